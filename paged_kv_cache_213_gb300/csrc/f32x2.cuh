// f32x2.cuh -- fp32 arithmetic on pairs, one instruction for both halves (the FMA
// units take a pair of registers a lane), the maximum of three, and exact quotients.
#pragma once

namespace pkv {

__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float b, float c) {
    return fma2(a, make_float2(b, b), make_float2(c, c));
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// x / scale, correctly rounded: the quotient by the reciprocal inv = RN(1 / scale),
// then twice corrected by its exact residual (Markstein: with a correctly rounded
// reciprocal and a quotient within one unit in the last place, one such correction
// gives the rounded quotient; the first brings it there).  Exact where the residual is
// a normal number, which holds for |x / scale| >= 2^-11 (smaller ones become code 0)
// and scales in [2^-60, 2^60].  x has to be finite.  A residual of 0 turns -0 into 0.
__device__ __forceinline__ float2 divide2_unsigned_zero(float2 x, float scale, float inv) {
    const float2 s = make_float2(-scale, -scale), y = make_float2(inv, inv);
    const float2 q0 = mul2(x, y);
    const float2 q1 = fma2(fma2(s, q0, x), y, q0);
    return fma2(fma2(s, q1, x), y, q1);
}

// The same with the sign of x.
__device__ __forceinline__ float2 divide2_finite(float2 x, float scale, float inv) {
    const float2 q = divide2_unsigned_zero(x, scale, inv);
    return make_float2(copysignf(q.x, x.x), copysignf(q.y, x.y));
}

// The same for any x: a quotient that is not finite stays as it is.
__device__ __forceinline__ float2 divide2(float2 x, float scale, float inv) {
    const float2 q0 = mul2(x, make_float2(inv, inv)), q = divide2_finite(x, scale, inv);
    return make_float2(fabsf(q0.x) < 1e30f ? q.x : q0.x, fabsf(q0.y) < 1e30f ? q.y : q0.y);
}

}  // namespace pkv
