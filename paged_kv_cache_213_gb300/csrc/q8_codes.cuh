// q8_codes.cuh -- codes of the 8-bit caches with block scales: fp32 to codes and
// codes to fp16.  KIND is PKV_Q8_E4M3 or PKV_Q8_INT8.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "pagedkv_q8.h"

namespace pkv {

template <int KIND>
__device__ __forceinline__ constexpr float q8_limit() {
    return KIND == PKV_Q8_E4M3 ? 448.f : 127.f;
}

// Four quotients to four codes, the first in the low byte: to nearest even,
// saturated; NaN to the NaN code, or 0 for int8.  PLAIN: all are numbers that need no
// saturation (they round to a code).
template <int KIND, bool PLAIN = false>
__device__ __forceinline__ uint32_t q8_encode4(float2 a, float2 b) {
    if (KIND == PKV_Q8_E4M3)
        return __nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3) |
               static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3)) << 16;
    // 1.5 * 2^23 leaves the whole number, rounded to even, in the sum's low byte (a
    // conversion instruction has a quarter of the additions' rate)
    auto low = [](float x) {
        if (!PLAIN) x = x == x ? fminf(fmaxf(x, -127.f), 127.f) : 0.f;
        return __float_as_uint(x + 12582912.f);
    };
    return __byte_perm(__byte_perm(low(a.x), low(a.y), 0x0040), __byte_perm(low(b.x), low(b.y), 0x0040), 0x5410);
}

// Codes 0, 1 (HI 0) or 2, 3 (HI 1) of four to fp16: exact.
template <int KIND, int HI>
__device__ __forceinline__ uint32_t q8_widen(uint32_t w) {
    uint32_t r;
    if (KIND == PKV_Q8_E4M3) {
        const uint16_t s = static_cast<uint16_t>(HI ? w >> 16 : w);
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(s));
    } else {
        // byte + 128 behind the exponent of 1024 is the fp16 number 1152 + code
        const uint32_t u = __byte_perm(w ^ 0x80808080u, 0x64646464u, HI ? 0x4342 : 0x4140);
        const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&u), __floats2half2_rn(1152.f, 1152.f));
        r = *reinterpret_cast<const uint32_t *>(&h);
    }
    return r;
}

// The least reference of sums of values, whose scales go up to 2^64.  A weight's rounding (half a
// subnormal step of fp16, 2^-25, times the code) is below 2^-41 there, nothing in an fp16
// result, and so is what smaller scales lose.  The sums' factor from one reference to the next
// is between 2^-90 and 2^90: finite, so that a sum of 0 stays 0, and exact enough where it is
// small.  A sum that overflows by it is one of values above 2^102.
constexpr float kQ8LeastReference = 0x1p-26f;

}  // namespace pkv
