// calls.cpp -- the marshalling of rope.py's, latent.py's and q8.py's calls, natively.
//
// A call for a few tokens takes the GPU 2 to 9 us and took the host 15 to 20, nearly
// all of it in Python: attributes of tensors, one wrapper object each, and the
// conversion of some 25 arguments.  Each function below does the same checks on the
// tensors themselves, allocates what the caller did not give and calls the C entry on
// the current stream.  It returns None, having launched nothing, for whatever is not
// the plain case (a wrong type, shape or device, a refusal of the C entry, an
// exception); the Python code then goes through its own checks, which raise.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cstdint>
#include <initializer_list>

#include "pagedkv_latent.h"
#include "pagedkv_q8.h"
#include "pagedkv_rope.h"

namespace {

using at::Tensor;

// The arguments of a call, in order; `ok` stays true while they are plain.
struct Args {
    PyObject *const *args;
    Py_ssize_t left;
    int dev = -1;  // of the first tensor; the others have to be there too
    bool ok = true;

    PyObject *next() {
        if (left <= 0) {
            ok = false;
            return Py_None;
        }
        --left;
        return *args++;
    }
    // A CUDA tensor of this type, contiguous unless `strided`; null for None where
    // that is allowed.
    const Tensor *tensor(at::ScalarType type, bool optional = false, bool strided = false) {
        PyObject *o = next();
        if (!ok || (optional && o == Py_None)) return nullptr;
        ok = THPVariable_Check(o);
        if (!ok) return nullptr;
        const Tensor &t = THPVariable_Unpack(o);
        ok = t.is_cuda() && t.scalar_type() == type && (dev < 0 || t.get_device() == dev) &&
             (strided || t.is_contiguous());
        if (ok) dev = static_cast<int>(t.get_device());
        return ok ? &t : nullptr;
    }
    long long integer(long long low = INT_MIN, long long high = INT_MAX) {
        PyObject *o = next();
        ok = ok && PyLong_Check(o);
        if (!ok) return 0;
        int over = 0;
        const long long v = PyLong_AsLongLongAndOverflow(o, &over);
        ok = over == 0 && v >= low && v <= high;
        return ok ? v : 0;
    }
    int int32() { return static_cast<int>(integer()); }
    double number() {
        PyObject *o = next();
        ok = ok && (PyFloat_Check(o) || PyLong_CheckExact(o));
        if (!ok) return 0;
        const double v = PyFloat_AsDouble(o);
        if (v == -1.0 && PyErr_Occurred()) {
            PyErr_Clear();
            ok = false;
        }
        return v;
    }
    bool flag() {
        PyObject *o = next();
        ok = ok && PyBool_Check(o);
        return o == Py_True;
    }
    // All read, all plain, and their device the current one.
    bool plain() const { return ok && left == 0 && dev >= 0 && c10::cuda::current_device() == dev; }
    void *stream() const {
        return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    }
    Tensor make(std::initializer_list<int64_t> shape, at::ScalarType type = at::kHalf) const {
        return at::empty(shape, at::TensorOptions().dtype(type).device(
                                    at::kCUDA, static_cast<c10::DeviceIndex>(dev)));
    }
};

void *at_of(const Tensor *t) { return t ? t->data_ptr() : nullptr; }

bool is(const Tensor *t, std::initializer_list<int64_t> shape) {
    return !t || t->sizes() == at::IntArrayRef(shape);
}

bool fits(std::initializer_list<int64_t> sizes) {  // the C entries' int arguments
    for (int64_t s : sizes)
        if (s < 0 || s > INT_MAX) return false;
    return true;
}

// Elements between tokens of t [T, H, d], whose heads are contiguous; -1: they are not.
int64_t token_stride(const Tensor &t, int64_t T, int64_t H, int64_t d) {
    if ((t.stride(2) != 1 && d > 1) || (t.stride(1) != d && H > 1)) return -1;
    return T > 1 ? t.stride(0) : H * d;
}

// Other Python threads run while a launch waits for room in the queue.
struct Unlocked {
    PyThreadState *state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};
template <typename F>
int unlocked(F f) {
    Unlocked u;
    return f();
}

template <PyObject *(*F)(Args &)>
PyObject *guarded(PyObject *, PyObject *const *args, Py_ssize_t n) {
    try {
        Args a{args, n};
        return F(a);
    } catch (...) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

// q, k, v, q_weight, k_weight, eps, cos_sin, positions, slots, k_cache, v_cache,
// interleaved, q_out, err_word and, for E4M3, k_scale, v_scale
template <bool F8>
PyObject *qk_append(Args &a) {
    const at::ScalarType kind = F8 ? at::kByte : at::kHalf;
    const Tensor *q = a.tensor(at::kHalf, false, true), *k = a.tensor(at::kHalf, false, true),
                 *v = a.tensor(at::kHalf, false, true);
    const Tensor *qw = a.tensor(at::kHalf, true), *kw = a.tensor(at::kHalf, true);
    const float eps = static_cast<float>(a.number());
    const Tensor *cs = a.tensor(at::kFloat, true), *pos = a.tensor(at::kInt, true);
    const Tensor *slots = a.tensor(at::kLong), *kc = a.tensor(kind), *vc = a.tensor(kind);
    const int interleaved = a.flag();
    PyObject *given = a.left > 0 ? a.args[0] : Py_None;
    const Tensor *out = a.tensor(at::kHalf, true), *err = a.tensor(at::kInt, true);
    const float ks = F8 ? static_cast<float>(a.number()) : 1.f;
    const float vs = F8 ? static_cast<float>(a.number()) : 1.f;
    if (!a.plain() || kc->dim() != 4 || vc->sizes() != kc->sizes() || q->dim() != 3 || !!cs != !!pos)
        Py_RETURN_NONE;
    const int64_t NB = kc->size(0), Hk = kc->size(1), bs = kc->size(2), d = kc->size(3);
    const int64_t T = q->size(0), H = q->size(1);
    if (q->size(2) != d || !is(k, {T, Hk, d}) || !is(v, {T, Hk, d}) || !is(qw, {d}) || !is(kw, {d}) ||
        !is(slots, {T}) || !is(pos, {T}) || (cs && cs->dim() != 2) || !is(out, {T, H, d}))
        Py_RETURN_NONE;
    const int64_t table = cs ? cs->size(0) : 0, rot = cs ? cs->size(1) : 0;
    const int64_t qs = token_stride(*q, T, H, d), kst = token_stride(*k, T, Hk, d),
                  vst = token_stride(*v, T, Hk, d);
    if (qs < 0 || kst < 0 || vst < 0 || !fits({T, H, Hk, d, bs, table, rot})) Py_RETURN_NONE;
    Tensor made;
    if (!out) made = a.make({T, H, d});
    void *op = out ? out->data_ptr() : made.data_ptr();
    int rc;
    if (F8)
        rc = unlocked([&] { return paged_qk_norm_rope_append_fp8(
            op, q->data_ptr(), k->data_ptr(), v->data_ptr(), qs, kst, vst, at_of(qw), at_of(kw), eps,
            static_cast<const float *>(at_of(cs)), static_cast<const int32_t *>(at_of(pos)),
            static_cast<int>(table), static_cast<int>(rot), interleaved,
            static_cast<const int64_t *>(at_of(slots)), at_of(kc), at_of(vc), static_cast<int>(T),
            static_cast<int>(H), static_cast<int>(Hk), static_cast<int>(d), static_cast<int>(bs), NB, ks,
            vs, static_cast<int32_t *>(at_of(err)), a.stream()); });
    else
        rc = unlocked([&] { return paged_qk_norm_rope_append(
            op, q->data_ptr(), k->data_ptr(), v->data_ptr(), qs, kst, vst, at_of(qw), at_of(kw), eps,
            static_cast<const float *>(at_of(cs)), static_cast<const int32_t *>(at_of(pos)),
            static_cast<int>(table), static_cast<int>(rot), interleaved,
            static_cast<const int64_t *>(at_of(slots)), at_of(kc), at_of(vc), static_cast<int>(T),
            static_cast<int>(H), static_cast<int>(Hk), static_cast<int>(d), static_cast<int>(bs), NB,
            static_cast<int32_t *>(at_of(err)), a.stream()); });
    if (rc != PKV_OK) Py_RETURN_NONE;
    return out ? Py_NewRef(given) : THPVariable_Wrap(std::move(made));
}

// kv, weight, eps, cos_sin, positions, slots, cache, q_rope, q_out, interleaved,
// err_word; True
PyObject *latent_append(Args &a) {
    const Tensor *kv = a.tensor(at::kHalf, false, true), *w = a.tensor(at::kHalf, true);
    const float eps = static_cast<float>(a.number());
    const Tensor *cs = a.tensor(at::kFloat), *pos = a.tensor(at::kInt), *slots = a.tensor(at::kLong);
    const Tensor *cache = a.tensor(at::kHalf);
    const Tensor *q = a.tensor(at::kHalf, true, true), *out = a.tensor(at::kHalf, true, true);
    const int interleaved = a.flag();
    const Tensor *err = a.tensor(at::kInt, true);
    if (!a.plain() || cache->dim() != 3 || kv->dim() != 2 || cs->dim() != 2 || !!q != !!out)
        Py_RETURN_NONE;
    const int64_t NB = cache->size(0), bs = cache->size(1), E = cache->size(2);
    const int64_t T = kv->size(0), table = cs->size(0), P = cs->size(1), R = E - P;
    if (kv->size(1) != E || (E > 1 && kv->stride(1) != 1) || !is(pos, {T}) || !is(slots, {T}) || R <= 0 ||
        !is(w, {R}) || !fits({T, R, P, bs, table}))
        Py_RETURN_NONE;
    int64_t H = 0, qt = 0, qh = 0, ot = 0, oh = 0;
    if (q) {
        if (q->dim() != 3) Py_RETURN_NONE;
        H = q->size(1);
        if (!is(q, {T, H, P}) || !is(out, {T, H, P}) || !fits({H}) ||
            (P > 1 && (q->stride(2) != 1 || out->stride(2) != 1)))
            Py_RETURN_NONE;
        qh = H == 1 ? P : q->stride(1);
        oh = H == 1 ? P : out->stride(1);
        qt = T > 1 ? q->stride(0) : H * qh;
        ot = T > 1 ? out->stride(0) : H * oh;
    }
    const int rc = unlocked([&] { return paged_latent_append(
        kv->data_ptr(), T > 1 ? kv->stride(0) : E, at_of(w), eps, static_cast<const float *>(at_of(cs)),
        static_cast<const int32_t *>(at_of(pos)), static_cast<int>(table), interleaved,
        static_cast<const int64_t *>(at_of(slots)), at_of(cache), at_of(q), qt, qh, at_of(out), ot, oh,
        static_cast<int>(H), static_cast<int>(T), static_cast<int>(R), static_cast<int>(P),
        static_cast<int>(bs), NB, static_cast<int32_t *>(at_of(err)), a.stream()); });
    if (rc != PKV_OK) Py_RETURN_NONE;
    Py_RETURN_TRUE;
}

// q, cache, block_tables, context_lens, scale, latent_dim, query_start, max_q_len,
// max_context_len, out, workspace, lse, err_word
PyObject *latent_attention(Args &a) {
    const Tensor *q = a.tensor(at::kHalf), *cache = a.tensor(at::kHalf);
    const Tensor *tables = a.tensor(at::kInt), *lens = a.tensor(at::kInt);
    const float scale = static_cast<float>(a.number());
    const int64_t R = a.int32();
    const Tensor *start = a.tensor(at::kInt, true);
    const int most = a.int32(), longest = a.int32();
    PyObject *given = a.left > 0 ? a.args[0] : Py_None;
    const Tensor *out = a.tensor(at::kHalf, true), *ws = a.tensor(at::kByte, true),
                 *lse = a.tensor(at::kFloat, true), *err = a.tensor(at::kInt, true);
    if (!a.plain() || cache->dim() != 3 || q->dim() != 3 || tables->dim() != 2) Py_RETURN_NONE;
    const int64_t NB = cache->size(0), bs = cache->size(1), E = cache->size(2);
    const int64_t TQ = q->size(0), H = q->size(1), B = tables->size(0), MB = tables->size(1);
    if (q->size(2) != E || R <= 0 || R >= E || !is(lens, {B}) || !is(start, {B + 1}) ||
        (!start && (TQ != B || most != 1)) || !is(out, {TQ, H, R}) || !is(lse, {TQ, H}) ||
        !fits({bs, E, TQ, H, B, MB}))
        Py_RETURN_NONE;
    Tensor made, scratch;
    if (!out) made = a.make({TQ, H, R});
    if (!ws) {
        size_t bytes = 0;
        if (paged_latent_plan(static_cast<int>(B), static_cast<int>(TQ), most, static_cast<int>(H),
                              static_cast<int>(R), static_cast<int>(E - R), static_cast<int>(bs),
                              static_cast<int>(MB), longest, &bytes) != PKV_OK)
            Py_RETURN_NONE;
        scratch = a.make({static_cast<int64_t>(bytes)}, at::kByte);
        ws = &scratch;
    }
    const int rc = unlocked([&] { return paged_latent_attention(
        out ? out->data_ptr() : made.data_ptr(), q->data_ptr(), at_of(cache),
        static_cast<const int32_t *>(at_of(tables)), static_cast<const int32_t *>(at_of(lens)),
        static_cast<const int32_t *>(at_of(start)), static_cast<int>(B), static_cast<int>(TQ), most,
        static_cast<int>(MB), NB, scale, static_cast<int>(H), static_cast<int>(R),
        static_cast<int>(E - R), static_cast<int>(bs), longest, at_of(ws),
        static_cast<size_t>(ws->numel()), static_cast<float *>(at_of(lse)),
        static_cast<int32_t *>(at_of(err)), a.stream()); });
    if (rc != PKV_OK) Py_RETURN_NONE;
    return out ? Py_NewRef(given) : THPVariable_Wrap(std::move(made));
}

// cache, block_tables, start, total, latent_dim, latents, ropes, err_word; a pair
PyObject *latent_gather(Args &a) {
    const Tensor *cache = a.tensor(at::kHalf), *tables = a.tensor(at::kInt), *start = a.tensor(at::kInt);
    const int64_t total = a.int32(), R = a.int32();
    PyObject *l = a.left > 0 ? a.args[0] : Py_None, *r = a.left > 1 ? a.args[1] : Py_None;
    const Tensor *latents = a.tensor(at::kHalf, true), *ropes = a.tensor(at::kHalf, true),
                 *err = a.tensor(at::kInt, true);
    if (!a.plain() || cache->dim() != 3 || tables->dim() != 2) Py_RETURN_NONE;
    const int64_t NB = cache->size(0), bs = cache->size(1), E = cache->size(2), B = tables->size(0),
                  MB = tables->size(1);
    if (R <= 0 || R >= E || total < 0 || !is(start, {B + 1}) || !is(latents, {total, R}) ||
        !is(ropes, {total, E - R}) || !fits({bs, E, B, MB}))
        Py_RETURN_NONE;
    Tensor made_l, made_r;
    if (!latents) made_l = a.make({total, R});
    if (!ropes) made_r = a.make({total, E - R});
    const int rc = unlocked([&] { return paged_latent_gather(
        latents ? latents->data_ptr() : made_l.data_ptr(), ropes ? ropes->data_ptr() : made_r.data_ptr(),
        at_of(cache), static_cast<const int32_t *>(at_of(tables)),
        static_cast<const int32_t *>(at_of(start)), static_cast<int>(B), total, static_cast<int>(MB), NB,
        static_cast<int>(R), static_cast<int>(E - R), static_cast<int>(bs),
        static_cast<int32_t *>(at_of(err)), a.stream()); });
    if (rc != PKV_OK) Py_RETURN_NONE;
    PyObject *x = latents ? Py_NewRef(l) : THPVariable_Wrap(std::move(made_l));
    PyObject *y = ropes ? Py_NewRef(r) : THPVariable_Wrap(std::move(made_r));
    PyObject *pair = x && y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return pair;
}

// q, kv, k_rope, q_start, kv_start, scale, max_q_len, max_kv_len, out, lse, err_word
PyObject *latent_prefill(Args &a) {
    const Tensor *q = a.tensor(at::kHalf), *kv = a.tensor(at::kHalf), *kr = a.tensor(at::kHalf);
    const Tensor *qs = a.tensor(at::kInt), *ks = a.tensor(at::kInt);
    const float scale = static_cast<float>(a.number());
    const int most_q = a.int32(), most_kv = a.int32();
    PyObject *given = a.left > 0 ? a.args[0] : Py_None;
    const Tensor *out = a.tensor(at::kHalf, true), *lse = a.tensor(at::kFloat, true),
                 *err = a.tensor(at::kInt, true);
    if (!a.plain() || q->dim() != 3 || kv->dim() != 3 || kr->dim() != 2 || qs->dim() != 1)
        Py_RETURN_NONE;
    const int64_t TQ = q->size(0), H = q->size(1), TK = kr->size(0), P = kr->size(1),
                  d = q->size(2) - P, B = qs->size(0) - 1;
    if (B < 0 || d <= 0 || !is(kv, {TK, H, 2 * d}) || !is(ks, {B + 1}) || !is(out, {TQ, H, d}) ||
        !is(lse, {TQ, H}) || !fits({TQ, H, TK, P, d, B}))
        Py_RETURN_NONE;
    Tensor made;
    if (!out) made = a.make({TQ, H, d});
    const int rc = unlocked([&] { return latent_prefill_attention(
        out ? out->data_ptr() : made.data_ptr(), q->data_ptr(), kv->data_ptr(), kr->data_ptr(),
        static_cast<const int32_t *>(at_of(qs)), static_cast<const int32_t *>(at_of(ks)),
        static_cast<int>(B), static_cast<int>(TQ), static_cast<int>(TK), most_q, most_kv, scale,
        static_cast<int>(H), static_cast<int>(d), static_cast<int>(P), static_cast<float *>(at_of(lse)),
        static_cast<int32_t *>(at_of(err)), a.stream()); });
    if (rc != PKV_OK) Py_RETURN_NONE;
    return out ? Py_NewRef(given) : THPVariable_Wrap(std::move(made));
}

// The 8-bit caches of a call: k_cache, v_cache, k_scales, v_scales.
struct Q8 {
    const Tensor *k, *v, *ks, *vs;
    int kind = PKV_Q8_E4M3;
    int64_t NB = 0, Hk = 0, bs = 0, d = 0;
    bool ok = false;

    explicit Q8(Args &a) {
        at::ScalarType type = at::kByte;
        if (a.left > 0 && THPVariable_Check(a.args[0]) &&
            THPVariable_Unpack(a.args[0]).scalar_type() == at::kChar) {
            type = at::kChar;
            kind = PKV_Q8_INT8;
        }
        k = a.tensor(type);
        v = a.tensor(type);
        ks = a.tensor(at::kFloat);
        vs = a.tensor(at::kFloat);
        if (!a.ok || k->dim() != 4 || v->sizes() != k->sizes()) return;
        NB = k->size(0), Hk = k->size(1), bs = k->size(2), d = k->size(3);
        ok = Hk > 0 && is(ks, {NB, Hk}) && is(vs, {NB, Hk}) && fits({Hk, bs, d});
    }
    float *k_scales() const { return static_cast<float *>(ks->data_ptr()); }
    float *v_scales() const { return static_cast<float *>(vs->data_ptr()); }
};

// k_new, v_new, the cache, block_tables, context_lens, query_start, max_q_len,
// err_word; True
PyObject *append_q8(Args &a) {
    const Tensor *k = a.tensor(at::kHalf, false, true), *v = a.tensor(at::kHalf, false, true);
    const Q8 c(a);
    const Tensor *tables = a.tensor(at::kInt), *lens = a.tensor(at::kInt), *start = a.tensor(at::kInt, true);
    const int most = a.int32();
    const Tensor *err = a.tensor(at::kInt, true);
    if (!a.plain() || !c.ok || k->dim() != 3 || tables->dim() != 2) Py_RETURN_NONE;
    const int64_t T = k->size(0), B = tables->size(0), MB = tables->size(1);
    if (!is(k, {T, c.Hk, c.d}) || !is(v, {T, c.Hk, c.d}) || !is(lens, {B}) || !is(start, {B + 1}) ||
        (!start && (T != B || most != 1)) || !fits({T, B, MB}))
        Py_RETURN_NONE;
    const int64_t ks = token_stride(*k, T, c.Hk, c.d), vs = token_stride(*v, T, c.Hk, c.d);
    if (ks < 0 || vs < 0) Py_RETURN_NONE;
    const int rc = unlocked([&] { return paged_kv_append_q8(
        k->data_ptr(), v->data_ptr(), ks, vs, static_cast<const int32_t *>(at_of(start)),
        static_cast<const int32_t *>(at_of(tables)), static_cast<const int32_t *>(at_of(lens)),
        static_cast<int>(B), static_cast<int>(T), most, static_cast<int>(MB), at_of(c.k), at_of(c.v),
        c.k_scales(), c.v_scales(), c.kind, static_cast<int>(c.Hk), static_cast<int>(c.d),
        static_cast<int>(c.bs), c.NB, static_cast<int32_t *>(at_of(err)), a.stream()); });
    if (rc != PKV_OK) Py_RETURN_NONE;
    Py_RETURN_TRUE;
}

// q, the cache, block_tables, context_lens, scale, query_start, max_q_len,
// max_context_len, out, workspace, lse, err_word, flags
PyObject *attention_q8(Args &a) {
    const Tensor *q = a.tensor(at::kHalf, false, true);
    const Q8 c(a);
    const Tensor *tables = a.tensor(at::kInt), *lens = a.tensor(at::kInt);
    const float scale = static_cast<float>(a.number());
    const Tensor *start = a.tensor(at::kInt, true);
    const int most = a.int32(), longest = a.int32();
    PyObject *given = a.left > 0 ? a.args[0] : Py_None;
    const Tensor *out = a.tensor(at::kHalf, true), *ws = a.tensor(at::kByte, true),
                 *lse = a.tensor(at::kFloat, true), *err = a.tensor(at::kInt, true);
    const uint32_t flags = static_cast<uint32_t>(a.integer(0, UINT_MAX));
    // without a workspace one has to be zero-filled: the Python code does that
    if (!a.plain() || !c.ok || !ws || q->dim() != 3 || tables->dim() != 2) Py_RETURN_NONE;
    const int64_t TQ = q->size(0), H = q->size(1), B = tables->size(0), MB = tables->size(1);
    if (q->size(2) != c.d || H % c.Hk != 0 || !is(lens, {B}) || !is(start, {B + 1}) ||
        (!start && (TQ != B || most != 1)) || !is(out, {TQ, H, c.d}) || !is(lse, {TQ, H}) ||
        !fits({TQ, H, B, MB}))
        Py_RETURN_NONE;
    const int64_t qs = token_stride(*q, TQ, H, c.d);
    if (qs < 0) Py_RETURN_NONE;
    Tensor made;
    if (!out) made = a.make({TQ, H, c.d});
    const int rc = unlocked([&] { return paged_decode_attention_q8(
        out ? out->data_ptr() : made.data_ptr(), q->data_ptr(), qs, at_of(c.k), at_of(c.v), c.k_scales(),
        c.v_scales(), c.kind, static_cast<const int32_t *>(at_of(tables)),
        static_cast<const int32_t *>(at_of(lens)), static_cast<const int32_t *>(at_of(start)),
        static_cast<int>(B), static_cast<int>(TQ), most, static_cast<int>(MB), c.NB, scale,
        static_cast<int>(H), static_cast<int>(c.Hk), static_cast<int>(c.d), static_cast<int>(c.bs), longest,
        at_of(ws), static_cast<size_t>(ws->numel()), static_cast<float *>(at_of(lse)),
        static_cast<int32_t *>(at_of(err)), a.stream(), flags); });
    if (rc != PKV_OK) Py_RETURN_NONE;
    return out ? Py_NewRef(given) : THPVariable_Wrap(std::move(made));
}

// the cache, block_tables, start, total, k, v, err_word; a pair
PyObject *gather_q8(Args &a) {
    const Q8 c(a);
    const Tensor *tables = a.tensor(at::kInt), *start = a.tensor(at::kInt);
    const int64_t total = a.int32();
    PyObject *gk = a.left > 0 ? a.args[0] : Py_None, *gv = a.left > 1 ? a.args[1] : Py_None;
    const Tensor *k = a.tensor(at::kHalf, true), *v = a.tensor(at::kHalf, true), *err = a.tensor(at::kInt, true);
    if (!a.plain() || !c.ok || tables->dim() != 2) Py_RETURN_NONE;
    const int64_t B = tables->size(0), MB = tables->size(1);
    if (total < 0 || !is(start, {B + 1}) || !is(k, {total, c.Hk, c.d}) || !is(v, {total, c.Hk, c.d}) ||
        !fits({B, MB}))
        Py_RETURN_NONE;
    Tensor made_k, made_v;
    if (!k) made_k = a.make({total, c.Hk, c.d});
    if (!v) made_v = a.make({total, c.Hk, c.d});
    const int rc = unlocked([&] { return paged_kv_gather_q8(
        k ? k->data_ptr() : made_k.data_ptr(), v ? v->data_ptr() : made_v.data_ptr(), at_of(c.k), at_of(c.v),
        c.k_scales(), c.v_scales(), c.kind, static_cast<const int32_t *>(at_of(tables)),
        static_cast<const int32_t *>(at_of(start)), static_cast<int>(B), total, static_cast<int>(MB), c.NB,
        static_cast<int>(c.Hk), static_cast<int>(c.d), static_cast<int>(c.bs),
        static_cast<int32_t *>(at_of(err)), a.stream()); });
    if (rc != PKV_OK) Py_RETURN_NONE;
    PyObject *x = k ? Py_NewRef(gk) : THPVariable_Wrap(std::move(made_k));
    PyObject *y = v ? Py_NewRef(gv) : THPVariable_Wrap(std::move(made_v));
    PyObject *pair = x && y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return pair;
}

#define ENTRY(name, f) \
    {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<f>)), METH_FASTCALL, nullptr}

PyMethodDef methods[] = {ENTRY("qk_append", qk_append<false>),
                         ENTRY("qk_append_fp8", qk_append<true>),
                         ENTRY("latent_append", latent_append),
                         ENTRY("latent_attention", latent_attention),
                         ENTRY("latent_gather", latent_gather),
                         ENTRY("latent_prefill", latent_prefill),
                         ENTRY("append_q8", append_q8),
                         ENTRY("attention_q8", attention_q8),
                         ENTRY("gather_q8", gather_q8),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pagedkv_calls", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pagedkv_calls() { return PyModule_Create(&module); }
