// ssm_device.h -- device helpers shared by the state space kernels: 16-byte
// vectors of the three io types, the packed-sequence slots, the step size.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn_device.h"

namespace gdn {

typedef __bf16 bf16;

// ---- 16-byte vectors of the io types: 4 fp32 or 8 fp16 / bf16 -------------
template <typename T> struct Vec16 {
    static constexpr int n = 16 / sizeof(T);
    typedef T type __attribute__((ext_vector_type(16 / sizeof(T))));
};

template <typename T>
__device__ __forceinline__ typename Vec16<T>::type ld16(const T *p)
{
    return *reinterpret_cast<const typename Vec16<T>::type *>(p);
}
template <typename T>
__device__ __forceinline__ void st16(T *p, typename Vec16<T>::type v)
{
    *reinterpret_cast<typename Vec16<T>::type *>(p) = v;
}

// 16 bytes at a uniform base and a 32-bit byte offset of the lane: one register
// for the addresses of all rows a thread moves
template <typename T>
__device__ __forceinline__ typename Vec16<T>::type ld16_at(const T *base, uint32_t bytes)
{
    return ld16(reinterpret_cast<const T *>(reinterpret_cast<const char *>(base) + bytes));
}
template <typename T>
__device__ __forceinline__ void st16_at(T *base, uint32_t bytes, typename Vec16<T>::type v)
{
    st16(reinterpret_cast<T *>(reinterpret_cast<char *>(base) + bytes), v);
}

// 8 consecutive elements widened to fp32, and narrowed (to nearest even) back
template <typename T>
__device__ __forceinline__ void load8f(const T *p, float (&x)[8])
{
    constexpr int n = Vec16<T>::n;
#pragma unroll
    for (int b = 0; b < 8 / n; ++b) {
        const typename Vec16<T>::type v = ld16(p + b * n);
#pragma unroll
        for (int i = 0; i < n; ++i) x[b * n + i] = (float)v[i];
    }
}
template <typename T>
__device__ __forceinline__ void store8f(T *p, const float (&x)[8])
{
    constexpr int n = Vec16<T>::n;
#pragma unroll
    for (int b = 0; b < 8 / n; ++b) {
        typename Vec16<T>::type v;
#pragma unroll
        for (int i = 0; i < n; ++i) v[i] = (T)x[b * n + i];
        st16(p + b * n, v);
    }
}

// ---- packed sequences -----------------------------------------------------
// cu[n], kept inside [0, T] whatever it holds
__device__ __forceinline__ int seq_bound(const int32_t *__restrict__ cu, int n, int64_t T)
{
    const int v = cu[n];
    return v < 0 ? 0 : (int64_t)v > T ? (int)T : v;
}

// Tiles of `tile` tokens counted from each sequence's first token are numbered
// by slots: tile c of sequence n has slot cu[n] / tile + n + c.  Distinct tiles
// get distinct slots below T / tile + n_seq, some of which stay empty, so a
// launch needs no list of tiles.  Finds a slot's sequence by bisection (the
// slot of tile 0 grows with n) and its token range; false: an empty slot.
// A sequence of no tokens has its tile 0 all the same (begin == end).
struct SeqTile {
    int n, c;        // sequence, tile
    int begin, end;  // the sequence's tokens
};
__device__ __forceinline__ bool find_tile(const int32_t *__restrict__ cu, int n_seq, int64_t T,
                                          int tile, int slot, SeqTile &out)
{
    int lo = 0, hi = n_seq;  // first slot of lo <= slot < that of hi
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (seq_bound(cu, mid, T) / tile + mid <= slot) lo = mid;
        else hi = mid;
    }
    out.n = lo;
    out.begin = seq_bound(cu, lo, T);
    out.end = seq_bound(cu, lo + 1, T);
    if (out.end < out.begin) out.end = out.begin;
    out.c = slot - (out.begin / tile + lo);
    if (out.c < 0) return false;  // (cu does not start at 0)
    return out.c == 0 || (int64_t)out.c * tile < (int64_t)out.end - out.begin;
}

// ---- step size and log decay ----------------------------------------------
// e^x for x <= 0 to about 2 ulp at any size: the rounding of x log2(e), which
// the hardware's 2^p does not see, is put back to first order
__device__ __forceinline__ float exp_neg(float x)
{
    const float p = x * 1.44269502f;
    float r = __builtin_fmaf(x, 1.44269502f, -p);
    r = __builtin_fmaf(x, 1.92596299e-8f, r);  // log2(e) beyond its first float
    return __builtin_amdgcn_exp2f(p) * __builtin_fmaf(r, 0.693147181f, 1.0f);
}

// log(1 + e) for 0 <= e <= 1 to about 3 ulp: 2 atanh(s), s = e / (2 + e) <= 1/3,
// by its series; what follows s^15 / 15 is below 2^-29 of the sum
__device__ __forceinline__ float log1p_unit(float e)
{
    const float d = 2.0f + e, q = __builtin_amdgcn_rcpf(d);
    float s = e * q;
    s = __builtin_fmaf(__builtin_fmaf(-s, d, e), q, s);
    const float t = s * s;
    float v = 1.0f / 15.0f;
    v = __builtin_fmaf(v, t, 1.0f / 13.0f);
    v = __builtin_fmaf(v, t, 1.0f / 11.0f);
    v = __builtin_fmaf(v, t, 1.0f / 9.0f);
    v = __builtin_fmaf(v, t, 1.0f / 7.0f);
    v = __builtin_fmaf(v, t, 1.0f / 5.0f);
    v = __builtin_fmaf(v, t, 1.0f / 3.0f);
    return 2.0f * __builtin_fmaf(s * t, v, s);
}

// dt = clamp(softplus(raw + bias)), lam = -exp(A_log) dt.  A NaN stays one (the
// comparisons fail).  lam is bounded at -200, e^-200 being 0 in fp32, so that
// sums of log decays stay finite and their differences exact.
__device__ __forceinline__ void step_size(float raw, float bias, float neg_a, float dt_min,
                                          float dt_max, float &dt, float &lam)
{
    const float u = raw + bias, m = fabsf(u);
    float v = (u > 0.f ? u : 0.f) + log1p_unit(exp_neg(m > 150.f ? -150.f : -m));
    v = u != u ? u : v;
    v = v < dt_min ? dt_min : v;
    v = v > dt_max ? dt_max : v;
    dt = v;
    const float l = neg_a * v;
    lam = l < -200.f ? -200.f : l;
}

// dispatch over io x out types: `out` is fp32 or the io type
#define GDN_SSM_IO(io, ...)                          \
    switch (io) {                                    \
    case GDN_F32: { using TI = float; __VA_ARGS__ } break;    \
    case GDN_F16: { using TI = _Float16; __VA_ARGS__ } break; \
    default: { using TI = gdn::bf16; __VA_ARGS__ } break;     \
    }

} // namespace gdn
