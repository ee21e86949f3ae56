// attn_device.h -- device helpers shared by the attention kernels: where a
// sequence's tokens stand and where its pages lie.
#pragma once

#include "attn_internal.h"
#include "ssm_device.h"

namespace gdn {

// kv_len[n], kept inside [0, max_kv] whatever it holds
__device__ __forceinline__ int kv_bound(const AttnDims &d, const int32_t *__restrict__ kv_len, int n)
{
    const int v = kv_len[n];
    return v < 0 ? 0 : v > d.max_kv ? d.max_kv : v;
}

// a page number, kept inside the cache
__device__ __forceinline__ int page_bound(const AttnDims &d, int page)
{
    return page < 0 ? 0 : page >= d.n_pages ? d.n_pages - 1 : page;
}

// the first key that a query at position p sees
__device__ __forceinline__ int first_key(const AttnDims &d, int p)
{
    return p >= d.window ? p - d.window + 1 : 0;
}

// First element of a head's row of a page
__device__ __forceinline__ int64_t cache_row(const AttnDims &d, int page, int kv_head, int row)
{
    return page * d.page_stride + ((int64_t)kv_head * d.page + row) * d.D;
}

// the same for all lanes, which the compiler does not see
__device__ __forceinline__ int scalar(int x) { return __builtin_amdgcn_readfirstlane(x); }

// 4 channels of an output row: its gate's values, and o r, gated
template <typename T> struct Quad {
    typedef T t4 __attribute__((ext_vector_type(4)));
};
template <typename T>
__device__ __forceinline__ typename Quad<T>::t4 gate_of(const AttnDims &d, const AttnArgs &a, int64_t row, int head, int col)
{
    return *reinterpret_cast<const typename Quad<T>::t4 *>(static_cast<const T *>(a.gate) + row * d.gate_stride + head * d.D + col);
}
template <typename T, typename F4>
__device__ __forceinline__ typename Quad<T>::t4 finished(const AttnArgs &a, F4 o, float r, typename Quad<T>::t4 gate)
{
    typename Quad<T>::t4 y;
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = (T)(a.gate ? o[i] * r * __builtin_amdgcn_rcpf(1.0f + exp_fast(-(float)gate[i])) : o[i] * r);
    return y;
}
template <typename T, typename F4>
__device__ __forceinline__ void finish(const AttnDims &d, const AttnArgs &a, int64_t row, int head, int col, F4 o, float r,
                                       typename Quad<T>::t4 gate)
{
    *reinterpret_cast<typename Quad<T>::t4 *>(static_cast<T *>(a.out) + (row * d.H + head) * d.D + col) = finished<T>(a, o, r, gate);
}
// 1 / sum of weights; no key: o and the sum are 0 (a NaN stays one)
__device__ __forceinline__ float inverse_sum(float l) { return l > 0.f ? 1.0f / l : l; }

// N pieces of a row (maximum and sum of weights, 4 channels of o) put to what is there
template <int N, typename F4>
__device__ __forceinline__ void join(const float2 (&ml)[N], const F4 (&x)[N], float &m, float &l, F4 &o)
{
    float big = m;
#pragma unroll
    for (int u = 0; u < N; ++u) big = fmaxf(big, ml[u].x);
    const float big0 = big == -INFINITY ? 0.f : big, keep = __builtin_amdgcn_exp2f(m - big0);
    m = big;
    l *= keep;
    o *= keep;
#pragma unroll
    for (int u = 0; u < N; ++u) {
        const float f = __builtin_amdgcn_exp2f(ml[u].x - big0);
        l += f * ml[u].y;
        o += f * x[u];
    }
}

// What this wave's lanes wrote to LDS before is read by its lanes after (LDS takes a wave's accesses in order)
__device__ __forceinline__ void wave_sync() { __asm__ volatile("" ::: "memory"); }

// 16 bytes a lane from memory (base and the lane's offset) to LDS (`to`, lane after lane).  Written in
// assembly because the compiler does not count it then: it would put a wait for all of them before
// the next LDS read.  wait_vmem_all() and a barrier stand before the data is read.
// ONCE: past the caches' order.
// The waits that the compiler would put there stand in the assembly too: a load may read a scalar register 5 wait
// states after a vector instruction (readlane) wrote it, M0 1 after it was written; sooner it could go to the
// address that the registers held before.  s_mov is one of the 5, s_nop 3 the others.
template <bool ONCE = false>
__device__ __forceinline__ void copy_to_lds(const void *base, unsigned offset, unsigned to)
{
#ifdef __HIP_DEVICE_COMPILE__
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // (that nobody saves m0 for us: nothing here keeps it)
    const unsigned at = __builtin_amdgcn_readfirstlane(to);
    if (ONCE)
        __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %1, %2 nt" ::"s"(at), "v"(offset), "s"(base) : "memory", "m0");
    else
        __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(at), "v"(offset), "s"(base) : "memory", "m0");
#pragma clang diagnostic pop
#endif
}

} // namespace gdn
