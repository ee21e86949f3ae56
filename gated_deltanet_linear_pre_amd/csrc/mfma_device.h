// mfma_device.h -- matrix operands of the three io types, fp32 values in parts of a
// matrix type, and what goes with them, shared by the scan and the attention kernels.
#pragma once

#include "ssm_device.h"

namespace gdn {

typedef float f4 __attribute__((ext_vector_type(4)));

// ---- matrix operands: 8 values of a 32-deep contraction a lane -------------
template <typename T> struct Mat;
template <> struct Mat<bf16> {
    typedef bf16 frag __attribute__((ext_vector_type(8)));
    static constexpr int PARTS = 3;
    static constexpr bool scaled = false;
    static __device__ __forceinline__ f4 mma(frag a, frag b, f4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};
template <> struct Mat<_Float16> {
    typedef _Float16 frag __attribute__((ext_vector_type(8)));
    static constexpr int PARTS = 2;
    static constexpr bool scaled = true;
    static __device__ __forceinline__ f4 mma(frag a, frag b, f4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};
// fp32: eight 4-deep products; product i contracts value i of every lane group
template <> struct Mat<float> {
    typedef float frag __attribute__((ext_vector_type(8)));
    static constexpr int PARTS = 1;
    static constexpr bool scaled = false;
    static __device__ __forceinline__ f4 mma(frag a, frag b, f4 c)
    {
#pragma unroll
        for (int i = 0; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
        return c;
    }
};

// an operand's 8 values in memory, on 16 bytes
template <typename T> struct Frag16 {
    typedef typename Mat<T>::frag type __attribute__((aligned(16)));
};

// v = sum of PARTS values of the matrix type, each the nearest to what the
// ones before it leave.  Two values at a time: their conversion and packing
// are one instruction.
template <typename T> struct Pair {
    typedef T t2 __attribute__((ext_vector_type(2)));
    typedef float f2 __attribute__((ext_vector_type(2)));
    static __device__ __forceinline__ t2 narrow(f2 v) { return __builtin_convertvector(v, t2); }
    static __device__ __forceinline__ f2 widen(t2 v) { return f2{(float)v[0], (float)v[1]}; }
};
template <typename T, int PARTS, int NV>
__device__ __forceinline__ void split(const float *v, T (*out)[NV])
{
#pragma unroll
    for (int i = 0; i < NV; i += 2) {
        typename Pair<T>::f2 r = {v[i], v[i + 1]};
#pragma unroll
        for (int p = 0; p < PARTS; ++p) {
            const typename Pair<T>::t2 h = Pair<T>::narrow(r);
            out[p][i] = h[0];
            out[p][i + 1] = h[1];
            if (p + 1 < PARTS) {
                const typename Pair<T>::f2 w = Pair<T>::widen(h);
                r[0] -= w[0];
                r[1] -= w[1];
            }
        }
    }
}
template <typename T, int PARTS>
__device__ __forceinline__ void split8(const float (&v)[8], typename Mat<T>::frag (&out)[PARTS])
{
    T o[PARTS][8];
    split<T, PARTS, 8>(v, o);
#pragma unroll
    for (int p = 0; p < PARTS; ++p)
#pragma unroll
        for (int i = 0; i < 8; ++i) out[p][i] = o[p][i];
}

// the largest of the four lanes that share lane & 15: a lane-half
// swap of x with itself leaves the two halves' values side by side, and a
// swap of 16-lane rows likewise
__device__ __forceinline__ float max_of_groups(float x)
{
    const unsigned u = __float_as_uint(x);
    const auto h = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const unsigned v = __float_as_uint(fmaxf(__uint_as_float(h[0]), __uint_as_float(h[1])));
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// Barrier that orders LDS only: global loads and stores in flight stay so.
__device__ __forceinline__ void lds_sync()
{
    __asm__ volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __asm__ volatile("" ::: "memory");
}

} // namespace gdn
