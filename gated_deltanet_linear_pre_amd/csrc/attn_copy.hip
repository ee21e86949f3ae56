// attn_copy.hip -- pages of the key-value cache copied to other pages.
//
// gfx950 mapping.  Bytes in and out once, as a copy: bound by HBM bandwidth, and by
// latency for one page.  A block of 256 threads moves BATCH vectors of 16 bytes a
// thread of one page of K or of V, all loads before the first store.
#include "attn_device.h"

namespace gdn {

namespace {

constexpr int BLOCK = 256, BATCH = 4;
typedef float v4 __attribute__((ext_vector_type(4)));

__global__ __launch_bounds__(BLOCK) void copy_pages_kernel(const int32_t *__restrict__ pairs, int64_t n, int n_pages,
                                                           int64_t stride, int size, v4 *k_cache, v4 *v_cache)
{
    const int64_t i = (int64_t)blockIdx.z * gridDim.y + blockIdx.y;
    if (i >= 2 * n) return;
    const int from = pairs[i & ~(int64_t)1], to = pairs[i | 1];
    if (from < 0 || from >= n_pages || to < 0 || to >= n_pages || from == to) return;
    v4 *cache = i & 1 ? v_cache : k_cache;
    const v4 *src = cache + from * stride;
    v4 *dst = cache + to * stride;
    const int c0 = blockIdx.x * (BLOCK * BATCH) + threadIdx.x;
    v4 x[BATCH];
#pragma unroll
    for (int b = 0; b < BATCH; ++b)
        if (c0 + b * BLOCK < size) x[b] = __builtin_nontemporal_load(src + c0 + b * BLOCK);
#pragma unroll
    for (int b = 0; b < BATCH; ++b)
        if (c0 + b * BLOCK < size) __builtin_nontemporal_store(x[b], dst + c0 + b * BLOCK);
}

} // namespace

hipError_t launch_attn_copy_pages(const gdn_attn_shape &s, const int32_t *pairs, int64_t n, void *k_cache,
                                  void *v_cache, hipStream_t st)
{
    const AttnDims d = attn_dims(s);
    const int per = 16 / (s.io_dtype == GDN_F32 ? 4 : 2);  // elements of a vector
    const int size = d.KV * d.page * d.D / per;
    const int64_t gy = 2 * n < 32768 ? 2 * n : 32768;
    const dim3 grid((size + BLOCK * BATCH - 1) / (BLOCK * BATCH), (unsigned)gy, (unsigned)((2 * n + gy - 1) / gy));
    hipLaunchKernelGGL(copy_pages_kernel, grid, dim3(BLOCK), 0, st, pairs, n, d.n_pages, d.page_stride / per, size,
                       static_cast<v4 *>(k_cache), static_cast<v4 *>(v_cache));
    return hipGetLastError();
}

} // namespace gdn
