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

} // namespace gdn
