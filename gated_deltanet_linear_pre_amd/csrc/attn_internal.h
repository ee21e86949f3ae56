// attn_internal.h -- launchers behind the C ABI of include/gdn_attn.h.  Each one
// assumes its arguments were validated by the ABI layer and only enqueues.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/gdn_attn.h"

namespace gdn {

// The sizes the kernels take by value, strides resolved.
struct AttnDims {
    int H, KV, D, g;   // g: query heads of a key-value head
    int page, log_page;
    int n_seq, table_pages, n_pages;
    int max_T, max_kv;
    int64_t T, page_stride, q_stride, k_stride, v_stride, gate_stride;
    int window;        // INT32_MAX: none
    float scale;
};

inline AttnDims attn_dims(const gdn_attn_shape &s)
{
    AttnDims d;
    d.H = s.heads;
    d.KV = s.kv_heads;
    d.D = s.head_dim;
    d.g = s.heads / s.kv_heads;
    d.page = s.page_size;
    d.log_page = __builtin_ctz(s.page_size);
    d.n_seq = s.n_seq;
    d.table_pages = (int)s.table_pages;
    d.n_pages = (int)s.n_pages;
    d.max_T = (int)s.max_T;
    d.max_kv = (int)s.max_kv;
    d.T = s.total_T;
    d.page_stride = s.page_stride ? s.page_stride : (int64_t)s.kv_heads * s.page_size * s.head_dim;
    d.q_stride = s.q_stride ? s.q_stride : (int64_t)s.heads * s.head_dim;
    d.k_stride = s.k_stride ? s.k_stride : (int64_t)s.kv_heads * s.head_dim;
    d.v_stride = s.v_stride ? s.v_stride : (int64_t)s.kv_heads * s.head_dim;
    d.gate_stride = s.gate_stride ? s.gate_stride : (int64_t)s.heads * s.head_dim;
    d.window = s.window == 0 || s.window > s.max_kv ? INT32_MAX : (int)s.window;
    d.scale = s.scale;
    return d;
}

struct AttnAppendArgs {
    const int32_t *cu, *kv_len, *table, *positions;
    const void *q, *k, *v;
    const float *inv_freq;
    const void *q_norm, *k_norm;
    void *q_out, *k_cache, *v_cache;
};

struct AttnArgs {
    const int32_t *cu;  // NULL: one token a sequence
    const int32_t *kv_len, *table;
    const void *q, *k_cache, *v_cache, *gate;
    void *out, *ws;
};

size_t attn_prefill_workspace_bytes(const gdn_attn_shape &s);
size_t attn_step_workspace_bytes(const gdn_attn_shape &s);

hipError_t launch_attn_append(const gdn_attn_shape &s, const AttnAppendArgs &a, hipStream_t st);
hipError_t launch_attn_prefill(const gdn_attn_shape &s, const AttnArgs &a, hipStream_t st);
hipError_t launch_attn_step(const gdn_attn_shape &s, const AttnArgs &a, hipStream_t st);
hipError_t launch_attn_copy_pages(const gdn_attn_shape &s, const int32_t *pairs, int64_t n,
                                  void *k_cache, void *v_cache, hipStream_t st);

} // namespace gdn
