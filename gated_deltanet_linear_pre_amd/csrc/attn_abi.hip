// attn_abi.hip -- the extern "C" entry points of include/gdn_attn.h: argument
// checks (all before anything is enqueued), then the launchers.
#include <math.h>
#include <stdint.h>

#include "attn_internal.h"

namespace {

using gdn::AttnAppendArgs;
using gdn::AttnArgs;

constexpr int kMaxHeads = 1 << 12;
constexpr int kMaxGroup = 128;
constexpr int kMaxSeqs = 1 << 16;
constexpr int64_t kMaxRows = (int64_t)1 << 26;  // (8 rows a block of 256 threads: a launch has less than 2^32 of them)
constexpr int64_t kMaxKv = (int64_t)1 << 30;
constexpr int64_t kMaxStride = (int64_t)1 << 40;
constexpr int64_t kMaxCache = (int64_t)1 << 56;  // elements
constexpr int64_t kMaxPairs = (int64_t)1 << 24;
constexpr float kMaxScale = 0x1p127f;  // (times log2 e it is still finite: an infinite one would make a score of 0 NaN)

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
int elem(int32_t t) { return t == GDN_F32 ? 4 : 2; }
int launch_status(hipError_t e) { return e == hipSuccess ? GDN_OK : GDN_E_LAUNCH; }

#define REQ(p)                                  \
    do {                                        \
        if (!(p)) return GDN_E_NULL;            \
    } while (0)
#define ALN(p, a)                               \
    do {                                        \
        if (!aligned((p), (a))) return GDN_E_ALIGN; \
    } while (0)

bool stride_ok(int64_t s, int64_t least) { return s == 0 || (s >= least && s <= kMaxStride); }

int check_shape(const gdn_attn_shape *s)
{
    if (!s) return GDN_E_NULL;
    if (s->io_dtype != GDN_F32 && s->io_dtype != GDN_F16 && s->io_dtype != GDN_BF16) return GDN_E_DTYPE;
    if (s->kv_heads < 1 || s->heads < 1 || s->heads > kMaxHeads || s->heads % s->kv_heads) return GDN_E_SHAPE;
    if (s->heads / s->kv_heads > kMaxGroup) return GDN_E_SHAPE;
    const int D = s->head_dim;
    if (D != 64 && D != 96 && D != 128 && D != 192 && D != 256) return GDN_E_SHAPE;
    if (s->page_size < 16 || s->page_size > 1024 || (s->page_size & (s->page_size - 1))) return GDN_E_SHAPE;
    if (s->n_seq < 1 || s->n_seq > kMaxSeqs) return GDN_E_SHAPE;
    if (s->total_T < 0 || s->total_T > kMaxRows) return GDN_E_SHAPE;
    if (s->max_T < 0 || s->max_T > s->total_T) return GDN_E_SHAPE;
    if (s->n_pages < 1 || s->n_pages > INT32_MAX) return GDN_E_SHAPE;
    if (s->table_pages < 1 || s->table_pages > kMaxKv) return GDN_E_SHAPE;
    if (s->max_kv < 0 || s->max_kv > kMaxKv || s->max_kv > s->table_pages * s->page_size) return GDN_E_SHAPE;
    const int64_t page = (int64_t)s->kv_heads * s->page_size * D;
    if (!stride_ok(s->page_stride, page)) return GDN_E_SHAPE;
    if (s->n_pages > kMaxCache / (s->page_stride ? s->page_stride : page)) return GDN_E_SHAPE;
    const int64_t qrow = (int64_t)s->heads * D, krow = (int64_t)s->kv_heads * D;
    if (!stride_ok(s->q_stride, qrow) || !stride_ok(s->gate_stride, qrow)) return GDN_E_SHAPE;
    if (!stride_ok(s->k_stride, krow) || !stride_ok(s->v_stride, krow)) return GDN_E_SHAPE;
    if (s->rope_dim < 0 || s->rope_dim > D || s->rope_dim % 16) return GDN_E_SHAPE;
    if (s->flags & ~GDN_ROPE_PAIRS || s->reserved) return GDN_E_SHAPE;
    if (s->window < 0) return GDN_E_SHAPE;
    if (!(s->scale > 0.f && s->scale <= kMaxScale)) return GDN_E_SHAPE;
    if (!(isfinite(s->rope_scale) && s->rope_scale >= 0.f) || !(isfinite(s->eps) && s->eps >= 0.f)) return GDN_E_SHAPE;
    const int e = elem(s->io_dtype);
    if (s->page_stride * e % 16 || s->q_stride * e % 16 || s->k_stride * e % 16 || s->v_stride * e % 16 ||
        s->gate_stride * e % 16)
        return GDN_E_ALIGN;
    return GDN_OK;
}

} // namespace

extern "C" {

int gdn_attn_append(const gdn_attn_shape *shape, const int32_t *cu_seqlens, const int32_t *kv_len,
                    const int32_t *page_table, const int32_t *positions, const void *q,
                    const void *k, const void *v, const float *inv_freq, const void *q_norm,
                    const void *k_norm, void *q_out, void *k_cache, void *v_cache, void *stream)
{
    const int st = check_shape(shape);
    if (st) return st;
    REQ(cu_seqlens); REQ(kv_len); REQ(page_table); REQ(k_cache); REQ(v_cache);
    if (shape->rope_dim > 0) REQ(inv_freq);
    if (shape->total_T > 0) { REQ(q); REQ(k); REQ(v); REQ(q_out); }  // (buffers of no rows may have no address)
    ALN(cu_seqlens, 4); ALN(kv_len, 4); ALN(page_table, 4); ALN(positions, 4); ALN(inv_freq, 4);
    ALN(q, 16); ALN(k, 16); ALN(v, 16); ALN(q_norm, 16); ALN(k_norm, 16); ALN(q_out, 16);
    ALN(k_cache, 16); ALN(v_cache, 16);
    if (shape->total_T == 0 || shape->max_T == 0) return GDN_OK;
    const AttnAppendArgs a{cu_seqlens, kv_len, page_table, positions, q, k, v, inv_freq, q_norm, k_norm,
                           q_out, k_cache, v_cache};
    return launch_status(gdn::launch_attn_append(*shape, a, (hipStream_t)stream));
}

size_t gdn_attn_prefill_workspace_bytes(const gdn_attn_shape *shape)
{
    return check_shape(shape) == GDN_OK ? gdn::attn_prefill_workspace_bytes(*shape) : 0;
}

int gdn_attn_prefill(const gdn_attn_shape *shape, const int32_t *cu_seqlens, const int32_t *kv_len,
                     const int32_t *page_table, const void *q, const void *k_cache,
                     const void *v_cache, const void *gate, void *out, void *workspace,
                     size_t workspace_bytes, void *stream)
{
    const int st = check_shape(shape);
    if (st) return st;
    REQ(cu_seqlens); REQ(kv_len); REQ(page_table); REQ(k_cache); REQ(v_cache);
    if (shape->total_T > 0) { REQ(q); REQ(out); }
    ALN(cu_seqlens, 4); ALN(kv_len, 4); ALN(page_table, 4);
    ALN(q, 16); ALN(k_cache, 16); ALN(v_cache, 16); ALN(gate, 16); ALN(out, 16);
    const size_t need = gdn::attn_prefill_workspace_bytes(*shape);
    if (need > 0) REQ(workspace);
    ALN(workspace, 256);
    if (workspace_bytes < need) return GDN_E_WORKSPACE;
    if (shape->total_T == 0 || shape->max_T == 0) return GDN_OK;
    const AttnArgs a{cu_seqlens, kv_len, page_table, q, k_cache, v_cache, gate, out, workspace};
    return launch_status(gdn::launch_attn_prefill(*shape, a, (hipStream_t)stream));
}

size_t gdn_attn_step_workspace_bytes(const gdn_attn_shape *shape)
{
    return check_shape(shape) == GDN_OK ? gdn::attn_step_workspace_bytes(*shape) : 0;
}

int gdn_attn_step(const gdn_attn_shape *shape, const int32_t *kv_len, const int32_t *page_table,
                  const void *q, const void *k_cache, const void *v_cache, const void *gate,
                  void *out, void *workspace, size_t workspace_bytes, void *stream)
{
    const int st = check_shape(shape);
    if (st) return st;
    if (shape->total_T != shape->n_seq || shape->max_T != 1) return GDN_E_SHAPE;
    REQ(kv_len); REQ(page_table); REQ(q); REQ(k_cache); REQ(v_cache); REQ(out);
    ALN(kv_len, 4); ALN(page_table, 4);
    ALN(q, 16); ALN(k_cache, 16); ALN(v_cache, 16); ALN(gate, 16); ALN(out, 16);
    const size_t need = gdn::attn_step_workspace_bytes(*shape);
    if (need > 0) REQ(workspace);
    ALN(workspace, 256);
    if (workspace_bytes < need) return GDN_E_WORKSPACE;
    const AttnArgs a{nullptr, kv_len, page_table, q, k_cache, v_cache, gate, out, workspace};
    return launch_status(gdn::launch_attn_step(*shape, a, (hipStream_t)stream));
}

int gdn_attn_copy_pages(const gdn_attn_shape *shape, const int32_t *pairs, int64_t n,
                        void *k_cache, void *v_cache, void *stream)
{
    const int st = check_shape(shape);
    if (st) return st;
    if (n < 0 || n > kMaxPairs) return GDN_E_SHAPE;
    REQ(k_cache); REQ(v_cache);
    if (n > 0) REQ(pairs);
    ALN(pairs, 4); ALN(k_cache, 16); ALN(v_cache, 16);
    if (n == 0) return GDN_OK;
    return launch_status(gdn::launch_attn_copy_pages(*shape, pairs, n, k_cache, v_cache, (hipStream_t)stream));
}

int gdn_attn_rope_freqs(const gdn_rope *rope, float *inv_freq, float *rope_scale)
{
    REQ(rope); REQ(inv_freq); REQ(rope_scale);
    const int r = rope->rope_dim, kind = rope->kind;
    if (kind < GDN_ROPE_PLAIN || kind > GDN_ROPE_PARTS) return GDN_E_SHAPE;
    if (r < 16 || r > 256 || r % 16) return GDN_E_SHAPE;
    if (!(isfinite(rope->base) && rope->base > 1.0)) return GDN_E_SHAPE;
    if (kind != GDN_ROPE_PLAIN && !(isfinite(rope->factor) && rope->factor >= 1.0)) return GDN_E_SHAPE;
    if (kind == GDN_ROPE_PARTS &&
        (!(isfinite(rope->trained) && rope->trained >= 1.0) || !(rope->slow >= 0.0) ||
         !(rope->fast > rope->slow) || !isfinite(rope->fast)))
        return GDN_E_SHAPE;
    double base = rope->base;
    if (kind == GDN_ROPE_BASE) base *= pow(rope->factor, (double)r / (r - 2));
    for (int i = 0; i < r / 2; ++i) {
        double f = pow(base, -2.0 * i / r);
        if (kind == GDN_ROPE_LINEAR) f /= rope->factor;
        if (kind == GDN_ROPE_PARTS) {
            const double u = rope->trained * f / (2.0 * M_PI);
            const double keep = fmin(1.0, fmax(0.0, (u - rope->slow) / (rope->fast - rope->slow)));
            f *= keep + (1.0 - keep) / rope->factor;
        }
        inv_freq[i] = (float)f;
    }
    *rope_scale = kind == GDN_ROPE_PARTS ? (float)(0.1 * log(rope->factor) + 1.0) : 1.0f;
    return GDN_OK;
}

} // extern "C"
