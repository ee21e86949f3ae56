/*
 * gdn_attn.h -- C ABI of the attention layers that stand between Gated
 * DeltaNet layers in hybrid models: norm and rotary positions with the write
 * to a paged key-value cache, causal attention of prompts and of single tokens
 * over that cache, and the copy of its pages.
 *
 *   gdn_attn_append      q and k normed and rotated, k and v to the cache.
 *   gdn_attn_prefill     attention of whole prompts, or of chunks that go on
 *                        from what the cache holds.
 *   gdn_attn_step        attention of one decode token per sequence.
 *   gdn_attn_copy_pages  pages copied to other pages (a sequence is forked, a
 *                        cache compacted).
 *   gdn_attn_rope_freqs  host only: the table of rotary frequencies.
 *
 * The conventions of gdn.h hold: device pointers on the current HIP device,
 * a host `shape` read during the call only, a hipStream_t passed as void*,
 * nothing synchronises or allocates, the library keeps no state, every
 * argument check runs before anything is enqueued, and the return value is a
 * gdn_status.  A call that enqueues several kernels returns GDN_E_LAUNCH when
 * the runtime refuses one of them; its outputs are then undefined.
 *
 * Symbols and layouts (row-major).  H = heads, KV = kv_heads, D = head_dim,
 * "io" = shape->io_dtype (GDN_F32, GDN_F16 or GDN_BF16) of every buffer but
 * the integers and inv_freq.
 *   cu_seqlens [n_seq+1] int32  sequence n owns the token rows [cu[n],
 *                               cu[n+1]): T_n of them; cu[0] = 0,
 *                               non-decreasing, no T_n above max_T, cu[n_seq]
 *                               <= total_T.  Rows from cu[n_seq] on belong to
 *                               no sequence: they are not read and their
 *                               outputs are left as they were.
 *   kv_len  [n_seq] int32       tokens of the sequence with the new ones: token
 *                               t of its T_n stands at position
 *                               p = kv_len[n] - T_n + t
 *   page_table [n_seq][table_pages] int32  position p of sequence n lies in
 *                               row p % page_size of page
 *                               page_table[n][p / page_size]; entries from
 *                               ceil(kv_len / page_size) on are not read
 *   k_cache, v_cache [n_pages][KV][page_size][D]  page_stride elements from
 *                               page to page (both may lie in one buffer, and
 *                               a page of all layers in one piece)
 *   q       [total_T][H][D]     head h reads key-value head h / (H/KV)
 *   k, v    [total_T][KV][D]
 *   gate    [total_T][H][D]     or NULL (no gate)
 *   out, q_out [total_T][H][D]  dense
 * q, k, v and gate may be column blocks of a wider projection: the strides
 * give the elements between token rows.  The heads of a row lie side by side: a
 * projection that leaves q and gate of a head next to each other has its weights'
 * rows put in order once, when they are loaded.
 * The integers on the device are preconditions, since checking them would take
 * a synchronisation.  No access leaves the buffers whatever they hold: cu_seqlens
 * outside [0, total_T] and kv_len outside [0, max_kv] are taken as the nearer
 * end, a page to be read outside [0, n_pages) too; one to be written is left out.
 * Alignment: workspaces 256-byte; the integers and inv_freq 4-byte; the rest, rows and
 * pages too, 16-byte (GDN_E_ALIGN otherwise).
 * No two buffers may overlap.
 */
#ifndef GDN_ATTN_H
#define GDN_ATTN_H

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

#ifndef GDN_BF16
#define GDN_BF16 2 /* beside GDN_F32 and GDN_F16 */
#endif

/* gdn_attn_shape.flags */
#define GDN_ROPE_PAIRS 1 /* rotated pairs are neighbours (2i, 2i+1); else (i, i + rope_dim/2) */

/* Sizes of one call.  Supported: 1 <= kv_heads, heads % kv_heads == 0,
 * heads / kv_heads <= 128, heads <= 4096; head_dim 64, 96, 128, 192 or 256;
 * page_size a power of two from 16 to 1024; 1 <= n_seq <= 65536; 0 <= max_T <=
 * total_T <= 2^26; 1 <= n_pages; 1 <= table_pages; 0 <= max_kv <= 2^30 and
 * max_kv <= table_pages * page_size; strides 0 or a row's (page's) elements up
 * to 2^40; n_pages * page_stride <= 2^56; rope_dim a multiple of 16 up to
 * head_dim; window >= 0; 0 < scale <= 2^127; rope_scale and eps >= 0, both finite.
 * Every entry point checks all of it, whichever fields it reads. */
typedef struct gdn_attn_shape {
    int32_t heads, kv_heads, head_dim, page_size;
    int32_t n_seq;
    int32_t io_dtype;
    int32_t rope_dim;    /* leading values of a head that are rotated (0: none) */
    int32_t flags;
    int64_t total_T;     /* token rows of the buffers */
    int64_t max_T;       /* host copy of max_n T_n, or more */
    int64_t max_kv;      /* host copy of max_n kv_len[n], or more */
    int64_t n_pages;
    int64_t table_pages; /* entries of a row of the page table */
    int64_t page_stride; /* elements between pages; 0: KV*page_size*D */
    int64_t q_stride;    /* elements between token rows; 0: H*D */
    int64_t k_stride;    /* 0: KV*D */
    int64_t v_stride;    /* 0: KV*D */
    int64_t gate_stride; /* 0: H*D */
    int64_t window;      /* keys a query sees, its own among them; 0: all before it */
    float scale;         /* of q.k */
    float rope_scale;    /* of the rotated values */
    float eps;           /* of the norms */
    int32_t reserved;    /* must be 0 */
} gdn_attn_shape;

/*
 * gdn_attn_append -- for every token and each head row x of q and k:
 *   x = x / sqrt(mean(x^2) + eps) * w       (w = q_norm or k_norm [D]; NULL: as it is)
 *   with a = P inv_freq[i] for i < rope_dim/2, and x_a, x_b the i-th pair:
 *   x_a, x_b = rope_scale (x_a cos a - x_b sin a), rope_scale (x_b cos a + x_a sin a)
 *   q_out <- x of q;  the cache's rows at the token's position p <- x of k, and v as it is
 * P is positions[t] ([total_T] int32) or, with positions NULL, p.  Norm and
 * rotation in fp32, one rounding to io; the angle is formed in 64 bits, so that it is
 * as exact for a far position as for the first (2^-21 at position 2^30).
 * Tokens at a position p below 0 or not below max_kv are not written to the cache.
 * No two tokens of a call may fall on one row of a page, or it may hold a mixture
 * (sequences that share a page which they still write to are forked first,
 * gdn_attn_copy_pages).
 * inv_freq [rope_dim/2] fp32 (may be NULL with rope_dim 0).
 * In: cu_seqlens, kv_len, page_table, positions, q, k, v, inv_freq, q_norm,
 * k_norm.  Out: q_out; k_cache, v_cache (the written rows only).
 */
int gdn_attn_append(const gdn_attn_shape *shape, const int32_t *cu_seqlens, const int32_t *kv_len,
                    const int32_t *page_table, const int32_t *positions, const void *q,
                    const void *k, const void *v, const float *inv_freq, const void *q_norm,
                    const void *k_norm, void *q_out, void *k_cache, void *v_cache, void *stream);

/*
 * gdn_attn_prefill -- for token t of sequence n at position p and head h, over
 * the keys j with max(0, p - window + 1) <= j <= p (from 0 with window 0):
 *   w_j = exp(scale q[t][h] . K_j - max),  o = sum_j w_j V_j / sum_j w_j
 *   out = o, or o sigmoid(gate[t][h])
 * A query that sees no key (p < 0) has o = 0.  The keys of the new tokens are in the
 * cache already (gdn_attn_append).  Scores, maxima, sums and o are fp32; with 16-bit
 * io the weights w_j are rounded to io as operands of the product with V (their sum
 * is not).  Keys and values that a query does not see, and rows of pages that no
 * token was written to, do not change its output, whatever they hold.  A value that
 * is not finite makes undefined: q its own output row, K those that see it, V those
 * that see it in its channel, gate its own value.  Scores times log2 e, and sums over
 * the keys of up to 2^8 |V_j|, have to stay inside fp32's range, or the row or the
 * channel is undefined too.  Where few rows meet many keys the keys of all of them are
 * dealt to the blocks, as in gdn_attn_step: a row's last bits may then depend on the
 * call's other rows, which say where its keys are cut.  The same call repeats bit for bit.
 * workspace: device scratch of >= gdn_attn_prefill_workspace_bytes(shape)
 * bytes, 256-byte aligned (NULL where that is 0); its contents are undefined
 * after the call, and it must not be shared by calls in flight at the same time.
 */
int gdn_attn_prefill(const gdn_attn_shape *shape, const int32_t *cu_seqlens, const int32_t *kv_len,
                     const int32_t *page_table, const void *q, const void *k_cache,
                     const void *v_cache, const void *gate, void *out, void *workspace,
                     size_t workspace_bytes, void *stream);

/* Bytes of scratch gdn_attn_prefill needs for `shape` (0 also if the shape is
 * invalid, which gdn_attn_prefill reports).  The need is each shape's own: one of fewer
 * tokens or shorter caches may need more (few rows have their keys dealt, many do not:
 * with 16 heads of 256 over 2 and max_kv 32768, 1024 tokens need 68 MB and 8192 none).  To allocate once,
 * take the bound for all shapes of a head_dim and type, 8 P R (head_dim + 2) + 32 P bytes, with P = 512
 * for head_dim up to 128 and 256 above, R = 128 and for GDN_F32 64. */
size_t gdn_attn_prefill_workspace_bytes(const gdn_attn_shape *shape);

/*
 * gdn_attn_step -- one token for each of n_seq sequences: the arithmetic of
 * gdn_attn_prefill with total_T == n_seq and max_T == 1 (token row n belongs to
 * sequence n and stands at kv_len[n] - 1; no cu_seqlens), the weights w_j kept to
 * 16 bits at least.  The keys of all sequences are dealt to the blocks in equal
 * parts, from kv_len on the device: a captured call stays balanced as lengths grow
 * up to max_kv.  The result does not depend on the other sequences but for the
 * places where its keys are cut.
 */
int gdn_attn_step(const gdn_attn_shape *shape, const int32_t *kv_len, const int32_t *page_table,
                  const void *q, const void *k_cache, const void *v_cache, const void *gate,
                  void *out, void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of scratch gdn_attn_step needs for `shape` (0 also if the shape is
 * invalid).  With the same heads and type it falls with no size but `window` (0 needs the most). */
size_t gdn_attn_step_workspace_bytes(const gdn_attn_shape *shape);

/*
 * gdn_attn_copy_pages -- for each of n pairs (from, to) of `pairs` [n][2] int32:
 * page `to` of k_cache and v_cache <- page `from`, bit for bit.  No page may be
 * `to` of two pairs, or `to` of one and `from` of another (either may then hold a
 * mixture); pairs with a page outside [0, n_pages), or of a page with itself, are
 * left out.  0 <= n <= 2^24.  Reads kv_heads, head_dim, page_size, n_pages,
 * page_stride and io_dtype of the shape.
 */
int gdn_attn_copy_pages(const gdn_attn_shape *shape, const int32_t *pairs, int64_t n,
                        void *k_cache, void *v_cache, void *stream);

/* Rotary frequencies f_i = base^(-2i/rope_dim), i < rope_dim/2, for contexts `factor`
 * times as long as the `trained` positions:
 *   GDN_ROPE_PLAIN   as they are
 *   GDN_ROPE_LINEAR  f_i / factor
 *   GDN_ROPE_BASE    with base factor^(rope_dim / (rope_dim - 2)) in base's place,
 *                    which divides the slowest by factor and leaves the fastest
 *   GDN_ROPE_PARTS   by the turns u = trained f_i / (2 pi) of a pair: f_i where u >=
 *                    fast, f_i / factor where u <= slow, in between
 *                    f_i (r + (1 - r) / factor), r = (u - slow) / (fast - slow);
 *                    rope_scale 0.1 ln(factor) + 1.  The ramp is linear in the turns; a
 *                    model whose ramp is linear in the pair's index has other frequencies
 *                    between the two ends, and passes a table of its own
 * rope_scale is 1 for the others. */
typedef enum gdn_rope_kind {
    GDN_ROPE_PLAIN = 0,
    GDN_ROPE_LINEAR = 1,
    GDN_ROPE_BASE = 2,
    GDN_ROPE_PARTS = 3
} gdn_rope_kind;

typedef struct gdn_rope {
    int32_t kind;     /* gdn_rope_kind */
    int32_t rope_dim; /* a multiple of 16 from 16 to 256 */
    double base;      /* > 1 */
    double factor;    /* >= 1; all but PLAIN */
    double trained;   /* >= 1; PARTS */
    double slow, fast; /* 0 <= slow < fast; PARTS */
} gdn_rope;

/* Host only: inv_freq [rope_dim/2] and *rope_scale are HOST addresses.  Formed in 64
 * bits, rounded once.  GDN_E_NULL or GDN_E_SHAPE on bad arguments. */
int gdn_attn_rope_freqs(const gdn_rope *rope, float *inv_freq, float *rope_scale);

#ifdef __cplusplus
}
#endif

#endif /* GDN_ATTN_H */
