// attn_append.hip -- norm and rotary positions of q and k, and the write of k and
// v to the paged cache.
//
//   x <- x / sqrt(mean x^2 + eps) w;   (x_a, x_b) <- s (x_a cos t - x_b sin t, x_b cos t + x_a sin t),
//   t = P f_i;   q -> q_out, k and v -> row p % page of page table[n][p / page]
//
// gfx950 mapping.  Every value goes in and out once for a handful of flop: bound by
// HBM bandwidth, and by latency for a single token.  A block takes TOKENS tokens; its
// threads first form the cosines and sines of those tokens' pairs in LDS (one a
// thread and round: formed beside the rows, once for every head, they would cost
// more than the traffic), then walk the tokens' head rows (H of q, KV of k, KV of v).
// A team of TEAM lanes owns a head row, 16 values a lane in two vectors of 8: the
// two halves of 8 rotated pairs, or 16 values that pass; a rotation never leaves its
// lane, and the norm's sum runs over the team.
#include "attn_device.h"

namespace gdn {

namespace {

constexpr int BLOCK = 256;

// cos and sin of p f: the turns are formed in 64 bits (p f has 55 bits at most), whole
// ones taken off, and what is left is exact to 2^-24 of a turn
__device__ __forceinline__ float2 turn(int p, float f, float scale)
{
    double u = (double)p * (double)f * 0.15915494309189535;
    u -= rint(u);
    float c, s;
    sincospif((float)(2.0 * u), &s, &c);
    return make_float2(scale * c, scale * s);
}

template <typename T, int D>
__global__ __launch_bounds__(BLOCK) void append_kernel(AttnDims d, int tokens, int rope, bool pairs, float rope_scale,
                                                       float eps, const int32_t *__restrict__ cu,
                                                       const int32_t *__restrict__ kv_len,
                                                       const int32_t *__restrict__ table,
                                                       const int32_t *__restrict__ positions, const T *__restrict__ q,
                                                       const T *__restrict__ k, const T *__restrict__ v,
                                                       const float *__restrict__ inv_freq, const T *__restrict__ q_norm,
                                                       const T *__restrict__ k_norm, T *__restrict__ q_out,
                                                       T *__restrict__ k_cache, T *__restrict__ v_cache)
{
    constexpr int LANES = D / 16;  // that hold values
    constexpr int TEAM = LANES <= 4 ? 4 : LANES <= 8 ? 8 : 16;
    extern __shared__ float2 cs[];  // [tokens][rope/2]
    __shared__ int64_t at[16];      // a token's row in the cache, in elements (without its head); -1: none
    __shared__ int pos[16];
    __shared__ bool live[16];
    const int64_t t0 = (int64_t)blockIdx.x * tokens;
    const int half = rope / 2;

    if (threadIdx.x < tokens) {
        const int64_t t = t0 + threadIdx.x;
        bool in = t < d.T && t < seq_bound(cu, d.n_seq, d.T);
        int64_t where = -1;
        int p = 0;
        if (in) {
            int lo = 0, hi = d.n_seq;  // the last sequence that begins at t or before
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (seq_bound(cu, mid, d.T) <= t) lo = mid;
                else hi = mid;
            }
            const int end = seq_bound(cu, lo + 1, d.T);
            in = t >= seq_bound(cu, lo, d.T) && t < end;  // (false where cu is not in order)
            p = kv_bound(d, kv_len, lo) - end + (int)t;
            if (in && p >= 0 && p < d.max_kv) {
                const int page = table[(int64_t)lo * d.table_pages + (p >> d.log_page)];
                if (page >= 0 && page < d.n_pages) where = cache_row(d, page, 0, p & (d.page - 1));
            }
            if (in && positions) p = positions[t];
        }
        at[threadIdx.x] = where;
        pos[threadIdx.x] = p;
        live[threadIdx.x] = in;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < tokens * half; i += BLOCK) {
        const int t = i / half;
        if (live[t]) cs[i] = turn(pos[t], inv_freq[i - t * half], rope_scale);
    }
    __syncthreads();

    const int lane = threadIdx.x & (TEAM - 1);
    const int rows = d.H + 2 * d.KV;
    // this lane's two vectors: of the pairs 8 lane.., or of values behind the rotated ones
    const bool turned = lane < rope / 16, in = lane < LANES;
    const int a = pairs || !turned ? 16 * lane : 8 * lane, b = pairs || !turned ? a + 8 : a + half;
    for (int i = blockIdx.y * (BLOCK / TEAM) + threadIdx.x / TEAM; i < tokens * rows; i += gridDim.y * (BLOCK / TEAM)) {
        const int t = i / rows, r = i - t * rows;
        if (!live[t]) continue;
        const T *from;
        T *to;
        const T *w = nullptr;
        const int64_t tok = t0 + t;
        if (r < d.H) {
            from = q + tok * d.q_stride + r * D;
            to = q_out + (tok * d.H + r) * D;
            w = q_norm;
        } else {
            const bool key = r < d.H + d.KV;
            const int h = key ? r - d.H : r - d.H - d.KV;
            if (at[t] < 0) continue;
            from = key ? k + tok * d.k_stride + h * D : v + tok * d.v_stride + h * D;
            to = (key ? k_cache : v_cache) + at[t] + (int64_t)h * d.page * D;
            if (key) w = k_norm;
        }
        const bool value = r >= d.H + d.KV;
        float x[2][8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[0][j] = x[1][j] = 0.f;
        if (in) {
            load8f(from + a, x[0]);
            load8f(from + b, x[1]);
        }
        if (w) {
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(x[0][j], x[0][j], fmaf(x[1][j], x[1][j], ss));
#pragma unroll
            for (int m = TEAM / 2; m > 0; m >>= 1) ss += __shfl_xor(ss, m, 64);
            const float n = 1.0f / sqrtf(ss * (1.0f / D) + eps);
            if (in) {
                float wa[8], wb[8];
                load8f(w + a, wa);
                load8f(w + b, wb);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    x[0][j] = x[0][j] * n * wa[j];
                    x[1][j] = x[1][j] * n * wb[j];
                }
            }
        }
        if (turned && !value) {
            const float2 *c = cs + t * half + 8 * lane;
            if (pairs) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int j = 0; j < 8; j += 2) {
                        const float2 e = c[4 * u + j / 2];
                        const float xa = x[u][j], xb = x[u][j + 1];
                        x[u][j] = xa * e.x - xb * e.y;
                        x[u][j + 1] = xb * e.x + xa * e.y;
                    }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 e = c[j];
                    const float xa = x[0][j], xb = x[1][j];
                    x[0][j] = xa * e.x - xb * e.y;
                    x[1][j] = xb * e.x + xa * e.y;
                }
            }
        }
        if (in) {
            store8f(to + a, x[0]);
            store8f(to + b, x[1]);
        }
    }
}

template <typename T, int D>
void launch_append_t(const AttnDims &d, const gdn_attn_shape &s, const AttnAppendArgs &a, hipStream_t st)
{
    constexpr int LANES = D / 16, TEAM = LANES <= 4 ? 4 : LANES <= 8 ? 8 : 16;
    // 8 tokens a block; fewer where the launch would have less than 4 blocks a CU, and
    // then several blocks for a token's rows
    const int rows = d.H + 2 * d.KV;
    int tokens = 8;
    while (tokens > 1 && d.T / tokens < 1024) tokens >>= 1;
    int split = 1;
    while (d.T / tokens * split < 1024 && split * (BLOCK / TEAM) < tokens * rows) split <<= 1;
    const dim3 grid((unsigned)((d.T + tokens - 1) / tokens), split);
    hipLaunchKernelGGL((append_kernel<T, D>), grid, dim3(BLOCK), (size_t)tokens * s.rope_dim / 2 * sizeof(float2), st, d, tokens,
                       s.rope_dim, (s.flags & GDN_ROPE_PAIRS) != 0, s.rope_scale, s.eps, a.cu, a.kv_len, a.table,
                       a.positions, static_cast<const T *>(a.q), static_cast<const T *>(a.k),
                       static_cast<const T *>(a.v), a.inv_freq, static_cast<const T *>(a.q_norm),
                       static_cast<const T *>(a.k_norm), static_cast<T *>(a.q_out), static_cast<T *>(a.k_cache),
                       static_cast<T *>(a.v_cache));
}

} // namespace

hipError_t launch_attn_append(const gdn_attn_shape &s, const AttnAppendArgs &a, hipStream_t st)
{
    const AttnDims d = attn_dims(s);
    GDN_SSM_IO(s.io_dtype,
        switch (s.head_dim) {
        case 64: launch_append_t<TI, 64>(d, s, a, st); break;
        case 96: launch_append_t<TI, 96>(d, s, a, st); break;
        case 128: launch_append_t<TI, 128>(d, s, a, st); break;
        case 192: launch_append_t<TI, 192>(d, s, a, st); break;
        default: launch_append_t<TI, 256>(d, s, a, st); break;
        })
    return hipGetLastError();
}

} // namespace gdn
