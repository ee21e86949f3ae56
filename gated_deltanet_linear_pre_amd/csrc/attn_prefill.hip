// attn_prefill.hip -- causal attention over the paged cache.
//
//   o = sum_j w_j V_j / sum_j w_j,  w_j = exp(scale q.K_j - max)
//
// The simplest right form: one wave a (token, head), a key a lane for the scores and
// D / 64 channels a lane for the sums.
#include "attn_device.h"

namespace gdn {

namespace {

template <typename T, int D>
__global__ __launch_bounds__(64) void attend_kernel(AttnDims d, AttnArgs a)
{
    __shared__ float sq[D];
    constexpr int DD = (D + 63) / 64;
    const int64_t t = blockIdx.x;
    const int h = blockIdx.y, lane = threadIdx.x, kh = h / d.g;
    int n = (int)t, p;
    if (a.cu) {
        if (t >= seq_bound(a.cu, d.n_seq, d.T)) return;
        int lo = 0, hi = d.n_seq;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (seq_bound(a.cu, mid, d.T) <= t) lo = mid;
            else hi = mid;
        }
        n = lo;
        const int end = seq_bound(a.cu, lo + 1, d.T);
        if (t < seq_bound(a.cu, lo, d.T) || t >= end) return;
        p = kv_bound(d, a.kv_len, n) - end + (int)t;
    } else {
        p = kv_bound(d, a.kv_len, n) - 1;
    }
    const T *q = static_cast<const T *>(a.q) + t * d.q_stride + h * D;
    for (int i = lane; i < D; i += 64) sq[i] = (float)q[i] * d.scale;
    __syncthreads();
    float m = -INFINITY, l = 0.f, o[DD];
#pragma unroll
    for (int i = 0; i < DD; ++i) o[i] = 0.f;
    const int32_t *table = a.table + (int64_t)n * d.table_pages;
    const T *K = static_cast<const T *>(a.k_cache), *V = static_cast<const T *>(a.v_cache);
    for (int j0 = first_key(d, p); j0 <= p; j0 += 64) {
        const int j = j0 + lane;
        float s = -INFINITY;
        if (j <= p) {
            const T *k = K + cache_row(d, page_bound(d, table[j >> d.log_page]), kh, j & (d.page - 1));
            s = 0.f;
            for (int i = 0; i < D; i += 8) {
                float x[8];
                load8f(k + i, x);
#pragma unroll
                for (int u = 0; u < 8; ++u) s = fmaf(x[u], sq[i + u], s);
            }
        }
        float most = s;
#pragma unroll
        for (int u = 32; u > 0; u >>= 1) most = fmaxf(most, __shfl_xor(most, u, 64));
        const float m1 = fmaxf(m, most), safe = m1 == -INFINITY ? 0.f : m1;
        const float w = j <= p ? expf(s - safe) : 0.f, keep = expf(m - safe);
        m = m1;
        float sum = w;
#pragma unroll
        for (int u = 32; u > 0; u >>= 1) sum += __shfl_xor(sum, u, 64);
        l = l * keep + sum;
#pragma unroll
        for (int i = 0; i < DD; ++i) o[i] *= keep;
        for (int u = 0; u < 64 && j0 + u <= p; ++u) {
            const float wu = __shfl(w, u, 64);
            const T *v = V + cache_row(d, page_bound(d, table[(j0 + u) >> d.log_page]), kh, (j0 + u) & (d.page - 1));
#pragma unroll
            for (int i = 0; i < DD; ++i)
                if (i * 64 + lane < D) o[i] = fmaf(wu, (float)v[i * 64 + lane], o[i]);
        }
    }
    T *out = static_cast<T *>(a.out) + (t * d.H + h) * D;
    const T *gate = static_cast<const T *>(a.gate) + t * d.gate_stride + h * D;
#pragma unroll
    for (int i = 0; i < DD; ++i)
        if (i * 64 + lane < D) {
            float v = p >= 0 ? o[i] / l : 0.f;
            if (a.gate) v = v / (1.f + expf(-(float)gate[i * 64 + lane]));
            out[i * 64 + lane] = (T)v;
        }
}

template <typename T, int D>
void launch_attend_t(const AttnDims &d, const AttnArgs &a, hipStream_t st)
{
    hipLaunchKernelGGL((attend_kernel<T, D>), dim3((unsigned)d.T, d.H), dim3(64), 0, st, d, a);
}

hipError_t attend(const gdn_attn_shape &s, const AttnArgs &a, hipStream_t st)
{
    const AttnDims d = attn_dims(s);
    GDN_SSM_IO(s.io_dtype,
        switch (s.head_dim) {
        case 64: launch_attend_t<TI, 64>(d, a, st); break;
        case 96: launch_attend_t<TI, 96>(d, a, st); break;
        case 128: launch_attend_t<TI, 128>(d, a, st); break;
        case 192: launch_attend_t<TI, 192>(d, a, st); break;
        default: launch_attend_t<TI, 256>(d, a, st); break;
        })
    return hipGetLastError();
}

} // namespace

size_t attn_prefill_workspace_bytes(const gdn_attn_shape &) { return 0; }
hipError_t launch_attn_prefill(const gdn_attn_shape &s, const AttnArgs &a, hipStream_t st) { return attend(s, a, st); }

} // namespace gdn
