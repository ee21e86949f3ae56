// ssm_conv.hip -- K-tap causal depthwise conv over the packed x|B|C channels
// with a carried history, bias and SiLU.
//
//   X = [hist; token rows]  ((K-1+T) x C)
//   out[t][c] = SiLU(b[c] + sum_{k<K} w[c][k] X[t+k][c]),  hist_out = last K-1 rows of X
//
// gfx950 mapping.  One read and one write of an element for about 2K+5 flop:
// bound by HBM bandwidth.  A lane owns one 16-byte vector of channels (8 of 16
// bits, 4 of fp32) and a run of 4 consecutive tokens, so every memory
// instruction of a wave moves 1 KB of one token row; the K-1 rows before a run
// are read again by the next run (an L2 hit).  All loads of a run are issued
// before its first store, so they are in flight together.  The four waves of
// a block take four runs in turn of the same channels.  Measured: 27135 tokens of
// 6144 bf16 channels 148 to 156 us, 4.3 to 4.5 TB/s, where a copy of 4 GB reaches
// 4.76; 2048 of 4352 fp16 9.9 us, 3.6 TB/s, 3 us of it a launch.
// History without a race when it is updated in place: only the run at a
// sequence's first token reads the old history (later runs start K-1 or more
// tokens in), and the same lanes write the new one after their reads.
#include "ssm_device.h"
#include "ssm_internal.h"

namespace gdn {

// Tokens of a wave's run.  Longer runs read a run's K-1 leading rows again less
// often, shorter ones make more waves.  Measured, by 4 and by 8: 37 tokens of 512
// fp32 channels 3.3 and 4.7 us, 2048 of 4352 fp16 9.9 and 11.3, 27135 of 6144 bf16
// 147.5 and 147.6.
constexpr int RUN = 4;

template <typename TI, int K>
__global__ __launch_bounds__(256) void ssm_conv_kernel(SsmDims d, const int32_t *__restrict__ cu,
                                                       const TI *__restrict__ xbc,
                                                       const TI *__restrict__ w,
                                                       const TI *__restrict__ bias,
                                                       const TI *hist, TI *hist_out,
                                                       TI *__restrict__ out)
{
    constexpr int V = Vec16<TI>::n;
    typedef typename Vec16<TI>::type vec;
    const int c0 = (blockIdx.y * 64 + (threadIdx.x & 63)) * V;
    if (c0 >= d.C) return;
    vec wk[K], b = vec(TI(0));  // (asked for before the trips to cu)
#pragma unroll
    for (int k = 0; k < K; ++k) wk[k] = ld16(w + (int64_t)c0 * K + k * V);
    if (bias) b = ld16(bias + c0);
    SeqTile st;
    if (!find_tile(cu, d.n_seq, d.T, 4 * RUN, blockIdx.x, st)) return;
    const int len = st.end - st.begin;
    const int t0 = st.c * 4 * RUN + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * RUN;
    if (t0 >= len && t0 > 0) return;

    // rows are the wave's, channels the lane's: one register for all addresses
    const uint32_t at_c = (uint32_t)c0 * sizeof(TI);
    const TI *row0 = xbc + st.begin * d.xbc_stride;
    const TI *h0 = hist + (int64_t)st.n * (K - 1) * d.C;
    // row e of X (e < K-1: history)
    auto load = [&](int e) -> vec {
        if (e >= K - 1) return ld16_at(row0 + (e - (K - 1)) * d.xbc_stride, at_c);
        return hist ? ld16_at(h0 + (int64_t)e * d.C, at_c) : vec(TI(0));
    };

    vec x[RUN + K - 1], nh[K - 1];
#pragma unroll
    for (int i = 0; i < RUN + K - 1; ++i) x[i] = t0 + i < len + K - 1 ? load(t0 + i) : vec(TI(0));
    const bool carry = t0 == 0 && hist_out;
    if (carry) {
#pragma unroll
        for (int j = 0; j < K - 1; ++j) nh[j] = load(len + j);
    }

    // half of the channels at a time, or all weights would be held widened: 102
    // registers instead of 82, and one more round of blocks (10.2 and 9.8 us a
    // prompt of 2048 tokens)
    vec o[RUN];
#pragma unroll
    for (int v0 = 0; v0 < V; v0 += V / 2) {
#pragma unroll
        for (int i = 0; i < RUN; ++i)
#pragma unroll
            for (int v = v0; v < v0 + V / 2; ++v) {
                float acc = (float)b[v];
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const int at = v * K + k;  // place in the V*K weights of these channels
                    acc = fmaf((float)wk[at / V][at % V], (float)x[i + k][v], acc);
                }
                o[i][v] = (TI)silu_fast(acc);
            }
#pragma unroll
        for (int i = 0; i < RUN; ++i) __asm__ volatile("" : "+v"(o[i]));
        __builtin_amdgcn_sched_barrier(0);
    }
    TI *o0 = out + (int64_t)(st.begin + t0) * d.C;
#pragma unroll
    for (int i = 0; i < RUN; ++i)
        if (t0 + i < len) st16_at(o0 + (int64_t)i * d.C, at_c, o[i]);
    if (carry) {
        TI *n0 = hist_out + (int64_t)st.n * (K - 1) * d.C;
#pragma unroll
        for (int j = 0; j < K - 1; ++j) st16_at(n0 + (int64_t)j * d.C, at_c, nh[j]);
    }
}

template <typename TI, int K>
static void launch_conv_k(const SsmDims &d, const SsmConvArgs &a, hipStream_t st)
{
    constexpr int V = Vec16<TI>::n;
    const dim3 grid((unsigned)(d.T / (4 * RUN) + d.n_seq), (unsigned)((d.C / V + 63) / 64));
    hipLaunchKernelGGL((ssm_conv_kernel<TI, K>), grid, dim3(256), 0, st, d, a.cu,
                       static_cast<const TI *>(a.xbc), static_cast<const TI *>(a.conv_w),
                       static_cast<const TI *>(a.conv_b), static_cast<const TI *>(a.hist),
                       static_cast<TI *>(a.hist_out), static_cast<TI *>(a.out));
}

hipError_t launch_ssm_conv(const gdn_ssm_shape &s, const SsmConvArgs &a, hipStream_t st)
{
    const SsmDims d = ssm_dims(s);
    GDN_SSM_IO(s.io_dtype,
        if (s.conv_width == 2) launch_conv_k<TI, 2>(d, a, st);
        else if (s.conv_width == 3) launch_conv_k<TI, 3>(d, a, st);
        else launch_conv_k<TI, 4>(d, a, st);)
    return hipGetLastError();
}

} // namespace gdn
