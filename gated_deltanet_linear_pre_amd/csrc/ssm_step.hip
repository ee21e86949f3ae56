// ssm_step.hip -- one token per sequence through conv and recurrence.
//
//   X = [hist; xbc row];  s = SiLU(b + sum_k w[c][k] X[k][c]) = x | B | C
//   S <- exp(-exp(A_log) dt) S + dt x B^T,  y = S C + D x,  hist_out = X[1..K-1]
//
// gfx950 mapping.  The state goes in and out once (8 bytes an element) for 5
// flop: bound by HBM bandwidth in a batch and by latency for one sequence.  A
// 256-thread block takes up to 32*R rows p of one (sequence, head).  Each
// thread issues the loads of its state elements first, so that they are in
// flight while the block forms x, B and C in LDS.  8 lanes own a row and cover
// one whole 128-byte line of it with every load and store; y's sum over N runs
// over a lane's elements, then over the 8 lanes.  Measured, 64 heads of 64,
// N = 128: 64 sequences 50 us, 5.5 TB/s (some of the state stays in the 256 MB
// cache between calls); one sequence 4 us, most of it a launch and two dependent
// trips to memory.
// With a separate hist_out this kernel writes it too: each block the x
// channels of its rows, the first block of each group those of B and C.  In
// place a second launch shifts the history, since every head of a group reads
// the group's old B and C rows: 6.1 us for one sequence and 3.7 with two buffers,
// 53.9 and 49.9 for 64 (from a graph).
#include "ssm_device.h"
#include "ssm_internal.h"

namespace gdn {

template <typename TI, typename TO, int N, int K, int R>
__global__ __launch_bounds__(256) void ssm_step_kernel(
    SsmDims d, int tiles, const TI *__restrict__ xbc, const TI *__restrict__ w,
    const TI *__restrict__ bias, const TI *__restrict__ dt_raw, const float *__restrict__ A_log,
    const float *__restrict__ dt_bias, const float *__restrict__ D, const TI *__restrict__ hist,
    TI *__restrict__ hist_out, const float *state, float *state_out, TO *__restrict__ y)
{
    constexpr int ROWS = 32 * R, NV = N / 32;
    __shared__ float sx[ROWS], sb[N], sc[N];
    const int64_t n = (int64_t)blockIdx.z * gridDim.y + blockIdx.y;
    if (n >= d.n_seq) return;
    const int h = blockIdx.x / tiles, tile = blockIdx.x - h * tiles;
    const int grp = h / d.hg;
    const int p0 = tile * ROWS;
    const int rows = d.P - p0 < ROWS ? d.P - p0 : ROWS;
    const int e = threadIdx.x & 7, r0 = threadIdx.x >> 3;

    float4 S[R][NV];
    const int64_t base = ((n * d.H + h) * d.P + p0) * N + e * 4;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int row = r * 32 + r0;
            S[r][j] = state && row < rows ? load4_nt(state + base + (int64_t)row * N + j * 32)
                                          : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    float dt, lam;
    step_size((float)dt_raw[n * d.dt_stride + h], dt_bias[h], -expf(A_log[h]), d.dt_min, d.dt_max, dt, lam);
    const float a = expf(lam);
    const bool first = tile == 0 && h == grp * d.hg;  // writes the group's B and C history

    for (int i = threadIdx.x; i < rows + 2 * N; i += 256) {
        int c;
        float *to;
        if (i < rows) { c = h * d.P + p0 + i; to = sx + i; }
        else if (i < rows + N) { c = d.H * d.P + grp * N + i - rows; to = sb + i - rows; }
        else { c = d.H * d.P + (d.G + grp) * N + i - rows - N; to = sc + i - rows - N; }
        TI X[K];
#pragma unroll
        for (int k = 0; k < K - 1; ++k) X[k] = hist ? hist[(n * (K - 1) + k) * d.C + c] : TI(0);
        X[K - 1] = xbc[n * d.xbc_stride + c];
        float acc = bias ? (float)bias[c] : 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) acc = fmaf((float)w[(int64_t)c * K + k], (float)X[k], acc);
        *to = silu_fast(acc);
        if (hist_out && (i < rows || first)) {
#pragma unroll
            for (int k = 0; k < K - 1; ++k) hist_out[(n * (K - 1) + k) * d.C + c] = X[k + 1];
        }
    }
    __syncthreads();

    float4 Bv[NV], Cv[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        Bv[j] = *reinterpret_cast<const float4 *>(sb + j * 32 + e * 4);
        Cv[j] = *reinterpret_cast<const float4 *>(sc + j * 32 + e * 4);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int row = r * 32 + r0;
        const float xv = row < rows ? sx[row] : 0.f;
        const float u = dt * xv;
        float acc = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float4 v = S[r][j];
            v.x = fmaf(a, v.x, u * Bv[j].x);
            v.y = fmaf(a, v.y, u * Bv[j].y);
            v.z = fmaf(a, v.z, u * Bv[j].z);
            v.w = fmaf(a, v.w, u * Bv[j].w);
            acc = fmaf(v.x, Cv[j].x, acc);
            acc = fmaf(v.y, Cv[j].y, acc);
            acc = fmaf(v.z, Cv[j].z, acc);
            acc = fmaf(v.w, Cv[j].w, acc);
            if (state_out && row < rows) store4_nt(state_out + base + (int64_t)row * N + j * 32, v);
        }
        acc += __shfl_xor(acc, 1, 64);
        acc += __shfl_xor(acc, 2, 64);
        acc += __shfl_xor(acc, 4, 64);
        if (e == 0 && row < rows)
            y[(n * d.H + h) * d.P + p0 + row] = (TO)(D ? fmaf(D[h], xv, acc) : acc);
    }
}

// hist <- [hist rows 1..K-2; xbc row], 16 bytes of channels a thread
template <typename TI>
__global__ __launch_bounds__(256) void ssm_hist_shift_kernel(SsmDims d, int K, const TI *__restrict__ xbc, TI *hist)
{
    constexpr int V = Vec16<TI>::n;
    const int c = (blockIdx.x * 256 + threadIdx.x) * V;
    const int64_t n = (int64_t)blockIdx.z * gridDim.y + blockIdx.y;
    if (n >= d.n_seq || c >= d.C) return;
    TI *h = hist + n * (K - 1) * d.C + c;
    for (int k = 0; k < K - 2; ++k) st16(h + (int64_t)k * d.C, ld16(h + (int64_t)(k + 1) * d.C));
    st16(h + (int64_t)(K - 2) * d.C, ld16(xbc + n * d.xbc_stride + c));
}

// 64 rows a block (R = 2) form a head's B and C half as often as 32 do; 32 make
// more blocks, which a launch of less than 2048 (8 a CU) needs.  Measured, 64
// heads of 64, N = 128: one sequence 4.6 us by 64, 4.2 by 32; 64 sequences 50.6
// (5.4 TB/s) and 52.3.
template <typename TI, typename TO, int N, int K>
static void launch_step_t(const SsmDims &d, const SsmStepArgs &a, hipStream_t st)
{
    const bool in_place = a.hist_out && a.hist_out == a.hist;
    const bool wide = (int64_t)d.n_seq * d.H * ((d.P + 31) / 32) >= 2048 && d.P > 32;
    const int tiles = (d.P + (wide ? 63 : 31)) / (wide ? 64 : 32);
    const unsigned gy = d.n_seq < 32768 ? d.n_seq : 32768;
    const dim3 grid(d.H * tiles, gy, (d.n_seq + gy - 1) / gy);
    hipLaunchKernelGGL((wide ? ssm_step_kernel<TI, TO, N, K, 2> : ssm_step_kernel<TI, TO, N, K, 1>), grid, dim3(256), 0, st, d,
                       tiles, static_cast<const TI *>(a.xbc), static_cast<const TI *>(a.conv_w),
                       static_cast<const TI *>(a.conv_b), static_cast<const TI *>(a.dt), a.A_log,
                       a.dt_bias, a.D, static_cast<const TI *>(a.hist),
                       in_place ? nullptr : static_cast<TI *>(a.hist_out), a.state, a.state_out,
                       static_cast<TO *>(a.y));
    if (in_place) {
        constexpr int V = Vec16<TI>::n;
        const dim3 sg((d.C / V + 255) / 256, gy, (d.n_seq + gy - 1) / gy);
        hipLaunchKernelGGL((ssm_hist_shift_kernel<TI>), sg, dim3(256), 0, st, d, K,
                           static_cast<const TI *>(a.xbc), static_cast<TI *>(a.hist_out));
    }
}

template <typename TI, typename TO, int N>
static void launch_step_k(const SsmDims &d, int K, const SsmStepArgs &a, hipStream_t st)
{
    if (K == 2) launch_step_t<TI, TO, N, 2>(d, a, st);
    else if (K == 3) launch_step_t<TI, TO, N, 3>(d, a, st);
    else launch_step_t<TI, TO, N, 4>(d, a, st);
}

template <typename TI, typename TO>
static void launch_step_n(const SsmDims &d, int K, const SsmStepArgs &a, hipStream_t st)
{
    if (d.N == 32) launch_step_k<TI, TO, 32>(d, K, a, st);
    else if (d.N == 64) launch_step_k<TI, TO, 64>(d, K, a, st);
    else if (d.N == 128) launch_step_k<TI, TO, 128>(d, K, a, st);
    else launch_step_k<TI, TO, 256>(d, K, a, st);
}

hipError_t launch_ssm_step(const gdn_ssm_shape &s, const SsmStepArgs &a, hipStream_t st)
{
    const SsmDims d = ssm_dims(s);
    GDN_SSM_IO(s.io_dtype,
        if (s.out_dtype == GDN_F32) launch_step_n<TI, float>(d, s.conv_width, a, st);
        else launch_step_n<TI, TI>(d, s.conv_width, a, st);)
    return hipGetLastError();
}

} // namespace gdn
