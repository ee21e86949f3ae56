// ssm_scan.hip -- the selective state space recurrence over whole prompts.
//
//   dt = clamp(softplus(dt_raw + dt_bias)), a = exp(-exp(A_log) dt)
//   S <- a S + dt x B^T,  y = S C + D x      per token, S the P x N state of a head
//
// One wave per (sequence, head, row p of the state), token by token: lane l
// holds the state elements n = l, l + 64, ...  Bound by the latency of a
// token's loads and its sum over the wave.
#include "ssm_device.h"
#include "ssm_internal.h"

namespace gdn {

template <typename TI, typename TO, int N>
__global__ __launch_bounds__(256) void ssm_scan_kernel(
    SsmDims d, const int32_t *__restrict__ cu, const TI *__restrict__ xbc,
    const TI *__restrict__ dt_raw, const float *__restrict__ A_log,
    const float *__restrict__ dt_bias, const float *__restrict__ D, const float *state,
    float *state_out, TO *__restrict__ y)
{
    constexpr int NL = N < 64 ? 1 : N / 64;
    const int64_t n = (int64_t)blockIdx.z * gridDim.y + blockIdx.y;
    if (n >= d.n_seq) return;
    const int l = threadIdx.x & 63;
    const int col = blockIdx.x * 4 + (threadIdx.x >> 6);  // h*P + p
    const int h = col / d.P, grp = h / d.hg;
    const int begin = seq_bound(cu, n, d.T), end = seq_bound(cu, n + 1, d.T);
    const int64_t at = (n * d.H * d.P + col) * N;
    float S[NL];
#pragma unroll
    for (int j = 0; j < NL; ++j) S[j] = state && l + 64 * j < N ? state[at + l + 64 * j] : 0.f;
    const float na = -expf(A_log[h]), bias = dt_bias[h], Dh = D ? D[h] : 0.f;
    for (int t = begin; t < end; ++t) {
        const TI *row = xbc + (int64_t)t * d.C;
        float dt, lam;
        step_size((float)dt_raw[t * d.dt_stride + h], bias, na, d.dt_min, d.dt_max, dt, lam);
        const float a = expf(lam), xv = (float)row[col];
        const TI *B = row + d.H * d.P + grp * N, *C = B + d.G * N;
        float acc = 0.f;
#pragma unroll
        for (int j = 0; j < NL; ++j) {
            const bool in = l + 64 * j < N;
            S[j] = fmaf(a, S[j], dt * xv * (in ? (float)B[l + 64 * j] : 0.f));
            acc = fmaf(S[j], in ? (float)C[l + 64 * j] : 0.f, acc);
        }
        for (int m = 32; m > 0; m >>= 1) acc += __shfl_xor(acc, m, 64);
        if (l == 0) y[(int64_t)t * d.H * d.P + col] = (TO)(D ? fmaf(Dh, xv, acc) : acc);
    }
    if (state_out) {
#pragma unroll
        for (int j = 0; j < NL; ++j)
            if (l + 64 * j < N) state_out[at + l + 64 * j] = S[j];
    }
}

size_t ssm_scan_workspace_bytes(const gdn_ssm_shape &) { return 0; }

template <typename TI, typename TO, int N>
static void launch_scan_t(const SsmDims &d, const SsmScanArgs &a, hipStream_t st)
{
    const unsigned gy = d.n_seq < 32768 ? d.n_seq : 32768;
    hipLaunchKernelGGL((ssm_scan_kernel<TI, TO, N>), dim3(d.H * d.P / 4, gy, (d.n_seq + gy - 1) / gy),
                       dim3(256), 0, st, d, a.cu, static_cast<const TI *>(a.xbc),
                       static_cast<const TI *>(a.dt), a.A_log, a.dt_bias, a.D, a.state, a.state_out,
                       static_cast<TO *>(a.y));
}

template <typename TI, typename TO>
static void launch_scan_n(const SsmDims &d, const SsmScanArgs &a, hipStream_t st)
{
    if (d.N == 32) launch_scan_t<TI, TO, 32>(d, a, st);
    else if (d.N == 64) launch_scan_t<TI, TO, 64>(d, a, st);
    else if (d.N == 128) launch_scan_t<TI, TO, 128>(d, a, st);
    else launch_scan_t<TI, TO, 256>(d, a, st);
}

hipError_t launch_ssm_scan(const gdn_ssm_shape &s, const SsmScanArgs &a, hipStream_t st)
{
    const SsmDims d = ssm_dims(s);
    GDN_SSM_IO(s.io_dtype,
        if (s.out_dtype == GDN_F32) launch_scan_n<TI, float>(d, a, st);
        else launch_scan_n<TI, TI>(d, a, st);)
    return hipGetLastError();
}

} // namespace gdn
