// ssm_norm.hip -- per-token group norm (RMS or centred) with a SiLU gate before
// or after it, over the consecutive channels of a token row.
//
//   v = x SiLU(z) (gate first) or x;  m = mean_g v (centred) or 0
//   y = (v - m) / sqrt(mean_g (v - m)^2 + eps) w + b  (times SiLU(z), gate last)
//
// gfx950 mapping.  One read of x and z and one write of y for about 12 flop:
// bound by HBM bandwidth, and by latency for a single row.  A team of `TEAM`
// lanes (a power of two, 8 to 256) owns one group of a row and keeps its
// values in registers between the sums and the output, V vectors of 8 channels
// a lane, vector i of lane l at 8 (i TEAM + l): whole lines per instruction.
// The squares are those of v - m, from the registers, so no precision is lost
// to a large mean.  Sums run over the lane's values, then across the team.
// Measured: 27135 rows of 64 groups of 64 bf16 channels 124 us, 5.4 TB/s; 2048
// rows of 8 groups of 512, x fp32, 13 us, 5.1 TB/s; one row of 4096 3.4 us.
#include "ssm_device.h"
#include "ssm_internal.h"

namespace gdn {

// Sum over a team of TEAM consecutive lanes (teams of more than a wave: over
// the block, through `part`); every lane gets the same bits.
template <int TEAM>
__device__ __forceinline__ float team_sum(float x, float *part)
{
#pragma unroll
    for (int m = (TEAM < 64 ? TEAM : 64) / 2; m > 0; m >>= 1) x += __shfl_xor(x, m, 64);
    if (TEAM > 64) {
        const int wave = threadIdx.x >> 6;
        __syncthreads();  // (the previous sum has been read)
        if ((threadIdx.x & 63) == 0) part[wave] = x;
        __syncthreads();
        constexpr int W = TEAM / 64;
        const int w0 = wave / (W > 0 ? W : 1) * W;
        x = 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i) x += part[w0 + i];
    }
    return x;
}

struct NormDims {
    int64_t units, x_stride, z_stride;  // units: rows * groups
    int channels, groups, size;         // size: channels of a group
    float eps;
};

template <typename TX, typename TI, int TEAM, int V>
__global__ __launch_bounds__(256) void group_norm_kernel(NormDims d, const TX *__restrict__ x,
                                                         const TI *__restrict__ z,
                                                         const TI *__restrict__ w,
                                                         const TI *__restrict__ bias,
                                                         TI *__restrict__ y, int flags)
{
    __shared__ float part[4];
    const int lane = threadIdx.x & (TEAM - 1);
    const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    const int64_t unit = block * (256 / TEAM) + threadIdx.x / TEAM;
    // a team past the last unit leaves as a whole, except that the lanes of a
    // multi-wave team all stay for the block's barriers
    const bool live = unit < d.units;
    if (TEAM <= 64 && !live) return;
    const int64_t row = live ? unit / d.groups : 0;
    const int ch0 = live ? (int)(unit - row * d.groups) * d.size : 0;
    const bool last = flags & GDN_NORM_GATE_LAST, centre = flags & GDN_NORM_CENTRE;

    float v[V][8], g[V][8];
    bool in[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = (i * TEAM + lane) * 8;
        in[i] = live && c < d.size;
#pragma unroll
        for (int j = 0; j < 8; ++j) { v[i][j] = 0.f; g[i][j] = 1.f; }
        if (in[i]) {
            load8f(x + row * d.x_stride + ch0 + c, v[i]);
            if (z) load8f(z + row * d.z_stride + ch0 + c, g[i]);
        }
    }
    if (z) {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) g[i][j] = silu_fast(g[i][j]);
        if (!last) {
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = in[i] ? v[i][j] * g[i][j] : 0.f;
        }
    }
    const float inv_n = 1.0f / (float)d.size;
    float mean = 0.f;
    if (centre) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) s += v[i][j];
        mean = team_sum<TEAM>(s, part) * inv_n;
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[i][j] -= mean;
            ss = in[i] ? fmaf(v[i][j], v[i][j], ss) : ss;
        }
    const float r = 1.0f / sqrtf(team_sum<TEAM>(ss, part) * inv_n + d.eps);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (!in[i]) continue;
        const int c = ch0 + (i * TEAM + lane) * 8;
        float wv[8], bv[8], o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) { wv[j] = 1.f; bv[j] = 0.f; }
        if (w) load8f(w + c, wv);
        if (bias) load8f(bias + c, bv);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            o[j] = fmaf(v[i][j] * r, wv[j], bv[j]);
            if (last) o[j] *= g[i][j];
        }
        store8f(y + row * d.channels + c, o);
    }
}

template <typename TX, typename TI, int TEAM, int V>
static void launch_norm_t(const NormDims &d, const NormArgs &a, int flags, hipStream_t st)
{
    const int64_t blocks = (d.units + 256 / TEAM - 1) / (256 / TEAM);
    const int64_t gx = blocks < (1 << 22) ? blocks : 1 << 22;
    hipLaunchKernelGGL((group_norm_kernel<TX, TI, TEAM, V>), dim3((unsigned)gx, (unsigned)((blocks + gx - 1) / gx)),
                       dim3(256), 0, st, d, static_cast<const TX *>(a.x), static_cast<const TI *>(a.z),
                       static_cast<const TI *>(a.weight), static_cast<const TI *>(a.bias),
                       static_cast<TI *>(a.y), flags);
}

// Teams of the smallest power of two that gives a lane one vector; above 256
// lanes (2048 channels) 2, 4 or 8 vectors a lane.
template <typename TX, typename TI>
static void launch_norm_size(const NormDims &d, const NormArgs &a, int flags, hipStream_t st)
{
    const int n = d.size / 8;
    if (n <= 8) launch_norm_t<TX, TI, 8, 1>(d, a, flags, st);
    else if (n <= 16) launch_norm_t<TX, TI, 16, 1>(d, a, flags, st);
    else if (n <= 32) launch_norm_t<TX, TI, 32, 1>(d, a, flags, st);
    else if (n <= 64) launch_norm_t<TX, TI, 64, 1>(d, a, flags, st);
    else if (n <= 128) launch_norm_t<TX, TI, 128, 1>(d, a, flags, st);
    else if (n <= 256) launch_norm_t<TX, TI, 256, 1>(d, a, flags, st);
    else if (n <= 512) launch_norm_t<TX, TI, 256, 2>(d, a, flags, st);
    else if (n <= 1024) launch_norm_t<TX, TI, 256, 4>(d, a, flags, st);
    else launch_norm_t<TX, TI, 256, 8>(d, a, flags, st);
}

hipError_t launch_group_norm(const gdn_norm_shape &s, const NormArgs &a, hipStream_t st)
{
    NormDims d;
    d.units = s.rows * s.groups;
    d.channels = s.channels;
    d.groups = s.groups;
    d.size = s.channels / s.groups;
    d.x_stride = s.x_stride ? s.x_stride : s.channels;
    d.z_stride = s.z_stride ? s.z_stride : s.channels;
    d.eps = s.eps;
    GDN_SSM_IO(s.io_dtype,
        if (s.x_dtype == GDN_F32) launch_norm_size<float, TI>(d, a, s.flags, st);
        else launch_norm_size<TI, TI>(d, a, s.flags, st);)
    return hipGetLastError();
}

} // namespace gdn
