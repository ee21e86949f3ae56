// ssm_internal.h -- launchers behind the C ABI of include/gdn_ssm.h.  Each
// one assumes its arguments were validated by the ABI layer and only enqueues.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/gdn_ssm.h"

namespace gdn {

// The sizes the kernels take by value, strides resolved.
struct SsmDims {
    int H, P, G, N, C, n_seq;
    int hg;  // heads of a group
    int64_t T, xbc_stride, dt_stride;
    float dt_min, dt_max;
};

inline SsmDims ssm_dims(const gdn_ssm_shape &s)
{
    SsmDims d;
    d.H = s.heads;
    d.P = s.head_dim;
    d.G = s.groups;
    d.N = s.state_dim;
    d.C = s.heads * s.head_dim + 2 * s.groups * s.state_dim;
    d.n_seq = s.n_seq;
    d.hg = s.heads / s.groups;
    d.T = s.total_T;
    d.xbc_stride = s.xbc_stride ? s.xbc_stride : d.C;
    d.dt_stride = s.dt_stride ? s.dt_stride : d.H;
    d.dt_min = s.dt_min;
    d.dt_max = s.dt_max;
    return d;
}

struct SsmConvArgs {
    const int32_t *cu;
    const void *xbc, *conv_w, *conv_b, *hist;
    void *hist_out, *out;
};

struct SsmScanArgs {
    const int32_t *cu;
    const void *xbc, *dt;
    const float *A_log, *dt_bias, *D, *state;
    float *state_out;
    void *y;
    void *ws;
};

struct SsmStepArgs {
    const void *xbc, *conv_w, *conv_b, *dt;
    const float *A_log, *dt_bias, *D;
    const void *hist;
    void *hist_out;  // hist itself: shifted in place by a second launch
    const float *state;
    float *state_out;
    void *y;
};

struct NormArgs {
    const void *x, *z, *weight, *bias;
    void *y;
};

size_t ssm_scan_workspace_bytes(const gdn_ssm_shape &s);

hipError_t launch_ssm_conv(const gdn_ssm_shape &s, const SsmConvArgs &a, hipStream_t st);
hipError_t launch_ssm_scan(const gdn_ssm_shape &s, const SsmScanArgs &a, hipStream_t st);
hipError_t launch_ssm_step(const gdn_ssm_shape &s, const SsmStepArgs &a, hipStream_t st);
hipError_t launch_group_norm(const gdn_norm_shape &s, const NormArgs &a, hipStream_t st);

} // namespace gdn
