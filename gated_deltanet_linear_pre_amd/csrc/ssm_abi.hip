// ssm_abi.hip -- the extern "C" entry points of include/gdn_ssm.h: argument
// checks (all before anything is enqueued), then the launchers.
#include <math.h>
#include <stdint.h>

#include "ssm_internal.h"

namespace {

using gdn::NormArgs;
using gdn::SsmConvArgs;
using gdn::SsmScanArgs;
using gdn::SsmStepArgs;

constexpr int kMaxHeads = 1 << 12;
constexpr int kMaxSeqs = 1 << 20;
constexpr int kMaxGroupChannels = 16384;
constexpr int kMaxRowChannels = 65536;
constexpr int64_t kMaxRows = (int64_t)1 << 27;  // (keeps every launch grid inside its limits)
constexpr int64_t kMaxStride = (int64_t)1 << 40;

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

bool dtype_ok(int32_t t) { return t == GDN_F32 || t == GDN_F16 || t == GDN_BF16; }
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

int check_shape(const gdn_ssm_shape *s)
{
    if (!s) return GDN_E_NULL;
    if (!dtype_ok(s->io_dtype)) return GDN_E_DTYPE;
    if (s->out_dtype != GDN_F32 && s->out_dtype != s->io_dtype) return GDN_E_DTYPE;
    if (s->groups < 1 || s->heads < 1 || s->heads > kMaxHeads || s->heads % s->groups) return GDN_E_SHAPE;
    if (s->head_dim < 16 || s->head_dim > 256 || s->head_dim % 16) return GDN_E_SHAPE;
    if (s->state_dim != 32 && s->state_dim != 64 && s->state_dim != 128 && s->state_dim != 256)
        return GDN_E_SHAPE;
    if (s->conv_width < 2 || s->conv_width > 4) return GDN_E_SHAPE;
    if (s->n_seq < 1 || s->n_seq > kMaxSeqs) return GDN_E_SHAPE;
    if (s->total_T < 0 || s->total_T > kMaxRows) return GDN_E_SHAPE;
    if (s->max_T < 0 || s->max_T > s->total_T) return GDN_E_SHAPE;
    if (!(s->dt_min >= 0.f) || !(s->dt_max >= s->dt_min)) return GDN_E_SHAPE;
    const int64_t C = (int64_t)s->heads * s->head_dim + 2 * (int64_t)s->groups * s->state_dim;
    if (s->xbc_stride != 0 && (s->xbc_stride < C || s->xbc_stride > kMaxStride)) return GDN_E_SHAPE;
    if (s->dt_stride != 0 && (s->dt_stride < s->heads || s->dt_stride > kMaxStride)) return GDN_E_SHAPE;
    return GDN_OK;
}

// rows of the raw xbc start on 16 bytes
int check_rows(const gdn_ssm_shape *s)
{
    return s->xbc_stride * elem(s->io_dtype) % 16 ? GDN_E_ALIGN : GDN_OK;
}

int check_norm(const gdn_norm_shape *s)
{
    if (!s) return GDN_E_NULL;
    if (!dtype_ok(s->io_dtype)) return GDN_E_DTYPE;
    if (s->x_dtype != GDN_F32 && s->x_dtype != s->io_dtype) return GDN_E_DTYPE;
    if (s->rows < 0 || s->rows > kMaxRows) return GDN_E_SHAPE;
    if (s->groups < 1 || s->channels < 1 || s->channels > kMaxRowChannels) return GDN_E_SHAPE;
    if (s->channels % s->groups || s->channels / s->groups % 8) return GDN_E_SHAPE;
    if (s->channels / s->groups > kMaxGroupChannels) return GDN_E_SHAPE;
    if (s->flags & ~(GDN_NORM_CENTRE | GDN_NORM_GATE_LAST)) return GDN_E_SHAPE;
    if (!(isfinite(s->eps) && s->eps >= 0.f)) return GDN_E_SHAPE;
    if (s->x_stride != 0 && (s->x_stride < s->channels || s->x_stride > kMaxStride)) return GDN_E_SHAPE;
    if (s->z_stride != 0 && (s->z_stride < s->channels || s->z_stride > kMaxStride)) return GDN_E_SHAPE;
    if (s->x_stride * elem(s->x_dtype) % 16 || s->z_stride * elem(s->io_dtype) % 16) return GDN_E_ALIGN;
    return GDN_OK;
}

} // namespace

extern "C" {

int gdn_ssm_conv(const gdn_ssm_shape *shape, const int32_t *cu_seqlens, const void *xbc,
                 const void *conv_w, const void *conv_b, const void *hist, void *hist_out,
                 void *out, void *stream)
{
    int st = check_shape(shape);
    if (st) return st;
    st = check_rows(shape);
    if (st) return st;
    REQ(cu_seqlens); REQ(conv_w);
    if (shape->total_T > 0) { REQ(xbc); REQ(out); }  // (buffers of no rows may have no address)
    ALN(cu_seqlens, 4); ALN(xbc, 16); ALN(conv_w, 16); ALN(conv_b, 16); ALN(hist, 16);
    ALN(hist_out, 16); ALN(out, 16);
    const SsmConvArgs a{cu_seqlens, xbc, conv_w, conv_b, hist, hist_out, out};
    return launch_status(gdn::launch_ssm_conv(*shape, a, (hipStream_t)stream));
}

size_t gdn_ssm_scan_workspace_bytes(const gdn_ssm_shape *shape)
{
    if (check_shape(shape) != GDN_OK) return 0;
    return gdn::ssm_scan_workspace_bytes(*shape);
}

int gdn_ssm_scan(const gdn_ssm_shape *shape, const int32_t *cu_seqlens, const void *xbc,
                 const void *dt, const float *A_log, const float *dt_bias, const float *D,
                 const float *state, float *state_out, void *y, void *workspace,
                 size_t workspace_bytes, void *stream)
{
    int st = check_shape(shape);
    if (st) return st;
    REQ(cu_seqlens); REQ(A_log); REQ(dt_bias);
    if (shape->total_T > 0) { REQ(xbc); REQ(dt); REQ(y); }
    ALN(cu_seqlens, 4); ALN(A_log, 4); ALN(dt_bias, 4); ALN(D, 4);
    ALN(dt, elem(shape->io_dtype));
    ALN(xbc, 16); ALN(state, 16); ALN(state_out, 16); ALN(y, 16);
    const size_t need = gdn::ssm_scan_workspace_bytes(*shape);
    if (need > 0) REQ(workspace);
    ALN(workspace, 256);
    if (workspace_bytes < need) return GDN_E_WORKSPACE;
    const SsmScanArgs a{cu_seqlens, xbc, dt, A_log, dt_bias, D, state, state_out, y, workspace};
    return launch_status(gdn::launch_ssm_scan(*shape, a, (hipStream_t)stream));
}

int gdn_ssm_step(const gdn_ssm_shape *shape, const void *xbc, const void *conv_w,
                 const void *conv_b, const void *dt, const float *A_log, const float *dt_bias,
                 const float *D, const void *hist, void *hist_out, const float *state,
                 float *state_out, void *y, void *stream)
{
    int st = check_shape(shape);
    if (st) return st;
    st = check_rows(shape);
    if (st) return st;
    if (shape->total_T != shape->n_seq || shape->max_T != 1) return GDN_E_SHAPE;
    REQ(xbc); REQ(conv_w); REQ(dt); REQ(A_log); REQ(dt_bias); REQ(y);
    ALN(A_log, 4); ALN(dt_bias, 4); ALN(D, 4); ALN(dt, elem(shape->io_dtype));
    ALN(xbc, 16); ALN(conv_w, 16); ALN(conv_b, 16); ALN(hist, 16); ALN(hist_out, 16);
    ALN(state, 16); ALN(state_out, 16); ALN(y, 16);
    const SsmStepArgs a{xbc, conv_w, conv_b, dt, A_log, dt_bias, D, hist, hist_out, state, state_out, y};
    return launch_status(gdn::launch_ssm_step(*shape, a, (hipStream_t)stream));
}

int gdn_group_norm(const gdn_norm_shape *shape, const void *x, const void *z, const void *weight,
                   const void *bias, void *y, void *stream)
{
    const int st = check_norm(shape);
    if (st) return st;
    if (shape->rows == 0) return GDN_OK;
    REQ(x); REQ(y);
    ALN(x, 16); ALN(z, 16); ALN(weight, 16); ALN(bias, 16); ALN(y, 16);
    const NormArgs a{x, z, weight, bias, y};
    return launch_status(gdn::launch_group_norm(*shape, a, (hipStream_t)stream));
}

} // extern "C"
