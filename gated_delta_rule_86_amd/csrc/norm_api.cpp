// norm_api.cpp -- host side of the norms around a block (kda_gated_norm*, kda_residual_norm* in include/kda.h):
// argument checks and launches.  The checks are plain host code that touches no HIP API.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <hip/hip_runtime.h>

#include "host_checks.h"
#include "kda.h"
#include "norm_internal.h"

namespace {

using kda::aligned;
using kda::kMaxElems;
using kda::overlap;
using kda::Range;
using kda::range_of;

int size_of(int dtype) { return dtype == KDA_DTYPE_FP32 ? 4 : 2; }
bool dtype_ok(int d) { return d == KDA_DTYPE_BF16 || d == KDA_DTYPE_FP32 || d == KDA_DTYPE_FP16; }

// Rows stay below 2^31: the kernels find a row's place with 32-bit numbers.
kda_status check_shape(int64_t B, int64_t T, int64_t H, int64_t D, int64_t most_d)
{
    if (B < 1 || T < 0 || H < 1 || H > 65536 || T >= ((int64_t)1 << 31) || B >= ((int64_t)1 << 31) ||
        (T > 0 && B > (((int64_t)1 << 31) - 1) / T) || (T > 0 && B * T > (((int64_t)1 << 31) - 1) / H))
        return KDA_ERR_SHAPE;
    if (D < 8 || D > most_d || D % 8)
        return KDA_ERR_HEAD_DIM;
    return KDA_OK;
}

// A strided input [B, T, H, D]: batch, token and head strides in elements, NULL = contiguous.
kda_status set_view(const void *p, const int64_t *st, int64_t B, int64_t T, int64_t H, int64_t D, int size,
                    kda::NormView *v, Range *r)
{
    v->p = static_cast<unsigned char *>(const_cast<void *>(p));
    v->sb = st ? st[0] : T * H * D;
    v->st = st ? st[1] : H * D;
    v->sh = st ? st[2] : D;
    const int64_t unit = 16 / size;
    if (v->sb < 0 || v->st < 0 || v->sh < 0 || v->sb % unit || v->st % unit || v->sh % unit || v->sb > kMaxElems ||
        v->st > kMaxElems || v->sh > kMaxElems || T > kMaxElems / (v->st + 1) || B > kMaxElems / (v->sb + 1) ||
        H > kMaxElems / (v->sh + 1))
        return KDA_ERR_STRIDE;
    if (!aligned(p, 16))
        return KDA_ERR_ALIGN;
    // a row's index alone gives its place: heads, tokens and batch rows follow each other (a dimension of size 1 always does)
    if (H == 1)
        v->sh = T == 1 ? (B == 1 ? 0 : v->sb) : v->st;
    const int64_t rows_t = H * v->sh;
    v->flat = (T == 1 || v->st == rows_t) && (B == 1 || v->sb == T * rows_t);
    *r = range_of(p, T > 0 ? (size_t)((B - 1) * v->sb + (T - 1) * v->st + (H == 1 ? 0 : (H - 1) * v->sh) + D) * (size_t)size
                           : 0);
    return KDA_OK;
}

void set_sizes(kda::NormArgs *a, int64_t B, int64_t T, int64_t H, int64_t D)
{
    a->T = T;
    a->H = (int)H;
    a->D = (int)D;
    a->rows = (int)(B * T * H);
    a->inv_h = 1.0 / (double)H;
    a->inv_t = T > 0 ? 1.0 / (double)T : 1.0;
}

// Outputs overlap no input (callers leave out one that an output replaces in place) and not each other.
bool clear(const Range *in, int n_in, const Range *out, int n_out)
{
    for (int i = 0; i < n_out; ++i) {
        for (int j = 0; j < n_in; ++j)
            if (overlap(out[i], in[j]))
                return false;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j]))
                return false;
    }
    return true;
}

// Contiguous, as an output that takes its place has to be: one row, or rows D apart (rows 0 apart are one row broadcast, which
// every other workgroup still reads when the first output row is written)
bool dense(const kda::NormView &v, const kda::NormArgs &a) { return a.rows == 1 || (v.flat && v.sh == a.D); }

}  // namespace

extern "C" {

kda_status kda_gated_norm(const void *x, const void *gate, const float *weight, void *out, int64_t B, int64_t T, int64_t H,
                          int64_t D, kda_dtype dtype, kda_gate activation, float eps, const int64_t *strides_host,
                          void *stream)
{
    if (T != 0 && (!x || !gate || !out))
        return KDA_ERR_NULL;
    kda_status st = check_shape(B, T, H, D, kda::kGatedMaxD);
    if (st != KDA_OK)
        return st;
    if (!dtype_ok(dtype))
        return KDA_ERR_DTYPE;
    if (activation != KDA_GATE_SIGMOID && activation != KDA_GATE_SILU)
        return KDA_ERR_FLAGS;
    if (!(eps >= 0.0f) || !isfinite(eps))
        return KDA_ERR_SCALE;
    kda::NormArgs a;
    memset(&a, 0, sizeof(a));
    set_sizes(&a, B, T, H, D);
    const int size = size_of(dtype);
    Range rx, rz;
    if ((st = set_view(x, strides_host, B, T, H, D, size, &a.x, &rx)) != KDA_OK ||
        (st = set_view(gate, strides_host ? strides_host + 3 : nullptr, B, T, H, D, size, &a.z, &rz)) != KDA_OK)
        return st;
    if (!aligned(out, 16) || !aligned(weight, 4))
        return KDA_ERR_ALIGN;
    const Range ro = range_of(out, (size_t)a.rows * (size_t)D * (size_t)size);
    // in place: each value of a row is read before any of the row is written, by the same lane
    const bool over_x = out == x && dense(a.x, a), over_z = out == gate && dense(a.z, a);
    const Range none = {0, 0};
    const Range in[] = {over_x ? none : rx, over_z ? none : rz, range_of(weight, (size_t)D * 4)};
    if (!clear(in, 3, &ro, 1))
        return KDA_ERR_ALIAS;
    a.y = static_cast<unsigned char *>(out);
    a.w = weight;
    a.dtype = (int)dtype;
    a.act = activation == KDA_GATE_SILU;
    a.eps = eps;
    if (a.rows == 0)
        return KDA_OK;
    return kda::gated_launch(a, static_cast<hipStream_t>(stream)) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

size_t kda_gated_norm_bwd_workspace_size(int64_t B, int64_t T, int64_t H, int64_t D, kda_dtype dtype)
{
    if (check_shape(B, T, H, D, kda::kGatedMaxD) != KDA_OK || !dtype_ok(dtype))
        return 0;
    return (size_t)kda::gated_groups(B * T * H, (int)D, (int)dtype) * (size_t)D * 4;
}

kda_status kda_gated_norm_bwd(const void *x, const void *gate, const float *weight, const void *dout, void *dx, void *dgate,
                              float *dweight, int64_t B, int64_t T, int64_t H, int64_t D, kda_dtype dtype,
                              kda_gate activation, float eps, const int64_t *strides_host, void *workspace,
                              size_t workspace_bytes, void *stream)
{
    if ((T != 0 && (!x || !gate || !dout || !dx || !dgate)) || (dweight && !weight))
        return KDA_ERR_NULL;
    kda_status st = check_shape(B, T, H, D, kda::kGatedMaxD);
    if (st != KDA_OK)
        return st;
    if (!dtype_ok(dtype))
        return KDA_ERR_DTYPE;
    if (activation != KDA_GATE_SIGMOID && activation != KDA_GATE_SILU)
        return KDA_ERR_FLAGS;
    if (!(eps >= 0.0f) || !isfinite(eps))
        return KDA_ERR_SCALE;
    kda::NormArgs a;
    memset(&a, 0, sizeof(a));
    set_sizes(&a, B, T, H, D);
    const int size = size_of(dtype);
    Range rx, rz;
    if ((st = set_view(x, strides_host, B, T, H, D, size, &a.x, &rx)) != KDA_OK ||
        (st = set_view(gate, strides_host ? strides_host + 3 : nullptr, B, T, H, D, size, &a.z, &rz)) != KDA_OK)
        return st;
    if (!aligned(dout, 16) || !aligned(dx, 16) || !aligned(dgate, 16) || !aligned(weight, 4) || !aligned(dweight, 4) ||
        !aligned(workspace, 256))
        return KDA_ERR_ALIGN;
    const size_t bytes = (size_t)a.rows * (size_t)D * (size_t)size, wb = (size_t)D * 4;
    const Range in[] = {rx, rz, range_of(dout, bytes), range_of(weight, wb)};
    const Range out[] = {range_of(dx, bytes), range_of(dgate, bytes), range_of(dweight, wb),
                         range_of(dweight ? workspace : nullptr, workspace_bytes)};
    if (!clear(in, 4, out, 4))
        return KDA_ERR_ALIAS;
    a.groups = kda::gated_groups(a.rows, (int)D, (int)dtype);
    if (dweight && (!workspace || workspace_bytes < (size_t)a.groups * wb))
        return KDA_ERR_WORKSPACE;
    a.dy = static_cast<const unsigned char *>(dout);
    a.y = static_cast<unsigned char *>(dx);
    a.zo = static_cast<unsigned char *>(dgate);
    a.w = weight;
    a.dw = dweight;
    a.part = static_cast<float *>(workspace);
    a.dtype = (int)dtype;
    a.act = activation == KDA_GATE_SILU;
    a.eps = eps;
    if (a.rows == 0 && !dweight)
        return KDA_OK;
    return kda::gated_launch_bwd(a, static_cast<hipStream_t>(stream)) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

kda_status kda_residual_norm(const void *x, const void *residual, const float *weight, const float *scale,
                             const float *post_weight, void *out, void *residual_out, int64_t B, int64_t T, int64_t D,
                             kda_dtype dtype, kda_dtype residual_dtype, kda_norm post_norm, float eps,
                             const int64_t *strides_host, void *stream)
{
    if (T != 0 && (!x || !residual || !out || !residual_out))
        return KDA_ERR_NULL;
    kda_status st = check_shape(B, T, 1, D, kda::kResidualMaxD);
    if (st != KDA_OK)
        return st;
    if (!dtype_ok(dtype) || (residual_dtype != dtype && residual_dtype != KDA_DTYPE_FP32))
        return KDA_ERR_DTYPE;
    if ((post_norm != KDA_NORM_NONE && post_norm != KDA_NORM_RMS) || (post_weight && post_norm == KDA_NORM_NONE))
        return KDA_ERR_FLAGS;
    if (!(eps >= 0.0f) || !isfinite(eps))
        return KDA_ERR_SCALE;
    kda::NormArgs a;
    memset(&a, 0, sizeof(a));
    set_sizes(&a, B, T, 1, D);
    const int size = size_of(dtype), rsize = size_of(residual_dtype);
    int64_t sx[3], sz[3];
    if (strides_host) {
        sx[0] = strides_host[0], sx[1] = strides_host[1], sx[2] = 0;
        sz[0] = strides_host[2], sz[1] = strides_host[3], sz[2] = 0;
    }
    Range rx, rz;
    if ((st = set_view(x, strides_host ? sx : nullptr, B, T, 1, D, size, &a.x, &rx)) != KDA_OK ||
        (st = set_view(residual, strides_host ? sz : nullptr, B, T, 1, D, rsize, &a.z, &rz)) != KDA_OK)
        return st;
    if (!aligned(out, 16) || !aligned(residual_out, 16) || !aligned(weight, 4) || !aligned(scale, 4) || !aligned(post_weight, 4))
        return KDA_ERR_ALIGN;
    const size_t values = (size_t)a.rows * (size_t)D, wb = (size_t)D * 4;
    const Range none = {0, 0};
    // in place: a row's values are in registers before any of it is written, by the threads that read them
    const bool over_x = out == x && dense(a.x, a), over_z = residual_out == residual && dense(a.z, a);
    const Range out_r[] = {range_of(out, values * (size_t)size), range_of(residual_out, values * (size_t)rsize)};
    const Range w_in[] = {range_of(weight, wb), range_of(scale, wb), range_of(post_weight, wb)};
    const Range for_out[] = {over_x ? none : rx, rz}, for_res[] = {rx, over_z ? none : rz};
    if (!clear(w_in, 3, out_r, 2) || !clear(for_out, 2, out_r, 1) || !clear(for_res, 2, out_r + 1, 1))
        return KDA_ERR_ALIAS;
    a.y = static_cast<unsigned char *>(out);
    a.zo = static_cast<unsigned char *>(residual_out);
    a.w = weight;
    a.scale = scale;
    a.post = post_weight;
    a.post_norm = post_norm == KDA_NORM_RMS;
    a.dtype = (int)dtype;
    a.rdtype = (int)residual_dtype;
    a.eps = eps;
    if (a.rows == 0)
        return KDA_OK;
    return kda::residual_launch(a, static_cast<hipStream_t>(stream)) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

size_t kda_residual_norm_bwd_workspace_size(int64_t B, int64_t T, int64_t D)
{
    if (check_shape(B, T, 1, D, kda::kResidualMaxD) != KDA_OK)
        return 0;
    return (size_t)kda::residual_groups(B * T, (int)D) * (size_t)D * 12;
}

kda_status kda_residual_norm_bwd(const void *x, const void *residual_out, const void *dout, const void *dresidual_out,
                                 const float *weight, const float *scale, const float *post_weight, void *dx,
                                 void *dresidual, float *dweight, float *dscale, float *dpost_weight, int64_t B, int64_t T,
                                 int64_t D, kda_dtype dtype, kda_dtype residual_dtype, kda_norm post_norm, float eps,
                                 const int64_t *strides_host, void *workspace, size_t workspace_bytes, void *stream)
{
    if ((T != 0 && (!x || !residual_out || !dout || !dx || !dresidual)) || (dweight && !weight) || (dscale && !scale) ||
        (dpost_weight && !post_weight))
        return KDA_ERR_NULL;
    kda_status st = check_shape(B, T, 1, D, kda::kResidualMaxD);
    if (st != KDA_OK)
        return st;
    if (!dtype_ok(dtype) || (residual_dtype != dtype && residual_dtype != KDA_DTYPE_FP32))
        return KDA_ERR_DTYPE;
    if ((post_norm != KDA_NORM_NONE && post_norm != KDA_NORM_RMS) || (post_weight && post_norm == KDA_NORM_NONE))
        return KDA_ERR_FLAGS;
    if (!(eps >= 0.0f) || !isfinite(eps))
        return KDA_ERR_SCALE;
    kda::NormArgs a;
    memset(&a, 0, sizeof(a));
    set_sizes(&a, B, T, 1, D);
    const int size = size_of(dtype), rsize = size_of(residual_dtype);
    int64_t sx[3], sz[3];
    if (strides_host) {
        sx[0] = strides_host[0], sx[1] = strides_host[1], sx[2] = 0;
        sz[0] = strides_host[2], sz[1] = strides_host[3], sz[2] = 0;
    }
    Range rx, rz;
    if ((st = set_view(x, strides_host ? sx : nullptr, B, T, 1, D, size, &a.x, &rx)) != KDA_OK ||
        (st = set_view(residual_out, strides_host ? sz : nullptr, B, T, 1, D, rsize, &a.z, &rz)) != KDA_OK)
        return st;
    const void *p16[] = {dout, dresidual_out, dx, dresidual};
    for (const void *p : p16)
        if (!aligned(p, 16))
            return KDA_ERR_ALIGN;
    const void *p4[] = {weight, scale, post_weight, dweight, dscale, dpost_weight};
    for (const void *p : p4)
        if (!aligned(p, 4))
            return KDA_ERR_ALIGN;
    if (!aligned(workspace, 256))
        return KDA_ERR_ALIGN;
    const bool sums = dweight || dscale || dpost_weight;
    const size_t values = (size_t)a.rows * (size_t)D, wb = (size_t)D * 4;
    const Range in[] = {rx, rz, range_of(dout, values * (size_t)size), range_of(dresidual_out, values * (size_t)rsize),
                        range_of(weight, wb), range_of(scale, wb), range_of(post_weight, wb)};
    const Range out[] = {range_of(dx, values * (size_t)size), range_of(dresidual, values * (size_t)rsize),
                         range_of(dweight, wb), range_of(dscale, wb), range_of(dpost_weight, wb),
                         range_of(sums ? workspace : nullptr, workspace_bytes)};
    if (!clear(in, 7, out, 6))
        return KDA_ERR_ALIAS;
    a.groups = kda::residual_groups(a.rows, (int)D);
    if (sums && (!workspace || workspace_bytes < 3 * (size_t)a.groups * wb))
        return KDA_ERR_WORKSPACE;
    a.dy = static_cast<const unsigned char *>(dout);
    a.dz = static_cast<const unsigned char *>(dresidual_out);
    a.y = static_cast<unsigned char *>(dx);
    a.zo = static_cast<unsigned char *>(dresidual);
    a.w = weight;
    a.scale = scale;
    a.post = post_weight;
    a.dw = dweight;
    a.dscale = dscale;
    a.dpost = dpost_weight;
    a.part = static_cast<float *>(workspace);
    a.post_norm = post_norm == KDA_NORM_RMS;
    a.dtype = (int)dtype;
    a.rdtype = (int)residual_dtype;
    a.eps = eps;
    if (a.rows == 0 && !sums)
        return KDA_OK;
    return kda::residual_launch_bwd(a, static_cast<hipStream_t>(stream)) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

}  // extern "C"
