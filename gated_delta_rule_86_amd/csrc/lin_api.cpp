// lin_api.cpp -- host side of the decayed linear attention (kda_lin_* in include/kda.h):
// argument checks, workspace layout, launches.  The checks are plain host code that touches no
// HIP API, so every error path can be exercised without a GPU.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <hip/hip_runtime.h>

#include "host_checks.h"
#include "kda.h"
#include "lin_internal.h"

namespace {

using kda::aligned;
using kda::check_cu;
using kda::dtype_ok;
using kda::kD;
using kda::overlap;
using kda::Range;
using kda::range_of;
using kda::set_tensor;
using kda::state_bytes;
using Sizes = kda::HeadSizes;

kda_status check_sizes(int64_t B, int64_t T, int64_t Hk, int64_t H, int64_t N, bool varlen, Sizes *z)
{
    const kda_status st = kda::check_head_sizes(B, T, Hk, H, N, varlen, z);
    if (st != KDA_OK)
        return st;
    return z->n_seq >= ((int64_t)1 << 29) || z->n_seq > (((int64_t)1 << 31) - 64) / (4 * H) ? KDA_ERR_SHAPE : KDA_OK;
}

bool make_layout(const Sizes &z, bool bwd, bool ddecay, kda::LinLayout *L)
{
    using kda::kAlign;
    L->plan = kda::lin_plan(z.B, z.T, z.H, z.N, z.varlen, bwd ? 3 : 1, ddecay ? kda::kLinGradSeg : 0);
    const kda::LinPlan &p = L->plan;
    // a launch holds less than 2^32 threads: 512 per segment and head at most, 8192 per row and head in the scan
    if (p.rows * p.P > (((int64_t)1 << 23) - 8) / z.H || (p.P > 1 && p.rows >= ((int64_t)1 << 19) / z.H))
        return false;
    size_t off = kAlign;  // status word
    auto take = [&](size_t bytes) {
        const size_t o = off;
        off = (off + bytes + kAlign - 1) / kAlign * kAlign;
        return o;
    };
    const size_t slots = (size_t)p.rows * (size_t)p.P * (size_t)z.H;
    L->off_fwd = L->off_flam = L->off_rev = L->off_rlam = L->off_dq = L->off_dk = 0;
    L->off_qd = L->off_kd = L->off_xfin = L->off_part = 0;
    if (p.P > 1) {
        L->off_fwd = take(slots * kda::kLinStateBytes);
        L->off_flam = take(slots * sizeof(float));
    }
    if (bwd) {
        const size_t rows = (size_t)z.B * (size_t)z.T;
        if (p.P > 1) {
            L->off_rev = take(slots * kda::kLinStateBytes);
            L->off_rlam = take(slots * sizeof(float));
        }
        if (z.Hk != z.H) {
            L->off_dq = take(rows * (size_t)z.H * kD * sizeof(float));
            L->off_dk = take(rows * (size_t)z.H * kD * sizeof(float));
        }
        if (ddecay) {
            L->off_qd = take(rows * (size_t)z.H * sizeof(float));
            L->off_kd = take(rows * (size_t)z.H * sizeof(float));
            L->off_xfin = take((size_t)z.n_seq * (size_t)z.H * sizeof(float));
            L->off_part = take(slots * sizeof(double));
        }
    }
    L->total = off;
    return true;
}

// Everything that the forward entry points check; fills role 0 and the sizes.
kda_status forward_args(const void *q, const void *k, const void *v, const float *decay, int per_token, float scale,
                        void *out, const void *h0, kda_state_dtype h0_dt, void *ht, kda_state_dtype ht_dt,
                        const int64_t *cu, const int64_t *cu_host, int64_t B, int64_t T, int64_t Hk, int64_t H,
                        int64_t N, int64_t K, int64_t V, const int64_t *strides, void *ws, size_t ws_bytes,
                        bool recurrent, kda::LinArgs *a, kda::LinLayout *lay)
{
    if ((!decay && !(per_token && T == 0)) || (T != 0 && (!q || !k || !v || !out)))
        return KDA_ERR_NULL;
    Sizes z;
    kda_status st = check_sizes(B, T, Hk, H, N, cu != nullptr, &z);
    if (st != KDA_OK)
        return st;
    if (K != kD || V != kD)
        return KDA_ERR_HEAD_DIM;
    if (!dtype_ok(h0_dt) || !dtype_ok(ht_dt) || (h0 == nullptr) != (h0_dt == KDA_STATE_NONE) ||
        (ht == nullptr) != (ht_dt == KDA_STATE_NONE) || (h0 && ht && h0_dt != ht_dt))
        return KDA_ERR_DTYPE;
    if (per_token != 0 && per_token != 1)
        return KDA_ERR_FLAGS;
    if (!isfinite(scale))
        return KDA_ERR_SCALE;
    // token by token nothing is cut, and a launch has 256 threads per sequence and head
    if (recurrent ? z.n_seq > (((int64_t)1 << 24) - 8) / H : !make_layout(z, false, false, lay))
        return KDA_ERR_SHAPE;
    memset(a, 0, sizeof(*a));
    kda::LinRole &r = a->role[0];
    Range rq, rk, rv;
    if ((st = set_tensor(q, strides, z, Hk, &r.q, &rq)) != KDA_OK ||
        (st = set_tensor(k, strides ? strides + 3 : nullptr, z, Hk, &r.k, &rk)) != KDA_OK ||
        (st = set_tensor(v, strides ? strides + 6 : nullptr, z, H, &r.v, &rv)) != KDA_OK)
        return st;
    if (!aligned(out, 16) || !aligned(decay, 4) || !aligned(h0, 16) || !aligned(ht, 16) || !aligned(cu, 8) ||
        !aligned(ws, kda::kAlign))
        return KDA_ERR_ALIGN;
    const size_t rows = (size_t)B * (size_t)T * (size_t)H;
    const Range ro = range_of(out, rows * kD * 2), rd = range_of(decay, (per_token ? rows : (size_t)H) * 4),
                rc = range_of(cu, cu ? (size_t)(N + 1) * 8 : 0),
                ri = range_of(h0, (size_t)z.n_seq * (size_t)H * state_bytes(h0_dt)),
                rf = range_of(ht, (size_t)z.n_seq * (size_t)H * state_bytes(ht_dt)), rw = range_of(ws, ws_bytes);
    const Range in[] = {rq, rk, rv, rd, rc};
    for (const Range &x : in)
        if (overlap(ro, x) || overlap(rf, x) || overlap(rw, x))
            return KDA_ERR_ALIAS;
    if (overlap(ro, ri) || overlap(ro, rf) || (h0 != ht && overlap(ri, rf)) || overlap(rw, ri) || overlap(rw, ro) ||
        overlap(rw, rf))
        return KDA_ERR_ALIAS;
    // token by token, the workspace holds the status word alone
    const size_t need = recurrent ? (cu ? kda::kAlign : 0) : lay->total;
    if (need && (!ws || ws_bytes < need))
        return KDA_ERR_WORKSPACE;
    if ((st = check_cu(cu, cu_host, z)) != KDA_OK)
        return st;
    unsigned char *w = static_cast<unsigned char *>(ws);
    r.init = h0;
    r.fin = ht;
    r.init_dt = (int)h0_dt;
    r.fin_dt = (int)ht_dt;
    r.out = out;
    if (!recurrent) {
        a->rows = lay->plan.rows;
        a->P = lay->plan.P;
        a->len = lay->plan.len;
    }
    if (a->P > 1) {
        r.slots = reinterpret_cast<float *>(w + lay->off_fwd);
        r.lam = reinterpret_cast<float *>(w + lay->off_flam);
        r.defer = ht && ht == h0 ? 1 : 0;
    }
    a->decay = decay;
    a->per_token = per_token;
    a->scale = scale;
    a->T = T;
    a->H = H;
    a->N = z.n_seq;
    a->cu = cu;
    a->status = reinterpret_cast<int32_t *>(w);
    return KDA_OK;
}

}  // namespace

extern "C" {

size_t kda_lin_fwd_workspace_size(int64_t B, int64_t T, int64_t H, int64_t N, int has_cu_seqlens)
{
    Sizes z;
    kda::LinLayout lay;
    if (check_sizes(B, T, H, H, N, has_cu_seqlens != 0, &z) != KDA_OK || !make_layout(z, false, false, &lay))
        return 0;
    return lay.total;
}

kda_status kda_lin_fwd(const void *q, const void *k, const void *v, const float *decay, int decay_per_token,
                       float scale, void *out, const void *initial_state, kda_state_dtype initial_state_dtype,
                       void *final_state, kda_state_dtype final_state_dtype, const int64_t *cu_seqlens,
                       const int64_t *cu_seqlens_host, int64_t B, int64_t T, int64_t Hk, int64_t H, int64_t N,
                       int64_t K, int64_t V, const int64_t *strides_host, void *workspace, size_t workspace_bytes,
                       void *stream)
{
    kda::LinArgs a;
    kda::LinLayout lay;
    const kda_status st = forward_args(q, k, v, decay, decay_per_token, scale, out, initial_state,
                                       initial_state_dtype, final_state, final_state_dtype, cu_seqlens,
                                       cu_seqlens_host, B, T, Hk, H, N, K, V, strides_host, workspace,
                                       workspace_bytes, false, &a, &lay);
    if (st != KDA_OK)
        return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (cu_seqlens && kda::lin_launch_check(cu_seqlens, a.N, T, a.status, s) != hipSuccess)
        return KDA_ERR_HIP;
    const int lead[1] = {0};
    return kda::lin_launch_walk(a, 1, lead, 1, s) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

kda_status kda_lin_fwd_recurrent(const void *q, const void *k, const void *v, const float *decay,
                                 int decay_per_token, float scale, void *out, const void *initial_state,
                                 kda_state_dtype initial_state_dtype, void *final_state,
                                 kda_state_dtype final_state_dtype, const int64_t *cu_seqlens,
                                 const int64_t *cu_seqlens_host, int64_t B, int64_t T, int64_t Hk, int64_t H,
                                 int64_t N, int64_t K, int64_t V, const int64_t *strides_host, void *workspace,
                                 size_t workspace_bytes, void *stream)
{
    kda::LinArgs a;
    kda::LinLayout lay;
    const kda_status st = forward_args(q, k, v, decay, decay_per_token, scale, out, initial_state,
                                       initial_state_dtype, final_state, final_state_dtype, cu_seqlens,
                                       cu_seqlens_host, B, T, Hk, H, N, K, V, strides_host, workspace,
                                       workspace_bytes, true, &a, &lay);
    if (st != KDA_OK)
        return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (cu_seqlens && kda::lin_launch_check(cu_seqlens, a.N, T, a.status, s) != hipSuccess)
        return KDA_ERR_HIP;
    return kda::lin_launch_recurrent(a, s) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

size_t kda_lin_bwd_workspace_size(int64_t B, int64_t T, int64_t Hk, int64_t H, int64_t N, int has_cu_seqlens,
                                  int need_ddecay)
{
    Sizes z;
    kda::LinLayout lay;
    if (check_sizes(B, T, Hk, H, N, has_cu_seqlens != 0, &z) != KDA_OK ||
        !make_layout(z, true, need_ddecay != 0, &lay))
        return 0;
    return lay.total;
}

kda_status kda_lin_bwd(const void *q, const void *k, const void *v, const float *decay, int decay_per_token,
                       float scale, const void *initial_state, kda_state_dtype initial_state_dtype, const void *dout,
                       const float *dfinal_state, void *dq, void *dk, void *dv, float *ddecay,
                       float *dinitial_state, const int64_t *cu_seqlens, const int64_t *cu_seqlens_host, int64_t B,
                       int64_t T, int64_t Hk, int64_t H, int64_t N, int64_t K, int64_t V,
                       const int64_t *strides_host, void *workspace, size_t workspace_bytes, void *stream)
{
    if ((!decay && !(decay_per_token && T == 0)) || (T != 0 && (!q || !k || !v || !dout || !dq || !dk || !dv)))
        return KDA_ERR_NULL;
    Sizes z;
    kda_status st = check_sizes(B, T, Hk, H, N, cu_seqlens != nullptr, &z);
    if (st != KDA_OK)
        return st;
    if (K != kD || V != kD)
        return KDA_ERR_HEAD_DIM;
    if (!dtype_ok(initial_state_dtype) || (initial_state == nullptr) != (initial_state_dtype == KDA_STATE_NONE))
        return KDA_ERR_DTYPE;
    if (decay_per_token != 0 && decay_per_token != 1)
        return KDA_ERR_FLAGS;
    if (!isfinite(scale))
        return KDA_ERR_SCALE;
    kda::LinTensor tq, tk, tv, td;
    Range rq, rk, rv, rdo;
    if ((st = set_tensor(q, strides_host, z, Hk, &tq, &rq)) != KDA_OK ||
        (st = set_tensor(k, strides_host ? strides_host + 3 : nullptr, z, Hk, &tk, &rk)) != KDA_OK ||
        (st = set_tensor(v, strides_host ? strides_host + 6 : nullptr, z, H, &tv, &rv)) != KDA_OK ||
        (st = set_tensor(dout, nullptr, z, H, &td, &rdo)) != KDA_OK)
        return st;
    const void *p16[] = {dq, dk, dv, initial_state, dfinal_state, dinitial_state};
    for (const void *p : p16)
        if (!aligned(p, 16))
            return KDA_ERR_ALIGN;
    if (!aligned(decay, 4) || !aligned(ddecay, 4) || !aligned(cu_seqlens, 8) || !aligned(workspace, kda::kAlign))
        return KDA_ERR_ALIGN;
    const size_t tokens = (size_t)B * (size_t)T, states = (size_t)z.n_seq * (size_t)H;
    const size_t decay_bytes = (decay_per_token ? tokens * (size_t)H : (size_t)H) * 4;
    const Range in[] = {rq, rk, rv, rdo, range_of(decay, decay_bytes),
                        range_of(initial_state, states * state_bytes(initial_state_dtype)),
                        range_of(dfinal_state, states * kda::kLinStateBytes),
                        range_of(cu_seqlens, cu_seqlens ? (size_t)(N + 1) * 8 : 0)};
    const Range out[] = {range_of(dq, tokens * (size_t)Hk * kD * 2), range_of(dk, tokens * (size_t)Hk * kD * 2),
                         range_of(dv, tokens * (size_t)H * kD * 2), range_of(ddecay, decay_bytes),
                         range_of(dinitial_state, states * kda::kLinStateBytes),
                         range_of(workspace, workspace_bytes)};
    const int n_out = (int)(sizeof(out) / sizeof(out[0]));
    for (int i = 0; i < n_out; ++i) {
        for (const Range &x : in)
            if (overlap(out[i], x))
                return KDA_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j]))
                return KDA_ERR_ALIAS;
    }
    kda::LinLayout lay;
    if (!make_layout(z, true, ddecay != nullptr, &lay))
        return KDA_ERR_SHAPE;
    if (!workspace || workspace_bytes < lay.total)
        return KDA_ERR_WORKSPACE;
    if ((st = check_cu(cu_seqlens, cu_seqlens_host, z)) != KDA_OK)
        return st;

    unsigned char *w = static_cast<unsigned char *>(workspace);
    auto f32 = [&](size_t off) { return reinterpret_cast<float *>(w + off); };
    kda::LinArgs a;
    memset(&a, 0, sizeof(a));
    a.decay = decay;
    a.per_token = decay_per_token;
    a.scale = scale;
    a.T = T;
    a.H = H;
    a.N = z.n_seq;
    a.rows = lay.plan.rows;
    a.P = lay.plan.P;
    a.len = lay.plan.len;
    a.cu = cu_seqlens;
    a.status = reinterpret_cast<int32_t *>(w);
    const bool shared = Hk != H;
    kda::LinRole &rdq = a.role[0], &rdk = a.role[1], &rdv = a.role[2];
    rdq.q = td;
    rdq.k = tv;
    rdq.v = tk;
    rdq.transposed = 1;
    rdq.init = initial_state;
    rdq.init_dt = (int)initial_state_dtype;
    rdk.q = tv;
    rdk.k = td;
    rdk.v = tq;
    rdk.rev = 1;
    rdk.transposed = 1;
    rdv.q = tk;
    rdv.k = tq;
    rdv.v = td;
    rdv.rev = 1;
    rdk.init = rdv.init = dfinal_state;
    rdk.init_dt = rdv.init_dt = (int)(dfinal_state ? KDA_STATE_FP32 : KDA_STATE_NONE);
    rdv.fin = dinitial_state;
    rdv.fin_dt = (int)KDA_STATE_FP32;
    if (a.P > 1) {
        rdq.slots = f32(lay.off_fwd);
        rdq.lam = f32(lay.off_flam);
        rdk.slots = rdv.slots = f32(lay.off_rev);
        rdk.lam = rdv.lam = f32(lay.off_rlam);
    }
    rdq.out = shared ? static_cast<void *>(f32(lay.off_dq)) : dq;
    rdk.out = shared ? static_cast<void *>(f32(lay.off_dk)) : dk;
    rdq.out_f32 = rdk.out_f32 = shared ? 1 : 0;
    rdv.out = dv;
    if (ddecay) {
        rdq.x = tq;
        rdq.dots = f32(lay.off_qd);
        rdk.x = tk;
        rdk.dots = f32(lay.off_kd);
        if (dfinal_state) {
            rdq.xst = dfinal_state;
            rdq.xfin = f32(lay.off_xfin);
        }
    }
    kda::LinBwdExtra e;
    memset(&e, 0, sizeof(e));
    e.Hk = Hk;
    e.dq = static_cast<uint16_t *>(dq);
    e.dk = static_cast<uint16_t *>(dk);
    if (shared) {
        e.dq_h = f32(lay.off_dq);
        e.dk_h = f32(lay.off_dk);
    }
    e.ddecay = ddecay;
    if (ddecay)
        e.part = reinterpret_cast<double *>(w + lay.off_part);
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (cu_seqlens && kda::lin_launch_check(cu_seqlens, a.N, T, a.status, s) != hipSuccess)
        return KDA_ERR_HIP;
    const int lead[2] = {0, 2};
    if (kda::lin_launch_walk(a, 3, lead, 2, s) != hipSuccess || kda::lin_launch_grad_tail(a, e, s) != hipSuccess)
        return KDA_ERR_HIP;
    return KDA_OK;
}

}  // extern "C"
