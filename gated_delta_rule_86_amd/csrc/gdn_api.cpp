// gdn_api.cpp -- host side of the gated delta rule (kda_gdn_* in include/kda.h): argument checks, workspace layout,
// launches.  The checks are plain host code that touches no HIP API, so every error path can be exercised without a GPU.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <hip/hip_runtime.h>

#include "gdn_internal.h"
#include "host_checks.h"
#include "kda.h"

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
    // a launch holds less than 2^32 threads: 256 for each of these
    return z->n_seq > (((int64_t)1 << 24) - 8) / H ? KDA_ERR_SHAPE : KDA_OK;
}

bool make_layout(const Sizes &z, bool bwd, kda::GdnLayout *L)
{
    using kda::kAlign;
    L->plan = kda::gdn_plan(z.B, z.T, z.H, z.varlen, bwd);
    const kda::GdnPlan &p = L->plan;
    L->slots = z.B * z.T / kda::kGC + z.n_seq + 1;
    L->blocks = z.B * z.T / kda::kGB + z.n_seq + 1;
    // 64 threads for each record, at most 512 for each block, 256 for each segment and head, 4096 for each row and head
    if (L->slots > (((int64_t)1 << 26) - 8) / z.H || (bwd && L->blocks > (((int64_t)1 << 23) - 8) / z.H) ||
        p.rows * p.P > (((int64_t)1 << 24) - 8) / z.H || (p.P > 1 && p.rows >= ((int64_t)1 << 20) / z.H))
        return false;
    size_t off = kAlign;  // status word
    auto take = [&](size_t bytes) {
        const size_t o = off;
        off = (off + bytes + kAlign - 1) / kAlign * kAlign;
        return o;
    };
    L->off_rec = L->off_seg = L->off_phi = L->off_keep = L->off_dseg = L->off_dead = L->off_norm = 0;
    L->off_before = L->off_dafter = L->off_res = L->off_dwrite = L->off_dq = L->off_dk = 0;
    const size_t recs = z.T > 0 ? (size_t)L->slots * (size_t)z.H : 0, blocks = z.T > 0 ? (size_t)L->blocks * (size_t)z.H : 0;
    L->off_rec = take(recs * (bwd ? kda::kGdnRecBwd : kda::kGdnRecFwd));
    if (p.P > 1) {
        const size_t segs = (size_t)p.rows * (size_t)p.P * (size_t)z.H * kda::kGdnStateBytes;
        L->off_seg = take(segs);
        L->off_phi = take(segs);
        (bwd ? L->off_dseg : L->off_keep) = take(segs);
        L->off_dead = take((size_t)p.rows * (size_t)p.P * (size_t)z.H * sizeof(int32_t));
        L->off_norm = take(recs * sizeof(float));
    }
    if (bwd) {
        L->off_before = take(blocks * kda::kGdnStateBytes);
        L->off_dafter = take(blocks * kda::kGdnStateBytes);
        L->off_res = take(recs * kda::kGC * kD * sizeof(float));
        L->off_dwrite = take(recs * kda::kGC * kD * sizeof(float));
        if (z.Hk != z.H) {
            const size_t rows = (size_t)z.B * (size_t)z.T * (size_t)z.H * kD * sizeof(float);
            L->off_dq = take(rows);
            L->off_dk = take(rows);
        }
    }
    L->total = off;
    return true;
}

// Everything that the forward entry points check; fills the kernels' arguments.
kda_status forward_args(const void *q, const void *k, const void *v, const float *decay, const float *beta, float scale,
                        void *out, const void *h0, kda_state_dtype h0_dt, void *ht, kda_state_dtype ht_dt,
                        const int64_t *cu, const int64_t *cu_host, int64_t B, int64_t T, int64_t Hk, int64_t H,
                        int64_t N, int64_t K, int64_t V, const int64_t *strides, void *ws, size_t ws_bytes,
                        bool recurrent, kda::GdnArgs *a)
{
    if (T != 0 && (!q || !k || !v || !decay || !beta || !out))
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
    if (!isfinite(scale))
        return KDA_ERR_SCALE;
    kda::GdnLayout lay;
    if (!recurrent && !make_layout(z, false, &lay))
        return KDA_ERR_SHAPE;
    memset(a, 0, sizeof(*a));
    Range rq, rk, rv;
    if ((st = set_tensor(q, strides, z, Hk, &a->q, &rq)) != KDA_OK ||
        (st = set_tensor(k, strides ? strides + 3 : nullptr, z, Hk, &a->k, &rk)) != KDA_OK ||
        (st = set_tensor(v, strides ? strides + 6 : nullptr, z, H, &a->v, &rv)) != KDA_OK)
        return st;
    if (!aligned(out, 16) || !aligned(decay, 4) || !aligned(beta, 4) || !aligned(h0, 16) || !aligned(ht, 16) ||
        !aligned(cu, 8) || !aligned(ws, kda::kAlign))
        return KDA_ERR_ALIGN;
    const size_t rows = (size_t)B * (size_t)T * (size_t)H, states = (size_t)z.n_seq * (size_t)H;
    const Range ro = range_of(out, rows * kD * 2), ri = range_of(h0, states * state_bytes(h0_dt)),
                rf = range_of(ht, states * state_bytes(ht_dt)), rw = range_of(ws, ws_bytes);
    const Range in[] = {rq, rk, rv, range_of(decay, rows * 4), range_of(beta, rows * 4),
                        range_of(cu, cu ? (size_t)(N + 1) * 8 : 0)};
    for (const Range &x : in)
        if (overlap(ro, x) || overlap(rf, x) || overlap(rw, x))
            return KDA_ERR_ALIAS;
    if (overlap(ro, ri) || overlap(ro, rf) || (h0 != ht && overlap(ri, rf)) || overlap(rw, ri) || overlap(rw, ro) ||
        overlap(rw, rf))
        return KDA_ERR_ALIAS;
    // token by token, the workspace holds the status word alone
    const size_t need = recurrent ? (cu ? kda::kAlign : 0) : lay.total;
    if (need && (!ws || ws_bytes < need))
        return KDA_ERR_WORKSPACE;
    if ((st = check_cu(cu, cu_host, z)) != KDA_OK)
        return st;
    a->decay = decay;
    a->beta = beta;
    a->scale = scale;
    a->T = T;
    a->H = H;
    a->N = z.n_seq;
    a->cu = cu;
    unsigned char *w = static_cast<unsigned char *>(ws);
    a->status = cu ? reinterpret_cast<int32_t *>(w) : nullptr;
    a->out = static_cast<uint16_t *>(out);
    a->init = h0;
    a->fin = ht;
    a->init_dt = (int)h0_dt;
    a->fin_dt = (int)ht_dt;
    if (!recurrent) {
        a->rows = lay.plan.rows;
        a->P = lay.plan.P;
        a->len = lay.plan.len;
        a->slots = lay.slots;
        a->blocks = lay.blocks;
        a->rec = w + lay.off_rec;
        a->rec_bytes = kda::kGdnRecFwd;
        if (a->P > 1) {
            a->seg = reinterpret_cast<float *>(w + lay.off_seg);
            a->phi = reinterpret_cast<float *>(w + lay.off_phi);
            a->dead = reinterpret_cast<int32_t *>(w + lay.off_dead);
            a->norm = reinterpret_cast<float *>(w + lay.off_norm);
            if (ht && ht == h0)
                a->keep = reinterpret_cast<float *>(w + lay.off_keep);
        }
    }
    return KDA_OK;
}

}  // namespace

extern "C" {

size_t kda_gdn_fwd_workspace_size(int64_t B, int64_t T, int64_t H, int64_t N, int has_cu_seqlens)
{
    Sizes z;
    kda::GdnLayout lay;
    if (check_sizes(B, T, H, H, N, has_cu_seqlens != 0, &z) != KDA_OK || !make_layout(z, false, &lay))
        return 0;
    return lay.total;
}

kda_status kda_gdn_fwd(const void *q, const void *k, const void *v, const float *decay, const float *beta, float scale,
                       void *out, const void *initial_state, kda_state_dtype initial_state_dtype, void *final_state,
                       kda_state_dtype final_state_dtype, const int64_t *cu_seqlens, const int64_t *cu_seqlens_host,
                       int64_t B, int64_t T, int64_t Hk, int64_t H, int64_t N, int64_t K, int64_t V,
                       const int64_t *strides_host, void *workspace, size_t workspace_bytes, void *stream)
{
    kda::GdnArgs a;
    const kda_status st =
        forward_args(q, k, v, decay, beta, scale, out, initial_state, initial_state_dtype, final_state, final_state_dtype,
                     cu_seqlens, cu_seqlens_host, B, T, Hk, H, N, K, V, strides_host, workspace, workspace_bytes, false, &a);
    if (st != KDA_OK)
        return st;
    return kda::gdn_launch_fwd(a, static_cast<int32_t *>(workspace), static_cast<hipStream_t>(stream)) == hipSuccess
               ? KDA_OK
               : KDA_ERR_HIP;
}

kda_status kda_gdn_fwd_recurrent(const void *q, const void *k, const void *v, const float *decay, const float *beta,
                                 float scale, void *out, const void *initial_state, kda_state_dtype initial_state_dtype,
                                 void *final_state, kda_state_dtype final_state_dtype, const int64_t *cu_seqlens,
                                 const int64_t *cu_seqlens_host, int64_t B, int64_t T, int64_t Hk, int64_t H, int64_t N,
                                 int64_t K, int64_t V, const int64_t *strides_host, void *workspace,
                                 size_t workspace_bytes, void *stream)
{
    kda::GdnArgs a;
    const kda_status st =
        forward_args(q, k, v, decay, beta, scale, out, initial_state, initial_state_dtype, final_state, final_state_dtype,
                     cu_seqlens, cu_seqlens_host, B, T, Hk, H, N, K, V, strides_host, workspace, workspace_bytes, true, &a);
    if (st != KDA_OK)
        return st;
    return kda::gdn_launch_recurrent(a, static_cast<int32_t *>(workspace), static_cast<hipStream_t>(stream)) == hipSuccess
               ? KDA_OK
               : KDA_ERR_HIP;
}

size_t kda_gdn_bwd_workspace_size(int64_t B, int64_t T, int64_t Hk, int64_t H, int64_t N, int has_cu_seqlens)
{
    Sizes z;
    kda::GdnLayout lay;
    if (check_sizes(B, T, Hk, H, N, has_cu_seqlens != 0, &z) != KDA_OK || !make_layout(z, true, &lay))
        return 0;
    return lay.total;
}

kda_status kda_gdn_bwd(const void *q, const void *k, const void *v, const float *decay, const float *beta, float scale,
                       const void *initial_state, kda_state_dtype initial_state_dtype, const void *dout,
                       const float *dfinal_state, void *dq, void *dk, void *dv, float *ddecay, float *dbeta,
                       float *dinitial_state, const int64_t *cu_seqlens, const int64_t *cu_seqlens_host, int64_t B,
                       int64_t T, int64_t Hk, int64_t H, int64_t N, int64_t K, int64_t V, const int64_t *strides_host,
                       void *workspace, size_t workspace_bytes, void *stream)
{
    if (T != 0 && (!q || !k || !v || !decay || !beta || !dout || !dq || !dk || !dv || !ddecay || !dbeta))
        return KDA_ERR_NULL;
    Sizes z;
    kda_status st = check_sizes(B, T, Hk, H, N, cu_seqlens != nullptr, &z);
    if (st != KDA_OK)
        return st;
    if (K != kD || V != kD)
        return KDA_ERR_HEAD_DIM;
    if (!dtype_ok(initial_state_dtype) || (initial_state == nullptr) != (initial_state_dtype == KDA_STATE_NONE))
        return KDA_ERR_DTYPE;
    if (!isfinite(scale))
        return KDA_ERR_SCALE;
    kda::GdnLayout lay;
    if (!make_layout(z, true, &lay))
        return KDA_ERR_SHAPE;
    kda::GdnArgs a;
    memset(&a, 0, sizeof(a));
    Range rq, rk, rv, rdo;
    if ((st = set_tensor(q, strides_host, z, Hk, &a.q, &rq)) != KDA_OK ||
        (st = set_tensor(k, strides_host ? strides_host + 3 : nullptr, z, Hk, &a.k, &rk)) != KDA_OK ||
        (st = set_tensor(v, strides_host ? strides_host + 6 : nullptr, z, H, &a.v, &rv)) != KDA_OK ||
        (st = set_tensor(dout, nullptr, z, H, &a.dout, &rdo)) != KDA_OK)
        return st;
    const void *p16[] = {dq, dk, dv, initial_state, dfinal_state, dinitial_state};
    for (const void *p : p16)
        if (!aligned(p, 16))
            return KDA_ERR_ALIGN;
    const void *p4[] = {decay, beta, ddecay, dbeta};
    for (const void *p : p4)
        if (!aligned(p, 4))
            return KDA_ERR_ALIGN;
    if (!aligned(cu_seqlens, 8) || !aligned(workspace, kda::kAlign))
        return KDA_ERR_ALIGN;
    const size_t tokens = (size_t)B * (size_t)T, states = (size_t)z.n_seq * (size_t)H, gates = tokens * (size_t)H * 4;
    const Range in[] = {rq, rk, rv, rdo, range_of(decay, gates), range_of(beta, gates),
                        range_of(initial_state, states * state_bytes(initial_state_dtype)),
                        range_of(dfinal_state, states * kda::kGdnStateBytes),
                        range_of(cu_seqlens, cu_seqlens ? (size_t)(N + 1) * 8 : 0)};
    const Range out[] = {range_of(dq, tokens * (size_t)Hk * kD * 2), range_of(dk, tokens * (size_t)Hk * kD * 2),
                         range_of(dv, tokens * (size_t)H * kD * 2), range_of(ddecay, gates), range_of(dbeta, gates),
                         range_of(dinitial_state, states * kda::kGdnStateBytes), range_of(workspace, workspace_bytes)};
    const int n_out = (int)(sizeof(out) / sizeof(out[0]));
    for (int i = 0; i < n_out; ++i) {
        for (const Range &x : in)
            if (overlap(out[i], x))
                return KDA_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j]))
                return KDA_ERR_ALIAS;
    }
    if (!workspace || workspace_bytes < lay.total)
        return KDA_ERR_WORKSPACE;
    if ((st = check_cu(cu_seqlens, cu_seqlens_host, z)) != KDA_OK)
        return st;
    unsigned char *w = static_cast<unsigned char *>(workspace);
    auto f32 = [&](size_t off) { return reinterpret_cast<float *>(w + off); };
    a.decay = decay;
    a.beta = beta;
    a.scale = scale;
    a.T = T;
    a.H = H;
    a.Hk = Hk;
    a.N = z.n_seq;
    a.rows = lay.plan.rows;
    a.P = lay.plan.P;
    a.len = lay.plan.len;
    a.cu = cu_seqlens;
    a.status = cu_seqlens ? reinterpret_cast<int32_t *>(w) : nullptr;
    a.init = initial_state;
    a.init_dt = (int)initial_state_dtype;
    a.rec = w + lay.off_rec;
    a.rec_bytes = kda::kGdnRecBwd;
    a.slots = lay.slots;
    a.blocks = lay.blocks;
    if (a.P > 1) {
        a.seg = f32(lay.off_seg);
        a.phi = f32(lay.off_phi);
        a.dead = reinterpret_cast<int32_t *>(w + lay.off_dead);
        a.norm = f32(lay.off_norm);
        a.dseg = f32(lay.off_dseg);
    }
    a.dfin = dfinal_state;
    a.dinit = dinitial_state;
    a.before = f32(lay.off_before);
    a.dafter = f32(lay.off_dafter);
    a.res = f32(lay.off_res);
    a.dwrite = f32(lay.off_dwrite);
    a.dq = static_cast<uint16_t *>(dq);
    a.dk = static_cast<uint16_t *>(dk);
    a.dv = static_cast<uint16_t *>(dv);
    if (Hk != H) {
        a.dq_h = f32(lay.off_dq);
        a.dk_h = f32(lay.off_dk);
    }
    a.ddecay = ddecay;
    a.dbeta = dbeta;
    return kda::gdn_launch_bwd(a, static_cast<int32_t *>(workspace), static_cast<hipStream_t>(stream)) == hipSuccess
               ? KDA_OK
               : KDA_ERR_HIP;
}

}  // extern "C"
