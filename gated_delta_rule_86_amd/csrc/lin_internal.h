// lin_internal.h -- shared by the host side (lin_api.cpp) and the gfx950 kernels
// (lin_attn.hip) of the decayed linear attention.  Not part of the public ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

#include "kda_internal.h"

namespace kda {

constexpr int kLC = 64;                       // tokens per chunk
constexpr int64_t kLinSlots = 512;            // workgroups that run at once: two on each of 256 CUs
constexpr int64_t kLinMinSeg = 256;           // shortest segment that a cut leaves, in tokens
// Longest segment when the decay's gradient is wanted: it sums rounding errors from the segment's end on.  B = 2,
// T = 4096, H = 16 against 64 bits: 1.5e-6 with 832 tokens (202 us), 1.2e-6 with 512 (201 us), 0.9e-6 with 256
// (231 us).
constexpr int64_t kLinGradSeg = 512;
constexpr size_t kLinStateBytes = (size_t)kD * kD * sizeof(float);

// Segments.  The packed tokens of a batch row (the one row of a varlen batch) are cut into P
// segments of `len` tokens whatever the sequences in it, so workgroups get equal work and
// no table is needed.  A sequence that crosses a segment boundary has its state there in
// slot [segment][head] of the workspace: the states pass forms each segment's own share, the
// scan joins them, and the output pass starts from them.
struct LinPlan {
    int64_t rows;      // batch rows (1 for varlen)
    int64_t P;         // segments per row
    int64_t len;       // tokens per segment, a multiple of kLC
    int64_t n_seq;     // N, or B without cu_seqlens
};

// Time of `groups` workgroups of `chunks` chunks each, in chunks of a full chip: rounds of kLinSlots, each with
// `fixed` for its state and first loads; at most one workgroup on a CU runs its chunks in about 0.6 of the time that
// two take side by side (T = 262144, H = 8: 815 us with 256 workgroups, 700 us with 512, when it was chosen).
inline double lin_rounds(int64_t groups, int64_t chunks, double fixed)
{
    const double round = (double)cdiv(groups, kLinSlots) * ((double)chunks + fixed);
    return groups <= kLinSlots / 2 ? 0.6 * round : round;
}

// walks: how many share the segments (1 forward; 3 backward, two of which need states).  The cut that takes the least
// time: the walks, the states pass (reads two of three inputs), the scan (128 KiB per slot at 5 TB/s against 9.6 us
// for a chunk of the full chip) and two more launches.  B = 2, T = 4096, H = 16: forward 98 us with P = 16, 89 us with
// P = 8, when it was chosen (86 by now).
inline LinPlan lin_plan(int64_t B, int64_t T, int64_t H, int64_t N, bool varlen, int64_t walks, int64_t max_len)
{
    LinPlan p;
    p.rows = varlen ? 1 : B;
    p.n_seq = varlen ? N : B;
    const int64_t chains = p.rows * H, leads = walks > 1 ? 2 : 1;
    const int64_t least = max_len > 0 ? cdiv(T, max_len) : 1;
    int64_t most = T / kLinMinSeg;
    if (most > cdiv(4 * kLinSlots, chains))
        most = cdiv(4 * kLinSlots, chains);
    if (most < least)
        most = least;
    if (most < 1)
        most = 1;
    double best = 0.0;
    p.P = 0;
    for (int64_t P = least < 1 ? 1 : least; P <= most; ++P) {
        int64_t len = cdiv(cdiv(T, P), kLC) * kLC;
        if (len < kLC)
            len = kLC;
        const int64_t got = T > 0 ? cdiv(T, len) : 1, chunks = len / kLC;
        double cost = lin_rounds(walks * chains * got, chunks, 2.5);
        if (got > 1)
            cost += 0.45 * lin_rounds(leads * chains * got, chunks, 1.5) + 0.0027 * (double)(leads * chains * got) + 0.4;
        if (p.P == 0 || cost < best) {
            best = cost;
            p.P = got;
            p.len = len;
        }
    }
    return p;
}

struct LinLayout {
    LinPlan plan;
    size_t off_fwd, off_flam;  // slots of the state and their decay factors [rows * P][H]
    size_t off_rev, off_rlam;  // slots of the state's gradient (backward pass)
    size_t off_dq, off_dk;     // fp32 per value head [B, T, H, 128], when q/k heads are shared
    size_t off_qd, off_kd;     // fp32 [B, T, H]: q.dq and k.dk, when the decay's gradient is wanted
    size_t off_xfin;           // fp32 [n_seq][H]: <S_final, dL/dS_final>
    size_t off_part;           // double [rows * P][H]: partial sums of a per-head decay's gradient
    size_t total;
};

struct LinTensor {  // bf16 [B, T, heads, 128] with element strides; head h of the pass reads head h / share
    const uint16_t *p;
    int64_t sb, st, sh;
    int64_t share;
};

// One walk over all tokens: out_t = sum over sources s of w(t, s) (q_t . k_s) v_s, with the
// sources at or before t, or (rev) at or behind it.
struct LinRole {
    LinTensor q, k, v;
    int rev;          // sources behind the token; the state runs from the end to the start
    int transposed;   // the state's [V][K] matrix is held as [k of the role][v of the role]
    const void *init; // [n_seq][H][128][128] or NULL
    void *fin;        // state after the last step, or NULL
    int init_dt, fin_dt;
    float *slots;     // [rows * P][H][128][128]
    float *lam;       // [rows * P][H]
    int defer;        // fin is init and P > 1: see lin_final_kernel
    void *out;        // [B, T, H, 128], bf16 or fp32 (out_f32), or NULL
    int out_f32;
    LinTensor x;      // dots[b, t, h] = out row . x row (x.p NULL: not wanted)
    float *dots;
    const float *xst; // fp32 [n_seq][H][128][128]: xfin = <final state, xst>
    float *xfin;
};

struct LinArgs {
    LinRole role[3];
    const float *decay;  // natural-log decay
    int per_token;       // decay [B, T, H], else [H]
    float scale;
    int64_t T, H, N;     // N = n_seq
    int64_t rows, P, len;
    int turns;           // walks on one CU keep close to each other
    const int64_t *cu;   // NULL: every row is one sequence
    int32_t *status;     // device status word (NULL without cu)
};

struct LinBwdExtra {
    int64_t Hk;
    uint16_t *dq, *dk;        // bf16 [B, T, Hk, 128]
    const float *dq_h, *dk_h; // fp32 per value head, or NULL when heads are not shared
    float *ddecay;            // NULL: not wanted
    double *part;
};

hipError_t lin_launch_check(const int64_t *cu, int64_t N, int64_t T, int32_t *status, hipStream_t s);
// n_roles walks in one launch; with P > 1 the states pass and the scan run first, for the
// roles that `lead` lists (roles that share slots need them once).
hipError_t lin_launch_walk(const LinArgs &a, int n_roles, const int *lead, int n_lead, hipStream_t s);
hipError_t lin_launch_grad_tail(const LinArgs &a, const LinBwdExtra &e, hipStream_t s);
hipError_t lin_launch_recurrent(const LinArgs &a, hipStream_t s);

}  // namespace kda
