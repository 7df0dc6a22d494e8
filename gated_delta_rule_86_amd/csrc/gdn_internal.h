// gdn_internal.h -- shared by the host side (gdn_api.cpp) and the gfx950 kernels (gdn.hip) of the gated delta
// rule.  Not part of the public ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

#include "kda_internal.h"

namespace kda {

constexpr int kGC = 32;                    // tokens per chunk
constexpr int kGB = 64;                    // tokens per block of the backward pass: one state is kept for two chunks
constexpr int64_t kGdnSlots = 512;         // workgroups of a walk that run at once: two on each of 256 CUs
constexpr size_t kGdnStateBytes = (size_t)kD * kD * sizeof(float);
constexpr int64_t kGdnMaxCuts = 1024;      // segments of a row, at most
constexpr int64_t kGdnMinSeg = 256;        // shortest segment that a cut leaves, in tokens

// Record of one (chunk, head) in the workspace, bytes: operands of the walks, in the order of their lanes.
//   forward:   T' | factors | A'
//   backward:  T' | factors | T^T | A^T   (A without beta)
// Each matrix is 32 x 32 in three bf16 terms.
constexpr int kGdnMat = 2 * 3 * 1024;
constexpr int kGdnVec = 1024;
constexpr int kGdnRecFwd = 2 * kGdnMat + kGdnVec;
constexpr int kGdnRecBwd = 3 * kGdnMat + kGdnVec;

// The tokens of a batch row (the one row of a packed batch) are cut into P segments of `len` tokens whatever the
// sequences in it.  A chunk belongs to the segment that holds its first token.  Where a sequence's chunks go on in the
// next segment, the state there is found before the output walk: each segment's own share F and, where it lies inside one
// sequence, its transition Phi (S_end = S_begin Phi + F), joined by a scan.
struct GdnPlan {
    int64_t rows, P, len;
};

// Time of `groups` workgroups of `chunks` chunks each, in chunks of a full chip: rounds of kGdnSlots; a workgroup alone on
// its CU takes about 0.6 of the time that two take side by side.
inline double gdn_rounds(int64_t groups, double chunks)
{
    const double round = (double)cdiv(groups, kGdnSlots) * chunks;
    return groups <= kGdnSlots / 2 ? 0.6 * round : round;
}

// The cut that takes the least time: the walks, and with a cut the shares and transitions of all but the last segment, the
// scans' steps and more launches.
inline GdnPlan gdn_plan(int64_t B, int64_t T, int64_t H, bool varlen, bool bwd)
{
    GdnPlan p;
    p.rows = varlen ? 1 : B;
    p.P = 1;
    p.len = T > 0 ? cdiv(T, kGB) * kGB : kGB;
    const int64_t chains = p.rows * H;
    int64_t most = T / kGdnMinSeg;
    if (most > 2 * kGdnSlots / chains)
        most = 2 * kGdnSlots / chains;  // at most kGdnMaxCuts
    double best = 0.0;
    for (int64_t P = 1; P <= (most > 1 ? most : 1); ++P) {
        const int64_t len = T > 0 ? cdiv(cdiv(T, P), kGB) * kGB : kGB, got = T > 0 ? cdiv(T, len) : 1;
        const double n = (double)(len / kGC) + 2.0;
        double cost = gdn_rounds(chains * got, bwd ? 1.7 * n : n);
        if (got > 1)
            cost += gdn_rounds(2 * chains * (got - 1), 0.65 * n) + (bwd ? gdn_rounds(chains * (got - 1), 1.0 * n) : 0.0) +
                    (bwd ? 2.0 : 1.0) * (0.3 * (double)got + 2.0);
        if (P == 1 || cost < best) {
            best = cost;
            p.P = got;
            p.len = len;
        }
    }
    return p;
}

struct GdnTensor {  // bf16 [B, T, heads, 128] with element strides; head h of the pass reads head h / share
    const uint16_t *p;
    int64_t sb, st, sh;
    int64_t share;
};

struct GdnArgs {
    GdnTensor q, k, v, dout;
    const float *decay, *beta;   // [B, T, H]
    float scale;
    int64_t T, H, N;             // N: sequences
    int64_t rows, P, len;
    const int64_t *cu;           // NULL: every row is one sequence
    const int32_t *status;       // device status word (NULL without cu)
    uint16_t *out;
    const void *init;
    void *fin;
    int init_dt, fin_dt;
    unsigned char *rec;          // [slots][H] records
    int64_t slots, blocks, rec_bytes;
    float *seg;                  // [rows * P][H]: state at a segment's start, of the sequence that crosses it
    float *phi;                  // [rows * P][H]
    int32_t *dead;               // [rows * P][H]: the transition counts as 0 (and is not formed)
    float *norm;                 // [slots][H]: log2 of a bound of each chunk's transition; NULL without cuts
    float *keep;                 // [rows * P][H]: initial state of the sequence that leaves the segment (in place), or NULL
    // backward pass
    int64_t Hk;
    const float *dfin;           // dL/dfinal_state or NULL
    float *dinit;                // dL/dinitial_state or NULL
    float *dseg;                 // [rows * P][H]: dL/dS at a segment's end, of the sequence that goes on behind it
    float *before, *dafter;      // [blocks][H] states before each block, dL/dS after it
    float *res, *dwrite;         // [slots][H][32][128]: residuals r_t, and dL/d(beta r)_t
    uint16_t *dq, *dk, *dv;
    float *dq_h, *dk_h;          // fp32 [B, T, H, 128] when q/k heads are shared, else NULL
    float *ddecay, *dbeta;
};

struct GdnLayout {
    GdnPlan plan;
    int64_t slots, blocks;
    size_t off_rec, off_seg, off_phi, off_keep, off_dead, off_norm;
    size_t off_dseg, off_before, off_dafter, off_res, off_dwrite, off_dq, off_dk;
    size_t total;
};

hipError_t gdn_launch_fwd(const GdnArgs &a, int32_t *status, hipStream_t s);
hipError_t gdn_launch_bwd(const GdnArgs &a, int32_t *status, hipStream_t s);
hipError_t gdn_launch_recurrent(const GdnArgs &a, int32_t *status, hipStream_t s);

}  // namespace kda
