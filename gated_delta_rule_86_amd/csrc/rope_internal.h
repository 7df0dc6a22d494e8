// rope_internal.h -- shared by the host side (rope_api.cpp) and the gfx950 kernels
// (qk_rope.hip) of the q/k normalisation and position rotation.  Not part of the public ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

namespace kda {

constexpr int kRopeMaxD = 512;          // largest head size
constexpr int kRopeThreads = 256;
constexpr int64_t kRopeGroups = 1024;   // most workgroups of the backward pass, one row of partial weight sums each

struct RopeView {  // [B, T, heads, D], element strides
    unsigned char *p;
    int64_t sb, st, sh;
};

struct RopeArgs {
    RopeView x[2];   // q, k
    RopeView dy[2];  // gradients of the outputs (backward pass)
    RopeView y[2];   // outputs, or gradients of the inputs
    const float *w[2];  // [D] or NULL
    const float *inv_freq;
    const int64_t *positions;  // [B, T] or NULL: the token's index in its row
    int64_t B, T;
    int heads[2];
    int D, R;
    int dtype;   // 1 bf16, 2 fp32, 3 fp16
    int norm;    // 0 none, 1 rms, 2 l2
    int interleaved;
    float eps, factor;
    int tokens;      // per workgroup (forward pass)
    int step[2];     // tokens per step, and workgroups, of q and k (backward pass)
    int groups[2];
    float *part;     // [groups[0] + groups[1]][D] partial weight sums (backward pass)
    float *dw[2];
};

// sets step and groups from B, T, heads, D and R
void rope_plan_bwd(RopeArgs *a);
hipError_t rope_launch(const RopeArgs &a, hipStream_t s);
hipError_t rope_launch_bwd(const RopeArgs &a, hipStream_t s);

}  // namespace kda
