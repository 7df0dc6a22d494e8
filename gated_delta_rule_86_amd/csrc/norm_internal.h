// norm_internal.h -- shared by the host side (norm_api.cpp) and the gfx950 kernels (block_norm.hip) of the norms around a
// block.  Not part of the public ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

namespace kda {

constexpr int kGatedMaxD = 512;       // one wave at most holds a row
constexpr int kResidualMaxD = 8192;   // one workgroup of 512 threads, 16 channels each
constexpr int kNormGroups = 1024;     // most workgroups of a backward pass: partial weight sums of each

struct NormView {  // [B, T, H, D], strides in elements; flat: row r begins at r * sh
    unsigned char *p;
    int64_t sb, st, sh;
    int flat;
};

struct NormArgs {
    NormView x, z;            // gated: x and the gate; residual: x and the residual (backward: the stored stream)
    const unsigned char *dy;  // contiguous gradients of the outputs
    const unsigned char *dz;  // of residual_out, or NULL
    unsigned char *y, *zo;    // contiguous outputs: out (dx), residual_out (dgate, dresidual)
    const float *w, *post, *scale;  // [D] or NULL
    float *part;              // [3][groups][D]: partial sums of the gradients of w, post and scale
    float *dw, *dpost, *dscale;
    int64_t T;
    int rows, H, D;
    int dtype, rdtype;        // 1 bf16, 2 fp32, 3 fp16
    int act;                  // 0 sigmoid, 1 silu
    int post_norm;
    float eps;
    double inv_h, inv_t;
    int groups;               // workgroups (backward)
};

// workgroups of a backward pass
int gated_groups(int64_t rows, int D, int dtype);
int residual_groups(int64_t rows, int D);
hipError_t gated_launch(const NormArgs &a, hipStream_t s);
hipError_t gated_launch_bwd(const NormArgs &a, hipStream_t s);
hipError_t residual_launch(const NormArgs &a, hipStream_t s);
hipError_t residual_launch_bwd(const NormArgs &a, hipStream_t s);

}  // namespace kda
