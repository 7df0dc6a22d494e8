// qk_rope.hip -- normalisation of queries and keys for each head with the position rotation in the same
// pass, and its backward pass, gfx950.
//
// Per token and head, x [D]:
//   r = (mean x^2 + eps)^-1/2 (rms), (sum x^2 + eps)^-1/2 (l2) or 1;   n = x r w   (w [D] or 1),
//   pairs of the first R channels: (a, b) -> m (a cos t - b sin t, a sin t + b cos t),
//   t = position * inv_freq[pair]; the channels from R on pass as n.
// Pairs are (i, i + R/2), or (2i, 2i + 1) when interleaved.  Backward, with dn the rotation of
// dy by -t (times m):
//   dw = sum over tokens and heads of dn x r,
//   dx = r w dn - x r^3 / D' sum(w dn x),   D' = D (rms), 1 (l2); dx = w dn without a norm.
//
// Angles: position * inv_freq / 2 pi in fp64, reduced to within 1/8 of a turn, then fp32 Taylor
// polynomials (next terms below 2^-28): a far position costs no accuracy.  They are formed once
// per token and shared by its heads through LDS.
//
// Bound by memory: every value is read once and written once (backward: read twice as many).
// A lane owns 16 channels of a row as two 16-byte pieces (four in fp32) that hold both
// halves of its pairs, D / 16 lanes (rounded up to a power of two) own the row.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "rope_internal.h"

namespace kda {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kBf16 = 1, kFp32 = 2, kFp16 = 3;

// 8 values from memory and back (one 16-byte piece, two in fp32); rounded once, to nearest even
template <int kT>
__device__ __forceinline__ void load8(const unsigned char *p, float *x)
{
    if constexpr (kT == kFp32) {
        const f32x4 a = reinterpret_cast<const f32x4 *>(p)[0], b = reinterpret_cast<const f32x4 *>(p)[1];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[e] = a[e];
            x[4 + e] = b[e];
        }
    } else {
        const u32x4 u = *reinterpret_cast<const u32x4 *>(p);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (kT == kBf16) {
                x[2 * e] = __uint_as_float(u[e] << 16);
                x[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
            } else {
                x[2 * e] = (float)__builtin_bit_cast(_Float16, (uint16_t)(u[e] & 0xffffu));
                x[2 * e + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(u[e] >> 16));
            }
        }
    }
}
template <int kT>
__device__ __forceinline__ void store8(unsigned char *p, const float *x)
{
    if constexpr (kT == kFp32) {
        reinterpret_cast<f32x4 *>(p)[0] = f32x4{x[0], x[1], x[2], x[3]};
        reinterpret_cast<f32x4 *>(p)[1] = f32x4{x[4], x[5], x[6], x[7]};
    } else {
        u32x4 u;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            uint16_t a, b;
            if constexpr (kT == kBf16) {
                a = __builtin_bit_cast(uint16_t, (__bf16)x[2 * e]);
                b = __builtin_bit_cast(uint16_t, (__bf16)x[2 * e + 1]);
            } else {
                a = __builtin_bit_cast(uint16_t, (_Float16)x[2 * e]);
                b = __builtin_bit_cast(uint16_t, (_Float16)x[2 * e + 1]);
            }
            u[e] = (uint32_t)a | ((uint32_t)b << 16);
        }
        *reinterpret_cast<u32x4 *>(p) = u;
    }
}

// cos and sin of position * f
__device__ __forceinline__ void turn(int64_t position, float f, float *c, float *s)
{
    constexpr double kPerTurn = 0.15915494309189535;  // 1 / 2 pi
    double t = (double)position * ((double)f * kPerTurn);
    t -= rint(t);
    const double q = rint(4.0 * t);
    const float x = (float)((t - 0.25 * q) * 6.283185307179586);
    const float z = x * x;
    const float sn =
        x * fmaf(z, fmaf(z, fmaf(z, fmaf(z, 1.0f / 362880, -1.0f / 5040), 1.0f / 120), -1.0f / 6), 1.0f);
    const float cs = fmaf(
        z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -1.0f / 3628800, 1.0f / 40320), -1.0f / 720), 1.0f / 24), -0.5f), 1.0f);
    const int k = (int)q & 3;
    *c = k == 0 ? cs : k == 1 ? -sn : k == 2 ? -cs : sn;
    *s = k == 0 ? sn : k == 1 ? cs : k == 2 ? -sn : -cs;
}

struct Unit {       // a lane's 16 channels of a row
    int lo, hi;     // first channels of its two groups of 8
    int pair;       // first of its 8 pairs, or -1: not rotated
    bool on;        // the row has this unit
};
__device__ __forceinline__ Unit unit_of(const RopeArgs &a, int u)
{
    Unit t;
    t.on = u < a.D / 16;
    t.pair = -1;
    if (16 * u < a.R && !a.interleaved) {
        t.lo = 8 * u;
        t.hi = a.R / 2 + 8 * u;
        t.pair = 8 * u;
    } else {
        t.lo = 16 * u;
        t.hi = 16 * u + 8;
        if (16 * u < a.R)
            t.pair = 8 * u;
    }
    return t;
}

// rotate 8 pairs held as x[0..7], x[8..15] (half) or neighbours (interleaved); back: by -t
__device__ __forceinline__ void rotate(float *x, const float *cs, bool interleaved, bool back)
{
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float c = cs[2 * e], s = back ? -cs[2 * e + 1] : cs[2 * e + 1];
        if (interleaved) {
            const float p = x[2 * e], q = x[2 * e + 1];
            x[2 * e] = p * c - q * s;
            x[2 * e + 1] = p * s + q * c;
        } else {
            const float p = x[e], q = x[e + 8];
            x[e] = p * c - q * s;
            x[e + 8] = p * s + q * c;
        }
    }
}

__device__ __forceinline__ float row_sum(float x, int lanes)
{
    for (int o = lanes >> 1; o > 0; o >>= 1)
        x += __shfl_xor(x, o);
    return x;
}

__device__ __forceinline__ float norm_factor(const RopeArgs &a, float ss)
{
    if (a.norm == 0)
        return 1.0f;
    return rsqrtf((a.norm == 1 ? ss / (float)a.D : ss) + a.eps);
}

// cos/sin of the step's tokens: [token][pair][2] in LDS
__device__ __forceinline__ void fill_turns(const RopeArgs &a, float *lds, int64_t t0, int n, int tid)
{
    const int pairs = a.R / 2;
    for (int i = tid; i < n * pairs; i += kRopeThreads) {
        const int tt = i / pairs, p = i - tt * pairs;
        const int64_t tok = t0 + tt;
        float c, s;
        turn(a.positions ? a.positions[tok] : tok % a.T, a.inv_freq[p], &c, &s);
        lds[2 * i] = c * a.factor;
        lds[2 * i + 1] = s * a.factor;
    }
}

template <int kT>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeArgs a)
{
    extern __shared__ __attribute__((aligned(16))) float turns[];
    constexpr int kSize = kT == kFp32 ? 4 : 2;
    const int tid = threadIdx.x;
    int lanes = 1;
    while (lanes * 16 < a.D)
        lanes <<= 1;
    const int group = tid / lanes, groups = kRopeThreads / lanes;
    const Unit u = unit_of(a, tid & (lanes - 1));
    const int64_t total = a.B * a.T;
    const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
    const int n = (int)(total - t0 < a.tokens ? total - t0 : a.tokens);
    fill_turns(a, turns, t0, n, tid);
    __syncthreads();
    const int heads = a.heads[0] + a.heads[1], rows = n * heads;
    for (int r = group; r < rows; r += groups) {
        const int tt = r / heads, hh = r - tt * heads;
        const int side = hh >= a.heads[0] ? 1 : 0, h = side ? hh - a.heads[0] : hh;
        const int64_t tok = t0 + tt, b = tok / a.T, t = tok - b * a.T;
        float x[16];
#pragma unroll
        for (int e = 0; e < 16; ++e)
            x[e] = 0.0f;
        const RopeView &in = a.x[side], &out = a.y[side];
        const unsigned char *p = in.p + (b * in.sb + t * in.st + h * in.sh) * kSize;
        if (u.on) {
            load8<kT>(p + u.lo * kSize, x);
            load8<kT>(p + u.hi * kSize, x + 8);
        }
        float ss = 0.0f;
#pragma unroll
        for (int e = 0; e < 16; ++e)
            ss = fmaf(x[e], x[e], ss);
        const float rn = norm_factor(a, row_sum(ss, lanes));
        const float *w = a.w[side];
        if (!u.on)
            continue;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[e] *= w ? rn * w[u.lo + e] : rn;
            x[8 + e] *= w ? rn * w[u.hi + e] : rn;
        }
        if (u.pair >= 0)
            rotate(x, turns + (tt * (a.R / 2) + u.pair) * 2, a.interleaved != 0, false);
        unsigned char *q = out.p + (b * out.sb + t * out.st + h * out.sh) * kSize;
        store8<kT>(q + u.lo * kSize, x);
        store8<kT>(q + u.hi * kSize, x + 8);
    }
}

template <int kT>
__global__ __launch_bounds__(kRopeThreads) void rope_bwd_kernel(RopeArgs a)
{
    extern __shared__ __attribute__((aligned(16))) float turns[];
    constexpr int kSize = kT == kFp32 ? 4 : 2;
    const int tid = threadIdx.x;
    int lanes = 1;
    while (lanes * 16 < a.D)
        lanes <<= 1;
    const int group = tid / lanes, groups = kRopeThreads / lanes;
    const Unit u = unit_of(a, tid & (lanes - 1));
    const int64_t total = a.B * a.T;
    float dw[2][16];
#pragma unroll
    for (int e = 0; e < 16; ++e)
        dw[0][e] = dw[1][e] = 0.0f;
    for (int64_t t0 = (int64_t)blockIdx.x * a.tokens; t0 < total; t0 += (int64_t)gridDim.x * a.tokens) {
        const int n = (int)(total - t0 < a.tokens ? total - t0 : a.tokens);
        __syncthreads();
        fill_turns(a, turns, t0, n, tid);
        __syncthreads();
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            const int heads = a.heads[side], rows = n * heads;
            const RopeView &in = a.x[side], &gr = a.dy[side], &out = a.y[side];
            const float *w = a.w[side];
            for (int r = group; r < rows; r += groups) {
                const int tt = r / heads, h = r - tt * heads;
                const int64_t tok = t0 + tt, b = tok / a.T, t = tok - b * a.T;
                float x[16], d[16];
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    x[e] = d[e] = 0.0f;
                const unsigned char *p = in.p + (b * in.sb + t * in.st + h * in.sh) * kSize;
                const unsigned char *g = gr.p + (b * gr.sb + t * gr.st + h * gr.sh) * kSize;
                if (u.on) {
                    load8<kT>(p + u.lo * kSize, x);
                    load8<kT>(p + u.hi * kSize, x + 8);
                    load8<kT>(g + u.lo * kSize, d);
                    load8<kT>(g + u.hi * kSize, d + 8);
                }
                if (u.pair >= 0)
                    rotate(d, turns + (tt * (a.R / 2) + u.pair) * 2, a.interleaved != 0, true);
                float ss = 0.0f, sd = 0.0f;
                float wd[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int ch = e < 8 ? u.lo + e : u.hi + e - 8;
                    wd[e] = w && u.on ? d[e] * w[ch] : d[e];
                    ss = fmaf(x[e], x[e], ss);
                    sd = fmaf(x[e], wd[e], sd);
                }
                const float rn = norm_factor(a, row_sum(ss, lanes));
                sd = row_sum(sd, lanes);
                const float back = a.norm == 0 ? 0.0f : sd * rn * rn * rn / (a.norm == 1 ? (float)a.D : 1.0f);
                float dx[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    dw[side][e] = fmaf(d[e], x[e] * rn, dw[side][e]);
                    dx[e] = rn * wd[e] - x[e] * back;
                }
                if (u.on) {
                    unsigned char *q = out.p + (b * out.sb + t * out.st + h * out.sh) * kSize;
                    store8<kT>(q + u.lo * kSize, dx);
                    store8<kT>(q + u.hi * kSize, dx + 8);
                }
            }
        }
    }
    // this workgroup's weight sums, groups added in order
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        if (!a.dw[side])
            continue;
        __syncthreads();
        if (u.on) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                turns[group * a.D + (e < 8 ? u.lo + e : u.hi + e - 8)] = dw[side][e];
        }
        __syncthreads();
        for (int ch = tid; ch < a.D; ch += kRopeThreads) {
            float s = 0.0f;
            for (int g = 0; g < groups; ++g)
                s += turns[g * a.D + ch];
            a.part[((int64_t)blockIdx.x * 2 + side) * a.D + ch] = s;
        }
    }
}

// dw[ch] = sum of the workgroups' parts, in a fixed order; one wave per channel and side
__global__ __launch_bounds__(256) void rope_dw_kernel(RopeArgs a, int64_t parts)
{
    const int side = blockIdx.y, ch = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
    if (ch >= a.D || !a.dw[side])
        return;
    double s = 0.0;
    for (int64_t n = lane; n < parts; n += 64)
        s += (double)a.part[(n * 2 + side) * a.D + ch];
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        s += __shfl_xor(s, o);
    if (lane == 0)
        a.dw[side][ch] = (float)s;
}

}  // namespace

int64_t rope_groups(int64_t tokens, int heads, int D, bool backward, int *per_step)
{
    int lanes = 1;
    while (lanes * 16 < D)
        lanes <<= 1;
    const int groups = kRopeThreads / lanes;
    // about four rows for each group of lanes and step, fewer where that would leave the chip empty
    int64_t n = (4 * groups + heads - 1) / heads;
    if (n > 16)
        n = 16;
    while (n > 1 && (tokens + n - 1) / n < 512)
        n >>= 1;
    *per_step = (int)n;
    int64_t steps = (tokens + n - 1) / n;
    if (steps < 1)
        steps = 1;
    return backward && steps > kRopeGroups ? kRopeGroups : steps;
}

hipError_t rope_launch(const RopeArgs &a0, hipStream_t s)
{
    RopeArgs a = a0;
    const int64_t grid = rope_groups(a.B * a.T, a.heads[0] + a.heads[1], a.D, false, &a.tokens);
    if (a.B * a.T == 0)
        return hipSuccess;
    const size_t lds = (size_t)a.tokens * a.R * sizeof(float);
    const dim3 g((unsigned)grid), b(kRopeThreads);
    if (a.dtype == kBf16)
        hipLaunchKernelGGL(rope_kernel<kBf16>, g, b, lds, s, a);
    else if (a.dtype == kFp32)
        hipLaunchKernelGGL(rope_kernel<kFp32>, g, b, lds, s, a);
    else
        hipLaunchKernelGGL(rope_kernel<kFp16>, g, b, lds, s, a);
    return hipGetLastError();
}

hipError_t rope_launch_bwd(const RopeArgs &a0, hipStream_t s)
{
    RopeArgs a = a0;
    const int64_t grid = rope_groups(a.B * a.T, a.heads[0] + a.heads[1], a.D, true, &a.tokens);
    int lanes = 1;
    while (lanes * 16 < a.D)
        lanes <<= 1;
    const size_t turns = (size_t)a.tokens * a.R * sizeof(float);
    const size_t sums = (size_t)(kRopeThreads / lanes) * a.D * sizeof(float);
    const size_t lds = turns > sums ? turns : sums;
    const dim3 g((unsigned)grid), b(kRopeThreads);
    if (a.dtype == kBf16)
        hipLaunchKernelGGL(rope_bwd_kernel<kBf16>, g, b, lds, s, a);
    else if (a.dtype == kFp32)
        hipLaunchKernelGGL(rope_bwd_kernel<kFp32>, g, b, lds, s, a);
    else
        hipLaunchKernelGGL(rope_bwd_kernel<kFp16>, g, b, lds, s, a);
    if (a.dw[0] || a.dw[1])
        hipLaunchKernelGGL(rope_dw_kernel, dim3((unsigned)((a.D + 3) / 4), 2), dim3(256), 0, s, a, grid);
    return hipGetLastError();
}

}  // namespace kda
