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
// Bound by memory: every value is read once and written once (backward: read twice as many).  Measured: 16384
// tokens x 40 heads of 128, bf16, forward 72 us from pass to pass (336 MB, 4.7 TB/s; a copy of that size 5.3), 78 us from
// its first wave to its last; backward B = 2, T = 4096, 16 + 16 heads 50 us from pass to pass with the weights' sums (201
// MB, 4.0 TB/s), 47 us the kernel alone (219 MB by the counters, 4.7 TB/s).  One row in flight per lane group ran at 2.5 TB/s; four (two
// backwards) keep enough loads on their way.  Small fp32 batches are bound by latency (3001 tokens, 12 + 1 heads: 26 us,
// of which the angles, one row's loads, the sums and the second launch follow each other).
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

// 16 bytes of memory as values and back; values are rounded once, to nearest even
template <int kT>
struct Piece {
    static constexpr int kSize = kT == kFp32 ? 4 : 2;
    static constexpr int kPer = 16 / kSize;       // values
    static constexpr int kCount = 8 / kPer;       // pieces of 8 values
};
template <int kT>
__device__ __forceinline__ void widen(const u32x4 *u, float *x)
{
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if constexpr (kT == kFp32) {
            x[e] = __uint_as_float(u[e >> 2][e & 3]);
        } else {
            const uint32_t w = u[0][e >> 1], half = e & 1 ? w >> 16 : w & 0xffffu;
            if constexpr (kT == kBf16)
                x[e] = __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16);
            else
                x[e] = (float)__builtin_bit_cast(_Float16, (uint16_t)half);
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
    if (!t.on) {  // reads the row's first unit, counts for nothing
        t.lo = 0;
        t.hi = 8;
        return t;
    }
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

// LDS of a step: cos and sin of its tokens [token][pair][2], and where each token's row of a tensor begins, in bytes.
constexpr int kMaxStep = 64;  // tokens
struct Starts {
    int64_t at[6][kMaxStep];  // q, k, their outputs (or gradients), ...
};

template <int kViews, int kSize>
__device__ __forceinline__ void fill_starts(const RopeArgs &a, Starts &s, int64_t t0, int n, int tid)
{
    for (int i = tid; i < kViews * kMaxStep; i += kRopeThreads) {
        const int view = i / kMaxStep, tt = i - view * kMaxStep;
        if (tt < n) {
            // the step's first token is divided once, as one value for the workgroup
            const int64_t b0 = t0 / a.T;
            int64_t b = b0, t = t0 - b0 * a.T + tt;
            while (t >= a.T) {
                t -= a.T;
                ++b;
            }
            const RopeView &v = view < 2 ? a.x[view] : kViews == 4 || view >= 4 ? a.y[view & 1] : a.dy[view & 1];
            s.at[view][tt] = (b * v.sb + t * v.st) * kSize;
        }
    }
}
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

// One tensor's rows (token, head) of a step, `groups` at a time.
struct Rows {
    int heads, count;
    float inv;

    __device__ Rows(int heads_, int n) : heads(heads_), count(n * heads_), inv(1.0f / (float)heads_) {}
    // r below 2^18, so that (r + 1/2) / heads is far enough from whole numbers for fp32
    __device__ int token(int r) const { return (int)(((float)r + 0.5f) * inv); }
};

template <int kT, int kRows>
struct RowLoads {
    u32x4 u[kRows][2 * Piece<kT>::kCount];
};
// kRows rows of this lane's group from row r on, `groups` apart; rows behind the last one repeat it
template <int kT, int kRows>
__device__ __forceinline__ void load_rows(RowLoads<kT, kRows> &f, const RopeView &v, const int64_t *starts, const Rows &ro,
                                          const Unit &u, int r, int groups)
{
    constexpr int kSize = Piece<kT>::kSize;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int rr = min(r + i * groups, ro.count - 1), tt = ro.token(rr), h = rr - tt * ro.heads;
        const unsigned char *p = v.p + starts[tt] + (int64_t)h * (v.sh * kSize);
#pragma unroll
        for (int c = 0; c < Piece<kT>::kCount; ++c) {
            f.u[i][c] = *reinterpret_cast<const u32x4 *>(p + u.lo * kSize + 16 * c);
            f.u[i][Piece<kT>::kCount + c] = *reinterpret_cast<const u32x4 *>(p + u.hi * kSize + 16 * c);
        }
    }
}

// A lane's 16 weights (1 without weights)
__device__ __forceinline__ void load_weights(float *w, const float *p, const Unit &u)
{
#pragma unroll
    for (int e = 0; e < 16; ++e)
        w[e] = p ? p[e < 8 ? u.lo + e : u.hi + e - 8] : 1.0f;
}

template <int kT>
__device__ __forceinline__ void rope_side(const RopeArgs &a, int side, int n, const Starts &st, const float *turns,
                                          const Unit &u, int group, int groups, int lanes, bool first)
{
    constexpr int kRows = kT == kFp32 ? 2 : 4, kSize = Piece<kT>::kSize, kC = Piece<kT>::kCount;
    const Rows ro(a.heads[side], n);
    float w[16];
    load_weights(w, a.w[side], u);
    RowLoads<kT, kRows> f;
    load_rows<kT, kRows>(f, a.x[side], st.at[side], ro, u, group, groups);
    if (first)  // every thread: the angles are ready; the first rows are on their way by then
        __syncthreads();
    for (int r = group; r < ro.count; r += kRows * groups) {
        if (r != group)
            load_rows<kT, kRows>(f, a.x[side], st.at[side], ro, u, r, groups);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int rr = r + i * groups;
            if (rr >= ro.count)
                break;
            float x[16];
            widen<kT>(f.u[i], x);
            widen<kT>(f.u[i] + kC, x + 8);
            float ss = 0.0f;
#pragma unroll
            for (int e = 0; e < 16; ++e)
                ss = fmaf(x[e], x[e], ss);
            const float rn = norm_factor(a, row_sum(u.on ? ss : 0.0f, lanes));
#pragma unroll
            for (int e = 0; e < 16; ++e)
                x[e] *= rn * w[e];
            const int tt = ro.token(rr), h = rr - tt * ro.heads;
            if (u.pair >= 0)
                rotate(x, turns + (tt * (a.R / 2) + u.pair) * 2, a.interleaved != 0, false);
            if (u.on) {
                unsigned char *q = a.y[side].p + st.at[2 + side][tt] + (int64_t)h * (a.y[side].sh * kSize);
                store8<kT>(q + u.lo * kSize, x);
                store8<kT>(q + u.hi * kSize, x + 8);
            }
        }
    }
}

template <int kT>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeArgs a)
{
    extern __shared__ __attribute__((aligned(16))) float turns[];
    __shared__ Starts st;
    const int tid = threadIdx.x;
    int lanes = 1;
    while (lanes * 16 < a.D)
        lanes <<= 1;
    const int group = tid / lanes, groups = kRopeThreads / lanes;
    const Unit u = unit_of(a, tid & (lanes - 1));
    const int64_t total = a.B * a.T;
    const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
    const int n = (int)(total - t0 < a.tokens ? total - t0 : a.tokens);
    fill_starts<4, Piece<kT>::kSize>(a, st, t0, n, tid);
    __syncthreads();
    fill_turns(a, turns, t0, n, tid);
    rope_side<kT>(a, 0, n, st, turns, u, group, groups, lanes, true);
    rope_side<kT>(a, 1, n, st, turns, u, group, groups, lanes, false);
}

template <int kT>
__device__ __forceinline__ void rope_bwd_side(const RopeArgs &a, int side, int n, const Starts &st, const float *turns,
                                              const Unit &u, int group, int groups, int lanes, float *dw)
{
    constexpr int kRows = kT == kFp32 ? 1 : 2, kSize = Piece<kT>::kSize, kC = Piece<kT>::kCount;
    const Rows ro(a.heads[side], n);
    float w[16];
    load_weights(w, a.w[side], u);
    for (int r = group; r < ro.count; r += kRows * groups) {
        RowLoads<kT, kRows> fx, fd;
        load_rows<kT, kRows>(fx, a.x[side], st.at[side], ro, u, r, groups);
        load_rows<kT, kRows>(fd, a.dy[side], st.at[2 + side], ro, u, r, groups);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int rr = r + i * groups;
            if (rr >= ro.count)
                break;
            const int tt = ro.token(rr), h = rr - tt * ro.heads;
            float x[16], d[16];
            widen<kT>(fx.u[i], x);
            widen<kT>(fx.u[i] + kC, x + 8);
            widen<kT>(fd.u[i], d);
            widen<kT>(fd.u[i] + kC, d + 8);
            if (u.pair >= 0)
                rotate(d, turns + (tt * (a.R / 2) + u.pair) * 2, a.interleaved != 0, true);
            float ss = 0.0f, sd = 0.0f;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                ss = fmaf(x[e], x[e], ss);
                sd = fmaf(x[e], d[e] * w[e], sd);
            }
            const float rn = norm_factor(a, row_sum(u.on ? ss : 0.0f, lanes));
            sd = row_sum(u.on ? sd : 0.0f, lanes);
            const float back = a.norm == 0 ? 0.0f : sd * rn * rn * rn / (a.norm == 1 ? (float)a.D : 1.0f);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                dw[e] = fmaf(d[e], x[e] * rn, dw[e]);
                d[e] = rn * (d[e] * w[e]) - x[e] * back;
            }
            if (u.on) {
                unsigned char *q = a.y[side].p + st.at[4 + side][tt] + (int64_t)h * (a.y[side].sh * kSize);
                store8<kT>(q + u.lo * kSize, d);
                store8<kT>(q + u.hi * kSize, d + 8);
            }
        }
    }
}

// Workgroups [0, groups_q) take q's rows, the others k's, in steps of tokens; each keeps its weight sums in registers.
template <int kT>
__global__ __launch_bounds__(kRopeThreads, 4) void rope_bwd_kernel(RopeArgs a)
{
    extern __shared__ __attribute__((aligned(16))) float turns[];
    __shared__ Starts st;
    const int tid = threadIdx.x;
    int lanes = 1;
    while (lanes * 16 < a.D)
        lanes <<= 1;
    const int group = tid / lanes, groups = kRopeThreads / lanes;
    const Unit u = unit_of(a, tid & (lanes - 1));
    const int64_t total = a.B * a.T;
    const int side = (int)blockIdx.x >= a.groups[0] ? 1 : 0, step = a.step[side];
    float dw[16];
#pragma unroll
    for (int e = 0; e < 16; ++e)
        dw[e] = 0.0f;
    for (int64_t t0 = (int64_t)(blockIdx.x - (side ? a.groups[0] : 0)) * step; t0 < total;
         t0 += (int64_t)a.groups[side] * step) {
        const int n = (int)(total - t0 < step ? total - t0 : step);
        __syncthreads();
        fill_starts<6, Piece<kT>::kSize>(a, st, t0, n, tid);
        fill_turns(a, turns, t0, n, tid);
        __syncthreads();
        rope_bwd_side<kT>(a, side, n, st, turns, u, group, groups, lanes, dw);
    }
    if (!a.dw[side])
        return;
    // this workgroup's weight sums, groups added in order
    __syncthreads();
    if (u.on) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
            turns[group * a.D + (e < 8 ? u.lo + e : u.hi + e - 8)] = dw[e];
    }
    __syncthreads();
    for (int ch = tid; ch < a.D; ch += kRopeThreads) {
        float s = 0.0f;
        for (int g = 0; g < groups; ++g)
            s += turns[g * a.D + ch];
        a.part[(int64_t)blockIdx.x * a.D + ch] = s;
    }
}

// dw[ch] = sum of the workgroups' parts, in a fixed order: 16 channels a workgroup, 64 runs of parts side by side
__global__ __launch_bounds__(1024) void rope_dw_kernel(RopeArgs a)
{
    __shared__ double sum[64][17];
    const int side = blockIdx.y, c = threadIdx.x & 15, run = threadIdx.x >> 4, ch = blockIdx.x * 16 + c;
    if (!a.dw[side])
        return;
    const float *p = a.part + (side ? (int64_t)a.groups[0] * a.D : 0) + ch;
    double s = 0.0;
#pragma unroll 4
    for (int n = run; n < a.groups[side]; n += 64)
        s += (double)p[(int64_t)n * a.D];
    sum[run][c] = s;
    __syncthreads();
    if (run == 0) {
        for (int i = 1; i < 64; ++i)
            s += sum[i][c];
        a.dw[side][ch] = (float)s;
    }
}

}  // namespace

namespace {

int lanes_of(int D)
{
    int lanes = 1;
    while (lanes * 16 < D)
        lanes <<= 1;
    return lanes;
}
// Tokens per step: about four rows for each group of lanes, fewer where that would leave the chip empty; cos and sin
// of a step fit 32 KiB.
int step_of(int64_t tokens, int heads, int D, int R, int64_t want)
{
    const int groups = kRopeThreads / lanes_of(D);
    int n = (4 * groups + heads - 1) / heads;
    const int most = R > 0 ? 8192 / R : kMaxStep;
    n = n > most ? most : n;
    n = n > kMaxStep ? kMaxStep : n;
    while (n > 1 && (tokens + n - 1) / n < want)
        n = (n + 1) / 2;
    return n;
}

}  // namespace

void rope_plan_bwd(RopeArgs *a)
{
    const int64_t tokens = a->B * a->T;
    const int64_t heads = a->heads[0] + a->heads[1];
    for (int side = 0; side < 2; ++side) {
        // workgroups by the share of rows, all resident at once: four on each of 256 CUs
        int64_t g = side ? kRopeGroups - kRopeGroups * a->heads[0] / heads : kRopeGroups * a->heads[0] / heads;
        g = g < 1 ? 1 : g > kRopeGroups - 1 ? kRopeGroups - 1 : g;
        a->step[side] = step_of(tokens, a->heads[side], a->D, a->R, g);
        const int64_t steps = (tokens + a->step[side] - 1) / a->step[side];
        a->groups[side] = (int)(steps < 1 ? 1 : steps < g ? steps : g);
    }
}

hipError_t rope_launch(const RopeArgs &a0, hipStream_t s)
{
    RopeArgs a = a0;
    const int64_t tokens = a.B * a.T;
    if (tokens == 0)
        return hipSuccess;
    a.tokens = step_of(tokens, a.heads[0] + a.heads[1], a.D, a.R, 512);
    const size_t lds = (size_t)a.tokens * a.R * sizeof(float);
    const dim3 g((unsigned)((tokens + a.tokens - 1) / a.tokens)), b(kRopeThreads);
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
    rope_plan_bwd(&a);
    const size_t turns = (size_t)(a.step[0] > a.step[1] ? a.step[0] : a.step[1]) * a.R * sizeof(float);
    const size_t sums = (size_t)(kRopeThreads / lanes_of(a.D)) * a.D * sizeof(float);
    const size_t lds = turns > sums ? turns : sums;
    const dim3 g((unsigned)(a.groups[0] + a.groups[1])), b(kRopeThreads);
    if (a.dtype == kBf16)
        hipLaunchKernelGGL(rope_bwd_kernel<kBf16>, g, b, lds, s, a);
    else if (a.dtype == kFp32)
        hipLaunchKernelGGL(rope_bwd_kernel<kFp32>, g, b, lds, s, a);
    else
        hipLaunchKernelGGL(rope_bwd_kernel<kFp16>, g, b, lds, s, a);
    if (a.dw[0] || a.dw[1])
        hipLaunchKernelGGL(rope_dw_kernel, dim3((unsigned)(a.D / 16), 2), dim3(1024), 0, s, a);
    return hipGetLastError();
}

}  // namespace kda
