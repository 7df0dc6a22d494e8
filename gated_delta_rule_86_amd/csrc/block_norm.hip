// block_norm.hip -- the norms before and after a block, fused with what stands between them, gfx950.
//
// Gated norm, per token and head, x, z (the gate) [D]:
//   r = (mean x^2 + eps)^-1/2,   out = x r w act(z),   act the sigmoid s or silu z s.
//   Backward, with d = dout act(z) w:
//   dx = r d - x r^3 mean(d x),   dz = dout x r w act'(z),   dw = sum over rows of dout act(z) x r.
// Residual norm, per token, x (a block's output), res [D]:
//   h = x, or x r_x post (a norm behind the block);   y = res + scale h;   residual_out = y, rounded to its type;
//   out = y r_y w (the norm before the next block), from the sum before it is rounded.
//   Backward, y the stored stream, g = dout w:
//   dy = dresidual_out + r_y g - y r_y^3 mean(g y) = dresidual,   dw = sum dout y r_y,   dscale = sum dy h,
//   dh = scale dy,   dx = dh, or r_x dh post - x r_x^3 mean(dh post x),   dpost = sum dh x r_x.
//
// Everything is fp32 and rounded once.  Bound by memory: every value is read once and written once, a row stays in the
// registers of its lanes.  A lane owns 8 neighbouring channels (16 bytes of a 2-byte type); D / 8 lanes, rounded up to a
// power of two, own a row of up to 512 channels, several rows in flight; longer rows take a workgroup of 256 or 512
// threads with one or two pieces each, the next row's loads on their way while one is worked on.
//
// Measured (a copy of 512 MiB: 5.33 TB/s): residual forward, 16384 rows of 4096 bf16 channels, both norms: 104 us, 5.2 TB/s;
// residual backward, 6002 rows of 2048, bf16 with an fp32 stream: 43 us, 5.3 TB/s, and 5 for the sums; 16384 rows of 4096 with
// both norms and their sums 178 us, 4.5 TB/s (without the norm behind the block 166), with an fp32 stream 240, 5.0 TB/s;
// gated backward, 131072 rows of 128: 34 us, 4.9 TB/s, and 4 for the sums: there a third of the issue slots are taken,
// the exponential and the divisions of the gate among them; gated forward of 1024 rows: 6 us, the launch; of 131072 rows
// 24 us, 4.2 TB/s, of 524288 77 us, 5.2 TB/s.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "norm_internal.h"

namespace kda {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kBf16 = 1, kFp32 = 2, kFp16 = 3;
constexpr int kThreads = 256;

// 8 values as they lie in memory; rounded once, to nearest even
template <int kT>
struct Raw {
    static constexpr int kWords = kT == kFp32 ? 2 : 1;
    static constexpr int kSize = kT == kFp32 ? 4 : 2;
    u32x4 u[kWords];

    __device__ void load(const unsigned char *p)
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            u[i] = reinterpret_cast<const u32x4 *>(p)[i];
    }
    __device__ void store(unsigned char *p) const
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            reinterpret_cast<u32x4 *>(p)[i] = u[i];
    }
    __device__ float get(int e) const
    {
        if constexpr (kT == kFp32) {
            return __uint_as_float(u[e >> 2][e & 3]);
        } else {
            const uint32_t w = u[0][e >> 1];
            if constexpr (kT == kBf16)
                return __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16);
            else
                return (float)__builtin_bit_cast(_Float16, (uint16_t)(e & 1 ? w >> 16 : w & 0xffffu));
        }
    }
    __device__ void set(const float *x)
    {
        if constexpr (kT == kFp32) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                u[e >> 2][e & 3] = __float_as_uint(x[e]);
        } else {
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
                u[0][e] = (uint32_t)a | ((uint32_t)b << 16);
            }
        }
    }
};

// First byte of row r (below 2^31, so that fp64 finds token and batch row exactly)
template <int kSize>
__device__ __forceinline__ const unsigned char *row_at(const NormArgs &a, const NormView &v, int r)
{
    if (v.flat)
        return v.p + (int64_t)r * v.sh * kSize;
    const int tok = (int)(((double)r + 0.5) * a.inv_h), h = r - tok * a.H;
    const int b = (int)(((double)tok + 0.5) * a.inv_t);
    return v.p + ((int64_t)b * v.sb + ((int64_t)tok - (int64_t)b * a.T) * v.st + (int64_t)h * v.sh) * kSize;
}

__device__ __forceinline__ float sum_lanes(float x, int lanes)
{
    for (int o = lanes >> 1; o > 0; o >>= 1)
        x += __shfl_xor(x, o);
    return x;
}

// e^-|z| and from it the sigmoid y of z and 1 - y, neither of which cancels
__device__ __forceinline__ void sigmoid(float z, float &y, float &rest)
{
    constexpr float kHi = 1.44269502f, kLo = 1.92596299e-8f;  // log2 e
    const float n = -fabsf(z), t = n * kHi, low = fmaf(n, kHi, -t) + n * kLo;
    const float e = __builtin_amdgcn_exp2f(t) * fmaf(low, 0.693147182f, 1.0f);
    const float f = n < -150.0f ? 0.0f : e;  // far out the low part is no number
    const float big = __builtin_amdgcn_rcpf(1.0f + f), small = f * big;
    y = z != z ? z : z >= 0.0f ? big : small;
    rest = z >= 0.0f ? small : big;
}

// ------------------------------------------------------------------------------ gated norm

struct Group {   // the lanes of a row
    int lanes, ch;
    bool on;     // this lane has channels; others read the row's first ones and count for nothing
};
__device__ __forceinline__ Group group_of(int D, int tid)
{
    Group g;
    g.lanes = 1;
    while (g.lanes * 8 < D)
        g.lanes <<= 1;
    const int i = tid & (g.lanes - 1);
    g.on = i * 8 < D;
    g.ch = g.on ? i * 8 : 0;
    return g;
}

template <int kT>
constexpr int kGatedRows = kT == kFp32 ? 2 : 4;  // rows in flight for each group of lanes

template <int kT>
__global__ __launch_bounds__(kThreads) void gated_kernel(NormArgs a)
{
    constexpr int kRows = kGatedRows<kT>, kSize = Raw<kT>::kSize;
    const Group g = group_of(a.D, threadIdx.x);
    const int groups = kThreads / g.lanes;
    float w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        w[e] = a.w ? a.w[g.ch + e] : 1.0f;
    const float inv_d = 1.0f / (float)a.D;
    for (int64_t r0 = (int64_t)blockIdx.x * (groups * kRows); r0 < a.rows; r0 += (int64_t)gridDim.x * (groups * kRows)) {
        Raw<kT> x[kRows], z[kRows];
        int row[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int64_t r = r0 + threadIdx.x / g.lanes + i * groups;
            row[i] = r < a.rows ? (int)r : -1;
            const int rr = r < a.rows ? (int)r : a.rows - 1;
            x[i].load(row_at<kSize>(a, a.x, rr) + g.ch * kSize);
            z[i].load(row_at<kSize>(a, a.z, rr) + g.ch * kSize);
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            float ss = 0.0f, y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                ss = fmaf(x[i].get(e), x[i].get(e), ss);
            const float rn = rsqrtf(fmaf(sum_lanes(g.on ? ss : 0.0f, g.lanes), inv_d, a.eps));
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float t = z[i].get(e);
                float s, rest;
                sigmoid(t, s, rest);
                y[e] = x[i].get(e) * rn * w[e] * (a.act ? t * s : s);
            }
            if (row[i] >= 0 && g.on) {
                Raw<kT> o;
                o.set(y);
                o.store(a.y + ((int64_t)row[i] * a.D + g.ch) * kSize);
            }
        }
    }
}

// Weight sums of the workgroup: its groups of lanes added in order
__device__ __forceinline__ void write_part(const NormArgs &a, const Group &g, const float *dw, float *out, float *lds)
{
    __syncthreads();
    if (g.on) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            lds[threadIdx.x / g.lanes * a.D + g.ch + e] = dw[e];
    }
    __syncthreads();
    for (int ch = threadIdx.x; ch < a.D; ch += kThreads) {
        float s = 0.0f;
        for (int n = 0; n < kThreads / g.lanes; ++n)
            s += lds[n * a.D + ch];
        out[(int64_t)blockIdx.x * a.D + ch] = s;
    }
}

template <int kT>
__global__ __launch_bounds__(kThreads) void gated_bwd_kernel(NormArgs a)
{
    constexpr int kRows = kGatedRows<kT> / 2, kSize = Raw<kT>::kSize;
    __shared__ float lds[kThreads * 8];
    const Group g = group_of(a.D, threadIdx.x);
    const int groups = kThreads / g.lanes;
    float w[8], dw[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        w[e] = a.w ? a.w[g.ch + e] : 1.0f;
        dw[e] = 0.0f;
    }
    const float inv_d = 1.0f / (float)a.D;
    for (int64_t r0 = (int64_t)blockIdx.x * (groups * kRows); r0 < a.rows; r0 += (int64_t)gridDim.x * (groups * kRows)) {
        Raw<kT> x[kRows], z[kRows], d[kRows];
        int row[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int64_t r = r0 + threadIdx.x / g.lanes + i * groups;
            row[i] = r < a.rows ? (int)r : -1;
            const int rr = r < a.rows ? (int)r : a.rows - 1;
            x[i].load(row_at<kSize>(a, a.x, rr) + g.ch * kSize);
            z[i].load(row_at<kSize>(a, a.z, rr) + g.ch * kSize);
            d[i].load(a.dy + ((int64_t)rr * a.D + g.ch) * kSize);
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            float ss = 0.0f, sd = 0.0f, act[8], dact[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float t = z[i].get(e), xe = x[i].get(e);
                float s, rest;
                sigmoid(t, s, rest);
                act[e] = a.act ? t * s : s;
                dact[e] = a.act ? s * fmaf(t, rest, 1.0f) : s * rest;
                ss = fmaf(xe, xe, ss);
                sd = fmaf(d[i].get(e) * act[e] * w[e], xe, sd);
            }
            const float rn = rsqrtf(fmaf(sum_lanes(g.on ? ss : 0.0f, g.lanes), inv_d, a.eps));
            const float back = sum_lanes(g.on ? sd : 0.0f, g.lanes) * inv_d * rn * rn * rn;
            if (row[i] < 0 || !g.on)
                continue;
            float dx[8], dz[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float n = x[i].get(e) * rn, da = d[i].get(e) * act[e];
                dw[e] = fmaf(da, n, dw[e]);
                dx[e] = da * w[e] * rn - x[i].get(e) * back;
                dz[e] = d[i].get(e) * n * w[e] * dact[e];
            }
            Raw<kT> o;
            o.set(dx);
            o.store(a.y + ((int64_t)row[i] * a.D + g.ch) * kSize);
            o.set(dz);
            o.store(a.zo + ((int64_t)row[i] * a.D + g.ch) * kSize);
        }
    }
    if (a.dw)
        write_part(a, g, dw, a.part, lds);
}

// ---------------------------------------------------------------------------- residual norm
//
// kBlock 0: rows of up to 512 channels, a group of lanes each, 256 threads; else a workgroup of kBlock threads for a
// row, kP pieces of 8 channels a thread.

template <int kBlock>
struct Sums {
    int lanes, turn;
    float (*red)[8];

    // sum over the row's threads; every one of them gets it
    __device__ float operator()(float x)
    {
        if constexpr (kBlock == 0) {
            return sum_lanes(x, lanes);
        } else {
            x = sum_lanes(x, 64);
            if ((threadIdx.x & 63) == 0)
                red[turn][threadIdx.x >> 6] = x;
            __syncthreads();
            float s = red[turn][0];
#pragma unroll
            for (int i = 1; i < kBlock / 64; ++i)
                s += red[turn][i];
            turn ^= 1;  // the other row: the next sum may begin before everyone has read this one
            return s;
        }
    }
};

template <int kBlock, int kP>
struct Place {
    int ch[kP];
    bool on[kP];

    __device__ Place(int D, int lanes)
    {
        const int i = kBlock ? (int)threadIdx.x : (int)threadIdx.x & (lanes - 1), n = kBlock ? kBlock : lanes;
#pragma unroll
        for (int p = 0; p < kP; ++p) {
            ch[p] = 8 * (i + p * n);
            on[p] = ch[p] < D;
            if (!on[p])
                ch[p] = 0;
        }
    }
    __device__ void load(float (*w)[8], const float *src, float none) const
    {
#pragma unroll
        for (int p = 0; p < kP; ++p)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                w[p][e] = src ? src[ch[p] + e] : none;
    }
};

template <int kT, int kR, int kBlock, int kP>
__global__ __launch_bounds__(kBlock ? kBlock : kThreads) void residual_kernel(NormArgs a)
{
    constexpr int kSize = Raw<kT>::kSize, kRSize = Raw<kR>::kSize;
    __shared__ float red[2][8];
    const int lanes = kBlock ? kBlock : group_of(a.D, 0).lanes;
    Sums<kBlock> sum{lanes, 0, red};
    const Place<kBlock, kP> at(a.D, lanes);
    const int groups = kBlock ? 1 : kThreads / lanes;
    float w[kP][8], post[kP][8], scale[kP][8];
    at.load(w, a.w, 1.0f);
    at.load(post, a.post, 1.0f);
    at.load(scale, a.scale, 1.0f);
    const float inv_d = 1.0f / (float)a.D;
    const int64_t step = (int64_t)gridDim.x * groups;
    int64_t r = (int64_t)blockIdx.x * groups + (kBlock ? 0 : threadIdx.x / lanes);
    Raw<kT> x[kP];
    Raw<kR> z[kP];
    auto fetch = [&](int64_t n) {
        const int rr = n < a.rows ? (int)n : a.rows - 1;
        const unsigned char *px = row_at<kSize>(a, a.x, rr), *pz = row_at<kRSize>(a, a.z, rr);
#pragma unroll
        for (int p = 0; p < kP; ++p) {
            x[p].load(px + at.ch[p] * kSize);
            z[p].load(pz + at.ch[p] * kRSize);
        }
    };
    if ((int64_t)blockIdx.x * groups < a.rows)
        fetch(r);
    // every thread of a workgroup takes as many steps: the sums hold barriers
    for (int64_t first = (int64_t)blockIdx.x * groups; first < a.rows; first += step, r += step) {
        float h[kP][8], y[kP][8], ss = 0.0f;
#pragma unroll
        for (int p = 0; p < kP; ++p)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                h[p][e] = x[p].get(e);
                y[p][e] = z[p].get(e);
                ss = at.on[p] ? fmaf(h[p][e], h[p][e], ss) : ss;
            }
        if (first + step < a.rows)
            fetch(r + step);
        const float rx = a.post_norm ? rsqrtf(fmaf(sum(ss), inv_d, a.eps)) : 1.0f;
        ss = 0.0f;
#pragma unroll
        for (int p = 0; p < kP; ++p)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                y[p][e] = fmaf(h[p][e] * rx * post[p][e], scale[p][e], y[p][e]);
                ss = at.on[p] ? fmaf(y[p][e], y[p][e], ss) : ss;
            }
        const float ry = rsqrtf(fmaf(sum(ss), inv_d, a.eps));
        if (r >= a.rows)
            continue;
#pragma unroll
        for (int p = 0; p < kP; ++p) {
            if (!at.on[p])
                continue;
            Raw<kR> zo;
            zo.set(y[p]);
            zo.store(a.zo + (r * a.D + at.ch[p]) * kRSize);
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                o[e] = y[p][e] * ry * w[p][e];
            Raw<kT> yo;
            yo.set(o);
            yo.store(a.y + (r * a.D + at.ch[p]) * kSize);
        }
    }
}

template <int kT, int kR, int kBlock, int kP>
__global__ __launch_bounds__(kBlock ? kBlock : kThreads) void residual_bwd_kernel(NormArgs a)
{
    constexpr int kSize = Raw<kT>::kSize, kRSize = Raw<kR>::kSize;
    __shared__ float red[2][8];
    __shared__ float lds[kBlock ? 1 : kThreads * 8];
    const int lanes = kBlock ? kBlock : group_of(a.D, 0).lanes;
    Sums<kBlock> sum{lanes, 0, red};
    const Place<kBlock, kP> at(a.D, lanes);
    const int groups = kBlock ? 1 : kThreads / lanes;
    float w[kP][8], post[kP][8], scale[kP][8], dw[kP][8], dpost[kP][8], dscale[kP][8];
    at.load(w, a.w, 1.0f);
    at.load(post, a.post, 1.0f);
    at.load(scale, a.scale, 1.0f);
    at.load(dw, nullptr, 0.0f);
    at.load(dpost, nullptr, 0.0f);
    at.load(dscale, nullptr, 0.0f);
    const float inv_d = 1.0f / (float)a.D;
    const bool need_x = a.post_norm || a.dscale;
    const int64_t step = (int64_t)gridDim.x * groups;
    int64_t r = (int64_t)blockIdx.x * groups + (kBlock ? 0 : threadIdx.x / lanes);
    Raw<kT> x[kP], d[kP];
    Raw<kR> z[kP], g[kP];
    auto fetch = [&](int64_t n) {
        const int rr = n < a.rows ? (int)n : a.rows - 1;
        const unsigned char *px = row_at<kSize>(a, a.x, rr), *pz = row_at<kRSize>(a, a.z, rr);
        const int64_t flat = (int64_t)rr * a.D;
#pragma unroll
        for (int p = 0; p < kP; ++p) {
            if (need_x)
                x[p].load(px + at.ch[p] * kSize);
            z[p].load(pz + at.ch[p] * kRSize);
            d[p].load(a.dy + (flat + at.ch[p]) * kSize);
            if (a.dz)
                g[p].load(a.dz + (flat + at.ch[p]) * kRSize);
        }
    };
    if ((int64_t)blockIdx.x * groups < a.rows)
        fetch(r);
    for (int64_t first = (int64_t)blockIdx.x * groups; first < a.rows; first += step, r += step) {
        const bool mine = r < a.rows;
        float h[kP][8], y[kP][8], dy[kP][8], dn[kP][8], ss = 0.0f, sd = 0.0f;
#pragma unroll
        for (int p = 0; p < kP; ++p)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                h[p][e] = need_x ? x[p].get(e) : 0.0f;
                y[p][e] = z[p].get(e);
                dn[p][e] = d[p].get(e);
                dy[p][e] = a.dz ? g[p].get(e) : 0.0f;
                if (at.on[p]) {
                    ss = fmaf(y[p][e], y[p][e], ss);
                    sd = fmaf(dn[p][e] * w[p][e], y[p][e], sd);
                }
            }
        if (first + step < a.rows)
            fetch(r + step);
        const float ry = rsqrtf(fmaf(sum(ss), inv_d, a.eps));
        const float back = sum(sd) * inv_d * ry * ry * ry;
        float rx = 1.0f, xback = 0.0f;
#pragma unroll
        for (int p = 0; p < kP; ++p)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (mine)
                    dw[p][e] = fmaf(dn[p][e], y[p][e] * ry, dw[p][e]);
                dy[p][e] += dn[p][e] * w[p][e] * ry - y[p][e] * back;
            }
        if (a.post_norm) {
            ss = sd = 0.0f;
#pragma unroll
            for (int p = 0; p < kP; ++p)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (at.on[p]) {
                        ss = fmaf(h[p][e], h[p][e], ss);
                        sd = fmaf(dy[p][e] * scale[p][e] * post[p][e], h[p][e], sd);
                    }
            rx = rsqrtf(fmaf(sum(ss), inv_d, a.eps));
            xback = sum(sd) * inv_d * rx * rx * rx;
        }
        if (!mine)
            continue;
#pragma unroll
        for (int p = 0; p < kP; ++p) {
            if (!at.on[p])
                continue;
            float dx[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float dh = dy[p][e] * scale[p][e], n = h[p][e] * rx;
                dpost[p][e] = fmaf(dh, n, dpost[p][e]);
                dscale[p][e] = fmaf(dy[p][e], n * post[p][e], dscale[p][e]);
                dx[e] = dh * post[p][e] * rx - h[p][e] * xback;
            }
            Raw<kR> zo;
            zo.set(dy[p]);
            zo.store(a.zo + (r * a.D + at.ch[p]) * kRSize);
            Raw<kT> yo;
            yo.set(dx);
            yo.store(a.y + (r * a.D + at.ch[p]) * kSize);
        }
    }
    const int64_t each = (int64_t)a.groups * a.D;
    if constexpr (kBlock == 0) {
        const Group gr = group_of(a.D, threadIdx.x);
        if (a.dw)
            write_part(a, gr, dw[0], a.part, lds);
        if (a.dpost)
            write_part(a, gr, dpost[0], a.part + each, lds);
        if (a.dscale)
            write_part(a, gr, dscale[0], a.part + 2 * each, lds);
    } else {
#pragma unroll
        for (int p = 0; p < kP; ++p) {
            if (!at.on[p])
                continue;
            float *q = a.part + (int64_t)blockIdx.x * a.D + at.ch[p];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (a.dw)
                    q[e] = dw[p][e];
                if (a.dpost)
                    q[each + e] = dpost[p][e];
                if (a.dscale)
                    q[2 * each + e] = dscale[p][e];
            }
        }
    }
}

// Sums of the workgroups' parts in a fixed order: 16 channels a workgroup, 64 runs of parts side by side
__global__ __launch_bounds__(1024) void norm_dw_kernel(NormArgs a)
{
    __shared__ double sum[64][17];
    float *out = blockIdx.y == 0 ? a.dw : blockIdx.y == 1 ? a.dpost : a.dscale;
    if (!out)
        return;
    const int c = threadIdx.x & 15, run = threadIdx.x >> 4, ch = blockIdx.x * 16 + c;
    const float *p = a.part + (int64_t)blockIdx.y * a.groups * a.D + ch;
    double s = 0.0;
    if (ch < a.D)
#pragma unroll 4
        for (int n = run; n < a.groups; n += 64)
            s += (double)p[(int64_t)n * a.D];
    sum[run][c] = s;
    __syncthreads();
    if (run == 0 && ch < a.D) {
        for (int i = 1; i < 64; ++i)
            s += sum[i][c];
        out[ch] = (float)s;
    }
}

int lanes_of(int D)
{
    int lanes = 1;
    while (lanes * 8 < D)
        lanes <<= 1;
    return lanes;
}

hipError_t launch_sums(const NormArgs &a, hipStream_t s)
{
    if (a.dw || a.dpost || a.dscale)
        hipLaunchKernelGGL(norm_dw_kernel, dim3((unsigned)((a.D + 15) / 16), a.dpost || a.dscale ? 3 : 1), dim3(1024), 0, s, a);
    return hipGetLastError();
}

template <int kT, int kR, bool kBack>
hipError_t launch_residual(const NormArgs &a, hipStream_t s)
{
    if (a.D <= 512) {
        const int per = kThreads / lanes_of(a.D);
        if constexpr (kBack)
            hipLaunchKernelGGL((residual_bwd_kernel<kT, kR, 0, 1>), dim3((unsigned)a.groups), dim3(kThreads), 0, s, a);
        else
            hipLaunchKernelGGL((residual_kernel<kT, kR, 0, 1>), dim3((unsigned)((a.rows + per - 1) / per > 65536 ? 65536 : (a.rows + per - 1) / per)), dim3(kThreads), 0, s, a);
    } else {
        // as many workgroups as run at once, each with its share of the rows
        const unsigned grid = kBack ? (unsigned)a.groups : (unsigned)(a.rows < 2048 ? a.rows : 2048);
#define KDA_RES(block, pieces)                                                                                    \
    if constexpr (kBack)                                                                                          \
        hipLaunchKernelGGL((residual_bwd_kernel<kT, kR, block, pieces>), dim3(grid), dim3(block), 0, s, a);       \
    else                                                                                                          \
        hipLaunchKernelGGL((residual_kernel<kT, kR, block, pieces>), dim3(grid), dim3(block), 0, s, a);
        if (a.D <= 2048) {
            KDA_RES(256, 1)
        } else if (a.D <= 4096) {
            KDA_RES(256, 2)
        } else {
            KDA_RES(512, 2)
        }
#undef KDA_RES
    }
    return hipGetLastError();
}

template <bool kBack>
hipError_t launch_residual_types(const NormArgs &a, hipStream_t s)
{
    if (a.dtype == kFp32)
        return launch_residual<kFp32, kFp32, kBack>(a, s);
    if (a.dtype == kBf16)
        return a.rdtype == kFp32 ? launch_residual<kBf16, kFp32, kBack>(a, s) : launch_residual<kBf16, kBf16, kBack>(a, s);
    return a.rdtype == kFp32 ? launch_residual<kFp16, kFp32, kBack>(a, s) : launch_residual<kFp16, kFp16, kBack>(a, s);
}

}  // namespace

int gated_groups(int64_t rows, int D, int dtype)
{
    const int64_t per = (int64_t)(kThreads / lanes_of(D)) * (dtype == kFp32 ? 1 : 2), n = (rows + per - 1) / per;
    return (int)(n < 1 ? 1 : n < kNormGroups ? n : kNormGroups);
}
int residual_groups(int64_t rows, int D)
{
    const int64_t per = D <= 512 ? kThreads / lanes_of(D) : 1, n = (rows + per - 1) / per;
    const int64_t most = D <= 512 ? kNormGroups : 512;
    return (int)(n < 1 ? 1 : n < most ? n : most);
}

hipError_t gated_launch(const NormArgs &a, hipStream_t s)
{
    const int64_t per = (int64_t)(kThreads / lanes_of(a.D)) * (a.dtype == kFp32 ? 2 : 4), n = (a.rows + per - 1) / per;
    const dim3 g((unsigned)(n < 65536 ? n : 65536)), b(kThreads);
    if (a.dtype == kBf16)
        hipLaunchKernelGGL(gated_kernel<kBf16>, g, b, 0, s, a);
    else if (a.dtype == kFp32)
        hipLaunchKernelGGL(gated_kernel<kFp32>, g, b, 0, s, a);
    else
        hipLaunchKernelGGL(gated_kernel<kFp16>, g, b, 0, s, a);
    return hipGetLastError();
}

hipError_t gated_launch_bwd(const NormArgs &a, hipStream_t s)
{
    const dim3 g((unsigned)a.groups), b(kThreads);
    if (a.dtype == kBf16)
        hipLaunchKernelGGL(gated_bwd_kernel<kBf16>, g, b, 0, s, a);
    else if (a.dtype == kFp32)
        hipLaunchKernelGGL(gated_bwd_kernel<kFp32>, g, b, 0, s, a);
    else
        hipLaunchKernelGGL(gated_bwd_kernel<kFp16>, g, b, 0, s, a);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? launch_sums(a, s) : e;
}

hipError_t residual_launch(const NormArgs &a, hipStream_t s) { return launch_residual_types<false>(a, s); }

hipError_t residual_launch_bwd(const NormArgs &a, hipStream_t s)
{
    const hipError_t e = launch_residual_types<true>(a, s);
    return e == hipSuccess ? launch_sums(a, s) : e;
}

}  // namespace kda
