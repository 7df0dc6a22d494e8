// gdn.hip -- gated delta rule with a decay for each head, gfx950.
//
// Per (sequence, head), state S [V = 128][K = 128], natural-log decay g_t <= 0, write strength beta_t:
//   S~ = e^{g_t} S_{t-1},   r_t = v_t - S~ k_t,   S_t = S~ + beta_t r_t k_t^T,   out_t = scale * S_t q_t.
// In chunks of C = 64 tokens, with b the inclusive running sum of g inside the chunk, L its last entry and
// S the state before the chunk, the residuals R (rows r_t) solve a unit triangular system:
//   r_t = x_t - sum_{s < t} e^{b_t - b_s} (k_t.k_s) beta_s r_s,   x_t = v_t - e^{b_t} S k_t,
//   so R = T' X with T' = (1 + M diag(beta))^-1, M_ts = e^{b_t - b_s} k_t.k_s for s < t;
//   out_t = scale * (e^{b_t} S q_t + sum_{s <= t} e^{b_t - b_s} (q_t.k_s) beta_s r_s),
//   S    <- e^{L} S + sum_s e^{L - b_s} beta_s r_s k_s^T.
// T' does not divide by beta (beta = 0 writes nothing and needs no case of its own).  It is formed as 1 - N diag(beta)
// with N = (1 + M diag(beta))^-1 M, from which the backward pass also has T = (1 + diag(beta) M)^-1 = 1 - diag(beta) N.
//
// Backward, with dS the gradient of the state after the chunk, A_ts = scale e^{b_t - b_s} q_t.k_s (s <= t), w = beta r the
// writes and dw their gradients, dx = beta dw those of x:
//   dw = T^T (A^T dO + tail (dS k_s)),  tail_s = e^{L - b_s},   dv = dx,   dbeta_t = dw_t.r_t,
//   dS_before = e^{L} dS + sum_t (scale e^{b_t} dO_t) q_t^T - (e^{b_t} dx_t) k_t^T,
//   dq_t = scale e^{b_t} S^T dO_t + sum_s P_ts k_s,           P_ts = scale e^{b_t - b_s} dO_t.w_s  (s <= t),
//   dk_s = tail_s dS^T w_s - e^{b_s} S^T dx_s + sum_t P_ts q_t + sum_t (G_ts + G_st) k_t,
//                                                             G_ts = -e^{b_t - b_s} dx_t.w_s     (s < t),
//   dg_t = sum over the chunk's u >= t of (q_u.dq_u - v_u.dv_u), plus <dS, S_after>,
// since <dS~, S~> at a token is that at the next one plus what the token's read adds and its write takes.
//
// Numbers: decays are used as min(max(g, -1000), 0); running sums of logarithms are fp64, a factor is the
// exponential of a difference and at most 1.  The products run on bf16 MFMA with fp32 accumulation; q, k, v are
// bf16 as they come, every other factor is cut into three bf16 terms, hi + mid + lo: the 24 bits of fp32.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn_internal.h"
#include "lin_internal.h"

namespace kda {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u4 __attribute__((vector_size(16)));   // as the buffer builtins want them
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void lds_void;

constexpr int kBf16 = 1;  // kda_state_dtype
constexpr float kLowest = -1000.0f;
constexpr double kLog2e64 = 1.4426950408889634;

__device__ __forceinline__ float lo_f(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_f(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    bf16x2 p;
    p[0] = (__bf16)a;
    p[1] = (__bf16)b;
    return __builtin_bit_cast(uint32_t, p);
}
__device__ __forceinline__ float clamp_decay(float g)
{
    return g < kLowest ? kLowest : (g > 0.0f ? 0.0f : g);  // NaN stays NaN
}

// v_mfma_f32_16x16x32_bf16: A[m][k] in lane m + 16*(k/8), element k%8; B[k][n] in lane n + 16*(k/8), element
// k%8; D[m][n] in lane n + 16*(m/4), element m%4.  The order of k is free as long as A and B agree: everywhere here
// element j of lane group g stands for k = 4g + j (j < 4) or 16 + 4g + j - 4, so two D tiles are one B (or A) operand.
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}
// v_mfma_f32_16x16x4_f32: A[m][k] in lane m + 16 k, B[k][n] in lane n + 16 k; step i of four takes k = 4g + i
__device__ __forceinline__ f32x4 mfma_f32(f32x4 a, f32x4 b, f32x4 c)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
    return c;
}

struct Terms {  // three bf16 terms of 8 floats
    u32x4 h, m, l;
};
// two floats into word e of each term
__device__ __forceinline__ void cut2(float x, float y, Terms &t, int e)
{
    uint32_t h = pack2(x, y);
    __asm__("" : "+v"(h));  // one conversion for both: else each value is converted again to get its rest
    t.h[e] = h;
    const float x1 = x - lo_f(t.h[e]), y1 = y - hi_f(t.h[e]);
    uint32_t m = pack2(x1, y1);
    __asm__("" : "+v"(m));
    t.m[e] = m;
    t.l[e] = pack2(x1 - lo_f(t.m[e]), y1 - hi_f(t.m[e]));
}
__device__ __forceinline__ void cut8(f32x4 a, f32x4 b, Terms &t)
{
    cut2(a[0], a[1], t, 0);
    cut2(a[2], a[3], t, 1);
    cut2(b[0], b[1], t, 2);
    cut2(b[2], b[3], t, 3);
}
// products with an exact factor, and of two cut factors (the terms left out are below 2^-24 of the product)
__device__ __forceinline__ f32x4 mfma3(u32x4 a, const Terms &b, f32x4 c)
{
    c = mfma(a, b.l, c);
    c = mfma(a, b.m, c);
    return mfma(a, b.h, c);
}
__device__ __forceinline__ f32x4 mfma3(const Terms &a, u32x4 b, f32x4 c)
{
    c = mfma(a.l, b, c);
    c = mfma(a.m, b, c);
    return mfma(a.h, b, c);
}
__device__ __forceinline__ f32x4 mfma6(const Terms &a, const Terms &b, f32x4 c)
{
    c = mfma(a.l, b.h, c);
    c = mfma(a.h, b.l, c);
    c = mfma(a.m, b.m, c);
    c = mfma(a.m, b.h, c);
    c = mfma(a.h, b.m, c);
    return mfma(a.h, b.h, c);
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void *base, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ u32x4 buf_b128(__amdgpu_buffer_rsrc_t r, uint32_t off)
{
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// Everything that this wave has in flight has arrived, and then the other waves' too.
__device__ __forceinline__ void arrive()
{
    __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
    __asm__ volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    __asm__ volatile("" ::: "memory");
}

// ------------------------------------------------------------------ sequences and chunks

// A value that is the same in all lanes, said so: descriptors and branches on it stay scalar.
__device__ __forceinline__ int64_t uniform(int64_t x)
{
    const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)x), hi = __builtin_amdgcn_readfirstlane((int)(x >> 32));
    return (int64_t)(((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ int64_t seq_begin(const GdnArgs &a, int64_t i) { return a.cu ? a.cu[i] : i * a.T; }

// First element of a tensor's row and head (heads are shared by small whole numbers: 32-bit division)
__device__ __forceinline__ const uint16_t *head_base(const GdnTensor &x, int64_t row, int64_t h)
{
    return x.p + uniform(row * x.sb + (int64_t)((uint32_t)h / (uint32_t)x.share) * x.sh);
}

// Records: chunk c of sequence i has slot floor(begin / 64) + i + c; the slots of different sequences differ.
__device__ __forceinline__ int64_t slot_of(int64_t begin, int64_t i) { return begin / kGC + i; }

// Largest i in [0, N) with key(i) <= x, for a key that does not decrease; key(0) <= x.
template <typename F>
__device__ __forceinline__ int64_t last_at_most(int64_t N, int64_t x, F key)
{
    int64_t lo = 0, hi = N;  // key(lo) <= x < key(hi)
    while (hi - lo > 1) {
        const int64_t m = (lo + hi) >> 1;
        if (key(m) <= x)
            lo = m;
        else
            hi = m;
    }
    return lo;
}

// The first chunk of segment p of a row (p = P: the row's end), as a sequence and a chunk of it.
struct Entry {
    int64_t seq, chunk;  // chunk > 0: the sequence comes from the segment before
};
__device__ __forceinline__ Entry entry_of(const GdnArgs &a, int64_t row, int64_t p)
{
    const int64_t at = p * a.len;
    if (!a.cu)
        return p >= a.P ? Entry{row + 1, 0} : Entry{row, at / kGC};  // len is a multiple of a chunk
    if (p >= a.P)
        return Entry{a.N, 0};
    if (p == 0)
        return Entry{0, 0};
    // the first sequence that begins at `at` or behind, or the one before it if it has a chunk there
    const int64_t m = uniform(a.cu[0]) >= at ? 0 : last_at_most(a.N + 1, at - 1, [&](int64_t n) { return uniform(a.cu[n]); });
    if (m >= a.N)
        return Entry{a.N, 0};
    const int64_t begin = uniform(a.cu[m]), c = (at - begin + kGC - 1) / kGC;
    return c * kGC < uniform(a.cu[m + 1]) - begin ? Entry{m, c} : Entry{m + 1, 0};
}

struct Chunk {
    int64_t seq, slot;
    int64_t t0;     // first token, in its row
    int len;        // 0: no chunk
    bool first, last;  // of the workgroup's piece of the sequence
    bool from_seg, to_seg;  // the piece begins (ends) at a cut
};

// The chunks from one entry to another, in order (or from the last to the first).
struct Walk {
    Entry e0, e1;
    int64_t i, c, c_lo, c_hi;  // current sequence, chunk, its piece [c_lo, c_hi)
    int64_t begin, len;
    bool rev;

    __device__ void init(const Entry &a0, const Entry &a1, bool rev_)
    {
        e0 = Entry{uniform(a0.seq), uniform(a0.chunk)};
        e1 = Entry{uniform(a1.seq), uniform(a1.chunk)};
        rev = rev_;
        i = rev ? e1.seq + 1 : e0.seq - 1;
        c = c_lo = c_hi = 0;
        begin = len = 0;
    }
    // The 64-bit comparisons run on the vector unit; said to be uniform once more, the results stay scalar.
    __device__ Chunk next(const GdnArgs &a)
    {
        Chunk k = advance(a);
        k.len = __builtin_amdgcn_readfirstlane(k.len);
        k.seq = uniform(k.seq);
        k.slot = uniform(k.slot);
        k.t0 = uniform(k.t0);
        return k;
    }
    __device__ Chunk advance(const GdnArgs &a)
    {
        Chunk k = {0, 0, 0, 0, false, false, false, false};
        c += rev ? -1 : 1;
        while (rev ? c < c_lo : c >= c_hi) {
            i += rev ? -1 : 1;
            if (rev ? i < e0.seq : (i > e1.seq || (i == e1.seq && e1.chunk == 0))) {
                c_lo = 0, c_hi = 0;  // from now on every call ends here
                c = rev ? -1 : 0;
                i = rev ? e0.seq : e1.seq;
                return k;
            }
            if (rev && i == e1.seq && e1.chunk == 0) {  // nothing of it belongs here
                c_lo = c_hi = 0;
                c = -1;
                continue;
            }
            begin = uniform(seq_begin(a, i));
            len = uniform(seq_begin(a, i + 1)) - begin;
            const int64_t n = (len + kGC - 1) / kGC;
            c_lo = i == e0.seq ? e0.chunk : 0;
            c_hi = i == e1.seq ? e1.chunk : n;
            if (c_lo >= c_hi) {
                c_lo = c_hi = 0;
                c = rev ? -1 : 0;
                continue;
            }
            c = rev ? c_hi - 1 : c_lo;
            k.first = true;
        }
        k.last = rev ? c == c_lo : c + 1 == c_hi;
        k.from_seg = rev ? i == e1.seq : c_lo > 0;
        k.to_seg = rev ? c_lo > 0 : i == e1.seq;
        const int64_t rest = len - c * kGC;
        k.len = (int)(rest < kGC ? rest : kGC);
        k.seq = i;
        k.slot = slot_of(begin, i) + c;
        k.t0 = (a.cu ? begin : 0) + c * kGC;
        return k;
    }
};

template <int kCtrl, int kRows>
__device__ __forceinline__ double dpp_f64(double x)  // 0 where the pattern has no source lane
{
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, kCtrl, kRows, 0xf, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), kCtrl, kRows, 0xf, false);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
// Inclusive sum over the lanes: shifts by 1, 2, 4, 8 inside each 16, then the last lane of row 0 and 2 to the next
// row, then lane 31 to the upper half.
__device__ __forceinline__ double running_sum(double b)
{
    b += dpp_f64<0x111, 0xf>(b);
    b += dpp_f64<0x112, 0xf>(b);
    b += dpp_f64<0x114, 0xf>(b);
    b += dpp_f64<0x118, 0xf>(b);
    b += dpp_f64<0x142, 0xa>(b);
    b += dpp_f64<0x143, 0xc>(b);
    return b;
}
__device__ __forceinline__ double last_lane(double b)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, b);
    return __builtin_bit_cast(double,
                              ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), 63) << 32) |
                                  (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, 63));
}

// ------------------------------------------------------------------------------- records
//
// Factors of a record, 64 floats each (token of the chunk):
constexpr int kVHead = 0;     // e^{b_t}
constexpr int kVWrite = 64;   // beta_s e^{L - b_s}
constexpr int kVOut = 128;    // scale e^{b_t}
constexpr int kVBeta = 192;   // beta_s
constexpr int kVTail = 256;   // e^{L - b_s}
constexpr int kVLast = 320;   // [0]: e^{L}
constexpr int kVSum = 384;    // b_t (log2), as a pair of floats: the second 64 behind the first

// block of a triangular matrix with rows in row tile r and the contraction in 32-column step ks
__device__ __forceinline__ constexpr int low_block(int r, int ks) { return r < 2 ? r : 2 + 2 * (r - 2) + ks; }  // ks <= r / 2
__device__ __forceinline__ constexpr int up_block(int r, int ks) { return r < 2 ? 2 * r + ks : 4 + (r - 2); }  // ks >= r / 2

__device__ __forceinline__ void store_terms(unsigned char *mat, int block, int lane, const Terms &t)
{
    u32x4 *p = reinterpret_cast<u32x4 *>(mat + block * 1024 + lane * 16);
    p[0] = t.h;
    p[6 * 64] = t.m;
    p[12 * 64] = t.l;
}

constexpr int kNRow = 68;  // floats per row of the triangular matrix in LDS

struct LdsPrep {
    float n[kGC * kNRow];
    float bh[kGC], bl[kGC], beta[kGC];
};

// One workgroup of 4 waves per (chunk, head).  Wave w forms row tile w of M = e^{b_t - b_s} k_t.k_s; the four
// 16 x 16 blocks on the diagonal of N are solved column by column, the blocks below them with fp32 matrix
// instructions, a wave per block column: N_IJ = (1 - N_II beta)(M_IJ - sum_{J <= K < I} M_IK beta N_KJ).
template <bool kBwd>
__global__ __launch_bounds__(256) void gdn_prep_kernel(GdnArgs a)
{
    __shared__ __attribute__((aligned(16))) LdsPrep s;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, m = lane & 15, g = lane >> 4;
    const int64_t slot = blockIdx.x / a.H, h = blockIdx.x - slot * a.H;
    if (a.status && *a.status != 0)
        return;
    const int64_t seq = last_at_most(a.N, slot, [&](int64_t i) { return slot_of(uniform(seq_begin(a, i)), i); });
    const int64_t begin = uniform(seq_begin(a, seq)), c = slot - slot_of(begin, seq),
                  rest = uniform(seq_begin(a, seq + 1)) - begin - c * kGC;
    if (rest <= 0)
        return;
    const int len = (int)(rest < kGC ? rest : kGC);
    const int64_t row = a.cu ? 0 : seq, t0 = (a.cu ? begin : 0) + c * kGC;
    unsigned char *rec = a.rec + (slot * a.H + h) * a.rec_bytes;

    auto tile = [&](const GdnTensor &x) {
        const uint32_t stride = (uint32_t)x.st * 2;
        return rsrc(head_base(x, row, h) + t0 * x.st, (uint32_t)(len - 1) * stride + 256u);
    };
    const __amdgpu_buffer_rsrc_t rk = tile(a.k), rq = tile(a.q);
    const uint32_t sk = (uint32_t)a.k.st * 2, sq = (uint32_t)a.q.st * 2;
    u32x4 kf[4][4], qf[4][4];  // row tiles, 32 channels each step; behind the chunk zeros
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int p = 0; p < 4; ++p)
            kf[r][p] = buf_b128(rk, (uint32_t)(16 * r + m) * sk + (uint32_t)(64 * p + 16 * g));
    // forward: A' of out rows 16 w ..; backward: A^T of source rows 16 w ..
#pragma unroll
    for (int r = 0; r < (kBwd ? 4 : 1); ++r)
#pragma unroll
        for (int p = 0; p < 4; ++p)
            qf[r][p] = buf_b128(rq, (uint32_t)(16 * (kBwd ? r : wave) + m) * sq + (uint32_t)(64 * p + 16 * g));

    const int64_t gate = ((row * a.T + t0) * a.H + h);
    const float dec = lane < len ? a.decay[gate + (int64_t)lane * a.H] : 0.0f;
    const float bet = lane < len ? a.beta[gate + (int64_t)lane * a.H] : 0.0f;
    const double b = running_sum((double)clamp_decay(dec) * kLog2e64), last = last_lane(b);
    if (wave == 0) {
        const float bh = (float)b;
        s.bh[lane] = bh;
        s.bl[lane] = (float)(b - (double)bh);
        s.beta[lane] = bet;
        float *v = reinterpret_cast<float *>(rec + kGdnMat);
        const float head = __builtin_amdgcn_exp2f((float)b), tail = __builtin_amdgcn_exp2f((float)(last - b));
        v[kVHead + lane] = head;
        v[kVWrite + lane] = bet * tail;
        v[kVOut + lane] = a.scale * head;
        v[kVBeta + lane] = bet;
        v[kVTail + lane] = tail;
        if constexpr (kBwd) {
            v[kVSum + lane] = bh;
            v[kVSum + 64 + lane] = (float)(b - (double)bh);
        }
        if (lane == 0)
            v[kVLast] = __builtin_amdgcn_exp2f((float)last);
    }
    __syncthreads();
    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
    // e^{b_t - b_s} for s <= t, else 0
    auto within = [&](int t, int u) {
        const float d = (s.bh[t] - s.bh[u]) + (s.bl[t] - s.bl[u]);
        return u <= t ? __builtin_amdgcn_exp2f(d) : 0.0f;
    };
    // row tile `wave` of M, strictly below the diagonal
    u32x4 kw[4];
#pragma unroll
    for (int p = 0; p < 4; ++p)
        kw[p] = wave == 0 ? kf[0][p] : wave == 1 ? kf[1][p] : wave == 2 ? kf[2][p] : kf[3][p];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (j > wave)
            continue;
        f32x4 d = zero;
#pragma unroll
        for (int p = 0; p < 4; ++p)
            d = mfma(kw[p], kf[j][p], d);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 16 * wave + 4 * g + i, u = 16 * j + m;
            s.n[t * kNRow + u] = u < t ? d[i] * within(t, u) : 0.0f;
        }
    }
    // A: products of q and k
    if constexpr (!kBwd) {
        f32x4 t4[4] = {zero, zero, zero, zero};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j > wave)
                continue;
            f32x4 d = zero;  // rows: sources 16 j .., columns: out tokens 16 w ..
#pragma unroll
            for (int p = 0; p < 4; ++p)
                d = mfma(kf[j][p], qf[0][p], d);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = 16 * wave + m, u = 16 * j + 4 * g + i;
                t4[j][i] = u <= t ? d[i] * (a.scale * within(t, u)) * s.beta[u] : 0.0f;
            }
        }
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            if (2 * ks > wave)
                continue;
            Terms t;
            cut8(t4[2 * ks], t4[2 * ks + 1], t);
            store_terms(rec + kGdnMat + kGdnVec, low_block(wave, ks), lane, t);
        }
    } else {
        f32x4 t4[4] = {zero, zero, zero, zero};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j < wave)
                continue;
            f32x4 d = zero;  // rows: out tokens 16 j .., columns: sources 16 w ..
#pragma unroll
            for (int p = 0; p < 4; ++p)
                d = mfma(qf[j][p], kw[p], d);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = 16 * j + 4 * g + i, u = 16 * wave + m;
                t4[j][i] = u <= t ? d[i] * (a.scale * within(t, u)) : 0.0f;
            }
        }
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            if (2 * ks + 1 < wave)
                continue;
            Terms t;
            cut8(t4[2 * ks], t4[2 * ks + 1], t);
            store_terms(rec + 2 * kGdnMat + kGdnVec, up_block(wave, ks), lane, t);
        }
    }
    // N's diagonal block: lane m its column m.  Rows of the wave's own block only; the four lane groups do the same.
    {
        float y[16];  // beta times the column so far
        float x[16];
        const float *blk = s.n + 16 * wave * (kNRow + 1);
        const float *bb = s.beta + 16 * wave;
        y[0] = x[0] = 0.0f;
#pragma unroll
        for (int i = 1; i < 16; ++i) {
            float z = blk[i * kNRow + m];
#pragma unroll
            for (int k = 1; k < i; ++k)
                z = fmaf(-blk[i * kNRow + k], y[k], z);
            x[i] = i > m ? z : 0.0f;
            y[i] = bb[i] * x[i];
        }
        __builtin_amdgcn_wave_barrier();
        if (g == 0) {
            float *w = s.n + 16 * wave * (kNRow + 1) + m;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                w[i * kNRow] = x[i];
        }
    }
    __syncthreads();
    // the blocks below it
    f32x4 n[3], y[4];
    {
        auto rows = [&](int bi, int bj) {  // D layout of a block
            f32x4 r;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                r[i] = s.n[(16 * bi + 4 * g + i) * kNRow + 16 * bj + m];
            return r;
        };
        auto left = [&](int bi, int bk) {  // minus a block, as A operand
            return -*reinterpret_cast<const f32x4 *>(&s.n[(16 * bi + m) * kNRow + 16 * bk + 4 * g]);
        };
        auto beta4 = [&](int bi) { return *reinterpret_cast<const f32x4 *>(&s.beta[16 * bi + 4 * g]); };
        y[0] = rows(wave, wave) * beta4(wave);
#pragma unroll
        for (int d = 1; d < 4; ++d) {
            if (wave + d > 3)
                break;
            const int bi = wave + d;
            f32x4 p = rows(bi, wave);
#pragma unroll
            for (int e = 0; e < d; ++e)
                p = mfma_f32(left(bi, wave + e), y[e], p);
            n[d - 1] = mfma_f32(left(bi, bi), p * beta4(bi), p);
            y[d] = n[d - 1] * beta4(bi);
        }
    }
    __syncthreads();
#pragma unroll
    for (int d = 1; d < 4; ++d)
        if (wave + d < 4)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                s.n[(16 * (wave + d) + 4 * g + i) * kNRow + 16 * wave + m] = n[d - 1][i];
    __syncthreads();
    // T' = 1 - N beta, rows 16 w ..
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
        if (2 * ks > wave)
            continue;
        const int t = 16 * wave + m;
        f32x4 x[2];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int u0 = 32 * ks + 16 * hf + 4 * g;
            const f32x4 nn = *reinterpret_cast<const f32x4 *>(&s.n[t * kNRow + u0]);
            const f32x4 bb = *reinterpret_cast<const f32x4 *>(&s.beta[u0]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[hf][i] = u0 + i < t ? -nn[i] * bb[i] : u0 + i == t ? 1.0f : 0.0f;
        }
        Terms tt;
        cut8(x[0], x[1], tt);
        store_terms(rec, low_block(wave, ks), lane, tt);
    }
    // T = 1 - beta N, transposed: rows are sources 16 w ..
    if constexpr (kBwd) {
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            if (2 * ks + 1 < wave)
                continue;
            const int u = 16 * wave + m;
            f32x4 x[2];
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = 32 * ks + 16 * hf + 4 * g + i;
                    x[hf][i] = u < t ? -s.n[t * kNRow + u] * s.beta[t] : u == t ? 1.0f : 0.0f;
                }
            Terms tt;
            cut8(x[0], x[1], tt);
            store_terms(rec + kGdnMat + kGdnVec, up_block(wave, ks), lane, tt);
        }
    }
}

// ------------------------------------------------------------------------- state in registers
//
// Wave w of 8 holds value columns 16w .. 16w+15 of the state, all 128 key channels: S[kt][i], lane = column + 16 g:
// channel 16 kt + 4 g + i, the D layout of S^T.  Nothing of it ever crosses waves.

struct State {
    f32x4 t[8];
};

__device__ __forceinline__ void state_load(State &S, const void *base, int dt, int wave, int lane)
{
    const int v = 16 * wave + (lane & 15), g = lane >> 4;
    if (dt == kBf16) {
        const uint16_t *p = static_cast<const uint16_t *>(base) + v * kD + 4 * g;
#pragma unroll
        for (int kt = 0; kt < 8; ++kt) {
            const u32x2 x = *reinterpret_cast<const u32x2 *>(p + 16 * kt);
            S.t[kt] = f32x4{lo_f(x[0]), hi_f(x[0]), lo_f(x[1]), hi_f(x[1])};
        }
    } else {
        const float *p = static_cast<const float *>(base) + v * kD + 4 * g;
#pragma unroll
        for (int kt = 0; kt < 8; ++kt)
            S.t[kt] = *reinterpret_cast<const f32x4 *>(p + 16 * kt);
    }
}
__device__ __forceinline__ void state_store(const State &S, void *base, int dt, int wave, int lane)
{
    const int v = 16 * wave + (lane & 15), g = lane >> 4;
    if (dt == kBf16) {
        uint16_t *p = static_cast<uint16_t *>(base) + v * kD + 4 * g;
#pragma unroll
        for (int kt = 0; kt < 8; ++kt)
            *reinterpret_cast<u32x2 *>(p + 16 * kt) =
                u32x2{pack2(S.t[kt][0], S.t[kt][1]), pack2(S.t[kt][2], S.t[kt][3])};
    } else {
        float *p = static_cast<float *>(base) + v * kD + 4 * g;
#pragma unroll
        for (int kt = 0; kt < 8; ++kt)
            *reinterpret_cast<f32x4 *>(p + 16 * kt) = S.t[kt];
    }
}
__device__ __forceinline__ void state_zero(State &S)
{
#pragma unroll
    for (int kt = 0; kt < 8; ++kt)
        S.t[kt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
}
__device__ __forceinline__ void state_one(State &S, int wave, int lane)
{
    const int v = 16 * wave + (lane & 15), g = lane >> 4;
#pragma unroll
    for (int kt = 0; kt < 8; ++kt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            S.t[kt][i] = 16 * kt + 4 * g + i == v ? 1.0f : 0.0f;
}
__device__ __forceinline__ size_t state_size(int dt) { return kGdnStateBytes / (dt == kBf16 ? 2 : 1); }

// ------------------------------------------------------------------------------- LDS
//
// Tiles of 64 tokens x 128 channels are rows of 256 bytes; the 16-byte pieces of a row are XORed with its number, so that
// 16 rows of one piece lie in different banks, whether read along the row or transposed.

constexpr int kTile = kGC * 256;
__device__ __forceinline__ int swz(int row) { return ((row & 7) << 1) | ((row >> 3) & 1); }

struct LdsWalk {
    unsigned char tile[2][3][kTile];  // k, v, q of two chunks
    unsigned char rec[kGdnMat * 2 + kGdnVec + 2048];
};

// A tile's 16 KiB straight into LDS: instruction n of 16 covers rows 4n .. 4n+3, wave w takes n = w and w + 8.
// Rows behind the chunk lie beyond the descriptor and arrive as zeros.
__device__ __forceinline__ void tile_fetch(unsigned char *lds, const GdnTensor &x, const uint16_t *base, int64_t t0, int len,
                                           int wave, int lane)
{
    const uint32_t stride = (uint32_t)x.st * 2;
    const uint32_t bytes = __builtin_amdgcn_readfirstlane((int)(len > 0 ? (uint32_t)(len - 1) * stride + 256u : 0u));
    const __amdgpu_buffer_rsrc_t r = rsrc(base + t0 * x.st, bytes);
    const int row = 4 * wave + (lane >> 4);
    const uint32_t off = (uint32_t)row * stride + (uint32_t)(((lane & 15) ^ swz(row)) << 4);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)(lds + 1024 * wave), 16, off, 0, 0, 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)(lds + 1024 * (wave + 8)), 16, off + 32 * stride, 0, 0, 0);
}
// kParts x 8 KiB of a record
template <int kParts>
__device__ __forceinline__ void rec_fetch(unsigned char *lds, const unsigned char *src, bool on, int wave, int lane)
{
    const __amdgpu_buffer_rsrc_t r = rsrc(src, on ? kParts * 8192u : 0u);
#pragma unroll
    for (int n = 0; n < kParts; ++n)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)(lds + 8192 * n + 1024 * wave), 16,
                                                 (uint32_t)(8192 * n + 1024 * wave + 16 * lane), 0, 0, 0);
}

__device__ __forceinline__ u32x2 lds_b64(const unsigned char *p) { return *reinterpret_cast<const u32x2 *>(p); }
// Transposing read: lane i of each 16 lanes gives the address of 4 channels of token i / 4 and gets channel i of
// the 16 for the 4 tokens.
__device__ __forceinline__ u32x2 lds_tr(const unsigned char *p)
{
    typedef __attribute__((address_space(3))) s16x4 lds_s4;
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)p));
}

// The same for four row tiles of one channel block, and of two.  While loads to LDS are on their way, the compiler waits for all of
// them before the builtin; these blocks wait for their own reads alone.
struct Col4 {
    u32x2 r[4];  // 4 tokens 16 r + 4 g .. each
};
__device__ __forceinline__ uint32_t lds_address(const unsigned char *p)
{
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const unsigned char *)p;
}
__device__ __forceinline__ Col4 lds_tr4(uint32_t at)
{
    Col4 x;
    __asm__ volatile("ds_read_b64_tr_b16 %0, %4\n\t"
                     "ds_read_b64_tr_b16 %1, %4 offset:4096\n\t"
                     "ds_read_b64_tr_b16 %2, %4 offset:8192\n\t"
                     "ds_read_b64_tr_b16 %3, %4 offset:12288\n\t"
                     "s_waitcnt lgkmcnt(0)"
                     : "=&v"(x.r[0]), "=&v"(x.r[1]), "=&v"(x.r[2]), "=&v"(x.r[3])
                     : "v"(at)
                     : "memory");
    return x;
}
__device__ __forceinline__ void lds_tr8(uint32_t at, uint32_t bt, Col4 &x, Col4 &y)
{
    __asm__ volatile("ds_read_b64_tr_b16 %0, %8\n\t"
                     "ds_read_b64_tr_b16 %1, %8 offset:4096\n\t"
                     "ds_read_b64_tr_b16 %2, %8 offset:8192\n\t"
                     "ds_read_b64_tr_b16 %3, %8 offset:12288\n\t"
                     "ds_read_b64_tr_b16 %4, %9\n\t"
                     "ds_read_b64_tr_b16 %5, %9 offset:4096\n\t"
                     "ds_read_b64_tr_b16 %6, %9 offset:8192\n\t"
                     "ds_read_b64_tr_b16 %7, %9 offset:12288\n\t"
                     "s_waitcnt lgkmcnt(0)"
                     : "=&v"(x.r[0]), "=&v"(x.r[1]), "=&v"(x.r[2]), "=&v"(x.r[3]), "=&v"(y.r[0]), "=&v"(y.r[1]),
                       "=&v"(y.r[2]), "=&v"(y.r[3])
                     : "v"(at), "v"(bt)
                     : "memory");
}
__device__ __forceinline__ u32x4 join(u32x2 x, u32x2 y) { return u32x4{x[0], x[1], y[0], y[1]}; }

// This lane's places in a tile; the channel block is XORed in.
struct Lanes {
    int row;  // token lane % 16 of a row tile, channels 4 g .. of 16
    int tr;   // transposing read: tokens 4 g .. of a row tile

    __device__ explicit Lanes(int lane)
    {
        const int m = lane & 15, g = lane >> 4, u = 4 * g + (m >> 2);
        row = m * 256 + (((g >> 1) ^ swz(m)) << 4) + 8 * (g & 1);
        tr = u * 256 + ((((m >> 1) & 1) ^ swz(u)) << 4) + 8 * (m & 1);
    }
};
// 32 channels 32 p .. of the tokens of row tile r: a lane's token is lane % 16
__device__ __forceinline__ u32x4 row_frag(const unsigned char *tile, const Lanes &ln, int r, int p)
{
    const u32x2 x = lds_b64(tile + 4096 * r + (ln.row ^ (64 * p))), y = lds_b64(tile + 4096 * r + (ln.row ^ (64 * p + 32)));
    return u32x4{x[0], x[1], y[0], y[1]};
}
// 4 tokens 16 r + 4 g .. of channel 16 kt + lane % 16
__device__ __forceinline__ u32x2 col_frag4(const unsigned char *tile, const Lanes &ln, int kt, int r)
{
    return lds_tr(tile + 4096 * r + (ln.tr ^ (32 * kt)));
}
// 32 tokens 32 ks .. of channel 16 kt + lane % 16
__device__ __forceinline__ u32x4 col_frag(const unsigned char *tile, const Lanes &ln, int kt, int ks)
{
    const u32x2 x = col_frag4(tile, ln, kt, 2 * ks), y = col_frag4(tile, ln, kt, 2 * ks + 1);
    return u32x4{x[0], x[1], y[0], y[1]};
}
// S += sum over the chunk's tokens of channel rows (tile) times value columns (u), the reads a step ahead of the products
__device__ __forceinline__ void state_add(State &S, const unsigned char *tile, const Lanes &ln, const Terms *u)
{
    const uint32_t at = lds_address(tile);
    Col4 x[2], y[2];
    lds_tr8(at + ln.tr, at + (ln.tr ^ 32), x[0], x[1]);
#pragma unroll
    for (int kt = 0; kt < 8; kt += 2) {
        if (kt < 6)
            lds_tr8(at + (ln.tr ^ (32 * kt + 64)), at + (ln.tr ^ (32 * kt + 96)), y[0], y[1]);
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int n = 0; n < 2; ++n)
                S.t[kt + n] = mfma3(join(x[n].r[2 * ks], x[n].r[2 * ks + 1]), u[ks], S.t[kt + n]);
        x[0] = y[0];
        x[1] = y[1];
    }
}
__device__ __forceinline__ f32x4 widen4(u32x2 x) { return f32x4{lo_f(x[0]), hi_f(x[0]), lo_f(x[1]), hi_f(x[1])}; }
__device__ __forceinline__ f32x4 vec4(const unsigned char *vec, int at)
{
    return *reinterpret_cast<const f32x4 *>(vec + 4 * at);
}
__device__ __forceinline__ Terms block_terms(const unsigned char *mat, int block, int lane)
{
    const u32x4 *p = reinterpret_cast<const u32x4 *>(mat + block * 1024 + lane * 16);
    return Terms{p[0], p[6 * 64], p[12 * 64]};
}

// --------------------------------------------------------------------------- forward walk

constexpr int kModeOut = 0;    // out and final states
constexpr int kModeShare = 1;  // a segment's share of the state at its end (F)
constexpr int kModePhi = 2;    // the transition: from S = 1, without values
constexpr int kModeStore = 3;  // backward pass: the state before each chunk and its residuals

__device__ __forceinline__ void state_scale(State &S, float f)
{
#pragma unroll
    for (int kt = 0; kt < 8; ++kt)
        S.t[kt] *= f;
}

// Sequences without tokens that belong to segment p: the state leaves as it came.  With invalid lengths all of them.
__device__ void empty_states(const GdnArgs &a, const Entry &e0, const Entry &e1, bool valid, int64_t p, int64_t h,
                             const void *init, int init_dt, void *fin, int fin_dt)
{
    if (!a.cu && a.T != 0)
        return;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t lo = !valid ? (p == 0 ? 0 : a.N) : e0.seq, hi = !valid ? a.N : p + 1 == a.P && a.cu ? a.N : e1.seq;
    for (int64_t b = lo; b < hi; b += 512) {
        const int64_t i = b + tid;
        const bool none = i < hi && (!valid || seq_begin(a, i) == seq_begin(a, i + 1));
        if (!__syncthreads_or(none))
            continue;
        for (int64_t n = b; n < b + 512 && n < hi; ++n) {
            if (valid && seq_begin(a, n) != seq_begin(a, n + 1))
                continue;
            State S;
            state_zero(S);
            const int64_t at = n * a.H + h;
            if (init)
                state_load(S, static_cast<const unsigned char *>(init) + at * state_size(init_dt), init_dt, wave, lane);
            state_store(S, static_cast<unsigned char *>(fin) + at * state_size(fin_dt), fin_dt, wave, lane);
        }
    }
}

// rows of a D tile (tokens 16 r + 4 g ..) into column `col` of a 64 x 128 matrix
__device__ __forceinline__ void rows_store(float *m, const f32x4 &x, int r, int g, int col)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        m[(16 * r + 4 * g + i) * kD + col] = x[i];
}

template <int kMode>
__device__ __forceinline__ void walk(const GdnArgs &a, LdsWalk &lds, int64_t row, int64_t p, int64_t h)
{
    constexpr bool kOut = kMode == kModeOut;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int m = lane & 15, g = lane >> 4;
    const int64_t segment = row * a.P + p;
    const bool valid = !a.status || *a.status == 0;
    Entry e0 = entry_of(a, row, p), e1 = entry_of(a, row, p + 1);
    if (!valid) {
        e0 = e1 = Entry{0, 0};
    } else if (kMode == kModeShare || kMode == kModePhi) {  // only the sequence that goes on in the next segment
        if (e1.chunk == 0 || (kMode == kModePhi && (e0.chunk == 0 || e0.seq != e1.seq)))
            return;
        if (e0.seq != e1.seq)
            e0 = Entry{e1.seq, 0};
    }
    if constexpr (kOut)
        if (a.fin && a.fin != a.init)
            empty_states(a, e0, e1, valid, p, h, a.init, a.init_dt, a.fin, a.fin_dt);
    Walk w;
    w.init(e0, e1, false);
    Chunk ch = w.next(a);
    if (ch.len == 0)
        return;
    const Lanes ln(lane);
    auto head_of = [&](const GdnTensor &x) { return head_base(x, row, h); };
    const uint16_t *pk = head_of(a.k), *pv = head_of(a.v), *pq = head_of(a.q);
    constexpr int kParts = kOut ? 5 : 3;
    auto fetch = [&](int buf, const Chunk &n) {
        tile_fetch(lds.tile[buf][0], a.k, pk, n.t0, n.len, wave, lane);
        if constexpr (kMode != kModePhi)
            tile_fetch(lds.tile[buf][1], a.v, pv, n.t0, n.len, wave, lane);
        if constexpr (kOut)
            tile_fetch(lds.tile[buf][2], a.q, pq, n.t0, n.len, wave, lane);
    };
    auto fetch_rec = [&](const Chunk &n) {
        rec_fetch<kParts>(lds.rec, a.rec + ((n.len ? n.slot : 0) * a.H + h) * a.rec_bytes, n.len != 0, wave, lane);
    };
    const unsigned char *mt = lds.rec, *vec = lds.rec + kGdnMat, *ma = vec + kGdnVec;
    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
    State S;
    state_zero(S);
    int buf = 0;
    fetch(0, ch);
    fetch_rec(ch);
    arrive();
    for (;;) {
        const unsigned char *tk = lds.tile[buf][0], *tv = lds.tile[buf][1], *tq = lds.tile[buf][2];
        if (ch.first) {
            if constexpr (kMode == kModePhi) {
                state_one(S, wave, lane);
            } else if (ch.from_seg) {
                if constexpr (kOut || kMode == kModeStore)
                    state_load(S, a.seg + (segment * a.H + h) * kD * kD, 2, wave, lane);
                else
                    state_zero(S);
            } else if (kOut && a.keep && ch.to_seg) {
                state_load(S, a.keep + (segment * a.H + h) * kD * kD, 2, wave, lane);
            } else if (a.init) {
                state_load(S, static_cast<const unsigned char *>(a.init) + (ch.seq * a.H + h) * state_size(a.init_dt),
                           a.init_dt, wave, lane);
                if constexpr (kMode == kModeShare)
                    if (a.keep)
                        state_store(S, a.keep + (segment * a.H + h) * kD * kD, 2, wave, lane);
            } else {
                state_zero(S);
            }
            // here, or the compiler waits behind the branch in every chunk, and for the loads to LDS with it
            __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
        }
        const Chunk nx = w.next(a);
        if constexpr (kMode == kModeStore)
            state_store(S, a.before + (ch.slot * a.H + h) * kD * kD, 2, wave, lane);
        Col4 cv;
        if constexpr (kMode != kModePhi)
            cv = lds_tr4(lds_address(tv) + (ln.tr ^ (32 * wave)));
        f32x4 Z[4], O[4];
        {
            Terms c[4];
#pragma unroll
            for (int x = 0; x < 4; ++x)
                cut8(S.t[2 * x], S.t[2 * x + 1], c[x]);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                Z[r] = O[r] = zero;
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    Z[r] = mfma3(row_frag(tk, ln, r, x), c[x], Z[r]);
                if constexpr (kOut)
#pragma unroll
                    for (int x = 0; x < 4; ++x)  // transposed: rows are value columns, a lane's token is lane % 16
                        O[r] = mfma3(c[x], row_frag(tq, ln, r, x), O[r]);
            }
        }
        arrive();  // this chunk's record is there; the other buffer is read by no one
        fetch(buf ^ 1, nx);
        Terms xr[2];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            f32x4 x[2];
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int r = 2 * ks + hf;
                x[hf] = -vec4(vec, kVHead + 16 * r + 4 * g) * Z[r];
                if constexpr (kMode != kModePhi)
                    x[hf] += widen4(cv.r[r]);
            }
            cut8(x[0], x[1], xr[ks]);
        }
        f32x4 R[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            R[r] = zero;
#pragma unroll
            for (int ks = 0; ks <= r / 2; ++ks)
                R[r] = mfma6(block_terms(mt, low_block(r, ks), lane), xr[ks], R[r]);
        }
        if constexpr (kOut) {
            const float *vo = reinterpret_cast<const float *>(vec) + kVOut;
            Terms rr[2];
            cut8(R[0], R[1], rr[0]);
            cut8(R[2], R[3], rr[1]);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                O[r] *= vo[16 * r + m];
#pragma unroll
                for (int ks = 0; ks <= r / 2; ++ks)
                    O[r] = mfma6(rr[ks], block_terms(ma, low_block(r, ks), lane), O[r]);
            }
        }
        Terms u[2];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
            cut8(R[2 * ks] * vec4(vec, kVWrite + 32 * ks + 4 * g), R[2 * ks + 1] * vec4(vec, kVWrite + 32 * ks + 16 + 4 * g),
                 u[ks]);
        const float carry = *reinterpret_cast<const float *>(vec + 4 * kVLast);
        arrive();  // the next chunk's tiles are there; the record is read by no one
        fetch_rec(nx);
        if constexpr (kOut) {
            const __amdgpu_buffer_rsrc_t ro = rsrc(a.out + ((row * a.T + ch.t0) * a.H + h) * kD,
                                                   (uint32_t)(ch.len - 1) * (uint32_t)a.H * 256u + 256u);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const u32x2 y = {pack2(O[r][0], O[r][1]), pack2(O[r][2], O[r][3])};
                typedef unsigned int u2 __attribute__((vector_size(8)));
                __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u2, y), ro,
                                                      (uint32_t)(16 * r + m) * (uint32_t)a.H * 256u + 32 * wave + 8 * g, 0, 0);
            }
        }
        if constexpr (kMode == kModeStore)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                rows_store(a.res + (ch.slot * a.H + h) * kGC * kD, R[r], r, g, 16 * wave + m);
        state_scale(S, carry);
        state_add(S, tk, ln, u);
        if (kMode != kModeStore && ch.last) {
            if constexpr (kMode == kModeShare)
                state_store(S, a.seg + ((segment + 1) * a.H + h) * kD * kD, 2, wave, lane);
            else if constexpr (kMode == kModePhi)
                state_store(S, a.phi + (segment * a.H + h) * kD * kD, 2, wave, lane);
            else if (a.fin && !ch.to_seg)
                state_store(S, static_cast<unsigned char *>(a.fin) + (ch.seq * a.H + h) * state_size(a.fin_dt), a.fin_dt,
                            wave, lane);
        }
        if (nx.len == 0)
            break;
        ch = nx;
        buf ^= 1;
    }
}

__global__ __launch_bounds__(512, 1) void gdn_out_kernel(GdnArgs a)
{
    extern __shared__ __attribute__((aligned(1024))) unsigned char raw[];
    LdsWalk &lds = *reinterpret_cast<LdsWalk *>(raw);
    const int64_t h = blockIdx.x % a.H, s = blockIdx.x / a.H, row = s / a.P;
    walk<kModeOut>(a, lds, row, s - row * a.P, h);
}
// y = 0: shares, y = 1: transitions
__global__ __launch_bounds__(512, 1) void gdn_cut_kernel(GdnArgs a)
{
    extern __shared__ __attribute__((aligned(1024))) unsigned char raw[];
    LdsWalk &lds = *reinterpret_cast<LdsWalk *>(raw);
    const int64_t h = blockIdx.x % a.H, s = blockIdx.x / a.H, row = s / a.P;
    if (blockIdx.y == 0)
        walk<kModeShare>(a, lds, row, s - row * a.P, h);
    else
        walk<kModePhi>(a, lds, row, s - row * a.P, h);
}

// ----------------------------------------------------------------------------------- scan
//
// State at each cut: S_{p+1} = S_p Phi_p + F_p where segment p lies inside one sequence (else F_p is the state).  A
// workgroup of 8 waves takes 16 value columns of one row and head; wave w forms key channels 16w ..
__global__ __launch_bounds__(512) void gdn_scan_kernel(GdnArgs a)
{
    __shared__ __attribute__((aligned(16))) float st[2][16][132];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, m = lane & 15, g = lane >> 4;
    const int64_t chain = blockIdx.x >> 3, row = chain / a.H, h = chain - row * a.H;
    const int v0 = (int)(blockIdx.x & 7) * 16;
    if (a.status && *a.status != 0)
        return;
    bool have = false;  // st[cur] holds the state at segment p's start
    int cur = 0;
    Entry e = entry_of(a, row, 1);
    for (int64_t p = 1; p + 1 < a.P; ++p) {
        const Entry n = entry_of(a, row, p + 1);
        const bool inside = e.chunk > 0 && n.chunk > 0 && e.seq == n.seq;
        e = n;
        if (!inside) {
            have = false;
            continue;
        }
        const size_t at = ((size_t)(row * a.P + p) * a.H + h) * kD * kD;
        if (!have) {
            __syncthreads();
            const f32x4 x = *reinterpret_cast<const f32x4 *>(a.seg + at + (size_t)(v0 + (tid >> 5)) * kD + (tid & 31) * 4);
            *reinterpret_cast<f32x4 *>(&st[cur][tid >> 5][(tid & 31) * 4]) = x;
            __syncthreads();
        }
        float *next = a.seg + at + (size_t)a.H * kD * kD + (size_t)(v0 + m) * kD + 16 * wave + 4 * g;
        f32x4 acc = *reinterpret_cast<const f32x4 *>(next);
        const float *phi = a.phi + at + 16 * wave + m;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            Terms s, f;
            cut8(*reinterpret_cast<const f32x4 *>(&st[cur][m][32 * x + 4 * g]),
                 *reinterpret_cast<const f32x4 *>(&st[cur][m][32 * x + 16 + 4 * g]), s);
            f32x4 y[2];
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    y[hf][i] = phi[(32 * x + 16 * hf + 4 * g + i) * kD];
            cut8(y[0], y[1], f);
            acc = mfma6(f, s, acc);  // rows: key channels, columns: value columns
        }
        *reinterpret_cast<f32x4 *>(next) = acc;
        cur ^= 1;
        *reinterpret_cast<f32x4 *>(&st[cur][m][16 * wave + 4 * g]) = acc;
        __syncthreads();
        have = true;
    }
}

// -------------------------------------------------------------------------- backward walk
//
// dL/dS from a sequence's end to its start, in the same layout; stores it after each chunk, and dw.

template <bool kShare>
__device__ __forceinline__ void walk_back(const GdnArgs &a, LdsWalk &lds, int64_t row, int64_t p, int64_t h)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int m = lane & 15, g = lane >> 4;
    const int64_t segment = row * a.P + p;
    const bool valid = !a.status || *a.status == 0;
    Entry e0 = entry_of(a, row, p), e1 = entry_of(a, row, p + 1);
    if (!valid) {
        e0 = e1 = Entry{0, 0};
    } else if (kShare) {  // only the sequence that comes from the segment before
        if (e0.chunk == 0)
            return;
        if (e0.seq != e1.seq)
            e1 = Entry{e0.seq + 1, 0};
    }
    if constexpr (!kShare)
        if (a.dinit)
            empty_states(a, e0, e1, valid, p, h, a.dfin, 2, a.dinit, 2);
    Walk w;
    w.init(e0, e1, true);
    Chunk ch = w.next(a);
    if (ch.len == 0)
        return;
    const Lanes ln(lane);
    auto head_of = [&](const GdnTensor &x) { return head_base(x, row, h); };
    const uint16_t *pk = head_of(a.k), *po = head_of(a.dout), *pq = head_of(a.q);
    auto fetch = [&](int buf, const Chunk &n) {
        tile_fetch(lds.tile[buf][0], a.k, pk, n.t0, n.len, wave, lane);
        tile_fetch(lds.tile[buf][1], a.dout, po, n.t0, n.len, wave, lane);
        tile_fetch(lds.tile[buf][2], a.q, pq, n.t0, n.len, wave, lane);
    };
    auto fetch_rec = [&](const Chunk &n) {
        rec_fetch<5>(lds.rec, a.rec + ((n.len ? n.slot : 0) * a.H + h) * a.rec_bytes + kGdnMat, n.len != 0, wave, lane);
    };
    const unsigned char *vec = lds.rec, *mt = vec + kGdnVec, *ma = mt + kGdnMat;
    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
    State S;
    state_zero(S);
    int buf = 0;
    fetch(0, ch);
    fetch_rec(ch);
    arrive();
    for (;;) {
        const unsigned char *tk = lds.tile[buf][0], *to = lds.tile[buf][1], *tq = lds.tile[buf][2];
        if (ch.first) {
            if (ch.from_seg) {
                if constexpr (kShare)
                    state_zero(S);
                else
                    state_load(S, a.dseg + (segment * a.H + h) * kD * kD, 2, wave, lane);
            } else if (a.dfin) {
                state_load(S, a.dfin + (ch.seq * a.H + h) * kD * kD, 2, wave, lane);
            } else {
                state_zero(S);
            }
            // here, or the compiler waits behind the branch in every chunk, and for the loads to LDS with it
            __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
        }
        const Chunk nx = w.next(a);
        if constexpr (!kShare)
            state_store(S, a.dafter + (ch.slot * a.H + h) * kD * kD, 2, wave, lane);
        const Col4 co = lds_tr4(lds_address(to) + (ln.tr ^ (32 * wave)));
        f32x4 Y[4];
        {
            Terms c[4];
#pragma unroll
            for (int x = 0; x < 4; ++x)
                cut8(S.t[2 * x], S.t[2 * x + 1], c[x]);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                Y[r] = zero;
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    Y[r] = mfma3(row_frag(tk, ln, r, x), c[x], Y[r]);
            }
        }
        arrive();  // this chunk's record is there; the other buffer is read by no one
        fetch(buf ^ 1, nx);
        const u32x4 o[2] = {join(co.r[0], co.r[1]), join(co.r[2], co.r[3])};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            Y[r] *= vec4(vec, kVTail + 16 * r + 4 * g);
#pragma unroll
            for (int ks = r / 2; ks < 2; ++ks)
                Y[r] = mfma3(block_terms(ma, up_block(r, ks), lane), o[ks], Y[r]);
        }
        Terms d[2];
        cut8(Y[0], Y[1], d[0]);
        cut8(Y[2], Y[3], d[1]);
        f32x4 W[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            W[r] = zero;
#pragma unroll
            for (int ks = r / 2; ks < 2; ++ks)
                W[r] = mfma6(block_terms(mt, up_block(r, ks), lane), d[ks], W[r]);
        }
        // what the tokens' reads and writes send to the state before the chunk
        Terms uo[2], uw[2];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            f32x4 x[2], y[2];
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int at = 32 * ks + 16 * hf + 4 * g;
                x[hf] = widen4(u32x2{o[ks][2 * hf], o[ks][2 * hf + 1]}) * vec4(vec, kVOut + at);
                y[hf] = -(W[2 * ks + hf] * (vec4(vec, kVBeta + at) * vec4(vec, kVHead + at)));
            }
            cut8(x[0], x[1], uo[ks]);
            cut8(y[0], y[1], uw[ks]);
        }
        const float carry = *reinterpret_cast<const float *>(vec + 4 * kVLast);
        arrive();  // the next chunk's tiles are there; the record is read by no one
        fetch_rec(nx);
        if constexpr (!kShare)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                rows_store(a.dwrite + (ch.slot * a.H + h) * kGC * kD, W[r], r, g, 16 * wave + m);
        state_scale(S, carry);
        state_add(S, tq, ln, uo);
        state_add(S, tk, ln, uw);
        if (ch.last) {
            if constexpr (kShare)
                state_store(S, a.dseg + ((segment - 1) * a.H + h) * kD * kD, 2, wave, lane);
            else if (a.dinit && !ch.to_seg)
                state_store(S, a.dinit + (ch.seq * a.H + h) * kD * kD, 2, wave, lane);
        }
        if (nx.len == 0)
            break;
        ch = nx;
        buf ^= 1;
    }
}

__global__ __launch_bounds__(512, 1) void gdn_store_kernel(GdnArgs a)
{
    extern __shared__ __attribute__((aligned(1024))) unsigned char raw[];
    LdsWalk &lds = *reinterpret_cast<LdsWalk *>(raw);
    const int64_t h = blockIdx.x % a.H, s = blockIdx.x / a.H, row = s / a.P;
    walk<kModeStore>(a, lds, row, s - row * a.P, h);
}
template <bool kShare>
__global__ __launch_bounds__(512, 1) void gdn_back_kernel(GdnArgs a)
{
    extern __shared__ __attribute__((aligned(1024))) unsigned char raw[];
    LdsWalk &lds = *reinterpret_cast<LdsWalk *>(raw);
    const int64_t h = blockIdx.x % a.H, s = blockIdx.x / a.H, row = s / a.P;
    walk_back<kShare>(a, lds, row, s - row * a.P, h);
}

// dL/dS at each cut, from the last to the first: dS_{p-1} = dS_p Phi_p^T + share, as gdn_scan_kernel.
__global__ __launch_bounds__(512) void gdn_scan_back_kernel(GdnArgs a)
{
    __shared__ __attribute__((aligned(16))) float st[2][16][132];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, m = lane & 15, g = lane >> 4;
    const int64_t chain = blockIdx.x >> 3, row = chain / a.H, h = chain - row * a.H;
    const int v0 = (int)(blockIdx.x & 7) * 16;
    if (a.status && *a.status != 0)
        return;
    bool have = false;  // st[cur] holds dL/dS at segment p's end
    int cur = 0;
    Entry e = entry_of(a, row, a.P - 1);
    for (int64_t p = a.P - 2; p > 0; --p) {
        const Entry n = e;
        e = entry_of(a, row, p);
        if (!(e.chunk > 0 && n.chunk > 0 && e.seq == n.seq)) {
            have = false;
            continue;
        }
        const size_t at = ((size_t)(row * a.P + p) * a.H + h) * kD * kD;
        if (!have) {
            __syncthreads();
            const f32x4 x = *reinterpret_cast<const f32x4 *>(a.dseg + at + (size_t)(v0 + (tid >> 5)) * kD + (tid & 31) * 4);
            *reinterpret_cast<f32x4 *>(&st[cur][tid >> 5][(tid & 31) * 4]) = x;
            __syncthreads();
        }
        float *next = a.dseg + at - (size_t)a.H * kD * kD + (size_t)(v0 + m) * kD + 16 * wave + 4 * g;
        f32x4 acc = *reinterpret_cast<const f32x4 *>(next);
        const float *phi = a.phi + at + (16 * wave + m) * kD + 4 * g;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            Terms s, f;
            cut8(*reinterpret_cast<const f32x4 *>(&st[cur][m][32 * x + 4 * g]),
                 *reinterpret_cast<const f32x4 *>(&st[cur][m][32 * x + 16 + 4 * g]), s);
            cut8(*reinterpret_cast<const f32x4 *>(phi + 32 * x), *reinterpret_cast<const f32x4 *>(phi + 32 * x + 16), f);
            acc = mfma6(f, s, acc);
        }
        *reinterpret_cast<f32x4 *>(next) = acc;
        cur ^= 1;
        *reinterpret_cast<f32x4 *>(&st[cur][m][16 * wave + 4 * g]) = acc;
        __syncthreads();
        have = true;
    }
}

// ------------------------------------------------------------------- gradients of a chunk
//
// One workgroup of 8 waves per (chunk, head).  w = beta r and dx = beta dw are cut into bf16 terms once, in LDS.  Wave w
// forms key channels 16w .. of dq and dk for all 64 tokens (rows: channels, a lane's token is lane % 16), and one 16 x 32
// block each of P, P^T and G + G^T, which pass through LDS to the other waves in the place of the terms.

struct LdsGrad {
    unsigned char k[kTile], q[kTile], o[kTile];
    unsigned char w[3][kTile], x[3][kTile];  // terms of w and dx; then the blocks of P, P^T, G + G^T
    float vec[kGdnVec / 4];
    float sums[8][kGC];   // q.dq of each wave's channels
    float vdv[kGC];
    float end[8];         // <dS, S_after>, a wave's share
};

__device__ __forceinline__ Terms row_terms(const unsigned char (*t)[kTile], const Lanes &ln, int r, int p)
{
    return Terms{row_frag(t[0], ln, r, p), row_frag(t[1], ln, r, p), row_frag(t[2], ln, r, p)};
}

__global__ __launch_bounds__(512, 1) void gdn_grad_kernel(GdnArgs a)
{
    __shared__ __attribute__((aligned(1024))) LdsGrad s;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int m = lane & 15, g = lane >> 4;
    const int64_t slot = blockIdx.x / a.H, h = blockIdx.x - slot * a.H;
    if (a.status && *a.status != 0)
        return;
    const int64_t seq = last_at_most(a.N, slot, [&](int64_t i) { return slot_of(uniform(seq_begin(a, i)), i); });
    const int64_t begin = uniform(seq_begin(a, seq)), c = slot - slot_of(begin, seq),
                  rest = uniform(seq_begin(a, seq + 1)) - begin - c * kGC;
    if (rest <= 0)
        return;
    const int len = (int)(rest < kGC ? rest : kGC);
    const int64_t row = a.cu ? 0 : seq, t0 = (a.cu ? begin : 0) + c * kGC, at = slot * a.H + h;
    const int64_t tok0 = row * a.T + t0;
    auto head_of = [&](const GdnTensor &x) { return head_base(x, row, h); };
    tile_fetch(s.k, a.k, head_of(a.k), t0, len, wave, lane);
    tile_fetch(s.q, a.q, head_of(a.q), t0, len, wave, lane);
    tile_fetch(s.o, a.dout, head_of(a.dout), t0, len, wave, lane);
    if (wave < 2)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc(a.rec + at * a.rec_bytes + kGdnMat, kGdnVec),
                                                 (lds_void *)(s.vec + 256 * wave), 16, 1024 * wave + 16 * lane, 0, 0, 0);
    // the states' columns of this wave: lane = key channel, 4 value rows 16 n + 4 g ..
    const float *sb = a.before + at * kD * kD + 16 * wave + m, *sd = a.dafter + at * kD * kD + 16 * wave + m;
    f32x4 S[8], dS[8];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            S[n][i] = sb[(16 * n + 4 * g + i) * kD];
    // rows of r and dw: thread = token tid / 8, value channels 16 (tid % 8) ..
    {
        const int t = tid >> 3, v0 = 16 * (tid & 7);
        const float *pr = a.res + at * kGC * kD + t * kD + v0, *pw = a.dwrite + at * kGC * kD + t * kD + v0;
        const float be = t < len ? a.beta[(tok0 + t) * a.H + h] : 0.0f;
        const uint16_t *pv = head_of(a.v) + (t0 + (t < len ? t : 0)) * a.v.st + v0;
        const u32x4 vv[2] = {*reinterpret_cast<const u32x4 *>(pv), *reinterpret_cast<const u32x4 *>(pv + 8)};
        float db = 0.0f, vd = 0.0f;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            f32x4 r[2], d[2], x[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                r[e] = *reinterpret_cast<const f32x4 *>(pr + 8 * hf + 4 * e);
                d[e] = *reinterpret_cast<const f32x4 *>(pw + 8 * hf + 4 * e);
                x[e] = d[e] * be;
                const f32x4 v4 = widen4(u32x2{vv[hf][2 * e], vv[hf][2 * e + 1]});
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    db = fmaf(d[e][i], r[e][i], db);
                    vd = fmaf(x[e][i], v4[i], vd);
                }
                r[e] *= be;
            }
            const int piece = 2 * (tid & 7) + hf, to = t * 256 + ((piece ^ swz(t)) << 4);
            Terms y;
            cut8(r[0], r[1], y);
            *reinterpret_cast<u32x4 *>(s.w[0] + to) = y.h;
            *reinterpret_cast<u32x4 *>(s.w[1] + to) = y.m;
            *reinterpret_cast<u32x4 *>(s.w[2] + to) = y.l;
            cut8(x[0], x[1], y);
            *reinterpret_cast<u32x4 *>(s.x[0] + to) = y.h;
            *reinterpret_cast<u32x4 *>(s.x[1] + to) = y.m;
            *reinterpret_cast<u32x4 *>(s.x[2] + to) = y.l;
            if (t < len)
                *reinterpret_cast<u32x4 *>(a.dv + ((tok0 + t) * a.H + h) * kD + v0 + 8 * hf) = y.h;
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) {
            db += __shfl_xor(db, o);
            vd += __shfl_xor(vd, o);
        }
        if ((tid & 7) == 0) {
            s.vdv[t] = vd;
            if (t < len)
                a.dbeta[(tok0 + t) * a.H + h] = db;
        }
    }
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            dS[n][i] = sd[(16 * n + 4 * g + i) * kD];
    arrive();
    const Lanes ln(lane);
    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
    // the states' shares
    f32x4 dq[4], dk[4];
    float dot = 0.0f;
    {
        Terms cs[4];
#pragma unroll
        for (int x = 0; x < 4; ++x)
            cut8(S[2 * x], S[2 * x + 1], cs[x]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            dq[r] = dk[r] = zero;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                dq[r] = mfma3(cs[x], row_frag(s.o, ln, r, x), dq[r]);
                dk[r] = mfma6(cs[x], row_terms(s.x, ln, r, x), dk[r]);
            }
            dq[r] *= s.vec[kVOut + 16 * r + m];
            dk[r] *= -s.vec[kVHead + 16 * r + m];
        }
    }
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            dot = fmaf(S[n][i], dS[n][i], dot);
    dot *= s.vec[kVLast];
    // channels 16 w + 4 g .. of token 16 r + m
    auto mine = [&](const unsigned char *tile, int r) {
        return widen4(lds_b64(tile + 4096 * r + (ln.row ^ (32 * wave))));
    };
    {
        Terms cs[4];
#pragma unroll
        for (int x = 0; x < 4; ++x)
            cut8(dS[2 * x], dS[2 * x + 1], cs[x]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            f32x4 y = zero;
#pragma unroll
            for (int x = 0; x < 4; ++x)
                y = mfma6(cs[x], row_terms(s.w, ln, r, x), y);
            y *= s.vec[kVTail + 16 * r + m];
            const f32x4 k4 = mine(s.k, r);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                dot = fmaf(y[i], k4[i], dot);
            dk[r] += y;
        }
    }
    // blocks of this wave: columns of tile cr, contraction 32 ck ..
    const int cr = wave >> 1, ck = wave & 1;
    auto within = [&](int t, int u) {  // e^{b_t - b_u} for u <= t
        const float d = (s.vec[kVSum + t] - s.vec[kVSum + u]) + (s.vec[kVSum + 64 + t] - s.vec[kVSum + 64 + u]);
        return u <= t ? __builtin_amdgcn_exp2f(d) : 0.0f;
    };
    Terms pa, pb, gs;
    {
        const int col = 16 * cr + m;
        f32x4 fa[2], fb[2], fg[2];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int rt = 2 * ck + hf;  // row tile
            f32x4 ya = zero, yb = zero, g1 = zero, g2 = zero;
            if (rt <= cr) {  // rows are sources, columns out tokens
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const Terms wt = row_terms(s.w, ln, rt, x);
                    ya = mfma3(wt, row_frag(s.o, ln, cr, x), ya);
                    g1 = mfma6(wt, row_terms(s.x, ln, cr, x), g1);
                }
            }
            if (rt >= cr) {  // rows are out tokens, columns sources
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const Terms wt = row_terms(s.w, ln, cr, x);
                    yb = mfma3(row_frag(s.o, ln, rt, x), wt, yb);
                    g2 = mfma6(row_terms(s.x, ln, rt, x), wt, g2);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int rw = 16 * rt + 4 * g + i;
                const float lo = within(col, rw), hi = within(rw, col);
                fa[hf][i] = rw <= col ? a.scale * lo * ya[i] : 0.0f;
                fb[hf][i] = rw >= col ? a.scale * hi * yb[i] : 0.0f;
                fg[hf][i] = rw < col ? -lo * g1[i] : rw > col ? -hi * g2[i] : 0.0f;
            }
        }
        cut8(fa[0], fa[1], pa);
        cut8(fb[0], fb[1], pb);
        cut8(fg[0], fg[1], gs);
    }
    __syncthreads();  // the terms of w and dx are read by no one
    unsigned char *mp = s.w[0], *mq = mp + 8 * 3 * 1024, *mg = mq + 8 * 3 * 1024;  // 72 KiB of their 96
    auto put = [&](unsigned char *mat, const Terms &t) {
        u32x4 *p = reinterpret_cast<u32x4 *>(mat + wave * 3072 + lane * 16);
        p[0] = t.h;
        p[64] = t.m;
        p[128] = t.l;
    };
    put(mp, pa);
    put(mq, pb);
    put(mg, gs);
    __syncthreads();
    auto block = [&](const unsigned char *mat, int r, int ks) {
        const u32x4 *p = reinterpret_cast<const u32x4 *>(mat + (2 * r + ks) * 3072 + lane * 16);
        return Terms{p[0], p[64], p[128]};
    };
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
        const u32x4 kc = col_frag(s.k, ln, wave, ks), qc = col_frag(s.q, ln, wave, ks);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if (ks <= r / 2)
                dq[r] = mfma3(kc, block(mp, r, ks), dq[r]);
            if (ks >= r / 2)
                dk[r] = mfma3(qc, block(mq, r, ks), dk[r]);
            dk[r] = mfma3(kc, block(mg, r, ks), dk[r]);
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const f32x4 q4 = mine(s.q, r);
        float y = dq[r][0] * q4[0];
#pragma unroll
        for (int i = 1; i < 4; ++i)
            y = fmaf(dq[r][i], q4[i], y);
        y += __shfl_xor(y, 16);
        y += __shfl_xor(y, 32);
        if (g == 0)
            s.sums[wave][16 * r + m] = y;
        const int t = 16 * r + m;
        if (t < len) {
            const int64_t to = ((tok0 + t) * a.H + h) * kD + 16 * wave + 4 * g;
            if (a.dq_h) {
                *reinterpret_cast<f32x4 *>(a.dq_h + to) = dq[r];
                *reinterpret_cast<f32x4 *>(a.dk_h + to) = dk[r];
            } else {
                *reinterpret_cast<u32x2 *>(a.dq + to) = u32x2{pack2(dq[r][0], dq[r][1]), pack2(dq[r][2], dq[r][3])};
                *reinterpret_cast<u32x2 *>(a.dk + to) = u32x2{pack2(dk[r][0], dk[r][1]), pack2(dk[r][2], dk[r][3])};
            }
        }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        dot += __shfl_xor(dot, o);
    if (lane == 0)
        s.end[wave] = dot;
    __syncthreads();
    if (wave != 0)
        return;
    float qd = 0.0f, end = 0.0f;
#pragma unroll
    for (int n = 0; n < 8; ++n) {
        qd += s.sums[n][lane];
        end += s.end[n];
    }
    const double each = lane < len ? (double)qd - (double)s.vdv[lane] : 0.0;
    const double upto = running_sum(each), total = last_lane(upto);  // by all lanes, those behind the chunk too
    if (lane < len) {
        const int64_t to = (tok0 + lane) * a.H + h;
        const float gd = a.decay[to];
        a.ddecay[to] = gd > kLowest && gd <= 0.0f ? (float)((total - upto) + each + (double)end) : 0.0f;
    }
}

// ------------------------------------------------------------------------- cu_seqlens

// The walks trust cu_seqlens, so nothing may run on one that leads out of the tensors.
__global__ __launch_bounds__(1024) void gdn_check_kernel(const int64_t *cu, int64_t N, int64_t T, int32_t *status)
{
    __shared__ int bits;
    if (threadIdx.x == 0)
        bits = (cu[0] != 0 ? 1 : 0) | (cu[N] != T ? 4 : 0);
    __syncthreads();
    int mine = 0;
    for (int64_t n = threadIdx.x; n < N; n += 1024)
        if (cu[n + 1] < cu[n])
            mine = 2;
    if (mine)
        atomicOr(&bits, mine);
    __syncthreads();
    if (threadIdx.x == 0)
        *status = bits;
}

// ------------------------------------------------------------------- token by token
//
// One wave per (sequence, head, 32 rows of the state); lane = row % 8 * 8 + q holds 16 channels of 4 rows: 16-byte
// pieces, interleaved with those of the row's other 7 lanes.  S q = S~ q + beta r (k.q), so one pass over the row
// gives both dot products.  The state is read once and written once, which bounds it.
template <bool kF32>
__global__ __launch_bounds__(256) void gdn_recurrent_kernel(GdnArgs a)
{
    constexpr int kPer = kF32 ? 4 : 8;     // channels per 16-byte piece
    constexpr int kPieces = 16 / kPer;     // pieces per row and lane
    const int lane = threadIdx.x & 63;
    const int64_t unit = (int64_t)blockIdx.x * (blockDim.x >> 6) + (threadIdx.x >> 6);
    const int64_t chain = unit >> 2;
    if (chain >= a.N * a.H)
        return;
    const int v0 = (int)(unit & 3) * 32, r8 = lane >> 3, q8 = lane & 7;
    const int64_t seq = chain / a.H, h = chain - seq * a.H;
    float S[4][16];
    const size_t mat = (size_t)chain * kD * kD;
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            const size_t at = mat + (size_t)(v0 + 8 * n + r8) * kD + (8 * p + q8) * kPer;
            if (!a.init) {
#pragma unroll
                for (int e = 0; e < kPer; ++e)
                    S[n][p * kPer + e] = 0.0f;
            } else if constexpr (kF32) {
                const f32x4 x = *reinterpret_cast<const f32x4 *>(static_cast<const float *>(a.init) + at);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    S[n][p * 4 + e] = x[e];
            } else {
                const u32x4 x = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(a.init) + at);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    S[n][p * 8 + 2 * e] = lo_f(x[e]);
                    S[n][p * 8 + 2 * e + 1] = hi_f(x[e]);
                }
            }
        }
    int64_t row = seq, t0 = 0, t1 = a.T;
    if (a.cu) {
        row = 0;
        t0 = t1 = 0;
        if (*a.status == 0) {
            t0 = a.cu[seq];
            t1 = a.cu[seq + 1];
        }
    }
    auto sum8 = [](float x) {
#pragma unroll
        for (int o = 4; o > 0; o >>= 1)
            x += __shfl_xor(x, o);
        return x;
    };
    for (int64_t t = t0; t < t1; ++t) {
        const uint16_t *qp = a.q.p + row * a.q.sb + t * a.q.st + (h / a.q.share) * a.q.sh;
        const uint16_t *kp = a.k.p + row * a.k.sb + t * a.k.st + (h / a.k.share) * a.k.sh;
        const uint16_t *vp = a.v.p + row * a.v.sb + t * a.v.st + (h / a.v.share) * a.v.sh;
        const int64_t tok = row * a.T + t;
        const float al = __builtin_amdgcn_exp2f((float)((double)clamp_decay(a.decay[tok * a.H + h]) * kLog2e64));
        const float be = a.beta[tok * a.H + h];
        float qv[16], kv[16], o[4];
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            const int ch = (8 * p + q8) * kPer;
#pragma unroll
            for (int e = 0; e < kPer; e += 4) {
                const f32x4 x = widen4(*reinterpret_cast<const u32x2 *>(qp + ch + e));
                const f32x4 y = widen4(*reinterpret_cast<const u32x2 *>(kp + ch + e));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    qv[p * kPer + e + i] = x[i];
                    kv[p * kPer + e + i] = y[i];
                }
            }
        }
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const float vv = __uint_as_float((uint32_t)vp[v0 + 8 * n + r8] << 16);
            float sk = 0.0f, sq = 0.0f;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                S[n][e] *= al;
                sk = fmaf(S[n][e], kv[e], sk);
            }
            const float u = be * (vv - sum8(sk));
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                S[n][e] = fmaf(u, kv[e], S[n][e]);
                sq = fmaf(S[n][e], qv[e], sq);
            }
            o[n] = sum8(sq) * a.scale;
        }
        const float mine = q8 == 0 ? o[0] : q8 == 1 ? o[1] : q8 == 2 ? o[2] : o[3];
        if (q8 < 4)
            a.out[(tok * a.H + h) * kD + v0 + 8 * q8 + r8] = __builtin_bit_cast(uint16_t, (__bf16)mine);
    }
    if (!a.fin)
        return;
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            const size_t at = mat + (size_t)(v0 + 8 * n + r8) * kD + (8 * p + q8) * kPer;
            if constexpr (kF32) {
                *reinterpret_cast<f32x4 *>(static_cast<float *>(a.fin) + at) =
                    f32x4{S[n][p * 4], S[n][p * 4 + 1], S[n][p * 4 + 2], S[n][p * 4 + 3]};
            } else {
                u32x4 x;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[e] = pack2(S[n][p * 8 + 2 * e], S[n][p * 8 + 2 * e + 1]);
                *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(a.fin) + at) = x;
            }
        }
}

hipError_t launch_check(const GdnArgs &a, int32_t *status, hipStream_t s)
{
    if (a.cu)
        hipLaunchKernelGGL(gdn_check_kernel, dim3(1), dim3(1024), 0, s, a.cu, a.N, a.T, status);
    return hipGetLastError();
}

}  // namespace

hipError_t gdn_launch_fwd(const GdnArgs &a, int32_t *status, hipStream_t s)
{
    hipError_t e = launch_check(a, status, s);
    if (e == hipSuccess && a.T > 0) {
        hipLaunchKernelGGL(gdn_prep_kernel<false>, dim3((unsigned)(a.slots * a.H)), dim3(256), 0, s, a);
        e = hipGetLastError();
    }
    const unsigned grid = (unsigned)(a.rows * a.P * a.H);
    if (e == hipSuccess && a.P > 1) {
        hipLaunchKernelGGL(gdn_cut_kernel, dim3(grid, 2), dim3(512), sizeof(LdsWalk), s, a);
        e = hipGetLastError();
        if (e == hipSuccess && a.P > 2) {
            hipLaunchKernelGGL(gdn_scan_kernel, dim3((unsigned)(8 * a.rows * a.H)), dim3(512), 0, s, a);
            e = hipGetLastError();
        }
    }
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL(gdn_out_kernel, dim3(grid), dim3(512), sizeof(LdsWalk), s, a);
    return hipGetLastError();
}

hipError_t gdn_launch_bwd(const GdnArgs &a, int32_t *status, hipStream_t s)
{
    hipError_t e = launch_check(a, status, s);
    if (e != hipSuccess)
        return e;
    const unsigned grid = (unsigned)(a.rows * a.P * a.H), recs = (unsigned)(a.slots * a.H);
    if (a.T > 0) {
        hipLaunchKernelGGL(gdn_prep_kernel<true>, dim3(recs), dim3(256), 0, s, a);
        if (a.P > 1) {
            hipLaunchKernelGGL(gdn_cut_kernel, dim3(grid, 2), dim3(512), sizeof(LdsWalk), s, a);
            if (a.P > 2)
                hipLaunchKernelGGL(gdn_scan_kernel, dim3((unsigned)(8 * a.rows * a.H)), dim3(512), 0, s, a);
            hipLaunchKernelGGL(gdn_back_kernel<true>, dim3(grid), dim3(512), sizeof(LdsWalk), s, a);
            if (a.P > 2)
                hipLaunchKernelGGL(gdn_scan_back_kernel, dim3((unsigned)(8 * a.rows * a.H)), dim3(512), 0, s, a);
        }
        hipLaunchKernelGGL(gdn_store_kernel, dim3(grid), dim3(512), sizeof(LdsWalk), s, a);
    }
    hipLaunchKernelGGL(gdn_back_kernel<false>, dim3(grid), dim3(512), sizeof(LdsWalk), s, a);
    if (a.T > 0)
        hipLaunchKernelGGL(gdn_grad_kernel, dim3(recs), dim3(512), 0, s, a);
    e = hipGetLastError();
    if (e != hipSuccess || !a.dq_h || a.T == 0)
        return e;
    return lin_launch_fold(a.dq_h, a.dk_h, a.dq, a.dk, (a.cu ? 1 : a.N) * a.T, a.Hk, a.H / a.Hk, a.status, s);
}

hipError_t gdn_launch_recurrent(const GdnArgs &a, int32_t *status, hipStream_t s)
{
    const hipError_t e = launch_check(a, status, s);
    if (e != hipSuccess)
        return e;
    const int64_t units = a.N * a.H * 4;
    const bool f32 = (a.init ? a.init_dt : a.fin_dt) != kBf16;
    const int threads = units < 4096 ? 64 : 256;
    const unsigned grid = (unsigned)cdiv(units, threads / 64);
    if (f32)
        hipLaunchKernelGGL(gdn_recurrent_kernel<true>, dim3(grid), dim3(threads), 0, s, a);
    else
        hipLaunchKernelGGL(gdn_recurrent_kernel<false>, dim3(grid), dim3(threads), 0, s, a);
    return hipGetLastError();
}

}  // namespace kda
