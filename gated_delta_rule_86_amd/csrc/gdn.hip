// gdn.hip -- gated delta rule with a decay for each head, gfx950.
//
// Per (sequence, head), state S [V = 128][K = 128], natural-log decay g_t <= 0, write strength beta_t:
//   S~ = e^{g_t} S_{t-1},   r_t = v_t - S~ k_t,   S_t = S~ + beta_t r_t k_t^T,   out_t = scale * S_t q_t.
// In chunks of C = 32 tokens, with b the inclusive running sum of g inside the chunk, L its last entry and
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
//   dg_t = <dS~_t, S~_t>, the sum of all that crosses the token:
//     e^{L} <dS, S> + sum_{s < t} tail_s w_s.(dS k_s) + sum_{u >= t} e^{b_u} (scale dO_u.(S q_u) - dx_u.(S k_u))
//     + sum_{s < t <= u} (P_us q_u.k_s + G_us k_u.k_s).
// Every term has e^{g_t} in it and none is taken away again, so dg_t is as exact where a head forgets as where it remembers.
// (The sums of q_u.dq_u - v_u.dv_u over u >= t are the same in exact arithmetic, but hold the token's own read and write,
// which e^{g_t} does not scale: in fp32 nothing is left of dg_t below g_t = -16.)
//
// Numbers: decays are used as min(max(g, -1000), 0); running sums of logarithms are fp64, a factor is the
// exponential of a difference and at most 1.  The products run on bf16 MFMA with fp32 accumulation; q, k, v are
// bf16 as they come, every other factor is cut into three bf16 terms, hi + mid + lo: the 24 bits of fp32.
//
// Passes: prep forms each chunk's triangular matrices; the cut walks each segment's share of the state at its end and its
// transition, the scan the states there (few rows: the chip has room for 512 walks); the output walk starts from them.
// Backwards the store walk keeps the state before each block of 64 tokens, the back walk its gradient behind it, and the
// gradients of the blocks follow from the two.  Times below are of B=2 T=4096 H=16 (a), 38350 packed tokens H=32 Hk=16 (b) and
// T=65536 H=8 (c), on a card at speed (after some 30 passes), with the decays that such models start training from: two thirds of the
// heads forget within a segment, and their transitions and most of their shares are left out.  Where every head remembers, the
// cut takes 70 us for 62 in (a), 569 for 289 in (b), 256 for 167 in (c), and each scan a fifth more.
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gdn_internal.h"
#include "lin_internal.h"

namespace kda {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

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


// The order of a product's contraction is free as long as both operands agree.
//
// v_mfma_f32_32x32x16_bf16: A[m][k] in lane m + 32*(k/8), element k%8; B[k][n] in lane n + 32*(k/8), element k%8;
// D[m][n] in lane n + 32*((m/4)%2), element 4*(m/8) + m%4.  Elements 8s .. 8s+7 of a D tile are the operand of a
// contraction over its rows 16s .. 16s+15 in the order 4h + j (j < 4), 8 + 4h + j - 4, with h = lane / 32.
__device__ __forceinline__ f32x16 mfma(u32x4 a, u32x4 b, f32x16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                   0);
}
// v_mfma_f32_16x16x32_bf16: lanes as above with 16 for 32; D[m][n] in lane n + 16*(m/4), element m%4: two tiles are the
// operand of a contraction over their 32 rows.
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
// Cuts: x = h + m + l exactly, towards 0 (cut2, cut8) or to the nearest (cut2n, cut8n).  A product with a bf16 factor is whole either
// way.  mfma6 leaves out m l + l m + l l of two cut factors, relative to the product (normal factors): both towards 0 2^-24.0 root mean
// square and 2^-21 at most, always on the side of 0; one of them to the nearest 2^-25.7 and 2^-22.4, both 2^-27.4 and 2^-24, on
// no side (a rounded fp32 product: 2^-25.2).  So one at least is: both where that costs nothing, in the walks the record's alone (the
// other too makes the calls 1 to 2 % longer: v_cvt_pk_bf16_f32 for v_perm_b32).
// Two floats into word e of each term: the upper 16 bits, those of what they leave, and the rest, which has 8 bits.
__device__ __forceinline__ void cut2(float x, float y, Terms &t, int e)
{
    constexpr uint32_t kUpper = 0x07060302u;  // the upper halves of two words
    const uint32_t a = __float_as_uint(x), b = __float_as_uint(y);
    t.h[e] = __builtin_amdgcn_perm(b, a, kUpper);
    const float x1 = x - __uint_as_float(a & 0xffff0000u), y1 = y - __uint_as_float(b & 0xffff0000u);
    const uint32_t a1 = __float_as_uint(x1), b1 = __float_as_uint(y1);
    t.m[e] = __builtin_amdgcn_perm(b1, a1, kUpper);
    const float x2 = x1 - __uint_as_float(a1 & 0xffff0000u), y2 = y1 - __uint_as_float(b1 & 0xffff0000u);
    t.l[e] = __builtin_amdgcn_perm(__float_as_uint(y2), __float_as_uint(x2), kUpper);
}
__device__ __forceinline__ Terms cut8(f32x4 a, f32x4 b)
{
    Terms t;
    cut2(a[0], a[1], t, 0);
    cut2(a[2], a[3], t, 1);
    cut2(b[0], b[1], t, 2);
    cut2(b[2], b[3], t, 3);
    return t;
}
__device__ __forceinline__ Terms cut8(const f32x16 &x, int s)
{
    Terms t;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        cut2(x[8 * s + 2 * e], x[8 * s + 2 * e + 1], t, e);
    return t;
}
// Two floats into word e of each term: the nearest bf16 value, that of what it leaves, and the rest, which has 8 bits with its sign.
__device__ __forceinline__ void cut2n(float x, float y, Terms &t, int e)
{
    t.h[e] = pack2(x, y);
    const float x1 = x - lo_f(t.h[e]), y1 = y - hi_f(t.h[e]);
    t.m[e] = pack2(x1, y1);
    t.l[e] = pack2(x1 - lo_f(t.m[e]), y1 - hi_f(t.m[e]));
}
__device__ __forceinline__ Terms cut8n(f32x4 a, f32x4 b)
{
    Terms t;
    cut2n(a[0], a[1], t, 0);
    cut2n(a[2], a[3], t, 1);
    cut2n(b[0], b[1], t, 2);
    cut2n(b[2], b[3], t, 3);
    return t;
}
__device__ __forceinline__ Terms cut8n(const f32x16 &x, int s)
{
    Terms t;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        cut2n(x[8 * s + 2 * e], x[8 * s + 2 * e + 1], t, e);
    return t;
}
// products with an exact factor, and of two cut factors (one at least to the nearest)
template <typename D>
__device__ __forceinline__ D mfma3(u32x4 a, const Terms &b, D c)
{
    c = mfma(a, b.l, c);
    c = mfma(a, b.m, c);
    return mfma(a, b.h, c);
}
template <typename D>
__device__ __forceinline__ D mfma3(const Terms &a, u32x4 b, D c)
{
    c = mfma(a.l, b, c);
    c = mfma(a.m, b, c);
    return mfma(a.h, b, c);
}
template <typename D>
__device__ __forceinline__ D mfma6(const Terms &a, const Terms &b, D c)
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

// 16 bytes a lane straight into LDS, 1 KiB from `lds` on in the order of the lanes.  In assembly, because the compiler would
// wait for all such loads before each transposing read of LDS; arrive() waits for them.  No register is written.
__device__ __forceinline__ void load_lds(const void *base, uint32_t bytes, uint32_t off, uint32_t lds)
{
    const uint64_t p = (uint64_t)(uintptr_t)base;
    const u32x4 r = {(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)p),
                     (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(p >> 32)) & 0xffffu,
                     (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes), 0x00020000u};
    __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                     :
                     : "s"(__builtin_amdgcn_readfirstlane((int)lds)), "v"(off), "s"(r)
                     : "memory");
}
typedef __attribute__((address_space(3))) unsigned char lds_byte;
#define lds_base(array) ((uint32_t)(uintptr_t)(lds_byte *)(array))
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

// Records: chunk c of sequence i has slot floor(begin / 32) + i + c, its block c / 2 of 64 tokens slot floor(begin / 64) +
// i + c / 2; the slots of different sequences differ.
__device__ __forceinline__ int64_t slot_of(int64_t begin, int64_t i) { return begin / kGC + i; }
__device__ __forceinline__ int64_t block_of(int64_t begin, int64_t i) { return begin / kGB + i; }

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
template <bool kUniform = true>  // the same segment for all lanes
__device__ __forceinline__ Entry entry_of(const GdnArgs &a, int64_t row, int64_t p)
{
    auto cu = [&](int64_t n) { return kUniform ? uniform(a.cu[n]) : a.cu[n]; };
    const int64_t at = p * a.len;
    if (!a.cu)
        return p >= a.P ? Entry{row + 1, 0} : Entry{row, at / kGC};  // len is a multiple of a chunk
    if (p >= a.P)
        return Entry{a.N, 0};
    if (p == 0)
        return Entry{0, 0};
    // the first sequence that begins at `at` or behind, or the one before it if it has a chunk there
    const int64_t m = cu(0) >= at ? 0 : last_at_most(a.N + 1, at - 1, cu);
    if (m >= a.N)
        return Entry{a.N, 0};
    const int64_t begin = cu(m), c = (at - begin + kGC - 1) / kGC;
    return c * kGC < cu(m + 1) - begin ? Entry{m, c} : Entry{m + 1, 0};
}

struct Chunk {
    int64_t seq, slot, block;
    int64_t t0;     // first token, in its row
    int len;        // 0: no chunk
    bool first, last;       // of the workgroup's piece of the sequence
    bool from_seg, to_seg;  // the piece begins (ends) at a cut
    bool opens, closes;     // the first (last) chunk of a block of 64 tokens
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
        k.block = uniform(k.block);
        k.t0 = uniform(k.t0);
        return k;
    }
    __device__ Chunk advance(const GdnArgs &a)
    {
        Chunk k = {0, 0, 0, 0, 0, false, false, false, false, false, false};
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
        k.block = block_of(begin, i) + (c >> 1);
        k.t0 = (a.cu ? begin : 0) + c * kGC;
        k.opens = (c & 1) == 0;
        k.closes = (c & 1) == 1 || rest <= kGC;
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
// Inclusive sum over the lanes of each half of the wave: shifts by 1, 2, 4, 8 inside each 16, then the last lane of row 0
// and 2 to the next row.
__device__ __forceinline__ double running_sum32(double b)
{
    b += dpp_f64<0x111, 0xf>(b);
    b += dpp_f64<0x112, 0xf>(b);
    b += dpp_f64<0x114, 0xf>(b);
    b += dpp_f64<0x118, 0xf>(b);
    b += dpp_f64<0x142, 0xa>(b);
    return b;
}
// The same over all 64: lane 31 to the upper half
__device__ __forceinline__ double running_sum64(double b)
{
    b = running_sum32(b);
    b += dpp_f64<0x143, 0xc>(b);
    return b;
}
__device__ __forceinline__ double of_lane(double b, int lane)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, b);
    return __builtin_bit_cast(double,
                              ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane) << 32) |
                                  (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane));
}

// A state that has passed transitions of a norm below 2^-150 counts as 0 (a finite one; others make their rows NaN).
constexpr float kDead = -150.0f;

// How many of the chunks [c_lo, c_hi) of a sequence, counted from the end (or from the start), a state has to pass until it counts
// as 0; one more than all of them if it never does.  By a wave, 64 chunks at a time.  What lies beyond is left out of shares and
// transitions: of a state of size 1 it is below the smallest fp32 number.
template <bool kFromEnd>
__device__ __forceinline__ int64_t live_chunks(const GdnArgs &a, int64_t slot0, int64_t c_lo, int64_t c_hi, int64_t h, int lane)
{
    double sum = 0.0;
    for (int64_t n = 0; n < c_hi - c_lo; n += 64) {
        const int64_t i = n + lane, c = kFromEnd ? c_hi - 1 - i : c_lo + i;
        const float x = i < c_hi - c_lo ? a.norm[(slot0 + c) * a.H + h] : 0.0f;
        const double upto = sum + running_sum64((double)x);
        const uint64_t hit = __ballot(i < c_hi - c_lo && upto < (double)kDead);
        if (hit)
            return uniform(n + __builtin_ctzll(hit) + 1);
        sum = of_lane(upto, 63);
    }
    return c_hi - c_lo + 1;
}

// ------------------------------------------------------------------------------- records
//
// Factors of a record, 32 floats each (token of the chunk):
constexpr int kVHead = 0;    // e^{b_t}
constexpr int kVWrite = 32;  // beta_s e^{L - b_s}
constexpr int kVOut = 64;    // scale e^{b_t}
constexpr int kVBeta = 96;   // beta_s
constexpr int kVTail = 128;  // e^{L - b_s}
constexpr int kVLast = 160;  // [0]: e^{L}

// The terms of one step (16 of the contraction) of a 32 x 32 matrix, in the order of the lanes
constexpr int kTermStep = 3 * 1024;
__device__ __forceinline__ void store_terms(unsigned char *mat, int step, int lane, const Terms &t)
{
    u32x4 *p = reinterpret_cast<u32x4 *>(mat + step * kTermStep + lane * 16);
    p[0] = t.h;
    p[64] = t.m;
    p[128] = t.l;
}
__device__ __forceinline__ Terms load_terms(const unsigned char *mat, int step, int lane)
{
    const u32x4 *p = reinterpret_cast<const u32x4 *>(mat + step * kTermStep + lane * 16);
    return Terms{p[0], p[64], p[128]};
}

constexpr int kNRow = 36;      // floats per row of the triangular matrix in LDS
constexpr int kPrepWaves = 4;

struct LdsPrep {
    float n[kGC * kNRow];
    float bh[kGC], bl[kGC], beta[kGC];
};

// Bound by memory, most of it the records that it writes: (a) 25 us, 5.1 TB/s; (b) 169 us, 5.3 TB/s; (c) 70 us, 5.1 TB/s.
// Records of chunks of 64 tokens, two waves each, took 2.2 times as long in (b): four times the matrix to solve and to write.
// One wave per (chunk, head), nothing shared between waves.  M = e^{b_t - b_s} k_t.k_s; N's two 16 x 16 blocks on the diagonal
// are solved column by column, the block below them with fp32 matrix instructions:
// N_10 = (1 - N_11 beta)(M_10 - M_10 beta N_00).
template <bool kBwd>
__global__ __launch_bounds__(64 * kPrepWaves) void gdn_prep_kernel(GdnArgs a)
{
    __shared__ __attribute__((aligned(16))) LdsPrep lds[kPrepWaves];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l32 = lane & 31,
              h = lane >> 5;
    LdsPrep &s = lds[wave];
    const uint32_t unit = blockIdx.x * kPrepWaves + wave;  // below 2^26
    const int64_t slot = unit / (uint32_t)a.H, head = unit - (uint32_t)slot * (uint32_t)a.H;
    if (slot >= a.slots || (a.status && *a.status != 0))
        return;
    const int64_t seq = last_at_most(a.N, slot, [&](int64_t i) { return slot_of(uniform(seq_begin(a, i)), i); });
    const int64_t begin = uniform(seq_begin(a, seq)), c = slot - slot_of(begin, seq),
                  rest = uniform(seq_begin(a, seq + 1)) - begin - c * kGC;
    if (rest <= 0)
        return;
    const int len = (int)(rest < kGC ? rest : kGC);
    const int64_t row = a.cu ? 0 : seq, t0 = (a.cu ? begin : 0) + c * kGC;
    unsigned char *rec = a.rec + (slot * a.H + head) * a.rec_bytes;

    auto tile = [&](const GdnTensor &x) {
        const uint32_t stride = (uint32_t)x.st * 2;
        return rsrc(head_base(x, row, head) + t0 * x.st, __builtin_amdgcn_readfirstlane((int)((uint32_t)(len - 1) * stride + 256u)));
    };
    const __amdgpu_buffer_rsrc_t rk = tile(a.k), rq = tile(a.q);
    const uint32_t ok = (uint32_t)l32 * (uint32_t)a.k.st * 2 + 16u * h, oq = (uint32_t)l32 * (uint32_t)a.q.st * 2 + 16u * h;
    u32x4 kf[8], qf[8];  // row lane % 32, 16 channels each step; behind the chunk zeros
#pragma unroll
    for (int x = 0; x < 8; ++x)
        kf[x] = buf_b128(rk, ok + 32u * x);
#pragma unroll
    for (int x = 0; x < 8; ++x)
        qf[x] = buf_b128(rq, oq + 32u * x);
    const int64_t gate = (row * a.T + t0) * a.H + head;
    const float dec = l32 < len ? a.decay[gate + (int64_t)l32 * a.H] : 0.0f;
    const float bet = l32 < len ? a.beta[gate + (int64_t)l32 * a.H] : 0.0f;
    const double b = running_sum32((double)clamp_decay(dec) * kLog2e64), last = of_lane(b, 31);
    const float bh = (float)b, bl = (float)(b - (double)bh);
    if (h == 0) {
        s.bh[l32] = bh;
        s.bl[l32] = bl;
        s.beta[l32] = bet;
        float *v = reinterpret_cast<float *>(rec + kGdnMat) + l32;
        const float from = __builtin_amdgcn_exp2f((float)b), tail = __builtin_amdgcn_exp2f((float)(last - b));
        v[kVHead] = from;
        v[kVWrite] = bet * tail;
        v[kVOut] = a.scale * from;
        v[kVBeta] = bet;
        v[kVTail] = tail;
        if (l32 == 0)
            v[kVLast] = __builtin_amdgcn_exp2f((float)last);
    }
    __builtin_amdgcn_wave_barrier();
    f32x16 kk, qk;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        kk[i] = qk[i] = 0.0f;
    // rows: sources 8 n + 4 h .., columns: tokens, a lane's is lane % 32
#pragma unroll
    for (int x = 0; x < 8; ++x)
        kk = mfma(kf[x], kf[x], kk);
#pragma unroll
    for (int x = 0; x < 8; ++x)
        qk = kBwd ? mfma(qf[x], kf[x], qk) : mfma(kf[x], qf[x], qk);
    auto vec4 = [&](const float *p, int n) { return *reinterpret_cast<const f32x4 *>(p + 8 * n + 4 * h); };
    if (a.norm) {  // log2 of a bound of the transition's norm: |e^g (1 - beta k k^T)| = e^g max(1, |1 - beta k.k|) for each token
        float own = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            own = 8 * (i >> 2) + 4 * h + (i & 3) == l32 ? kk[i] : own;
        own += __shfl_xor(own, 32);
        const float f = fabsf(1.0f - bet * own), grow = f > 1.0f ? __builtin_amdgcn_logf(f) : f != f ? f : 0.0f;
        const double bound = last + of_lane(running_sum32((double)grow), 31);
        if (lane == 0)
            a.norm[slot * a.H + head] = (float)bound;
    }
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        const f32x4 uh = vec4(s.bh, n), ul = vec4(s.bl, n), ub = vec4(s.beta, n);
        f32x4 m4;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int u = 8 * n + 4 * h + i;
            // e^{b_t - b_u}, t = lane % 32
            const float w = u <= l32 ? __builtin_amdgcn_exp2f((bh - uh[i]) + (bl - ul[i])) : 0.0f;
            m4[i] = u < l32 ? kk[4 * n + i] * w : 0.0f;
            if constexpr (!kBwd) {  // A'
                qk[4 * n + i] = u <= l32 ? qk[4 * n + i] * (a.scale * w) * ub[i] : 0.0f;
            } else {  // A, rows: tokens u, columns: sources, a lane's is lane % 32
                const float z = u >= l32 ? __builtin_amdgcn_exp2f((uh[i] - bh) + (ul[i] - bl)) : 0.0f;
                qk[4 * n + i] = u >= l32 ? qk[4 * n + i] * (a.scale * z) : 0.0f;
            }
        }
        *reinterpret_cast<f32x4 *>(&s.n[l32 * kNRow + 8 * n + 4 * h]) = m4;
    }
#pragma unroll
    for (int st = 0; st < 2; ++st)
        store_terms(rec + (kBwd ? 2 : 1) * kGdnMat + kGdnVec, st, lane, cut8n(qk, st));
    __builtin_amdgcn_wave_barrier();
    // N's diagonal blocks: lanes of block lane / 16 % 2, column lane % 16; both halves of the wave do the same
    {
        const int blk = l32 >> 4, m = l32 & 15;
        const float *p = s.n + 16 * blk * (kNRow + 1), *bb = s.beta + 16 * blk;
        float x[16], y[16];  // the column so far, and beta times it
        x[0] = y[0] = 0.0f;
#pragma unroll
        for (int i = 1; i < 16; ++i) {
            float z = p[i * kNRow + m];
#pragma unroll
            for (int k = 1; k < i; ++k)
                z = fmaf(-p[i * kNRow + k], y[k], z);
            x[i] = i > m ? z : 0.0f;
            y[i] = bb[i] * x[i];
        }
        __builtin_amdgcn_wave_barrier();
        if (h == 0) {
            float *w = s.n + 16 * blk * (kNRow + 1) + m;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                w[i * kNRow] = x[i];
        }
    }
    __builtin_amdgcn_wave_barrier();
    {
        const int m = lane & 15, g = lane >> 4;
        auto rows = [&](int bi, int bj) {  // D layout of a block
            f32x4 r;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                r[i] = s.n[(16 * bi + 4 * g + i) * kNRow + 16 * bj + m];
            return r;
        };
        auto minus = [&](int bi, int bk) {  // minus a block, as A operand
            return -*reinterpret_cast<const f32x4 *>(&s.n[(16 * bi + m) * kNRow + 16 * bk + 4 * g]);
        };
        auto beta4 = [&](int bi) { return *reinterpret_cast<const f32x4 *>(&s.beta[16 * bi + 4 * g]); };
        const f32x4 p = mfma_f32(minus(1, 0), rows(0, 0) * beta4(0), rows(1, 0));
        const f32x4 n = mfma_f32(minus(1, 1), p * beta4(1), p);
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int i = 0; i < 4; ++i)
            s.n[(16 + 4 * g + i) * kNRow + m] = n[i];
    }
    __builtin_amdgcn_wave_barrier();
    // T' = 1 - N beta, and for the backward pass T = 1 - beta N, transposed
#pragma unroll
    for (int st = 0; st < 2; ++st) {
        f32x4 x[2], y[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int u0 = 16 * st + 8 * e + 4 * h;
            const f32x4 nn = *reinterpret_cast<const f32x4 *>(&s.n[l32 * kNRow + u0]);
            const f32x4 bb = *reinterpret_cast<const f32x4 *>(&s.beta[u0]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[e][i] = u0 + i < l32 ? -nn[i] * bb[i] : u0 + i == l32 ? 1.0f : 0.0f;
                if constexpr (kBwd)
                    y[e][i] = u0 + i > l32 ? -s.n[(u0 + i) * kNRow + l32] * bb[i] : u0 + i == l32 ? 1.0f : 0.0f;
            }
        }
        store_terms(rec, st, lane, cut8n(x[0], x[1]));
        if constexpr (kBwd)
            store_terms(rec + kGdnMat + kGdnVec, st, lane, cut8n(y[0], y[1]));
    }
}

// ------------------------------------------------------------------------- state in registers
//
// Wave w of 4 holds 32 value columns of the state, all 128 key channels: S.t[kt][r], lane = column + 32 h: channel
// 32 kt + 16 (r / 8) + 8 h + r % 8, so that elements 8s .. 8s+7 are 8 neighbouring channels, as an operand wants them.
// Nothing of it ever crosses waves.  Lane n % 32 holds column n, or (where rows of out are stored) column
// 16 (n/4 % 2) + 4 (n/8) + n%4: a lane of an out tile then has 16 neighbouring channels.

struct State {
    f32x16 t[4];
};
template <bool kOut>
__device__ __forceinline__ int column_of(int n)
{
    return kOut ? 16 * ((n >> 2) & 1) + 4 * (n >> 3) + (n & 3) : n;
}

// v: the lane's value column
__device__ __forceinline__ void state_load(State &S, const void *base, int dt, int v, int lane)
{
    const int at = v * kD + 8 * (lane >> 5);
#pragma unroll
    for (int kt = 0; kt < 4; ++kt)
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            if (dt == kBf16) {
                const u32x4 x = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(base) + at + 32 * kt + 16 * st);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    S.t[kt][8 * st + 2 * e] = lo_f(x[e]);
                    S.t[kt][8 * st + 2 * e + 1] = hi_f(x[e]);
                }
            } else {
                const f32x4 *p = reinterpret_cast<const f32x4 *>(static_cast<const float *>(base) + at + 32 * kt + 16 * st);
                const f32x4 x = p[0], y = p[1];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    S.t[kt][8 * st + e] = x[e];
                    S.t[kt][8 * st + 4 + e] = y[e];
                }
            }
        }
}
__device__ __forceinline__ void state_store(const State &S, void *base, int dt, int v, int lane)
{
    const int at = v * kD + 8 * (lane >> 5);
#pragma unroll
    for (int kt = 0; kt < 4; ++kt)
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            if (dt == kBf16) {
                u32x4 x;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[e] = pack2(S.t[kt][8 * st + 2 * e], S.t[kt][8 * st + 2 * e + 1]);
                *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(base) + at + 32 * kt + 16 * st) = x;
            } else {
                f32x4 *p = reinterpret_cast<f32x4 *>(static_cast<float *>(base) + at + 32 * kt + 16 * st);
                p[0] = f32x4{S.t[kt][8 * st], S.t[kt][8 * st + 1], S.t[kt][8 * st + 2], S.t[kt][8 * st + 3]};
                p[1] = f32x4{S.t[kt][8 * st + 4], S.t[kt][8 * st + 5], S.t[kt][8 * st + 6], S.t[kt][8 * st + 7]};
            }
        }
}
__device__ __forceinline__ void state_zero(State &S)
{
#pragma unroll
    for (int kt = 0; kt < 4; ++kt)
#pragma unroll
        for (int r = 0; r < 16; ++r)
            S.t[kt][r] = 0.0f;
}
__device__ __forceinline__ void state_one(State &S, int v, int lane)
{
#pragma unroll
    for (int kt = 0; kt < 4; ++kt)
#pragma unroll
        for (int r = 0; r < 16; ++r)
            S.t[kt][r] = 32 * kt + 16 * (r >> 3) + 8 * (lane >> 5) + (r & 7) == v ? 1.0f : 0.0f;
}
// 0, or NaN where a value of the lane's column is not finite
__device__ __forceinline__ float state_lost(const State &S)
{
    float x = 0.0f;
#pragma unroll
    for (int kt = 0; kt < 4; ++kt)
#pragma unroll
        for (int r = 0; r < 16; ++r)
            x = fmaf(S.t[kt][r], 0.0f, x);
    return x + __shfl_xor(x, 32);
}
__device__ __forceinline__ void state_add1(State &S, float x)
{
#pragma unroll
    for (int kt = 0; kt < 4; ++kt)
        S.t[kt] += x;
}
__device__ __forceinline__ size_t state_size(int dt) { return kGdnStateBytes / (dt == kBf16 ? 2 : 1); }

// ------------------------------------------------------------------------------- LDS
//
// Tiles are rows (tokens) of 256 bytes (128 channels); the 16-byte pieces of a row are XORed with a function of its
// number modulo 8, so that 8 rows of one piece and 4 rows of two neighbouring pieces lie in different banks.

__device__ __forceinline__ int swz(int row) { return ((row & 3) << 1) | ((row >> 2) & 1); }

constexpr int kTile = kGC * 256;

struct LdsWalk {
    unsigned char tile[2][3][kTile];  // k, v, q of two chunks
    unsigned char rec[2][2 * kGdnMat + kGdnVec];
};

// Half n of a tile straight into LDS: 4 rows an instruction, wave w of kWaves takes rows 4w .. and those 4 kWaves behind
// them.  Rows behind the chunk lie beyond the descriptor and arrive as zeros.
template <int kWaves>
__device__ __forceinline__ void tile_half(uint32_t lds, const GdnTensor &x, const uint16_t *base, int64_t t0, int len,
                                          int n, int wave, int lane)
{
    const uint32_t stride = (uint32_t)x.st * 2;
    const int row = 4 * wave + (lane >> 4);
    const uint32_t off = (uint32_t)(row + 4 * kWaves * n) * stride + (uint32_t)(((lane & 15) ^ swz(row)) << 4);
    load_lds(base + t0 * x.st, len > 0 ? (uint32_t)(len - 1) * stride + 256u : 0u, off, lds + 1024 * (wave + kWaves * n));
}

// Transposing read: lane i of each 16 lanes gives the address of 4 channels of token i / 4 and gets channel i of
// the 16 for the 4 tokens.
__device__ __forceinline__ u32x2 lds_tr(const unsigned char *p)
{
    typedef __attribute__((address_space(3))) s16x4 lds_s4;
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)p));
}

// This lane's places in a tile; the channel block is XORed in.
struct Lanes {
    int row;  // row lane % 32, 8 channels 8 h .. of 16
    int key;  // transposing: tokens 4 h .. of 8, the 32 channels of a state's tile in the order of its registers
    int col;  // the same, 32 channels in the order of lanes
    int out;  // the same, in the order of column_of<true>

    __device__ explicit Lanes(int lane)
    {
        const int l32 = lane & 31, h = lane >> 5, g2 = (lane >> 4) & 1, i = lane & 15, t = 4 * h + (i >> 2), q = i & 3;
        auto at = [&](int channel) { return t * 256 + (((channel >> 3) ^ swz(t)) << 4) + 2 * (channel & 4); };
        row = l32 * 256 + ((h ^ swz(l32)) << 4);
        key = at(16 * g2 + 8 * (q & 1) + 4 * (q >> 1));
        col = at(16 * g2 + 4 * q);
        out = at(16 * (q & 1) + 8 * g2 + 4 * (q >> 1));
    }
};
// 16 channels 16 x .. of row lane % 32 of a block of 32 rows
__device__ __forceinline__ u32x4 row_frag(const unsigned char *tile, const Lanes &ln, int x, int block = 0)
{
    return *reinterpret_cast<const u32x4 *>(tile + 8192 * block + (ln.row ^ (32 * x)));
}
// tokens 8 n + 4 h .. of 32 channels 32 kt ..
__device__ __forceinline__ u32x2 col_frag4(const unsigned char *tile, int at, int kt, int n)
{
    return lds_tr(tile + 2048 * n + (at ^ (64 * kt)));
}
// 16 tokens 16 st .., as an operand of a contraction over tokens
__device__ __forceinline__ u32x4 col_frag(const unsigned char *tile, int at, int kt, int st)
{
    const u32x2 x = col_frag4(tile, at, kt, 2 * st), y = col_frag4(tile, at, kt, 2 * st + 1);
    return u32x4{x[0], x[1], y[0], y[1]};
}
__device__ __forceinline__ f32x4 widen4(u32x2 x) { return f32x4{lo_f(x[0]), hi_f(x[0]), lo_f(x[1]), hi_f(x[1])}; }
// factors of tokens 8 n + 4 h ..
__device__ __forceinline__ f32x4 vec4(const unsigned char *vec, int which, int n, int lane)
{
    return *reinterpret_cast<const f32x4 *>(vec + 4 * (which + 8 * n + 4 * (lane >> 5)));
}
__device__ __forceinline__ float vec1(const unsigned char *vec, int at)
{
    return *reinterpret_cast<const float *>(vec + 4 * at);
}
__device__ __forceinline__ f32x16 zero16()
{
    f32x16 z;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        z[i] = 0.0f;
    return z;
}

// Order of what stands since the last call: kN matrix instructions with kV vector instructions behind each, and no others
// across.  A matrix instruction takes 32 cycles, in which one wave can issue six others; left alone the compiler puts
// products and cuts behind each other, and neither the wave's own nor the other wave's overlap.
template <int kN, int kV>
__device__ __forceinline__ void mixed()
{
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, kV, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
}

// Key channels (rows: the state's registers) of tokens 16 st .. of a tile
struct KeyFrags {
    u32x4 t[4];
};
__device__ __forceinline__ KeyFrags key_frags(const unsigned char *tile, const Lanes &ln, int st)
{
    KeyFrags k;
#pragma unroll
    for (int kt = 0; kt < 4; ++kt)
        k.t[kt] = col_frag(tile, ln.key, kt, st);
    return k;
}
// S += keys times value columns, 12 products
__device__ __forceinline__ void state_add(State &S, const KeyFrags &k, const Terms &u)
{
#pragma unroll
    for (int kt = 0; kt < 4; ++kt)
        S.t[kt] = mfma3(k.t[kt], u, S.t[kt]);
}
__device__ __forceinline__ void state_scale(State &S, float f)
{
#pragma unroll
    for (int kt = 0; kt < 4; ++kt)
        S.t[kt] *= f;
}

// --------------------------------------------------------------------------- forward walk
//
// 32 value columns a wave on 32x32x16 matrix instructions, four waves a workgroup, two workgroups a CU; a chunk's tiles and record
// come into one of two LDS buffers while the other is worked on, with one barrier a chunk.  Per chunk and wave of the output
// walk: 96 matrix instructions (of 32 cycles), 750 other vector instructions, most of them cuts, 58 LDS reads.  A wave alone
// on its SIMD issues in 61 % of its cycles, which is what bounds (a) with 256 workgroups (62 us, 3.9 us a chunk; the matrix
// pipe busy 31 %) and (c) (212 us, 40 %); two a SIMD reach some 6 us for two chunks ((b): 462 us, matrix pipe 49 %, vector 58 %).
// With products and cuts in the compiler's order (b) took 12 % longer; chunks of 64 tokens with one workgroup a CU made all
// of the call's kernels together 11 % longer than these in that order.

constexpr int kModeOut = 0;    // out and final states
constexpr int kModeShare = 1;  // a segment's share of the state at its end (F)
constexpr int kModePhi = 2;    // the transition: from S = 1, without values
constexpr int kModeStore = 3;  // backward pass: the state before each block and the residuals
constexpr int kWalkWaves = 4;
constexpr int kWalkThreads = 64 * kWalkWaves;

// Sequences without tokens that belong to segment p: the state leaves as it came.  With invalid lengths all of them.
__device__ void empty_states(const GdnArgs &a, const Entry &e0, const Entry &e1, bool valid, int64_t p, int64_t h,
                             const void *init, int init_dt, void *fin, int fin_dt)
{
    if (!a.cu && a.T != 0)
        return;
    const int tid = threadIdx.x, lane = tid & 63, v = 32 * (tid >> 6) + (lane & 31);
    const int64_t lo = !valid ? (p == 0 ? 0 : a.N) : e0.seq, hi = !valid ? a.N : p + 1 == a.P && a.cu ? a.N : e1.seq;
    for (int64_t b = lo; b < hi; b += kWalkThreads) {
        const int64_t i = b + tid;
        const bool none = i < hi && (!valid || seq_begin(a, i) == seq_begin(a, i + 1));
        if (!__syncthreads_or(none))
            continue;
        for (int64_t n = b; n < b + kWalkThreads && n < hi; ++n) {
            if (valid && seq_begin(a, n) != seq_begin(a, n + 1))
                continue;
            State S;
            state_zero(S);
            const int64_t at = n * a.H + h;
            if (init)
                state_load(S, static_cast<const unsigned char *>(init) + at * state_size(init_dt), init_dt, v, lane);
            state_store(S, static_cast<unsigned char *>(fin) + at * state_size(fin_dt), fin_dt, v, lane);
        }
    }
}

// A D tile (rows: tokens, columns: lane % 32) into a 32 x 128 matrix, from its column on
__device__ __forceinline__ void rows_store(float *m, const f32x16 &x, int lane)
{
#pragma unroll
    for (int i = 0; i < 16; ++i)
        m[(8 * (i >> 2) + 4 * (lane >> 5) + (i & 3)) * kD + (lane & 31)] = x[i];
}

// at: where in LDS `lds` begins
template <int kMode>
__device__ __forceinline__ void walk(const GdnArgs &a, LdsWalk &lds, uint32_t at, int64_t row, int64_t p, int64_t h)
{
    constexpr bool kOut = kMode == kModeOut, kValues = kMode != kModePhi;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l32 = lane & 31;
    const int v = 32 * wave + column_of<kOut>(l32);
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
    float lost = 0.0f;    // NaN where a state that is not finite was left out
    bool skipped = false;  // chunks whose share of the state at the cut counts as 0
    if constexpr (kMode == kModeShare || kMode == kModePhi) {
        const int64_t begin = uniform(seq_begin(a, e1.seq)), n = e1.chunk - e0.chunk;
        const int64_t live = live_chunks<true>(a, slot_of(begin, e1.seq), e0.chunk, e1.chunk, h, lane);
        if constexpr (kMode == kModePhi) {
            if (tid == 0)
                a.dead[segment * a.H + h] = live <= n;
            if (live <= n)
                return;
        } else {
            if (e0.chunk == 0 && a.init && (a.keep || live <= n)) {
                State S;
                state_load(S, static_cast<const unsigned char *>(a.init) + (e0.seq * a.H + h) * state_size(a.init_dt),
                           a.init_dt, v, lane);
                if (a.keep)
                    state_store(S, a.keep + (segment * a.H + h) * kD * kD, 2, v, lane);
                lost = state_lost(S);
            }
            if (live <= n) {
                skipped = true;
                e0.chunk = e1.chunk - live;
            }
        }
    }
    Walk w;
    w.init(e0, e1, false);
    Chunk ch = w.next(a);
    if (ch.len == 0)
        return;
    const Lanes ln(lane);
    const uint16_t *pk = head_base(a.k, row, h), *pv = head_base(a.v, row, h), *pq = head_base(a.q, row, h);
    // A chunk's loads in kLoads parts: asked for all at once they fill the load queue and hold the wave up for some 2000 cycles.
    constexpr int kTiles = kOut ? 3 : kValues ? 2 : 1, kBytes = kOut ? 2 * kGdnMat + kGdnVec : kGdnMat + kGdnVec;
    constexpr int kLoads = 2 * kTiles + (kBytes / 1024 + kWalkWaves - 1) / kWalkWaves;
    auto fetch = [&](int buf, const Chunk &n, int part) {
        if (part >= kLoads)
            return;
        if (part < 2 * kTiles) {
            const int t = part >> 1;
            tile_half<kWalkWaves>(at + kTile * (3 * buf + t), t == 0 ? a.k : t == 1 ? a.v : a.q, t == 0 ? pk : t == 1 ? pv : pq, n.t0, n.len,
                                  part & 1, wave, lane);
        } else {
            int i = wave + kWalkWaves * (part - 2 * kTiles);  // the last KiB by several waves, rather than a branch
            i = i < kBytes / 1024 ? i : kBytes / 1024 - 1;
            load_lds(a.rec + (n.slot * a.H + h) * a.rec_bytes, n.len ? kBytes : 0, (uint32_t)(1024 * i + 16 * lane),
                     at + (int)offsetof(LdsWalk, rec) + (int)sizeof(lds.rec[0]) * buf + 1024 * i);
        }
    };
    State S;
    state_zero(S);
    int buf = 0;
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
        fetch(0, ch, i);
    Terms c = cut8(S.t[0], 0);  // of the state's first 16 channels
    // stored a chunk later, behind the wait for the loads: a store is then waited for a whole chunk after it
    u32x4 held[2];     // rows of out
    f32x16 held_r;     // residuals
    Chunk before = ch;
    before.len = 0;
    auto store_held = [&]() {
        if (before.len == 0)
            return;
        if constexpr (kOut) {
            if (l32 < before.len) {
                uint16_t *o = a.out + ((row * a.T + before.t0 + l32) * a.H + h) * kD + 32 * wave + 16 * (lane >> 5);
                reinterpret_cast<u32x4 *>(o)[0] = held[0];
                reinterpret_cast<u32x4 *>(o)[1] = held[1];
            }
        }
        if constexpr (kMode == kModeStore)
            rows_store(a.res + (before.slot * a.H + h) * kGC * kD + 32 * wave, held_r, lane);
    };
    for (;;) {
        const unsigned char *tk = lds.tile[buf][0], *tv = lds.tile[buf][1], *tq = lds.tile[buf][2], *mt = lds.rec[buf],
                            *vec = mt + kGdnMat, *ma = vec + kGdnVec;
        const Chunk nx = w.next(a);
        arrive();  // this chunk's tiles and record are there; the other buffer is read by no one
        store_held();
        if (ch.first) {
            if constexpr (kMode == kModePhi) {
                state_one(S, v, lane);
            } else if (ch.from_seg || skipped) {
                if constexpr (kOut || kMode == kModeStore)
                    state_load(S, a.seg + (segment * a.H + h) * kD * kD, 2, v, lane);
                else
                    state_zero(S);
            } else if (kOut && a.keep && ch.to_seg) {
                state_load(S, a.keep + (segment * a.H + h) * kD * kD, 2, v, lane);
            } else if (a.init) {
                state_load(S, static_cast<const unsigned char *>(a.init) + (ch.seq * a.H + h) * state_size(a.init_dt),
                           a.init_dt, v, lane);
            } else {
                state_zero(S);
            }
            // here, or the compiler waits behind the branch in every chunk
            __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
            c = cut8(S.t[0], 0);
        }
        if constexpr (kMode == kModeStore)
            if (ch.opens)
                state_store(S, a.before + (ch.block * a.H + h) * kD * kD, 2, v, lane);
        f32x16 Z = zero16(), O = zero16(), R = zero16();
        u32x4 kf = row_frag(tk, ln, 0), qf = kf;
        if constexpr (kOut)
            qf = row_frag(tq, ln, 0);
        Terms t0, t1, a0, a1;
        u32x2 v4[4];
        f32x4 f4[4];
        __builtin_amdgcn_sched_barrier(0);
        // what is read for a step, and the cut for it, stand in the step before
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            Terms cn = c;
            u32x4 kn = kf, qn = qf;
            if (x < 7) {
                kn = row_frag(tk, ln, x + 1);
                if constexpr (kOut)
                    qn = row_frag(tq, ln, x + 1);
                cn = cut8(S.t[(x + 1) >> 1], (x + 1) & 1);
            }
            if (x == 6) {
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    f4[n] = vec4(vec, kVHead, n, lane);
                    if constexpr (kValues)
                        v4[n] = col_frag4(tv, kOut ? ln.out : ln.col, wave, n);
                }
            }
            if (x == 7)
                t0 = load_terms(mt, 0, lane);
            Z = mfma(kf, c.l, Z);
            if constexpr (kOut)  // transposed: rows are value columns, a lane's token is lane % 32
                O = mfma(c.l, qf, O);
            Z = mfma(kf, c.m, Z);
            if constexpr (kOut)
                O = mfma(c.m, qf, O);
            Z = mfma(kf, c.h, Z);
            if constexpr (kOut)
                O = mfma(c.h, qf, O);
            fetch(buf ^ 1, nx, x);
            mixed<kOut ? 6 : 3, kOut ? 8 : 15>();
            c = cn;
            kf = kn;
            qf = qn;
        }
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                Z[4 * n + i] = kValues ? fmaf(-f4[n][i], Z[4 * n + i], i == 0   ? lo_f(v4[n][0])
                                                                       : i == 1 ? hi_f(v4[n][0])
                                                                       : i == 2 ? lo_f(v4[n][1])
                                                                                : hi_f(v4[n][1]))
                                       : -f4[n][i] * Z[4 * n + i];
        Terms x0 = cut8(Z, 0);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 8; i < kLoads; ++i)
            fetch(buf ^ 1, nx, i);
        t1 = load_terms(mt, 1, lane);
        R = mfma6(t0, x0, R);
        const Terms x1 = cut8(Z, 1);
        mixed<6, 8>();
        const float carry = vec1(vec, kVLast), vo = vec1(vec, kVOut + l32);
#pragma unroll
        for (int n = 0; n < 4; ++n)
            f4[n] = vec4(vec, kVWrite, n, lane);
        if constexpr (kOut)
            a0 = load_terms(ma, 0, lane);
        KeyFrags k0 = key_frags(tk, ln, 0);
        R = mfma6(t1, x1, R);
        state_scale(S, carry);
        if constexpr (kOut)
            O *= vo;
        mixed<6, kOut ? 14 : 11>();
        if constexpr (kOut) {
            const Terms r0 = cut8(R, 0);
            __builtin_amdgcn_sched_barrier(0);
            a1 = load_terms(ma, 1, lane);
            O = mfma6(r0, a0, O);
            const Terms r1 = cut8(R, 1);
            mixed<6, 8>();
            O = mfma6(r1, a1, O);
        }
        if constexpr (kMode == kModeStore)
            held_r = R;
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                R[4 * n + i] *= f4[n][i];
        const Terms u0 = cut8(R, 0);
        if constexpr (kOut)
            mixed<6, 10>();
        else
            __builtin_amdgcn_sched_barrier(0);
        const KeyFrags k1 = key_frags(tk, ln, 1);
        state_add(S, k0, u0);
        const Terms u1 = cut8(R, 1);
        mixed<12, 4>();
        state_add(S, k1, u1);
        c = cut8(S.t[0], 0);
        if constexpr (kOut)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                held[e >> 2][e & 3] = pack2(O[2 * e], O[2 * e + 1]);
        mixed<12, 5>();
        before = ch;
        if (kMode != kModeStore && ch.last) {
            if constexpr (kMode == kModeShare) {
                if (skipped)
                    state_add1(S, lost);
                state_store(S, a.seg + ((segment + 1) * a.H + h) * kD * kD, 2, v, lane);
            } else if constexpr (kMode == kModePhi)
                state_store(S, a.phi + (segment * a.H + h) * kD * kD, 2, v, lane);
            else if (a.fin && !ch.to_seg)
                state_store(S, static_cast<unsigned char *>(a.fin) + (ch.seq * a.H + h) * state_size(a.fin_dt), a.fin_dt,
                            v, lane);
        }
        if (nx.len == 0)
            break;
        ch = nx;
        buf ^= 1;
    }
    store_held();
}

// Workgroup b of a walk: segment b % (rows P) of head b / (rows P).  Neighbours run on different XCDs, so that each of them gets
// its share of every head (how long a share or transition takes depends on the head's decays), and heads that share q and k
// meet in one XCD's cache.
struct Place {
    int64_t row, p, h;

    __device__ explicit Place(const GdnArgs &a)
    {
        const uint32_t b = blockIdx.x, n = (uint32_t)(a.rows * a.P), s = b % n;
        h = b / n;
        row = s / (uint32_t)a.P;
        p = s - (uint32_t)row * (uint32_t)a.P;
    }
};

__global__ __launch_bounds__(kWalkThreads, 2) void gdn_out_kernel(GdnArgs a)
{
    extern __shared__ __attribute__((aligned(1024))) unsigned char raw[];
    const Place at(a);
    walk<kModeOut>(a, *reinterpret_cast<LdsWalk *>(raw), lds_base(raw), at.row, at.p, at.h);
}
// Head i in an order that puts, of each 64 heads, those first that forget slowly: their shares and transitions are whole segments,
// those of others end early, and workgroups begin in the order of their numbers.  Judged by the bounds of 8 chunks; any values
// there, of a slot without a chunk too, give an order of all heads.  It costs some 3 us before the walk, so only where segments
// are long (shares and transitions, without and with it): 512 tokens 67 and 70 us, 896 tokens 119 and 121, 2048 tokens 248
// and 206, 2432 tokens 437 and 367.
constexpr int64_t kOrderedSeg = 1024;
__device__ __forceinline__ int64_t slow_first(const GdnArgs &a, uint32_t i)
{
    if (a.len < kOrderedSeg)
        return i;
    const int lane = threadIdx.x & 63;
    const int64_t group = i & ~63u, left = a.H - group, n = left < 64 ? left : 64;
    float sum = 0.0f;
    if (lane < n)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            sum += a.norm[a.slots * (2 * j + 1) / 16 * a.H + group + lane];
    const int bits = __float_as_int(sum);
    const uint32_t key = (uint32_t)bits ^ (bits < 0 ? 0xffffffffu : 0x80000000u);  // in the order of the values
    int rank = 0;
    for (int k = 0; k < (int)n; ++k) {
        const uint32_t other = (uint32_t)__builtin_amdgcn_readlane((int)key, k);
        rank += other > key || (other == key && k < lane);
    }
    return group + __builtin_ctzll(__ballot(lane < n && rank == (int)(i - group)));
}
// All transitions, then all shares, or, in order, a head's transitions and its shares before the next head's
__global__ __launch_bounds__(kWalkThreads, 2) void gdn_cut_kernel(GdnArgs a)
{
    extern __shared__ __attribute__((aligned(1024))) unsigned char raw[];
    const bool ordered = a.len >= kOrderedSeg;
    const uint32_t n = (uint32_t)(a.rows * a.P), each = ordered ? 2 * n : n,
                   b = ordered ? blockIdx.y * gridDim.x + blockIdx.x : blockIdx.x, i = b / each, r = b - each * i;
    const int64_t h = slow_first(a, i), s = r < n ? r : r - n, row = s / a.P, p = s - row * a.P;
    if (ordered ? r < n : blockIdx.y == 0)
        walk<kModePhi>(a, *reinterpret_cast<LdsWalk *>(raw), lds_base(raw), row, p, h);
    else
        walk<kModeShare>(a, *reinterpret_cast<LdsWalk *>(raw), lds_base(raw), row, p, h);
}
__global__ __launch_bounds__(kWalkThreads, 2) void gdn_store_kernel(GdnArgs a)
{
    extern __shared__ __attribute__((aligned(1024))) unsigned char raw[];
    const Place at(a);
    walk<kModeStore>(a, *reinterpret_cast<LdsWalk *>(raw), lds_base(raw), at.row, at.p, at.h);
}

// ----------------------------------------------------------------------------------- scan
//
// State at each cut: S_{p+1} = S_p Phi_p + F_p where segment p lies inside one sequence (else F_p is the state); backwards
// (kRev) the gradients of the states at the cuts, dS_{p-1} = dS_p Phi_p^T + F_p.  A workgroup of 8 waves takes 16 value
// columns of one row and head; wave w forms key channels 16w .. of each state and hands its terms to the others
// through LDS.  The next step's Phi and F are on their way meanwhile.  A step takes some 2 us: each of a row's 8 workgroups
// reads the whole of Phi, 64 KiB at some 15 bytes a cycle ((a) 18 us for 6 steps, (c) 59 for 30).  Two steps' loads on their
// way took longer (20 and 73).
template <bool kRev>
__global__ __launch_bounds__(512) void gdn_scan_kernel(GdnArgs a)
{
    __shared__ __attribute__((aligned(16))) uint32_t terms[2][3][4][64][4];
    __shared__ float lost[2][8][16];
    __shared__ uint8_t kinds[kGdnMaxCuts];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, m = lane & 15, g = lane >> 4;
    const uint32_t chain = blockIdx.x >> 3, row = chain / (uint32_t)a.H, h = chain - row * (uint32_t)a.H;
    const int v = (int)(blockIdx.x & 7) * 16 + m;
    if (a.status && *a.status != 0)
        return;
    float *base = (kRev ? a.dseg : a.seg) + ((size_t)row * a.P * a.H + h) * kD * kD;
    const float *phis = a.phi + ((size_t)row * a.P * a.H + h) * kD * kD;
    const size_t step = (size_t)a.H * kD * kD;
    const int first = kRev ? (int)a.P - 2 : 1, dir = kRev ? -1 : 1;
    // what each segment is: 0 not inside one sequence, 1 inside, 2 inside and its transition counts as 0
    for (int p = tid; p < a.P; p += 512) {
        int kind = 0;
        if (p >= 1 && p <= a.P - 2) {
            const Entry e = entry_of<false>(a, row, p), n = entry_of<false>(a, row, p + 1);
            if (e.chunk > 0 && n.chunk > 0 && e.seq == n.seq)
                kind = a.dead[((int64_t)row * a.P + p) * a.H + h] ? 2 : 1;
        }
        kinds[p] = (uint8_t)kind;
    }
    __syncthreads();
    auto kind_of = [&](int p) { return p < 1 || p > a.P - 2 ? 0 : __builtin_amdgcn_readfirstlane((int)kinds[p]); };
    f32x4 f[8], acc, own;
    auto at = [&](int p) { return reinterpret_cast<f32x4 *>(base + (size_t)p * step + (size_t)v * kD + 16 * wave + 4 * g); };
    auto fetch = [&](int p) {
        acc = *at(p + dir);
        const float *phi = phis + (size_t)p * step;
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            if constexpr (kRev) {
                f[x] = *reinterpret_cast<const f32x4 *>(phi + (16 * wave + m) * kD + 16 * x + 4 * g);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    f[x][i] = phi[(16 * x + 4 * g + i) * kD + 16 * wave + m];
            }
        }
    };
    int cur = 0;
    bool have = false;  // `own` is the state that segment p begins (ends) with
    auto share_terms = [&]() {
        Terms t;
        cut2n(own[0], own[1], t, 0);
        cut2n(own[2], own[3], t, 1);
        const int x = wave >> 1, e = 2 * (wave & 1);
        *reinterpret_cast<u32x2 *>(&terms[cur][0][x][lane][e]) = u32x2{t.h[0], t.h[1]};
        *reinterpret_cast<u32x2 *>(&terms[cur][1][x][lane][e]) = u32x2{t.m[0], t.m[1]};
        *reinterpret_cast<u32x2 *>(&terms[cur][2][x][lane][e]) = u32x2{t.l[0], t.l[1]};
    };
    int kind = kind_of(first);
    if (kind == 1)
        fetch(first);
    for (int p = first; p >= 1 && p <= a.P - 2; p += dir) {
        const int next = kind_of(p + dir);
        if (kind == 0) {
            have = false;
        } else {
            if (!have)
                own = *at(p);
            if (kind == 2) {
                // nothing of the state is left, unless a row of it is not finite: that makes the row NaN
                float x = own[0] * 0.0f + own[1] * 0.0f + own[2] * 0.0f + own[3] * 0.0f;
                x += __shfl_xor(x, 16);
                x += __shfl_xor(x, 32);
                if (g == 0)
                    lost[cur][wave][m] = x;
                __syncthreads();
                x = 0.0f;
#pragma unroll
                for (int w = 0; w < 8; ++w)
                    x += lost[cur][w][m];
                own = *at(p + dir);
                if (x != x) {
                    own += x;
                    *at(p + dir) = own;
                }
            } else {
                share_terms();
                Terms ft[4];
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    ft[x] = cut8n(f[2 * x], f[2 * x + 1]);
                own = acc;
                if (next == 1)
                    fetch(p + dir);
                __syncthreads();
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const Terms s = {*reinterpret_cast<const u32x4 *>(terms[cur][0][x][lane]),
                                     *reinterpret_cast<const u32x4 *>(terms[cur][1][x][lane]),
                                     *reinterpret_cast<const u32x4 *>(terms[cur][2][x][lane])};
                    own = mfma6(ft[x], s, own);  // rows: key channels, columns: value columns
                }
                *at(p + dir) = own;
            }
            cur ^= 1;  // the next step's barrier keeps the writes two steps on behind these reads
            have = true;
        }
        if (kind != 1 && next == 1)
            fetch(p + dir);
        kind = next;
    }
}

// -------------------------------------------------------------------------- backward walk
//
// dL/dS from a sequence's end to its start, in the same layout; stores it after each block, and dw.  90 matrix instructions a
// chunk; (a) 85 us, the store walk 69, each writing 134 MB of states, and shares 61.

template <bool kShare>
__device__ __forceinline__ void walk_back(const GdnArgs &a, LdsWalk &lds, uint32_t at, int64_t row, int64_t p, int64_t h)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int v = 32 * wave + (lane & 31);
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
    float lost = 0.0f;
    bool skipped = false;  // as in the forward walk, from the segment's start on
    if (kShare && valid) {
        const int64_t begin = uniform(seq_begin(a, e0.seq)), len = uniform(seq_begin(a, e0.seq + 1)) - begin;
        const int64_t end = e1.seq == e0.seq ? e1.chunk : (len + kGC - 1) / kGC, n = end - e0.chunk;
        const int64_t live = live_chunks<false>(a, slot_of(begin, e0.seq), e0.chunk, end, h, lane);
        if (live <= n) {
            if (e1.seq != e0.seq && a.dfin) {
                State S;
                state_load(S, a.dfin + (e0.seq * a.H + h) * kD * kD, 2, v, lane);
                lost = state_lost(S);
            }
            skipped = true;
            e1 = Entry{e0.seq, e0.chunk + live};
        }
    }
    Walk w;
    w.init(e0, e1, true);
    Chunk ch = w.next(a);
    if (ch.len == 0)
        return;
    const uint16_t *pk = head_base(a.k, row, h), *po = head_base(a.dout, row, h), *pq = head_base(a.q, row, h);
    constexpr int kBytes = 2 * kGdnMat + kGdnVec, kLoads = 6 + (kBytes / 1024 + kWalkWaves - 1) / kWalkWaves;
    auto fetch = [&](int buf, const Chunk &n, int part) {  // in parts, as in the forward walk
        if (part >= kLoads)
            return;
        if (part < 6) {
            const int t = part >> 1;
            tile_half<kWalkWaves>(at + kTile * (3 * buf + t), t == 0 ? a.k : t == 1 ? a.dout : a.q, t == 0 ? pk : t == 1 ? po : pq, n.t0, n.len,
                                  part & 1, wave, lane);
        } else {
            int i = wave + kWalkWaves * (part - 6);
            i = i < kBytes / 1024 ? i : kBytes / 1024 - 1;
            load_lds(a.rec + (n.slot * a.H + h) * a.rec_bytes + kGdnMat, n.len ? kBytes : 0, (uint32_t)(1024 * i + 16 * lane),
                     at + (int)offsetof(LdsWalk, rec) + (int)sizeof(lds.rec[0]) * buf + 1024 * i);
        }
    };
    State S;
    state_zero(S);
    int buf = 0;
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
        fetch(0, ch, i);
    Terms c = cut8(S.t[0], 0);  // of the state's first 16 channels
    f32x16 held;  // dw, stored a chunk later as in the forward walk
    Chunk before = ch;
    before.len = 0;
    auto store_held = [&]() {
        if (!kShare && before.len)
            rows_store(a.dwrite + (before.slot * a.H + h) * kGC * kD + 32 * wave, held, lane);
    };
    for (;;) {
        const unsigned char *tk = lds.tile[buf][0], *to = lds.tile[buf][1], *tq = lds.tile[buf][2], *vec = lds.rec[buf],
                            *mt = vec + kGdnVec, *ma = mt + kGdnMat;
        const Chunk nx = w.next(a);
        int l = tid & 63;
        if constexpr (kShare)  // places formed anew: kept from chunk to chunk some would be in scratch, whose loads wait for the tiles'
            __asm__ volatile("" : "+v"(l));
        const int lane = l;
        const Lanes ln(lane);
        arrive();  // this chunk's tiles and record are there; the other buffer is read by no one
        store_held();
        if (ch.first) {
            if (ch.from_seg) {  // also where chunks were left out
                if constexpr (kShare)
                    state_zero(S);
                else
                    state_load(S, a.dseg + (segment * a.H + h) * kD * kD, 2, v, lane);
            } else if (a.dfin) {
                state_load(S, a.dfin + (ch.seq * a.H + h) * kD * kD, 2, v, lane);
            } else {
                state_zero(S);
            }
            // here, or the compiler waits behind the branch in every chunk
            __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
            c = cut8(S.t[0], 0);
        }
        if (!kShare && ch.closes)
            state_store(S, a.dafter + (ch.block * a.H + h) * kD * kD, 2, v, lane);
        f32x16 Y = zero16(), W = zero16();
        u32x4 kf = row_frag(tk, ln, 0), o[2];
        Terms a0, a1, t0, t1;
        f32x4 f4[4], fo[4], fb[4], fh[4];
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            Terms cn = c;
            u32x4 kn = kf;
            if (x < 7) {
                kn = row_frag(tk, ln, x + 1);
                cn = cut8(S.t[(x + 1) >> 1], (x + 1) & 1);
            }
            if (x == 6) {
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    f4[n] = vec4(vec, kVTail, n, lane);
                    fo[n] = vec4(vec, kVOut, n, lane);
                }
#pragma unroll
                for (int st = 0; st < 2; ++st)
                    o[st] = col_frag(to, ln.col, wave, st);
            }
            if (x == 7) {
                a0 = load_terms(ma, 0, lane);
                a1 = load_terms(ma, 1, lane);
            }
            Y = mfma3(kf, c, Y);
            fetch(buf ^ 1, nx, x);
            mixed<3, 15>();
            c = cn;
            kf = kn;
        }
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                Y[4 * n + i] *= f4[n][i];
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 8; i < kLoads; ++i)
            fetch(buf ^ 1, nx, i);
        t0 = load_terms(mt, 0, lane);
        Y = mfma3(a0, o[0], Y);
        Y = mfma3(a1, o[1], Y);
        // what the tokens' reads and writes send to the state before the chunk: first the reads
        f32x16 g;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const f32x4 o4 = widen4(u32x2{o[n >> 1][2 * (n & 1)], o[n >> 1][2 * (n & 1) + 1]});
#pragma unroll
            for (int i = 0; i < 4; ++i)
                g[4 * n + i] = o4[i] * fo[n][i];
        }
        const Terms g0 = cut8(g, 0);
        mixed<6, 12>();
        const float carry = vec1(vec, kVLast);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            fb[n] = vec4(vec, kVBeta, n, lane);
            fh[n] = vec4(vec, kVHead, n, lane);
        }
        t1 = load_terms(mt, 1, lane);
        const Terms y0 = cut8(Y, 0);
        __builtin_amdgcn_sched_barrier(0);
        KeyFrags k0 = key_frags(tq, ln, 0);
        W = mfma6(t0, y0, W);
        const Terms y1 = cut8(Y, 1);
        mixed<6, 8>();
        W = mfma6(t1, y1, W);
        state_scale(S, carry);
        const Terms g1 = cut8(g, 1);
        mixed<6, 18>();
        KeyFrags k1 = key_frags(tq, ln, 1);
        state_add(S, k0, g0);
        held = W;
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                W[4 * n + i] *= -(fb[n][i] * fh[n][i]);
        const Terms w0 = cut8(W, 0);
        mixed<12, 7>();
        k0 = key_frags(tk, ln, 0);
        state_add(S, k1, g1);
        const Terms w1 = cut8(W, 1);
        mixed<12, 4>();
        k1 = key_frags(tk, ln, 1);
        state_add(S, k0, w0);
        __builtin_amdgcn_sched_barrier(0);
        state_add(S, k1, w1);
        c = cut8(S.t[0], 0);
        mixed<12, 4>();
        before = ch;
        if (ch.last) {
            if constexpr (kShare) {
                if (skipped)
                    state_add1(S, lost);
                state_store(S, a.dseg + ((segment - 1) * a.H + h) * kD * kD, 2, v, lane);
            } else if (a.dinit && !ch.to_seg)
                state_store(S, a.dinit + (ch.seq * a.H + h) * kD * kD, 2, v, lane);
        }
        if (nx.len == 0)
            break;
        ch = nx;
        buf ^= 1;
    }
    store_held();
}

template <bool kShare>
__global__ __launch_bounds__(kWalkThreads, 2) void gdn_back_kernel(GdnArgs a)
{
    extern __shared__ __attribute__((aligned(1024))) unsigned char raw[];
    Place at(a);
    if constexpr (kShare)
        at.h = slow_first(a, (uint32_t)at.h);
    walk_back<kShare>(a, *reinterpret_cast<LdsWalk *>(raw), lds_base(raw), at.row, at.p, at.h);
}

// ------------------------------------------------------------------- gradients of a block
//
// One workgroup of 4 waves per (block of 64 tokens, head), two of them on a CU, so that one computes while the other's loads
// are on their way; the formulas hold for blocks of any length, r_t and dw_t are the tokens' own.  Each wave forms what the
// state before the block and its gradient behind it give to dq and dk, 32 key channels each (rows: channels, a lane's token
// is lane % 32): it takes them from memory, cut as they come.  w = beta r and dx = beta dw stay in LDS in fp32 and are cut
// where they are used, which takes less room and time than their terms would.  Then the waves share out the 32 x 32 tiles of
// P, P^T and G + G^T, which reach all of them through LDS, in the place of w and dx.
//
// 414 matrix and some 5250 other vector instructions a wave, three quarters of them cuts: issue bounds it (matrix pipe busy
// 26 %, vector 46 %), then memory, 3.4 TB/s.  (a) 184 us, some 5 of them what ddecay's terms add to the sums of q.dq - v.dv (the
// reads of v saved).  One workgroup of 8 waves with the terms in LDS took 37 % longer (its 36000 cycles of loads and 29000 of
// products did not overlap: a CU takes in some 10 bytes a cycle), with tiles shared out evenly 25 %; products and cuts
// interleaved by hand change nothing here, ddecay's products beside those of P (no branches) or its sums over lanes by
// DPP in place of LDS permutes do not either or make it slower (call 522 and 545 us).

// LDS: w and dx, 64 rows of 32 pieces of 16 bytes each, piece u of row t at u ^ (t % 16), and dout.  Behind the products with
// them: the matrices (steps of 3 KiB), k, q, and what is below.
constexpr int kGradX = kGB * 512, kGradO = 2 * kGradX, kGradLds = kGradO + kGB * 256;
// P: columns tokens t, contraction sources, steps 0 .. 1 + 2 t; P^T: columns sources s, contraction tokens, steps 2 s .. 3; then, in
// their place, G + G^T, all steps
constexpr int kGradP = 0, kGradPT = 6, kGradMats = 12;
constexpr int kGradK = kGradMats * kTermStep, kGradQ = kGradK + kGB * 256;
struct LdsGrad {
    float bh[4][kGB], bl[4][kGB];  // running sums of log2 decays as pairs, a copy for each wave
    // terms of dg (above): by source or token for each wave's channels, inside tiles 00 and 11 by token (of G and of P), and of
    // tile 01 by its tokens and by its sources (of P and of G)
    float writes[4][kGB], reads[4][kGB];
    float inside[2][kGB];
    float far_tok[2][kGC], far_src[2][kGC];
    float end[4];                  // e^L <dS, S>, a wave's share
};
constexpr int kGradRest = kGradQ + kGB * 256;
static_assert(kGradRest + sizeof(LdsGrad) <= kGradLds, "the second half reuses the first's room");

// This wave's writes to LDS are done, and then the other waves'; loads from memory stay in flight.
__device__ __forceinline__ void settle()
{
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
    __asm__ volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    __asm__ volatile("" ::: "memory");
}

__global__ __launch_bounds__(256, 2) void gdn_grad_kernel(GdnArgs a)
{
    extern __shared__ __attribute__((aligned(1024))) unsigned char raw[];
    const int tid = threadIdx.x, lane = tid & 63, kg = __builtin_amdgcn_readfirstlane(tid >> 6), l32 = lane & 31, h = lane >> 5;
    const int64_t block = blockIdx.x / (uint32_t)a.H, head = blockIdx.x - (uint32_t)block * (uint32_t)a.H;
    if (a.status && *a.status != 0)
        return;
    const int64_t seq = last_at_most(a.N, block, [&](int64_t i) { return block_of(uniform(seq_begin(a, i)), i); });
    const int64_t begin = uniform(seq_begin(a, seq)), c = block - block_of(begin, seq),
                  rest = uniform(seq_begin(a, seq + 1)) - begin - c * kGB;
    if (rest <= 0)
        return;
    const int len = (int)(rest < kGB ? rest : kGB);
    const int64_t row = a.cu ? 0 : seq, t0 = (a.cu ? begin : 0) + c * kGB, tok0 = row * a.T + t0;
    const int64_t slot = slot_of(begin, seq) + 2 * c;
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // two rows an instruction; a chunk without tokens has none and arrives as zeros
        const int n = kg + 4 * i, chunk = n >> 4, t = 2 * n + h;
        const int64_t from = ((slot + chunk) * a.H + head) * kGC * kD;
        const uint32_t off = (uint32_t)((t & 31) * 512 + ((l32 ^ (t & 15)) << 4)), bytes = len > kGC * chunk ? kGC * kD * 4 : 0;
        load_lds(a.res + from, bytes, off, lds_base(raw) + 1024 * n);
        load_lds(a.dwrite + from, bytes, off, lds_base(raw) + kGradX + 1024 * n);
    }
    auto load_tile = [&](const GdnTensor &x, int to) {
        const uint16_t *p = head_base(x, row, head);
#pragma unroll
        for (int n = 0; n < 4; ++n)
            tile_half<4>(lds_base(raw) + to, x, p, t0, len, n, kg, lane);
    };
    load_tile(a.dout, kGradO);
    // rows of dv: thread = token tid / 4, value channels 32 (tid % 4) ..
    const int rt = tid >> 2, v0 = 32 * (tid & 3);
    const bool on = rt < len;
    const float rb = on ? a.beta[(tok0 + rt) * a.H + head] : 0.0f;
    const float rg = lane < len ? a.decay[(tok0 + lane) * a.H + head] : 0.0f;
    // the states' columns of this wave: lane = key channel, element 8 x + j: value row 16 x + 8 h + j
    const int64_t at = (block * a.H + head) * kD * kD;
    const __amdgpu_buffer_rsrc_t rs = rsrc(a.before + at, kGdnStateBytes), rd = rsrc(a.dafter + at, kGdnStateBytes);
    const int lane_at = 4 * (8 * h * kD + 32 * kg + column_of<true>(l32));
    struct Piece {
        f32x4 a, b;
    };
    auto piece = [&](__amdgpu_buffer_rsrc_t r, int x) {
        Piece y;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            y.a[j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, lane_at + 4 * kD * j, 64 * kD * x, 0));
            y.b[j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, lane_at + 4 * kD * (4 + j), 64 * kD * x, 0));
        }
        return y;
    };
    // of each token in lane: its logarithm as a pair
    const double b64 = running_sum64((double)clamp_decay(rg) * kLog2e64), last64 = of_lane(b64, 63);
    const float bh = (float)b64, bl = (float)(b64 - (double)bh);
    const float from1 = __builtin_amdgcn_exp2f((float)b64), tail1 = __builtin_amdgcn_exp2f((float)(last64 - b64));
    const float last = __builtin_amdgcn_exp2f((float)last64);
    arrive();
    {
        float db = 0.0f;
        u32x4 rv[4];
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // scaled by beta in place
            const int p = rt * 512 + (((8 * (tid & 3) + i) ^ (rt & 15)) << 4);
            f32x4 r = *reinterpret_cast<const f32x4 *>(raw + p), d = *reinterpret_cast<const f32x4 *>(raw + kGradX + p);
            if (!on)
                r = d = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            const f32x4 x = d * rb;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                db = fmaf(d[e], r[e], db);
            *reinterpret_cast<f32x4 *>(raw + p) = r * rb;
            *reinterpret_cast<f32x4 *>(raw + kGradX + p) = x;
            rv[i >> 1][2 * (i & 1)] = pack2(x[0], x[1]);
            rv[i >> 1][2 * (i & 1) + 1] = pack2(x[2], x[3]);
        }
        if (on) {
            u32x4 *dv = reinterpret_cast<u32x4 *>(a.dv + ((tok0 + rt) * a.H + head) * kD + v0);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                dv[i] = rv[i];
        }
#pragma unroll
        for (int o = 2; o > 0; o >>= 1)
            db += __shfl_xor(db, o);
        if (on && (tid & 3) == 0)
            a.dbeta[(tok0 + rt) * a.H + head] = db;
    }
    Piece ps[2], pd[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        ps[x] = piece(rs, x);
        pd[x] = piece(rd, x);
    }
    settle();
    Lanes ln(lane);
    int row4 = l32 * 512 + (((2 * h) ^ (l32 & 15)) << 4);
    // 8 values 16 x + 8 h .. of row 32 th + lane % 32 of w or dx
    auto terms = [&](int which, int x, int th) {
        const unsigned char *p = raw + which + 16384 * th + 256 * (x >> 2);
        return cut8n(*reinterpret_cast<const f32x4 *>(p + (row4 ^ (64 * (x & 3)))),
                    *reinterpret_cast<const f32x4 *>(p + (row4 ^ (64 * (x & 3) + 16))));
    };
    float dot = 0.0f;  // <dS, S>, this lane's share
    float writes[2], reads[2];
    f32x16 dq[2], dk[2], put[4];
    {
        f32x16 dw[2];
        dq[0] = dq[1] = dk[0] = dk[1] = dw[0] = dw[1] = zero16();
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            const Piece s = ps[x & 1], d = pd[x & 1];
            if (x < 6) {
                ps[x & 1] = piece(rs, x + 2);
                pd[x & 1] = piece(rd, x + 2);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                dot = fmaf(s.b[j], d.b[j], fmaf(s.a[j], d.a[j], dot));
            __asm__ volatile("" : "+v"(dot));  // here: put off, it would keep the pieces
            const Terms cs = cut8n(s.a, s.b), cd = cut8n(d.a, d.b);
#pragma unroll
            for (int th = 0; th < 2; ++th) {
                dq[th] = mfma3(cs, row_frag(raw + kGradO, ln, x, th), dq[th]);
                dk[th] = mfma6(cs, terms(kGradX, x, th), dk[th]);
                dw[th] = mfma6(cd, terms(0, x, th), dw[th]);
            }
            __builtin_amdgcn_sched_barrier(0);  // one step at a time: more of them in flight do not fit the registers
        }
        dot *= last;
        const uint16_t *pk = head_base(a.k, row, head);
#pragma unroll
        for (int th = 0; th < 2; ++th) {
            const int t = 32 * th + l32;
            const float from = __shfl(from1, t), tail = __shfl(tail1, t);
            const int64_t at = t0 + (t < len ? t : 0);  // behind the block all sums are 0
            const u32x4 *p = reinterpret_cast<const u32x4 *>(pk + at * a.k.st + 32 * kg + 16 * h);
            const u32x4 k16[2] = {p[0], p[1]};
            dq[th] *= a.scale * from;
            float wk = 0.0f, rd = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float y = dw[th][i] * tail, z = from * dk[th][i];
                const uint32_t u = k16[i >> 3][(i & 7) >> 1];
                const float ke = i & 1 ? hi_f(u) : lo_f(u);
                wk = fmaf(y, ke, wk);
                rd = fmaf(-z, ke, rd);
                dk[th][i] = y - z;
            }
            writes[th] = wk + __shfl_xor(wk, 32);
            reads[th] = rd;  // without dq.q yet
            __asm__ volatile("" : "+v"(dq[th]), "+v"(dk[th]), "+v"(writes[th]), "+v"(reads[th]));
        }
    }
    // The tiles, unscaled: the product of rows of token tile i by rows of token tile j, and the transposed one of the same
    // operands.  Their terms are cut anew, from places that the compiler cannot tell to be those above: kept from there they would
    // not fit the registers.
    __asm__ volatile("" : "+v"(row4), "+v"(ln.row));
    auto g_pair = [&](int i, int j, f32x16 &y, f32x16 &yt) {
        y = yt = zero16();
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            const Terms w = terms(0, x, i), d = terms(kGradX, x, j);
            y = mfma6(w, d, y);
            yt = mfma6(d, w, yt);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    auto p_pair = [&](int i, int j, f32x16 &y, f32x16 &yt) {
        y = yt = zero16();
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            const Terms w = terms(0, x, i);
            const u32x4 o = row_frag(raw + kGradO, ln, x, j);
            y = mfma3(w, o, y);
            yt = mfma3(o, w, yt);
            if (x & 1)
                __builtin_amdgcn_sched_barrier(0);
        }
    };
    // P(0, 1) or, transposed, P^T(1, 0)
    auto p_far = [&](bool low) {
        f32x16 y = zero16();
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            const Terms w = terms(0, x, 0);
            const u32x4 o = row_frag(raw + kGradO, ln, x, 1);
            y = low ? mfma3(w, o, y) : mfma3(o, w, y);
            if (x & 1)
                __builtin_amdgcn_sched_barrier(0);
        }
        return y;
    };
    // waves 0 .. 2: G and G^T of tiles 00, 11, 01; 3: the diagonal tiles of P and P^T; the others of P, P^T: waves 0 and 1
    if (kg < 3)
        g_pair(kg == 1, kg != 0, put[0], put[1]);
    if (kg == 0) {
        put[2] = p_far(true);
    } else if (kg == 1) {
        put[2] = p_far(false);
    } else if (kg == 3) {
        p_pair(0, 0, put[0], put[1]);
        p_pair(1, 1, put[2], put[3]);
    }
    settle();  // w, dx and dout are read by no one
    load_tile(a.k, kGradK);
    load_tile(a.q, kGradQ);
    LdsGrad &s = *reinterpret_cast<LdsGrad *>(raw + kGradRest);
    s.bh[kg][lane] = bh;
    s.bl[kg][lane] = bl;
    if (h == 0) {
#pragma unroll
        for (int th = 0; th < 2; ++th)
            s.writes[kg][32 * th + l32] = writes[th];
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        dot += __shfl_xor(dot, o);
    if (lane == 0)
        s.end[kg] = dot;
    // times f e^{b_t - b_u} for u <= t (strict: u < t), formed where it is used, and 0 elsewhere
    auto scaled = [&](int rt, int ct, f32x16 d, float f, bool low, bool strict) {
        const float ch = s.bh[kg][32 * ct + l32], cl = s.bl[kg][32 * ct + l32], sign = low ? 1.0f : -1.0f;
        const int c0 = 32 * (ct - rt) + l32 - 4 * h, side = low ? 1 : -1;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const f32x4 rh = *reinterpret_cast<const f32x4 *>(&s.bh[kg][32 * rt + 8 * n + 4 * h]);
            const f32x4 rl = *reinterpret_cast<const f32x4 *>(&s.bl[kg][32 * rt + 8 * n + 4 * h]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int ahead = side * (c0 - (8 * n + i));  // of the source, in tokens
                const float b = sign * ((ch - rh[i]) + (cl - rl[i]));
                const float z = d[4 * n + i] * f * __builtin_amdgcn_exp2f(ahead >= 0 ? b : 0.0f);
                d[4 * n + i] = ahead >= (strict ? 1 : 0) ? z : 0.0f;
            }
        }
        return d;
    };
    auto store = [&](int step, const f32x16 &y) {
        store_terms(raw, step, lane, cut8(y, 0));
        store_terms(raw, step + 1, lane, cut8(y, 1));
    };
    if (kg == 0) {
        put[2] = scaled(0, 1, put[2], a.scale, true, false);
        store(kGradP + 2, put[2]);
    } else if (kg == 1) {
        put[2] = scaled(1, 0, put[2], a.scale, false, false);
        store(kGradPT + 2, put[2]);
    } else if (kg == 3) {
        put[0] = scaled(0, 0, put[0], a.scale, true, false);
        store(kGradP, put[0]);
        store(kGradPT, scaled(0, 0, put[1], a.scale, false, false));
        put[2] = scaled(1, 1, put[2], a.scale, true, false);
        store(kGradP + 4, put[2]);
        store(kGradPT + 4, scaled(1, 1, put[3], a.scale, false, false));
    }
    f32x16 g, gt;
    if (kg < 3) {
        g = scaled(kg == 1, kg != 0, put[0], -1.0f, true, true);
        gt = scaled(kg != 0, kg == 1, put[1], -1.0f, false, true);
        if (kg < 2)  // both triangles of one tile
#pragma unroll
            for (int i = 0; i < 16; ++i)
                g[i] = (i & 3) + 8 * (i >> 2) + 4 * h < l32 ? g[i] : gt[i];
    }
    arrive();  // P, P^T, k, q
    // Terms of dg from tiles of P and G (rows: registers, columns: lane % 32), each times the dot products of the rows' and
    // columns' tokens: rows of x by columns of y
    auto dots = [&](f32x16 d, int x, int i, int y, int j) {
        f32x16 c = zero16();
#pragma unroll
        for (int n = 0; n < 8; ++n)
            c = mfma(row_frag(raw + x, ln, n, i), row_frag(raw + y, ln, n, j), c);
        return d * c;
    };
    auto over_rows = [&](const f32x16 &d, float *to) {
        float x = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            x += d[i];
        x += __shfl_xor(x, 32);
        if (h == 0)
            to[l32] = x;
    };
    // for each token t of a tile on the diagonal the sum over rows s < t and columns u >= t
    auto inside = [&](f32x16 d, float *to) {
        float upto = 0.0f;  // rows before 8 n
#pragma unroll
        for (int n = 0; n < 4; ++n) {  // d: the sum of the rows before this one, where the column is not before it
            float own = 0.0f, part[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                part[i] = own;
                own += d[4 * n + i];
            }
            const float other = __shfl_xor(own, 32), base = h ? upto + other : upto;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                d[4 * n + i] = 8 * n + 4 * h + i <= l32 ? base + part[i] : 0.0f;
            upto += own + other;
        }
        // over the columns: at each step lanes in pairs keep one half of the rows each
#pragma unroll
        for (int o = 1, n = 8; n > 0; o <<= 1, n >>= 1)
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const bool upper = lane & o;
                const float keep = upper ? d[i + n] : d[i], give = upper ? d[i] : d[i + n];
                d[i] = keep + __shfl_xor(give, o);
            }
        const float x = d[0] + __shfl_xor(d[0], 16);
        const int i = 8 * (lane & 1) + 2 * (lane & 2) + ((lane >> 1) & 2) + ((lane >> 3) & 1);  // its row
        if ((lane & 16) == 0)
            to[8 * (i >> 2) + 4 * h + (i & 3)] = x;
    };
#pragma unroll
    for (int th = 0; th < 2; ++th) {
        const int t = 32 * th + l32;
        float x = reads[th];
#pragma unroll
        for (int e = 0; e < 2; ++e) {  // 16 channels 32 kg + 16 h .. of token t
            const u32x4 u = *reinterpret_cast<const u32x4 *>(raw + kGradQ + t * 256 + (((4 * kg + 2 * h + e) ^ swz(t)) << 4));
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x = fmaf(dq[th][8 * e + 2 * i + 1], hi_f(u[i]), fmaf(dq[th][8 * e + 2 * i], lo_f(u[i]), x));
        }
        x += __shfl_xor(x, 32);
        if (h == 0)
            s.reads[kg][t] = x;
    }
    if (kg == 0) {
        over_rows(dots(put[2], kGradK, 0, kGradQ, 1), s.far_tok[0]);
        inside(dots(g, kGradK, 0, kGradK, 0), s.inside[0]);
    } else if (kg == 1) {
        over_rows(dots(put[2], kGradQ, 1, kGradK, 0), s.far_src[0]);
        inside(dots(g, kGradK, 1, kGradK, 1), s.inside[0] + kGC);
    } else if (kg == 2) {
        over_rows(dots(g, kGradK, 0, kGradK, 1), s.far_tok[1]);
        over_rows(dots(gt, kGradK, 1, kGradK, 0), s.far_src[1]);
    } else {
        inside(dots(put[0], kGradK, 0, kGradQ, 0), s.inside[1]);
        inside(dots(put[2], kGradK, 1, kGradQ, 1), s.inside[1] + kGC);
    }
    auto key = [&](int tile, int st) { return col_frag(raw + tile + 8192 * (st >> 1), ln.out, kg, st & 1); };
#pragma unroll
    for (int st = 0; st < 4; ++st) {  // 16 tokens each of the contraction
        const u32x4 kc4 = key(kGradK, st), qc4 = key(kGradQ, st);
#pragma unroll
        for (int th = 0; th < 2; ++th) {
            if (st < 2 + 2 * th)
                dq[th] = mfma3(kc4, load_terms(raw, kGradP + 2 * th + st, lane), dq[th]);
            if (st >= 2 * th)
                dk[th] = mfma3(qc4, load_terms(raw, kGradPT + 2 * th + st, lane), dk[th]);
        }
    }
    settle();
    if (kg < 3)
        store(kg == 2 ? 4 : 6 * kg, g);
    if (kg == 2)
        store(2, gt);
    settle();
#pragma unroll
    for (int st = 0; st < 4; ++st) {
        const u32x4 kc4 = key(kGradK, st);
#pragma unroll
        for (int th = 0; th < 2; ++th)
            dk[th] = mfma3(kc4, load_terms(raw, 4 * th + st, lane), dk[th]);
    }
#pragma unroll
    for (int th = 0; th < 2; ++th) {
        const int t = 32 * th + l32;
        if (t >= len)
            continue;
        const int64_t to = ((tok0 + t) * a.H + head) * kD + 32 * kg + 16 * h;
        if (a.dq_h) {
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                reinterpret_cast<f32x4 *>(a.dq_h + to)[n] = f32x4{dq[th][4 * n], dq[th][4 * n + 1], dq[th][4 * n + 2], dq[th][4 * n + 3]};
                reinterpret_cast<f32x4 *>(a.dk_h + to)[n] = f32x4{dk[th][4 * n], dk[th][4 * n + 1], dk[th][4 * n + 2], dk[th][4 * n + 3]};
            }
        } else {
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                u32x4 x, z;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[e] = pack2(dq[th][8 * n + 2 * e], dq[th][8 * n + 2 * e + 1]);
                    z[e] = pack2(dk[th][8 * n + 2 * e], dk[th][8 * n + 2 * e + 1]);
                }
                reinterpret_cast<u32x4 *>(a.dq + to)[n] = x;
                reinterpret_cast<u32x4 *>(a.dk + to)[n] = z;
            }
        }
    }
    if (kg != 0)
        return;
    // dg: sums over the tokens before (without the lane's own) run forwards, those over tokens from the lane's on backwards, by
    // lanes in the opposite order; of tile 01 in tokens of the upper half over its tokens, of the lower half over its sources
    float end = 0.0f, written = 0.0f, read = 0.0f;
    const int past = lane > 0 ? lane - 1 : 0, turned = 63 - lane;
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        end += s.end[n];
        written += s.writes[n][past];
        read += s.reads[n][turned];
    }
    const float src = s.far_src[0][past & 31] + s.far_src[1][past & 31], tok = s.far_tok[0][turned & 31] + s.far_tok[1][turned & 31];
    const double before = running_sum64(lane > 0 ? (double)written : 0.0) + running_sum32(lane > 0 && h == 0 ? (double)src : 0.0);
    const double behind = running_sum64((double)read) + running_sum32(h == 0 ? (double)tok : 0.0);
    const double dg = (double)end + before + __shfl(behind, turned) + (double)s.inside[0][lane] + (double)s.inside[1][lane];
    if (lane < len)
        a.ddecay[(tok0 + lane) * a.H + head] = rg > kLowest && rg <= 0.0f ? (float)dg : 0.0f;
}

// ------------------------------------------------------------------- token by token
//
// One wave per (sequence, head, 32 rows of the state); lane = row % 8 * 8 + q holds 16 channels of 4 rows: 16-byte
// pieces, interleaved with those of the row's other 7 lanes.  S q = S~ q + beta r (k.q), so one pass over the row
// gives both dot products.  The state is read once and written once, which bounds it: 256 sequences of 32 heads, fp32
// states, 207 us, 5.2 TB/s (a copy: 5.33); bf16 states 110 us, 5.0 TB/s.
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

// The walks trust cu_seqlens, so nothing may run on one that leads out of the tensors.
hipError_t launch_check(const GdnArgs &a, int32_t *status, hipStream_t s)
{
    return a.cu ? lin_launch_check(a.cu, a.N, a.T, status, s) : hipSuccess;
}

}  // namespace

hipError_t gdn_launch_fwd(const GdnArgs &a, int32_t *status, hipStream_t s)
{
    const hipError_t e = launch_check(a, status, s);
    if (e != hipSuccess)
        return e;
    const unsigned grid = (unsigned)(a.rows * a.P * a.H);
    if (a.T > 0) {
        hipLaunchKernelGGL(gdn_prep_kernel<false>, dim3((unsigned)cdiv(a.slots * a.H, kPrepWaves)), dim3(64 * kPrepWaves), 0, s, a);
        if (a.P > 1)
            hipLaunchKernelGGL(gdn_cut_kernel, dim3(grid, 2), dim3(kWalkThreads), sizeof(LdsWalk), s, a);
        if (a.P > 2)
            hipLaunchKernelGGL(gdn_scan_kernel<false>, dim3((unsigned)(8 * a.rows * a.H)), dim3(512), 0, s, a);
    }
    hipLaunchKernelGGL(gdn_out_kernel, dim3(grid), dim3(kWalkThreads), sizeof(LdsWalk), s, a);
    return hipGetLastError();
}

hipError_t gdn_launch_bwd(const GdnArgs &a, int32_t *status, hipStream_t s)
{
    hipError_t e = launch_check(a, status, s);
    if (e != hipSuccess)
        return e;
    const unsigned grid = (unsigned)(a.rows * a.P * a.H), scan = (unsigned)(8 * a.rows * a.H);
    if (a.T > 0) {
        hipLaunchKernelGGL(gdn_prep_kernel<true>, dim3((unsigned)cdiv(a.slots * a.H, kPrepWaves)), dim3(64 * kPrepWaves), 0, s, a);
        if (a.P > 1) {
            hipLaunchKernelGGL(gdn_cut_kernel, dim3(grid, 2), dim3(kWalkThreads), sizeof(LdsWalk), s, a);
            if (a.P > 2)
                hipLaunchKernelGGL(gdn_scan_kernel<false>, dim3(scan), dim3(512), 0, s, a);
            hipLaunchKernelGGL(gdn_back_kernel<true>, dim3(grid), dim3(kWalkThreads), sizeof(LdsWalk), s, a);
            if (a.P > 2)
                hipLaunchKernelGGL(gdn_scan_kernel<true>, dim3(scan), dim3(512), 0, s, a);
        }
        hipLaunchKernelGGL(gdn_store_kernel, dim3(grid), dim3(kWalkThreads), sizeof(LdsWalk), s, a);
    }
    hipLaunchKernelGGL(gdn_back_kernel<false>, dim3(grid), dim3(kWalkThreads), sizeof(LdsWalk), s, a);
    if (a.T > 0)
        hipLaunchKernelGGL(gdn_grad_kernel, dim3((unsigned)(a.blocks * a.H)), dim3(256), kGradLds, s, a);
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
