// lin_attn.hip -- linear attention with a decay for each head, gfx950.
//
// Per (sequence, head), state S [V = 128][K = 128], natural-log decay g_t <= 0:
//   S_t = e^{g_t} S_{t-1} + v_t k_t^T,     out_t = scale * S_t q_t.
// In chunks of C = 64 tokens, with b the inclusive running sum of g inside the chunk and L
// its last entry:
//   out_t = scale * ( sum_{s <= t} e^{b_t - b_s} (q_t.k_s) v_s  +  e^{b_t} S q_t ),
//   S    <- e^{L} S + sum_s e^{L - b_s} v_s k_s^T.
// All three gradients are walks of the same form on other operands: dq takes (dO, v, k) in
// the place of (q, k, v), forwards, with the transposed state; dv takes (k, q, dO) and dk
// (v, dO, q) with the sources behind the token, the state dL/dS running from the end:
//   out_s = scale * sum_{t >= s} e^{b_t - b_s} (k_s.q_t) dO_t  +  e^{L - b_s} dS k_s,
//   dS   <- e^{L} dS + scale * sum_t e^{b_t} dO_t q_t^T.
// The decay's gradient follows from the others: with db_t = q_t.dq_t - k_t.dk_t,
//   dg_t = sum_{u >= t} db_u + <S_end, dS_end>, the sum up to the end of the segment.
// A token's own pair (t = s) adds the same to q.dq and k.dk and is left out of both.
//
// Numbers: decays are used as min(max(g, -1000), 0) (below -1000 the factor is 0 in fp32 long
// since, so -inf means "forget").  Running sums of logarithms are fp64 and kept as pairs of
// floats; a factor is the exponential of a difference, at most 1.  The products run on
// bf16 MFMA with fp32 accumulation; factors that are not bf16 inputs (the state, the weights, the weighted rows) are
// cut into three bf16 terms, hi + mid + lo: the 24 bits of fp32, whatever type the states have in memory.  Two terms
// (16 bits) took less time (T = 262144, H = 8: 618 us against 692; 38000 packed tokens, H = 32, Hk = 8: 385 against 472;
// B = 2, T = 4096, H = 16: 81 against 86), but where terms cancel they lose what fp32 keeps.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lin_internal.h"

namespace kda {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u2 __attribute__((vector_size(8)));   // as the buffer builtins want them
typedef unsigned int u4 __attribute__((vector_size(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kBf16 = 1, kFp32 = 2;  // kda_state_dtype
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
__device__ __forceinline__ uint16_t to_bf16(float a) { return __builtin_bit_cast(uint16_t, (__bf16)a); }

__device__ __forceinline__ float clamp_decay(float g)
{
    return g < kLowest ? kLowest : (g > 0.0f ? 0.0f : g);  // NaN stays NaN
}

// v_mfma_f32_32x32x16_bf16: A[m][k] in lane m + 32*(k/8), element k%8; B[k][n] in lane
// n + 32*(k/8), element k%8; D[m][n] in lane n + 32*((m/4)%2), element 4*(m/8) + m%4.
__device__ __forceinline__ f32x16 mfma(u32x4 a, u32x4 b, f32x16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                   0, 0, 0);
}

// Barrier for LDS hand-offs: global loads and stores stay in flight.
__device__ __forceinline__ void lds_barrier()
{
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
    __asm__ volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    __asm__ volatile("" ::: "memory");
}

// LDS tiles are rows of 256 bytes (64 tokens x 128 channels); the 16-byte pieces of a row are
// XORed with its number so that both 8 rows of one piece (the row-wise reads) and 4 rows
// of two neighbouring pieces (the transposing reads) lie in different banks.
__device__ __forceinline__ int swz(int row) { return ((row & 3) << 1) | ((row >> 2) & 1); }
__device__ __forceinline__ int tile_at(int row, int piece) { return row * 256 + ((piece ^ swz(row)) << 4); }

__device__ __forceinline__ u32x4 lds_b128(const unsigned char *p) { return *reinterpret_cast<const u32x4 *>(p); }
// Transposing read: lane i of each 16 lanes gives the address of 4 channels of token i / 4
// and gets channel i of the 16 for the 4 tokens.
__device__ __forceinline__ u32x2 lds_tr(const unsigned char *p)
{
    typedef __attribute__((address_space(3))) s16x4 lds_s4;
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)p));
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void *base, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ u32x4 buf_b128(__amdgpu_buffer_rsrc_t r, uint32_t off)
{
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// ------------------------------------------------------------------ sequences and pieces

constexpr int kPieceStart = 1, kPieceEnd = 2, kFromSlot = 4, kToFinal = 8;

struct Chunk {
    int64_t t0;   // first token (in its row)
    int64_t seq;
    int len;      // 0: no chunk
    int flags;
};

// The chunks that a workgroup walks: the pieces of sequences inside tokens [r0, r1) of its
// row, in the walk's direction.  Sequences are cut into chunks from their first token in
// the range on; a reverse walk takes the same chunks from the last to the first.
struct Walk {
    const int64_t *cu;
    int64_t row, T, r0, r1;
    int64_t first, last;   // sequences to visit
    int64_t i;             // the current one
    int64_t p0, p1;        // its piece
    int64_t t, left, nc;   // first token of the current chunk, chunks of the piece after it, chunks of it
    int pflags;
    bool rev;

    __device__ int64_t start(int64_t n) const { return cu ? cu[n] : 0; }
    __device__ int64_t end(int64_t n) const { return cu ? cu[n + 1] : T; }

    // first index with cu[index] >= x
    __device__ int64_t lower(int64_t N, int64_t x) const
    {
        int64_t lo = 0, hi = N + 1;
        while (lo < hi) {
            const int64_t m = (lo + hi) >> 1;
            if (cu[m] < x)
                lo = m + 1;
            else
                hi = m;
        }
        return lo;
    }
    __device__ void init(const LinArgs &a, int64_t row_, int64_t j, bool rev_)
    {
        cu = a.cu;
        row = row_;
        T = a.T;
        rev = rev_;
        r0 = j * a.len;
        r1 = r0 + a.len < T ? r0 + a.len : T;
        if (!cu) {
            first = last = 0;
        } else {
            const int64_t m = lower(a.N, r0);
            first = m > 0 && (m > a.N || cu[m] > r0) ? m - 1 : m;
            if (first > a.N - 1)
                first = a.N - 1;
            last = r1 == T ? a.N - 1 : lower(a.N, r1) - 1;
            if (last > a.N - 1)
                last = a.N - 1;
        }
        i = rev ? last + 1 : first - 1;
        p0 = p1 = t = left = nc = 0;
        pflags = 0;
    }
    __device__ int64_t seq_index() const { return cu ? i : row; }
    __device__ void set_piece()
    {
        const int64_t s0 = start(i), s1 = end(i);
        p0 = s0 > r0 ? s0 : r0;
        p1 = s1 < r1 ? s1 : r1;
        nc = p1 > p0 ? (p1 - p0 + kLC - 1) / kLC : 0;
        pflags = 0;
        if (rev)
            pflags = (s1 > r1 ? kFromSlot : 0) | (s0 >= r0 ? kToFinal : 0);
        else
            pflags = (s0 < r0 ? kFromSlot : 0) | (s1 <= r1 ? kToFinal : 0);
    }
    __device__ Chunk next()
    {
        Chunk k;
        int first_one = 0;
        --left;
        t += rev ? -kLC : kLC;
        while (left < 0) {  // the next piece with tokens
            i += rev ? -1 : 1;
            if (rev ? i < first : i > last)
                break;
            set_piece();
            left = nc - 1;
            t = rev ? p0 + left * kLC : p0;
            first_one = kPieceStart;
        }
        const int64_t rest = p1 - t;
        k.len = left < 0 ? 0 : (int)(rest < kLC ? rest : kLC);
        k.flags = pflags | first_one | (left == 0 ? kPieceEnd : 0);
        k.t0 = t;
        k.seq = seq_index();
        return k;
    }
};

// ------------------------------------------------------------------------- state in registers
//
// Wave w of 4 holds columns 32w .. 32w+31 of the role's v channels, all 128 k channels:
// S[kt][r], kt = 0..3, lane = column + 32 * half: channel 32 kt + 16 (r / 8) + 8 half + r % 8.
// A lane's registers 8m .. 8m+7 of a tile are then 8 neighbouring channels, as the operand of a
// 16-channel MFMA step wants them; the K operand of the update is read with its rows in
// the matching order.

struct State {
    f32x16 t[4];
};

__device__ __forceinline__ const void *matrix_of(const void *base, int64_t n, size_t bytes)
{
    return base ? static_cast<const unsigned char *>(base) + (size_t)n * bytes : nullptr;
}

// channel of register n = 16 kt + r for half 0 (half 1: 8 more)
__device__ constexpr int first_channel(int n) { return 32 * (n >> 4) + 16 * ((n >> 3) & 1) + (n & 7); }

// One 128 x 128 matrix at `base` (dt: 1 bf16, 2 fp32; NULL: zeros) into registers or back.  Buffer
// instructions: one lane offset serves all 64 entries, the rest sits in the instruction.
__device__ __forceinline__ void state_load(State &S, const void *base, int dt, bool tr, int wave, int lane)
{
    const int col = 32 * wave + (lane & 31), half = lane >> 5;
    const int size = dt == kBf16 ? 2 : 4;
    const __amdgpu_buffer_rsrc_t r = rsrc(base, base ? (uint32_t)(kD * kD * size) : 0u);
    const int vo = (tr ? 8 * half * kD + col : col * kD + 8 * half) * size;
    if (dt == kBf16 && tr) {
#pragma unroll
        for (int n = 0; n < 64; ++n)
            S.t[n >> 4][n & 15] = __uint_as_float(
                (uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, vo, first_channel(n) * kD * 2, 0) << 16);
    } else if (dt == kBf16) {
#pragma unroll
        for (int n = 0; n < 64; n += 8) {
            const u32x4 x =
                __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, vo, first_channel(n) * 2, 0));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                S.t[n >> 4][(n & 15) + 2 * e] = lo_f(x[e]);
                S.t[n >> 4][(n & 15) + 2 * e + 1] = hi_f(x[e]);
            }
        }
    } else if (tr) {
#pragma unroll
        for (int n = 0; n < 64; ++n)
            S.t[n >> 4][n & 15] =
                __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, vo, first_channel(n) * kD * 4, 0));
    } else {
#pragma unroll
        for (int n = 0; n < 64; n += 4) {
            const u32x4 x =
                __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, vo, first_channel(n) * 4, 0));
#pragma unroll
            for (int e = 0; e < 4; ++e)
                S.t[n >> 4][(n & 15) + e] = __uint_as_float(x[e]);
        }
    }
}

__device__ __forceinline__ void state_store(const State &S, void *base, int dt, bool tr, int wave, int lane)
{
    const int col = 32 * wave + (lane & 31), half = lane >> 5;
    const int size = dt == kBf16 ? 2 : 4;
    const __amdgpu_buffer_rsrc_t r = rsrc(base, (uint32_t)(kD * kD * size));
    const int vo = (tr ? 8 * half * kD + col : col * kD + 8 * half) * size;
    if (dt == kBf16 && tr) {
#pragma unroll
        for (int n = 0; n < 64; ++n)
            __builtin_amdgcn_raw_buffer_store_b16((short)to_bf16(S.t[n >> 4][n & 15]), r, vo,
                                                  first_channel(n) * kD * 2, 0);
    } else if (dt == kBf16) {
#pragma unroll
        for (int n = 0; n < 64; n += 8) {
            u32x4 x;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                x[e] = pack2(S.t[n >> 4][(n & 15) + 2 * e], S.t[n >> 4][(n & 15) + 2 * e + 1]);
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4, x), r, vo, first_channel(n) * 2, 0);
        }
    } else if (tr) {
#pragma unroll
        for (int n = 0; n < 64; ++n)
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S.t[n >> 4][n & 15]), r, vo,
                                                  first_channel(n) * kD * 4, 0);
    } else {
#pragma unroll
        for (int n = 0; n < 64; n += 4) {
            const f32x4 x = {S.t[n >> 4][n & 15], S.t[n >> 4][(n & 15) + 1], S.t[n >> 4][(n & 15) + 2],
                             S.t[n >> 4][(n & 15) + 3]};
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4, x), r, vo, first_channel(n) * 4, 0);
        }
    }
}

// <S, X> over the workgroup's 128 x 128 entries (X fp32), this thread's share
__device__ __forceinline__ float state_dot(const State &S, const float *base, bool tr, int wave, int lane)
{
    const int col = 32 * wave + (lane & 31), half = lane >> 5;
    const __amdgpu_buffer_rsrc_t r = rsrc(base, (uint32_t)kLinStateBytes);
    const int vo = (tr ? 8 * half * kD + col : col * kD + 8 * half) * 4, step = (tr ? kD : 1) * 4;
    float d = 0.0f;
#pragma unroll
    for (int n = 0; n < 64; ++n)
        d = fmaf(S.t[n >> 4][n & 15],
                 __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, vo, first_channel(n) * step, 0)), d);
    return d;
}

__device__ __forceinline__ void state_scale(State &S, float f)
{
#pragma unroll
    for (int n = 0; n < 64; ++n)
        S.t[n >> 4][n & 15] *= f;
}

// ------------------------------------------------------------------------------- LDS

struct Decays {           // of one chunk, natural order of tokens
    float bh[kLC], bl[kLC];  // running sum of log2 decays, as a pair
    float wout[kLC];         // factor of the state's share of an output row
    float win[kLC];          // factor of a source row on its way into the state
    double held;             // log2 of the factor that the registers' state lacks after the chunk
    float mul;               // factor to put into the registers' state now; 1: none
    float pad;
};

// The state in registers lacks a common factor 2^held, -16 < held <= 0: decays gather there and reach the 64 registers
// when they come to 2^-16 or less.  Slow decays would otherwise round the state in every chunk, by the same
// factor each time, and drift.  Rows go in with 2^-held and come out with 2^held.
constexpr double kMostHeld = -16.0;

constexpr int kTile = kLC * 256;
constexpr int kPRow = 128;  // bytes per row of the 64 x 64 weight matrix

struct LdsWalk {
    unsigned char k[kTile], v[kTile], q[kTile];
    unsigned char p[3][kLC * kPRow];  // weights, hi, mid and lo terms, [out token][source token]
    Decays d[2];
};
struct LdsWalkDots {
    LdsWalk w;
    float red[4][kLC];
    float own[kLC];                 // weights of the tokens' own pairs
};
struct LdsStates {
    unsigned char k[2][kTile], v[2][kTile];
    float win[2][kLC];
    double after[2];  // log2 of the factor between the chunk's far end and the segment's boundary
    int nan[4];       // a wave's share of the rows that were not read has a decay that is NaN
};

template <int kCtrl, int kRows>
__device__ __forceinline__ double dpp_f64(double x)  // 0 where the pattern has no source lane
{
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, kCtrl, kRows, 0xf, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), kCtrl, kRows, 0xf, false);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// Running sum of the chunk's log2 decays (lane = token), and their sum.
__device__ __forceinline__ void decay_sums(float g, int len, int lane, double &b, double &last)
{
    b = lane < len ? (double)clamp_decay(g) * kLog2e64 : 0.0;
    // inclusive sum: shifts by 1, 2, 4, 8 inside each 16 lanes, then the last lane of row 0 and 2 to the next
    // row, then lane 31 to the upper half
    b += dpp_f64<0x111, 0xf>(b);
    b += dpp_f64<0x112, 0xf>(b);
    b += dpp_f64<0x114, 0xf>(b);
    b += dpp_f64<0x118, 0xf>(b);
    b += dpp_f64<0x142, 0xa>(b);
    b += dpp_f64<0x143, 0xc>(b);
    const uint64_t u = __builtin_bit_cast(uint64_t, b);
    last = __builtin_bit_cast(
        double, ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), 63) << 32) |
                    (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, 63));
}

// `held` as it stands before the chunk, and after it
__device__ __forceinline__ void make_decays(Decays &d, double &held, float g, const Chunk &c, int lane, bool rev, float scale)
{
    if (c.flags & kPieceStart)
        held = 0.0;
    double b, last;
    decay_sums(g, c.len, lane, b, last);
    const double after = held + last;
    const bool apply = !(after > kMostHeld);  // also for NaN
    const float bh = (float)b;
    d.bh[lane] = bh;
    d.bl[lane] = (float)(b - (double)bh);
    const double head = b, tail = last - b, in = apply ? 0.0 : after;
    d.wout[lane] = (rev ? 1.0f : scale) * __builtin_amdgcn_exp2f((float)((rev ? tail : head) + held));
    d.win[lane] = (rev ? scale : 1.0f) * __builtin_amdgcn_exp2f((float)((rev ? head : tail) - in));
    if (lane == 0) {
        d.held = in;
        d.mul = apply ? __builtin_amdgcn_exp2f((float)after) : 1.0f;
    }
    held = in;
}

// The decay of token `lane` of the chunk (0 behind it, and all 0 without a chunk); p: this workgroup's row and head
__device__ __forceinline__ float load_decay(const LinArgs &a, const float *p, const Chunk &c, int lane)
{
    const uint32_t step = a.per_token ? (uint32_t)a.H * 4u : 0u;
    const __amdgpu_buffer_rsrc_t r =
        rsrc(p + (a.per_token ? c.t0 * a.H : 0), c.len > 0 ? (uint32_t)(c.len - 1) * step + 4u : 0u);
    return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, (uint32_t)lane * step, 0, 0));
}
__device__ __forceinline__ const float *decay_of(const LinArgs &a, int64_t row, int64_t h)
{
    return a.decay + (a.per_token ? row * a.T * a.H : 0) + h;
}

// One input of the walk: this workgroup's row and head.
struct TileSrc {
    const uint16_t *p;
    uint32_t st;  // elements from token to token, below 2^24
};
__device__ __forceinline__ TileSrc tile_src(const LinTensor &x, int64_t row, int64_t h)
{
    // heads are shared by small whole numbers: 32-bit division
    return TileSrc{x.p + row * x.sb + (int64_t)((uint32_t)h / (uint32_t)x.share) * x.sh, (uint32_t)x.st};
}
struct TileLoad {
    u32x4 r[4];
};
// 64 rows of 256 bytes; rows behind the chunk lie beyond the descriptor (the token stride is at least
// a row, see lin_api.cpp) and read as zeros.  Without a chunk (len 0) nothing is read, by the same instructions: a
// branch around them would make the compiler wait for all loads wherever older ones are used.
__device__ __forceinline__ void tile_fetch(TileLoad &f, const TileSrc &x, const Chunk &c, int tid)
{
    const uint32_t stride = x.st * 2;
    const __amdgpu_buffer_rsrc_t r = rsrc(x.p + c.t0 * x.st, c.len > 0 ? (uint32_t)(c.len - 1) * stride + 256u : 0u);
    __asm__ volatile("" : "+v"(tid));  // the offsets are formed anew: kept from chunk to chunk they would cost 12 registers
    const uint32_t off = (uint32_t)(tid >> 4) * stride + (uint32_t)(tid & 15) * 16u;
#pragma unroll
    for (int n = 0; n < 4; ++n)
        f.r[n] = buf_b128(r, off + (uint32_t)n * 16u * stride);
}

// This lane's places in the LDS tiles, as byte offsets.  The XOR of tile_at() reaches the three low bits of a
// piece's number only, so a few bases and the instruction's own offset reach everything.
struct Lanes {
    int put;        // row tid / 16 (+ 16 n), piece tid % 16 of a tile
    int row[4];     // row lane % 32 (+ 32), piece 2 v + half (+ 8)
    int trv[2];     // transposing read of this wave's columns: token 8 half (+ 16 j) + 4 n
    int trk[2][2];  // [kt % 2][n]: the same of channels 32 kt .. (+ 64), in the order of the state's registers
    int w[4];       // weights of out token lane % 32 (+ 32), source piece 2 v + half

    __device__ Lanes(int tid)
    {
        const int lane = tid & 63, wave = tid >> 6, l32 = lane & 31, half = lane >> 5, i = lane & 15, g2 = (lane >> 4) & 1;
        const int fg = ((i & 1) << 1) | ((i >> 1) & 1);
        put = tile_at(tid >> 4, tid & 15);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            row[v] = tile_at(l32, 2 * v + half);
            w[v] = l32 * kPRow + (((2 * v + half) ^ (l32 & 7)) << 4);
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int tok = 8 * half + 4 * n + (i >> 2);
            trv[n] = tile_at(tok, 4 * wave + 2 * g2 + ((i & 3) >> 1)) + 8 * (i & 1);
#pragma unroll
            for (int kt = 0; kt < 2; ++kt)
                trk[kt][n] = tile_at(tok, 4 * kt + 2 * g2 + (fg >> 1)) + 8 * (fg & 1);
        }
    }
};

__device__ __forceinline__ void tile_put(const TileLoad &f, unsigned char *tile, const Lanes &ln)
{
#pragma unroll
    for (int n = 0; n < 4; ++n)
        *reinterpret_cast<u32x4 *>(tile + ln.put + 4096 * n) = f.r[n];
}
// 16 channels, 16 jj .., of row lane % 32 of a block of 32 rows
__device__ __forceinline__ u32x4 row_frag(const unsigned char *tile, const Lanes &ln, int block, int jj)
{
    return lds_b128(tile + ln.row[jj & 3] + 8192 * block + 128 * (jj >> 2));
}
// 8 of the 16 tokens 16 j .. of this lane's column
__device__ __forceinline__ u32x4 col_frag(const unsigned char *tile, const Lanes &ln, int j)
{
    const u32x2 x = lds_tr(tile + ln.trv[0] + 4096 * j), y = lds_tr(tile + ln.trv[1] + 4096 * j);
    return u32x4{x[0], x[1], y[0], y[1]};
}
__device__ __forceinline__ u32x4 key_frag(const unsigned char *tile, const Lanes &ln, int kt, int j)
{
    const int off = 4096 * j + 128 * (kt >> 1);
    const u32x2 x = lds_tr(tile + ln.trk[kt & 1][0] + off), y = lds_tr(tile + ln.trk[kt & 1][1] + off);
    return u32x4{x[0], x[1], y[0], y[1]};
}

// Cutting floats into bf16 terms: what a rounded pair leaves of each, x - hi(x), exact.
struct Cutter {
    __device__ float rest0(uint32_t pair, float x) const { return x - lo_f(pair); }
    __device__ float rest1(uint32_t pair, float x) const { return x - hi_f(pair); }
};
// The same as one dot product each, (hi0, hi1).(-1, 0) + x: fewer registers, but dot products wait for the matrix pipe.
// The two constants live in registers: as an instruction's constant the compiler puts both into the same half.
struct DotCutter {
    uint32_t neg0, neg1;

    __device__ DotCutter() : neg0(0x0000bf80u), neg1(0xbf800000u) { __asm__ volatile("" : "+v"(neg0), "+v"(neg1)); }
    __device__ float rest0(uint32_t pair, float x) const
    {
        return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, pair), __builtin_bit_cast(bf16x2, neg0), x,
                                               false);
    }
    __device__ float rest1(uint32_t pair, float x) const
    {
        return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, pair), __builtin_bit_cast(bf16x2, neg1), x,
                                               false);
    }
};
template <bool kDots>
struct CutterOf {
    using type = Cutter;
};
template <>
struct CutterOf<true> {
    using type = DotCutter;
};
struct Terms3 {
    u32x4 h, m, l;
};
template <typename Cut>
__device__ __forceinline__ void cut_terms(const float *x, Terms3 &t, const Cut &cut)
{
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        t.h[e] = pack2(x[2 * e], x[2 * e + 1]);
        const float a1 = cut.rest0(t.h[e], x[2 * e]), b1 = cut.rest1(t.h[e], x[2 * e + 1]);
        t.m[e] = pack2(a1, b1);
        t.l[e] = pack2(cut.rest0(t.m[e], a1), cut.rest1(t.m[e], b1));
    }
}

// S += sum over the chunk's tokens of (win v) k^T.  Source rows are weighted on the way in,
// in fp32, and go into the product as three bf16 terms.
//
// Steps of 16 tokens, in a pipeline by hand: while a step's 12 matrix instructions run, the next step's K
// operand is on its way from LDS and its weighted rows are cut.
template <typename Cut>
__device__ __forceinline__ void weighted_terms(Terms3 &t, const u32x4 &v, const float *win, int tok, const Cut &cut)
{
    const f32x4 w0 = *reinterpret_cast<const f32x4 *>(&win[tok]);
    const f32x4 w1 = *reinterpret_cast<const f32x4 *>(&win[tok + 4]);
    float x[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        x[2 * e] = lo_f(v[e]) * (e < 2 ? w0[2 * e] : w1[2 * e - 4]);
        x[2 * e + 1] = hi_f(v[e]) * (e < 2 ? w0[2 * e + 1] : w1[2 * e - 3]);
    }
    cut_terms(x, t, cut);
}

// The scheduler keeps the order of these groups: n x { 1 matrix instruction, v vector instructions }.
template <int kN, int kV>
__device__ __forceinline__ void interleave()
{
#pragma unroll
    for (int x = 0; x < kN; ++x) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, kV, 0);
    }
}

template <bool kAhead, typename Cut>
__device__ __forceinline__ void state_update(State &S, const unsigned char *ktile, const u32x4 *vf, const float *win,
                                             const Lanes &ln, int half, const Cut &cut)
{
    if constexpr (!kAhead) {  // where registers are short
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            u32x4 kf[4];
            Terms3 t;
#pragma unroll
            for (int kt = 0; kt < 4; ++kt)
                kf[kt] = key_frag(ktile, ln, kt, j);
            weighted_terms(t, vf[j], win, 16 * j + 8 * half, cut);
#pragma unroll
            for (int kt = 0; kt < 4; ++kt)
                S.t[kt] = mfma(kf[kt], t.l, S.t[kt]);
#pragma unroll
            for (int kt = 0; kt < 4; ++kt)
                S.t[kt] = mfma(kf[kt], t.m, S.t[kt]);
#pragma unroll
            for (int kt = 0; kt < 4; ++kt)
                S.t[kt] = mfma(kf[kt], t.h, S.t[kt]);
            __builtin_amdgcn_sched_barrier(0);
        }
        return;
    }
    u32x4 kf[2][4];
    Terms3 t[2];
#pragma unroll
    for (int kt = 0; kt < 4; ++kt)
        kf[0][kt] = key_frag(ktile, ln, kt, 0);
    weighted_terms(t[0], vf[0], win, 8 * half, cut);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int c = j & 1;
        if (j < 3) {
#pragma unroll
            for (int kt = 0; kt < 4; ++kt)
                kf[c ^ 1][kt] = key_frag(ktile, ln, kt, j + 1);
            __builtin_amdgcn_sched_barrier(0);
            weighted_terms(t[c ^ 1], vf[j + 1], win, 16 * (j + 1) + 8 * half, cut);
        }
#pragma unroll
        for (int kt = 0; kt < 4; ++kt)
            S.t[kt] = mfma(kf[c][kt], t[c].l, S.t[kt]);
#pragma unroll
        for (int kt = 0; kt < 4; ++kt)
            S.t[kt] = mfma(kf[c][kt], t[c].m, S.t[kt]);
#pragma unroll
        for (int kt = 0; kt < 4; ++kt)
            S.t[kt] = mfma(kf[c][kt], t[c].h, S.t[kt]);
        if (j < 3)
            interleave<12, 5>();
        __builtin_amdgcn_sched_barrier(0);
    }
}

// Two workgroups share a CU, and the older one's waves go first: it would finish at nearly full speed, then the younger one
// would run its second half alone.  Priorities that fall over 8 chunks and start again keep them close: the one behind goes
// first.  T = 262144, H = 8: 673 -> 646 us in all, when it was built.  Only where all workgroups run at once: with more, the place that one
// leaves early goes to the next (B = 2, T = 4096, H = 16 backwards, 768 workgroups, then: 205 us, 213 with turns).
__device__ __forceinline__ void take_turn(uint32_t token)
{
    const uint32_t p = (token / (2 * kLC)) & 3;
    if (p == 0)
        __builtin_amdgcn_s_setprio(3);
    else if (p == 1)
        __builtin_amdgcn_s_setprio(2);
    else if (p == 2)
        __builtin_amdgcn_s_setprio(1);
    else
        __builtin_amdgcn_s_setprio(0);
}

// Block -> (segment, head): the blocks of one XCD (every eighth) take neighbouring heads, so that
// heads that share q/k rows, and the lines of per-token decays, meet in one L2.
__device__ __forceinline__ int64_t xcd_order(int64_t id, int64_t total)
{
    const int64_t per = (total + 7) >> 3;
    return (id & 7) * per + (id >> 3);
}

__device__ __forceinline__ bool device_bad(const LinArgs &a) { return a.cu && *a.status != 0; }

// ------------------------------------------------------------------------- states pass
//
// Each segment's share of the state at its boundary: the last sequence of a forward walk if it
// goes on behind the segment, the first one of a reverse walk if it began before it.  lam:
// the factor on the state at the segment's other boundary, or -1 when the share is the whole
// state (the sequence starts inside), -2 when there is none.
//
// The chunks are taken from the boundary inwards, each row weighted with its whole factor up to the boundary,
// so the sum itself is never scaled; once that factor is below 2^-150, 0 in fp32, the chunks further in
// add nothing and are not read, but for their decays: one that is NaN makes the share NaN.  Tiles are in LDS twice, 64 KiB, one barrier a chunk.  Bound by memory (T = 262144,
// H = 8, per-token decays: 65 us, 3.6 TB/s) where segments are short, else by a chunk's latency, 2.5 us.
constexpr double kGone = -150.0;

__device__ __forceinline__ void states(const LinArgs &a, const LinRole &ro, int64_t seg, int64_t h, LdsStates &lds)
{
    const int64_t row = seg / a.P, j = seg - row * a.P;
    const bool rev = ro.rev != 0, tr = ro.transposed != 0;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), half = lane >> 5;
    const int64_t slot = seg * a.H + h;
    float *lam = ro.lam + slot;
    const bool edge = rev ? j == 0 : j == a.P - 1;  // nothing beyond this boundary
    Walk w;
    w.init(a, row, j, rev);
    w.i = rev ? w.first : w.last;
    if (!edge && !device_bad(a))
        w.set_piece();
    const int64_t nc = w.nc;
    if (nc == 0 || (w.pflags & kToFinal)) {
        if (tid == 0)
            *lam = -2.0f;
        return;
    }
    auto chunk = [&](int64_t n) {  // the n-th from the boundary
        Chunk c;
        const int64_t at_n = rev ? n : nc - 1 - n;
        c.t0 = w.p0 + at_n * kLC;
        const int64_t rest = w.p1 - c.t0;
        c.len = (int)(rest < kLC ? rest : kLC);
        c.seq = 0;
        c.flags = 0;
        return c;
    };
    const TileSrc sk = tile_src(ro.k, row, h), sv = tile_src(ro.v, row, h);
    const float *dp = decay_of(a, row, h);
    const Lanes ln(tid);
    const DotCutter cut;
    State S;
#pragma unroll
    for (int n = 0; n < 64; ++n)
        S.t[n >> 4][n & 15] = 0.0f;
    TileLoad fk, fv;
    Chunk c = chunk(0);
    float g = load_decay(a, dp, c, lane);
    tile_fetch(fk, sk, c, tid);
    tile_fetch(fv, sv, c, tid);
    double gone = 0.0;  // wave 3: log2 factor from the boundary to the next chunk's near end
    auto sources = [&](int buf, float gn, int len) {
        double b, last;
        decay_sums(gn, len, lane, b, last);
        lds.win[buf][lane] =
            (rev ? a.scale : 1.0f) * __builtin_amdgcn_exp2f((float)((rev ? b : last - b) + gone));
        gone += last;
        if (lane == 0)
            lds.after[buf] = gone;
    };
    if (wave == 3)
        sources(0, g, c.len);
    if (nc > 1)
        g = load_decay(a, dp, chunk(1), lane);
    double after = 0.0;
    int64_t n = 0;
    for (;; ++n) {
        const int buf = (int)(n & 1);
        tile_put(fk, lds.k[buf], ln);
        tile_put(fv, lds.v[buf], ln);
        lds_barrier();
        after = lds.after[buf];
        const bool more = n + 1 < nc && !(after < kGone);
        Chunk next = c;
        if (more) {
            next = chunk(n + 1);
            tile_fetch(fk, sk, next, tid);
            tile_fetch(fv, sv, next, tid);
        }
        u32x4 vf[4];
#pragma unroll
        for (int jj = 0; jj < 4; ++jj)
            vf[jj] = col_frag(lds.v[buf], ln, jj);
        state_update<true>(S, lds.k[buf], vf, lds.win[buf], ln, half, cut);
        if (!more)
            break;
        if (wave == 3)
            sources(buf ^ 1, g, next.len);
        if (n + 2 < nc)
            g = load_decay(a, dp, chunk(n + 2), lane);
        c = next;
    }
    const bool starts = !(w.pflags & kFromSlot);
    bool whole = starts;
    const float f = after < kGone ? 0.0f : __builtin_amdgcn_exp2f((float)after);
    if (a.per_token && n + 1 < nc) {
        const int64_t t0 = rev ? w.p0 + (n + 1) * kLC : w.p0, t1 = rev ? w.p1 : w.p0 + (nc - 1 - n) * kLC;
        bool nan = false;
        for (int64_t t = t0 + tid; t < t1; t += 256) {
            const float d = dp[t * a.H];
            nan = nan || d != d;
        }
        const bool any = __any(nan);
        if (lane == 0)
            lds.nan[wave] = any;
        lds_barrier();
        if (lds.nan[0] | lds.nan[1] | lds.nan[2] | lds.nan[3]) {
            whole = true;
#pragma unroll
            for (int e = 0; e < 64; ++e)
                S.t[e >> 4][e & 15] = __builtin_nanf("");
        }
    }
    if (starts && ro.init) {  // also with a factor of 0: what is not finite lasts
        State X;
        state_load(X, matrix_of(ro.init, w.seq_index() * a.H + h, kLinStateBytes / (ro.init_dt == kBf16 ? 2 : 1)),
                   ro.init_dt, tr, wave, lane);
#pragma unroll
        for (int n = 0; n < 64; ++n)
            S.t[n >> 4][n & 15] = fmaf(f, X.t[n >> 4][n & 15], S.t[n >> 4][n & 15]);
    }
    state_store(S, ro.slots + (size_t)slot * kD * kD, kFp32, tr, wave, lane);
    if (tid == 0)
        *lam = whole ? -1.0f : f;
}

__global__ __launch_bounds__(256, 2) void lin_states_kernel(LinArgs a, int lead0, int lead1)
{
    __shared__ __attribute__((aligned(16))) LdsStates lds;
    const int64_t total = a.rows * a.P * a.H;
    const int64_t at = xcd_order(blockIdx.x, total);
    if (at >= total || (int64_t)(blockIdx.x >> 3) >= ((total + 7) >> 3))
        return;
    const LinRole &ro = a.role[blockIdx.y == 0 ? lead0 : lead1];
    const int64_t seg = at / a.H, h = at - seg * a.H;
    states(a, ro, seg, h, lds);
}

// ---------------------------------------------------------------------------- scan
//
// slot_j <- share_j + lam_j * slot_{j-1} (forwards; backwards from the other end), so that slot
// j is the state at the boundary behind (before) segment j.  Every entry is its own chain: P steps of one fma, bound by
// memory.  Two entries a thread, the loads of 8 segments on their way together: B = 2, T = 4096, H = 16 backwards
// (512 slots of 64 KiB) 11 us, 4.9 TB/s.
constexpr unsigned kScanParts = kD * kD / 512;  // workgroups per matrix

__global__ __launch_bounds__(256) void lin_scan_kernel(LinArgs a, int lead0, int lead1)
{
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const LinRole &ro = a.role[blockIdx.y == 0 ? lead0 : lead1];
    const int64_t rh = blockIdx.x / kScanParts, row = rh / a.H, h = rh - row * a.H;
    const int e = ((blockIdx.x % kScanParts) * 256 + threadIdx.x) * 2;
    f32x2 s = {0.0f, 0.0f};
    const int64_t last = a.P - 2;  // steps 0 .. P - 2
    for (int64_t n = 0; n <= last; n += 8) {
        f32x2 f[8];
        float lam[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            const int64_t m = n + x <= last ? n + x : last;
            const int64_t slot = (row * a.P + (ro.rev ? a.P - 1 - m : m)) * a.H + h;
            lam[x] = ro.lam[slot];
            f[x] = *reinterpret_cast<const f32x2 *>(ro.slots + (size_t)slot * kD * kD + e);
        }
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            if (n + x > last || lam[x] == -2.0f)
                continue;
            // a factor of 0 joins what is not finite: it lasts
            if (!(lam[x] <= 0.0f) || (lam[x] == 0.0f && !(isfinite(s[0]) && isfinite(s[1])))) {
                const int64_t slot = (row * a.P + (ro.rev ? a.P - 1 - (n + x) : n + x)) * a.H + h;
                f[x][0] = fmaf(lam[x], s[0], f[x][0]);
                f[x][1] = fmaf(lam[x], s[1], f[x][1]);
                *reinterpret_cast<f32x2 *>(ro.slots + (size_t)slot * kD * kD + e) = f[x];
            }
            s = f[x];
        }
    }
}

// ---------------------------------------------------------------------------- output pass
//
// One workgroup walks the chunks of one segment and head: out^T[v][t] = S q^T scaled by wout, plus V^T times the
// 64 x 64 weights, then the state's update.  4 waves split the 128 v channels, so each holds 128 x 32 of the state in 64
// registers a lane from chunk to chunk and the transposed products need no exchange between waves; the weights,
// one 32 x 32 block a wave, are the one thing they share.  74 KiB of LDS and 256 registers a lane let two workgroups
// share a CU.  The next chunk's rows are loaded into registers while this one is worked on; three barriers a chunk.
//
// Per chunk a wave issues 122 matrix instructions (weights 8, the state's share 48, the weights' products 18, the update
// 48) and, counted, some 1130 other vector instructions (the greater part of them the cuts of state, weights and rows into
// bf16 terms), 150 scalar, 143 LDS and 17 memory ones; two waves a SIMD, it is the issue of these that bounds the walk.
// T = 262144, H = 8: 616 us, 2.2 GB at 3.6 TB/s; the same loads and stores without the arithmetic took 466 us.  38000
// packed tokens, H = 32, Hk = 8: 337 us, 2.5 TB/s.  The three walks of a backward pass with dots (75 KiB), B = 2, T = 4096,
// H = 16: 141 us, 3.6 TB/s.  512 threads with the state's channels in halves, one workgroup a CU, was slower (T = 262144:
// 740 us in all against 667, with two terms).

// kDots: roles with dots also give the rows' products with x's rows, the tokens' own pairs left
// out.  Their sums over many tokens cancel, so the own pairs are added to the rows outside the matrix product.
template <bool kDots, bool rev>
__device__ __forceinline__ void walk(const LinArgs &a, const LinRole &ro, int64_t seg, int64_t h, unsigned char *lds_raw)
{
    LdsWalk &lds = *reinterpret_cast<LdsWalk *>(lds_raw);
    LdsWalkDots &ldx = *reinterpret_cast<LdsWalkDots *>(lds_raw);  // behind lds only with kDots
    const int64_t row = seg / a.P, j = seg - row * a.P;
    const bool tr = ro.transposed != 0;
    const bool dots = kDots && ro.dots != nullptr;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int half = lane >> 5, l32 = lane & 31;
    const Lanes ln(tid);
    const typename CutterOf<kDots>::type cut;
    const size_t init_bytes = kLinStateBytes / (ro.init_dt == kBf16 ? 2 : 1);
    const size_t fin_bytes = kLinStateBytes / (ro.fin_dt == kBf16 ? 2 : 1);
    State S;

    Walk w;
    const bool bad = device_bad(a);
    if (!bad)
        w.init(a, row, j, rev);
    // sequences without tokens keep their state
    if (ro.fin && (a.cu || a.T == 0)) {
        const int64_t lo = bad ? 0 : w.first, hi = bad ? (seg == 0 ? a.N - 1 : -1) : w.last;
        for (int64_t n = lo; n <= hi; ++n) {
            const int64_t s0 = a.cu && !bad ? a.cu[n] : 0, s1 = a.cu && !bad ? a.cu[n + 1] : 0;
            if (s0 != s1 || (!bad && s0 < w.r0))
                continue;
            const int64_t sq = a.cu ? n : row;
            state_load(S, matrix_of(ro.init, sq * a.H + h, init_bytes), ro.init_dt, tr, wave, lane);
            state_store(S, static_cast<unsigned char *>(ro.fin) + (size_t)(sq * a.H + h) * fin_bytes, ro.fin_dt, tr,
                        wave, lane);
        }
    }
    if (bad)
        return;

    Chunk c = w.next();
    if (c.len == 0)
        return;
    TileLoad fq, fk, fv;
    const TileSrc sq = tile_src(ro.q, row, h), sk = tile_src(ro.k, row, h), sv = tile_src(ro.v, row, h);
    TileSrc sx = {nullptr, 0};
    if (dots)
        sx = tile_src(ro.x, row, h);
    tile_fetch(fq, sq, c, tid);
    tile_fetch(fk, sk, c, tid);
    tile_fetch(fv, sv, c, tid);
    const float *dp = decay_of(a, row, h);
    float g = load_decay(a, dp, c, lane);
    double held = 0.0;
    if (wave == 3)
        make_decays(lds.d[0], held, g, c, lane, rev, a.scale);
    int buf = 0;
    while (c.len > 0) {
        if (a.turns)
            take_turn(rev ? ~(uint32_t)c.t0 : (uint32_t)c.t0);
        tile_put(fq, lds.q, ln);
        tile_put(fk, lds.k, ln);
        tile_put(fv, lds.v, ln);
        const Chunk n = w.next();
        u32x2 xr[2][4];  // x's rows of this chunk, older than the next chunk's rows: waiting for them does not wait for those
        if (dots) {
            const uint32_t xs = sx.st * 2;
            int tx = l32;
            __asm__ volatile("" : "+v"(tx));
            const __amdgpu_buffer_rsrc_t rx = rsrc(sx.p + c.t0 * sx.st, (uint32_t)(c.len - 1) * xs + 256u);
#pragma unroll
            for (int tt = 0; tt < 2; ++tt)
#pragma unroll
                for (int a4 = 0; a4 < 4; ++a4)
                    xr[tt][a4] = __builtin_bit_cast(
                        u32x2, __builtin_amdgcn_raw_buffer_load_b64(
                                   rx, (uint32_t)(32 * tt + tx) * xs + (32 * wave + 4 * half + 8 * a4) * 2, 0, 0));
        }
        g = load_decay(a, dp, n, lane);
        // the other rows follow further down: 12 loads at once would fill the queue and hold the wave up (packed prompts 397 ->
        // 379 us in all, with two terms)
        tile_fetch(fq, sq, n, tid);
        if (c.flags & kPieceStart) {
            const bool slot = (c.flags & kFromSlot) != 0;
            state_load(S,
                       slot ? matrix_of(ro.slots, (seg + (rev ? 1 : -1)) * a.H + h, kLinStateBytes)
                            : matrix_of(ro.init, c.seq * a.H + h, init_bytes),
                       slot ? (int)kFp32 : ro.init_dt, tr, wave, lane);
            // here, or the compiler waits in every chunk, for the rows on their way too
            __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
        }
        lds_barrier();
        const Decays &d = lds.d[buf];

        // The weights of one 32 x 32 block (sources sb, outputs ob) per wave, in three terms (wave 3's block lies beyond
        // the diagonal: zeros, never read), and the state's share of the outputs, O^T[v][t].  In steps of 16 channels: a
        // step's products with the state run while the next 16 channels of the state are cut and every other step makes
        // 4 of the lane's 16 weights.
        f32x16 O[2];
        {
            const int sb = wave == 0 ? 0 : wave == 2 ? 1 : (wave == 1) == rev ? 1 : 0;
            const int ob = wave == 0 ? 0 : wave == 2 ? 1 : (wave == 1) == rev ? 0 : 1;
            f32x16 p;
#pragma unroll
            for (int r = 0; r < 16; ++r)
                p[r] = O[0][r] = O[1][r] = 0.0f;
            constexpr int kGroup = kDots ? 4 : 8;  // operands on their way together
#pragma unroll
            for (int j0 = 0; j0 < 8; j0 += kGroup) {
                u32x4 kr[kGroup], qr[kGroup];
#pragma unroll
                for (int jj = 0; jj < kGroup; ++jj) {
                    kr[jj] = row_frag(lds.k, ln, sb, j0 + jj);
                    qr[jj] = row_frag(lds.q, ln, ob, j0 + jj);
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int jj = 0; jj < kGroup; ++jj)
                    p = mfma(kr[jj], qr[jj], p);
            }
            __builtin_amdgcn_sched_barrier(0);
            tile_fetch(fk, sk, n, tid);
            __builtin_amdgcn_sched_barrier(0);
            int to = 32 * ob + l32;
            __asm__ volatile("" : "+v"(to));  // keep the comparisons below in the loop: 16 masks would not stay in SGPRs
            const float bho = d.bh[to], blo = d.bl[to];
            auto weights = [&](int a4) {
                const int s = 32 * sb + 8 * a4 + 4 * half;
                const f32x4 bhs = *reinterpret_cast<const f32x4 *>(&d.bh[s]);
                const f32x4 bls = *reinterpret_cast<const f32x4 *>(&d.bl[s]);
                float x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float df = rev ? (bhs[e] - bho) + (bls[e] - blo) : (bho - bhs[e]) + (blo - bls[e]);
                    const bool on = rev ? s + e >= to : s + e <= to;  // a token behind the row's (before it) weighs nothing
                    x[e] = on ? p[4 * a4 + e] * (a.scale * __builtin_amdgcn_exp2f(df)) : 0.0f;
                    if (dots && s + e == to) {
                        ldx.own[to] = x[e];
                        x[e] = 0.0f;
                    }
                }
                const u32x2 hi = {pack2(x[0], x[1]), pack2(x[2], x[3])};
                const float y[4] = {cut.rest0(hi[0], x[0]), cut.rest1(hi[0], x[1]), cut.rest0(hi[1], x[2]),
                                    cut.rest1(hi[1], x[3])};
                const u32x2 mid = {pack2(y[0], y[1]), pack2(y[2], y[3])};
                const int off = to * kPRow + (((4 * sb + a4) ^ (to & 7)) << 4) + 8 * half;
                *reinterpret_cast<u32x2 *>(lds.p[0] + off) = hi;
                *reinterpret_cast<u32x2 *>(lds.p[1] + off) = mid;
                *reinterpret_cast<u32x2 *>(lds.p[2] + off) =
                    u32x2{pack2(cut.rest0(mid[0], y[0]), cut.rest1(mid[0], y[1])),
                          pack2(cut.rest0(mid[1], y[2]), cut.rest1(mid[1], y[3]))};
            };
            u32x4 qf[2][2];
            Terms3 sc[2];
            auto cut_state = [&](int jj) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    x[e] = S.t[jj >> 1][8 * (jj & 1) + e];
                cut_terms(x, sc[jj & 1], cut);
            };
            if constexpr (kDots) {  // registers are short: no step ahead
#pragma unroll
                for (int jj = 0; jj < 8; ++jj) {
                    qf[0][0] = row_frag(lds.q, ln, 0, jj);
                    qf[0][1] = row_frag(lds.q, ln, 1, jj);
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        x[e] = S.t[jj >> 1][8 * (jj & 1) + e];
                    cut_terms(x, sc[0], cut);
#pragma unroll
                    for (int tt = 0; tt < 2; ++tt)
                        O[tt] = mfma(sc[0].l, qf[0][tt], O[tt]);
#pragma unroll
                    for (int tt = 0; tt < 2; ++tt)
                        O[tt] = mfma(sc[0].m, qf[0][tt], O[tt]);
#pragma unroll
                    for (int tt = 0; tt < 2; ++tt)
                        O[tt] = mfma(sc[0].h, qf[0][tt], O[tt]);
                    if (jj & 1)
                        weights(jj >> 1);
                    __builtin_amdgcn_sched_barrier(0);
                }
            } else {
                qf[0][0] = row_frag(lds.q, ln, 0, 0);
                qf[0][1] = row_frag(lds.q, ln, 1, 0);
                cut_state(0);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int jj = 0; jj < 8; ++jj) {
                    const int b = jj & 1;
                    if (jj < 7) {
                        qf[b ^ 1][0] = row_frag(lds.q, ln, 0, jj + 1);
                        qf[b ^ 1][1] = row_frag(lds.q, ln, 1, jj + 1);
                        __builtin_amdgcn_sched_barrier(0);
                        cut_state(jj + 1);
                    }
                    if (jj & 1)
                        weights(jj >> 1);
#pragma unroll
                    for (int tt = 0; tt < 2; ++tt)
                        O[tt] = mfma(sc[b].l, qf[b][tt], O[tt]);
#pragma unroll
                    for (int tt = 0; tt < 2; ++tt)
                        O[tt] = mfma(sc[b].m, qf[b][tt], O[tt]);
#pragma unroll
                    for (int tt = 0; tt < 2; ++tt)
                        O[tt] = mfma(sc[b].h, qf[b][tt], O[tt]);
                    if (jj & 1)
                        interleave<6, 14>();
                    else
                        interleave<6, 5>();
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
            const float wo = d.wout[32 * tt + l32];
#pragma unroll
            for (int r = 0; r < 16; ++r)
                O[tt][r] *= wo;
        }
        u32x4 vf[4];
#pragma unroll
        for (int jj = 0; jj < 4; ++jj)
            vf[jj] = col_frag(lds.v, ln, jj);
        __builtin_amdgcn_sched_barrier(0);
        tile_fetch(fv, sv, n, tid);
        __builtin_amdgcn_sched_barrier(0);
        lds_barrier();  // the weights are there
        {
            // weight operands: of each 16 sources the diagonal block's, and the block beside it for half of them
            constexpr int kBeside = rev ? 0 : 1;  // output block that sees all sources
            constexpr int kGroup = 2;
#pragma unroll
            for (int x0 = 0; x0 < 6; x0 += kGroup) {
                u32x4 wh[kGroup], wm[kGroup], wl[kGroup];
#pragma unroll
                for (int y = 0; y < kGroup; ++y) {
                    const int x = x0 + y, jj = x < 4 ? x : (rev ? x - 2 : x - 4), block = x < 4 ? x >> 1 : kBeside;
                    const int off = ln.w[jj] + 32 * kPRow * block;
                    wl[y] = lds_b128(lds.p[2] + off);
                    wm[y] = lds_b128(lds.p[1] + off);
                    wh[y] = lds_b128(lds.p[0] + off);
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int y = 0; y < kGroup; ++y) {
                    const int x = x0 + y, jj = x < 4 ? x : (rev ? x - 2 : x - 4), block = x < 4 ? x >> 1 : kBeside;
                    O[block] = mfma(vf[jj], wl[y], O[block]);
                    O[block] = mfma(vf[jj], wm[y], O[block]);
                    O[block] = mfma(vf[jj], wh[y], O[block]);
                }
            }
        }

        // Rows out; those behind the chunk lie beyond the descriptor.  A lane holds 4 neighbouring channels of a token:
        // stored like that, an instruction would touch 32 rows.  They change places in this wave's part of the
        // query and value tiles (read for the last time before the barrier above), so that it touches 16 (8 with fp32),
        // and leave after the state's update.  With dots registers are short and the value rows needed: stored as they are.
        const bool out_f32 = ro.out_f32 != 0;
        const uint32_t size = out_f32 ? 4 : 2, stride = (uint32_t)a.H * (kD * size);
        const __amdgpu_buffer_rsrc_t ra =
            rsrc(static_cast<unsigned char *>(ro.out) +
                     ((size_t)(row * a.T + c.t0) * (size_t)a.H + (size_t)h) * (kD * size),
                 (uint32_t)(c.len - 1) * stride + kD * size);
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
            const int t = 32 * tt + l32;
            int tv = l32;
            __asm__ volatile("" : "+v"(tv));  // as above: addresses formed anew
            if constexpr (kDots) {
                if (dots) {
                    const float own = ldx.own[t];
                    float dot = 0.0f;
#pragma unroll
                    for (int a4 = 0; a4 < 4; ++a4) {
                        f32x4 y = {O[tt][4 * a4], O[tt][4 * a4 + 1], O[tt][4 * a4 + 2], O[tt][4 * a4 + 3]};
                        const u32x2 xw = xr[tt][a4];
                        dot += (lo_f(xw[0]) * y[0] + hi_f(xw[0]) * y[1]) + (lo_f(xw[1]) * y[2] + hi_f(xw[1]) * y[3]);
                        const u32x2 vr = *reinterpret_cast<const u32x2 *>(lds.v + tile_at(tv, 4 * wave + a4) + 8 * half +
                                                                          8192 * tt);
                        O[tt][4 * a4] = fmaf(own, lo_f(vr[0]), y[0]);
                        O[tt][4 * a4 + 1] = fmaf(own, hi_f(vr[0]), y[1]);
                        O[tt][4 * a4 + 2] = fmaf(own, lo_f(vr[1]), y[2]);
                        O[tt][4 * a4 + 3] = fmaf(own, hi_f(vr[1]), y[3]);
                    }
                    dot += __shfl_xor(dot, 32);
                    if (half == 0)
                        ldx.red[wave][t] = dot;
                }
                const uint32_t o = (uint32_t)t * stride + (32 * wave + 4 * half) * size;
#pragma unroll
                for (int a4 = 0; a4 < 4; ++a4) {
                    const f32x4 y = {O[tt][4 * a4], O[tt][4 * a4 + 1], O[tt][4 * a4 + 2], O[tt][4 * a4 + 3]};
                    if (out_f32)
                        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4, y), ra, o + 32 * a4, 0, 0);
                    else
                        __builtin_amdgcn_raw_buffer_store_b64(
                            __builtin_bit_cast(u2, u32x2{pack2(y[0], y[1]), pack2(y[2], y[3])}), ra, o + 16 * a4, 0, 0);
                }
            } else if (out_f32) {  // 32 rows of 512 bytes, piece 8 wave + 2 a4 + half
                unsigned char *stage = tt ? lds.v : lds.q;
#pragma unroll
                for (int a4 = 0; a4 < 4; ++a4) {
                    const f32x4 y = {O[tt][4 * a4], O[tt][4 * a4 + 1], O[tt][4 * a4 + 2], O[tt][4 * a4 + 3]};
                    *reinterpret_cast<f32x4 *>(stage + tv * 512 + ((8 * wave + ((2 * a4 + half) ^ (tv & 7))) << 4)) = y;
                }
            } else {
#pragma unroll
                for (int a4 = 0; a4 < 4; ++a4)
                    *reinterpret_cast<u32x2 *>(lds.q + tile_at(tv, 4 * wave + a4) + 8 * half + 8192 * tt) =
                        u32x2{pack2(O[tt][4 * a4], O[tt][4 * a4 + 1]), pack2(O[tt][4 * a4 + 2], O[tt][4 * a4 + 3])};
            }
        }
        if (d.mul != 1.0f)
            state_scale(S, d.mul);
        state_update<!kDots>(S, lds.k, vf, d.win, ln, half, cut);
        if constexpr (!kDots) {
            int to = lane;
            __asm__ volatile("" : "+v"(to));
            if (out_f32) {
#pragma unroll
                for (int n8 = 0; n8 < 8; ++n8) {
                    const int t8 = 8 * (n8 & 3) + (to >> 3), pc = to & 7;
                    const u32x4 y = lds_b128((n8 < 4 ? lds.q : lds.v) + t8 * 512 + ((8 * wave + (pc ^ (t8 & 7))) << 4));
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4, y), ra,
                                                           (uint32_t)(32 * (n8 >> 2) + t8) * stride + (8 * wave + pc) * 16,
                                                           0, 0);
                }
            } else {
#pragma unroll
                for (int n4 = 0; n4 < 4; ++n4) {
                    const int t4 = to >> 2, pc = 4 * wave + (to & 3);
                    const u32x4 y = lds_b128(lds.q + tile_at(t4, pc) + 4096 * n4);
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4, y), ra,
                                                           (uint32_t)(16 * n4 + t4) * stride + pc * 16, 0, 0);
                }
            }
        }
        const double held_now = d.held;
        if (wave == 3 && n.len > 0)
            make_decays(lds.d[buf ^ 1], held, g, n, lane, rev, a.scale);
        lds_barrier();  // every read of this chunk's tiles is done
        if (dots && tid < c.len)
            ro.dots[(row * a.T + c.t0 + tid) * a.H + h] =
                (ldx.red[0][tid] + ldx.red[1][tid]) + (ldx.red[2][tid] + ldx.red[3][tid]);
        if ((c.flags & kPieceEnd) && (c.flags & kToFinal) && (ro.fin || (kDots && ro.xfin))) {
            state_scale(S, __builtin_amdgcn_exp2f((float)held_now));
            if (ro.fin && ro.defer && (c.flags & kFromSlot))
                state_store(S, ro.slots + (size_t)((seg - 1) * a.H + h) * kD * kD, kFp32, tr, wave, lane);
            else if (ro.fin)
                state_store(S, static_cast<unsigned char *>(ro.fin) + (size_t)(c.seq * a.H + h) * fin_bytes, ro.fin_dt,
                            tr, wave, lane);
            if (kDots && ro.xfin) {
                float x = state_dot(S, ro.xst + (size_t)(c.seq * a.H + h) * kD * kD, tr, wave, lane);
#pragma unroll
                for (int o = 32; o > 0; o >>= 1)
                    x += __shfl_xor(x, o);
                lds_barrier();
                if (lane == 0)
                    ldx.red[wave][0] = x;
                lds_barrier();
                if (tid == 0)
                    ro.xfin[c.seq * a.H + h] =
                        (ldx.red[0][0] + ldx.red[1][0]) + (ldx.red[2][0] + ldx.red[3][0]);
                lds_barrier();
            }
        }
        c = n;
        buf ^= 1;
    }
}

template <bool kDots>
__global__ __launch_bounds__(256, 2) void lin_walk_kernel(LinArgs a)
{
    __shared__ __attribute__((aligned(16))) unsigned char lds_raw[kDots ? sizeof(LdsWalkDots) : sizeof(LdsWalk)];
    const int64_t total = a.rows * a.P * a.H;
    const int64_t at = xcd_order(blockIdx.x, total);
    if (at >= total || (int64_t)(blockIdx.x >> 3) >= ((total + 7) >> 3))
        return;
    if (!a.cu && a.status && at == 0 && blockIdx.y == 0 && threadIdx.x == 0)
        *a.status = 0;
    const LinRole &ro = a.role[blockIdx.y];
    const int64_t seg = at / a.H, h = at - seg * a.H;
    if constexpr (kDots) {
        if (!ro.rev)
            walk<true, false>(a, ro, seg, h, lds_raw);
        else if (ro.dots)
            walk<true, true>(a, ro, seg, h, lds_raw);
        else
            walk<false, true>(a, ro, seg, h, lds_raw);
    } else {
        if (ro.rev)
            walk<false, true>(a, ro, seg, h, lds_raw);
        else
            walk<false, false>(a, ro, seg, h, lds_raw);
    }
}

// In-place state carry with cut rows: the workgroup that ends a sequence may finish before the one
// that starts it has read the initial state.  Final states of sequences that cross a
// boundary therefore wait in the slot that their last segment started from (it has been read,
// by the same threads) and move to their place here.
__global__ __launch_bounds__(256) void lin_final_kernel(LinArgs a)
{
    const LinRole &ro = a.role[0];
    const int64_t seg = blockIdx.x / a.H, h = blockIdx.x - seg * a.H;
    const int64_t row = seg / a.P, j = seg - row * a.P;
    if (j == 0 || device_bad(a))
        return;
    Walk w;
    w.init(a, row, j, false);
    w.i = w.first;
    w.set_piece();
    if (w.nc == 0 || !(w.pflags & kFromSlot) || !(w.pflags & kToFinal))
        return;
    const f32x4 *x = reinterpret_cast<const f32x4 *>(ro.slots + (size_t)((seg - 1) * a.H + h) * kD * kD);
    const size_t at = (size_t)(w.seq_index() * a.H + h) * kD * kD;
    for (int e = threadIdx.x; e < kD * kD / 4; e += 256) {
        const f32x4 y = x[e];
        if (ro.fin_dt == kFp32)
            reinterpret_cast<f32x4 *>(static_cast<float *>(ro.fin) + at)[e] = y;
        else
            reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(ro.fin) + at)[e] = u32x2{pack2(y[0], y[1]), pack2(y[2], y[3])};
    }
}

// ------------------------------------------------------------------- cu_seqlens, checked once
//
// The walks trust cu_seqlens, so nothing may run on one that leads out of the tensors.  One workgroup: a launch, 4.7 us.

__global__ __launch_bounds__(1024) void lin_check_kernel(const int64_t *cu, int64_t N, int64_t T, int32_t *status)
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

// ------------------------------------------------------------------- backward pass, tail

// Sum of the value heads that share a q/k head, in head order, rounded once.  One thread per 4 channels.  Bound by
// memory: 13500 tokens, H = 16, Hk = 4: 42 us, 5.9 TB/s.  Folding in the walk would need the states of all
// sharing heads in one workgroup, 64 KiB of registers each.
__global__ __launch_bounds__(256) void lin_fold_kernel(const float *xq, const float *xk, uint16_t *yq, uint16_t *yk,
                                                       int64_t rows, int64_t Hk, int64_t G, const int32_t *status)
{
    if (status && *status != 0)
        return;
    const float *x = blockIdx.y ? xk : xq;
    uint16_t *y = blockIdx.y ? yk : yq;
    const int64_t n = rows * Hk * (kD / 4);
    for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < n; at += (int64_t)gridDim.x * 256) {
        const int64_t r = at / (kD / 4);  // (token, q/k head)
        const float *p = x + r * G * kD + (at - r * (kD / 4)) * 4;
        f32x4 s = *reinterpret_cast<const f32x4 *>(p);
        for (int64_t g = 1; g < G; ++g)
            s += *reinterpret_cast<const f32x4 *>(p + g * kD);
        *reinterpret_cast<u32x2 *>(y + at * 4) = u32x2{pack2(s[0], s[1]), pack2(s[2], s[3])};
    }
}

constexpr int kGradThreads = (int)kLinGradSeg;  // a thread for each token of a segment

// Sum over the threads of a workgroup, in a fixed order; every thread gets it.
__device__ __forceinline__ double wg_sum(double x, double *red, int tid)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        x += __shfl_xor(x, o);
    __syncthreads();
    if ((tid & 63) == 0)
        red[tid >> 6] = x;
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int w = 0; w < kGradThreads / 64; ++w)
        s += red[w];
    return s;
}

// dg of one segment and head: from the end of each piece, where <S, dS> is known, back to its start.  Latency:
// the tokens' dots and the states are asked for together (T = 4096, H = 16, 5 segments: 14 -> 10 us against 256
// threads that took four turns).
__global__ __launch_bounds__(kGradThreads) void lin_ddecay_kernel(LinArgs a, float *ddecay, double *part)
{
    __shared__ double red[kGradThreads / 64];
    const int64_t seg = blockIdx.x / a.H, h = blockIdx.x - seg * a.H;
    const int64_t row = seg / a.P, j = seg - row * a.P;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    if (device_bad(a)) {
        if (!a.per_token && tid == 0)
            part[seg * a.H + h] = 0.0;
        return;
    }
    const LinRole &rq = a.role[0], &rk = a.role[1];
    Walk w;
    w.init(a, row, j, true);
    double total = 0.0;
    for (int64_t n = w.last; n >= w.first; --n) {
        w.i = n;
        w.set_piece();
        if (w.p1 <= w.p0)
            continue;
        // one token per thread: a piece is at most a segment long, see lin_plan
        const int64_t t = w.p0 + tid, at = (row * a.T + t) * a.H + h;
        const bool on = t < w.p1;
        const double x = on ? (double)rq.dots[at] - (double)rk.dots[at] : 0.0;
        double end = 0.0;
        if (w.pflags & kFromSlot) {
            const f32x4 *p = reinterpret_cast<const f32x4 *>(rq.slots + (size_t)(seg * a.H + h) * kD * kD);
            const f32x4 *q = reinterpret_cast<const f32x4 *>(rk.slots + (size_t)((seg + 1) * a.H + h) * kD * kD);
            float d = 0.0f;
#pragma unroll
            for (int e = 0; e < kD * kD / 4; e += kGradThreads) {
                const f32x4 y = p[e + tid], z = q[e + tid];
                d += (y[0] * z[0] + y[1] * z[1]) + (y[2] * z[2] + y[3] * z[3]);
            }
            end = wg_sum((double)d, red, tid);
        } else if (rq.xfin) {
            end = (double)rq.xfin[w.seq_index() * a.H + h];
        }
        double s = x;  // sum over this and the later tokens
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const double u = __shfl_down(s, o);
            if (lane + o < 64)
                s += u;
        }
        __syncthreads();
        if (lane == 0)
            red[wave] = s;
        __syncthreads();
        for (int k = kGradThreads / 64 - 1; k > wave; --k)
            end += red[k];
        if (on) {
            const double dg = end + s;
            if (a.per_token) {
                const float g = a.decay[at];
                ddecay[at] = g > kLowest && g <= 0.0f ? (float)dg : 0.0f;
            } else {
                total += dg;
            }
        }
    }
    if (!a.per_token) {
        total = wg_sum(total, red, tid);
        if (tid == 0)
            part[seg * a.H + h] = total;
    }
}

__global__ __launch_bounds__(64) void lin_ddecay_sum_kernel(LinArgs a, const double *part, float *ddecay)
{
    const int64_t h = blockIdx.x;
    double s = 0.0;
    for (int64_t n = threadIdx.x; n < a.rows * a.P; n += 64)
        s += part[n * a.H + h];
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        s += __shfl_xor(s, o);
    if (threadIdx.x == 0) {
        const float g = a.decay[h];
        ddecay[h] = g > kLowest && g <= 0.0f ? (float)s : 0.0f;
    }
}

// ------------------------------------------------------------------- token by token
//
// One wave per (sequence, head, 32 rows of the state); lane = row % 8 * 8 + q holds 16 channels
// of 4 rows: 16-byte pieces, interleaved with those of the row's other 7 lanes.  The state is read once and written once,
// which bounds it: 256 sequences, H = 32, fp32: 207 us, 5.2 TB/s.  Waves share nothing; few of them are
// launched as workgroups of one wave, to reach more CUs (H = 8, one sequence: 4.5 us).
template <bool kF32>
__global__ __launch_bounds__(256) void lin_recurrent_kernel(LinArgs a)
{
    constexpr int kPer = kF32 ? 4 : 8;     // channels per 16-byte piece
    constexpr int kPieces = 16 / kPer;     // pieces per row and lane
    const LinRole &ro = a.role[0];
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
    for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            const size_t at = mat + (size_t)(v0 + 8 * g + r8) * kD + (8 * p + q8) * kPer;
            if (!ro.init) {
#pragma unroll
                for (int e = 0; e < kPer; ++e)
                    S[g][p * kPer + e] = 0.0f;
            } else if constexpr (kF32) {
                const f32x4 x = *reinterpret_cast<const f32x4 *>(static_cast<const float *>(ro.init) + at);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    S[g][p * 4 + e] = x[e];
            } else {
                const u32x4 x = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(ro.init) + at);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    S[g][p * 8 + 2 * e] = lo_f(x[e]);
                    S[g][p * 8 + 2 * e + 1] = hi_f(x[e]);
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
    for (int64_t t = t0; t < t1; ++t) {
        const uint16_t *qp = ro.q.p + row * ro.q.sb + t * ro.q.st + (h / ro.q.share) * ro.q.sh;
        const uint16_t *kp = ro.k.p + row * ro.k.sb + t * ro.k.st + (h / ro.k.share) * ro.k.sh;
        const uint16_t *vp = ro.v.p + row * ro.v.sb + t * ro.v.st + (h / ro.v.share) * ro.v.sh;
        const int64_t tok = row * a.T + t;
        const float al = __builtin_amdgcn_exp2f(
            (float)((double)clamp_decay(a.per_token ? a.decay[tok * a.H + h] : a.decay[h]) * kLog2e64));
        float qv[16], kv[16], o[4];
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            const int ch = (8 * p + q8) * kPer;
#pragma unroll
            for (int e = 0; e < kPer; e += 4) {
                const u32x2 x = *reinterpret_cast<const u32x2 *>(qp + ch + e);
                const u32x2 y = *reinterpret_cast<const u32x2 *>(kp + ch + e);
                qv[p * kPer + e] = lo_f(x[0]);
                qv[p * kPer + e + 1] = hi_f(x[0]);
                qv[p * kPer + e + 2] = lo_f(x[1]);
                qv[p * kPer + e + 3] = hi_f(x[1]);
                kv[p * kPer + e] = lo_f(y[0]);
                kv[p * kPer + e + 1] = hi_f(y[0]);
                kv[p * kPer + e + 2] = lo_f(y[1]);
                kv[p * kPer + e + 3] = hi_f(y[1]);
            }
        }
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const float vv = __uint_as_float((uint32_t)vp[v0 + 8 * g + r8] << 16);
            float s = 0.0f;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                S[g][e] = fmaf(vv, kv[e], S[g][e] * al);
                s = fmaf(S[g][e], qv[e], s);
            }
#pragma unroll
            for (int x = 4; x > 0; x >>= 1)
                s += __shfl_xor(s, x);
            o[g] = s * a.scale;
        }
        const float mine = q8 == 0 ? o[0] : q8 == 1 ? o[1] : q8 == 2 ? o[2] : o[3];
        if (q8 < 4)
            static_cast<uint16_t *>(ro.out)[(tok * a.H + h) * kD + v0 + 8 * q8 + r8] = to_bf16(mine);
    }
    if (!ro.fin)
        return;
#pragma unroll
    for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            const size_t at = mat + (size_t)(v0 + 8 * g + r8) * kD + (8 * p + q8) * kPer;
            if constexpr (kF32) {
                *reinterpret_cast<f32x4 *>(static_cast<float *>(ro.fin) + at) =
                    f32x4{S[g][p * 4], S[g][p * 4 + 1], S[g][p * 4 + 2], S[g][p * 4 + 3]};
            } else {
                u32x4 x;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[e] = pack2(S[g][p * 8 + 2 * e], S[g][p * 8 + 2 * e + 1]);
                *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(ro.fin) + at) = x;
            }
        }
}

}  // namespace

hipError_t lin_launch_check(const int64_t *cu, int64_t N, int64_t T, int32_t *status, hipStream_t s)
{
    hipLaunchKernelGGL(lin_check_kernel, dim3(1), dim3(1024), 0, s, cu, N, T, status);
    return hipGetLastError();
}

hipError_t lin_launch_walk(const LinArgs &a0, int n_roles, const int *lead, int n_lead, hipStream_t s)
{
    LinArgs a = a0;
    const int64_t total = a.rows * a.P * a.H;
    const unsigned grid = (unsigned)(8 * cdiv(total, 8));
    if (a.P > 1) {
        const int l0 = lead[0], l1 = lead[n_lead - 1];
        hipLaunchKernelGGL(lin_states_kernel, dim3(grid, n_lead), dim3(256), 0, s, a, l0, l1);
        hipLaunchKernelGGL(lin_scan_kernel, dim3((unsigned)(kScanParts * a.rows * a.H), n_lead), dim3(256), 0, s, a,
                           l0, l1);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    bool dots = false;
    for (int i = 0; i < n_roles; ++i)
        dots = dots || a.role[i].dots;
    a.turns = total * n_roles <= kLinSlots;
    if (dots)
        hipLaunchKernelGGL(lin_walk_kernel<true>, dim3(grid, n_roles), dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL(lin_walk_kernel<false>, dim3(grid, n_roles), dim3(256), 0, s, a);
    if (a.role[0].defer)
        hipLaunchKernelGGL(lin_final_kernel, dim3((unsigned)total), dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t lin_launch_fold(const float *xq, const float *xk, uint16_t *yq, uint16_t *yk, int64_t rows, int64_t Hk, int64_t G,
                           const int32_t *status, hipStream_t s)
{
    const int64_t n = rows * Hk * (kD / 4);
    const int64_t blocks = cdiv(n, 256) < 4096 ? cdiv(n, 256) : 4096;
    hipLaunchKernelGGL(lin_fold_kernel, dim3((unsigned)blocks, 2), dim3(256), 0, s, xq, xk, yq, yk, rows, Hk, G, status);
    return hipGetLastError();
}

hipError_t lin_launch_grad_tail(const LinArgs &a, const LinBwdExtra &e, hipStream_t s)
{
    if (e.dq_h && a.T > 0) {
        const hipError_t err = lin_launch_fold(e.dq_h, e.dk_h, e.dq, e.dk, a.rows * a.T, e.Hk, a.H / e.Hk,
                                               a.cu ? a.status : nullptr, s);
        if (err != hipSuccess)
            return err;
    }
    if (e.ddecay) {
        hipLaunchKernelGGL(lin_ddecay_kernel, dim3((unsigned)(a.rows * a.P * a.H)), dim3(kGradThreads), 0, s, a, e.ddecay,
                           e.part);
        if (!a.per_token)
            hipLaunchKernelGGL(lin_ddecay_sum_kernel, dim3((unsigned)a.H), dim3(64), 0, s, a, e.part, e.ddecay);
    }
    return hipGetLastError();
}

hipError_t lin_launch_recurrent(const LinArgs &a, hipStream_t s)
{
    const int64_t units = a.N * a.H * 4;
    const LinRole &ro = a.role[0];
    const bool f32 = (ro.init ? ro.init_dt : ro.fin_dt) != kBf16;
    const int threads = units < 4096 ? 64 : 256;
    const unsigned grid = (unsigned)cdiv(units, threads / 64);
    if (f32)
        hipLaunchKernelGGL(lin_recurrent_kernel<true>, dim3(grid), dim3(threads), 0, s, a);
    else
        hipLaunchKernelGGL(lin_recurrent_kernel<false>, dim3(grid), dim3(threads), 0, s, a);
    return hipGetLastError();
}

}  // namespace kda
