// host_checks.h -- argument checks that the host sides of the operators (*_api.cpp) share.  Plain host code that touches no HIP API.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "kda.h"
#include "kda_internal.h"

namespace kda {

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct Range {
    uintptr_t lo, hi;  // [lo, hi)
};
inline Range range_of(const void *p, size_t bytes)
{
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Range{lo, p ? lo + bytes : lo};
}
inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.lo != a.hi && b.lo != b.hi; }

constexpr int64_t kMaxTokenStride = (int64_t)1 << 24;  // elements: 64 rows stay below 2^31 bytes
constexpr int64_t kMaxElems = (int64_t)1 << 46;

// Operators with one decay per head: Hk q/k heads shared by H value heads, a state [128][128] for each sequence and head
struct HeadSizes {
    int64_t B, T, Hk, H, N, n_seq;
    bool varlen;
};

// B, T, Hk, H, N and the sizes that follow from them; launches have limits of their own
inline kda_status check_head_sizes(int64_t B, int64_t T, int64_t Hk, int64_t H, int64_t N, bool varlen, HeadSizes *z)
{
    if (B < 1 || T < 0 || H < 1)
        return KDA_ERR_SHAPE;
    if (Hk < 1 || H % Hk != 0)
        return KDA_ERR_HEADS;
    if (varlen ? (B != 1 || N < 1) : (N != 0 && N != B))
        return KDA_ERR_SHAPE;
    if (H > ((int64_t)1 << 16) || T >= ((int64_t)1 << 35) || T > ((int64_t)1 << 40) / B ||
        B * T > kMaxElems / (H * kD))
        return KDA_ERR_SHAPE;
    *z = HeadSizes{B, T, Hk, H, N, varlen ? N : B, varlen};
    return KDA_OK;
}

inline bool dtype_ok(kda_state_dtype d) { return d == KDA_STATE_NONE || d == KDA_STATE_BF16 || d == KDA_STATE_FP32; }

inline size_t state_bytes(kda_state_dtype d) { return (size_t)kD * kD * (d == KDA_STATE_BF16 ? 2 : 4); }

// One strided input [B, T, heads, 128]; strides in elements (batch, token, head), NULL = contiguous.
template <typename Tensor>
inline kda_status set_tensor(const void *p, const int64_t *st, const HeadSizes &z, int64_t heads, Tensor *t, Range *r)
{
    t->p = static_cast<const uint16_t *>(p);
    t->share = z.H / heads;
    t->sb = st ? st[0] : z.T * heads * kD;
    t->st = st ? st[1] : heads * kD;
    t->sh = st ? st[2] : kD;
    if (t->sb < 0 || t->st < 0 || t->sh < 0 || t->sb % 8 || t->st % 8 || t->sh % 8 || t->st > kMaxTokenStride ||
        t->sb > kMaxElems || t->sh > kMaxElems)
        return KDA_ERR_STRIDE;
    if (z.T == 1)
        t->st = kD;  // never a step, but the kernels take a row's end from it
    if (!aligned(p, 16))
        return KDA_ERR_ALIGN;
    if (z.T > kMaxElems / (t->st + 1) || (z.T > 1 && t->st < kD))  // tokens' rows do not overlap
        return KDA_ERR_STRIDE;
    const size_t last = (size_t)(z.B - 1) * (size_t)t->sb + (size_t)(z.T > 0 ? z.T - 1 : 0) * (size_t)t->st +
                        (size_t)(heads - 1) * (size_t)t->sh + kD;
    *r = range_of(p, z.T > 0 ? last * 2 : 0);
    return KDA_OK;
}

inline kda_status check_cu(const int64_t *cu, const int64_t *host, const HeadSizes &z)
{
    if (!cu || !host)
        return KDA_OK;
    if (host[0] != 0 || host[z.N] != z.T)
        return KDA_ERR_CU_SEQLENS;
    for (int64_t i = 0; i < z.N; ++i)
        if (host[i + 1] < host[i])
            return KDA_ERR_CU_SEQLENS;
    return KDA_OK;
}

}  // namespace kda
