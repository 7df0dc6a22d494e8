// rope_api.cpp -- host side of the q/k normalisation and position rotation (kda_qk_rope* in
// include/kda.h): argument checks and launches.  The checks are plain host code that touches
// no HIP API.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <hip/hip_runtime.h>

#include "kda.h"
#include "rope_internal.h"

namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int64_t kMaxElems = (int64_t)1 << 46;

struct Span {  // a strided view and the bytes it touches
    uintptr_t lo, hi;
    int64_t sb, st, sh;  // elements
    int64_t B, T, heads, D;
    int size;
};

bool plain_overlap(uintptr_t lo, uintptr_t hi, const Span &s)
{
    return lo < s.hi && s.lo < hi && lo != hi && s.lo != s.hi;
}

// What a view covers of a period of p elements: dimensions whose stride is a multiple of p repeat it.
int64_t width(const Span &s, int64_t p)
{
    const int64_t n[3] = {s.B, s.T, s.heads}, st[3] = {s.sb, s.st, s.sh};
    int64_t w = s.D;
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && st[i] % p)
            w += (n[i] - 1) * st[i];
    return w;
}
// True when two views certainly share no byte: disjoint ranges, or disjoint places in a common period (the rows of one buffer
// with q's heads beside k's, or its batch rows with q's heads before k's), tried for every stride.
bool disjoint(const Span &x, const Span &y)
{
    if (!(x.lo < y.hi && y.lo < x.hi) || x.lo == x.hi || y.lo == y.hi)
        return true;
    const int64_t n[6] = {x.B, x.T, x.heads, y.B, y.T, y.heads}, st[6] = {x.sb, x.st, x.sh, y.sb, y.st, y.sh};
    for (int i = 0; i < 6; ++i) {
        const int64_t p = st[i];
        if (n[i] < 2 || p <= 0)
            continue;
        const int64_t period = p * x.size, wx = width(x, p) * x.size, wy = width(y, p) * y.size;
        const int64_t up = (int64_t)((y.lo - x.lo) % (uintptr_t)period), down = (int64_t)((x.lo - y.lo) % (uintptr_t)period);
        const int64_t at = y.lo >= x.lo ? up : (down ? period - down : 0);  // y's place in a period that starts with x
        if (at >= wx && at + wy <= period)
            return true;
    }
    return false;
}
bool same_view(const Span &x, const Span &y)
{
    return x.lo == y.lo && (x.B == 1 || x.sb == y.sb) && (x.T == 1 || x.st == y.st) && (x.heads == 1 || x.sh == y.sh);
}
// A view that is written must not hit itself: from the smallest stride on, each steps over all that the smaller ones cover.
bool injective(const Span &s)
{
    int64_t n[3] = {s.B, s.T, s.heads}, st[3] = {s.sb, s.st, s.sh}, covered = s.D;
    for (int done = 0; done < 3; ++done) {
        int least = done;
        for (int i = done + 1; i < 3; ++i)
            if (st[i] < st[least])
                least = i;
        const int64_t many = n[least], step = st[least];
        n[least] = n[done];
        st[least] = st[done];
        if (many < 2)
            continue;
        if (step < covered)
            return false;
        covered += (many - 1) * step;
    }
    return true;
}

kda_status set_view(const void *p, const int64_t *st, int64_t B, int64_t T, int64_t heads, int64_t D, int size,
                    kda::RopeView *v, Span *s)
{
    v->p = static_cast<unsigned char *>(const_cast<void *>(p));
    v->sb = st ? st[0] : T * heads * D;
    v->st = st ? st[1] : heads * D;
    v->sh = st ? st[2] : D;
    const int64_t unit = 16 / size;
    if (v->sb < 0 || v->st < 0 || v->sh < 0 || v->sb % unit || v->st % unit || v->sh % unit || v->sb > kMaxElems ||
        v->st > kMaxElems || v->sh > kMaxElems || T > kMaxElems / (v->st + 1) || B > kMaxElems / (v->sb + 1) ||
        heads > kMaxElems / (v->sh + 1))
        return KDA_ERR_STRIDE;
    if (!aligned(p, 16))
        return KDA_ERR_ALIGN;
    s->lo = reinterpret_cast<uintptr_t>(p);
    s->hi = T > 0 ? s->lo + (size_t)((B - 1) * v->sb + (T - 1) * v->st + (heads - 1) * v->sh + D) * (size_t)size : s->lo;
    s->sb = v->sb;
    s->st = v->st;
    s->sh = v->sh;
    s->B = B;
    s->T = T;
    s->heads = heads;
    s->D = D;
    s->size = size;
    return KDA_OK;
}

kda_status check_shape(int64_t B, int64_t T, int64_t Hq, int64_t Hk, int64_t D, int64_t R)
{
    if (B < 1 || T < 0 || Hq < 1 || Hk < 1 || Hq > 4096 || Hk > 4096 ||
        T > (((int64_t)1 << 30) - 64) / B)  // a launch holds less than 2^32 threads: 256 for up to 64 tokens
        return KDA_ERR_SHAPE;
    if (D < 16 || D > kda::kRopeMaxD || D % 16 || R < 0 || R > D || R % 16)
        return KDA_ERR_ROTARY;
    return KDA_OK;
}

// What both directions check; `views` are q, k, then their outputs (forward), or the outputs' gradients
// and the inputs' gradients (backward).
kda_status common(const void *const *p, int n_views, const int64_t *strides, const float *wq, const float *wk,
                  const float *inv_freq, const int64_t *positions, int64_t B, int64_t T, int64_t Hq, int64_t Hk,
                  int64_t D, int64_t R, int dtype, int norm, float eps, int interleaved, float factor,
                  kda::RopeArgs *a, Span *span)
{
    kda_status st = check_shape(B, T, Hq, Hk, D, R);
    if (st != KDA_OK)
        return st;
    if (dtype != KDA_DTYPE_BF16 && dtype != KDA_DTYPE_FP32 && dtype != KDA_DTYPE_FP16)
        return KDA_ERR_DTYPE;
    if (norm < KDA_NORM_NONE || norm > KDA_NORM_L2 || (interleaved != 0 && interleaved != 1))
        return KDA_ERR_FLAGS;
    if (!(eps >= 0.0f) || !isfinite(eps) || !isfinite(factor))
        return KDA_ERR_SCALE;
    if (R > 0 && !inv_freq)
        return KDA_ERR_NULL;
    memset(a, 0, sizeof(*a));
    const int size = dtype == KDA_DTYPE_FP32 ? 4 : 2;
    kda::RopeView *to[] = {&a->x[0], &a->x[1], n_views == 4 ? &a->y[0] : &a->dy[0],
                           n_views == 4 ? &a->y[1] : &a->dy[1], &a->y[0], &a->y[1]};
    for (int i = 0; i < n_views; ++i) {
        if (T > 0 && !p[i])
            return KDA_ERR_NULL;
        if ((st = set_view(p[i], strides ? strides + 3 * i : nullptr, B, T, i % 2 ? Hk : Hq, D, size, to[i],
                           &span[i])) != KDA_OK)
            return st;
    }
    if (!aligned(wq, 4) || !aligned(wk, 4) || !aligned(inv_freq, 4) || !aligned(positions, 8))
        return KDA_ERR_ALIGN;
    // the two tensors written (the last two views): clear of each other, of themselves, and of every input but
    // the one they may replace in place, element for element
    const Span &oq = span[n_views - 2], &ok = span[n_views - 1];
    if (T > 0) {
        if (!injective(oq) || !injective(ok) || !disjoint(oq, ok))
            return KDA_ERR_ALIAS;
        for (int i = 0; i < n_views - 2; ++i) {
            if (!disjoint(oq, span[i]) && !(i % 2 == 0 && same_view(oq, span[i])))
                return KDA_ERR_ALIAS;
            if (!disjoint(ok, span[i]) && !(i % 2 == 1 && same_view(ok, span[i])))
                return KDA_ERR_ALIAS;
        }
    }
    const struct {
        const void *p;
        size_t bytes;
    } small[] = {{wq, (size_t)D * 4}, {wk, (size_t)D * 4}, {inv_freq, (size_t)R * 2}, {positions, (size_t)(B * T) * 8}};
    for (const auto &x : small) {
        const uintptr_t lo = reinterpret_cast<uintptr_t>(x.p);
        if (x.p && (plain_overlap(lo, lo + x.bytes, oq) || plain_overlap(lo, lo + x.bytes, ok)))
            return KDA_ERR_ALIAS;
    }
    a->w[0] = wq;
    a->w[1] = wk;
    a->inv_freq = inv_freq;
    a->positions = positions;
    a->B = B;
    a->T = T;
    a->heads[0] = (int)Hq;
    a->heads[1] = (int)Hk;
    a->D = (int)D;
    a->R = (int)R;
    a->dtype = dtype;
    a->norm = norm;
    a->interleaved = interleaved;
    a->eps = eps;
    a->factor = factor;
    return KDA_OK;
}

}  // namespace

extern "C" {

kda_status kda_qk_rope(const void *q, const void *k, void *q_out, void *k_out, const float *q_weight,
                       const float *k_weight, const float *inv_freq, const int64_t *positions, int64_t B, int64_t T,
                       int64_t Hq, int64_t Hk, int64_t D, int64_t rotary_dim, kda_dtype dtype, kda_norm norm,
                       float eps, int interleaved, float attention_factor, const int64_t *strides_host, void *stream)
{
    const void *p[] = {q, k, q_out, k_out};
    kda::RopeArgs a;
    Span span[4];
    const kda_status st = common(p, 4, strides_host, q_weight, k_weight, inv_freq, positions, B, T, Hq, Hk, D,
                                 rotary_dim, (int)dtype, (int)norm, eps, interleaved, attention_factor, &a, span);
    if (st != KDA_OK)
        return st;
    return kda::rope_launch(a, static_cast<hipStream_t>(stream)) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

size_t kda_qk_rope_bwd_workspace_size(int64_t B, int64_t T, int64_t Hq, int64_t Hk, int64_t D)
{
    if (check_shape(B, T, Hq, Hk, D, 0) != KDA_OK)
        return 0;
    return (size_t)kda::kRopeGroups * (size_t)D * sizeof(float);
}

kda_status kda_qk_rope_bwd(const void *q, const void *k, const void *dq_out, const void *dk_out, void *dq, void *dk,
                           const float *q_weight, const float *k_weight, float *dq_weight, float *dk_weight,
                           const float *inv_freq, const int64_t *positions, int64_t B, int64_t T, int64_t Hq,
                           int64_t Hk, int64_t D, int64_t rotary_dim, kda_dtype dtype, kda_norm norm, float eps,
                           int interleaved, float attention_factor, const int64_t *strides_host, void *workspace,
                           size_t workspace_bytes, void *stream)
{
    const void *p[] = {q, k, dq_out, dk_out, dq, dk};
    kda::RopeArgs a;
    Span span[6];
    const kda_status st = common(p, 6, strides_host, q_weight, k_weight, inv_freq, positions, B, T, Hq, Hk, D,
                                 rotary_dim, (int)dtype, (int)norm, eps, interleaved, attention_factor, &a, span);
    if (st != KDA_OK)
        return st;
    if ((dq_weight && !q_weight) || (dk_weight && !k_weight))
        return KDA_ERR_NULL;
    if (!aligned(dq_weight, 4) || !aligned(dk_weight, 4) || !aligned(workspace, 256))
        return KDA_ERR_ALIGN;
    const bool sums = dq_weight || dk_weight;
    const size_t need = kda_qk_rope_bwd_workspace_size(B, T, Hq, Hk, D);
    const struct {
        const void *p;
        size_t bytes;
    } out[] = {{dq_weight, (size_t)D * 4}, {dk_weight, (size_t)D * 4}, {sums ? workspace : nullptr, need}},
      in[] = {{q_weight, (size_t)D * 4}, {k_weight, (size_t)D * 4}, {inv_freq, (size_t)rotary_dim * 2},
              {positions, (size_t)(B * T) * 8}};
    for (int i = 0; i < 3; ++i) {
        const uintptr_t lo = reinterpret_cast<uintptr_t>(out[i].p), hi = lo + (out[i].p ? out[i].bytes : 0);
        for (const Span &s : span)
            if (plain_overlap(lo, hi, s))
                return KDA_ERR_ALIAS;
        auto hits = [&](const void *p2, size_t bytes) {
            const uintptr_t l2 = reinterpret_cast<uintptr_t>(p2), h2 = l2 + (p2 ? bytes : 0);
            return lo < h2 && l2 < hi && lo != hi && l2 != h2;
        };
        for (const auto &x : in)
            if (hits(x.p, x.bytes))
                return KDA_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (hits(out[j].p, out[j].bytes))
                return KDA_ERR_ALIAS;
    }
    if (sums && (!workspace || workspace_bytes < need))
        return KDA_ERR_WORKSPACE;
    a.part = static_cast<float *>(workspace);
    a.dw[0] = dq_weight;
    a.dw[1] = dk_weight;
    return kda::rope_launch_bwd(a, static_cast<hipStream_t>(stream)) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

}  // extern "C"
