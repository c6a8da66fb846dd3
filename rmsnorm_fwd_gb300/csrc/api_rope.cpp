// api_rope.cpp -- the C ABI of the head operators with a position rotation
// and of the gradients: argument checks and launches.
#include <algorithm>
#include <array>
#include <climits>
#include <cmath>
#include <cstdint>

#include "rope_args.h"
#include "strides.h"

using namespace rmsnorm;

namespace {

constexpr int64_t kMostHeads = 1 << 20;
constexpr int64_t kMostElements = INT64_MAX / 16; // offsets in bytes stay in 63 bits

int64_t elem_size(int dtype) { return dtype == RMSNORM_F32 ? 4 : 2; }
bool known_dtype(int dtype)
{
    return dtype == RMSNORM_F32 || dtype == RMSNORM_BF16 || dtype == RMSNORM_F16;
}
uintptr_t addr(const void *p) { return reinterpret_cast<uintptr_t>(p); }

// a * b + c for non-negative values, false beyond kMostElements.
bool mul_add(int64_t a, int64_t b, int64_t c, int64_t *out)
{
    if (a != 0 && b > (kMostElements - c) / a)
        return false;
    *out = a * b + c;
    return true;
}

// A tensor's heads with the default strides filled in.
struct Heads {
    uintptr_t p = 0;
    int64_t ts = 0, hs = 0;       // elements
    int64_t tokens = 0, heads = 0, dim = 0, es = 0;
    int64_t extent = 0;           // bytes from p that the heads span
    HeadsView view() const { return {reinterpret_cast<char *>(p), ts, hs}; }
    bool same(const Heads &o) const { return p == o.p && ts == o.ts && hs == o.hs; }
};

// Fills `out`; false when a pointer is missing, a stride is negative or too
// large, or two heads of the tensor share an element.
bool make_heads(const rmsnorm_heads_t *t, int64_t tokens, int64_t heads, int64_t dim, int64_t es,
                Heads *out)
{
    Heads v;
    v.tokens = tokens;
    v.heads = heads;
    v.dim = dim;
    v.es = es;
    if (heads == 0 || tokens == 0) {
        *out = v;
        return true;
    }
    if (!t || !t->data || t->token_stride < 0 || t->head_stride < 0)
        return false;
    v.p = addr(t->data);
    v.hs = t->head_stride ? t->head_stride : dim;
    if (v.hs > kMostElements / heads)
        return false;
    v.ts = t->token_stride ? t->token_stride : heads * v.hs;
    // A single token's or head's stride is never taken; one value for it
    // keeps layouts comparable.
    if (heads == 1)
        v.hs = dim;
    if (tokens == 1)
        v.ts = heads * v.hs;
    int64_t last = 0;
    if (!mul_add(tokens - 1, v.ts, dim, &last) || !mul_add(heads - 1, v.hs, last, &last))
        return false;
    const bool token_major = v.hs >= dim && v.ts >= (heads - 1) * v.hs + dim;
    const bool head_major = v.ts >= dim && (heads == 1 || v.hs >= (tokens - 1) * v.ts + dim);
    if (!token_major && !head_major)
        return false;
    v.extent = last * es;
    *out = v;
    return true;
}

// Whether two tensors' heads can share a byte.  Exact where both have the
// same strides and either contiguous heads or evenly spaced ones; layouts
// that interleave otherwise count as overlapping.
bool heads_overlap(const Heads &a, const Heads &b)
{
    if (!a.extent || !b.extent || !bytes_overlap(a.p, a.extent, b.p, b.extent))
        return false;
    const int64_t es = a.es, da = a.dim * es;
    if (a.es != b.es || a.dim != b.dim)
        return true;
    if (a.hs == a.dim && b.hs == b.dim && a.ts >= a.heads * a.dim && b.ts >= b.heads * b.dim)
        return strided_overlap(a.p, a.ts * es, a.heads * da, b.p, b.ts * es, b.heads * da,
                               a.tokens);
    if (a.ts == a.heads * a.hs && b.ts == b.heads * b.hs && a.heads == b.heads) // head by head
        return strided_overlap(a.p, a.hs * es, da, b.p, b.hs * es, da, a.tokens * a.heads);
    return true;
}

// Whether the interval [w, w + bytes) can meet a tensor's heads.
bool interval_overlaps(const Heads &a, uintptr_t w, int64_t bytes)
{
    if (!a.extent || !w || bytes <= 0 || !bytes_overlap(a.p, a.extent, w, bytes))
        return false;
    const int64_t es = a.es;
    if (a.hs == a.dim && a.ts >= a.heads * a.dim)
        return interval_hits_strided(a.p, a.ts * es, a.heads * a.dim * es, a.tokens, w, bytes);
    if (a.ts == a.heads * a.hs)
        return interval_hits_strided(a.p, a.hs * es, a.dim * es, a.tokens * a.heads, w, bytes);
    return true;
}

// Sizes and scalars that the head operators share.
int check_sizes(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t head_dim, float bias,
                float eps, int dtype, const rmsnorm_rope_t *rope)
{
    if (!known_dtype(dtype))
        return RMSNORM_ERR_UNSUPPORTED_DTYPE;
    if (tokens < 0 || q_heads < 0 || k_heads < 0 || q_heads > kMostHeads ||
        k_heads > kMostHeads || head_dim < 1 || head_dim > kMaxHeadDim || !(eps >= 0.f) ||
        !std::isfinite(eps) || !std::isfinite(bias) || !rope)
        return RMSNORM_ERR_INVALID_ARG;
    if (tokens > kMostElements / ((q_heads + 2 * k_heads + 1) * head_dim))
        return RMSNORM_ERR_INVALID_ARG;
    if (rope->rotary_dim < 0 || rope->rotary_dim > head_dim || rope->rotary_dim % 2 != 0 ||
        (rope->interleaved != 0 && rope->interleaved != 1))
        return RMSNORM_ERR_INVALID_ARG;
    if (rope->rotary_dim > 0) {
        if (rope->max_position < 0 ||
            rope->max_position > kMostElements / rope->rotary_dim)
            return RMSNORM_ERR_INVALID_ARG;
        if (tokens > 0 && (!rope->positions || (rope->max_position > 0 && !rope->cos_sin)))
            return RMSNORM_ERR_INVALID_ARG;
        if (addr(rope->positions) % 8 != 0 || addr(rope->cos_sin) % 4 != 0)
            return RMSNORM_ERR_MISALIGNED;
    }
    return RMSNORM_OK;
}

RopeTable table_of(const rmsnorm_rope_t &r)
{
    return {r.cos_sin, r.positions, r.max_position, r.rotary_dim, r.interleaved};
}

// Whether a written tensor meets any of the read-only arrays of a call.
bool hits_inputs(const Heads &out, const rmsnorm_rope_t &r, const void *qw, const void *kw)
{
    if (!out.extent)
        return false;
    const int64_t wb = out.dim * out.es;
    if (interval_overlaps(out, addr(qw), wb) || interval_overlaps(out, addr(kw), wb))
        return true;
    return r.rotary_dim > 0 &&
           (interval_overlaps(out, addr(r.positions), out.tokens * 8) ||
            interval_overlaps(out, addr(r.cos_sin), r.max_position * r.rotary_dim * 4));
}

// Whether a written tensor may overlap the tensor it is formed from.
bool bad_alias(const Heads &out, const Heads &in)
{
    return !(out.p == in.p && out.same(in)) && heads_overlap(out, in);
}

LaunchArgs launch_base(const CallContext &ctx, void *stream)
{
    LaunchArgs b{};
    b.stream = static_cast<cudaStream_t>(stream);
    b.pdl = ctx.pdl;
    b.status = ctx.status;
    return b;
}

struct Dim {
    int64_t n, s; // size and stride, elements
};
using Dims = std::array<Dim, 3>;
void sort_dims(Dims &d)
{
    std::sort(d.begin(), d.end(), [](const Dim &a, const Dim &b) { return a.s < b.s; });
}

// Whether two arrays of the same strides, `d` bytes apart, lie in each
// other's gaps: below some dimension the other array starts behind what the
// inner dimensions span, and every dimension from there on steps over both.
bool fits_in_gaps(int64_t d, int64_t es, int64_t dim, Dims dims)
{
    sort_dims(dims);
    int64_t inner = dim * es;
    for (int i = 0; i <= 3; ++i) {
        int64_t both = d + inner;
        bool ok = d >= inner;
        for (int j = i; ok && j < 3; ++j) {
            if (dims[j].n <= 1)
                continue;
            ok = dims[j].s * es >= both;
            both += (dims[j].n - 1) * dims[j].s * es;
        }
        if (ok)
            return true;
        if (i < 3 && dims[i].n > 1)
            inner += (dims[i].n - 1) * dims[i].s * es;
    }
    return false;
}

// The cache's strides with the defaults filled in; false when they are
// negative, too large, or let two of its heads share an element.
bool cache_strides(const rmsnorm_paged_cache_t &c, int64_t heads, int64_t dim, int64_t *ps,
                   int64_t *ss, int64_t *hs, int64_t *elements)
{
    if (c.pages < 0 || c.page_size < 1 || c.page_stride < 0 || c.slot_stride < 0 ||
        c.head_stride < 0)
        return false;
    int64_t slots = 0;
    if (!mul_add(c.pages, c.page_size, 0, &slots))
        return false;
    *ps = c.page_stride;
    *ss = c.slot_stride;
    *hs = c.head_stride;
    if (!*ps && !*ss && !*hs) {
        *hs = dim;
        *ss = heads * dim;
        if (!mul_add(c.page_size, *ss, 0, ps))
            return false;
    }
    Dims d = {{{c.pages, *ps}, {c.page_size, *ss}, {heads, *hs}}};
    sort_dims(d);
    int64_t span = dim; // each dimension must step over what the smaller ones span
    for (const Dim &e : d) {
        if (e.n <= 1)
            continue;
        if (e.s < span || !mul_add(e.n - 1, e.s, span, &span))
            return false;
    }
    *elements = c.pages ? span : 0;
    return true;
}

} // namespace

extern "C" {

int rmsnorm_qk_norm_rope(const rmsnorm_heads_t *q, const rmsnorm_heads_t *k,
                         const rmsnorm_heads_t *q_out, const rmsnorm_heads_t *k_out,
                         const void *q_weight, const void *k_weight, const rmsnorm_rope_t *rope,
                         int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t head_dim,
                         float weight_bias, float eps, int dtype, void *stream)
{
    int rc = check_sizes(tokens, q_heads, k_heads, head_dim, weight_bias, eps, dtype, rope);
    if (rc != RMSNORM_OK)
        return rc;
    const int64_t es = elem_size(dtype);
    Heads qi, ki, qo, ko;
    if ((q_heads > 0 && !q_weight) || (k_heads > 0 && !k_weight) ||
        !make_heads(q, tokens, q_heads, head_dim, es, &qi) ||
        !make_heads(k, tokens, k_heads, head_dim, es, &ki) ||
        !make_heads(q_out ? q_out : q, tokens, q_heads, head_dim, es, &qo) ||
        !make_heads(k_out ? k_out : k, tokens, k_heads, head_dim, es, &ko))
        return RMSNORM_ERR_INVALID_ARG;
    for (const Heads *h : {&qi, &ki, &qo, &ko})
        if (h->p % es != 0)
            return RMSNORM_ERR_MISALIGNED;
    if (addr(q_weight) % es != 0 || addr(k_weight) % es != 0)
        return RMSNORM_ERR_MISALIGNED;
    if (bad_alias(qo, qi) || bad_alias(ko, ki) || heads_overlap(qo, ko) || heads_overlap(qo, ki) ||
        heads_overlap(ko, qi) || hits_inputs(qo, *rope, q_weight, k_weight) ||
        hits_inputs(ko, *rope, q_weight, k_weight))
        return RMSNORM_ERR_ALIASING;
    CallContext ctx;
    rc = call_context(&ctx);
    if (rc != RMSNORM_OK)
        return rc;
    if (tokens == 0 || q_heads + k_heads == 0)
        return RMSNORM_OK;
    RopeArgs a{};
    a.base = launch_base(ctx, stream);
    a.q = qi.view();
    a.k = ki.view();
    a.qo = qo.view();
    a.ko = ko.view();
    a.qw = q_weight;
    a.kw = k_weight;
    a.rope = table_of(*rope);
    a.tokens = tokens;
    a.q_heads = static_cast<int32_t>(q_heads);
    a.k_heads = static_cast<int32_t>(k_heads);
    a.head_dim = static_cast<int32_t>(head_dim);
    a.bias = weight_bias;
    a.eps = eps;
    a.sm_count = ctx.sm_count;
    return launch_rope(a, dtype) == cudaSuccess ? RMSNORM_OK : RMSNORM_ERR_CUDA;
}

int rmsnorm_qk_norm_rope_append(const rmsnorm_heads_t *q, const rmsnorm_heads_t *k,
                                const rmsnorm_heads_t *v, const rmsnorm_heads_t *q_out,
                                const void *q_weight, const void *k_weight,
                                const rmsnorm_rope_t *rope, const rmsnorm_paged_cache_t *cache,
                                const int64_t *slots, int64_t tokens, int64_t q_heads,
                                int64_t k_heads, int64_t head_dim, float weight_bias, float eps,
                                int dtype, void *stream)
{
    int rc = check_sizes(tokens, q_heads, k_heads, head_dim, weight_bias, eps, dtype, rope);
    if (rc != RMSNORM_OK)
        return rc;
    const int64_t es = elem_size(dtype);
    if (!cache || k_heads < 1 || (cache->e4m3 != 0 && cache->e4m3 != 1))
        return RMSNORM_ERR_INVALID_ARG;
    const bool norm = q_weight || k_weight;
    if (norm && (!k_weight || (q_heads > 0 && !q_weight)))
        return RMSNORM_ERR_INVALID_ARG;
    float k_inv = 1.f, v_inv = 1.f;
    if (cache->e4m3) {
        k_inv = 1.f / cache->k_scale;
        v_inv = 1.f / cache->v_scale;
        for (float s : {cache->k_scale, cache->v_scale, k_inv, v_inv})
            if (!(s > 0.f) || !std::isfinite(s))
                return RMSNORM_ERR_INVALID_ARG;
    }
    int64_t ps = 0, ss = 0, hs = 0, span = 0;
    Heads qi, ki, vi, qo;
    if (!cache_strides(*cache, k_heads, head_dim, &ps, &ss, &hs, &span) ||
        (span > 0 && (!cache->k || !cache->v)) || (tokens > 0 && !slots) ||
        !make_heads(q, tokens, q_heads, head_dim, es, &qi) ||
        !make_heads(k, tokens, k_heads, head_dim, es, &ki) ||
        !make_heads(v, tokens, k_heads, head_dim, es, &vi) ||
        !make_heads(q_out ? q_out : q, tokens, q_heads, head_dim, es, &qo))
        return RMSNORM_ERR_INVALID_ARG;
    const int64_t ces = cache->e4m3 ? 1 : es;
    for (const Heads *h : {&qi, &ki, &vi, &qo})
        if (h->p % es != 0)
            return RMSNORM_ERR_MISALIGNED;
    if (addr(q_weight) % es != 0 || addr(k_weight) % es != 0)
        return RMSNORM_ERR_MISALIGNED;
    if (addr(cache->k) % ces != 0 || addr(cache->v) % ces != 0 || addr(slots) % 8 != 0)
        return RMSNORM_ERR_MISALIGNED;
    if (bad_alias(qo, qi) || heads_overlap(qo, ki) || heads_overlap(qo, vi) ||
        hits_inputs(qo, *rope, q_weight, k_weight) ||
        interval_overlaps(qo, addr(slots), tokens * 8))
        return RMSNORM_ERR_ALIASING;
    // Each cache as a whole interval, between its strides' gaps too -- but for
    // the other cache, whose pages may lie in those gaps ([page, 2, ...]).
    const int64_t cbytes = span * ces, wb = head_dim * es;
    for (const void *c : {cache->k, cache->v}) {
        const uintptr_t cp = addr(c);
        if (!c || !cbytes || tokens == 0)
            continue;
        for (const Heads *h : {&qi, &ki, &vi, &qo})
            if (interval_overlaps(*h, cp, cbytes))
                return RMSNORM_ERR_ALIASING;
        if ((q_weight && bytes_overlap(cp, cbytes, addr(q_weight), wb)) ||
            (k_weight && bytes_overlap(cp, cbytes, addr(k_weight), wb)) ||
            bytes_overlap(cp, cbytes, addr(slots), tokens * 8) ||
            (rope->rotary_dim > 0 &&
             (bytes_overlap(cp, cbytes, addr(rope->positions), tokens * 8) ||
              bytes_overlap(cp, cbytes, addr(rope->cos_sin),
                            rope->max_position * rope->rotary_dim * 4))))
            return RMSNORM_ERR_ALIASING;
    }
    if (cbytes && bytes_overlap(addr(cache->k), cbytes, addr(cache->v), cbytes)) {
        // One cache in the other's gaps, both with the same strides, as
        // [pages, 2, ...] or [..., head_dim of k | head_dim of v] have it.
        const int64_t d = static_cast<int64_t>(std::max(addr(cache->k), addr(cache->v)) -
                                               std::min(addr(cache->k), addr(cache->v)));
        if (!fits_in_gaps(d, ces, head_dim,
                          {{{cache->pages, ps}, {cache->page_size, ss}, {k_heads, hs}}}))
            return RMSNORM_ERR_ALIASING;
    }
    CallContext ctx;
    rc = call_context(&ctx);
    if (rc != RMSNORM_OK)
        return rc;
    if (tokens == 0)
        return RMSNORM_OK;
    RopeArgs a{};
    a.base = launch_base(ctx, stream);
    a.q = qi.view();
    a.k = ki.view();
    a.v = vi.view();
    a.qo = qo.view();
    a.qw = q_weight;
    a.kw = k_weight;
    a.rope = table_of(*rope);
    a.tokens = tokens;
    a.q_heads = static_cast<int32_t>(q_heads);
    a.k_heads = static_cast<int32_t>(k_heads);
    a.head_dim = static_cast<int32_t>(head_dim);
    a.bias = weight_bias;
    a.eps = eps;
    a.slots = slots;
    a.kc = static_cast<char *>(cache->k);
    a.vc = static_cast<char *>(cache->v);
    a.num_slots = cache->pages * cache->page_size;
    a.page_size = cache->page_size;
    a.page_stride = ps;
    a.slot_stride = ss;
    a.cache_hs = hs;
    a.e4m3 = cache->e4m3;
    a.k_inv = k_inv;
    a.v_inv = v_inv;
    a.sm_count = ctx.sm_count;
    return launch_rope(a, dtype) == cudaSuccess ? RMSNORM_OK : RMSNORM_ERR_CUDA;
}

int rmsnorm_qk_norm_rope_bwd_workspace(int64_t head_dim, int sm_count, size_t *bytes)
{
    if (!bytes || head_dim < 1 || head_dim > kMaxHeadDim || sm_count < 1 || sm_count > 4096)
        return RMSNORM_ERR_INVALID_ARG;
    *bytes = static_cast<size_t>(rope_bwd_max_blocks(sm_count)) * head_dim * sizeof(float);
    return RMSNORM_OK;
}

int rmsnorm_qk_norm_rope_bwd(const rmsnorm_heads_t *dq_out, const rmsnorm_heads_t *dk_out,
                             const rmsnorm_heads_t *q, const rmsnorm_heads_t *k,
                             const rmsnorm_heads_t *dq, const rmsnorm_heads_t *dk,
                             const void *q_weight, const void *k_weight, float *dq_weight,
                             float *dk_weight, const rmsnorm_rope_t *rope, void *workspace,
                             size_t workspace_bytes, int64_t tokens, int64_t q_heads,
                             int64_t k_heads, int64_t head_dim, float weight_bias, float eps,
                             int dtype, void *stream)
{
    int rc = check_sizes(tokens, q_heads, k_heads, head_dim, weight_bias, eps, dtype, rope);
    if (rc != RMSNORM_OK)
        return rc;
    const int64_t es = elem_size(dtype);
    const bool grads = dq_weight || dk_weight;
    Heads qy, ky, qi, ki, qd, kd;
    if ((q_heads > 0 && !q_weight) || (k_heads > 0 && !k_weight) ||
        (grads && (!dq_weight || !dk_weight)) ||
        !make_heads(dq_out, tokens, q_heads, head_dim, es, &qy) ||
        !make_heads(dk_out, tokens, k_heads, head_dim, es, &ky) ||
        !make_heads(q, tokens, q_heads, head_dim, es, &qi) ||
        !make_heads(k, tokens, k_heads, head_dim, es, &ki) ||
        !make_heads(dq, tokens, q_heads, head_dim, es, &qd) ||
        !make_heads(dk, tokens, k_heads, head_dim, es, &kd))
        return RMSNORM_ERR_INVALID_ARG;
    for (const Heads *h : {&qy, &ky, &qi, &ki, &qd, &kd})
        if (h->p % es != 0)
            return RMSNORM_ERR_MISALIGNED;
    if (addr(q_weight) % es != 0 || addr(k_weight) % es != 0)
        return RMSNORM_ERR_MISALIGNED;
    if (bad_alias(qd, qy) || bad_alias(qd, qi) || bad_alias(kd, ky) || bad_alias(kd, ki) ||
        heads_overlap(qd, kd) || heads_overlap(qd, ky) || heads_overlap(qd, ki) ||
        heads_overlap(kd, qy) || heads_overlap(kd, qi) ||
        hits_inputs(qd, *rope, q_weight, k_weight) || hits_inputs(kd, *rope, q_weight, k_weight))
        return RMSNORM_ERR_ALIASING;
    CallContext ctx;
    rc = call_context(&ctx);
    if (rc != RMSNORM_OK)
        return rc;
    if (grads) {
        size_t need = 0;
        rmsnorm_qk_norm_rope_bwd_workspace(head_dim, ctx.sm_count, &need);
        if (!workspace || workspace_bytes < need)
            return RMSNORM_ERR_INVALID_ARG;
        if (addr(workspace) % 16 != 0 || addr(dq_weight) % 4 != 0 || addr(dk_weight) % 4 != 0)
            return RMSNORM_ERR_MISALIGNED;
        // The fp32 results and the workspace are written: apart from
        // everything else, and from one another.
        const struct {
            uintptr_t p;
            int64_t n;
        } w[] = {{addr(workspace), static_cast<int64_t>(need)},
                 {addr(dq_weight), head_dim * 4},
                 {addr(dk_weight), head_dim * 4}};
        for (int i = 0; i < 3; ++i) {
            for (int j = i + 1; j < 3; ++j)
                if (bytes_overlap(w[i].p, w[i].n, w[j].p, w[j].n))
                    return RMSNORM_ERR_ALIASING;
            for (const Heads *h : {&qy, &ky, &qi, &ki, &qd, &kd})
                if (interval_overlaps(*h, w[i].p, w[i].n))
                    return RMSNORM_ERR_ALIASING;
            for (const void *x : {q_weight, k_weight})
                if (x && bytes_overlap(w[i].p, w[i].n, addr(x), head_dim * es))
                    return RMSNORM_ERR_ALIASING;
            if (rope->rotary_dim > 0 && tokens > 0 &&
                (bytes_overlap(w[i].p, w[i].n, addr(rope->positions), tokens * 8) ||
                 bytes_overlap(w[i].p, w[i].n, addr(rope->cos_sin),
                               rope->max_position * rope->rotary_dim * 4)))
                return RMSNORM_ERR_ALIASING;
        }
    }
    if (!grads && (tokens == 0 || q_heads + k_heads == 0))
        return RMSNORM_OK;
    RopeBwdArgs a{};
    a.base = launch_base(ctx, stream);
    a.qdy = qy.view();
    a.kdy = ky.view();
    a.q = qi.view();
    a.k = ki.view();
    a.dq = qd.view();
    a.dk = kd.view();
    a.qw = q_weight;
    a.kw = k_weight;
    a.dqw = dq_weight;
    a.dkw = dk_weight;
    a.part = grads ? static_cast<float *>(workspace) : nullptr;
    a.rope = table_of(*rope);
    a.tokens = tokens;
    a.q_heads = static_cast<int32_t>(q_heads);
    a.k_heads = static_cast<int32_t>(k_heads);
    a.head_dim = static_cast<int32_t>(head_dim);
    a.bias = weight_bias;
    a.eps = eps;
    a.sm_count = ctx.sm_count;
    return launch_rope_bwd(a, dtype) == cudaSuccess ? RMSNORM_OK : RMSNORM_ERR_CUDA;
}

int rmsnorm_bwd_workspace(int64_t rows, int64_t hidden, int dtype, int sm_count, size_t *bytes)
{
    if (!known_dtype(dtype))
        return RMSNORM_ERR_UNSUPPORTED_DTYPE;
    if (!bytes || rows < 0 || hidden < 1 || sm_count < 1 || sm_count > 4096 ||
        rows > kMostElements / hidden)
        return RMSNORM_ERR_INVALID_ARG;
    *bytes = rms_bwd_workspace(rows, hidden, dtype, sm_count);
    return RMSNORM_OK;
}

int rmsnorm_bwd(const void *dy, const void *x, const void *weight, void *dx, float *dweight,
                void *workspace, size_t workspace_bytes, int64_t rows, int64_t hidden,
                float weight_bias, float eps, int dtype, void *stream)
{
    if (!known_dtype(dtype))
        return RMSNORM_ERR_UNSUPPORTED_DTYPE;
    if (rows < 0 || hidden < 1 || !(eps >= 0.f) || !std::isfinite(eps) ||
        !std::isfinite(weight_bias) || !weight || rows > kMostElements / hidden)
        return RMSNORM_ERR_INVALID_ARG;
    if (rows > 0 && (!dy || !x || !dx))
        return RMSNORM_ERR_INVALID_ARG;
    const int64_t es = elem_size(dtype), bytes = rows * hidden * es, wb = hidden * es;
    if (addr(dy) % es || addr(x) % es || addr(dx) % es || addr(weight) % es || addr(dweight) % 4)
        return RMSNORM_ERR_MISALIGNED;
    if (rows > 0 && ((dx != dy && bytes_overlap(addr(dx), bytes, addr(dy), bytes)) ||
                     (dx != x && bytes_overlap(addr(dx), bytes, addr(x), bytes)) ||
                     bytes_overlap(addr(dx), bytes, addr(weight), wb)))
        return RMSNORM_ERR_ALIASING;
    CallContext ctx;
    const int rc = call_context(&ctx);
    if (rc != RMSNORM_OK)
        return rc;
    const size_t need = rms_bwd_workspace(rows, hidden, dtype, ctx.sm_count);
    if (rows > 0 && (!workspace || workspace_bytes < need))
        return RMSNORM_ERR_INVALID_ARG;
    if (rows > 0 && addr(workspace) % 16 != 0)
        return RMSNORM_ERR_MISALIGNED;
    const struct {
        const void *p;
        int64_t n;
    } written[] = {{rows > 0 ? workspace : nullptr, static_cast<int64_t>(need)},
                   {dweight, hidden * 4}};
    for (const auto &w : written) {
        if (!w.p)
            continue;
        for (const void *t : {dy, x, static_cast<const void *>(dx)})
            if (rows > 0 && bytes_overlap(addr(w.p), w.n, addr(t), bytes))
                return RMSNORM_ERR_ALIASING;
        if (bytes_overlap(addr(w.p), w.n, addr(weight), wb))
            return RMSNORM_ERR_ALIASING;
    }
    if (rows > 0 && dweight &&
        bytes_overlap(addr(workspace), static_cast<int64_t>(need), addr(dweight), hidden * 4))
        return RMSNORM_ERR_ALIASING;
    const LaunchArgs base = launch_base(ctx, stream);
    if (rows == 0) {
        if (!dweight)
            return RMSNORM_OK;
        return launch_colsum({nullptr, dweight, 0, hidden, hidden}, {}, base) == cudaSuccess
                   ? RMSNORM_OK
                   : RMSNORM_ERR_CUDA;
    }
    RmsBwdArgs a{};
    a.base = base;
    a.dy = dy;
    a.x = x;
    a.w = weight;
    a.dx = dx;
    a.dw = dweight;
    a.ws = workspace;
    a.rows = rows;
    a.hidden = hidden;
    a.bias = weight_bias;
    a.eps = eps;
    a.sm_count = ctx.sm_count;
    return launch_rms_bwd(a, dtype) == cudaSuccess ? RMSNORM_OK : RMSNORM_ERR_CUDA;
}

} // extern "C"
