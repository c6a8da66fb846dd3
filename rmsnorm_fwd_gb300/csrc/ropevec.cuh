// ropevec.cuh -- the vector body of the per-head QK norm with its rotation and
// paged-cache append; instantiated by rope_f32.cu, rope_bf16.cu, rope_f16.cu.
#pragma once

#include <algorithm>

#include "rope.cuh"

namespace rmsnorm {
namespace {

// N codes from a vector's first words, in one store.
template <int N, int VB> __device__ inline void st_e4m3(char *dst, const Vec<VB> &v)
{
    uint32_t w[(N + 3) / 4];
#pragma unroll
    for (int i = 0; i < (N + 3) / 4; ++i)
        w[i] = v.w[i];
    st_codes<N>(dst, w);
}

// Elements e .. e + C back in the element type or as E4M3 codes of value * inv
// (in word e / 4).
template <int DT, int VB, int C>
__device__ inline void put(Vec<VB> &v, int e, const float (&f)[C], bool code, float inv)
{
    if (code)
        v.w[e / 4] = e4m3x4(f[0] * inv, f[1] * inv, C == 4 ? f[C - 2] * inv : 0.f,
                            C == 4 ? f[C - 1] * inv : 0.f);
    else
        put<DT, VB, C>(v, e, f);
}

// How a call's heads are cut into warps: parts of per heads each, q's, then
// k's, then (appending) v's; a part lies within one tensor.
struct Parts {
    uint32_t q, k, all;
};

// Heads in vectors (rope.cuh): a warp takes U * (32 / TPR) heads of one
// tensor and token at once.  Only the heads' vectors wait in registers; the
// token's angles and the weights are loaded where they are used, once for the
// U heads of a lane:
//   y_a = x_a r (g_a cos) - x_b r (g_b sin),  y_b = x_b r (g_b cos) + x_a r (g_a sin)
//
// Memory bounds it once the warps on an SM have enough bytes on the way and
// few enough instructions between load and store.  Measured (16384 tokens of
// 32 + 8 bf16 heads of 128, 338 MB, floor 50.6 us at the copy bandwidth): the
// scalar body 326.8 us; this one 52.5 us (6.44 TB/s, 96 %).  On the way: one
// head a lane with its angles in registers 90 us (80 registers, half the
// warps); a warp within one tensor instead of choosing q or k lane by lane
// 84 -> 58 us; the pairing as a template 58 -> 55 us; four heads a lane instead of
// two 55 -> 53 us.  Slots that hold a warp's vectors in whole lines (slot_vectors)
// took 5003 tokens of 16 + 8 f16 heads of 256, 64 rotated as neighbours, from
// 28.0 to 22.7 us (floor 18.5).  Register caps: 64 for four heads (80: 3 %
// slower), 48 for two (64: 2 % slower, 40: 19 % slower).  Blocks of four warps (of
// eight, whose places wait for the slowest: 53.3 us; appending 67.0 for 65.1).
constexpr int kFwdWarps = 4; // of a block
//
// BY_TOKEN: each lane group takes a token of its own and U of its heads, for
// tensors of so few heads that a warp within one token would stand half empty.
template <int DT, int VB, int TPR, int NP, int U, bool APPEND, int MODE, bool BY_TOKEN>
__global__ void __launch_bounds__(kFwdWarps * 32, NP == 4 ? 2 : NP == 2 ? 4 : U == 2 ? 10 : 8)
rope_kernel(const __grid_constant__ RopeArgs a, Parts parts)
{
    using E = Elem<DT>;
    constexpr int N = kVpe<DT, VB>;
    constexpr int G = 32 / TPR;
    constexpr int C = N < 4 ? N : 4; // elements of each vector at a time
    pdl_begin();
    const int t = threadIdx.x % TPR;
    const int g = (threadIdx.x & 31) / TPR;
    const uint32_t item = __shfl_sync(0xFFFFFFFFu, blockIdx.x * kFwdWarps + (threadIdx.x >> 5), 0);
    constexpr int HS = BY_TOKEN ? 1 : G; // heads between a lane's
    const uint32_t unit = item / parts.all; // a token, or G tokens
    uint32_t part = item - unit * parts.all;
    const int64_t tok = BY_TOKEN ? static_cast<int64_t>(unit) * G + g : unit;
    if (static_cast<int64_t>(unit) * (BY_TOKEN ? G : 1) >= a.tokens)
        return; // the whole warp
    bool ok = !BY_TOKEN || tok < a.tokens; // this lane's token is there, and good
    const bool isq = part < parts.q;
    const bool isv = APPEND && part >= parts.q + parts.k;
    part -= isq ? 0 : isv ? parts.q + parts.k : parts.q;
    const int heads = isq ? a.q_heads : a.k_heads;
    const int h0 = static_cast<int>(part) * (U * HS); // this warp's first head
    const int own = BY_TOKEN ? 0 : g;                 // this lane's first, behind it
    const int slots = a.head_dim / (2 * N), half_v = a.rope.rd / (2 * N);
    constexpr bool inter = MODE == kInterleaved;

    const int64_t pos = a.rope.rd && ok ? a.rope.pos[tok] : 0;
    const int64_t slot = APPEND && ok ? a.slots[tok] : 0;

    const char *src = isq ? a.q.p : isv ? a.v.p : a.k.p;
    const int64_t sts = isq ? a.q.ts : isv ? a.v.ts : a.k.ts;
    const int64_t shs = isq ? a.q.hs : isv ? a.v.hs : a.k.hs;
    src += (tok * sts + (h0 + own) * shs) * E::kSize;
    int va[NP], vb[NP];
#pragma unroll
    for (int j = 0; j < NP; ++j)
        slot_vectors(t + j * TPR, slots, half_v, inter, va[j], vb[j]);
    Vec<VB> x[U][NP][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            if (ok && h0 + u * HS + own < heads && t + j * TPR < slots) {
                ld_head(x[u][j][0], src + va[j] * VB);
                ld_head(x[u][j][1], src + vb[j] * VB);
            } else {
                vzero(x[u][j][0]);
                vzero(x[u][j][1]);
            }
        }
        src += HS * shs * E::kSize;
    }
    {
        const bool pad = APPEND && slot < 0;
        const bool bad = (a.rope.rd && (pos < 0 || pos >= a.rope.max_pos)) ||
                         (APPEND && slot >= a.num_slots);
        if (ok && !pad && bad && t == 0)
            record_bad_index(a.base.status);
        ok = ok && !pad && !bad;
        if (BY_TOKEN ? !__any_sync(0xFFFFFFFFu, ok) : !ok)
            return; // the whole warp
    }
    const bool cached = APPEND && !isq;
    const bool code = cached && a.e4m3;
    const float inv = isv ? a.v_inv : a.k_inv;
    if (!isv) {
        const float *cs = a.rope.cs + pos * a.rope.rd;
        const RowCount n = row_count(a.head_dim);
        const char *w = static_cast<const char *>(isq ? a.qw : a.kw);
        const bool norm = !APPEND || w != nullptr;
        float r[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            r[u] = 1.f;
            if (!norm || h0 + u * HS >= heads)
                continue; // the whole warp
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < NP; ++j)
                sum = sumsq_mixed<DT, VB>(x[u][j][1], sumsq_mixed<DT, VB>(x[u][j][0], sum));
            sum = group_allreduce<TPR>(sum);
            r[u] = row_factor(sum, n, a.eps);
            if constexpr (kRangeGuard<DT>) {
                // Range guard (device_common.cuh), warp-uniform, from the
                // registers.
                const bool redo = sum_needs_rescale(sum, a.eps);
                if (__any_sync(0xFFFFFFFFu, redo)) {
                    const float k = rescale_k(sum);
                    float sk = 0.f;
#pragma unroll
                    for (int j = 0; j < NP; ++j)
                        sk = sumsq_k<DT, VB>(x[u][j][1], k, sumsq_k<DT, VB>(x[u][j][0], k, sk));
                    const Factor f = rescaled_factor(group_allreduce<TPR>(sk), k, n.n, a.eps);
                    if (redo) {
                        r[u] = f.r;
                        if (f.up) {
#pragma unroll
                            for (int j = 0; j < NP; ++j) {
                                scale_up<DT, VB>(x[u][j][0]);
                                scale_up<DT, VB>(x[u][j][1]);
                            }
                        }
                    }
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                reuse_barrier(x[u][j][0]);
                reuse_barrier(x[u][j][1]);
            }
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            const int p = t + j * TPR;
            if (p >= slots)
                continue;
            // Whether each vector is rotated, and its angles.
            const bool on_a = (!BY_TOKEN || ok) && (MODE == kHalvesFull ||
                                                    (inter ? va[j] * N < a.rope.rd : p < half_v));
            const bool on_b = inter ? (!BY_TOKEN || ok) && vb[j] * N < a.rope.rd : on_a;
            const float *ca = cs + (inter ? va[j] * (N / 2) : p * N), *cb = cs + vb[j] * (N / 2);
#pragma unroll
            for (int e = 0; e < N; e += C) {
                // What A r and B r are multiplied by.
                Two ac[C / 2], as[C / 2], bc[C / 2], bs[C / 2], c[C / 2], s[C / 2];
                Which on[C / 2];
                float wa[C], wb[C];
#pragma unroll
                for (int i = 0; i < C; ++i)
                    wa[i] = wb[i] = 1.f;
                if (norm) {
                    ld_weights<DT, C>(wa, w + va[j] * VB + e * E::kSize);
                    ld_weights<DT, C>(wb, w + vb[j] * VB + e * E::kSize);
#pragma unroll
                    for (int i = 0; i < C; ++i) {
                        wa[i] += a.bias;
                        wb[i] += a.bias;
                    }
                }
                couple<C, inter>(ac, bc, wa, wb);
                ld_couples<C, inter>(c, ca, cb, e, on_a, on_b);
                ld_couples<C, inter>(s, ca + a.rope.rd / 2, cb + a.rope.rd / 2, e, on_a, on_b);
#pragma unroll
                for (int i = 0; i < C / 2; ++i) {
                    // An element without a rotation has 1 and 0 here and takes 0
                    // for its partner, not 0 times it, which could be a NaN.
                    on[i] = rotated<C, inter>(i, on_a, on_b);
                    as[i] = ac[i] * s[i];
                    bs[i] = bc[i] * s[i];
                    ac[i] = ac[i] * or_one(c[i], on[i]);
                    bc[i] = bc[i] * or_one(c[i], on[i]);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (h0 + u * HS >= heads)
                        continue; // the whole warp
                    float fa[C], fb[C];
                    Two A[C / 2], B[C / 2];
                    get<DT, VB, C>(fa, x[u][j][0], e);
                    get<DT, VB, C>(fb, x[u][j][1], e);
                    couple<C, inter>(A, B, fa, fb);
#pragma unroll
                    for (int i = 0; i < C / 2; ++i) {
                        const Two xa = A[i] * r[u], xb = B[i] * r[u];
                        A[i] = fma2(xa, ac[i], -(pick(xb, on[i]) * bs[i]));
                        B[i] = fma2(xb, bc[i], pick(xa, on[i]) * as[i]);
                    }
                    uncouple<C, inter>(fa, fb, A, B);
                    put<DT, VB, C>(x[u][j][0], e, fa, code, inv);
                    put<DT, VB, C>(x[u][j][1], e, fb, code, inv);
                }
            }
        }
    } else if (code) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < NP; ++j)
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int e = 0; e < N; e += C) {
                        float f[C];
                        get<DT, VB, C>(f, x[u][j][b], e);
                        put<DT, VB, C>(x[u][j][b], e, f, true, inv);
                    }
    }
    // Out: in place of x, to the output tensor, or to the slot in the cache.
    char *dst;
    int64_t dhs;
    const int64_t h = h0 + own;
    if (cached) {
        const int64_t page = slot / a.page_size;
        dhs = a.cache_hs * (code ? 1 : E::kSize);
        dst = (isv ? a.vc : a.kc) +
              (page * a.page_stride + (slot - page * a.page_size) * a.slot_stride) *
                  (code ? 1 : E::kSize) + h * dhs;
    } else {
        dhs = (isq ? a.qo.hs : a.ko.hs) * E::kSize;
        dst = (isq ? a.qo.p : a.ko.p) + tok * (isq ? a.qo.ts : a.ko.ts) * E::kSize + h * dhs;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            if (!ok || h0 + u * HS + own >= heads || t + j * TPR >= slots)
                continue;
            if (code) {
                st_e4m3<N>(dst + va[j] * N, x[u][j][0]);
                st_e4m3<N>(dst + vb[j] * N, x[u][j][1]);
            } else {
                st_head(dst + va[j] * VB, x[u][j][0]);
                st_head(dst + vb[j] * VB, x[u][j][1]);
            }
        }
        dst += HS * dhs;
    }
}

constexpr int kMostSlots = 128; // 32 lanes with four slots each

// Whether vectors of vb bytes can read and write every head of the call.
bool takes_vectors(const RopeArgs &a, int64_t es, int64_t vb)
{
    const int64_t n = vb / es;
    if (!multiple(a.head_dim, 2 * n) || !multiple(a.rope.rd, a.rope.interleaved ? n : 2 * n) ||
        a.head_dim / (2 * n) > kMostSlots ||
        !aligned(a.rope.cs, std::min<int64_t>(16, 4 * n)) || !aligned(a.qw, vb) ||
        !aligned(a.kw, vb))
        return false;
    for (const HeadsView *v : {&a.q, &a.k, &a.qo, &a.ko, &a.v})
        if (v->p && !view_aligned(*v, es, vb))
            return false;
    if (!a.slots)
        return true;
    const int64_t ces = a.e4m3 ? 1 : es, to = n * ces;
    return aligned(a.kc, to) && aligned(a.vc, to) && multiple(a.page_stride * ces, to) &&
           multiple(a.slot_stride * ces, to) && multiple(a.cache_hs * ces, to);
}

template <int DT, int VB, int TPR, int NP, int U, bool APPEND, int MODE, bool BY_TOKEN = false>
cudaError_t launch_vec(const RopeArgs &a)
{
    constexpr int G = 32 / TPR, per = BY_TOKEN ? U : U * G; // heads of a token a warp takes
    const uint32_t q = (a.q_heads + per - 1) / per, k = (a.k_heads + per - 1) / per;
    const Parts parts = {q, k, q + k * (APPEND ? 2 : 1)};
    const int64_t units = BY_TOKEN ? (a.tokens + G - 1) / G : a.tokens;
    const int64_t blocks = (units * parts.all + kFwdWarps - 1) / kFwdWarps;
    return launch_kernel(rope_kernel<DT, VB, TPR, NP, U, APPEND, MODE, BY_TOKEN>,
                         static_cast<int>(blocks), kFwdWarps * 32, 0, a.base, a, parts);
}

// Heads a lane takes.  One, while that leaves fewer than 20 warps an SM: short
// calls are latency (128 tokens of 32 + 8 heads of 128: 3.4 us, with two 3.4 - 4.1,
// with four 4.1).  Four, when they make three full waves of 32 warps an SM and
// leave few places in a tensor's last warp empty: 16384 tokens 52.9 us, with two
// 54.6; but 2048 tokens 10.2 us, with two 9.6, and 16 + 16 heads of 64, half of
// whose places would be empty, 28.2 us, with two 24.6.  Tensors of so few heads that a
// third of the places would be empty even with two: a token a lane group (appending
// 15274 tokens of 1 + 1 heads of 192: 25.4 -> 14.4 us; 9361 of 6 + 2 of 80: 17.8 -> 10.4).
// The same for vectors of 8 and 4 bytes (5226 tokens of 128 + 16 heads of 80, 20
// elements rotated: 97.8 us; with one head a lane 197).
template <int DT, int VB, int TPR, bool APPEND, int MODE> cudaError_t launch_heads(const RopeArgs &a)
{
    const int64_t tensors = APPEND ? 2 : 1;
    auto places = [&](int64_t per) { // heads with each tensor's last warp filled up
        return (a.q_heads + per - 1) / per * per + tensors * ((a.k_heads + per - 1) / per * per);
    };
    constexpr int G = 32 / TPR;
    if (a.tokens * places(G) / G < 20 * a.sm_count)
        return launch_vec<DT, VB, TPR, 1, 1, APPEND, MODE>(a);
    if constexpr (VB == 16 && G > 1)
        if (2 * places(2 * G) >= 3 * (a.q_heads + tensors * a.k_heads))
            return launch_vec<DT, VB, TPR, 1, 2, APPEND, MODE, true>(a);
    if (4 * places(4 * G) <= 5 * places(2 * G) &&
        a.tokens * places(4 * G) / (4 * G) >= 3 * 32 * a.sm_count)
        return launch_vec<DT, VB, TPR, 1, 4, APPEND, MODE>(a);
    return launch_vec<DT, VB, TPR, 1, 2, APPEND, MODE>(a);
}

// The lanes of a head: the fewest that hold its slots, one each, else 32 with
// up to four slots.
template <int DT, int VB, bool APPEND, int MODE> cudaError_t launch_lanes(const RopeArgs &a)
{
    const int slots = a.head_dim / (2 * kVpe<DT, VB>);
    if constexpr (VB == 16) {
        if (slots <= 4)
            return launch_heads<DT, VB, 4, APPEND, MODE>(a);
        if (slots <= 8)
            return launch_heads<DT, VB, 8, APPEND, MODE>(a);
    }
    if (slots <= 16)
        return launch_heads<DT, VB, 16, APPEND, MODE>(a);
    if (slots <= 32) {
        if constexpr (VB == 16)
            return launch_vec<DT, VB, 32, 1, 1, APPEND, MODE>(a);
        else
            return launch_heads<DT, VB, 32, APPEND, MODE>(a);
    }
    if constexpr (VB < 16 || Elem<DT>::kSize == 4)
        if (slots > 64)
            return launch_vec<DT, VB, 32, 4, 1, APPEND, MODE>(a);
    return launch_vec<DT, VB, 32, 2, 1, APPEND, MODE>(a); // up to 64 (head_dim <= 1024)
}

template <int DT, int VB, bool APPEND> cudaError_t launch_mode(const RopeArgs &a)
{
    if (a.rope.interleaved)
        return launch_lanes<DT, VB, APPEND, kInterleaved>(a);
    if (VB == 16 && a.rope.rd == a.head_dim)
        return launch_lanes<DT, VB, APPEND, VB == 16 ? kHalvesFull : kHalves>(a);
    return launch_lanes<DT, VB, APPEND, kHalves>(a);
}

template <int DT, bool APPEND> cudaError_t launch_append(const RopeArgs &a, bool *taken)
{
    constexpr int64_t es = Elem<DT>::kSize;
    *taken = true;
    // Warps, of a head each at least, are counted in 32 bits.
    if (a.tokens <= (int64_t(1) << 31) / (a.q_heads + 2 * a.k_heads)) {
        if (takes_vectors(a, es, 16))
            return launch_mode<DT, 16, APPEND>(a);
        if (takes_vectors(a, es, 8))
            return launch_mode<DT, 8, APPEND>(a);
        if constexpr (es == 2)
            if (takes_vectors(a, es, 4))
                return launch_mode<DT, 4, APPEND>(a);
    }
    *taken = false;
    return cudaSuccess;
}

// Launches a vector body if one takes the call.
template <int DT> cudaError_t launch_vectors(const RopeArgs &a, bool *taken)
{
    return a.slots ? launch_append<DT, true>(a, taken) : launch_append<DT, false>(a, taken);
}

} // namespace
} // namespace rmsnorm
