// rope_bwd.cu -- the gradient of the per-head QK norm with its rotation.
//
//   du = rotate back(dy),  xh = x r,  g = w + bias
//   dx = r (du g - xh m),  m = sum(du g xh) / head_dim
//   dw = sum over tokens and heads of du xh
//
// Two inputs read and one output written once: memory bounds it.  A block
// works on q or on k alone and keeps its part of dw on chip; it leaves one
// row of the workspace, and launch_colsum adds the rows up in a fixed order.
#include <algorithm>

#include "rope.cuh"

namespace rmsnorm {

#ifndef MINB
#define MINB 4
#endif
#ifndef STAGES
#define STAGES 3
#endif
#ifndef ITERS
#define ITERS 4
#endif
#ifndef ITEMS
#define ITEMS 8
#endif
// A workspace row per block: MINB blocks on every SM, and one more for each
// tensor's rounding.
int rope_bwd_max_blocks(int sm_count) { return MINB * sm_count + 2; }

namespace {

constexpr int kBwdThreads = 128; // of the vector bodies

// Blocks that take q; the others take k.  In proportion to the heads, at
// least one for a tensor that has any.
struct BlockSplit {
    int q, k;
};

// Any alignment and head size: a warp per head of a token, scalar accesses;
// each warp sums its dw in its own row of shared memory.
template <int DT>
__global__ void __launch_bounds__(256) rope_bwd_scalar_kernel(const RopeBwdArgs a, BlockSplit split)
{
    using E = Elem<DT>;
    extern __shared__ float acc[]; // [8][head_dim]
    pdl_begin();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int D = a.head_dim, rd = a.rope.rd, half = rd / 2;
    const bool isq = static_cast<int>(blockIdx.x) < split.q;
    const int block = isq ? blockIdx.x : blockIdx.x - split.q;
    const int blocks = isq ? split.q : split.k;
    const int heads = isq ? a.q_heads : a.k_heads;
    const HeadsView vdy = isq ? a.qdy : a.kdy, vx = isq ? a.q : a.k, vdx = isq ? a.dq : a.dk;
    const void *w = isq ? a.qw : a.kw;
    const float n = static_cast<float>(D);
    float *mine = acc + warp * D;
    for (int d = lane; d < D; d += 32)
        mine[d] = 0.f;
    __syncwarp();
    const int64_t total = a.tokens * heads;
    for (int64_t item = static_cast<int64_t>(block) * 8 + warp; item < total;
         item += static_cast<int64_t>(blocks) * 8) {
        const int64_t tok = item / heads;
        const int h = static_cast<int>(item - tok * heads);
        const float *cs;
        if (!rope_row(a.rope, tok, cs)) {
            if (lane == 0 && h == 0)
                record_bad_index(a.base.status);
            continue;
        }
        const char *x = vx.p + (tok * vx.ts + h * vx.hs) * E::kSize;
        const char *dy = vdy.p + (tok * vdy.ts + h * vdy.hs) * E::kSize;
        char *dx = vdx.p + (tok * vdx.ts + h * vdx.hs) * E::kSize;
        auto sum = [&](float k) {
            float s = 0.f;
            for (int d = lane; d < D; d += 32) {
                const float v = E::widen1(x, d) * k;
                s = fmaf(v, v, s);
            }
            return group_allreduce<32>(s);
        };
        const RowScale f = row_scale<DT>(sum(1.f), n, a.eps, sum);
        // Elements a and b of pair i (i >= half: one unrotated element, db < 0)
        // with their du and xh.
        struct Pair {
            int da, db;
            float dua, dub, xa, xb;
        };
        auto pair = [&](int i) {
            Pair p;
            if (i >= half) {
                p.da = i + half;
                p.db = -1;
                p.dua = E::widen1(dy, p.da);
                p.dub = p.xb = 0.f;
            } else {
                p.da = a.rope.interleaved ? 2 * i : i;
                p.db = a.rope.interleaved ? 2 * i + 1 : i + half;
                const float ya = E::widen1(dy, p.da), yb = E::widen1(dy, p.db);
                const float c = cs[i], s = cs[half + i];
                p.dua = fmaf(ya, c, yb * s);
                p.dub = fmaf(yb, c, -(ya * s));
                p.xb = E::widen1(x, p.db) * f.pre * f.r;
            }
            p.xa = E::widen1(x, p.da) * f.pre * f.r;
            return p;
        };
        float m = 0.f;
        for (int i = lane; i < D - half; i += 32) {
            const Pair p = pair(i);
            m = fmaf(p.dua * (E::widen1(w, p.da) + a.bias), p.xa, m);
            mine[p.da] = fmaf(p.dua, p.xa, mine[p.da]);
            if (p.db >= 0) {
                m = fmaf(p.dub * (E::widen1(w, p.db) + a.bias), p.xb, m);
                mine[p.db] = fmaf(p.dub, p.xb, mine[p.db]);
            }
        }
        m = group_allreduce<32>(m) / n;
        for (int i = lane; i < D - half; i += 32) {
            const Pair p = pair(i);
            const float va = fmaf(p.dua, E::widen1(w, p.da) + a.bias, -(p.xa * m));
            E::store1(dx, p.da, va * f.r * f.pre);
            if (p.db >= 0) {
                const float vb = fmaf(p.dub, E::widen1(w, p.db) + a.bias, -(p.xb * m));
                E::store1(dx, p.db, vb * f.r * f.pre);
            }
        }
        __syncwarp();
    }
    if (!a.part)
        return;
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += 256) {
        float s = 0.f;
        for (int v = 0; v < 8; ++v)
            s += acc[v * D + d];
        a.part[static_cast<int64_t>(blockIdx.x) * D + d] = s;
    }
}

// ---- heads in vectors (rope.cuh)
//
// Each lane copies its own vectors of x and dy ahead into a ring in shared
// memory (cp.async; no lane reads another's, so only its own copies are
// waited for), which keeps the bytes on the way out of the registers that
// dw's sums, the angles and the weights take.  A warp keeps to one tensor and
// goes through chunks of a token's heads, 32 / TPR at a time.

template <int VB> __device__ inline void cp_async(uint32_t dst, const void *src)
{
    if constexpr (VB == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(VB)
                     : "memory");
}
template <int VB> __device__ inline void ld_ring(Vec<VB> &v, uint32_t p)
{
    if constexpr (VB == 16)
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3])
                     : "r"(p)
                     : "memory");
    else if constexpr (VB == 8)
        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];"
                     : "=r"(v.w[0]), "=r"(v.w[1])
                     : "r"(p)
                     : "memory");
    else
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v.w[0]) : "r"(p) : "memory");
}

// How tokens' heads are cut: chunks of a token's heads, iters steps of
// 32 / TPR heads each.
struct Chunks {
    uint32_t per_token, iters;
};

// A warp's place in its chunks.
struct Cursor {
    uint32_t item, tok, step, end; // step .. end: steps of the token in this chunk
    __device__ inline void start(uint32_t i, const Chunks &c, uint32_t steps)
    {
        item = i;
        tok = i / c.per_token;
        step = (i - tok * c.per_token) * c.iters;
        end = min(step + c.iters, steps);
    }
    __device__ inline void next(uint32_t stride, const Chunks &c, uint32_t steps)
    {
        if (++step == end)
            start(item + stride, c, steps);
    }
};

template <int DT, int VB, int TPR, int NP, int MODE>
__global__ void __launch_bounds__(kBwdThreads, NP == 1 ? MINB : 1)
rope_bwd_kernel(const __grid_constant__ RopeBwdArgs a, BlockSplit split, Chunks qc, Chunks kc)
{
    using E = Elem<DT>;
    constexpr int N = kVpe<DT, VB>;
    constexpr int G = 32 / TPR;
    constexpr int C = N < 4 ? N : 4;
    constexpr int S = NP == 1 ? STAGES : NP == 2 ? 2 : 1; // ring stages
    constexpr int kAhead = S > 1 ? S - 1 : 1;        // steps asked for ahead
    constexpr int kStage = NP * 4 * 32 * VB;         // bytes of a warp's stage
    constexpr int kWarps = kBwdThreads / 32;
    constexpr bool inter = MODE == kInterleaved;
    __shared__ alignas(16) char ring[kWarps * S * kStage];
    pdl_begin();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = lane % TPR, g = lane / TPR;
    const bool isq = static_cast<int>(blockIdx.x) < split.q;
    const Chunks ch = isq ? qc : kc;
    const int heads = isq ? a.q_heads : a.k_heads;
    const uint32_t steps = (heads + G - 1) / G;
    const uint32_t items = static_cast<uint32_t>(a.tokens) * ch.per_token;
    const uint32_t block = isq ? blockIdx.x : blockIdx.x - split.q;
    const uint32_t stride = (isq ? split.q : split.k) * kWarps;
    const int slots = a.head_dim / (2 * N), half_v = a.rope.rd / (2 * N);
    const char *xb = isq ? a.q.p : a.k.p, *yb = isq ? a.qdy.p : a.kdy.p;
    char *ob = isq ? a.dq.p : a.dk.p;
    const int64_t xts = isq ? a.q.ts : a.k.ts, xhs = isq ? a.q.hs : a.k.hs;
    const int64_t yts = isq ? a.qdy.ts : a.kdy.ts, yhs = isq ? a.qdy.hs : a.kdy.hs;
    const int64_t ots = isq ? a.dq.ts : a.dk.ts, ohs = isq ? a.dq.hs : a.dk.hs;
    const RowCount n = row_count(a.head_dim);
    int va[NP], vb[NP];
#pragma unroll
    for (int j = 0; j < NP; ++j)
        slot_vectors(t + j * TPR, slots, half_v, inter, va[j], vb[j]);

    // This lane's weights, and its sums of dw as couples.
    Vec<VB> w[NP][2];
    uint64_t accA[NP][N / 2], accB[NP][N / 2];
#pragma unroll
    for (int j = 0; j < NP; ++j) {
        vzero(w[j][0]);
        vzero(w[j][1]);
        if (t + j * TPR < slots) {
            const char *ws = static_cast<const char *>(isq ? a.qw : a.kw);
            ld_const(w[j][0], ws + va[j] * VB);
            ld_const(w[j][1], ws + vb[j] * VB);
        }
#pragma unroll
        for (int i = 0; i < N / 2; ++i)
            accA[j][i] = accB[j][i] = 0;
    }

    const uint32_t my = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) +
                        warp * (S * kStage) + lane * VB;
    // Asks a step's vectors into a stage (its two vectors of x, then of dy).
    auto ask = [&](const Cursor &c, uint32_t stage) {
        const int h = static_cast<int>(c.step) * G + g;
        if (c.item < items && h < heads) {
            const char *x = xb + (c.tok * xts + h * xhs) * E::kSize;
            const char *y = yb + (c.tok * yts + h * yhs) * E::kSize;
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                if (t + j * TPR >= slots)
                    continue;
                const uint32_t p = my + stage * kStage + j * (4 * 32 * VB);
                cp_async<VB>(p, x + va[j] * VB);
                cp_async<VB>(p + 32 * VB, x + vb[j] * VB);
                cp_async<VB>(p + 64 * VB, y + va[j] * VB);
                cp_async<VB>(p + 96 * VB, y + vb[j] * VB);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    Cursor at, ahead;
    at.start(block * kWarps + warp, ch, steps);
    ahead = at;
    auto ask_next = [&](uint32_t stage) {
        ask(ahead, stage);
        if (ahead.item < items)
            ahead.next(stride, ch, steps);
    };
#pragma unroll
    for (int s = 0; s < kAhead; ++s)
        ask_next(s);
    uint32_t stage = 0;
    bool fresh = true, bad = false;
    // The token's angles as the couples take them.
    uint64_t cc[NP][N / 2], ss[NP][N / 2];
    int64_t next_pos = a.rope.rd && at.item < items ? a.rope.pos[at.tok] : 0;
    while (at.item < items) {
        if (fresh) {
            const int64_t pos = next_pos;
            bad = a.rope.rd && (pos < 0 || pos >= a.rope.max_pos);
            if (bad && lane == 0 && at.step == 0)
                record_bad_index(a.base.status);
            const uint32_t after = at.item + stride;
            if (a.rope.rd && after < items)
                next_pos = a.rope.pos[after / ch.per_token];
            const float *cs = a.rope.cs + (bad ? 0 : pos) * a.rope.rd;
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                const int p = t + j * TPR;
                const bool on_a = !bad && p < slots &&
                                  (inter ? va[j] * N < a.rope.rd : p < half_v);
                const bool on_b = inter ? !bad && p < slots && vb[j] * N < a.rope.rd : on_a;
                const float *ca = cs + (inter ? va[j] * (N / 2) : p * N);
                const float *cb = cs + vb[j] * (N / 2);
#pragma unroll
                for (int e = 0; e < N; e += C) {
                    uint64_t c[C / 2], s[C / 2];
                    ld_couples<C, inter>(c, ca, cb, e, on_a, on_b);
                    ld_couples<C, inter>(s, ca + a.rope.rd / 2, cb + a.rope.rd / 2, e, on_a, on_b);
#pragma unroll
                    for (int i = 0; i < C / 2; ++i) {
                        const uint64_t on = couple_mask<C, inter>(i, on_a, on_b);
                        cc[j][e / 2 + i] = c[i] | (~on & f2(1.f, 1.f));
                        ss[j][e / 2 + i] = s[i];
                    }
                }
            }
        }
        // All but the newest kAhead - 1 of this lane's groups have arrived.
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
        const int h = static_cast<int>(at.step) * G + g;
        const bool live = h < heads;
        Vec<VB> x[NP][2], y[NP][2];
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            if (live && t + j * TPR < slots) {
                const uint32_t p = my + stage * kStage + j * (4 * 32 * VB);
                ld_ring(x[j][0], p);
                ld_ring(x[j][1], p + 32 * VB);
                ld_ring(y[j][0], p + 64 * VB);
                ld_ring(y[j][1], p + 96 * VB);
            } else {
                vzero(x[j][0]);
                vzero(x[j][1]);
                vzero(y[j][0]);
                vzero(y[j][1]);
            }
        }
        if constexpr (S > 1) // into the stage of the step before, whose values are used
            ask_next(stage == 0 ? S - 1 : stage - 1);
        stage = stage + 1 == S ? 0 : stage + 1;
        if (!bad) {
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < NP; ++j)
                sum = sumsq_mixed<DT, VB>(x[j][1], sumsq_mixed<DT, VB>(x[j][0], sum));
            // A group without a head keeps finite numbers: its zeros are summed.
            sum = group_allreduce<TPR>(sum);
            if (!live)
                sum = 1.f;
            float r = row_factor(sum, n, a.eps), k = 1.f;
            const bool redo = bwd_rescales<DT>(sum, a.eps);
            const bool rare = kRangeGuard<DT> && __any_sync(0xFFFFFFFFu, redo);
            if (rare) {
                const float kk = redo ? bwd_rescale_k(sum, a.eps) : 1.f;
                float sk = 0.f;
#pragma unroll
                for (int j = 0; j < NP; ++j) {
                    scale_by<DT, VB>(x[j][0], kk);
                    scale_by<DT, VB>(x[j][1], kk);
                    sk = sumsq<DT, VB>(x[j][1], sumsq<DT, VB>(x[j][0], sk));
                }
                k = kk;
                r = row_factor(group_allreduce<TPR>(sk), n, (a.eps * kk) * kk);
            }
            // du, and sum(du g x); dw's sums take du * (x r).
            uint64_t eA[NP][N / 2], eB[NP][N / 2], dot = 0;
            const uint64_t r2 = f2(r, r);
#pragma unroll
            for (int j = 0; j < NP; ++j)
#pragma unroll
                for (int e = 0; e < N; e += C) {
                    float fa[C], fb[C];
                    uint64_t gA[C / 2], gB[C / 2], xA[C / 2], xB[C / 2], yA[C / 2], yB[C / 2];
                    get<DT, VB, C>(fa, w[j][0], e);
                    get<DT, VB, C>(fb, w[j][1], e);
                    couple<C, inter>(gA, gB, fa, fb);
                    get<DT, VB, C>(fa, x[j][0], e);
                    get<DT, VB, C>(fb, x[j][1], e);
                    couple<C, inter>(xA, xB, fa, fb);
                    get<DT, VB, C>(fa, y[j][0], e);
                    get<DT, VB, C>(fb, y[j][1], e);
                    couple<C, inter>(yA, yB, fa, fb);
                    const bool on_a = MODE == kHalvesFull ||
                                      (inter ? va[j] * N < a.rope.rd : t + j * TPR < half_v);
                    const bool on_b = inter ? vb[j] * N < a.rope.rd : on_a;
#pragma unroll
                    for (int i = 0; i < C / 2; ++i) {
                        const uint64_t on = couple_mask<C, inter>(i, on_a, on_b);
                        const uint64_t c = cc[j][e / 2 + i], s = ss[j][e / 2 + i];
                        const uint64_t duA = fma2(yA[i], c, mul2(yB[i] & on, s));
                        const uint64_t duB = fma2(yB[i], c, neg2(mul2(yA[i] & on, s)));
                        const uint64_t b2 = f2(a.bias, a.bias);
                        uint64_t &aA = accA[j][e / 2 + i], &aB = accB[j][e / 2 + i];
                        aA = fma2(duA, mul2(xA[i], r2), aA);
                        aB = fma2(duB, mul2(xB[i], r2), aB);
                        eA[j][e / 2 + i] = mul2(duA, add2(gA[i], b2));
                        eB[j][e / 2 + i] = mul2(duB, add2(gB[i], b2));
                        dot = fma2(eA[j][e / 2 + i], xA[i], dot);
                        dot = fma2(eB[j][e / 2 + i], xB[i], dot);
                    }
                }
            float d0, d1;
            f2split(dot, d0, d1);
            const float total = group_allreduce<TPR>(d0 + d1);
            // dx = r (e - x r m), m = r total / n
            const float m = n.pow2 ? total * n.inv : total / n.n;
            const float q = -(r * m) * r;
            const uint64_t q2 = f2(q, q);
            char *o = ob + (at.tok * ots + h * ohs) * E::kSize;
#pragma unroll
            for (int j = 0; j < NP; ++j) {
#pragma unroll
                for (int e = 0; e < N; e += C) {
                    float fa[C], fb[C];
                    uint64_t xA[C / 2], xB[C / 2];
                    get<DT, VB, C>(fa, x[j][0], e);
                    get<DT, VB, C>(fb, x[j][1], e);
                    couple<C, inter>(xA, xB, fa, fb);
#pragma unroll
                    for (int i = 0; i < C / 2; ++i) {
                        xA[i] = mul2(fma2(xA[i], q2, eA[j][e / 2 + i]), r2);
                        xB[i] = mul2(fma2(xB[i], q2, eB[j][e / 2 + i]), r2);
                    }
                    uncouple<C, inter>(fa, fb, xA, xB);
                    if (rare) {
#pragma unroll
                        for (int i = 0; i < C; ++i) {
                            fa[i] *= k;
                            fb[i] *= k;
                        }
                    }
                    put<DT, VB, C>(x[j][0], e, fa);
                    put<DT, VB, C>(x[j][1], e, fb);
                }
                if (live && t + j * TPR < slots) {
                    st_head(o + va[j] * VB, x[j][0]);
                    st_head(o + vb[j] * VB, x[j][1]);
                }
            }
        }
        if constexpr (S == 1)
            ask_next(0);
        const uint32_t item = at.item;
        at.next(stride, ch, steps);
        fresh = at.item != item;
    }
    if (!a.part)
        return;
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads(); // every warp is done with its ring
    // The block's sums: over the groups of a warp, then over the warps, in order.
    float *sums = reinterpret_cast<float *>(ring); // [kWarps][head_dim]
#pragma unroll
    for (int j = 0; j < NP; ++j)
#pragma unroll
        for (int e = 0; e < N; e += C) {
            uint64_t A[C / 2], B[C / 2];
            float fa[C], fb[C];
#pragma unroll
            for (int i = 0; i < C / 2; ++i) {
                A[i] = accA[j][e / 2 + i];
                B[i] = accB[j][e / 2 + i];
            }
            uncouple<C, inter>(fa, fb, A, B);
#pragma unroll
            for (int i = 0; i < C; ++i) {
#pragma unroll
                for (int off = TPR; off < 32; off <<= 1) {
                    fa[i] += __shfl_xor_sync(0xFFFFFFFFu, fa[i], off);
                    fb[i] += __shfl_xor_sync(0xFFFFFFFFu, fb[i], off);
                }
                if (g == 0 && t + j * TPR < slots) {
                    sums[warp * a.head_dim + va[j] * N + e + i] = fa[i];
                    sums[warp * a.head_dim + vb[j] * N + e + i] = fb[i];
                }
            }
        }
    __syncthreads();
    for (int d = threadIdx.x; d < a.head_dim; d += kBwdThreads) {
        float s = 0.f;
#pragma unroll
        for (int v = 0; v < kWarps; ++v)
            s += sums[v * a.head_dim + d];
        a.part[static_cast<int64_t>(blockIdx.x) * a.head_dim + d] = s;
    }
}

constexpr int kMostSlots = 128;

// Whether vectors of vb bytes can read and write every head of the call.
bool takes_vectors(const RopeBwdArgs &a, int64_t es, int64_t vb)
{
    const int64_t n = vb / es;
    if (!multiple(a.head_dim, 2 * n) || !multiple(a.rope.rd, 2 * n) ||
        a.head_dim / (2 * n) > kMostSlots ||
        !aligned(a.rope.cs, std::min<int64_t>(16, 4 * n)) || !aligned(a.qw, vb) ||
        !aligned(a.kw, vb))
        return false;
    for (const HeadsView *v : {&a.qdy, &a.kdy, &a.q, &a.k, &a.dq, &a.dk})
        if (v->p && !view_aligned(*v, es, vb))
            return false;
    return true;
}

template <int DT, int VB, int TPR, int NP, int MODE> cudaError_t launch_vec(const RopeBwdArgs &a, BlockSplit *split)
{
    constexpr int G = 32 / TPR, kWarps = kBwdThreads / 32;
    const int64_t most = rope_bwd_max_blocks(a.sm_count) - 2; // blocks on all SMs
    const int64_t heads = int64_t(a.q_heads) + a.k_heads;
    auto cut = [&](int64_t h, int *blocks) {
        Chunks c = {1, 1};
        *blocks = 0;
        if (!h)
            return c;
        const int64_t steps = (h + G - 1) / G, share = std::max<int64_t>(1, most * h / heads);
        // The longest chunks (up to ITERS steps) that leave every warp ITEMS of them.
        int64_t iters = std::min<int64_t>(steps, ITERS);
        while (iters > 1 && a.tokens * ((steps + iters - 1) / iters) < ITEMS * share * kWarps)
            iters = (iters + 1) / 2;
        c.iters = static_cast<uint32_t>(iters);
        c.per_token = static_cast<uint32_t>((steps + iters - 1) / iters);
        const int64_t items = a.tokens * c.per_token;
        *blocks = static_cast<int>(std::max<int64_t>(1, std::min(share, (items + kWarps - 1) / kWarps)));
        return c;
    };
    const Chunks q = cut(a.q_heads, &split->q), k = cut(a.k_heads, &split->k);
    return launch_kernel(rope_bwd_kernel<DT, VB, TPR, NP, MODE>, split->q + split->k, kBwdThreads,
                         0, a.base, a, *split, q, k);
}

template <int DT, int VB, int MODE> cudaError_t launch_lanes(const RopeBwdArgs &a, BlockSplit *split)
{
    const int slots = a.head_dim / (2 * kVpe<DT, VB>);
    if constexpr (VB == 16) {
        if (slots <= 4)
            return launch_vec<DT, VB, 4, 1, MODE>(a, split);
        if (slots <= 8)
            return launch_vec<DT, VB, 8, 1, MODE>(a, split);
    }
    if (slots <= 16)
        return launch_vec<DT, VB, 16, 1, MODE>(a, split);
    if (slots <= 32)
        return launch_vec<DT, VB, 32, 1, MODE>(a, split);
    if constexpr (VB < 16 || Elem<DT>::kSize == 4)
        if (slots > 64)
            return launch_vec<DT, VB, 32, 4, MODE>(a, split);
    return launch_vec<DT, VB, 32, 2, MODE>(a, split); // up to 64 (head_dim <= 1024)
}

template <int DT, int VB> cudaError_t launch_mode(const RopeBwdArgs &a, BlockSplit *split)
{
    if (a.rope.interleaved)
        return launch_lanes<DT, VB, kInterleaved>(a, split);
    if (VB == 16 && a.rope.rd == a.head_dim)
        return launch_lanes<DT, VB, VB == 16 ? kHalvesFull : kHalves>(a, split);
    return launch_lanes<DT, VB, kHalves>(a, split);
}

template <int DT> cudaError_t launch_scalar(const RopeBwdArgs &a, BlockSplit *split)
{
    const int64_t heads = int64_t(a.q_heads) + a.k_heads, most = 4 * a.sm_count;
    auto take = [&](int64_t h) {
        const int64_t want = (a.tokens * h + 7) / 8;
        return h ? std::max<int64_t>(1, std::min(want, (most * h + heads - 1) / heads)) : 0;
    };
    *split = {static_cast<int>(take(a.q_heads)), static_cast<int>(take(a.k_heads))};
    return launch_kernel(rope_bwd_scalar_kernel<DT>, split->q + split->k, 256, 8 * a.head_dim * 4,
                         a.base, a, *split);
}

template <int DT> cudaError_t launch(const RopeBwdArgs &a)
{
    constexpr int64_t es = Elem<DT>::kSize;
    BlockSplit split = {0, 0};
    cudaError_t err = cudaSuccess;
    const int64_t heads = int64_t(a.q_heads) + a.k_heads;
    if (heads > 0) {
        // Steps of heads are counted in 32 bits.
        const bool counts = a.tokens <= (int64_t(1) << 30) / heads;
        if (counts && takes_vectors(a, es, 16))
            err = launch_mode<DT, 16>(a, &split);
        else if (counts && takes_vectors(a, es, 8))
            err = launch_mode<DT, 8>(a, &split);
        else if (counts && es == 2 && takes_vectors(a, es, 4))
            err = launch_mode<DT, es == 2 ? 4 : 8>(a, &split);
        else
            err = launch_scalar<DT>(a, &split);
    }
    if (err != cudaSuccess || !a.part)
        return err;
    const int64_t D = a.head_dim;
    return launch_colsum({a.part, a.dqw, split.q, D, D},
                         {a.part + split.q * D, a.dkw, split.k, D, D}, a.base);
}

} // namespace

cudaError_t launch_rope_bwd(const RopeBwdArgs &a, int dtype)
{
    return dtype == RMSNORM_F32    ? launch<RMSNORM_F32>(a)
           : dtype == RMSNORM_BF16 ? launch<RMSNORM_BF16>(a)
                                   : launch<RMSNORM_F16>(a);
}

} // namespace rmsnorm
