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

constexpr int kBwdBlocksPerSm = 4; // of 128 threads with up to 128 registers

// A workspace row per block: all SMs' blocks, and one more for each tensor's
// rounding.
int rope_bwd_max_blocks(int sm_count) { return kBwdBlocksPerSm * sm_count + 2; }

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
// A warp keeps to one tensor and goes through a run of consecutive steps, 32 /
// TPR heads of a token each.  Every lane copies its own vectors of x and dy
// ahead into a ring in shared memory (cp.async; no lane reads another's, so
// only its own copies are waited for): the bytes on the way take no registers,
// which dw's sums, the angles and g fill.  The angles are loaded once a token.
//
// What bounds it: instructions first (the same time without its loads or
// stores), memory close behind.  Measured with launch_colsum (16384 tokens of
// 32 + 8 bf16 heads of 128, 505 MB, floor 75.7 us at the copy bandwidth): scalar
// body 521 us, this one 86.8 us (5.83 TB/s, 87 %).  On the way: warps that take
// short chunks of many tokens in turn 96.8 us (61 M warp instructions for 49 M: a
// division and the angles every chunk); two passes over x and dy in registers,
// 24 warps an SM and no ring, 114 us (67 M: widening and angles twice), the same
// without the packed instructions 122 us (81 M).  128 registers and 16 warps an SM
// (96 and 20: 114 us, spills); 3 stages (4: 92.9 us: the larger ring leaves L1 no
// room for the angles).
//
// BY_TOKEN: each lane group takes a token of its own and goes through its heads,
// for tensors of so few heads that a warp within one token would stand half empty.
template <int DT, int VB, int TPR, int NP, int MODE, bool BY_TOKEN>
__global__ void __launch_bounds__(kBwdThreads, NP == 1 ? kBwdBlocksPerSm : 1)
rope_bwd_kernel(const __grid_constant__ RopeBwdArgs a, BlockSplit split)
{
    using E = Elem<DT>;
    constexpr int N = kVpe<DT, VB>;
    constexpr int G = 32 / TPR;
    constexpr int C = N < 4 ? N : 4;
    constexpr int S = NP == 1 ? 3 : NP == 2 ? 2 : 1; // ring stages
    constexpr int kAhead = S > 1 ? S - 1 : 1;        // steps asked for ahead
    constexpr int kStage = NP * 4 * 32 * VB;         // bytes of a warp's stage
    constexpr int kWarps = kBwdThreads / 32;
    constexpr bool inter = MODE == kInterleaved;
    __shared__ alignas(16) char ring[kWarps * S * kStage];
    pdl_begin();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = lane % TPR, g = lane / TPR;
    const bool isq = static_cast<int>(blockIdx.x) < split.q;
    const int heads = isq ? a.q_heads : a.k_heads;
    // A unit is a token, or G of them; its steps go through the heads.
    constexpr int HS = BY_TOKEN ? 1 : G; // heads between a lane's
    const uint32_t steps = (heads + HS - 1) / HS;
    const int own = BY_TOKEN ? 0 : g;    // this lane's first head
    auto token = [&](uint32_t unit) -> int64_t {
        return BY_TOKEN ? static_cast<int64_t>(unit) * G + g : unit;
    };
    const int slots = a.head_dim / (2 * N), half_v = a.rope.rd / (2 * N);
    const char *xb = isq ? a.q.p : a.k.p, *yb = isq ? a.qdy.p : a.kdy.p;
    char *ob = isq ? a.dq.p : a.dk.p;
    const int64_t xts = (isq ? a.q.ts : a.k.ts) * E::kSize, xhs = (isq ? a.q.hs : a.k.hs) * E::kSize;
    const int64_t yts = (isq ? a.qdy.ts : a.kdy.ts) * E::kSize,
                  yhs = (isq ? a.qdy.hs : a.kdy.hs) * E::kSize;
    const int64_t ots = (isq ? a.dq.ts : a.dk.ts) * E::kSize,
                  ohs = (isq ? a.dq.hs : a.dk.hs) * E::kSize;
    const float inv_n = 1.f / static_cast<float>(a.head_dim);
    int va[NP], vb[NP];
#pragma unroll
    for (int j = 0; j < NP; ++j)
        slot_vectors(t + j * TPR, slots, half_v, inter, va[j], vb[j]);

    // This warp's steps: an even share of the tensor's, in order.
    uint32_t left, first;
    {
        const uint64_t all =
            static_cast<uint64_t>(BY_TOKEN ? (a.tokens + G - 1) / G : a.tokens) * steps;
        const uint64_t block = isq ? blockIdx.x : blockIdx.x - split.q;
        const uint64_t warps = static_cast<uint64_t>(isq ? split.q : split.k) * kWarps;
        const uint64_t i = block * kWarps + __shfl_sync(0xFFFFFFFFu, warp, 0);
        first = static_cast<uint32_t>(all * i / warps);
        left = static_cast<uint32_t>(all * (i + 1) / warps) - first;
    }

    // This lane's g = w + bias, and its sums of dw, as couples.
    Two gA[NP][N / 2], gB[NP][N / 2], accA[NP][N / 2], accB[NP][N / 2];
#pragma unroll
    for (int j = 0; j < NP; ++j) {
        Vec<VB> w[2];
        vzero(w[0]);
        vzero(w[1]);
        if (t + j * TPR < slots) {
            const char *ws = static_cast<const char *>(isq ? a.qw : a.kw);
            ld_const(w[0], ws + va[j] * VB);
            ld_const(w[1], ws + vb[j] * VB);
        }
#pragma unroll
        for (int e = 0; e < N; e += C) {
            float fa[C], fb[C];
            Two A[C / 2], B[C / 2];
            get<DT, VB, C>(fa, w[0], e);
            get<DT, VB, C>(fb, w[1], e);
            couple<C, inter>(A, B, fa, fb);
#pragma unroll
            for (int i = 0; i < C / 2; ++i) {
                gA[j][e / 2 + i] = A[i] + a.bias;
                gB[j][e / 2 + i] = B[i] + a.bias;
                accA[j][e / 2 + i] = accB[j][e / 2 + i] = two(0.f, 0.f);
            }
        }
    }

    const uint32_t my = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) +
                        warp * (S * kStage) + lane * VB;
    // The step asked for next, and the step worked on.
    uint32_t unit_in = first / steps, in = first - unit_in * steps, left_in = left;
    uint32_t unit = unit_in, step = in;
    const char *px = xb + token(unit_in) * xts + (int64_t(in) * HS + own) * xhs;
    const char *py = yb + token(unit_in) * yts + (int64_t(in) * HS + own) * yhs;
    char *po = ob + token(unit) * ots + (int64_t(step) * HS + own) * ohs;
    // Asks a step's vectors into a stage (its two vectors of x, then of dy).
    auto ask_next = [&](uint32_t stage) {
        if (left_in) {
            if (BY_TOKEN ? token(unit_in) < a.tokens : static_cast<int>(in) * G + g < heads) {
#pragma unroll
                for (int j = 0; j < NP; ++j) {
                    if (t + j * TPR >= slots)
                        continue;
                    const uint32_t p = my + stage * kStage + j * (4 * 32 * VB);
                    cp_async<VB>(p, px + va[j] * VB);
                    cp_async<VB>(p + 32 * VB, px + vb[j] * VB);
                    cp_async<VB>(p + 64 * VB, py + va[j] * VB);
                    cp_async<VB>(p + 96 * VB, py + vb[j] * VB);
                }
            }
            --left_in;
            px += HS * xhs;
            py += HS * yhs;
            if (++in == steps) {
                in = 0;
                ++unit_in;
                px = xb + token(unit_in) * xts + own * xhs;
                py = yb + token(unit_in) * yts + own * yhs;
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int s = 0; s < kAhead; ++s)
        ask_next(s);
    uint32_t stage = 0;
    bool fresh = true, bad = false;
    // The token's angles as the couples take them.
    Two cc[NP][N / 2], ss[NP][N / 2];
    auto position = [&](uint32_t u) -> int64_t {
        return a.rope.rd && token(u) < a.tokens ? a.rope.pos[token(u)] : 0;
    };
    int64_t next_pos = left ? position(unit) : 0;
    for (; left; --left) {
        if (fresh) {
            const int64_t pos = next_pos;
            bad = a.rope.rd && (pos < 0 || pos >= a.rope.max_pos);
            const bool there = !BY_TOKEN || token(unit) < a.tokens;
            if (bad && there && t == 0)
                record_bad_index(a.base.status);
            bad = bad || !there;
            next_pos = position(unit + 1);
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
                    Two c[C / 2], s[C / 2];
                    ld_couples<C, inter>(c, ca, cb, e, on_a, on_b);
                    ld_couples<C, inter>(s, ca + a.rope.rd / 2, cb + a.rope.rd / 2, e, on_a, on_b);
#pragma unroll
                    for (int i = 0; i < C / 2; ++i) {
                        cc[j][e / 2 + i] = or_one(c[i], rotated<C, inter>(i, on_a, on_b));
                        ss[j][e / 2 + i] = s[i];
                    }
                }
            }
        }
        // All but the newest kAhead - 1 of this lane's groups have arrived.
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
        const bool live = BY_TOKEN ? !bad : static_cast<int>(step) * G + g < heads;
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
        if (BY_TOKEN || !bad) { // else the whole warp's token
            // du, and the two sums of a head: x^2 and du g x.
            Two dA[NP][N / 2], dB[NP][N / 2], xA[NP][N / 2], xB[NP][N / 2];
            Two dotA = two(0.f, 0.f), dotB = dotA;
            float sq[2] = {};
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                const bool on_a = MODE == kHalvesFull ||
                                  (inter ? va[j] * N < a.rope.rd : t + j * TPR < half_v);
                const bool on_b = inter ? vb[j] * N < a.rope.rd : on_a;
                sq[0] = sumsq_mixed<DT, VB>(x[j][0], sq[0]);
                sq[1] = sumsq_mixed<DT, VB>(x[j][1], sq[1]);
#pragma unroll
                for (int e = 0; e < N; e += C) {
                    float fa[C], fb[C];
                    Two yA[C / 2], yB[C / 2], cA[C / 2], cB[C / 2];
                    get<DT, VB, C>(fa, x[j][0], e);
                    get<DT, VB, C>(fb, x[j][1], e);
                    couple<C, inter>(cA, cB, fa, fb);
                    get<DT, VB, C>(fa, y[j][0], e);
                    get<DT, VB, C>(fb, y[j][1], e);
                    couple<C, inter>(yA, yB, fa, fb);
#pragma unroll
                    for (int i = 0; i < C / 2; ++i) {
                        const int m = e / 2 + i;
                        const Which on = rotated<C, inter>(i, on_a, on_b);
                        const Two c = cc[j][m], s = ss[j][m];
                        xA[j][m] = cA[i];
                        xB[j][m] = cB[i];
                        dA[j][m] = fma2(yA[i], c, pick(yB[i], on) * s);
                        dB[j][m] = fma2(yB[i], c, -(pick(yA[i], on) * s));
                        dotA = fma2(dA[j][m] * gA[j][m], cA[i], dotA);
                        dotB = fma2(dB[j][m] * gB[j][m], cB[i], dotB);
                    }
                }
            }
            float d0, d1;
            untwo(dotA + dotB, d0, d1);
            float sum = sq[0] + sq[1], dot = d0 + d1;
#pragma unroll
            for (int off = TPR / 2; off > 0; off >>= 1) {
                sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);
                dot += __shfl_xor_sync(0xFFFFFFFFu, dot, off);
            }
            // A group without a head keeps finite numbers: its zeros are summed.
            if (!live)
                sum = 1.f;
            float r = rsqrtf(fmaf(sum, inv_n, a.eps)), k = 1.f;
            const bool redo = bwd_rescales<DT>(sum, a.eps);
            const bool rare = kRangeGuard<DT> && __any_sync(0xFFFFFFFFu, redo);
            if (rare) {
                k = redo ? bwd_rescale_k(sum, a.eps) : 1.f;
                Two s2 = two(0.f, 0.f), t2 = s2;
#pragma unroll
                for (int j = 0; j < NP; ++j)
#pragma unroll
                    for (int m = 0; m < N / 2; ++m) {
                        xA[j][m] = xA[j][m] * k;
                        xB[j][m] = xB[j][m] * k;
                        s2 = fma2(xA[j][m], xA[j][m], fma2(xB[j][m], xB[j][m], s2));
                        t2 = fma2(dA[j][m] * gA[j][m], xA[j][m], t2);
                        t2 = fma2(dB[j][m] * gB[j][m], xB[j][m], t2);
                    }
                float s0, s1;
                untwo(s2, s0, s1);
                untwo(t2, d0, d1);
                dot = group_allreduce<TPR>(d0 + d1);
                s0 = group_allreduce<TPR>(s0 + s1);
                r = rsqrtf(fmaf(live ? s0 : 1.f, inv_n, (a.eps * k) * k));
            }
            // xh = x r, dw += du xh, dx = r (du g - xh m), m = r sum(du g x) / n
            const float m = r * (dot * inv_n);
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                Vec<VB> oa, ox;
#pragma unroll
                for (int e = 0; e < N; e += C) {
                    float fa[C], fb[C];
                    Two A[C / 2], B[C / 2];
#pragma unroll
                    for (int i = 0; i < C / 2; ++i) {
                        const int v = e / 2 + i;
                        const Two hA = xA[j][v] * r, hB = xB[j][v] * r;
                        accA[j][v] = fma2(dA[j][v], hA, accA[j][v]);
                        accB[j][v] = fma2(dB[j][v], hB, accB[j][v]);
                        A[i] = fma2(hA, -m, dA[j][v] * gA[j][v]) * r;
                        B[i] = fma2(hB, -m, dB[j][v] * gB[j][v]) * r;
                    }
                    uncouple<C, inter>(fa, fb, A, B);
                    if (rare) {
#pragma unroll
                        for (int i = 0; i < C; ++i) {
                            fa[i] *= k;
                            fb[i] *= k;
                        }
                    }
                    put<DT, VB, C>(oa, e, fa);
                    put<DT, VB, C>(ox, e, fb);
                }
                if (live && t + j * TPR < slots) {
                    st_head(po + va[j] * VB, oa);
                    st_head(po + vb[j] * VB, ox);
                }
            }
        }
        if constexpr (S == 1)
            ask_next(0);
        po += HS * ohs;
        fresh = ++step == steps;
        if (fresh) {
            step = 0;
            ++unit;
            po = ob + token(unit) * ots + own * ohs;
        }
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
            Two A[C / 2], B[C / 2];
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
    if (!multiple(a.head_dim, 2 * n) || !multiple(a.rope.rd, a.rope.interleaved ? n : 2 * n) ||
        a.head_dim / (2 * n) > kMostSlots ||
        !aligned(a.rope.cs, std::min<int64_t>(16, 4 * n)) || !aligned(a.qw, vb) ||
        !aligned(a.kw, vb))
        return false;
    for (const HeadsView *v : {&a.qdy, &a.kdy, &a.q, &a.k, &a.dq, &a.dk})
        if (v->p && !view_aligned(*v, es, vb))
            return false;
    return true;
}

template <int DT, int VB, int TPR, int NP, int MODE, bool BY_TOKEN = false>
cudaError_t launch_vec(const RopeBwdArgs &a, BlockSplit *split)
{
    constexpr int G = 32 / TPR, HS = BY_TOKEN ? 1 : G, kWarps = kBwdThreads / 32;
    const int64_t most = rope_bwd_max_blocks(a.sm_count) - 2; // blocks on all SMs
    const int64_t units = BY_TOKEN ? (a.tokens + G - 1) / G : a.tokens;
    const int64_t qs = (a.q_heads + HS - 1) / HS, ks = (a.k_heads + HS - 1) / HS;
    auto blocks = [&](int64_t steps) { // a step a warp at least
        const int64_t want = (units * steps + kWarps - 1) / kWarps;
        const int64_t share = (most * steps + (qs + ks) / 2) / (qs + ks);
        return steps ? static_cast<int>(std::max<int64_t>(1, std::min(want, share))) : 0;
    };
    *split = {blocks(qs), blocks(ks)};
    return launch_kernel(rope_bwd_kernel<DT, VB, TPR, NP, MODE, BY_TOKEN>, split->q + split->k,
                         kBwdThreads, 0, a.base, a, *split);
}

// By tokens, where a third of the lanes would have no head (bf16, by heads and by
// tokens: 14875 tokens of 3 + 1 heads of 80 21.8 and 15.2 us; 16384 of 1 + 1 of 128
// 22.6 and 11.0, of 4 + 1 of 128 25.3 and 20.3, of 12 + 4 of 64 33.4 and 23.5; but
// 32 + 8 of 128, where no lane is idle, 86.8 by heads, whose warp shares the angles).
template <int DT, int TPR, int MODE>
cudaError_t launch_groups(const RopeBwdArgs &a, BlockSplit *split)
{
    constexpr int G = 32 / TPR;
    const int64_t qs = (a.q_heads + G - 1) / G, ks = (a.k_heads + G - 1) / G;
    if (2 * G * (qs + ks) >= 3 * (int64_t(a.q_heads) + a.k_heads) && a.tokens >= G)
        return launch_vec<DT, 16, TPR, 1, MODE, true>(a, split);
    return launch_vec<DT, 16, TPR, 1, MODE>(a, split);
}

template <int DT, int VB, int MODE> cudaError_t launch_lanes(const RopeBwdArgs &a, BlockSplit *split)
{
    const int slots = a.head_dim / (2 * kVpe<DT, VB>);
    if constexpr (VB == 16) {
        if (slots <= 4)
            return launch_groups<DT, 4, MODE>(a, split);
        if (slots <= 8)
            return launch_groups<DT, 8, MODE>(a, split);
        if (slots <= 16)
            return launch_groups<DT, 16, MODE>(a, split);
    } else if (slots <= 16) {
        return launch_vec<DT, VB, 16, 1, MODE>(a, split);
    }
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
    const int64_t heads = int64_t(a.q_heads) + a.k_heads;
    const int64_t most = rope_bwd_max_blocks(a.sm_count) - 2;
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
                         a.dkw ? ColSum{a.part + split.q * D, a.dkw, split.k, D, D} : ColSum{},
                         a.base);
}

} // namespace

cudaError_t launch_rope_bwd(const RopeBwdArgs &a, int dtype)
{
    return dtype == RMSNORM_F32    ? launch<RMSNORM_F32>(a)
           : dtype == RMSNORM_BF16 ? launch<RMSNORM_BF16>(a)
                                   : launch<RMSNORM_F16>(a);
}

} // namespace rmsnorm
