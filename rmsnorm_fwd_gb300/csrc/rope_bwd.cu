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

// A workspace row per block: four blocks on every SM, and one more for each
// tensor's rounding.
int rope_bwd_max_blocks(int sm_count) { return 4 * sm_count + 2; }

namespace {

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

BlockSplit split_blocks(const RopeBwdArgs &a, int64_t per_block)
{
    const int64_t heads = int64_t(a.q_heads) + a.k_heads;
    auto want = [&](int64_t h) { return (a.tokens * h + per_block - 1) / per_block; };
    const int64_t most = 4 * a.sm_count;
    auto take = [&](int64_t h) {
        return h ? std::max<int64_t>(1, std::min(want(h), (most * h + heads - 1) / heads)) : 0;
    };
    return {static_cast<int>(take(a.q_heads)), static_cast<int>(take(a.k_heads))};
}

template <int DT> cudaError_t launch(const RopeBwdArgs &a)
{
    const BlockSplit split = split_blocks(a, 8);
    cudaError_t err = cudaSuccess;
    if (split.q + split.k > 0)
        err = launch_kernel(rope_bwd_scalar_kernel<DT>, split.q + split.k, 256,
                            8 * a.head_dim * 4, a.base, a, split);
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
