// rope.cu -- per-head QK norm and position rotation in one pass, and the same
// with keys and values appended to a paged cache: the scalar body, and which
// body takes a call.
//
//   u[d] = (x[d] * r) * (w[d] + bias),  r = rsqrt(mean x^2 + eps)
//   y_a = u_a cos - u_b sin,  y_b = u_b cos + u_a sin   for each rotated pair
//
// Every element is read once and written once, so memory bounds it.
#include <algorithm>

#include "rope.cuh"

namespace rmsnorm {
namespace {

// Where a head's result goes: a tensor of the element type, or the cache, in
// the element type or as E4M3 codes of value * inv (nearest-even, saturating).
template <int DT>
__device__ inline void store_out(char *dst, int64_t i, float v, bool code, float inv)
{
    if (code)
        reinterpret_cast<uint8_t *>(dst)[i] = static_cast<uint8_t>(e4m3_code(v * inv));
    else
        Elem<DT>::store1(dst, i, v);
}

// Any alignment and head size: a warp per head of a token, scalar accesses.
// Heads of a token: q, then k, then (appending) v.
template <int DT>
__global__ void __launch_bounds__(256) rope_scalar_kernel(const RopeArgs a)
{
    using E = Elem<DT>;
    pdl_begin();
    const int lane = threadIdx.x & 31;
    const int warps = blockDim.x >> 5;
    const bool append = a.slots != nullptr;
    const int heads = a.q_heads + a.k_heads * (append ? 2 : 1);
    const int64_t total = a.tokens * heads;
    const int D = a.head_dim, rd = a.rope.rd, half = rd / 2;
    for (int64_t item = static_cast<int64_t>(blockIdx.x) * warps + (threadIdx.x >> 5);
         item < total; item += static_cast<int64_t>(gridDim.x) * warps) {
        const int64_t tok = item / heads;
        int h = static_cast<int>(item - tok * heads);
        int64_t slot = 0;
        if (append) {
            slot = a.slots[tok];
            if (slot < 0)
                continue; // padding
        }
        const float *cs;
        if (!rope_row(a.rope, tok, cs) || (append && slot >= a.num_slots)) {
            if (lane == 0 && h == 0)
                record_bad_index(a.base.status);
            continue;
        }
        const bool isq = h < a.q_heads;
        const bool isv = !isq && h - a.q_heads >= a.k_heads;
        if (!isq)
            h -= a.q_heads + (isv ? a.k_heads : 0);
        const HeadsView &in = isq ? a.q : isv ? a.v : a.k;
        const char *x = in.p + (tok * in.ts + h * in.hs) * E::kSize;
        char *y;
        bool code = false;
        float inv = 1.f;
        if (isq || !append) {
            const HeadsView &o = isq ? a.qo : a.ko;
            y = o.p + (tok * o.ts + h * o.hs) * E::kSize;
        } else {
            const int64_t page = slot / a.page_size;
            code = a.e4m3 != 0;
            inv = isv ? a.v_inv : a.k_inv;
            y = (isv ? a.vc : a.kc) +
                (page * a.page_stride + (slot - page * a.page_size) * a.slot_stride +
                 h * a.cache_hs) * (code ? 1 : E::kSize);
        }
        if (isv) {
            for (int d = lane; d < D; d += 32)
                store_out<DT>(y, d, E::widen1(x, d), code, inv);
            continue;
        }
        const void *w = isq ? a.qw : a.kw;
        RowScale f = {1.f, 1.f};
        if (w) {
            auto sum = [&](float k) {
                float s = 0.f;
                for (int d = lane; d < D; d += 32) {
                    const float v = E::widen1(x, d) * k;
                    s = fmaf(v, v, s);
                }
                return group_allreduce<32>(s);
            };
            f = row_scale<DT>(sum(1.f), static_cast<float>(D), a.eps, sum);
        }
        auto u = [&](int d) {
            const float v = E::widen1(x, d);
            return w ? (v * f.pre * f.r) * (E::widen1(w, d) + a.bias) : v;
        };
        for (int i = lane; i < half; i += 32) {
            const int da = a.rope.interleaved ? 2 * i : i;
            const int db = a.rope.interleaved ? 2 * i + 1 : i + half;
            const float ua = u(da), ub = u(db), c = cs[i], s = cs[half + i];
            store_out<DT>(y, da, fmaf(ua, c, -(ub * s)), code, inv);
            store_out<DT>(y, db, fmaf(ub, c, ua * s), code, inv);
        }
        for (int d = rd + lane; d < D; d += 32)
            store_out<DT>(y, d, u(d), code, inv);
    }
}

template <int DT> cudaError_t launch_scalar(const RopeArgs &a)
{
    const int64_t items = a.tokens * (a.q_heads + a.k_heads * (a.slots ? 2 : 1));
    const int64_t grid = std::min<int64_t>((items + 7) / 8, 1 << 30);
    return launch_kernel(rope_scalar_kernel<DT>, static_cast<int>(grid), 256, 0, a.base, a);
}

} // namespace

cudaError_t launch_rope(const RopeArgs &a, int dtype)
{
    const auto vec = dtype == RMSNORM_F32    ? launch_rope_vec_f32
                     : dtype == RMSNORM_BF16 ? launch_rope_vec_bf16
                                             : launch_rope_vec_f16;
    bool taken = false;
    const cudaError_t err = vec(a, &taken);
    if (taken)
        return err;
    return dtype == RMSNORM_F32    ? launch_scalar<RMSNORM_F32>(a)
           : dtype == RMSNORM_BF16 ? launch_scalar<RMSNORM_BF16>(a)
                                   : launch_scalar<RMSNORM_F16>(a);
}

} // namespace rmsnorm
