// rope.cuh -- what the head kernels with a position rotation share (rope.cu,
// rope_bwd.cu): a token's row of the angle table and the row factor of a head.
#pragma once

#include "rope_args.h"
#include "device_common.cuh"

namespace rmsnorm {

__device__ inline void record_bad_index(int *status)
{
    atomicCAS(status, 0, static_cast<int>(RMSNORM_ERR_BAD_INDEX));
}

// The token's row of the table (null without a rotation); false when its
// position lies outside the table.
__device__ inline bool rope_row(const RopeTable &t, int64_t token, const float *&row)
{
    row = nullptr;
    if (t.rd == 0)
        return true;
    const int64_t p = t.pos[token];
    if (p < 0 || p >= t.max_pos)
        return false;
    row = t.cs + p * t.rd;
    return true;
}

// The factor of a row held as x = (x * pre) * r: pre is 1 but where the range
// guard scales x up by 2^100 (device_common.cuh).  For the bodies that read a
// head or row again from memory; `resum(k)` returns the sum of (k x)^2.
struct RowScale {
    float r, pre;
};
template <int DT, typename Resum>
__device__ inline RowScale row_scale(float S, float n, float eps, Resum resum)
{
    RowScale f = {row_factor(S, n, eps), 1.f};
    if constexpr (kRangeGuard<DT>) {
        if (sum_needs_rescale(S, eps)) {
            const float k = rescale_k(S);
            const Factor g = rescaled_factor(resum(k), k, n, eps);
            f.r = g.r;
            f.pre = g.up ? 0x1p100f : 1.f;
        }
    }
    return f;
}

// ---- heads in vectors
//
// A head is cut into slots of two VB-byte vectors, so that a slot holds whole
// pairs: with halves, slot p of the rotated part holds vectors p and
// p + rd / 2 / VPE, and the slots behind it hold the others; with neighbours
// any two vectors do.  This asks that rd and head_dim are multiples of 2 * VPE.
// TPR lanes of a warp own a head; lane t has slots t, t + TPR, ... (NP of them).

template <int DT, int VB> constexpr int kVpe = VB / Elem<DT>::kSize;

__device__ inline void ld_stream8(Vec<8> &v, const void *p)
{
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];"
                 : "=r"(v.w[0]), "=r"(v.w[1])
                 : "l"(p));
}
template <int VB> __device__ inline void ld_head(Vec<VB> &v, const void *p)
{
    if constexpr (VB == 16)
        ld_stream<0>(v, p);
    else if constexpr (VB == 8)
        ld_stream8(v, p);
    else
        asm volatile("ld.global.L1::no_allocate.u32 %0, [%1];" : "=r"(v.w[0]) : "l"(p));
}
template <int VB> __device__ inline void ld_const(Vec<VB> &v, const void *p)
{
    if constexpr (VB == 16)
        ld_weight(v, p);
    else if constexpr (VB == 8)
        asm volatile("ld.global.nc.v2.u32 {%0,%1}, [%2];" : "=r"(v.w[0]), "=r"(v.w[1]) : "l"(p));
    else
        asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(v.w[0]) : "l"(p));
}
template <int VB> __device__ inline void st_head(void *p, const Vec<VB> &v)
{
    if constexpr (VB == 16)
        st_stream<0>(p, v);
    else if constexpr (VB == 8)
        asm volatile("st.global.L1::no_allocate.v2.u32 [%0], {%1,%2};" ::"l"(p), "r"(v.w[0]),
                     "r"(v.w[1])
                     : "memory");
    else
        asm volatile("st.global.L1::no_allocate.u32 [%0], %1;" ::"l"(p), "r"(v.w[0]) : "memory");
}
template <int VB> __device__ inline void vzero(Vec<VB> &v)
{
#pragma unroll
    for (int i = 0; i < Vec<VB>::kWords; ++i)
        v.w[i] = 0u;
}

// N = 2, 4 or 8 floats of the angle table.
template <int N> __device__ inline void ld_angles(float (&f)[N], const float *p)
{
    if constexpr (N >= 4) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 v = __ldg(reinterpret_cast<const float4 *>(p + i));
            f[i] = v.x, f[i + 1] = v.y, f[i + 2] = v.z, f[i + 3] = v.w;
        }
    } else {
        const float2 v = __ldg(reinterpret_cast<const float2 *>(p));
        f[0] = v.x, f[1] = v.y;
    }
}

template <int DT, int VB>
__device__ inline void widen_vec(float (&f)[kVpe<DT, VB>], const Vec<VB> &v)
{
#pragma unroll
    for (int k = 0; k < Vec<VB>::kWords; ++k) {
        if constexpr (Elem<DT>::kPerWord == 2)
            Elem<DT>::widen(v.w[k], f[2 * k], f[2 * k + 1]);
        else
            f[k] = __uint_as_float(v.w[k]);
    }
}
template <int DT, int VB>
__device__ inline void narrow_vec(Vec<VB> &v, const float (&f)[kVpe<DT, VB>])
{
#pragma unroll
    for (int k = 0; k < Vec<VB>::kWords; ++k) {
        if constexpr (Elem<DT>::kPerWord == 2)
            v.w[k] = Elem<DT>::narrow(f[2 * k], f[2 * k + 1]);
        else
            v.w[k] = __float_as_uint(f[k]);
    }
}

// Vectors of slot p: the slots' first vectors follow one another, and so do
// the second ones, so that a warp's loads are whole lines.
__device__ inline void slot_vectors(int p, int slots, int half_v, bool interleaved, int &va,
                                    int &vb)
{
    if (interleaved) {
        va = p;
        vb = p + slots;
    } else {
        const bool turned = p < half_v;
        va = turned ? p : p + half_v;
        vb = va + (turned ? half_v : slots - half_v);
    }
}

} // namespace rmsnorm
