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

// The gradient bodies that keep x in registers form sum(du g x) before r is
// known, so they trust the plain sum S in a narrower range: S <= 2^80, and
// S >= 2^-60 unless eps >= 2^-40 bounds r.  There no product of dy, g and x
// leaves fp32's range for dy g within 2^+-60.  Otherwise x is replaced by k x
// (k a power of two: exact but for elements below 2^-46 of the largest), eps
// by eps k^2, and dx is multiplied by k at the end.  k keeps both the new sum
// and eps k^2 finite: 2^-80 above; below, 2^100 where S < 2^-100 and
// eps < 2^-120 (then S k^2 < 2^100, eps k^2 < 2^80, and the smallest element's
// square is 2^-98), else 2^50 (S k^2 <= 2^40, eps k^2 < 2^60).
template <int DT> __device__ inline bool bwd_rescales(float S, float eps)
{
    return kRangeGuard<DT> && !(S <= 0x1p80f && (S >= 0x1p-60f || eps >= 0x1p-40f));
}
__device__ inline float bwd_rescale_k(float S, float eps)
{
    return S > 0x1p80f ? 0x1p-80f : S < 0x1p-100f && eps < 0x1p-120f ? 0x1p100f : 0x1p50f;
}
// x <- k x in the element type.
template <int DT, int VB> __device__ inline void scale_by(Vec<VB> &v, float k)
{
#pragma unroll
    for (int i = 0; i < Vec<VB>::kWords; ++i) {
        float a, b = 0.f;
        Elem<DT>::widen(v.w[i], a, b);
        v.w[i] = Elem<DT>::narrow(a * k, b * k);
    }
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

// The pairing of the rotated elements, compiled apart: halves over the whole
// head, halves over a part of it, neighbours (over any part).
enum { kHalvesFull = 0, kHalves = 1, kInterleaved = 2 };

// ---- couples

// Two fp32 values in one register pair, worked on by the packed instructions
// (two IEEE operations each).
struct Two {
    uint64_t v;
};
__device__ inline Two two(float a, float b) { return {f2(a, b)}; }
__device__ inline void untwo(Two p, float &a, float &b) { f2split(p.v, a, b); }
__device__ inline Two operator*(Two p, Two q) { return {mul2(p.v, q.v)}; }
__device__ inline Two operator*(Two p, float q) { return {mul2(p.v, f2(q, q))}; }
__device__ inline Two operator+(Two p, Two q) { return {add2(p.v, q.v)}; }
__device__ inline Two operator+(Two p, float q) { return {add2(p.v, f2(q, q))}; }
__device__ inline Two operator-(Two p) { return {p.v ^ 0x8000000080000000ull}; }
__device__ inline Two fma2(Two p, Two q, Two c)
{
    Two r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(p.v), "l"(q.v), "l"(c.v));
    return r;
}
__device__ inline Two fma2(Two p, float q, Two c) { return fma2(p, two(q, q), c); }
// Which of the two are rotated: the others are 0 (pick), or 1 in place of 0
// (or_one).
struct Which {
    uint64_t mask;
};
__device__ inline Two pick(Two p, Which w) { return {p.v & w.mask}; }
__device__ inline Two or_one(Two p, Which w) { return {p.v | (~w.mask & f2(1.f, 1.f))}; }

// Loads at their place (volatile: they are not moved up into registers that
// wait): C = 2 or 4 floats, C elements of a weight widened.
template <int C> __device__ inline void ld_floats(float (&f)[C], const float *p)
{
    if constexpr (C == 4)
        asm volatile("ld.global.nc.v4.f32 {%0,%1,%2,%3}, [%4];"
                     : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3])
                     : "l"(p));
    else if constexpr (C == 2)
        asm volatile("ld.global.nc.v2.f32 {%0,%1}, [%2];" : "=f"(f[0]), "=f"(f[1]) : "l"(p));
    else
        asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(f[0]) : "l"(p));
}
template <int DT, int C> __device__ inline void ld_weights(float (&f)[C], const char *w)
{
    if constexpr (Elem<DT>::kPerWord == 1) {
        ld_floats(f, reinterpret_cast<const float *>(w));
    } else {
        Vec<2 * C> v;
        if constexpr (C == 4)
            asm volatile("ld.global.nc.v2.u32 {%0,%1}, [%2];"
                         : "=r"(v.w[0]), "=r"(v.w[1])
                         : "l"(w));
        else
            asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(v.w[0]) : "l"(w));
        widen_vec<DT, 2 * C>(f, v);
    }
}

// Elements e .. e + C of a slot's two vectors (C = 2 or 4), or of their
// weights, as couples (A_i, B_i) of which A_i is to be rotated with B_i:
// halves: A from the first vector and B from the second; neighbours: A the
// even elements and B the odd ones.
template <int C, bool INTER>
__device__ inline void couple(Two (&A)[C / 2], Two (&B)[C / 2], const float (&a)[C],
                              const float (&b)[C])
{
    if constexpr (!INTER) {
#pragma unroll
        for (int i = 0; i < C / 2; ++i) {
            A[i] = two(a[2 * i], a[2 * i + 1]);
            B[i] = two(b[2 * i], b[2 * i + 1]);
        }
    } else if constexpr (C == 4) {
        A[0] = two(a[0], a[2]), B[0] = two(a[1], a[3]);
        A[1] = two(b[0], b[2]), B[1] = two(b[1], b[3]);
    } else {
        A[0] = two(a[0], b[0]), B[0] = two(a[1], b[1]);
    }
}
template <int C, bool INTER>
__device__ inline void uncouple(float (&a)[C], float (&b)[C], const Two (&A)[C / 2],
                                const Two (&B)[C / 2])
{
    if constexpr (!INTER) {
#pragma unroll
        for (int i = 0; i < C / 2; ++i) {
            untwo(A[i], a[2 * i], a[2 * i + 1]);
            untwo(B[i], b[2 * i], b[2 * i + 1]);
        }
    } else if constexpr (C == 4) {
        untwo(A[0], a[0], a[2]), untwo(B[0], a[1], a[3]);
        untwo(A[1], b[0], b[2]), untwo(B[1], b[1], b[3]);
    } else {
        untwo(A[0], a[0], b[0]), untwo(B[0], a[1], b[1]);
    }
}
// The cosines (or sines) of the couples: halves from pa + e, neighbours from
// pa + e / 2 for the first vector and pb + e / 2 for the second.
template <int C, bool INTER>
__device__ inline void ld_couples(Two (&c)[C / 2], const float *pa, const float *pb, int e,
                                  bool on_a, bool on_b)
{
    if constexpr (!INTER) {
        float f[C] = {};
        if (on_a)
            ld_floats(f, pa + e);
#pragma unroll
        for (int i = 0; i < C / 2; ++i)
            c[i] = two(f[2 * i], f[2 * i + 1]);
    } else {
        float f0[C / 2] = {}, f1[C / 2] = {};
        if (on_a)
            ld_floats(f0, pa + e / 2);
        if (on_b)
            ld_floats(f1, pb + e / 2);
        if constexpr (C == 4)
            c[0] = two(f0[0], f0[1]), c[1] = two(f1[0], f1[1]);
        else
            c[0] = two(f0[0], f1[0]);
    }
}
// Which of couple i's elements are rotated.
template <int C, bool INTER>
__device__ inline Which rotated(int i, bool on_a, bool on_b)
{
    if constexpr (!INTER)
        return {on_a ? ~0ull : 0ull};
    else if constexpr (C == 4)
        return {(i == 0 ? on_a : on_b) ? ~0ull : 0ull};
    else
        return {(on_a ? 0xFFFFFFFFull : 0ull) | (on_b ? 0xFFFFFFFFull << 32 : 0ull)};
}

// Elements e .. e + C of a vector.
template <int DT, int VB, int C>
__device__ inline void get(float (&f)[C], const Vec<VB> &v, int e)
{
#pragma unroll
    for (int i = 0; i < C / 2; ++i) {
        if constexpr (Elem<DT>::kPerWord == 2) {
            Elem<DT>::widen(v.w[e / 2 + i], f[2 * i], f[2 * i + 1]);
        } else {
            f[2 * i] = __uint_as_float(v.w[e + 2 * i]);
            f[2 * i + 1] = __uint_as_float(v.w[e + 2 * i + 1]);
        }
    }
}
// Elements e .. e + C back in the element type.
template <int DT, int VB, int C>
__device__ inline void put(Vec<VB> &v, int e, const float (&f)[C])
{
#pragma unroll
    for (int i = 0; i < C / 2; ++i) {
        if constexpr (Elem<DT>::kPerWord == 2) {
            v.w[e / 2 + i] = Elem<DT>::narrow(f[2 * i], f[2 * i + 1]);
        } else {
            v.w[e + 2 * i] = __float_as_uint(f[2 * i]);
            v.w[e + 2 * i + 1] = __float_as_uint(f[2 * i + 1]);
        }
    }
}

// ---- a lane's own ring of copies

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

// (16-byte vectors only: what no ring copy brings)
__device__ inline void st_ring(uint32_t p, const Vec<16> &v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(p), "r"(v.w[0]), "r"(v.w[1]),
                 "r"(v.w[2]), "r"(v.w[3])
                 : "memory");
}

// ---- host: alignment of a call's tensors

inline bool multiple(int64_t v, int64_t of) { return v % of == 0; }
inline bool aligned(const void *p, int64_t to)
{
    return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(to) == 0;
}
inline bool view_aligned(const HeadsView &v, int64_t es, int64_t to)
{
    return aligned(v.p, to) && multiple(v.ts * es, to) && multiple(v.hs * es, to);
}

} // namespace rmsnorm
