// rms_bwd.cu -- the gradient of the row RMSNorm.
//
//   xh = x r,  g = w + bias,  r = rsqrt(mean x^2 + eps)
//   dx = r (dy g - xh m),  m = sum(dy g xh) / hidden
//   dw = sum over rows of dy xh
//
// Two inputs read and one output written once: memory bounds it.
#include <algorithm>
#include <mutex>

#include "rope.cuh"

namespace rmsnorm {
namespace {

// ---- rows too long for the registers: statistics, columns, then dx.  Three
// passes, because such a row does not fit on chip and dx may overwrite dy or
// x, which the columns' sums still need (two where it does not).  2000 x 30000
// bf16 (360 MB, floor 53.9 us): 157 us; element by element, as odd rows are, 358.

struct RowStat {
    float r, pre, m;
};

// Sum over the block of one value for each thread, in a fixed order.
__device__ inline float block_sum(float s, float *part)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    s = group_allreduce<32>(s);
    __syncthreads();
    if (lane == 0)
        part[warp] = s;
    __syncthreads();
    return group_allreduce<32>(lane < warps ? part[lane] : 0.f);
}

// N elements from element j on: a vector, or one by itself.
template <int DT, int N> __device__ inline void ld_row(float (&f)[N], const char *p, int64_t j)
{
    if constexpr (N == 1) {
        f[0] = Elem<DT>::widen1(p, j);
    } else {
        Vec<16> v;
        ld_head(v, p + j * Elem<DT>::kSize);
        widen_vec<DT, 16>(f, v);
    }
}
template <int DT, int N> __device__ inline void st_row(char *p, int64_t j, const float (&f)[N])
{
    if constexpr (N == 1) {
        Elem<DT>::store1(p, j, f[0]);
    } else {
        Vec<16> v;
        narrow_vec<DT, 16>(v, f);
        st_head(p + j * Elem<DT>::kSize, v);
    }
}

// dx of one row.
template <int DT, int N>
__device__ inline void row_dx(const char *dy, const char *x, const char *w, char *dx, int64_t base,
                              int64_t hidden, float bias, const RowStat &f)
{
    for (int64_t j = threadIdx.x * N; j < hidden; j += blockDim.x * N) {
        float a[N], b[N], g[N];
        ld_row<DT>(a, x, base + j);
        ld_row<DT>(b, dy, base + j);
        ld_row<DT>(g, w, j);
#pragma unroll
        for (int i = 0; i < N; ++i)
            a[i] = fmaf(b[i], g[i] + bias, -(a[i] * f.pre * f.r * f.m)) * f.r * f.pre;
        st_row<DT>(dx, base + j, a);
    }
}

// A row's statistics and, where dx overwrites neither dy nor x (`with_dx`),
// dx, while the row is still in L2.
template <int DT, int N>
__global__ void __launch_bounds__(512)
rms_bwd_stats_kernel(const char *dy, const char *x, const char *w, char *dx, RowStat *stat,
                     int64_t rows, int64_t hidden, float bias, float eps, bool with_dx)
{
    __shared__ float part[32];
    pdl_begin();
    const float n = static_cast<float>(hidden);
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const int64_t base = row * hidden;
        auto sum = [&](float k) {
            float s = 0.f;
            for (int64_t j = threadIdx.x * N; j < hidden; j += blockDim.x * N) {
                float a[N];
                ld_row<DT>(a, x, base + j);
#pragma unroll
                for (int i = 0; i < N; ++i)
                    s = fmaf(a[i] * k, a[i] * k, s);
            }
            return block_sum(s, part);
        };
        const RowScale f = row_scale<DT>(sum(1.f), n, eps, sum);
        float m = 0.f;
        for (int64_t j = threadIdx.x * N; j < hidden; j += blockDim.x * N) {
            float a[N], b[N], g[N];
            ld_row<DT>(a, x, base + j);
            ld_row<DT>(b, dy, base + j);
            ld_row<DT>(g, w, j);
#pragma unroll
            for (int i = 0; i < N; ++i)
                m = fmaf(b[i] * (g[i] + bias), a[i] * f.pre * f.r, m);
        }
        m = block_sum(m, part) / n;
        const RowStat s = {f.r, f.pre, m};
        if (threadIdx.x == 0)
            stat[row] = s;
        if (with_dx)
            row_dx<DT, N>(dy, x, w, dx, base, hidden, bias, s);
    }
}

// Columns: block (column block, chunk of rows); a thread for N columns.
template <int DT, int N>
__global__ void __launch_bounds__(256)
rms_bwd_columns_kernel(const char *dy, const char *x, const RowStat *stat, float *part,
                       int64_t rows, int64_t hidden, int64_t col_blocks, int chunks)
{
    pdl_begin();
    const int64_t chunk = blockIdx.x / col_blocks;
    const int64_t col = ((blockIdx.x - chunk * col_blocks) * 256 + threadIdx.x) * N;
    if (col >= hidden)
        return;
    float s[N] = {};
    for (int64_t row = chunk; row < rows; row += chunks) {
        const RowStat f = stat[row];
        float a[N], b[N];
        ld_row<DT>(a, x, row * hidden + col);
        ld_row<DT>(b, dy, row * hidden + col);
#pragma unroll
        for (int i = 0; i < N; ++i)
            s[i] = fmaf(b[i], a[i] * f.pre * f.r, s[i]);
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        part[chunk * hidden + col + i] = s[i];
}

template <int DT, int N>
__global__ void __launch_bounds__(512)
rms_bwd_dx_kernel(const char *dy, const char *x, const char *w, char *dx, const RowStat *stat,
                  int64_t rows, int64_t hidden, float bias)
{
    pdl_begin();
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x)
        row_dx<DT, N>(dy, x, w, dx, row * hidden, hidden, bias, stat[row]);
}

// Chunks of rows whose columns are summed apart (n columns a thread).
int64_t generic_chunks(int64_t rows, int64_t hidden, int sm_count, int n)
{
    const int64_t col_blocks = (hidden + 256 * n - 1) / (256 * n);
    const int64_t want = std::max<int64_t>(1, 8 * int64_t(sm_count) / col_blocks);
    return std::max<int64_t>(1, std::min(want, rows));
}

size_t stat_bytes(int64_t rows)
{
    return (static_cast<size_t>(rows) * sizeof(RowStat) + 15) / 16 * 16;
}

template <int DT, int N> cudaError_t launch_generic(const RmsBwdArgs &a)
{
    RowStat *stat = static_cast<RowStat *>(a.ws);
    float *part = reinterpret_cast<float *>(static_cast<char *>(a.ws) + stat_bytes(a.rows));
    const char *dy = static_cast<const char *>(a.dy), *x = static_cast<const char *>(a.x);
    const char *w = static_cast<const char *>(a.w);
    char *dx = static_cast<char *>(a.dx);
    const int grid = static_cast<int>(std::min<int64_t>(a.rows, 1 << 30));
    const bool with_dx = dx != dy && dx != x;
    cudaError_t err = launch_kernel(rms_bwd_stats_kernel<DT, N>, grid, 512, 0, a.base, dy, x, w, dx,
                                    stat, a.rows, a.hidden, a.bias, a.eps, with_dx);
    if (err == cudaSuccess && a.dw) {
        const int64_t chunks = generic_chunks(a.rows, a.hidden, a.sm_count, N);
        const int64_t col_blocks = (a.hidden + 256 * N - 1) / (256 * N);
        err = launch_kernel(rms_bwd_columns_kernel<DT, N>, static_cast<int>(chunks * col_blocks),
                            256, 0, a.base, dy, x, stat, part, a.rows, a.hidden, col_blocks,
                            static_cast<int>(chunks));
        if (err == cudaSuccess)
            err = launch_colsum({part, a.dw, chunks, a.hidden, a.hidden}, {}, a.base);
    }
    if (err == cudaSuccess && !with_dx)
        err = launch_kernel(rms_bwd_dx_kernel<DT, N>, grid, 512, 0, a.base, dy, x, w, dx, stat,
                            a.rows, a.hidden, a.bias);
    return err;
}

// ---- rows in registers
//
// A group of warps works on a row at a time, every thread on the same
// columns of each of the group's rows, so that dw's sums stay in registers.
// With g = w + bias both sums of a row, x^2 and dy g x, are formed at once and
// meet in shared memory; dx = r (dy g - x r m), m = r sum(dy g x) / hidden.
//   VB = 16 or 4: vectors of so many bytes; each thread copies its own ahead into
//        a ring in shared memory (cp.async; only its own copies are waited for).
//   SHIFT: rows that are no whole 16-byte vectors, in tensors that begin on a
//        boundary.  Rows a multiple of N apart lie alike between the boundaries, so a
//        block takes such rows alone and a thread's columns stay its own; what a
//        row's first and last vector hold of its neighbours is taken as zeros (it
//        may change meanwhile, where dx overwrites) and not written.
//   VB = 0: single elements, for any row length and alignment.
//
// Memory bounds it.  Measured with launch_colsum (16384 x 4096 bf16, 403 MB, floor
// 60.3 us at the copy bandwidth): three passes 383.9 us; this 65.9 us (6.11 TB/s,
// 91 %), two blocks of 256 threads on an SM; a ring of two stages 74.9 us; x and
// dy read again from the ring instead of kept (92 registers for 120) 70.4 us; but
// 16384 x 5120, where ten warps of 120 registers leave room for one block, 103 us
// with them kept and 84.7 us (floor 75.3) without.  Capped to 112 registers for a
// third block of six warps: 34.6 us for 32.9 us (9001 x 2880 f16, floor 23.3).
// Rows that are no whole vectors, shifted: 9001 x 2881 40.1 us, element by element
// 73.1; 9001 x 2882 40.3 us, with 4-byte vectors 45.4; 4000 x 12001 71.1 us, in the
// three passes above 208.  The edges cost 7 us of the 40 (9001 x 2880: 32.9).

// Ring stages: as many as leave an SM its blocks (f32 vectors hold half as
// many values, so a row's take twice the room).
template <int DT, int EPT, int VB>
constexpr int kRowStages = VB == 0 ? 0 : Elem<DT>::kSize == 2 ? 3 : EPT <= 16 ? 2 : 1;

// The first `bytes` of 16, the others as zeros.
__device__ inline void cp_async_part(uint32_t to, const char *from, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes)
                 : "memory");
}

template <int N> __device__ inline void zero_first(float (&f)[N], int n)
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        f[i] = i < n ? 0.f : f[i];
}

struct RowGroups {
    int warps;  // of a group
    int groups; // of a block
};

template <int DT, int EPT, int VB, bool KEEP, bool SHIFT>
__global__ void __launch_bounds__(512, 1)
rms_bwd_rows_kernel(const char *dy, const char *x, const char *w, char *dx, float *part,
                    int64_t rows, int32_t hidden, float bias, float eps, RowGroups rg)
{
    using E = Elem<DT>;
    constexpr bool VEC = VB > 0;
    constexpr int N = VEC ? VB / E::kSize : 1; // elements of an access
    constexpr int NV = EPT / N;
    constexpr int S = kRowStages<DT, EPT, VB>;
    constexpr int kAhead = S > 1 ? S - 1 : 1;
    constexpr bool kKeep = KEEP;
    static_assert(KEEP || VEC, "single elements are always kept");
    extern __shared__ __align__(16) char ring[];
    __shared__ float2 sums[2][16];
    pdl_begin();
    const int lane = threadIdx.x & 31;
    const int threads = rg.warps * 32; // of a group
    const int group = threadIdx.x / threads, t = threadIdx.x - group * threads;
    const int warp = t >> 5;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * rg.groups;
    const int64_t row0 = SHIFT ? blockIdx.x + static_cast<int64_t>(gridDim.x) * group
                               : static_cast<int64_t>(blockIdx.x) * rg.groups + group;
    // SHIFT: elements between a vector's boundary and the row, the same for all
    // rows of the block; column c lies at place c + shift of the vectors.
    const int shift = SHIFT ? static_cast<int>(blockIdx.x * static_cast<uint64_t>(hidden) % N) : 0;
    const int end = hidden + shift, nvec = SHIFT ? (end + N - 1) / N : hidden / N;
    const int64_t row_bytes = static_cast<int64_t>(hidden) * E::kSize;
    const float inv_n = 1.f / static_cast<float>(hidden);

    auto barrier = [&] { // of the group
        asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(threads) : "memory");
    };
    // Sums of two values over the group, in a fixed order.
    int turn = 0;
    auto group_sums = [&](float &a, float &b) {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            a += __shfl_xor_sync(0xFFFFFFFFu, a, off);
            b += __shfl_xor_sync(0xFFFFFFFFu, b, off);
        }
        if (rg.warps == 1)
            return;
        // Two sets in turn: a set is written again after a barrier that all
        // have reached with the set read.
        float2 *mine = &sums[turn][group * rg.warps];
        turn ^= 1;
        if (lane == 0)
            mine[warp] = make_float2(a, b);
        barrier();
        const int from = lane & 15;
        const float2 v = from < rg.warps ? mine[from] : make_float2(0.f, 0.f);
        a = v.x, b = v.y;
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) {
            a += __shfl_xor_sync(0xFFFFFFFFu, a, off);
            b += __shfl_xor_sync(0xFFFFFFFFu, b, off);
        }
    };

    const uint32_t my = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) +
                        threadIdx.x * VB;
    const uint32_t step = blockDim.x * VB; // bytes between a thread's vectors
    // g and dw's sums.
    Two acc[EPT / 2], g2[kKeep ? EPT / 2 : 1];
#pragma unroll
    for (int i = 0; i < EPT / 2; ++i)
        acc[i] = two(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int v = t + j * threads;
        if constexpr (VEC) {
            Vec<VB> u;
            vzero(u);
            if constexpr (SHIFT) {
                float f[N];
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int c = v * N + i - shift;
                    f[i] = c >= 0 && c < hidden ? E::widen1(w, c) : 0.f;
                }
                put<DT, VB, N>(u, 0, f);
            } else if (v < nvec) {
                ld_const(u, w + v * VB);
            }
            if constexpr (kKeep) {
                float f[N];
                get<DT, VB, N>(f, u, 0);
#pragma unroll
                for (int i = 0; i < N; i += 2)
                    g2[(j * N + i) / 2] = two(f[i], f[i + 1]) + bias;
            } else {
                st_ring(my + (S * 2 * NV + j) * step, u);
            }
        } else if (j % 2 == 0) {
            g2[j / 2] = two(v < nvec ? E::widen1(w, v) + bias : 0.f,
                            v + threads < nvec ? E::widen1(w, v + threads) + bias : 0.f);
        }
    }

    int64_t next = row0;
    auto ask_next = [&](int stage) {
        if constexpr (VEC) {
            if (next < rows) {
                const int64_t at = next * row_bytes - shift * E::kSize;
                const char *px = x + at, *py = dy + at;
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const int v = t + j * threads;
                    if (v < nvec) {
                        const uint32_t p = my + (stage * 2 * NV + 2 * j) * step;
                        if constexpr (SHIFT) { // nothing behind the row's end
                            const int bytes = min(VB, (end - v * N) * E::kSize);
                            cp_async_part(p, px + v * VB, bytes);
                            cp_async_part(p + step, py + v * VB, bytes);
                        } else {
                            cp_async<VB>(p, px + v * VB);
                            cp_async<VB>(p + step, py + v * VB);
                        }
                    }
                }
            }
            next += stride;
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    };
#pragma unroll
    for (int s = 0; s < kAhead; ++s)
        ask_next(s);
    int stage = 0;
    // Of this thread's first vector, the elements of the row before: taken as zeros.
    const int before = SHIFT && t == 0 ? shift : 0;
    for (int64_t row = row0; row < rows; row += stride) {
        const uint32_t here = my + stage * 2 * NV * step;
        Two x2[kKeep ? EPT / 2 : 1], y2[kKeep ? EPT / 2 : 1];
        if constexpr (VEC) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
            if constexpr (S > 1) // into the stage of the row before, whose values are used
                ask_next(stage == 0 ? S - 1 : stage - 1);
            stage = stage + 1 >= S ? 0 : stage + 1;
        } else {
            const char *px = x + row * row_bytes, *py = dy + row * row_bytes;
#pragma unroll
            for (int i = 0; i < EPT; i += 2) {
                const int c0 = t + i * threads, c1 = c0 + threads;
                x2[i / 2] = two(c0 < hidden ? E::widen1(px, c0) : 0.f,
                                c1 < hidden ? E::widen1(px, c1) : 0.f);
                y2[i / 2] = two(c0 < hidden ? E::widen1(py, c0) : 0.f,
                                c1 < hidden ? E::widen1(py, c1) : 0.f);
            }
        }
        // Vector j's values, from registers or widened (again): x, dy and g.
        auto values = [&](int j, Two (&xv)[N > 1 ? N / 2 : 1], Two (&yv)[N > 1 ? N / 2 : 1],
                          Two (&gv)[N > 1 ? N / 2 : 1], bool first) {
            if constexpr (!VEC) {
                xv[0] = x2[j], yv[0] = y2[j], gv[0] = g2[j];
            } else {
                const bool in = t + j * threads < nvec;
                if (first || !kKeep) {
                    Vec<VB> v;
                    float f[N];
                    vzero(v);
                    if (in)
                        ld_ring(v, here + 2 * j * step);
                    get<DT, VB, N>(f, v, 0);
                    if (SHIFT && j == 0)
                        zero_first<N>(f, before);
#pragma unroll
                    for (int i = 0; i < N / 2; ++i)
                        xv[i] = two(f[2 * i], f[2 * i + 1]);
                    vzero(v);
                    if (in)
                        ld_ring(v, here + (2 * j + 1) * step);
                    get<DT, VB, N>(f, v, 0);
                    if (SHIFT && j == 0)
                        zero_first<N>(f, before);
#pragma unroll
                    for (int i = 0; i < N / 2; ++i)
                        yv[i] = two(f[2 * i], f[2 * i + 1]);
                }
                if constexpr (kKeep) {
#pragma unroll
                    for (int i = 0; i < N / 2; ++i) {
                        const int m = j * (N / 2) + i;
                        if (first)
                            x2[m] = xv[i], y2[m] = yv[i];
                        else
                            xv[i] = x2[m], yv[i] = y2[m];
                        gv[i] = g2[m];
                    }
                } else {
                    Vec<VB> v;
                    float f[N];
                    ld_ring(v, my + (S * 2 * NV + j) * step);
                    get<DT, VB, N>(f, v, 0);
#pragma unroll
                    for (int i = 0; i < N / 2; ++i)
                        gv[i] = two(f[2 * i], f[2 * i + 1]) + bias;
                }
            }
        };
        constexpr int kSteps = VEC ? NV : NV / 2, kHalf = N > 1 ? N / 2 : 1;
        float sum, dot, k = 1.f;
        {
            Two s2 = two(0.f, 0.f), t2 = s2, s3 = s2, t3 = s2;
#pragma unroll
            for (int j = 0; j < kSteps; ++j) {
                Two xv[kHalf], yv[kHalf], gv[kHalf];
                values(j, xv, yv, gv, true);
#pragma unroll
                for (int i = 0; i < kHalf; ++i) {
                    if ((i + j * kHalf) % 2 == 0) {
                        s2 = fma2(xv[i], xv[i], s2);
                        t2 = fma2(yv[i] * gv[i], xv[i], t2);
                    } else {
                        s3 = fma2(xv[i], xv[i], s3);
                        t3 = fma2(yv[i] * gv[i], xv[i], t3);
                    }
                }
            }
            float a0, a1, b0, b1;
            untwo(s2 + s3, a0, a1);
            untwo(t2 + t3, b0, b1);
            sum = a0 + a1;
            dot = b0 + b1;
        }
        group_sums(sum, dot);
        float r = rsqrtf(fmaf(sum, inv_n, eps));
        const bool rare = bwd_rescales<DT>(sum, eps); // the same for the group
        if (rare) {
            // Again from k x (rope.cuh).
            k = bwd_rescale_k(sum, eps);
            sum = dot = 0.f;
#pragma unroll
            for (int j = 0; j < kSteps; ++j) {
                Two xv[kHalf], yv[kHalf], gv[kHalf];
                values(j, xv, yv, gv, false);
#pragma unroll
                for (int i = 0; i < kHalf; ++i) {
                    const Two xk = xv[i] * k;
                    float a0, a1, b0, b1;
                    untwo(xk * xk, a0, a1);
                    untwo(yv[i] * gv[i] * xk, b0, b1);
                    sum += a0 + a1;
                    dot += b0 + b1;
                }
            }
            group_sums(sum, dot);
            r = rsqrtf(fmaf(sum, inv_n, (eps * k) * k));
        }
        // xh = x r, dw += dy xh
        const float m = r * (dot * inv_n);
        char *po = dx + row * row_bytes;
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
            Two xv[kHalf], yv[kHalf], gv[kHalf];
            values(j, xv, yv, gv, false);
            float f[2 * kHalf];
#pragma unroll
            for (int i = 0; i < kHalf; ++i) {
                const Two h = (rare ? xv[i] * k : xv[i]) * r;
                Two &a = acc[j * kHalf + i];
                a = fma2(yv[i], h, a);
                untwo(fma2(h, -m, yv[i] * gv[i]) * r, f[2 * i], f[2 * i + 1]);
            }
            if (rare) {
#pragma unroll
                for (int i = 0; i < 2 * kHalf; ++i)
                    f[i] *= k;
            }
            if constexpr (VEC) {
                const int v = t + j * threads;
                if (!SHIFT || (v * N >= shift && v * N + N <= end)) {
                    Vec<VB> o;
                    put<DT, VB, N>(o, 0, f);
                    if (SHIFT || v < nvec)
                        st_head(po - shift * E::kSize + v * VB, o);
                } else {
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const int c = v * N + i - shift;
                        if (c >= 0 && c < hidden)
                            E::store1(po, c, f[i]);
                    }
                }
            } else {
                const int c0 = t + 2 * j * threads, c1 = c0 + threads;
                if (c0 < hidden)
                    E::store1(po, c0, f[0]);
                if (c1 < hidden)
                    E::store1(po, c1, f[1]);
            }
        }
        if constexpr (VEC && S == 1) {
            ask_next(0);
        }
    }
    if (!part)
        return;
    if constexpr (VEC)
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    // The block's sums, over its groups in order: each group in turn adds
    // to shared memory (columns of a thread lie together).
    float *out = part + static_cast<int64_t>(blockIdx.x) * hidden;
    float4 *buf = reinterpret_cast<float4 *>(ring) + t; // [EPT / 4][threads]
    for (int q = 0; q < rg.groups; ++q) {
        if (SHIFT || rg.groups > 1)
            __syncthreads();
        if (group != q)
            continue;
#pragma unroll
        for (int i = 0; i < EPT / 4; ++i) {
            float4 v;
            untwo(acc[2 * i], v.x, v.y);
            untwo(acc[2 * i + 1], v.z, v.w);
            if (q > 0) {
                const float4 o = buf[i * threads];
                v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
            }
            if (SHIFT || q < rg.groups - 1) {
                buf[i * threads] = v;
                continue;
            }
            if constexpr (N >= 4) {
                const int c = (t + i * 4 / N * threads) * N + i * 4 % N;
                if (c < hidden)
                    *reinterpret_cast<float4 *>(out + c) = v;
            } else {
                const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int c = (t + (4 * i + e) / N * threads) * N + e % N;
                    if (c < hidden)
                        out[c] = f[e];
                }
            }
        }
    }
    if constexpr (SHIFT) {
        // From there in order of columns: a thread's own lie N floats apart, and with
        // single stores so far apart 419 x 15495 took 27.5 us for 23.9.
        __syncthreads();
        const float *all = reinterpret_cast<const float *>(ring);
#pragma unroll 1
        for (int j = 0; j < NV; ++j) {
            for (int i = threadIdx.x; i < threads * N; i += blockDim.x) {
                const int c = j * threads * N + i - shift, e = i % N;
                if (c >= 0 && c < hidden)
                    out[c] = all[((j * N + e) / 4 * threads + i / N) * 4 + e % 4];
            }
        }
    }
}

// The groups for rows of `accesses` accesses, nv of them a thread.
RowGroups row_groups(int64_t accesses, int nv)
{
    const int warps = static_cast<int>((accesses + 32 * nv - 1) / (32 * nv));
    return {warps, std::max(1, 8 / warps)};
}

// Blocks on an SM, a workspace row each: no more than 1024 threads (the bodies
// have 61 registers and more, 64 as they are given out).
int row_blocks(const RowGroups &rg) { return std::max(1, 32 / (rg.warps * rg.groups)); }

// Blocks of a kernel that an SM holds, with the kernel's shared memory raised
// to what it asks; remembered for a device and launch shape.
cudaError_t row_occupancy(const void *kernel, int threads, int smem, int *blocks)
{
    struct Entry {
        const void *kernel;
        int device, threads, smem, blocks;
    };
    constexpr int kMost = 256;
    static std::mutex mu;
    static Entry known[kMost];
    static int count = 0;
    int device = 0;
    cudaError_t err = cudaGetDevice(&device);
    if (err != cudaSuccess)
        return err;
    std::lock_guard<std::mutex> lk(mu);
    int most = smem; // the attribute only grows
    for (int i = 0; i < count; ++i) {
        const Entry &e = known[i];
        if (e.kernel != kernel || e.device != device)
            continue;
        if (e.threads == threads && e.smem == smem) {
            *blocks = e.blocks;
            return cudaSuccess;
        }
        most = std::max(most, e.smem);
    }
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (err == cudaSuccess)
        err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(blocks, kernel, threads, smem);
    if (err != cudaSuccess)
        return err;
    if (*blocks < 1)
        return cudaErrorInvalidConfiguration;
    if (count < kMost)
        known[count++] = {kernel, device, threads, smem, *blocks};
    return cudaSuccess;
}

// Vectors of n elements that a row may take when it starts anywhere in the first.
int64_t shifted_vectors(int64_t hidden, int n) { return (hidden + 2 * n - 2) / n; }

template <int DT, int EPT, int VB, bool KEEP, bool SHIFT = false>
cudaError_t launch_rows(const RmsBwdArgs &a)
{
    constexpr int N = VB ? VB / Elem<DT>::kSize : 1;
    constexpr int NV = EPT / N, S = kRowStages<DT, EPT, VB>;
    const RowGroups rg = row_groups(SHIFT ? shifted_vectors(a.hidden, N) : a.hidden / N, NV);
    const int threads = rg.warps * rg.groups * 32;
    // The ring (and g), and the sums of dw over the groups.
    const int smem = std::max((S * 2 + (KEEP ? 0 : 1)) * NV * VB * threads,
                              SHIFT || rg.groups > 1 ? rg.warps * 32 * EPT * 4 : 0);
    auto *kernel = rms_bwd_rows_kernel<DT, EPT, VB, KEEP, SHIFT>;
    int blocks_per_sm = 0;
    cudaError_t err = row_occupancy(reinterpret_cast<const void *>(kernel), threads, smem,
                                    &blocks_per_sm);
    if (err != cudaSuccess)
        return err;
    const int64_t want = (a.rows + rg.groups - 1) / rg.groups;
    const int64_t most = int64_t(std::min(blocks_per_sm, row_blocks(rg))) * a.sm_count;
    int64_t blocks = std::min(want, most);
    if (SHIFT) { // rows a grid apart start alike
        blocks = (blocks + N - 1) / N * N;
        blocks = std::min(blocks <= most ? blocks : blocks - N, a.rows);
    }
    const int grid = static_cast<int>(blocks);
    float *part = a.dw ? static_cast<float *>(a.ws) : nullptr;
    err = launch_kernel(kernel, grid, threads, smem, a.base, static_cast<const char *>(a.dy),
                        static_cast<const char *>(a.x), static_cast<const char *>(a.w),
                        static_cast<char *>(a.dx), part, a.rows, static_cast<int32_t>(a.hidden),
                        a.bias, a.eps, rg);
    if (err != cudaSuccess || !part)
        return err;
    return launch_colsum({part, a.dw, grid, a.hidden, a.hidden}, {}, a.base);
}

constexpr int64_t kMostRow = 512 * 32; // elements of a row in registers
constexpr int64_t kHeadRow = 256;      // of one that goes as a head

template <int DT> cudaError_t launch(const RmsBwdArgs &a)
{
    constexpr int es = Elem<DT>::kSize;
    auto fits = [&](int64_t to) {
        return multiple(a.hidden * es, to) && aligned(a.dy, to) && aligned(a.x, to) &&
               aligned(a.w, to) && aligned(a.dx, to);
    };
    // Short rows: as the heads of one token, several a warp (rope_bwd.cu).  65536
    // rows of 128: 13.8 us, 26.7 us with a warp a row; of 256: 21.2 us and 27.3 us;
    // 40000 of 384: 22.5 us and 21.2 us.
    if (a.hidden <= kHeadRow && a.rows <= (1 << 30) && fits(std::min<int64_t>(16, 2 * es)) &&
        multiple(a.hidden, 4)) {
        RopeBwdArgs h{};
        h.base = a.base;
        auto view = [&](const void *p) {
            return HeadsView{static_cast<char *>(const_cast<void *>(p)), a.rows * a.hidden,
                             a.hidden};
        };
        h.qdy = view(a.dy);
        h.q = view(a.x);
        h.dq = view(a.dx);
        h.qw = a.w;
        h.dqw = a.dw;
        h.part = a.dw ? static_cast<float *>(a.ws) : nullptr;
        h.tokens = 1;
        h.q_heads = static_cast<int32_t>(a.rows);
        h.head_dim = static_cast<int32_t>(a.hidden);
        h.bias = a.bias;
        h.eps = a.eps;
        h.sm_count = a.sm_count;
        return launch_rope_bwd(h, DT);
    }
    // Many rows that two warps would half fill: one warp a row (bf16 27063 x 576 24.6 us,
    // with two 29.0; 22130 x 723 29.1 us, with two 32.9; but 3151 x 723 11.6 us, with two
    // 10.3, and f32 22130 x 723 41.2 us, with two 37.7).
    [[maybe_unused]] auto one_warp = [&](int64_t n) {
        return n > 512 && n <= 24 * 32 && a.rows >= 64 * int64_t(a.sm_count);
    };
    if (fits(16)) {
        if constexpr (es == 2)
            if (one_warp(a.hidden))
                return launch_rows<DT, 24, 16, false>(a);
        // Ten warps a row: a second block on an SM fits without x and dy kept.
        if (a.hidden > 9 * 512 && a.hidden <= 10 * 512)
            return launch_rows<DT, 16, 16, false>(a);
        if (a.hidden <= 512 * 16)
            return launch_rows<DT, 16, 16, true>(a);
        if (a.hidden <= kMostRow)
            return launch_rows<DT, 32, 16, false>(a);
        return launch_generic<DT, 16 / es>(a);
    }
    // Vectors over the rows' boundaries, beyond rows of 128 (65536 rows of 129: 26.5 us,
    // 41.3 by single elements; of 65: 25.9 us and 17.8).
    if (a.hidden > 32 * 4 && aligned(a.dy, 16) && aligned(a.x, 16) && aligned(a.dx, 16) &&
        a.sm_count >= 16 / es) {
        const int64_t places = shifted_vectors(a.hidden, 16 / es) * (16 / es);
        if (places <= 32 * 8)
            return launch_rows<DT, 8, 16, true, true>(a);
        if constexpr (es == 2)
            if (one_warp(places))
                return launch_rows<DT, 24, 16, false, true>(a);
        if (places <= 512 * 16) // ten warps a row too: 16384 x 5001 122 us, not kept 136
            return launch_rows<DT, 16, 16, true, true>(a);
        if (places <= kMostRow)
            return launch_rows<DT, 32, 16, false, true>(a);
    }
    if constexpr (es == 2) {
        if (a.hidden <= 512 * 16 && fits(4))
            return a.hidden <= 32 * 4   ? launch_rows<DT, 4, 4, true>(a)
                   : a.hidden <= 32 * 8 ? launch_rows<DT, 8, 4, true>(a)
                                        : launch_rows<DT, 16, 4, true>(a);
    }
    return a.hidden <= 32 * 4     ? launch_rows<DT, 4, 0, true>(a)
           : a.hidden <= 32 * 8   ? launch_rows<DT, 8, 0, true>(a)
           : a.hidden <= 512 * 16 ? launch_rows<DT, 16, 0, true>(a)
                                  : launch_generic<DT, 1>(a);
}

} // namespace

// A row of partial sums for every block of any body that may run (the pointers
// decide which), or the three passes' statistics and chunks.
size_t rms_bwd_workspace(int64_t rows, int64_t hidden, int, int sm_count)
{
    const size_t row = static_cast<size_t>(hidden) * sizeof(float);
    size_t blocks = 0;
    for (int ept : {4, 8, 16, 24, 32})
        if (hidden <= 512 * ept && hidden <= kMostRow)
            for (int n : {1, 4, 8}) // single elements or whole vectors, or shifted vectors
                if (ept >= n)
                    blocks = std::max(blocks, static_cast<size_t>(row_blocks(row_groups(
                                                  shifted_vectors(hidden, n), ept / n))) * sm_count);
    if (hidden <= kHeadRow)
        blocks = std::max(blocks, static_cast<size_t>(rope_bwd_max_blocks(sm_count)));
    blocks = std::min(blocks, static_cast<size_t>(rows));
    const size_t passes = stat_bytes(rows) + std::max(generic_chunks(rows, hidden, sm_count, 1),
                                                              generic_chunks(rows, hidden, sm_count, 8)) * row;
    return hidden <= 512 * 16 ? blocks * row : std::max(blocks * row, passes);
}

cudaError_t launch_rms_bwd(const RmsBwdArgs &a, int dtype)
{
    return dtype == RMSNORM_F32    ? launch<RMSNORM_F32>(a)
           : dtype == RMSNORM_BF16 ? launch<RMSNORM_BF16>(a)
                                   : launch<RMSNORM_F16>(a);
}

} // namespace rmsnorm
