// rms_bwd.cu -- the gradient of the row RMSNorm.
//
//   xh = x r,  g = w + bias,  r = rsqrt(mean x^2 + eps)
//   dx = r (dy g - xh m),  m = sum(dy g xh) / hidden
//   dw = sum over rows of dy xh
//
// Two inputs read and one output written once: memory bounds it.
#include <algorithm>

#include "rope.cuh"

namespace rmsnorm {
namespace {

// ---- any row length and alignment: statistics, columns, then dx.  Three
// passes, because a long row does not fit on chip and dx may overwrite dy or
// x, which the columns' sums still need.

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

template <int DT>
__global__ void __launch_bounds__(512)
rms_bwd_stats_kernel(const void *dy, const void *x, const void *w, RowStat *stat, int64_t rows,
                     int64_t hidden, float bias, float eps)
{
    using E = Elem<DT>;
    __shared__ float part[32];
    pdl_begin();
    const float n = static_cast<float>(hidden);
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const int64_t base = row * hidden;
        auto sum = [&](float k) {
            float s = 0.f;
            for (int64_t j = threadIdx.x; j < hidden; j += blockDim.x) {
                const float v = E::widen1(x, base + j) * k;
                s = fmaf(v, v, s);
            }
            return block_sum(s, part);
        };
        const RowScale f = row_scale<DT>(sum(1.f), n, eps, sum);
        float m = 0.f;
        for (int64_t j = threadIdx.x; j < hidden; j += blockDim.x)
            m = fmaf(E::widen1(dy, base + j) * (E::widen1(w, j) + bias),
                     E::widen1(x, base + j) * f.pre * f.r, m);
        m = block_sum(m, part) / n;
        if (threadIdx.x == 0)
            stat[row] = {f.r, f.pre, m};
    }
}

// Columns: block (column block, chunk of rows); a thread per column.
template <int DT>
__global__ void __launch_bounds__(256)
rms_bwd_columns_kernel(const void *dy, const void *x, const RowStat *stat, float *part,
                       int64_t rows, int64_t hidden, int64_t col_blocks, int chunks)
{
    using E = Elem<DT>;
    pdl_begin();
    const int64_t chunk = blockIdx.x / col_blocks;
    const int64_t col = (blockIdx.x - chunk * col_blocks) * 256 + threadIdx.x;
    if (col >= hidden)
        return;
    float s = 0.f;
    for (int64_t row = chunk; row < rows; row += chunks) {
        const RowStat f = stat[row];
        s = fmaf(E::widen1(dy, row * hidden + col),
                 E::widen1(x, row * hidden + col) * f.pre * f.r, s);
    }
    part[chunk * hidden + col] = s;
}

template <int DT>
__global__ void __launch_bounds__(512)
rms_bwd_dx_kernel(const void *dy, const void *x, const void *w, void *dx, const RowStat *stat,
                  int64_t rows, int64_t hidden, float bias)
{
    using E = Elem<DT>;
    pdl_begin();
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const int64_t base = row * hidden;
        const RowStat f = stat[row];
        for (int64_t j = threadIdx.x; j < hidden; j += blockDim.x) {
            const float v = fmaf(E::widen1(dy, base + j), E::widen1(w, j) + bias,
                                 -(E::widen1(x, base + j) * f.pre * f.r * f.m));
            E::store1(dx, base + j, v * f.r * f.pre);
        }
    }
}

int64_t generic_chunks(int64_t rows, int64_t hidden, int sm_count)
{
    const int64_t col_blocks = (hidden + 255) / 256;
    const int64_t want = std::max<int64_t>(1, 8 * int64_t(sm_count) / col_blocks);
    return std::max<int64_t>(1, std::min(want, rows));
}

size_t stat_bytes(int64_t rows)
{
    return (static_cast<size_t>(rows) * sizeof(RowStat) + 15) / 16 * 16;
}

template <int DT> cudaError_t launch_generic(const RmsBwdArgs &a)
{
    RowStat *stat = static_cast<RowStat *>(a.ws);
    float *part = reinterpret_cast<float *>(static_cast<char *>(a.ws) + stat_bytes(a.rows));
    const int grid = static_cast<int>(std::min<int64_t>(a.rows, 1 << 30));
    cudaError_t err = launch_kernel(rms_bwd_stats_kernel<DT>, grid, 512, 0, a.base, a.dy, a.x, a.w,
                                    stat, a.rows, a.hidden, a.bias, a.eps);
    if (err == cudaSuccess && a.dw) {
        const int64_t chunks = generic_chunks(a.rows, a.hidden, a.sm_count);
        const int64_t col_blocks = (a.hidden + 255) / 256;
        err = launch_kernel(rms_bwd_columns_kernel<DT>, static_cast<int>(chunks * col_blocks), 256,
                            0, a.base, a.dy, a.x, stat, part, a.rows, a.hidden, col_blocks,
                            static_cast<int>(chunks));
        if (err == cudaSuccess)
            err = launch_colsum({part, a.dw, chunks, a.hidden, a.hidden}, {}, a.base);
    }
    if (err == cudaSuccess)
        err = launch_kernel(rms_bwd_dx_kernel<DT>, grid, 512, 0, a.base, a.dy, a.x, a.w, a.dx, stat,
                            a.rows, a.hidden, a.bias);
    return err;
}

} // namespace

size_t rms_bwd_workspace(int64_t rows, int64_t hidden, int, int sm_count)
{
    return stat_bytes(rows) +
           static_cast<size_t>(generic_chunks(rows, hidden, sm_count)) * hidden * sizeof(float);
}

cudaError_t launch_rms_bwd(const RmsBwdArgs &a, int dtype)
{
    return dtype == RMSNORM_F32    ? launch_generic<RMSNORM_F32>(a)
           : dtype == RMSNORM_BF16 ? launch_generic<RMSNORM_BF16>(a)
                                   : launch_generic<RMSNORM_F16>(a);
}

} // namespace rmsnorm
