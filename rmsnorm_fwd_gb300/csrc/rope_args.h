// rope_args.h -- shared between the host side (api_rope.cpp) and the kernels of
// the head operators with a position rotation and of the gradients.
#pragma once

#include "internal.h"
#include "rmsnorm_rope.h"

namespace rmsnorm {

// What a call needs of the current device's context (api.cpp).
struct CallContext {
    int sm_count;
    int smem_optin;
    int *status; // device status word
    bool pdl;
};
int call_context(CallContext *out);

// Heads with a position rotation (rope.cu, rope_bwd.cu).  A negative extent
// never occurs: api_rope.cpp has checked every size, stride and overlap.
struct HeadsView {
    char *p;
    int64_t ts, hs; // elements between tokens, between heads
};
struct RopeTable {
    const float *cs;
    const int64_t *pos;
    int64_t max_pos;
    int32_t rd; // rotated elements of a head, even
    int32_t interleaved;
};
constexpr int32_t kMaxHeadDim = 1024;

struct RopeArgs {
    LaunchArgs base; // stream, launch attributes and status word
    HeadsView q, k, qo, ko; // ko unused when appending
    const void *qw, *kw;    // both null: no norm (appending only)
    RopeTable rope;
    int64_t tokens;
    int32_t q_heads, k_heads, head_dim;
    float bias, eps;
    // Appending (slots != null): v, the cache and its strides.
    HeadsView v;
    const int64_t *slots;
    char *kc, *vc;
    int64_t num_slots, page_size;          // num_slots = pages * page_size
    int64_t page_stride, slot_stride, cache_hs; // elements
    int32_t e4m3;
    float k_inv, v_inv; // 1 / scale
    int sm_count;
};
cudaError_t launch_rope(const RopeArgs &a, int dtype);
// The vector bodies; *taken is false when none takes the call.
cudaError_t launch_rope_vec_f32(const RopeArgs &a, bool *taken);
cudaError_t launch_rope_vec_bf16(const RopeArgs &a, bool *taken);
cudaError_t launch_rope_vec_f16(const RopeArgs &a, bool *taken);

struct RopeBwdArgs {
    LaunchArgs base;
    HeadsView qdy, kdy, q, k, dq, dk;
    const void *qw, *kw;
    float *dqw, *dkw; // null: not wanted
    float *part;      // workspace: a row of head_dim per block
    RopeTable rope;
    int64_t tokens;
    int32_t q_heads, k_heads, head_dim;
    float bias, eps;
    int sm_count;
};
cudaError_t launch_rope_bwd(const RopeBwdArgs &a, int dtype);
int rope_bwd_max_blocks(int sm_count); // rows of the workspace

// out[j] = sum over i < rows of part[i * ld + j], j < cols, in a fixed order
// (colsum.cu).  Two sums in one launch; a second of no columns is left out.
struct ColSum {
    const float *part;
    float *out;
    int64_t rows, cols, ld;
};
cudaError_t launch_colsum(const ColSum &a, const ColSum &b, const LaunchArgs &base);

// Row gradient (rms_bwd.cu).
struct RmsBwdArgs {
    LaunchArgs base;
    const void *dy, *x, *w;
    void *dx;
    float *dw; // null: not wanted
    void *ws;
    int64_t rows, hidden;
    float bias, eps;
    int sm_count;
};
cudaError_t launch_rms_bwd(const RmsBwdArgs &a, int dtype);
size_t rms_bwd_workspace(int64_t rows, int64_t hidden, int dtype, int sm_count);

} // namespace rmsnorm
