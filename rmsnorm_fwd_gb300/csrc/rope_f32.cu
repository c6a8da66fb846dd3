#include "ropevec.cuh"

namespace rmsnorm {

cudaError_t launch_rope_vec_f32(const RopeArgs &a, bool *taken)
{
    return launch_vectors<RMSNORM_F32>(a, taken);
}

} // namespace rmsnorm
