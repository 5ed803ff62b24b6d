#include "layernorm_fwd.cuh"

namespace dwk {
cudaError_t layernorm_fwd_rows_f32(const ResidualArgs &a, cudaStream_t s) { return lnf::launch_rows<float>(a, s); }
}  // namespace dwk
