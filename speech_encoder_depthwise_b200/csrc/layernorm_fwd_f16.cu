#include "layernorm_fwd.cuh"

namespace dwk {
cudaError_t layernorm_fwd_rows_f16(const ResidualArgs &a, cudaStream_t s) { return lnf::launch_rows<f16>(a, s); }
}  // namespace dwk
