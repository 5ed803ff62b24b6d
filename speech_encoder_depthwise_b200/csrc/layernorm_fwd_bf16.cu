#include "layernorm_fwd.cuh"

namespace dwk {
cudaError_t layernorm_fwd_rows_bf16(const ResidualArgs &a, cudaStream_t s) { return lnf::launch_rows<bf16>(a, s); }
}  // namespace dwk
