#include "layernorm_bwd.cuh"

namespace dwk {
cudaError_t layernorm_bwd_rows_f16(const ResidualArgs &a, int *G, cudaStream_t s) {
    return lnb::launch_rows<f16>(a, G, s);
}
}  // namespace dwk
