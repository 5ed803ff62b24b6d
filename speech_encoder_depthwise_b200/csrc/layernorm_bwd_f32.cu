#include "layernorm_bwd.cuh"

namespace dwk {
cudaError_t layernorm_bwd_rows_f32(const ResidualArgs &a, int *G, cudaStream_t s) {
    return lnb::launch_rows<float>(a, G, s);
}
}  // namespace dwk
