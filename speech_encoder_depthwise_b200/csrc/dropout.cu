// Dropout with the residual add, forward and (without a residual) backward:
//   y[e] = [valid] (res[e] + [kept] mult x[e]).
// Elementwise; the mask is drawn from the element's index, never stored.
#include "dw_internal.h"
#include "residual.cuh"

namespace dwk {
namespace {

// A thread takes the 8 elements of one mask block, element by element.
template <typename T>
__global__ void __launch_bounds__(256)
dropout_add_general_kernel(const T *__restrict__ x, const T *__restrict__ res, T *__restrict__ y,
                           const int32_t *__restrict__ lengths, const unsigned long long *__restrict__ rng,
                           uint32_t thr, float mult, int64_t B, int64_t Tn, int64_t C) {
    launch_dependents();
    grid_dependency_wait();
    DropoutRng R = {};
    if (thr) R.load(rng);
    const int64_t TC = Tn * C, N = B * TC;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x * 8;
    for (int64_t e0 = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) * 8; e0 < N; e0 += stride) {
        const uint4 w4 = thr ? R.block(static_cast<uint64_t>(e0) >> 3) : make_uint4(0, 0, 0, 0);
        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
        int64_t b = e0 / TC, i = e0 - b * TC, lim = clamp_len(lengths, b, Tn) * C;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t e = e0 + j;
            if (e >= N) break;
            if (i >= TC) {
                i = 0;
                lim = clamp_len(lengths, ++b, Tn) * C;
            }
            float v = 0.f;
            if (i < lim) {
                if (res) v = load1(res + e);
                if (((w[j / 2] >> (16 * (j % 2))) & 0xffffu) >= thr) v = fmaf(mult, load1(x + e), v);
            }
            store1(y + e, v);
            ++i;
        }
    }
}

}  // namespace

cudaError_t dropout_add_launch(const ResidualArgs &a, cudaStream_t s) {
    const int64_t groups = (a.B * a.T * a.C + 7) / 8;
    const int64_t blocks = (groups + 255) / 256, most = static_cast<int64_t>(sm_count()) * 8;
    const dim3 grid(static_cast<unsigned>(blocks < most ? blocks : most));
    return with_dtype(a.dtype, [&](auto t) {
        using T = decltype(t);
        return launch_programmatic(dropout_add_general_kernel<T>, grid, dim3(256), 0, s, static_cast<const T *>(a.x),
                                   static_cast<const T *>(a.res), static_cast<T *>(a.y), a.lengths, a.rng, a.thr,
                                   a.mult, a.B, a.T, a.C);
    });
}

}  // namespace dwk
