// Layer norm forward, alone or fused behind dropout and the residual add:
//   s = res + [kept] mult x,  h = s rounded,  y = (s - mean) rstd gamma + beta  over the C channels.
// Statistics in float32: the mean first, then the variance of the centred values (no
// E[s^2] - mean^2 cancellation).
#include "dw_internal.h"
#include "residual.cuh"

namespace dwk {
namespace {

// Any C, any alignment: a block per row, three passes over the row (the second and third hit L1/L2),
// s computed anew in each, one element at a time.  Bound by instructions: 4096 rows of 12288 bf16
// 261 us (0.12 of the measured copy bandwidth), with dropout a whole mask block per element and pass.
template <typename T>
__global__ void __launch_bounds__(256)
layernorm_fwd_general_kernel(const ResidualArgs a) {
    __shared__ float2 red[2][8];
    launch_dependents();
    grid_dependency_wait();
    DropoutRng R = {};
    if (a.thr) R.load(a.rng);
    const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.res);
    T *y = static_cast<T *>(a.y), *h = static_cast<T *>(a.h);
    const int64_t rows = a.B * a.T;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const int64_t base = r * a.C, b = r / a.T;
        if (r - b * a.T >= clamp_len(a.lengths, b, a.T)) {
            for (int64_t c = threadIdx.x; c < a.C; c += 256) {
                store1(y + base + c, 0.f);
                if (h) store1(h + base + c, 0.f);
            }
            if (threadIdx.x == 0) {
                if (a.mean) a.mean[r] = 0.f;
                if (a.rstd) a.rstd[r] = 0.f;
            }
            continue;
        }
        auto sum_at = [&](int64_t c) {
            const int64_t e = base + c;
            const float v = res ? load1(res + e) : 0.f;
            return a.thr == 0 || R.kept(static_cast<uint64_t>(e), a.thr) ? fmaf(a.mult, load1(x + e), v) : v;
        };
        float2 acc = make_float2(0.f, 0.f);
        for (int64_t c = threadIdx.x; c < a.C; c += 256) acc.x += sum_at(c);
        const float mean = block_sum2<8>(acc, red[0]).x / static_cast<float>(a.C);
        acc.x = 0.f;
        for (int64_t c = threadIdx.x; c < a.C; c += 256) {
            const float d = sum_at(c) - mean;
            acc.x = fmaf(d, d, acc.x);
        }
        const float rstd = 1.f / sqrtf(block_sum2<8>(acc, red[1]).x / static_cast<float>(a.C) + a.eps);
        for (int64_t c = threadIdx.x; c < a.C; c += 256) {
            const float v = sum_at(c);
            if (h) store1(h + base + c, v);
            const float ga = a.gamma ? __ldg(a.gamma + c) : 1.f, be = a.beta ? __ldg(a.beta + c) : 0.f;
            store1(y + base + c, fmaf((v - mean) * rstd, ga, be));
        }
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
    }
}

}  // namespace

cudaError_t layernorm_fwd_launch(const ResidualArgs &a, cudaStream_t s) {
    const cudaError_t e = a.dtype == 1   ? layernorm_fwd_rows_bf16(a, s)
                          : a.dtype == 2 ? layernorm_fwd_rows_f16(a, s)
                                         : layernorm_fwd_rows_f32(a, s);
    if (e != cudaErrorNotSupported) return e;
    const int64_t rows = a.B * a.T, most = static_cast<int64_t>(sm_count()) * 8;
    const dim3 grid(static_cast<unsigned>(rows < most ? rows : most));
    return with_dtype(a.dtype, [&](auto t) {
        return launch_programmatic(layernorm_fwd_general_kernel<decltype(t)>, grid, dim3(256), 0, s, a);
    });
}

}  // namespace dwk
