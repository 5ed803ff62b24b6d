// Layer norm backward, alone or fused with the gradients of dropout and the residual add:
//   xh = (x - mean) rstd,  g = dy gamma,  ds = dh + rstd (g - mean_c(g) - xh mean_c(g xh)),
//   dres = ds,  dx = [kept] mult ds,  dgamma = sum_rows dy xh,  dbeta = sum_rows dy.
// Two kernels:
//  1. row kernel: every block walks rows and adds their dgamma/dbeta terms to a partial row of its
//     own in the workspace, [G][2][ceil4(C)];
//  2. finalize kernel: the partial rows added in a fixed order.
// No atomics: bitwise reproducible for given sizes on a given GPU model.
#include "dw_internal.h"
#include "residual.cuh"

namespace dwk {
namespace {

// Any C, any alignment: a block per row, two passes over it; the block's partial row lives in the
// workspace (a thread only touches its own columns, so no synchronization is needed).
template <typename T>
__global__ void __launch_bounds__(256)
layernorm_bwd_general_kernel(const ResidualArgs a) {
    __shared__ float2 red[2][8];
    launch_dependents();
    grid_dependency_wait();
    DropoutRng R = {};
    if (a.thr) R.load(a.rng);
    const T *x = static_cast<const T *>(a.x), *dy = static_cast<const T *>(a.dy), *dh = static_cast<const T *>(a.dh);
    T *dx = static_cast<T *>(a.dx), *dres = static_cast<T *>(a.dres);
    const bool params = a.dgamma || a.dbeta;
    const int64_t rows = a.B * a.T, Cp = (a.C + 3) / 4 * 4;
    float *pg = params ? a.partials + static_cast<int64_t>(blockIdx.x) * 2 * Cp : nullptr;
    if (params)
        for (int64_t c = threadIdx.x; c < a.C; c += 256) pg[c] = pg[Cp + c] = 0.f;
    int flip = 0;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const int64_t base = r * a.C, b = r / a.T;
        if (r - b * a.T >= clamp_len(a.lengths, b, a.T)) {
            for (int64_t c = threadIdx.x; c < a.C; c += 256) {
                store1(dx + base + c, 0.f);
                if (dres) store1(dres + base + c, 0.f);
            }
            continue;
        }
        const float mean = __ldg(a.mean + r), rstd = __ldg(a.rstd + r);
        float2 acc = make_float2(0.f, 0.f);
        for (int64_t c = threadIdx.x; c < a.C; c += 256) {
            const float xh = (load1(x + base + c) - mean) * rstd, d = load1(dy + base + c);
            const float g = a.gamma ? d * __ldg(a.gamma + c) : d;
            acc.x += g;
            acc.y = fmaf(g, xh, acc.y);
            if (params) {
                pg[c] = fmaf(d, xh, pg[c]);
                pg[Cp + c] += d;
            }
        }
        acc = block_sum2<8>(acc, red[flip]);
        flip ^= 1;
        const float c1 = acc.x / static_cast<float>(a.C), c2 = acc.y / static_cast<float>(a.C);
        for (int64_t c = threadIdx.x; c < a.C; c += 256) {
            const int64_t e = base + c;
            const float xh = (load1(x + e) - mean) * rstd, d = load1(dy + e);
            const float g = a.gamma ? d * __ldg(a.gamma + c) : d;
            float ds = rstd * (g - c1 - xh * c2);
            if (dh) ds += load1(dh + e);
            if (dres) store1(dres + e, ds);
            const bool keep = a.thr == 0 || R.kept(static_cast<uint64_t>(e), a.thr);
            store1(dx + e, keep ? a.mult * ds : 0.f);
        }
    }
}

// dgamma[c], dbeta[c] = the G partial rows' entries added in order.  A block covers 32 entries of
// the 2 ceil4(C) with 8 row groups; group r adds rows r, r + 8, ... in order, then the 8 group sums
// are added in a fixed tree.
__global__ void __launch_bounds__(256)
layernorm_bwd_finalize_kernel(const float *__restrict__ partials, float *__restrict__ dgamma,
                              float *__restrict__ dbeta, int G, int64_t C) {
    __shared__ float red[8][33];
    launch_dependents();
    grid_dependency_wait();
    const int col = threadIdx.x % 32, rg = threadIdx.x / 32;
    const int64_t Cp = (C + 3) / 4 * 4, E = 2 * Cp, e = static_cast<int64_t>(blockIdx.x) * 32 + col;
    const int64_t c = e < Cp ? e : e - Cp;
    const bool live = e < E && c < C;
    float s = 0.f;
    if (live) {
#pragma unroll 4
        for (int g = rg; g < G; g += 8) s += __ldg(partials + static_cast<int64_t>(g) * E + e);
    }
    red[rg][col] = s;
    __syncthreads();
    if (rg == 0 && live) {
        const float t = ((red[0][col] + red[1][col]) + (red[2][col] + red[3][col])) +
                        ((red[4][col] + red[5][col]) + (red[6][col] + red[7][col]));
        float *o = e < Cp ? dgamma : dbeta;
        if (o) o[c] = t;
    }
}

}  // namespace

// One partial row per block; at most 64 MiB of them (and at least one).
int layernorm_bwd_partial_rows(int64_t B, int64_t T, int64_t C) {
    const int64_t rows = B * T, row_bytes = 2 * ((C + 3) / 4 * 4) * 4;
    int64_t g = (int64_t(64) << 20) / row_bytes;
    if (g > 256) g = 256;
    if (g > rows) g = rows;
    return static_cast<int>(g < 1 ? 1 : g);
}

size_t layernorm_bwd_workspace_bytes(int64_t B, int64_t T, int64_t C) {
    return static_cast<size_t>(layernorm_bwd_partial_rows(B, T, C)) * 2 * ((C + 3) / 4 * 4) * sizeof(float);
}

// With no rows only the finalize runs, over no partial rows: zeros.
cudaError_t layernorm_bwd_launch(const ResidualArgs &a, cudaStream_t s) {
    const bool params = a.dgamma || a.dbeta;
    int G = 0;
    if (a.B * a.T > 0) {
        G = a.G;
        const cudaError_t e = with_dtype(a.dtype, [&](auto t) {
            return launch_programmatic(layernorm_bwd_general_kernel<decltype(t)>, dim3(static_cast<unsigned>(G)),
                                       dim3(256), 0, s, a);
        });
        if (e != cudaSuccess) return e;
    }
    if (!params) return cudaSuccess;
    const int64_t blocks = (2 * ((a.C + 3) / 4 * 4) + 31) / 32;
    return launch_programmatic(layernorm_bwd_finalize_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s,
                               static_cast<const float *>(a.partials), a.dgamma, a.dbeta, G, a.C);
}

}  // namespace dwk
