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

// Partial rows: at most two blocks on each of 148 SMs, and at most 64 MiB of them (at least one).
constexpr int kMaxPartialRows = 296;

// Any C, any alignment: a block per row, two passes over it, one element at a time; the block's
// partial row lives in the workspace (a thread only touches its own columns, so no synchronization is
// needed).  4096 rows of 12288 bf16: 666 us (0.07 of the measured copy bandwidth).
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

// dgamma[c], dbeta[c] = the G partial rows' entries in a fixed order.  A block covers 16 entries of the
// 2 ceil4(C) with 8 row groups; group q adds rows q, q + 8, ... in order, its loads in flight together,
// then the 8 group sums are added in a fixed tree.  Blocks of 128 threads with 32 registers fit
// beside the row kernel's on an SM, so they are resident and waiting when it ends.
__global__ void __launch_bounds__(128, 16)
layernorm_bwd_finalize_kernel(const float *__restrict__ partials, float *__restrict__ dgamma,
                              float *__restrict__ dbeta, int G, int64_t C) {
    __shared__ float red[8][17];
    launch_dependents();
    const int lane = threadIdx.x % 16, q = threadIdx.x / 16;
    const int64_t Cp = (C + 3) / 4 * 4, E = 2 * Cp, e = static_cast<int64_t>(blockIdx.x) * 16 + lane;
    const float *p = partials + q * E + e;
    const bool live = e < E;
    grid_dependency_wait();
    float s = 0.f;
    for (int r0 = 0; r0 < G; r0 += 160) {
        float v[20];
#pragma unroll
        for (int i = 0; i < 20; ++i) v[i] = live && r0 + q + 8 * i < G ? __ldg(p + (r0 + 8 * i) * E) : 0.f;
#pragma unroll
        for (int i = 0; i < 20; ++i) s += v[i];
    }
    red[q][lane] = s;
    __syncthreads();
    if (q == 0 && live) {
        const float t = ((red[0][lane] + red[1][lane]) + (red[2][lane] + red[3][lane])) +
                        ((red[4][lane] + red[5][lane]) + (red[6][lane] + red[7][lane]));
        const int64_t c = e < Cp ? e : e - Cp;
        float *out = e < Cp ? dgamma : dbeta;
        if (c < C && out) out[c] = t;
    }
}

}  // namespace

int layernorm_bwd_partial_rows(int64_t B, int64_t T, int64_t C) {
    const int64_t rows = B * T, row_bytes = 2 * ((C + 3) / 4 * 4) * 4;
    int64_t g = (int64_t(64) << 20) / row_bytes;
    if (g > kMaxPartialRows) g = kMaxPartialRows;
    if (g > rows) g = rows;
    return static_cast<int>(g < 1 ? 1 : g);
}

size_t layernorm_bwd_workspace_bytes(int64_t B, int64_t T, int64_t C) {
    return static_cast<size_t>(layernorm_bwd_partial_rows(B, T, C)) * 2 * ((C + 3) / 4 * 4) * sizeof(float);
}

// With no rows only the finalize runs, over no partial rows: zeros.
cudaError_t layernorm_bwd_launch(const ResidualArgs &a, cudaStream_t s) {
    int G = 0;
    if (a.B * a.T > 0) {
        cudaError_t e = a.dtype == 1   ? layernorm_bwd_rows_bf16(a, &G, s)
                        : a.dtype == 2 ? layernorm_bwd_rows_f16(a, &G, s)
                                       : layernorm_bwd_rows_f32(a, &G, s);
        if (e == cudaErrorNotSupported) {
            G = a.G;
            e = with_dtype(a.dtype, [&](auto t) {
                return launch_programmatic(layernorm_bwd_general_kernel<decltype(t)>, dim3(static_cast<unsigned>(G)),
                                           dim3(256), 0, s, a);
            });
        }
        if (e != cudaSuccess || G == 0) return e;  // G == 0: the row kernel wrote dgamma and dbeta
    }
    if (!a.dgamma && !a.dbeta) return cudaSuccess;
    const int64_t blocks = (2 * ((a.C + 3) / 4 * 4) + 15) / 16;
    return launch_programmatic(layernorm_bwd_finalize_kernel, dim3(static_cast<unsigned>(blocks)), dim3(128), 0, s,
                               static_cast<const float *>(a.partials), a.dgamma, a.dbeta, G, a.C);
}

}  // namespace dwk
