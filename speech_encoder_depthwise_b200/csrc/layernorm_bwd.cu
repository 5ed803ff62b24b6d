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

// dgamma[c], dbeta[c] = the G <= 32 R partial rows' entries in a fixed order.  A block covers 32
// entries of the 2 ceil4(C) (8 lanes of a float4) with 32 row groups; group q adds rows q, q + 32, ...
// in order, all loads of a thread in flight at once, then the group sums are added in a fixed tree.
constexpr int kFinalizeRows = (kMaxPartialRows + 31) / 32;
__global__ void __launch_bounds__(256)
layernorm_bwd_finalize_kernel(const float *__restrict__ partials, float *__restrict__ dgamma,
                              float *__restrict__ dbeta, int G, int64_t C) {
    __shared__ float4 red[32][9];
    launch_dependents();
    grid_dependency_wait();
    const int lane = threadIdx.x % 8, q = threadIdx.x / 8;
    const int64_t Cp = (C + 3) / 4 * 4, E = 2 * Cp, e = static_cast<int64_t>(blockIdx.x) * 32 + lane * 4;
    float4 v[kFinalizeRows], s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kFinalizeRows; ++i) {
        const int r = q + 32 * i;
        v[i] = e < E && r < G ? __ldg(reinterpret_cast<const float4 *>(partials + r * E + e)) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int i = 0; i < kFinalizeRows; ++i) {
        s.x += v[i].x;
        s.y += v[i].y;
        s.z += v[i].z;
        s.w += v[i].w;
    }
    red[q][lane] = s;
    __syncthreads();
    if (threadIdx.x < 32) {
        const float *p = &red[0][0].x + threadIdx.x;
        float t[32];
#pragma unroll
        for (int r = 0; r < 32; ++r) t[r] = p[r * 36];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1)
#pragma unroll
            for (int r = 0; r + d < 32; r += 2 * d) t[r] += t[r + d];
        const int64_t o = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x, c = o < Cp ? o : o - Cp;
        float *out = o < Cp ? dgamma : dbeta;
        if (o < E && c < C && out) out[c] = t[0];
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
        if (e != cudaSuccess) return e;
    }
    if (!a.dgamma && !a.dbeta) return cudaSuccess;
    const int64_t blocks = (2 * ((a.C + 3) / 4 * 4) + 31) / 32;
    return launch_programmatic(layernorm_bwd_finalize_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s,
                               static_cast<const float *>(a.partials), a.dgamma, a.dbeta, G, a.C);
}

}  // namespace dwk
