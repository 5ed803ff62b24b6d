// The row kernel of layer norm forward (alone, or behind dropout and the residual add) and its
// dispatch; instantiated per element type in layernorm_fwd_{bf16,f16,f32}.cu.
#pragma once

#include "dw_internal.h"
#include "residual.cuh"

namespace dwk {
namespace lnf {

// TPR threads hold a row's NO octets each in registers: one read of x (and res), the mean, then
// the variance of the centred values, then the outputs.  SHIFT: rows that do not start on an octet
// (C not a multiple of 8); gamma and beta are then read from shared memory, channel by channel.
template <typename T, int TPR, int NO, bool SHIFT, bool DROP>
__global__ void __launch_bounds__(TPR > 256 ? TPR : 256)
layernorm_fwd_rows_kernel(const ResidualArgs a) {
    constexpr int kThreads = TPR > 256 ? TPR : 256, GPB = kThreads / TPR;
    __shared__ float red[2 * (TPR > 32 ? TPR / 32 : 1)];
    extern __shared__ float sp[];  // SHIFT: gamma, then beta, padded
    launch_dependents();
    const int lane = threadIdx.x % TPR, g = threadIdx.x / TPR;
    const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.res);
    T *y = static_cast<T *>(a.y), *h = static_cast<T *>(a.h);
    const int64_t N = a.B * a.T * a.C, grid = gridDim.x;
    const int C = static_cast<int>(a.C);
    grid_dependency_wait();
    const int P = pad32(C - 1) + 1;
    if constexpr (SHIFT) {
        for (int c = threadIdx.x; c < C; c += kThreads) {
            sp[pad32(c)] = a.gamma ? __ldg(a.gamma + c) : 1.f;
            sp[P + pad32(c)] = a.beta ? __ldg(a.beta + c) : 0.f;
        }
        __syncthreads();
    }
    Dropper D;
    if constexpr (DROP) D.start(a.rng, a.thr);
    RowWalk w;
    w.start(a.lengths, blockIdx.x + grid * g, grid * GPB, a.B, a.T);
    const int s = SHIFT ? static_cast<int>((w.r * a.C) % 8) : 0;
    const float inv = 1.f / static_cast<float>(C);
    int flip = 0;
    // groups of one warp walk together (their sums share its shuffles)
    const int64_t lead = TPR < 32 ? blockIdx.x + grid * (threadIdx.x / 32 * (32 / TPR)) : 0;
    for (int64_t k = 0; TPR < 32 ? lead + k * w.step < w.rows : w.in(); ++k, w.next()) {
        const bool live = TPR < 32 ? (w.in() && w.valid()) : w.valid();
        if (TPR >= 32 ? !live : (w.in() && !live)) {
            const float zero[8] = {};
#pragma unroll
            for (int j = 0; j < NO; ++j) {
                const OctAt<T, SHIFT> at(w.r, a.C, j * TPR + lane, s);
                if (!at.any()) continue;
                at.store(y, zero);
                if (h) at.store(h, zero);
            }
            if (lane == 0) {
                if (a.mean) a.mean[w.r] = 0.f;
                if (a.rstd) a.rstd[w.r] = 0.f;
            }
            if (TPR >= 32) continue;
        }
        float v[NO][8];
        float sum = 0.f;
        {
            Oct<T> xo[NO], ro[NO];
#pragma unroll
            for (int j = 0; j < NO; ++j) {
                const OctAt<T, SHIFT> at(w.r, a.C, j * TPR + lane, s);
                xo[j].zero();
                ro[j].zero();
                if (live && at.any()) {
                    at.load(x, xo[j], N);
                    if (res) at.load(res, ro[j], N);
                }
            }
#pragma unroll
            for (int j = 0; j < NO; ++j) {
                const OctAt<T, SHIFT> at(w.r, a.C, j * TPR + lane, s);
                float f[8], q[8];
                xo[j].get(f);
                ro[j].get(q);
                if constexpr (DROP) D.apply(static_cast<uint64_t>(at.e0) >> 3, f);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[j][i] = at.has(i) ? fmaf(a.mult, f[i], q[i]) : 0.f;
                    sum += v[j][i];
                }
            }
        }
        const float mean = row_sum<TPR>(sum, red, flip) * inv;
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < NO; ++j) {
            const OctAt<T, SHIFT> at(w.r, a.C, j * TPR + lane, s);
            if (!at.any()) continue;
            if (h && live) at.store(h, v[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[j][i] -= mean;
                if (at.has(i)) ss = fmaf(v[j][i], v[j][i], ss);
            }
        }
        const float rstd = 1.f / sqrtf(row_sum<TPR>(ss, red, flip) * inv + a.eps);
#pragma unroll
        for (int j = 0; j < NO; ++j) {
            const OctAt<T, SHIFT> at(w.r, a.C, j * TPR + lane, s);
            if (!at.any() || !live) continue;
            float ga[8], be[8], o[8];
            if constexpr (SHIFT) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int c = at.has(i) ? pad32(at.c0 + i) : 0;
                    ga[i] = sp[c];
                    be[i] = sp[P + c];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; i += 4) {
                    const float4 p = a.gamma ? __ldg(reinterpret_cast<const float4 *>(a.gamma + at.c0 + i)) : make_float4(1.f, 1.f, 1.f, 1.f);
                    const float4 q = a.beta ? __ldg(reinterpret_cast<const float4 *>(a.beta + at.c0 + i)) : make_float4(0.f, 0.f, 0.f, 0.f);
                    ga[i] = p.x; ga[i + 1] = p.y; ga[i + 2] = p.z; ga[i + 3] = p.w;
                    be[i] = q.x; be[i + 1] = q.y; be[i + 2] = q.z; be[i + 3] = q.w;
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = fmaf(v[j][i] * rstd, ga[i], be[i]);
            at.store(y, o);
        }
        if (lane == 0 && live) {
            if (a.mean) a.mean[w.r] = mean;
            if (a.rstd) a.rstd[w.r] = rstd;
        }
    }
}

template <typename T, int TPR, int NO, bool SHIFT, bool DROP>
cudaError_t launch(const ResidualArgs &a, cudaStream_t s) {
    constexpr int kThreads = TPR > 256 ? TPR : 256, GPB = kThreads / TPR;
    const auto kern = layernorm_fwd_rows_kernel<T, TPR, NO, SHIFT, DROP>;
    const size_t smem = SHIFT ? 2 * ((a.C - 1) + ((a.C - 1) >> 5) + 1) * sizeof(float) : 0;
    if (SHIFT) {
        const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(kern), static_cast<int>(smem));
        if (e != cudaSuccess) return e;
    }
    const int64_t rows = a.B * a.T;
    const int64_t fit = SHIFT ? (200 * 1024) / static_cast<int64_t>(smem + 1024) : 8;
    int64_t per_sm = 2048 / kThreads;
    if (per_sm > fit) per_sm = fit < 1 ? 1 : fit;
    const int64_t most = sm_count() * per_sm * GPB;                 // rows in flight
    const int64_t passes = (rows + most - 1) / most;
    int64_t grid = (rows + passes * GPB - 1) / (passes * GPB);
    if (SHIFT && passes > 1 && GPB % 8 != 0) grid = (grid + 7) / 8 * 8;  // a group's rows stay 8 k apart
    return launch_programmatic(kern, dim3(static_cast<unsigned>(grid)), dim3(kThreads), smem, s, a);
}

template <typename T, int TPR, int NO, bool SHIFT>
cudaError_t launch(const ResidualArgs &a, cudaStream_t s) {
    return a.thr ? launch<T, TPR, NO, SHIFT, true>(a, s) : launch<T, TPR, NO, SHIFT, false>(a, s);
}

// cudaErrorNotSupported: no row kernel for these sizes or this alignment.
template <typename T>
cudaError_t launch_rows(const ResidualArgs &a, cudaStream_t s) {
    if (!a.vec_oct || a.C > 8192) return cudaErrorNotSupported;
    const bool params16 = reinterpret_cast<uintptr_t>(a.gamma) % 16 == 0 && reinterpret_cast<uintptr_t>(a.beta) % 16 == 0;
    if (a.C % 8 == 0 && params16) {
        const int64_t n = a.C / 8;
        if (n <= 8) return launch<T, 8, 1, false>(a, s);
        if (n <= 16) return launch<T, 16, 1, false>(a, s);
        if (n <= 32) return launch<T, 32, 1, false>(a, s);
        if (n <= 64) return launch<T, 32, 2, false>(a, s);
        if (n <= 96) return launch<T, 32, 3, false>(a, s);
        if (n <= 128) return launch<T, 32, 4, false>(a, s);
        if (n <= 160) return launch<T, 32, 5, false>(a, s);
        if (n <= 256) return launch<T, 256, 1, false>(a, s);
        if (n <= 512) return launch<T, 512, 1, false>(a, s);
        return launch<T, 1024, 1, false>(a, s);
    }
    const int64_t n = (a.C + 14) / 8;  // octets a row may touch: up to 7 elements before its first
    if (n <= 32) return launch<T, 32, 1, true>(a, s);
    if (n <= 64) return launch<T, 32, 2, true>(a, s);
    if (n <= 96) return launch<T, 32, 3, true>(a, s);
    if (n <= 128) return launch<T, 32, 4, true>(a, s);
    if (n <= 160) return launch<T, 32, 5, true>(a, s);
    if (n <= 256) return launch<T, 256, 1, true>(a, s);
    if (n <= 512) return launch<T, 512, 1, true>(a, s);
    if (n <= 1024) return launch<T, 1024, 1, true>(a, s);
    return cudaErrorNotSupported;
}

}  // namespace lnf
}  // namespace dwk
