// The row kernel of layer norm backward (alone, or with the gradients of dropout and the residual
// add) and its dispatch; instantiated per element type in layernorm_bwd_{bf16,f16,f32}.cu.
#pragma once

#include "dw_internal.h"
#include "residual.cuh"

namespace dwk {
namespace lnb {

// TPR threads hold a row's NO octets each in registers.  Every thread keeps its channels from row to
// row, so dgamma and dbeta add up in registers over all its rows; the block's groups are then added
// in a fixed order through shared memory into the block's partial row.
template <typename T, int TPR, int NO, int THREADS, bool SHIFT, bool DROP>
__global__ void __launch_bounds__(THREADS)
layernorm_bwd_rows_kernel(const ResidualArgs a) {
    constexpr int GPB = THREADS / TPR, W = THREADS / 32;
    __shared__ float2 red[2 * (TPR > 32 ? TPR / 32 : 1)];
    extern __shared__ float sp[];  // SHIFT: gamma, padded; at the end the warps' dgamma, dbeta
    launch_dependents();
    const int lane = threadIdx.x % TPR, g = threadIdx.x / TPR;
    const T *x = static_cast<const T *>(a.x), *dy = static_cast<const T *>(a.dy), *dh = static_cast<const T *>(a.dh);
    T *dx = static_cast<T *>(a.dx), *dres = static_cast<T *>(a.dres);
    const int64_t N = a.B * a.T * a.C, grid = gridDim.x;
    const int C = static_cast<int>(a.C);
    grid_dependency_wait();
    if constexpr (SHIFT) {
        for (int c = threadIdx.x; c < C; c += THREADS) sp[pad32(c)] = a.gamma ? __ldg(a.gamma + c) : 1.f;
        __syncthreads();
    }
    Dropper D;
    if constexpr (DROP) D.start(a.rng, a.thr);
    RowWalk w;
    w.start(a.lengths, blockIdx.x + grid * g, grid * GPB, a.B, a.T);
    const int s = SHIFT ? static_cast<int>((w.r * a.C) % 8) : 0;
    const float inv = 1.f / static_cast<float>(C);
    int flip = 0;
    float ag[NO][8] = {}, ab[NO][8] = {};
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
                at.store(dx, zero);
                if (dres) at.store(dres, zero);
            }
            if (TPR >= 32) continue;
        }
        Oct<T> xo[NO], go[NO], ho[NO];
        float mean = 0.f, rstd = 0.f;
        if (live) {
            mean = __ldg(a.mean + w.r);
            rstd = __ldg(a.rstd + w.r);
        }
#pragma unroll
        for (int j = 0; j < NO; ++j) {
            const OctAt<T, SHIFT> at(w.r, a.C, j * TPR + lane, s);
            xo[j].zero();
            go[j].zero();
            ho[j].zero();
            if (live && at.any()) {
                at.load(x, xo[j], N);
                at.load(dy, go[j], N);
                if (dh) at.load(dh, ho[j], N);
            }
        }
        float2 sum = make_float2(0.f, 0.f);
        float gg[NO][8];
#pragma unroll
        for (int j = 0; j < NO; ++j) {
            const OctAt<T, SHIFT> at(w.r, a.C, j * TPR + lane, s);
            if (!at.any()) continue;
            float f[8], ga[8];
            xo[j].get(f);
            go[j].get(gg[j]);
            if constexpr (SHIFT) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    ga[i] = sp[at.has(i) ? pad32(at.c0 + i) : 0];
                    f[i] = at.has(i) ? f[i] : 0.f;
                    gg[j][i] = at.has(i) ? gg[j][i] : 0.f;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; i += 4) {
                    const float4 p = a.gamma ? __ldg(reinterpret_cast<const float4 *>(a.gamma + at.c0 + i)) : make_float4(1.f, 1.f, 1.f, 1.f);
                    ga[i] = p.x; ga[i + 1] = p.y; ga[i + 2] = p.z; ga[i + 3] = p.w;
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float xh = (f[i] - mean) * rstd, d = gg[j][i];
                ag[j][i] = fmaf(d, xh, ag[j][i]);
                ab[j][i] += d;
                gg[j][i] = d * ga[i];
                sum.x += gg[j][i];
                sum.y = fmaf(gg[j][i], xh, sum.y);
            }
        }
        sum = row_sum2<TPR>(sum, red, flip);
        const float c1 = sum.x * inv, c2 = sum.y * inv;
#pragma unroll
        for (int j = 0; j < NO; ++j) {
            const OctAt<T, SHIFT> at(w.r, a.C, j * TPR + lane, s);
            if (!at.any() || !live) continue;
            float f[8], d[8];
            xo[j].get(f);
            ho[j].get(d);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float xh = (f[i] - mean) * rstd;
                f[i] = fmaf(rstd, gg[j][i] - fmaf(xh, c2, c1), d[i]);
            }
            if (dres) at.store(dres, f);
            if constexpr (DROP) D.apply(static_cast<uint64_t>(at.e0) >> 3, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] *= a.mult;
            at.store(dx, f);
        }
    }
    if (!a.dgamma && !a.dbeta) return;
    const int64_t Cp = (a.C + 3) / 4 * 4;
    float *pg = a.partials + static_cast<int64_t>(blockIdx.x) * 2 * Cp;
    if constexpr (TPR > 32) {  // one group: its channels straight to the partial row
#pragma unroll
        for (int j = 0; j < NO; ++j) {
            const OctAt<T, SHIFT> at(0, a.C, j * TPR + lane, s);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (at.any() && at.has(i)) {
                    pg[at.c0 + i] = ag[j][i];
                    pg[Cp + at.c0 + i] = ab[j][i];
                }
        }
    } else {
        if constexpr (TPR < 32) {  // the warp's groups hold the same channels (no SHIFT here)
#pragma unroll
            for (int o = TPR; o < 32; o <<= 1)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    ag[0][i] += __shfl_xor_sync(0xffffffffu, ag[0][i], o);
                    ab[0][i] += __shfl_xor_sync(0xffffffffu, ab[0][i], o);
                }
        }
        // warps HALF .. W-1 store, warps 0 .. HALF-1 add to them, then the HALF slots are added in order
        constexpr int HALF = W / 2;
        const int P = pad32(C - 1) + 1, warp = threadIdx.x / 32;
        if constexpr (SHIFT) __syncthreads();  // gamma is no longer read
#pragma unroll
        for (int phase = 0; phase < 2; ++phase) {
            float *slot = sp + (phase == 0 ? warp - HALF : warp) * 2 * P;
            if ((phase == 0) == (warp >= HALF) && (TPR == 32 || threadIdx.x % 32 < TPR)) {
#pragma unroll
                for (int j = 0; j < NO; ++j) {
                    const OctAt<T, SHIFT> at(0, a.C, j * TPR + lane, s);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (at.any() && at.has(i)) {
                            const int c = pad32(at.c0 + i);
                            slot[c] = phase == 0 ? ag[j][i] : slot[c] + ag[j][i];
                            slot[P + c] = phase == 0 ? ab[j][i] : slot[P + c] + ab[j][i];
                        }
                }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < 2 * C; c += THREADS) {
            const int which = c >= C, ch = which ? c - C : c;
            const float *p = sp + which * P + pad32(ch);
            float t = p[0];
#pragma unroll
            for (int q = 1; q < HALF; ++q) t += p[q * 2 * P];
            pg[which * Cp + ch] = t;
        }
    }
}

template <typename T, int TPR, int NO, int THREADS, bool SHIFT, bool DROP>
cudaError_t launch(const ResidualArgs &a, int *G, cudaStream_t s) {
    constexpr int GPB = THREADS / TPR, HALF = THREADS / 64;
    const auto kern = layernorm_bwd_rows_kernel<T, TPR, NO, THREADS, SHIFT, DROP>;
    const size_t P = static_cast<size_t>((a.C - 1) + ((a.C - 1) >> 5) + 1);
    size_t smem = SHIFT ? P * sizeof(float) : 0;
    if (TPR <= 32) smem = HALF * 2 * P * sizeof(float);
    const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(kern), static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    constexpr int kPerSm = TPR == 256 || (TPR == 512 && NO == 1) ? 2 : 1;
    const int64_t rows = a.B * a.T;
    int64_t grid = sm_count() * kPerSm;
    if (grid > a.G) grid = a.G;
    if (SHIFT && rows > grid * GPB) {  // more than one row a group: keep them a multiple of 8 apart
        constexpr int kMult = GPB % 8 == 0 ? 1 : (GPB % 4 == 0 ? 2 : (GPB % 2 == 0 ? 4 : 8));
        if (grid < kMult) return cudaErrorNotSupported;
        grid = grid / kMult * kMult;
    }
    *G = static_cast<int>(grid);
    return launch_programmatic(kern, dim3(static_cast<unsigned>(grid)), dim3(THREADS), smem, s, a);
}

// Threads of a block (one or two blocks on an SM): as many as the registers of NO octets leave room
// for, a multiple of 64.
template <typename T> constexpr int threads_for(int NO) {
    return sizeof(T) == 2 ? (NO == 1 ? 1024 : NO == 2 ? 640 : NO == 3 ? 512 : NO == 4 ? 384 : 320)
                          : (NO == 1 ? 768 : NO == 2 ? 512 : NO == 3 ? 384 : NO == 4 ? 320 : 256);
}

template <typename T, int TPR, int NO, bool SHIFT>
cudaError_t launch(const ResidualArgs &a, int *G, cudaStream_t s) {
    constexpr int kThreads = TPR > 32 ? TPR : threads_for<T>(NO);
    return a.thr ? launch<T, TPR, NO, kThreads, SHIFT, true>(a, G, s) : launch<T, TPR, NO, kThreads, SHIFT, false>(a, G, s);
}

// cudaErrorNotSupported: no row kernel for these sizes or this alignment.
template <typename T>
cudaError_t launch_rows(const ResidualArgs &a, int *G, cudaStream_t s) {
    if (!a.vec_oct || a.C > 8192) return cudaErrorNotSupported;
    if (a.C % 8 == 0 && reinterpret_cast<uintptr_t>(a.gamma) % 16 == 0) {
        const int64_t n = a.C / 8;
        if (n <= 8) return launch<T, 8, 1, false>(a, G, s);
        if (n <= 16) return launch<T, 16, 1, false>(a, G, s);
        if (n <= 32) return launch<T, 32, 1, false>(a, G, s);
        if (n <= 64) return launch<T, 32, 2, false>(a, G, s);
        if (n <= 96) return launch<T, 32, 3, false>(a, G, s);
        if (n <= 128) return launch<T, 32, 4, false>(a, G, s);
        if (n <= 160) return launch<T, 32, 5, false>(a, G, s);
        if (n <= 256) return launch<T, 256, 1, false>(a, G, s);
        if (n <= 512) return launch<T, 512, 1, false>(a, G, s);
        return launch<T, 512, 2, false>(a, G, s);
    }
    const int64_t n = (a.C + 14) / 8;  // octets a row may touch: up to 7 elements before its first
    if (n <= 32) return launch<T, 32, 1, true>(a, G, s);
    if (n <= 64) return launch<T, 32, 2, true>(a, G, s);
    if (n <= 96) return launch<T, 32, 3, true>(a, G, s);
    if (n <= 128) return launch<T, 32, 4, true>(a, G, s);
    if (n <= 160) return launch<T, 32, 5, true>(a, G, s);
    if (n <= 256) return launch<T, 256, 1, true>(a, G, s);
    if (n <= 512) return launch<T, 512, 1, true>(a, G, s);
    if (n <= 1024) return launch<T, 512, 2, true>(a, G, s);
    return cudaErrorNotSupported;
}

}  // namespace lnb
}  // namespace dwk
