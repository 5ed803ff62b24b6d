// The row kernel of layer norm backward (alone, or with the gradients of dropout and the residual
// add) and its dispatch; instantiated per element type in layernorm_bwd_{bf16,f16,f32}.cu.
#pragma once

#include "dw_internal.h"
#include "residual.cuh"

namespace dwk {
namespace lnb {

enum Mode { kPlain, kFused, kFusedDrop };  // layer norm alone; with residual add; with dropout too

// TPR threads hold a row's NO octets each in registers.  Every thread keeps its channels from row to
// row, so dgamma and dbeta add up in registers over all its rows; the block's groups are then added
// in a fixed order through shared memory into the block's partial row.  SHIFT: rows that do not
// start on an octet (C not a multiple of 8).
template <typename T, int TPR, int NO, int THREADS, bool SHIFT, int MODE>
__global__ void __launch_bounds__(THREADS)
layernorm_bwd_rows_kernel(const ResidualArgs a) {
    constexpr int GPB = THREADS / TPR, W = THREADS / 32, HALF = W / 2;
    __shared__ float2 red[2 * (TPR > 32 ? TPR / 32 : 1)];
    extern __shared__ float sp[];  // SHIFT: gamma; at the end the warps' dgamma, dbeta
    launch_dependents();
    const int g = threadIdx.x / TPR, grid = gridDim.x, rows = static_cast<int>(a.B * a.T);
    const T *x = static_cast<const T *>(a.x), *dy = static_cast<const T *>(a.dy), *dh = MODE == kPlain ? nullptr : static_cast<const T *>(a.dh);
    T *dx = static_cast<T *>(a.dx), *dres = MODE == kPlain ? nullptr : static_cast<T *>(a.dres);
    using Ch = Channels<T, TPR, NO, SHIFT>;
    __shared__ __align__(32) T scratch[SHIFT ? THREADS / Ch::kGroup * 16 : 1];
    Ch ch;
    const int first = blockIdx.x + grid * g;
    ch.start(static_cast<int>(a.C), rows, first, scratch);
    const int Q = shifted_q(ch.C);
    int off[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) off[i] = shifted_off(i, ch.s, Q) + ch.lane;
    grid_dependency_wait();
    if constexpr (SHIFT) {
        for (int i = threadIdx.x; i < 8 * Q; i += THREADS) {
            const int c = i / Q + 8 * (i % Q - 1);
            sp[i] = c < 0 || c >= ch.C ? 0.f : a.gamma ? __ldg(a.gamma + c) : 1.f;
        }
        __syncthreads();
    }
    Dropper D;
    if constexpr (MODE == kFusedDrop) D.start(a.rng, a.thr);
    const float inv = 1.f / static_cast<float>(ch.C);
    int flip = 0;
    float2 ag[NO][4] = {}, ab[NO][4] = {};
    RowWalk w;
    w.start(a.lengths, first, grid * GPB, rows, static_cast<int>(a.T));
    // groups of one warp walk together (their sums share its shuffles): until the first one is done
    int lead = TPR < 32 ? blockIdx.x + grid * (threadIdx.x / 32 * (32 / TPR)) : first;
    for (; lead < rows; lead += w.step, w.next()) {
        const bool in = w.in(), live = in && w.valid();
        const int64_t e = ch.at(w.r);
        Oct<T> xo[NO], go[NO], ho[NO];
        float mean = 0.f, rstd = 0.f;
        if (live) {
            mean = __ldg(a.mean + w.r);
            rstd = __ldg(a.rstd + w.r);
        }
#pragma unroll
        for (int j = 0; j < NO; ++j) {
            if (!(TPR >= 32 && j < NO - 1)) {
                xo[j].zero();
                go[j].zero();
            }
            ho[j].zero();
        }
        if (live) {
            ch.load_row(x, e, w.r, xo);
            ch.load_row(dy, e, w.r, go);
            if (MODE != kPlain && dh) ch.load_row(dh, e, w.r, ho);
        }
        if (in && !live) {
            ch.store_zeros(dx, e, true);
            if (dres) ch.store_zeros(dres, e, true);
        }
        if (TPR >= 32 && !live) continue;
        float2 s1 = make_float2(0.f, 0.f), s2 = s1;
        float2 gg[NO][4], xh[NO][4];
#pragma unroll
        for (int j = 0; j < NO; ++j) {
            float2 ga[4];
            ch.get(j, xo[j], xh[j]);
            ch.get(j, go[j], gg[j]);
            if constexpr (SHIFT) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    ga[i] = ch.any(j) ? make_float2(sp[off[2 * i] + j * TPR], sp[off[2 * i + 1] + j * TPR]) : make_float2(0.f, 0.f);
            } else {
                // behind the row: any channel's gamma will do, dy is zero there
                load_params8(a.gamma + (ch.any(j) ? ch.c0(j) : 0), ga);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                xh[j][i] = fmul2(fadd2(xh[j][i], both(-mean)), both(rstd));
                ag[j][i] = ffma2(gg[j][i], xh[j][i], ag[j][i]);
                ab[j][i] = fadd2(ab[j][i], gg[j][i]);
                gg[j][i] = fmul2(gg[j][i], ga[i]);
                s1 = fadd2(s1, gg[j][i]);
                s2 = ffma2(gg[j][i], xh[j][i], s2);
            }
        }
        const float2 sum = row_sum<TPR>(make_float2(s1.x + s1.y, s2.x + s2.y), red, flip);
        const float c1 = sum.x * inv, c2 = sum.y * inv;
#pragma unroll
        for (int j = 0; j < NO; ++j) {
            float2 d[4] = {};
            if constexpr (MODE != kPlain) ho[j].get(d);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 t = fadd2(gg[j][i], ffma2(xh[j][i], both(-c2), both(-c1)));
                gg[j][i] = MODE == kPlain ? fmul2(both(rstd), t) : ffma2(both(rstd), t, d[i]);
            }
        }
        if (MODE != kPlain && dres) ch.store_row(dres, e, live, gg);
        if constexpr (MODE != kPlain) {
            if constexpr (MODE == kFusedDrop) D.apply(static_cast<uint32_t>(e >> 3), TPR, gg);
#pragma unroll
            for (int j = 0; j < NO; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) gg[j][i] = fmul2(gg[j][i], both(a.mult));
        }
        ch.store_row(dx, e, live, gg);
    }
    if (!a.dgamma && !a.dbeta) return;
    // a warp's or block's sums by channel, in the shifted layout: dgamma at slot[at], dbeta at slot[8 Q + at]
    const int64_t Cp = (a.C + 3) / 4 * 4;
    float *pg = a.partials + static_cast<int64_t>(blockIdx.x) * 2 * Cp;
    if constexpr (TPR > 32) {  // one group: its channels straight to the partial row
#pragma unroll
        for (int j = 0; j < NO; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (ch.any(j) && ch.has(j, i)) {
                    pg[ch.c0(j) + i] = i % 2 ? ag[j][i / 2].y : ag[j][i / 2].x;
                    pg[Cp + ch.c0(j) + i] = i % 2 ? ab[j][i / 2].y : ab[j][i / 2].x;
                }
    } else {
        // warps HALF .. W-1 store, warps 0 .. HALF-1 add to them, then the HALF slots are added in
        // order; the groups of one warp take turns
        const int warp = threadIdx.x / 32;
        __syncthreads();  // SHIFT: gamma is no longer read
#pragma unroll 1
        for (int phase = 0; phase < 2; ++phase) {
            float *slot = sp + (phase == 0 ? warp - HALF : warp) * 16 * Q;
#pragma unroll 1
            for (int turn = 0; turn < 32 / TPR; ++turn) {
                const bool add = phase > 0 || turn > 0;
                if ((phase == 0) == (warp >= HALF) && static_cast<int>(threadIdx.x % 32) / TPR == turn) {
#pragma unroll
                    for (int j = 0; j < NO; ++j)
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (ch.any(j) && ch.has(j, i)) {
                                float *p = slot + off[i] + j * TPR;
                                const float vg = i % 2 ? ag[j][i / 2].y : ag[j][i / 2].x, vb = i % 2 ? ab[j][i / 2].y : ab[j][i / 2].x;
                                p[0] = add ? p[0] + vg : vg;
                                p[8 * Q] = add ? p[8 * Q] + vb : vb;
                            }
                }
                __syncwarp();
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < 2 * ch.C; c += THREADS) {
            const int which = c >= ch.C, k = which ? c - ch.C : c;
            const float *p = sp + which * 8 * Q + (k % 8) * Q + k / 8 + 1;
            float t = p[0];
#pragma unroll
            for (int q = 1; q < HALF; ++q) t += p[q * 16 * Q];
            pg[which * Cp + k] = t;
        }
    }
}

template <typename T, int TPR, int NO, int THREADS, bool SHIFT, int MODE>
cudaError_t launch(const ResidualArgs &a, int *G, cudaStream_t s) {
    constexpr int GPB = THREADS / TPR, HALF = THREADS / 64;
    const auto kern = layernorm_bwd_rows_kernel<T, TPR, NO, THREADS, SHIFT, MODE>;
    const size_t words = 8 * static_cast<size_t>((a.C + 7) / 8 + 2);
    size_t smem = SHIFT ? words * sizeof(float) : 0;
    if (TPR <= 32) smem = HALF * 2 * words * sizeof(float);
    const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(kern), static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    constexpr int kPerSm = THREADS <= 256 && TPR > 32 && NO <= 2 ? 2 : 1;
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
    return sizeof(T) == 2 ? (NO == 1 ? 1024 : NO == 2 ? 640 : NO == 3 ? 512 : NO == 4 ? 384 : 256)
                          : (NO == 1 ? 768 : NO == 2 ? 512 : NO == 3 ? 384 : 256);
}

template <typename T, int TPR, int NO, bool SHIFT>
cudaError_t launch(const ResidualArgs &a, int *G, cudaStream_t s) {
    constexpr int kThreads = TPR > 32 ? TPR : threads_for<T>(NO);
    if (a.thr) return launch<T, TPR, NO, kThreads, SHIFT, kFusedDrop>(a, G, s);
    if (a.dh || a.dres || a.mult != 1.f) return launch<T, TPR, NO, kThreads, SHIFT, kFused>(a, G, s);
    return launch<T, TPR, NO, kThreads, SHIFT, kPlain>(a, G, s);
}

template <typename T, bool SHIFT>
cudaError_t launch_octets(const ResidualArgs &a, int64_t n, int *G, cudaStream_t s) {
    if (n <= 8) return launch<T, 8, 1, SHIFT>(a, G, s);
    if (n <= 16) return launch<T, 8, 2, SHIFT>(a, G, s);
    if (n <= 32) return launch<T, 16, 2, SHIFT>(a, G, s);
    if (n <= 64) return launch<T, 32, 2, SHIFT>(a, G, s);
    if (n <= 96) return launch<T, 32, 3, SHIFT>(a, G, s);
    if (n <= 128) return launch<T, 32, 4, SHIFT>(a, G, s);
    if (n <= 160) return launch<T, 32, 5, SHIFT>(a, G, s);
    if (n <= 256) return launch<T, 256, 1, SHIFT>(a, G, s);
    if (n <= 512) return launch<T, 256, 2, SHIFT>(a, G, s);
    if (n <= 768) return launch<T, 384, 2, SHIFT>(a, G, s);
    if (n <= 1024) return launch<T, 512, 2, SHIFT>(a, G, s);
    return cudaErrorNotSupported;
}

// cudaErrorNotSupported: no row kernel for these sizes or this alignment.
template <typename T>
cudaError_t launch_rows(const ResidualArgs &a, int *G, cudaStream_t s) {
    if (!a.vec_oct || a.C > 8192 || a.B * a.T >= (int64_t(1) << 30) || a.thr >= 65536u ||
        a.B * a.T * a.C >= (int64_t(1) << 35)) return cudaErrorNotSupported;
    if (a.C % 8 == 0 && a.gamma && reinterpret_cast<uintptr_t>(a.gamma) % 32 == 0) return launch_octets<T, false>(a, a.C / 8, G, s);
    return launch_octets<T, true>(a, (a.C + 14) / 8, G, s);  // a row may touch 7 elements before its first
}

}  // namespace lnb
}  // namespace dwk
