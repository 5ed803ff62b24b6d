// The row kernel of layer norm forward (alone, or behind dropout and the residual add) and its
// dispatch; instantiated per element type in layernorm_fwd_{bf16,f16,f32}.cu.
#pragma once

#include "dw_internal.h"
#include "residual.cuh"

namespace dwk {
namespace lnf {

constexpr int threads_for(int TPR) { return TPR > 256 ? TPR : 256; }

enum Mode { kPlain, kFused, kFusedDrop };  // layer norm alone; with residual add; with dropout too

// TPR threads hold a row's NO octets each in registers: one read of x (and res), the mean, then
// the variance of the centred values, then the outputs; the next row's octets are requested first.
// SHIFT: rows that do not start on an octet (C not a multiple of 8), or a parameter missing or
// misaligned; gamma and beta then come from shared memory instead of L1.
template <typename T, int TPR, int NO, bool SHIFT, int MODE>
__global__ void __launch_bounds__(threads_for(TPR), 2)
layernorm_fwd_rows_kernel(const ResidualArgs a) {
    constexpr int kThreads = threads_for(TPR), GPB = kThreads / TPR;
    __shared__ float red[2 * (TPR > 32 ? TPR / 32 : 1)];
    extern __shared__ float2 sp[];  // SHIFT: {gamma, beta} per channel
    launch_dependents();
    const int g = threadIdx.x / TPR, grid = gridDim.x, rows = static_cast<int>(a.B * a.T);
    const T *x = static_cast<const T *>(a.x), *res = MODE == kPlain ? nullptr : static_cast<const T *>(a.res);
    T *y = static_cast<T *>(a.y), *h = MODE == kPlain ? nullptr : static_cast<T *>(a.h);
    using Ch = Channels<T, TPR, NO, SHIFT>;
    __shared__ __align__(32) T scratch[SHIFT ? kThreads / Ch::kGroup * 16 : 1];
    Ch ch;
    const int first = blockIdx.x + grid * g;
    ch.start(static_cast<int>(a.C), rows, first, scratch);
    int off[8];
    grid_dependency_wait();
    if constexpr (SHIFT) {
        const int Q = shifted_q(ch.C);
        for (int i = threadIdx.x; i < 8 * Q; i += kThreads) {
            const int c = i / Q + 8 * (i % Q - 1);
            const bool in = c >= 0 && c < ch.C;
            sp[i] = make_float2(!in ? 0.f : a.gamma ? __ldg(a.gamma + c) : 1.f, in && a.beta ? __ldg(a.beta + c) : 0.f);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) off[i] = shifted_off(i, ch.s, Q) + ch.lane;
        __syncthreads();
    }
    Dropper D;
    if constexpr (MODE == kFusedDrop) D.start(a.rng, a.thr);
    const float inv = 1.f / static_cast<float>(ch.C);
    int flip = 0;
    Oct<T> xo[NO], ro[NO];
    const auto fetch = [&](const RowWalk &w) {
        if (!w.in() || !w.valid()) return;
        const int64_t e = ch.at(w.r);
        ch.load_row(x, e, w.r, xo);
        if (MODE != kPlain && res) ch.load_row(res, e, w.r, ro);
    };
#pragma unroll
    for (int j = 0; j < NO; ++j) {
        xo[j].zero();
        ro[j].zero();
    }
    // the next row is requested ahead where two rows fit 128 registers a thread
    constexpr bool kAhead = NO * sizeof(T) * (MODE == kPlain ? 1 : 2) <= 16;
    RowWalk w;
    w.start(a.lengths, first, grid * GPB, rows, static_cast<int>(a.T));
    if (kAhead) fetch(w);
    // groups of one warp walk together (their sums share its shuffles): until the first one is done
    int lead = TPR < 32 ? blockIdx.x + grid * (threadIdx.x / 32 * (32 / TPR)) : first;
    for (; lead < rows; lead += w.step) {
        if (!kAhead) fetch(w);
        const bool in = w.in(), live = in && w.valid();
        const int r = w.r;
        const int64_t e = ch.at(r);
        float2 v[NO][4], sum = make_float2(0.f, 0.f);
        if constexpr (MODE == kFusedDrop) {
#pragma unroll
            for (int j = 0; j < NO; ++j) ch.get(j, xo[j], v[j]);
            D.apply(static_cast<uint32_t>(e >> 3), TPR, v);
        }
#pragma unroll
        for (int j = 0; j < NO; ++j) {
            if constexpr (MODE != kFusedDrop) ch.get(j, xo[j], v[j]);
            if constexpr (MODE != kPlain) {
                float2 p[4];
                ch.get(j, ro[j], p);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[j][i] = ffma2(both(a.mult), v[j][i], p[i]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) sum = fadd2(sum, v[j][i]);
        }
        w.next();
        if (kAhead) fetch(w);
        if (in && !live) {
            ch.store_zeros(y, e, true);
            if (h) ch.store_zeros(h, e, true);
            if (ch.lane == 0) {
                if (a.mean) a.mean[r] = 0.f;
                if (a.rstd) a.rstd[r] = 0.f;
            }
        }
        if (TPR >= 32 && !live) continue;
        const float mean = row_sum<TPR>(sum.x + sum.y, red, flip) * inv;
        if (MODE != kPlain && h) ch.store_row(h, e, live, v);
        float2 ss = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < NO; ++j) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[j][i] = fadd2(v[j][i], both(-mean));
            ch.clear_outside(j, v[j]);
#pragma unroll
            for (int i = 0; i < 4; ++i) ss = ffma2(v[j][i], v[j][i], ss);
        }
        const float rstd = rsqrt_newton(fmaf(row_sum<TPR>(ss.x + ss.y, red, flip), inv, a.eps));
#pragma unroll
        for (int j = 0; j < NO; ++j) {
            const bool any = ch.any(j);  // behind the row: any channel's parameters will do
            if constexpr (SHIFT) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 p = sp[any ? off[2 * i] + j * TPR : 0], q = sp[any ? off[2 * i + 1] + j * TPR : 0];
                    const float2 t = fmul2(v[j][i], both(rstd));
                    v[j][i] = make_float2(fmaf(t.x, p.x, p.y), fmaf(t.y, q.x, q.y));
                }
            } else {
                float2 ga[4], be[4];
                load_params8(a.gamma + (any ? ch.c0(j) : 0), ga);
                load_params8(a.beta + (any ? ch.c0(j) : 0), be);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[j][i] = ffma2(fmul2(v[j][i], both(rstd)), ga[i], be[i]);
            }
        }
        ch.store_row(y, e, live, v);
        if (ch.lane == 0 && live) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
    }
}

template <typename T, int TPR, int NO, bool SHIFT, int MODE>
cudaError_t launch(const ResidualArgs &a, cudaStream_t s) {
    constexpr int kThreads = threads_for(TPR), GPB = kThreads / TPR;
    const auto kern = layernorm_fwd_rows_kernel<T, TPR, NO, SHIFT, MODE>;
    const size_t smem = SHIFT ? 8 * ((a.C + 7) / 8 + 2) * sizeof(float2) : 0;
    static const int regs_per_sm = [&] {
        int n = 0;
        return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, kThreads, 0) == cudaSuccess && n > 0 ? n : 1;
    }();
    if (SHIFT) {
        const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(kern), static_cast<int>(smem));
        if (e != cudaSuccess) return e;
    }
    int64_t per_sm = regs_per_sm;
    if (SHIFT && per_sm > 220 * 1024 / static_cast<int64_t>(smem + 1024)) per_sm = 220 * 1024 / (smem + 1024);
    const int64_t rows = a.B * a.T, most = sm_count() * per_sm * GPB;  // most: rows in flight
    const int64_t passes = (rows + most - 1) / most;
    int64_t grid = (rows + passes * GPB - 1) / (passes * GPB);
    if (SHIFT && passes > 1 && GPB % 8 != 0) grid = (grid + 7) / 8 * 8;  // a group's rows stay 8 k apart
    return launch_programmatic(kern, dim3(static_cast<unsigned>(grid)), dim3(kThreads), smem, s, a);
}

template <typename T, int TPR, int NO, bool SHIFT>
cudaError_t launch(const ResidualArgs &a, cudaStream_t s) {
    if (a.thr) return launch<T, TPR, NO, SHIFT, kFusedDrop>(a, s);
    if (a.res || a.h || a.mult != 1.f) return launch<T, TPR, NO, SHIFT, kFused>(a, s);
    return launch<T, TPR, NO, SHIFT, kPlain>(a, s);
}

template <typename T, bool SHIFT>
cudaError_t launch_octets(const ResidualArgs &a, int64_t n, cudaStream_t s) {
    if (n <= 8) return launch<T, 8, 1, SHIFT>(a, s);
    if (n <= 16) return launch<T, 8, 2, SHIFT>(a, s);
    if (n <= 24) return launch<T, 8, 3, SHIFT>(a, s);
    if (n <= 32) return launch<T, 8, 4, SHIFT>(a, s);
    if (n <= 48) return launch<T, 16, 3, SHIFT>(a, s);
    if (n <= 64) return launch<T, 16, 4, SHIFT>(a, s);
    if (n <= 80) return launch<T, 16, 5, SHIFT>(a, s);
    if (n <= 96) return launch<T, 32, 3, SHIFT>(a, s);
    if (n <= 128) return launch<T, 32, 4, SHIFT>(a, s);
    if (n <= 160) return launch<T, 32, 5, SHIFT>(a, s);
    if (n <= 256) return launch<T, 256, 1, SHIFT>(a, s);
    if (n <= 512) return launch<T, 256, 2, SHIFT>(a, s);
    if (n <= 768) return launch<T, 256, 3, SHIFT>(a, s);
    if (n <= 1024) return launch<T, 256, 4, SHIFT>(a, s);
    return cudaErrorNotSupported;
}

// cudaErrorNotSupported: no row kernel for these sizes or this alignment.
template <typename T>
cudaError_t launch_rows(const ResidualArgs &a, cudaStream_t s) {
    if (!a.vec_oct || a.C > 8192 || a.B * a.T >= (int64_t(1) << 30) || a.thr >= 65536u ||
        a.B * a.T * a.C >= (int64_t(1) << 35)) return cudaErrorNotSupported;
    const bool params32 = a.gamma && a.beta && reinterpret_cast<uintptr_t>(a.gamma) % 32 == 0 && reinterpret_cast<uintptr_t>(a.beta) % 32 == 0;
    if (a.C % 8 == 0 && params32) return launch_octets<T, false>(a, a.C / 8, s);
    return launch_octets<T, true>(a, (a.C + 14) / 8, s);  // a row may touch 7 elements before its first
}

}  // namespace lnf
}  // namespace dwk
