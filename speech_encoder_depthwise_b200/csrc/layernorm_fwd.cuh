// The row kernel of layer norm forward (alone, or behind dropout and the residual add) and its
// dispatch; instantiated per element type in layernorm_fwd_{bf16,f16,f32}.cu.
#pragma once

#include "dw_internal.h"
#include "residual.cuh"

namespace dwk {
namespace lnf {

constexpr int kThreads = 256;

// Three blocks where their 80 registers a thread suffice without spills (32x1500x255 bf16 12.4 us instead
// of 13.7); float32 and the wider shapes of few rows lose by it (32x1500x1024 float32 60.5 / 55.9 us, 1500 rows of
// 512 bf16 2.4 / 2.0).
constexpr int blocks_per_sm(int TPR, int NO, int element) {
    return NO == 1 || (NO == 2 && TPR <= 16 && element == 2) ? 3 : 2;
}

enum Mode { kPlain, kFused, kFusedDrop };  // layer norm alone; with residual add; with dropout too

// TPR threads hold a row's NO octets each in registers: one read of x (and res), the mean, then
// the variance of the centred values, then the outputs; the next row's octets are requested first.
// SHIFT: C or the tensors' address not a multiple of 8 elements, or a parameter missing or misaligned;
// gamma and beta then come from shared memory instead of L1.
//
// Bound by HBM: 8 flops an element against 4 bytes.  What it took to get there was instructions, not
// bytes in flight (a ring of bulk copies four rows deep was slower than plain loads): packed float32
// arithmetic, rows shared by half a warp so that two rows share one reduction's shuffles, modes and
// widths as instances instead of branches: 413 -> 140 instructions a row of 512 bf16.
// Measured (graph replay, cold inputs; fraction of the measured copy bandwidth): 64x3000x1024 bf16
// 111.7 us (0.94), 32x1500x1024 float32 56.0 us (0.94), 16x1500x512 bf16 9.9 us (0.66: about 3.4 us
// of launch, first load and last store), 64 rows of 512 1.6 us; with dropout and residual 32x1500x1024
// bf16 59.4 us (0.89), 16x1500x512 17.0 us (0.77), 16x1499x1023 fp16 34.3 us (0.76; 36.6 with edges converted
// where they are loaded, which waits for them).
template <typename T, int TPR, int NO, bool SHIFT, int MODE>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(TPR, NO, sizeof(T)))
layernorm_fwd_rows_kernel(const ResidualArgs a) {
    constexpr int GPB = kThreads / TPR;
    static_assert(TPR <= 32 || GPB <= 15, "a named barrier per group, numbers 1 to 15");
    __shared__ float red_all[GPB][2 * (TPR > 32 ? TPR / 32 : 1)];
    extern __shared__ float2 sp[];  // SHIFT: {gamma, beta} per channel
    launch_dependents();
    const int g = threadIdx.x / TPR, grid = gridDim.x, rows = static_cast<int>(a.B * a.T);
    const T *x = static_cast<const T *>(a.x), *res = MODE == kPlain ? nullptr : static_cast<const T *>(a.res);
    T *y = static_cast<T *>(a.y), *h = MODE == kPlain ? nullptr : static_cast<T *>(a.h);
    float *red = red_all[g];
    const int first = blockIdx.x + grid * g;
    Channels<T, TPR, NO, SHIFT> ch;
    ch.start(static_cast<int>(a.C), first, a.phase);
    int off[8];
    float2 pe = make_float2(0.f, 0.f);
    // the only row of each group on its way into L2 while the previous kernel drains (1500 rows of 512 bf16:
    // 2.0 us instead of 2.2; with more rows a group it gains nothing)
    if (first < rows && rows <= grid * GPB) {
        ch.prefetch_row(x, first);
        if (res) ch.prefetch_row(res, first);
        if (ch.lane == 0 && a.lengths) prefetch_l2(a.lengths + first / static_cast<int>(a.T));
    }
    grid_dependency_wait();
    if constexpr (SHIFT) {
        const int Q = shifted_q(ch.C);
        for (int c = threadIdx.x; c < ch.C; c += kThreads)
            sp[shifted_at(c, Q)] = make_float2(a.gamma ? load_global(a.gamma + c) : 1.f,
                                               a.beta ? load_global(a.beta + c) : 0.f);
#pragma unroll
        for (int i = 0; i < 8; ++i) off[i] = shifted_at(ch.head + i, Q) + ch.lane;
        __syncthreads();
        if (ch.edge()) pe = sp[shifted_at(ch.ce, Q)];
    }
    Dropper D;
    if constexpr (MODE == kFusedDrop) D.start(a.rng, a.thr);
    const float inv = 1.f / static_cast<float>(ch.C);
    int flip = 0;
    Oct<T> xo[NO], ro[NO];
    T xe = zero1<T>(), re = xe;  // as loaded: a conversion in `fetch` would wait for the load
    const auto fetch = [&](const RowWalk &w, bool any = false) {
        if (!w.in() || !(any || w.valid())) return;
        const int64_t e = ch.at(w.r);
        ch.load_row(x, e, xo);
        if (MODE != kPlain && res) ch.load_row(res, e, ro);
        if (ch.edge()) {
            xe = x[ch.edge_at(w.r)];
            if (MODE != kPlain && res) re = res[ch.edge_at(w.r)];
        }
    };
#pragma unroll
    for (int j = 0; j < NO; ++j) {
        xo[j].zero();
        ro[j].zero();
    }
    // the next row is requested ahead where two rows fit 128 registers a thread (five octets with the residual spill
    // up to 36 bytes)
    constexpr bool kAhead = NO * sizeof(T) * (MODE == kPlain ? 1 : 2) <= 16;
    // few rows of a 16-bit type behind a residual add: gamma and beta together with the row, since their loads can
    // pass neither the sums' barriers nor the stores of h (600 rows of 1024 bf16 with dropout 2.95 us, behind them
    // 3.07; 64 rows of 512 1.94 / 2.14).  float32 lacks the registers (16x1500x1024 60.6 / 59.6), and without h it
    // gains nothing (1500 rows of 512 2.04 / 2.02)
    constexpr bool kEarly = !SHIFT && MODE != kPlain && sizeof(T) == 2 && NO == 2 && TPR >= 32;
    RowWalk w;
    w.start(a.lengths, first, grid * GPB, rows, static_cast<int>(a.T));
    if (kAhead) fetch(w, true);  // whatever its length says: the two loads' latencies overlap
    // groups of one warp walk together (their sums share its shuffles): until the first one is done
    int lead = TPR < 32 ? blockIdx.x + grid * (threadIdx.x / 32 * (32 / TPR)) : first;
    for (; lead < rows; lead += w.step) {
        if (!kAhead) fetch(w);
        const bool in = w.in(), live = in && w.valid();
        const int r = w.r;
        const int64_t e = ch.at(r);
        float2 v[NO][4], sum = make_float2(0.f, 0.f);
        float ve = 0.f;
        float2 ga[NO][4], be[NO][4];
        const auto params = [&](int j) {
            load_params8(a.gamma + ch.c0(j), ga[j]);
            load_params8(a.beta + ch.c0(j), be[j]);
        };
        if constexpr (kEarly) {
#pragma unroll
            for (int j = 0; j < NO; ++j)
                if (ch.any(j)) params(j);
        }
#pragma unroll
        for (int j = 0; j < NO; ++j) xo[j].get(v[j]);
        if constexpr (SHIFT) ve = load1(&xe);
        if constexpr (MODE == kFusedDrop) {
            if constexpr (SHIFT) D.apply(static_cast<uint32_t>(e >> 3), TPR, v, ch.edge_at(r), ve);
            else D.apply(static_cast<uint32_t>(e >> 3), TPR, v);
        }
#pragma unroll
        for (int j = 0; j < NO; ++j) {
            if constexpr (MODE != kPlain) {
                float2 p[4];
                ro[j].get(p);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[j][i] = ffma2(both(a.mult), v[j][i], p[i]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) sum = fadd2(sum, v[j][i]);
        }
        if constexpr (SHIFT) {
            if constexpr (MODE != kPlain) ve = fmaf(a.mult, ve, load1(&re));
            sum.x += ve;  // zero where the thread has no edge channel
        }
        w.next();
        if (kAhead) fetch(w);
        if (in && !live) {
            ch.store_zeros(y, r);
            if (h) ch.store_zeros(h, r);
            if (ch.lane == 0) {
                if (a.mean) a.mean[r] = 0.f;
                if (a.rstd) a.rstd[r] = 0.f;
            }
        }
        if (TPR >= 32 && !live) continue;
        const float mean = row_sum<TPR>(sum.x + sum.y, red, flip) * inv;
        if (MODE != kPlain && h && live) {
            ch.store_row(h, e, v);
            if (ch.edge()) store1(h + ch.edge_at(r), ve);
        }
        float2 ss = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < NO; ++j) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[j][i] = fadd2(v[j][i], both(-mean));
            ch.clear_behind(j, v[j]);
#pragma unroll
            for (int i = 0; i < 4; ++i) ss = ffma2(v[j][i], v[j][i], ss);
        }
        if constexpr (SHIFT) {
            ve = ch.edge() ? ve - mean : 0.f;
            ss.x = fmaf(ve, ve, ss.x);
        }
        const float rstd = rsqrt_newton(fmaf(row_sum<TPR>(ss.x + ss.y, red, flip), inv, a.eps));
        if (!live) continue;
#pragma unroll
        for (int j = 0; j < NO; ++j) {
            if (!ch.any(j)) continue;
            if constexpr (SHIFT) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 p = sp[off[2 * i] + j * TPR], q = sp[off[2 * i + 1] + j * TPR];
                    const float2 t = fmul2(v[j][i], both(rstd));
                    v[j][i] = make_float2(fmaf(t.x, p.x, p.y), fmaf(t.y, q.x, q.y));
                }
            } else {
                if constexpr (!kEarly) params(j);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[j][i] = ffma2(fmul2(v[j][i], both(rstd)), ga[j][i], be[j][i]);
            }
        }
        ch.store_row(y, e, v);  // behind every octet's gamma and beta, whose loads cannot pass a store
        if (ch.edge()) store1(y + ch.edge_at(r), fmaf(ve * rstd, pe.x, pe.y));
        if (ch.lane == 0) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
    }
}

template <typename T, int TPR, int NO, bool SHIFT, int MODE>
cudaError_t launch(const ResidualArgs &a, cudaStream_t s) {
    constexpr int GPB = kThreads / TPR;
    const auto kern = layernorm_fwd_rows_kernel<T, TPR, NO, SHIFT, MODE>;
    const size_t smem = SHIFT ? 8 * shifted_q(static_cast<int>(a.C)) * sizeof(float2) : 0;
    static const int regs_per_sm = [&] {
        int n = 0;
        return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, kThreads, 0) == cudaSuccess && n > 0 ? n : 1;
    }();
    if (SHIFT) {
        static SmemGrant grant;
        const cudaError_t e = grant(reinterpret_cast<const void *>(kern), static_cast<int>(smem), -1);
        if (e != cudaSuccess) return e;
    }
    int64_t per_sm = regs_per_sm;
    if (SHIFT && per_sm > 220 * 1024 / static_cast<int64_t>(smem + 1024)) per_sm = 220 * 1024 / (smem + 1024);
    const int64_t rows = a.B * a.T, need = (rows + GPB - 1) / GPB;
    int64_t grid = sm_count() * per_sm;
    constexpr int kMult = GPB >= 8 ? 1 : 8 / GPB;
    if (grid > need) grid = need;
    else if (SHIFT) grid = grid / kMult * kMult;  // a group's rows stay 8 k apart
    return launch_programmatic(kern, dim3(static_cast<unsigned>(grid)), dim3(kThreads), smem, s, a);
}

template <typename T, int TPR, int NO, bool SHIFT>
cudaError_t launch(const ResidualArgs &a, cudaStream_t s) {
    if (a.thr) return launch<T, TPR, NO, SHIFT, kFusedDrop>(a, s);
    if (a.res || a.h || a.mult != 1.f) return launch<T, TPR, NO, SHIFT, kFused>(a, s);
    return launch<T, TPR, NO, SHIFT, kPlain>(a, s);
}

// n: the octets of a row, C / 8 rounded down (edges need 16 lanes).  Two octets a thread for float32
// and for few rows (up to 1024 octets per SM), where the latency of one row counts; three to five of a
// 16-bit type otherwise, which share the sums' shuffles and gamma's loads among more channels.  Both
// ways, us: float32 32x1500x1024 56.4 / 62.7; bf16 64 rows of 512 1.59 / 1.93, 1024 rows of
// 1024 2.20 / 2.70; 16384 rows of 1024 15.5 / 13.0, 16x1500x512 11.1 / 9.9.
template <typename T, bool SHIFT>
cudaError_t launch_octets(const ResidualArgs &a, int64_t n, cudaStream_t s) {
    if (!SHIFT && n <= 8) return launch<T, 8, 1, false>(a, s);
    if (sizeof(T) == 4 || a.B * a.T * n <= 1024 * static_cast<int64_t>(sm_count())) {
        if (n <= 16) return launch<T, 16, 1, SHIFT>(a, s);
        if (n <= 32) return launch<T, 32, 1, SHIFT>(a, s);
        if (n <= 64) return launch<T, 32, 2, SHIFT>(a, s);
        if (n <= 128) return launch<T, 64, 2, SHIFT>(a, s);
        if (n <= 192) return launch<T, 64, 3, SHIFT>(a, s);
        if (n <= 256) return launch<T, 128, 2, SHIFT>(a, s);
        if (n <= 384) return launch<T, 128, 3, SHIFT>(a, s);
        if (n <= 512) return launch<T, 256, 2, SHIFT>(a, s);
        if (n <= 768) return launch<T, 256, 3, SHIFT>(a, s);
        if (n <= 1024) return launch<T, 256, 4, SHIFT>(a, s);
        return cudaErrorNotSupported;
    }
    if constexpr (sizeof(T) == 2) {
        if constexpr (!SHIFT) {
            if (n <= 16) return launch<T, 8, 2, SHIFT>(a, s);
            if (n <= 24) return launch<T, 8, 3, SHIFT>(a, s);
            if (n <= 32) return launch<T, 8, 4, SHIFT>(a, s);
        } else {
            if (n <= 16) return launch<T, 16, 1, SHIFT>(a, s);
            if (n <= 32) return launch<T, 16, 2, SHIFT>(a, s);
        }
        if (n <= 48) return launch<T, 16, 3, SHIFT>(a, s);
        if (n <= 64) return launch<T, 16, 4, SHIFT>(a, s);
        if (n <= 80) return launch<T, 16, 5, SHIFT>(a, s);
        if (n <= 96) return launch<T, 32, 3, SHIFT>(a, s);
        if (n <= 128) return launch<T, 32, 4, SHIFT>(a, s);
        if (n <= 192) return launch<T, 64, 3, SHIFT>(a, s);
        if (n <= 256) return launch<T, 64, 4, SHIFT>(a, s);
        if (n <= 384) return launch<T, 128, 3, SHIFT>(a, s);
        if (n <= 512) return launch<T, 128, 4, SHIFT>(a, s);
        if (n <= 768) return launch<T, 256, 3, SHIFT>(a, s);
        if (n <= 1024) return launch<T, 256, 4, SHIFT>(a, s);
    }
    return cudaErrorNotSupported;
}

// cudaErrorNotSupported: no row kernel for these sizes or this alignment.
template <typename T>
cudaError_t launch_rows(const ResidualArgs &a, cudaStream_t s) {
    if (!row_kernels_serve(a)) return cudaErrorNotSupported;
    const bool params32 = a.gamma && a.beta && reinterpret_cast<uintptr_t>(a.gamma) % 32 == 0 &&
                          reinterpret_cast<uintptr_t>(a.beta) % 32 == 0;
    if (a.C % 8 == 0 && a.phase == 0 && params32) return launch_octets<T, false>(a, a.C / 8, s);
    return launch_octets<T, true>(a, a.C / 8, s);
}

}  // namespace lnf
}  // namespace dwk
