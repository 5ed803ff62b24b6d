// Layer norm backward, alone or fused with the gradients of dropout and the residual add:
//   xh = (x - mean) rstd,  g = dy gamma,  ds = dh + rstd (g - mean_c(g) - xh mean_c(g xh)),
//   dres = ds,  dx = [kept] mult ds,  dgamma = sum_rows dy xh,  dbeta = sum_rows dy.
// Two kernels:
//  1. row kernel: every block walks rows and adds their dgamma/dbeta terms to a partial row of its
//     own in the workspace, [G][2][ceil4(C)];
//  2. finalize kernel: the partial rows added in a fixed order.
// No atomics: bitwise reproducible for given sizes, pointer alignments and NULL operands on a given GPU model
// (alignment and gamma choose the kernel, which orders a row's and the rows' sums).
#include "dw_internal.h"
#include "residual.cuh"

namespace dwk {
namespace {

// Partial rows: at most two blocks on each of 148 SMs, and at most 64 MiB of them (at least one).
constexpr int kMaxPartialRows = 296;

// Any C, any alignment: a block per row, two passes over it, one element at a time; the block's
// partial row lives in the workspace (a thread only touches its own columns, so no synchronization is
// needed).  4096 rows of 12288 bf16 at alignments that differ, so that the wide kernel does not take them: 691 us
// (0.07 of the measured copy bandwidth).
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
        const float mean = a.mean[r], rstd = a.rstd[r];
        float2 acc = make_float2(0.f, 0.f);
        for (int64_t c = threadIdx.x; c < a.C; c += 256) {
            const float xh = (load1(x + base + c) - mean) * rstd, d = load1(dy + base + c);
            const float g = a.gamma ? d * load_global(a.gamma + c) : d;
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
            const float g = a.gamma ? d * load_global(a.gamma + c) : d;
            float ds = rstd * (g - c1 - xh * c2);
            if (dh) ds += load1(dh + e);
            if (dres) store1(dres + e, ds);
            const bool keep = a.thr == 0 || R.kept(static_cast<uint64_t>(e), a.thr);
            store1(dx + e, keep ? a.mult * ds : 0.f);
        }
    }
}

// Rows too long for registers (C a multiple of 8, the block's dgamma and dbeta in shared memory: up to
// 25600 channels): a block per row, every thread on octets of its own; the second pass reads x and dy
// again (L2).  4096 rows of 12288 bf16 123 us (0.37 of the measured copy bandwidth, general kernel 691 us);
// 2048 with dropout and dh 84 us (0.46); 1024 rows of 25600, one block per SM, 111 us (0.22).  Bound by the
// wait for the loads: a row has few octets per thread.  Two or three octets at a time, as in the forward,
// spill at the 64 registers of two blocks per SM and are slower (136 and 152 us).
constexpr int kWideThreads = 512;
template <typename T>
__global__ void __launch_bounds__(kWideThreads, 2)
layernorm_bwd_wide_kernel(const ResidualArgs a) {
    constexpr int W = kWideThreads / 32;
    __shared__ float2 red[2][W];
    extern __shared__ float4 part[];  // dgamma, then dbeta: [2][n] each, see the forward
    launch_dependents();
    grid_dependency_wait();
    Dropper D;
    if (a.thr) D.start(a.rng, a.thr);
    const T *x = static_cast<const T *>(a.x), *dy = static_cast<const T *>(a.dy), *dh = static_cast<const T *>(a.dh);
    T *dx = static_cast<T *>(a.dx), *dres = static_cast<T *>(a.dres);
    const int n = static_cast<int>(a.C / 8);
    const int64_t rows = a.B * a.T;
    const float inv = 1.f / static_cast<float>(a.C);
    for (int v = threadIdx.x; v < n; v += kWideThreads)
#pragma unroll
        for (int k = 0; k < 4; ++k) part[k * n + v] = make_float4(0.f, 0.f, 0.f, 0.f);
    int flip = 0;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const int64_t base = r * a.C, b = r / a.T;
        if (r - b * a.T >= clamp_len(a.lengths, b, a.T)) {
            const float2 zero[4] = {};
            for (int v = threadIdx.x; v < n; v += kWideThreads) {
                Oct<T>::store(dx + base + 8 * v, zero);
                if (dres) Oct<T>::store(dres + base + 8 * v, zero);
            }
            continue;
        }
        const float mean = a.mean[r], rstd = a.rstd[r];
        float2 s1 = make_float2(0.f, 0.f), s2 = s1;
        for (int v = threadIdx.x; v < n; v += kWideThreads) {
            Oct<T> xo, go;
            float2 xh[4], g[4], ga[4];
            xo.load(x + base + 8 * v);
            go.load(dy + base + 8 * v);
            any_params8(a.gamma, 1.f, 8 * v, ga);
            xo.get(xh);
            go.get(g);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float4 pg = part[k * n + v], pb = part[(2 + k) * n + v];
                float2 t[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) t[i] = fmul2(fadd2(xh[2 * k + i], both(-mean)), both(rstd));
                const float2 d0 = g[2 * k], d1 = g[2 * k + 1];
                const float2 q0 = ffma2(d0, t[0], make_float2(pg.x, pg.y));
                const float2 q1 = ffma2(d1, t[1], make_float2(pg.z, pg.w));
                part[k * n + v] = make_float4(q0.x, q0.y, q1.x, q1.y);
                part[(2 + k) * n + v] = make_float4(pb.x + d0.x, pb.y + d0.y, pb.z + d1.x, pb.w + d1.y);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 gg = fmul2(g[2 * k + i], ga[2 * k + i]);
                    s1 = fadd2(s1, gg);
                    s2 = ffma2(gg, t[i], s2);
                }
            }
        }
        const float2 c = block_sum2<W>(make_float2(s1.x + s1.y, s2.x + s2.y), red[flip]);
        flip ^= 1;
        const float c1 = c.x * inv, c2 = c.y * inv;
        for (int v = threadIdx.x; v < n; v += kWideThreads) {
            Oct<T> xo, go, ho;
            float2 f[1][4], g[4], ga[4], d[4];
            xo.load(x + base + 8 * v);
            go.load(dy + base + 8 * v);
            ho.zero();
            if (dh) ho.load(dh + base + 8 * v);
            any_params8(a.gamma, 1.f, 8 * v, ga);
            xo.get(f[0]);
            go.get(g);
            ho.get(d);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 xh = fmul2(fadd2(f[0][i], both(-mean)), both(rstd));
                const float2 t = fadd2(fmul2(g[i], ga[i]), ffma2(xh, both(-c2), both(-c1)));
                f[0][i] = ffma2(both(rstd), t, d[i]);
            }
            if (dres) Oct<T>::store(dres + base + 8 * v, f[0]);
            if (a.thr) D.apply(static_cast<uint32_t>((base + 8 * v) >> 3), 0, f);
#pragma unroll
            for (int i = 0; i < 4; ++i) f[0][i] = fmul2(f[0][i], both(a.mult));
            Oct<T>::store(dx + base + 8 * v, f[0]);
        }
    }
    if (!a.dgamma && !a.dbeta) return;
    float4 *pg = reinterpret_cast<float4 *>(a.partials + static_cast<int64_t>(blockIdx.x) * 2 * a.C);
    for (int v = threadIdx.x; v < n; v += kWideThreads)
#pragma unroll
        for (int k = 0; k < 4; ++k) pg[k / 2 * 2 * n + 2 * v + k % 2] = part[k * n + v];
}

template <typename T>
cudaError_t launch_wide(const ResidualArgs &a, int *G, cudaStream_t s) {
    const int64_t smem = a.C * 8;
    static SmemGrant grant;
    const void *const kernel = reinterpret_cast<const void *>(layernorm_bwd_wide_kernel<T>);
    const cudaError_t e = grant(kernel, static_cast<int>(smem), -1);
    if (e != cudaSuccess) return e;
    const int64_t most = static_cast<int64_t>(sm_count()) * (smem <= 100 * 1024 ? 2 : 1);
    *G = static_cast<int>(a.G < most ? a.G : most);
    return launch_programmatic(layernorm_bwd_wide_kernel<T>, dim3(static_cast<unsigned>(*G)), dim3(kWideThreads),
                               static_cast<size_t>(smem), s, a);
}

// dgamma[c], dbeta[c] = the G partial rows' entries in a fixed order.  A block covers 16 entries of the
// 2 ceil4(C) with 8 row groups; group q adds rows q, q + 8, ... in order, its loads in flight together,
// then the 8 group sums are added in a fixed tree.  Blocks of 128 threads with 32 registers fit
// beside the row kernel's on an SM, so they are resident and waiting when it ends (and read the partial
// rows, written meanwhile, from L2).
__global__ void __launch_bounds__(128, 16)
layernorm_bwd_finalize_kernel(const float *partials, float *dgamma, float *dbeta, int G, int64_t C) {
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
        for (int i = 0; i < 20; ++i) v[i] = live && r0 + q + 8 * i < G ? __ldcg(p + (r0 + 8 * i) * E) : 0.f;
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
        if (e == cudaErrorNotSupported && row_kernels_serve(a) && a.phase == 0 && a.C % 8 == 0 && a.C <= 25600)
            e = with_dtype(a.dtype, [&](auto t) { return launch_wide<decltype(t)>(a, &G, s); });
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
