// Layer norm forward, alone or fused behind dropout and the residual add:
//   s = res + [kept] mult x,  h = s rounded,  y = (s - mean) rstd gamma + beta  over the C channels.
// Statistics in float32: the mean first, then the variance of the centred values (no
// E[s^2] - mean^2 cancellation).
#include "dw_internal.h"
#include "residual.cuh"

namespace dwk {
namespace {

// Any C, any alignment: a block per row, three passes over the row (the second and third hit L1/L2),
// s computed anew in each, one element at a time.  Bound by instructions: 4096 rows of 12289 bf16
// 178 us (0.17 of the measured copy bandwidth), with dropout a whole mask block per element and pass.
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
            const float ga = a.gamma ? load_global(a.gamma + c) : 1.f, be = a.beta ? load_global(a.beta + c) : 0.f;
            store1(y + base + c, fmaf((v - mean) * rstd, ga, be));
        }
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
    }
}

// Rows too long for registers (C a multiple of 8, s in shared memory as float32: up to 51200 channels):
// a block per row, every thread on octets of its own, so the sums' barriers are the only ones.  The loads
// of U octets are in flight together: bound by the wait for them at the start of a row, which the SM's
// other block covers in part.  4096 rows of 12288 bf16 81 us (0.38 of the measured copy bandwidth; 154 us
// with one octet at a time, 169 us in the general kernel); 2048 with dropout and residual 55 us (0.56);
// 1024 rows of 51200 float32, one block per SM, 120 us (0.53).
constexpr int kWideThreads = 512;
template <typename T>
__global__ void __launch_bounds__(kWideThreads, 2)
layernorm_fwd_wide_kernel(const ResidualArgs a) {
    constexpr int W = kWideThreads / 32, U = sizeof(T) == 2 ? 3 : 2;
    __shared__ float2 red[2][W];
    extern __shared__ float4 sum[];  // [2][n]: the lower and the upper four channels of octet v at v and n + v
    launch_dependents();
    grid_dependency_wait();
    Dropper D;
    if (a.thr) D.start(a.rng, a.thr);
    const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.res);
    T *y = static_cast<T *>(a.y), *h = static_cast<T *>(a.h);
    const int n = static_cast<int>(a.C / 8);
    const int64_t rows = a.B * a.T;
    const float inv = 1.f / static_cast<float>(a.C);
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const int64_t base = r * a.C, b = r / a.T;
        if (r - b * a.T >= clamp_len(a.lengths, b, a.T)) {
            const float2 zero[4] = {};
            for (int v = threadIdx.x; v < n; v += kWideThreads) {
                Oct<T>::store(y + base + 8 * v, zero);
                if (h) Oct<T>::store(h + base + 8 * v, zero);
            }
            if (threadIdx.x == 0) {
                if (a.mean) a.mean[r] = 0.f;
                if (a.rstd) a.rstd[r] = 0.f;
            }
            continue;
        }
        float2 acc = make_float2(0.f, 0.f);
        for (int v0 = threadIdx.x; v0 < n; v0 += U * kWideThreads) {
            Oct<T> xo[U], ro[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t e = base + 8 * static_cast<int64_t>(v0 + u * kWideThreads);
                ro[u].zero();
                if (v0 + u * kWideThreads < n) {
                    xo[u].load(x + e);
                    if (res) ro[u].load(res + e);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int v = v0 + u * kWideThreads;
                if (v >= n) break;
                float2 f[1][4], p[4];
                xo[u].get(f[0]);
                ro[u].get(p);
                if (a.thr) D.apply(static_cast<uint32_t>((base + 8 * v) >> 3), 0, f);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f[0][i] = ffma2(both(a.mult), f[0][i], p[i]);
                    acc = fadd2(acc, f[0][i]);
                }
                sum[v] = make_float4(f[0][0].x, f[0][0].y, f[0][1].x, f[0][1].y);
                sum[n + v] = make_float4(f[0][2].x, f[0][2].y, f[0][3].x, f[0][3].y);
                if (h) Oct<T>::store(h + base + 8 * v, f[0]);
            }
        }
        const float mean = block_sum2<W>(make_float2(acc.x + acc.y, 0.f), red[0]).x * inv;
        acc = make_float2(0.f, 0.f);
        for (int v = threadIdx.x; v < n; v += kWideThreads) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float4 q = sum[k * n + v];
                const float2 d0 = fadd2(make_float2(q.x, q.y), both(-mean));
                const float2 d1 = fadd2(make_float2(q.z, q.w), both(-mean));
                acc = ffma2(d0, d0, ffma2(d1, d1, acc));
            }
        }
        const float rstd = rsqrt_newton(fmaf(block_sum2<W>(make_float2(acc.x + acc.y, 0.f), red[1]).x, inv, a.eps));
        for (int v = threadIdx.x; v < n; v += kWideThreads) {
            const float4 q0 = sum[v], q1 = sum[n + v];
            float2 f[4] = {make_float2(q0.x, q0.y), make_float2(q0.z, q0.w),
                           make_float2(q1.x, q1.y), make_float2(q1.z, q1.w)};
            float2 ga[4], be[4];
            any_params8(a.gamma, 1.f, 8 * v, ga);
            any_params8(a.beta, 0.f, 8 * v, be);
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = ffma2(fmul2(fadd2(f[i], both(-mean)), both(rstd)), ga[i], be[i]);
            Oct<T>::store(y + base + 8 * v, f);
        }
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
    }
}

template <typename T>
cudaError_t launch_wide(const ResidualArgs &a, cudaStream_t s) {
    const int64_t smem = a.C * 4;
    static SmemGrant grant;
    const void *const kernel = reinterpret_cast<const void *>(layernorm_fwd_wide_kernel<T>);
    const cudaError_t e = grant(kernel, static_cast<int>(smem), -1);
    if (e != cudaSuccess) return e;
    const int64_t rows = a.B * a.T, most = static_cast<int64_t>(sm_count()) * (smem <= 100 * 1024 ? 2 : 1);
    return launch_programmatic(layernorm_fwd_wide_kernel<T>, dim3(static_cast<unsigned>(rows < most ? rows : most)),
                               dim3(kWideThreads), static_cast<size_t>(smem), s, a);
}

}  // namespace

cudaError_t layernorm_fwd_launch(const ResidualArgs &a, cudaStream_t s) {
    const cudaError_t e = a.dtype == 1   ? layernorm_fwd_rows_bf16(a, s)
                          : a.dtype == 2 ? layernorm_fwd_rows_f16(a, s)
                                         : layernorm_fwd_rows_f32(a, s);
    if (e != cudaErrorNotSupported) return e;
    if (row_kernels_serve(a) && a.phase == 0 && a.C % 8 == 0 && a.C <= 51200)
        return with_dtype(a.dtype, [&](auto t) { return launch_wide<decltype(t)>(a, s); });
    const int64_t rows = a.B * a.T, most = static_cast<int64_t>(sm_count()) * 8;
    const dim3 grid(static_cast<unsigned>(rows < most ? rows : most));
    return with_dtype(a.dtype, [&](auto t) {
        return launch_programmatic(layernorm_fwd_general_kernel<decltype(t)>, grid, dim3(256), 0, s, a);
    });
}

}  // namespace dwk
