// Dropout with the residual add, forward and (without a residual) backward:
//   y[e] = [valid] (res[e] + [kept] mult x[e]).
// Elementwise; the mask is drawn from the element's index, never stored.
#include "dw_internal.h"
#include "residual.cuh"

namespace dwk {
namespace {

// x and res are read by ordinary loads, never as read-only data (no __restrict__, which would let the
// compiler take that path): the previous kernel may write them while this one is already resident.  A
// thread's loads come before its stores, which the compiler may no longer exchange.

// A thread takes the 8 elements of one mask block, element by element.
template <typename T>
__global__ void __launch_bounds__(256)
dropout_add_general_kernel(const T *x, const T *res, T *y, const int32_t *lengths, const unsigned long long *rng,
                           uint32_t thr, float mult, int64_t B, int64_t Tn, int64_t C) {
    launch_dependents();
    grid_dependency_wait();
    DropoutRng R = {};
    if (thr) R.load(rng);
    const int64_t TC = Tn * C, N = B * TC;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x * 8;
    for (int64_t e0 = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) * 8; e0 < N; e0 += stride) {
        const uint4 w4 = thr ? R.block(static_cast<uint64_t>(e0) >> 3) : make_uint4(0, 0, 0, 0);
        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
        int64_t b = e0 / TC, i = e0 - b * TC, lim = clamp_len(lengths, b, Tn) * C;
        T xv[8], rv[8];
        unsigned in = 0;  // bit j: element j is valid
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (e0 + j >= N) break;
            if (i >= TC) {
                i = 0;
                lim = clamp_len(lengths, ++b, Tn) * C;
            }
            if (i < lim) {
                in |= 1u << j;
                xv[j] = x[e0 + j];
                if (res) rv[j] = res[e0 + j];
            }
            ++i;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (e0 + j >= N) break;
            float v = 0.f;
            if (in >> j & 1u) {
                if (res) v = load1(&rv[j]);
                if (((w[j / 2] >> (16 * (j % 2))) & 0xffffu) >= thr) v = fmaf(mult, load1(&xv[j]), v);
            }
            store1(y + e0 + j, v);
        }
    }
}

// Octet-aligned tensors: a block takes a chunk of 256 U octets, all of a thread's loads first.  Most
// chunks lie wholly within the valid or the masked frames of one item, which one division per
// block tells; in the others every octet is looked at by itself, and those with an item's end or
// its last valid frame inside (or past the tensor's end) go element by element.
//
// Bound by HBM (4 to 6 bytes a 16-bit element) with the generator close behind: 18 wide
// multiplications an octet.  Measured (graph replay, cold inputs; fraction of the measured copy
// bandwidth): backward 32x1500x1024 fp16 28.7 us (0.91), forward 16x1500x512 bf16 11.7 us (0.80),
// forward 32x750x1024 float32 37.3 us (1.01).
constexpr int kChunkOctets = 4;
template <typename T, bool DROP, bool RES>
__global__ void __launch_bounds__(256)
dropout_add_octet_kernel(const T *x, const T *res, T *y, const int32_t *lengths, const unsigned long long *rng,
                         uint32_t thr, float mult, int64_t B, int64_t Tn, int64_t C) {
    constexpr int U = kChunkOctets, kStep = 256 * 8, kChunk = U * kStep;
    enum { kValid, kMasked, kMixed, kNone };
    launch_dependents();
    const int64_t TC = Tn * C, N = B * TC, first = static_cast<int64_t>(blockIdx.x) * kChunk;
    const bool narrow = N < (int64_t(1) << 32);
    const auto item_of = [&](int64_t e) -> int64_t {
        return narrow ? static_cast<uint32_t>(e) / static_cast<uint32_t>(TC) : e / TC;
    };
    const int64_t b = lengths ? item_of(first) : 0;
    grid_dependency_wait();
    Dropper D;
    if constexpr (DROP) D.start(rng, thr);
    const int64_t mine = first + threadIdx.x * 8;
    const int64_t start = b * TC, lim = lengths ? start + clamp_len(lengths, b, Tn) * C : N;
    Oct<T> xo[U], ro[U];
    if (first + kChunk <= lim) {
#pragma unroll
        for (int u = 0; u < U; ++u) xo[u].load(x + mine + u * kStep);
        if constexpr (RES) {
#pragma unroll
            for (int u = 0; u < U; ++u) ro[u].load(res + mine + u * kStep);
        }
        float2 f[U][4], q[4];
#pragma unroll
        for (int u = 0; u < U; ++u) xo[u].get(f[u]);
        if constexpr (DROP) D.apply(static_cast<uint32_t>(mine >> 3), kStep / 8, f);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if constexpr (RES) ro[u].get(q);
#pragma unroll
            for (int i = 0; i < 4; ++i) f[u][i] = RES ? ffma2(both(mult), f[u][i], q[i]) : fmul2(both(mult), f[u][i]);
            Oct<T>::store(y + mine + u * kStep, f[u]);
        }
        return;
    }
    if (first >= lim && first + kChunk <= start + TC && first + kChunk <= N) {
        const float2 zero[4] = {};
#pragma unroll
        for (int u = 0; u < U; ++u) Oct<T>::store(y + mine + u * kStep, zero);
        return;
    }
    int st[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t e = mine + u * kStep;
        st[u] = kNone;
        if (e >= N) continue;
        const int64_t item = lengths ? item_of(e) : 0, i0 = lengths ? item * TC : 0;
        const int64_t i1 = lengths ? i0 + clamp_len(lengths, item, Tn) * C : N, i2 = lengths ? i0 + TC : N;
        st[u] = e + 8 <= i1 ? kValid : (e >= i1 && e + 8 <= i2 ? kMasked : kMixed);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (st[u] != kValid) continue;
        xo[u].load(x + mine + u * kStep);
        if constexpr (RES) ro[u].load(res + mine + u * kStep);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float2 f[1][4] = {}, q[4] = {};
        if (st[u] == kValid) {
            xo[u].get(f[0]);
            if constexpr (RES) ro[u].get(q);
            if constexpr (DROP) D.apply(static_cast<uint32_t>((mine + u * kStep) >> 3), 0, f);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                f[0][i] = RES ? ffma2(both(mult), f[0][i], q[i]) : fmul2(both(mult), f[0][i]);
        }
        if (st[u] <= kMasked) Oct<T>::store(y + mine + u * kStep, f[0]);
    }
    unsigned mixed = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) mixed |= st[u] == kMixed ? 1u << u : 0u;
#pragma unroll 1
    for (int u = 0; mixed; ++u, mixed >>= 1) {
        if (!(mixed & 1u)) continue;
        const int64_t e0 = mine + u * kStep;
        float2 keep[1][4] = {{both(1.f), both(1.f), both(1.f), both(1.f)}};
        if constexpr (DROP) D.apply(static_cast<uint32_t>(e0 >> 3), 0, keep);
        int64_t item = lengths ? item_of(e0) : 0, next = lengths ? (item + 1) * TC : N;
        int64_t lim = lengths ? item * TC + clamp_len(lengths, item, Tn) * C : N;
        T xe[8], re[8];
        unsigned in = 0;  // bit i: element i is valid
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t e = e0 + i;
            if (e >= N) break;
            if (lengths && e >= next) {
                lim = next + clamp_len(lengths, ++item, Tn) * C;
                next += TC;
            }
            if (e < lim) {
                in |= 1u << i;
                xe[i] = x[e];
                if constexpr (RES) re[i] = res[e];
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (e0 + i >= N) break;
            float v = 0.f;
            if (in >> i & 1u) {
                if constexpr (RES) v = load1(&re[i]);
                if ((i % 2 ? keep[0][i / 2].y : keep[0][i / 2].x) != 0.f) v = fmaf(mult, load1(&xe[i]), v);
            }
            store1(y + e0 + i, v);
        }
    }
}

template <typename T>
cudaError_t launch_octets(const ResidualArgs &a, cudaStream_t s) {
    const int64_t chunk = 256 * kChunkOctets * 8, blocks = (a.B * a.T * a.C + chunk - 1) / chunk;
    const auto go = [&](auto kern) {
        return launch_programmatic(kern, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s,
                                   static_cast<const T *>(a.x), static_cast<const T *>(a.res), static_cast<T *>(a.y),
                                   a.lengths, a.rng, a.thr, a.mult, a.B, a.T, a.C);
    };
    if (a.thr)
        return a.res ? go(dropout_add_octet_kernel<T, true, true>) : go(dropout_add_octet_kernel<T, true, false>);
    return a.res ? go(dropout_add_octet_kernel<T, false, true>) : go(dropout_add_octet_kernel<T, false, false>);
}

}  // namespace

cudaError_t dropout_add_launch(const ResidualArgs &a, cudaStream_t s) {
    if (a.phase == 0 && a.thr < 65536u && a.B * a.T * a.C < (int64_t(1) << 35))
        return with_dtype(a.dtype, [&](auto t) { return launch_octets<decltype(t)>(a, s); });
    const int64_t groups = (a.B * a.T * a.C + 7) / 8;
    const int64_t blocks = (groups + 255) / 256, most = static_cast<int64_t>(sm_count()) * 8;
    const dim3 grid(static_cast<unsigned>(blocks < most ? blocks : most));
    return with_dtype(a.dtype, [&](auto t) {
        using T = decltype(t);
        return launch_programmatic(dropout_add_general_kernel<T>, grid, dim3(256), 0, s, static_cast<const T *>(a.x),
                                   static_cast<const T *>(a.res), static_cast<T *>(a.y), a.lengths, a.rng, a.thr,
                                   a.mult, a.B, a.T, a.C);
    });
}

}  // namespace dwk
