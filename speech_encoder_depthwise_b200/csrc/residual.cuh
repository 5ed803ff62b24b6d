// Device helpers shared by the residual-path kernels (layer norm, dropout with the residual add).
// Everything they read, parameters, lengths and generator state included, goes by ordinary loads: the previous
// kernel in the stream may write it while this one is already resident, so none of it is read-only data.
#pragma once

#include <atomic>
#include <mutex>

#include "dropout.cuh"
#include "dw_common.cuh"

namespace dwk {

// Dynamic shared memory beyond 48 KB, granted once per kernel, device and size (one of these per
// kernel); the grant only grows, so calls of different sizes at once cannot take each other's away.
// `carveout`: the shared-memory part of the SM's 256 KB, in percent of 228 KB (-1: what the kernel's
// own blocks need).
struct SmemGrant {
    std::mutex mu;
    std::atomic<int> bytes[32] = {};
    cudaError_t operator()(const void *kern, int want, int carveout) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (want < 48 * 1024) want = 48 * 1024;
        if (dev < 32 && bytes[dev].load(std::memory_order_acquire) >= want) return cudaSuccess;
        std::lock_guard<std::mutex> lock(mu);
        if (dev < 32 && bytes[dev].load(std::memory_order_relaxed) >= want) return cudaSuccess;
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, dev < 32 ? want : 226 * 1024);
        if (e == cudaSuccess && carveout >= 0)
            e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, carveout);
        if (e == cudaSuccess && dev < 32) bytes[dev].store(want, std::memory_order_release);
        return e;
    }
};

// One element of any type at any alignment, as float32 and back.
template <typename T> __device__ __forceinline__ float load1(const T *p) { return static_cast<float>(*p); }
template <typename T> __device__ __forceinline__ T zero1() { return static_cast<T>(0.f); }
template <typename T> __device__ __forceinline__ void store1(T *p, float v) {
    const float2 f[1] = {make_float2(v, 0.f)};
    Vec<T, 1>::store(p, f);
}

__device__ __forceinline__ float2 fadd2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 fmul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Eight consecutive elements, moved with one instruction (16 bytes of a 16-bit type, 32 of float32):
// the unit of the row kernels, and one block of the dropout generator.  Loads do not allocate in
// L1 (every activation is read once), which leaves it to gamma and beta.
template <typename T> struct Oct {
    using H = Half16<T>;
    uint4 r;
    __device__ __forceinline__ void load(const T *p) {
        asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
    }
    __device__ __forceinline__ void zero() { r = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float2 (&f)[4]) const {
        f[0] = H::unpack(r.x); f[1] = H::unpack(r.y); f[2] = H::unpack(r.z); f[3] = H::unpack(r.w);
    }
    __device__ __forceinline__ void set(const float2 (&f)[4]) {
        r = make_uint4(H::pack(f[0].x, f[0].y), H::pack(f[1].x, f[1].y), H::pack(f[2].x, f[2].y),
                       H::pack(f[3].x, f[3].y));
    }
    __device__ __forceinline__ void store_global(T *p) const { *reinterpret_cast<uint4 *>(p) = r; }
    static __device__ __forceinline__ void store(T *p, const float2 (&f)[4]) {
        Oct o;
        o.set(f);
        o.store_global(p);
    }
};

template <> struct Oct<float> {
    float2 v[4];
    __device__ __forceinline__ void load(const float *p) {
        asm volatile("ld.global.L1::no_allocate.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=f"(v[0].x), "=f"(v[0].y), "=f"(v[1].x), "=f"(v[1].y), "=f"(v[2].x), "=f"(v[2].y),
                       "=f"(v[3].x), "=f"(v[3].y)
                     : "l"(p) : "memory");
    }
    __device__ __forceinline__ void zero() { v[0] = v[1] = v[2] = v[3] = make_float2(0.f, 0.f); }
    __device__ __forceinline__ void get(float2 (&f)[4]) const { f[0] = v[0]; f[1] = v[1]; f[2] = v[2]; f[3] = v[3]; }
    __device__ __forceinline__ void set(const float2 (&f)[4]) { v[0] = f[0]; v[1] = f[1]; v[2] = f[2]; v[3] = f[3]; }
    __device__ __forceinline__ void store_global(float *p) const {
        asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0].x), "f"(v[0].y),
                     "f"(v[1].x), "f"(v[1].y), "f"(v[2].x), "f"(v[2].y), "f"(v[3].x), "f"(v[3].y)
                     : "memory");
    }
    static __device__ __forceinline__ void store(float *p, const float2 (&f)[4]) {
        Oct o;
        o.set(f);
        o.store_global(p);
    }
};

// Eight float32 parameters (32-byte aligned), kept in L1 for the rows to come.
__device__ __forceinline__ void load_params8(const float *p, float2 (&f)[4]) {
    asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(f[0].x), "=f"(f[0].y), "=f"(f[1].x), "=f"(f[1].y), "=f"(f[2].x), "=f"(f[2].y), "=f"(f[3].x),
                   "=f"(f[3].y)
                 : "l"(p) : "memory");
}

// The same of any alignment; `missing` where there is no parameter.
__device__ __forceinline__ void any_params8(const float *p, float missing, int64_t c, float2 (&f)[4]) {
    if (p == nullptr) {
        f[0] = f[1] = f[2] = f[3] = both(missing);
    } else if (reinterpret_cast<uintptr_t>(p) % 32 == 0) {
        load_params8(p + c, f);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = make_float2(load_global(p + c + 2 * i), load_global(p + c + 2 * i + 1));
    }
}

// The channels of one thread in a row kernel: NO octets, TPR apart, of a row held by TPR threads.
// Octets lie on multiples of 8 of the flat index (counted from the `phase` elements that the tensors
// lie past such a boundary), so every one is an aligned word whatever C is: row r has `head`
// channels before its first octet, m octets, and up to 7 channels behind them.  The channels before
// and behind (the edges) go one each to lanes 0 .. 6 and 8 .. 14, as scalars: no octet is ever
// partial and no neighbouring row is touched.  (Whole octets with masks at both ends instead, their
// places outside the row cleared, took 49.5 us where this takes 34.3: dropout, add and norm forward,
// 16x1499x1023 fp16.)  SHIFT false: C is a multiple of 8, no edges.  A thread's rows are a multiple of
// 8 apart, so it keeps its channels from row to row.  A row has at least TPR (NO - 1) octets, so only
// the last octet of a thread can lie behind them.
template <typename T, int TPR, int NO, bool SHIFT> struct Channels {
    int lane, C, head, m;
    int ce;  // the edge channel of this thread, or -1

    __device__ __forceinline__ void start(int C_, int first, int phase) {
        lane = static_cast<int>(threadIdx.x) % TPR;
        C = C_;
        head = 0;
        m = C / 8;
        ce = -1;
        if constexpr (SHIFT) {
            head = static_cast<int>(-(static_cast<int64_t>(first) * C + phase) & 7);
            if (head > C) head = C;
            m = (C - head) / 8;
            const int behind = head + 8 * m;
            if (lane < head) ce = lane;
            if (lane >= 8 && lane < 15 && behind + lane - 8 < C) ce = behind + lane - 8;
        }
    }
    __device__ __forceinline__ int c0(int j) const { return head + 8 * (j * TPR + lane); }
    __device__ __forceinline__ bool any(int j) const { return j < NO - 1 || j * TPR + lane < m; }
    __device__ __forceinline__ bool edge() const { return SHIFT && ce >= 0; }
    // Flat index of the thread's first octet in row r, and of its edge channel.
    __device__ __forceinline__ int64_t at(int r) const { return static_cast<int64_t>(r) * C + (head + 8 * lane); }
    __device__ __forceinline__ int64_t edge_at(int r) const { return static_cast<int64_t>(r) * C + ce; }
    __device__ __forceinline__ void load_row(const T *p, int64_t e, Oct<T> (&o)[NO]) const {
#pragma unroll
        for (int j = 0; j < NO; ++j)
            if (any(j)) o[j].load(p + e + 8 * j * TPR);
    }
    // Row r's lines into L2 (before the previous kernel in the stream has completed: see prefetch_l2).
    __device__ __forceinline__ void prefetch_row(const T *p, int r) const {
        if (lane % (128 / (8 * static_cast<int>(sizeof(T)))) == 0) {
#pragma unroll
            for (int j = 0; j < NO; ++j)
                if (any(j)) prefetch_l2(p + at(r) + 8 * j * TPR);
        }
    }
    __device__ __forceinline__ void store_row(T *p, int64_t e, const float2 (&f)[NO][4]) const {
#pragma unroll
        for (int j = 0; j < NO; ++j)
            if (any(j)) Oct<T>::store(p + e + 8 * j * TPR, f[j]);
    }
    __device__ __forceinline__ void store_zeros(T *p, int r) const {
        const float2 zero[4] = {};
        const int64_t e = at(r);
#pragma unroll
        for (int j = 0; j < NO; ++j)
            if (any(j)) Oct<T>::store(p + e + 8 * j * TPR, zero);
        if (edge()) store1(p + edge_at(r), 0.f);
    }
    // Zeros in an octet behind the row's.
    __device__ __forceinline__ void clear_behind(int j, float2 (&f)[4]) const {
        if (j < NO - 1) return;
        const bool in = any(j);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = in ? f[i] : make_float2(0.f, 0.f);
    }
};

// Parameters in shared memory for rows with edges: channel c at word (c % 8) Q + c / 8.  Element i of
// octet v is channel head + 8 v + i, at v + off(i) with off the same in every octet, so the lanes
// of a row read neighbouring words: no bank conflicts, and no address arithmetic but an immediate.
// Q is 4 more than a multiple of 8, so that neighbouring channels lie in different banks as well.
__host__ __device__ __forceinline__ int shifted_q(int C) { return ((C + 7) / 8 + 3) / 8 * 8 + 4; }
__device__ __forceinline__ int shifted_at(int c, int Q) { return (c & 7) * Q + (c >> 3); }
// Without edges: octet v's lower four channels are the 16 bytes v, its upper four the 16 bytes Q + v.
__device__ __forceinline__ int halves_at(int c, int Q) { return 4 * ((c >> 2 & 1) * Q + (c >> 3)) + (c & 3); }

// The rows of one thread group: first, first + step, ..., and whether each is valid (32-bit rows).
struct RowWalk {
    int r, rows, step, t, b, dt, db, T, len;
    const int32_t *lengths;
    __device__ __forceinline__ void start(const int32_t *lengths_, int first, int step_, int rows_, int T_) {
        r = first; rows = rows_; step = step_; T = T_; lengths = lengths_;
        t = b = dt = db = 0;
        len = 1;
        if (lengths) {
            b = static_cast<int>(static_cast<uint32_t>(first) / static_cast<uint32_t>(T));
            t = first - b * T;
            db = static_cast<int>(static_cast<uint32_t>(step) / static_cast<uint32_t>(T));
            dt = step - db * T;
            if (in()) len = load_global(lengths + b);
        }
    }
    __device__ __forceinline__ bool in() const { return r < rows; }
    __device__ __forceinline__ bool valid() const { return t < len; }  // t in [0, T): lengths need no clamp
    __device__ __forceinline__ void next() {
        r += step;
        if (lengths) {
            b += db;
            t += dt;
            if (t >= T) {
                t -= T;
                ++b;
            }
            if (in()) len = load_global(lengths + b);
        }
    }
};

// Which elements the dropout keeps: zeros where not, whatever was there.  thr < 65536.  The octets
// g, g + step, ... (32-bit numbers) go through the rounds together and share their keys (dropout
// backward 32x1500x1024 fp16 34.5 us -> 28.8: an octet by itself takes 106 instructions, four
// together 69 each); the first rounds' products that do not depend on the octet are the compiler's
// to hoist.
struct Dropper {
    DropoutRng R;
    uint32_t thr16;  // threshold in the upper half of a word
    __device__ __forceinline__ void start(const unsigned long long *rng, uint32_t thr) {
        R.load(rng);
        thr16 = thr << 16;
    }
    __device__ __forceinline__ void clear(const uint4 &w, float2 (&x)[4]) const {
        const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i].x = (q[i] << 16) < thr16 ? 0.f : x[i].x;
            x[i].y = q[i] < thr16 ? 0.f : x[i].y;
        }
    }
    template <int NO> __device__ __forceinline__ void apply(uint32_t g, uint32_t step, float2 (&x)[NO][4]) const {
        uint32_t gs[NO];
        uint4 w[NO];
#pragma unroll
        for (int j = 0; j < NO; ++j) gs[j] = g + j * step;
        R.blocks<NO>(gs, w);
#pragma unroll
        for (int j = 0; j < NO; ++j) clear(w[j], x[j]);
    }
    // The same with one element more, flat index e.
    template <int NO>
    __device__ __forceinline__ void apply(uint32_t g, uint32_t step, float2 (&x)[NO][4], int64_t e, float &xe) const {
        uint32_t gs[NO + 1];
        uint4 w[NO + 1];
#pragma unroll
        for (int j = 0; j < NO; ++j) gs[j] = g + j * step;
        gs[NO] = static_cast<uint32_t>(e >> 3);
        R.blocks<NO + 1>(gs, w);
#pragma unroll
        for (int j = 0; j < NO; ++j) clear(w[j], x[j]);
        const int i = static_cast<int>(e) & 7;
        const uint32_t lo = (i & 4) ? w[NO].z : w[NO].x, hi = (i & 4) ? w[NO].w : w[NO].y, q = (i & 2) ? hi : lo;
        if (((i & 1) ? q : q << 16) < thr16) xe = 0.f;
    }
};

// Sum over the TPR threads of a row (8, 16 or 32 lanes of a warp, or TPR/32 whole warps), the same
// in all of them.  Several warps: `red` holds 2 x TPR/32 values of the group, `flip` alternates
// its halves, so one barrier (the group's own, number 1 + group) per sum is enough.
__device__ __forceinline__ float2 plus(float2 a, float2 b) { return make_float2(a.x + b.x, a.y + b.y); }
__device__ __forceinline__ float plus(float a, float b) { return a + b; }
__device__ __forceinline__ float2 shfl_xor(float2 v, int o) {
    return make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o));
}
__device__ __forceinline__ float shfl_xor(float v, int o) { return __shfl_xor_sync(0xffffffffu, v, o); }
template <int TPR, typename V>
__device__ __forceinline__ V row_sum(V v, V *red, int &flip) {
    constexpr int W = TPR > 32 ? 32 : TPR;
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) v = plus(v, shfl_xor(v, o));
    if constexpr (TPR > 32) {
        V *half = red + flip * (TPR / 32);
        flip ^= 1;
        if (threadIdx.x % 32 == 0) half[threadIdx.x % TPR / 32] = v;
        asm volatile("bar.sync %0, %1;" ::"r"(1 + static_cast<int>(threadIdx.x) / TPR), "n"(TPR) : "memory");
        v = half[0];
#pragma unroll
        for (int w = 1; w < TPR / 32; ++w) v = plus(v, half[w]);
    }
    return v;
}

// 1 / sqrt(v): the approximate reciprocal square root and one Newton step, under 2 units of 2^-24.
// (0 and infinity keep the approximation's infinity and 0.)
__device__ __forceinline__ float rsqrt_newton(float v) {
    const float r = rsqrtf(v), e = fmaf(-v * r, r, 1.f);
    return v > 0.f && v < INFINITY ? fmaf(0.5f * r, e, r) : r;
}

// Sums of two values over a block of W warps, the same in every thread.  `red` holds 2 * W floats;
// the caller alternates two of them between calls, so one barrier per call is enough.
template <int W>
__device__ __forceinline__ float2 block_sum2(float2 v, float2 *red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    float2 s = red[0];
#pragma unroll
    for (int w = 1; w < W; ++w) {
        s.x += red[w].x;
        s.y += red[w].y;
    }
    return s;
}

}  // namespace dwk
