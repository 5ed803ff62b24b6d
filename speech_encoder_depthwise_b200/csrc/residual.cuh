// Device helpers shared by the residual-path kernels (layer norm, dropout with the residual add).
#pragma once

#include "dropout.cuh"
#include "dw_common.cuh"

namespace dwk {

// One element of any type at any alignment, as float32 and back.
template <typename T> __device__ __forceinline__ float load1(const T *p) {
    Vec<T, 1> v;
    float2 f[1];
    v.load(p);
    v.to_f2(f);
    return f[0].x;
}
template <typename T> __device__ __forceinline__ void store1(T *p, float v) {
    const float2 f[1] = {make_float2(v, 0.f)};
    Vec<T, 1>::store(p, f);
}

// Eight consecutive elements, moved with one instruction (16 bytes of a 16-bit type, 32 of float32):
// the unit of the row kernels, and one block of the dropout generator.  Loads do not allocate in
// L1 (every activation is read once), which leaves it to gamma and beta.
template <typename T> struct Oct {
    using H = Half16<T>;
    uint4 r;
    __device__ __forceinline__ void load(const T *p) {
        asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
    }
    __device__ __forceinline__ void zero() { r = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = H::unpack(w[i]);
            f[2 * i] = v.x;
            f[2 * i + 1] = v.y;
        }
    }
    __device__ __forceinline__ void set(const float (&f)[8]) {
        r = make_uint4(H::pack(f[0], f[1]), H::pack(f[2], f[3]), H::pack(f[4], f[5]), H::pack(f[6], f[7]));
    }
    static __device__ __forceinline__ void store(T *p, const float (&f)[8]) {
        Oct o;
        o.set(f);
        *reinterpret_cast<uint4 *>(p) = o.r;
    }
};

template <> struct Oct<float> {
    float v[8];
    __device__ __forceinline__ void load(const float *p) {
        asm volatile("ld.global.nc.L1::no_allocate.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                     : "l"(p) : "memory");
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = v[i];
    }
    __device__ __forceinline__ void set(const float (&f)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = f[i];
    }
    static __device__ __forceinline__ void store(float *p, const float (&f)[8]) {
        asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(f[0]), "f"(f[1]),
                     "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
                     : "memory");
    }
};

// Octet v of row r in a row kernel.  Octets lie on multiples of 8 of the flat index, so that every
// one is an aligned word whatever C is: row r starts s = (r C) mod 8 elements into its first octet,
// and octet v holds its channels 8 v - s .. 8 v - s + 7.  SHIFT false: C is a multiple of 8, s = 0.
// A thread's rows are a multiple of 8 apart, so it keeps its s and its channels.
template <typename T, bool SHIFT> struct OctAt {
    int64_t e0;  // flat index of its first element
    int c0;      // channel of its first element (may be negative)
    int C;
    __device__ __forceinline__ OctAt(int64_t r, int64_t C_, int v, int s)
        : e0(r * C_ + (8 * v - s)), c0(8 * v - s), C(static_cast<int>(C_)) {}
    __device__ __forceinline__ bool any() const { return c0 < C; }
    __device__ __forceinline__ bool has(int i) const { return !SHIFT || static_cast<unsigned>(c0 + i) < static_cast<unsigned>(C); }
    __device__ __forceinline__ bool full() const { return !SHIFT || (c0 >= 0 && c0 + 8 <= C); }
    // Neighbouring rows' elements come along and are ignored; only the last octet of a tensor of N
    // elements may reach past it.
    __device__ __forceinline__ void load(const T *p, Oct<T> &o, int64_t N) const {
        if (!SHIFT || e0 + 8 <= N) {
            o.load(p + e0);
        } else {
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = has(i) ? load1(p + e0 + i) : 0.f;
            o.set(f);
        }
    }
    __device__ __forceinline__ void store(T *p, const float (&f)[8]) const {
        if (full()) {
            Oct<T>::store(p + e0, f);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (has(i)) store1(p + e0 + i, f[i]);
        }
    }
};

// The rows of one thread group, k-th row blk + grid (g + groups k), and whether each is valid.
struct RowWalk {
    int64_t r, rows, step;
    int64_t b, t, db, dt, T;
    const int32_t *lengths;
    __device__ __forceinline__ void start(const int32_t *lengths_, int64_t first, int64_t step_, int64_t B, int64_t T_) {
        r = first;
        rows = B * T_;
        step = step_;
        lengths = lengths_;
        T = T_;
        if (lengths) {
            if (rows + step < (int64_t(1) << 31)) {
                const uint32_t T32 = static_cast<uint32_t>(T), f = static_cast<uint32_t>(first), s = static_cast<uint32_t>(step);
                b = f / T32;
                db = s / T32;
            } else {
                b = first / T;
                db = step / T;
            }
            t = first - b * T;
            dt = step - db * T;
        }
    }
    __device__ __forceinline__ bool in() const { return r < rows; }
    __device__ __forceinline__ bool valid() const { return lengths == nullptr || t < clamp_len(lengths, b, T); }
    __device__ __forceinline__ void next() {
        r += step;
        if (lengths) {
            b += db;
            t += dt;
            if (t >= T) {
                t -= T;
                ++b;
            }
        }
    }
};

// Which of an octet's elements the dropout keeps: x[i] = 0 where not.
struct Dropper {
    DropoutRng R;
    uint32_t thr16;  // threshold in the upper half of a word
    bool all;        // thr = 65536: nothing is kept
    __device__ __forceinline__ void start(const unsigned long long *rng, uint32_t thr) {
        R.load(rng);
        all = thr >= 65536u;
        thr16 = thr << 16;
    }
    __device__ __forceinline__ void apply(uint64_t g, float (&x)[8]) const {
        const uint4 w4 = R.block(g);
        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (all || (w[i] << 16) < thr16) x[2 * i] = 0.f;
            if (all || w[i] < thr16) x[2 * i + 1] = 0.f;
        }
    }
};

// Sum over the TPR threads of a row (8, 16 or 32 lanes of a warp, or a whole block of TPR), the
// same in all of them.  Blocks: `red` holds 2 x TPR/32 values; `flip` alternates its halves, so
// one barrier per sum is enough.
template <int TPR>
__device__ __forceinline__ float2 row_sum2(float2 v, float2 *red, int &flip) {
    constexpr int W = TPR > 32 ? 32 : TPR;
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    if constexpr (TPR > 32) {
        float2 *half = red + flip * (TPR / 32);
        flip ^= 1;
        if (threadIdx.x % 32 == 0) half[threadIdx.x / 32] = v;
        __syncthreads();
        v = half[0];
#pragma unroll
        for (int w = 1; w < TPR / 32; ++w) {
            const float2 q = half[w];
            v.x += q.x;
            v.y += q.y;
        }
    }
    return v;
}
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float *red, int &flip) {
    constexpr int W = TPR > 32 ? 32 : TPR;
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (TPR > 32) {
        float *half = red + flip * (TPR / 32);
        flip ^= 1;
        if (threadIdx.x % 32 == 0) half[threadIdx.x / 32] = v;
        __syncthreads();
        v = half[0];
#pragma unroll
        for (int w = 1; w < TPR / 32; ++w) v += half[w];
    }
    return v;
}

// Position of channel c in shared memory when a lane reads 8 consecutive channels one by one (the
// SHIFT kernels): one word of padding per 32 puts the 32 lanes' words in 32 banks.
__device__ __forceinline__ int pad32(int c) { return c + (c >> 5); }

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
