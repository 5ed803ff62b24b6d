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
        asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
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
    __device__ __forceinline__ void keep(const uint32_t (&m)[4]) { r = make_uint4(r.x & m[0], r.y & m[1], r.z & m[2], r.w & m[3]); }
    __device__ __forceinline__ void store_shared(T *p) const { *reinterpret_cast<uint4 *>(p) = r; }
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
        asm volatile("ld.global.nc.L1::no_allocate.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=f"(v[0].x), "=f"(v[0].y), "=f"(v[1].x), "=f"(v[1].y), "=f"(v[2].x), "=f"(v[2].y),
                       "=f"(v[3].x), "=f"(v[3].y)
                     : "l"(p) : "memory");
    }
    __device__ __forceinline__ void zero() { v[0] = v[1] = v[2] = v[3] = make_float2(0.f, 0.f); }
    __device__ __forceinline__ void get(float2 (&f)[4]) const { f[0] = v[0]; f[1] = v[1]; f[2] = v[2]; f[3] = v[3]; }
    __device__ __forceinline__ void set(const float2 (&f)[4]) { v[0] = f[0]; v[1] = f[1]; v[2] = f[2]; v[3] = f[3]; }
    __device__ __forceinline__ void store_shared(float *p) const {
        reinterpret_cast<float4 *>(p)[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
        reinterpret_cast<float4 *>(p)[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
    }
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
    asm volatile("ld.global.nc.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(f[0].x), "=f"(f[0].y), "=f"(f[1].x), "=f"(f[1].y), "=f"(f[2].x), "=f"(f[2].y), "=f"(f[3].x),
                   "=f"(f[3].y)
                 : "l"(p) : "memory");
}

// The channels of one thread in a row kernel: NO octets, TPR apart, of a row held by TPR threads.
// Octets lie on multiples of 8 of the flat index, so every one is an aligned word whatever C is: a row
// starts s = (r C) mod 8 elements into its first octet, and octet v holds its channels 8 v - s ..
// 8 v - s + 7.  SHIFT false: C is a multiple of 8, s = 0.  A thread's rows are a multiple of 8
// apart, so it keeps its s and its channels.  A row has more than TPR (NO - 1) octets (SHIFT: may touch
// that many), so only the last octet of a thread can lie behind the row, and only the first one
// and the last two can be partial.
template <typename T, int TPR, int NO, bool SHIFT> struct Channels {
    static constexpr int kGroup = TPR < 32 ? TPR : 32;  // lanes that store a row's partial octets together
    int lane, s, C, rows;
    bool two;                 // some lane's octet NO - 2 is partial (the same in the whole warp)
    uint32_t mask[2][4];      // the own elements of octets 0 and NO - 1, 16 bits each
    T *scratch;               // SHIFT: two octets of the group in shared memory
    int cf, ce;               // the channel of the first and of the last octet that this lane stores, or -1

    __device__ __forceinline__ void start(int C_, int rows_, int first, T *scratch_) {
        lane = static_cast<int>(threadIdx.x) % TPR;
        C = C_;
        rows = rows_;
        s = SHIFT ? static_cast<int>((static_cast<int64_t>(first) * C) % 8) : 0;
        two = false;
        if constexpr (SHIFT) {
            scratch = scratch_ + threadIdx.x / kGroup * 16;
            if (NO > 2) two = __any_sync(0xffffffffu, c0(NO - 2) + 8 > C);
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = k ? NO - 1 : 0;
                    mask[k][i] = (has(j, 2 * i) ? 0x0000ffffu : 0u) | (has(j, 2 * i + 1) ? 0xffff0000u : 0u);
                }
            const int q = lane % kGroup, vend = (C + s - 1) / 8, last = 8 * vend - s + q;
            cf = s > 0 && lane < 8 && q >= s && q - s < C ? q - s : -1;
            ce = (C + s) % 8 != 0 && (vend > 0 || s == 0) && q < 8 && last < C && vend % TPR / kGroup == lane / kGroup ? last : -1;
        }
    }
    __device__ __forceinline__ int c0(int j) const { return 8 * (j * TPR + lane) - s; }
    __device__ __forceinline__ bool any(int j) const { return j < NO - 1 || c0(j) < C; }
    __device__ __forceinline__ bool full(int j) const {
        if (!SHIFT || (j > 0 && j < NO - 2)) return true;
        if (j > 0 && j == NO - 2) return !two || c0(j) + 8 <= C;
        return c0(j) >= 0 && c0(j) + 8 <= C;
    }
    __device__ __forceinline__ bool has(int j, int i) const {
        return !SHIFT || static_cast<unsigned>(c0(j) + i) < static_cast<unsigned>(C);
    }
    // Flat index of the thread's first octet in row r.
    __device__ __forceinline__ int64_t at(int r) const { return static_cast<int64_t>(r) * C - s + 8 * lane; }
    // The octets of row r, e = at(r).  Neighbouring rows' elements come along in a row's first and last
    // octet and are ignored; the last octet of the tensor may reach past its end.
    __device__ __forceinline__ void load_row(const T *p, int64_t e, int r, Oct<T> (&o)[NO]) const {
        const T *q = p + e;
        if (!SHIFT || r < rows - 1) {
#pragma unroll
            for (int j = 0; j < NO; ++j)
                if (any(j)) o[j].load(q + 8 * j * TPR);
        } else if constexpr (SHIFT) {
#pragma unroll
            for (int j = 0; j < NO; ++j) {
                if (!any(j)) continue;
                float2 f[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f[i].x = has(j, 2 * i) ? load1(q + 8 * j * TPR + 2 * i) : 0.f;
                    f[i].y = has(j, 2 * i + 1) ? load1(q + 8 * j * TPR + 2 * i + 1) : 0.f;
                }
                o[j].set(f);
            }
        }
    }
    // A row's octets to p, by every lane of the warp (rows that are not `on` store nothing).  The
    // elements of the partial octets go through shared memory to lanes that store one each.
    __device__ __forceinline__ void store_row(T *p, int64_t e, bool on, const float2 (&f)[NO][4]) const {
        T *q = p + e;
#pragma unroll
        for (int j = 0; j < NO; ++j) {
            Oct<T> o;
            o.set(f[j]);
            if (on && any(j) && full(j)) o.store_global(q + 8 * j * TPR);
            if constexpr (SHIFT)
                if (!(j > 0 && j < NO - 2) && any(j) && !full(j)) o.store_shared(scratch + (j == 0 && c0(0) < 0 ? 0 : 8));
        }
        if constexpr (SHIFT) {
            __syncwarp();
            const T *row = scratch + static_cast<int>(threadIdx.x % kGroup);
            T *base = q - (8 * lane - s);
            if (on && cf >= 0) base[cf] = row[0];
            if (on && ce >= 0) base[ce] = row[8];
            __syncwarp();
        }
    }
    __device__ __forceinline__ void store_zeros(T *p, int64_t e, bool on) const {
        const float2 zero[4] = {};
        T *q = p + e;
#pragma unroll
        for (int j = 0; j < NO; ++j)
            if (on && any(j) && full(j)) Oct<T>::store(q + 8 * j * TPR, zero);
        if constexpr (SHIFT) {
            T *base = q - (8 * lane - s);
            if (on && cf >= 0) store1(base + cf, 0.f);
            if (on && ce >= 0) store1(base + ce, 0.f);
        }
    }
    // Octet j's values, zeros in the places that are not this row's.
    __device__ __forceinline__ void get(int j, const Oct<T> &o, float2 (&f)[4]) const {
        if constexpr (SHIFT && sizeof(T) == 2) {
            Oct<T> m = o;
            if (j == 0) m.keep(mask[0]);
            if (j == NO - 1 && NO > 1) m.keep(mask[1]);
            m.get(f);
            if (NO > 2 && j == NO - 2 && two) clear_partial(j, f);
        } else {
            o.get(f);
            clear_outside(j, f);
        }
    }
    __device__ __forceinline__ void clear_partial(int j, float2 (&f)[4]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (!has(j, 2 * i)) f[i].x = 0.f;
            if (!has(j, 2 * i + 1)) f[i].y = 0.f;
        }
    }
    // Zeros in the places of an octet that are not this row's.
    __device__ __forceinline__ void clear_outside(int j, float2 (&f)[4]) const {
        if constexpr (!SHIFT) {
            if (j == NO - 1) {
                const bool in = any(j);
#pragma unroll
                for (int i = 0; i < 4; ++i) f[i] = in ? f[i] : make_float2(0.f, 0.f);
            }
        } else if (j == 0 || j == NO - 1) {
            // an element's 16 mask bits, twice
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t m = mask[j == 0 ? 0 : 1][i];
                f[i].x = __uint_as_float(__float_as_uint(f[i].x) & __byte_perm(m, 0, 0x1010));
                f[i].y = __uint_as_float(__float_as_uint(f[i].y) & __byte_perm(m, 0, 0x3232));
            }
        } else if (j == NO - 2 && two) {
            clear_partial(j, f);
        }
    }
};

// Parameters in shared memory for rows that start inside an octet: channel c at word
// (c % 8) Q + c / 8 + 1.  Element i of octet v is channel 8 v + i - s, at v + off(i) with off the
// same in every octet, so the lanes of a row read neighbouring words: no bank conflicts, and no
// address arithmetic but an immediate.  Places without a channel hold zeros.
__device__ __forceinline__ int shifted_q(int C) { return (C + 7) / 8 + 2; }
__device__ __forceinline__ int shifted_off(int i, int s, int Q) { return ((i - s) & 7) * Q + (i < s ? 0 : 1); }

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
            if (in()) len = __ldg(lengths + b);
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
            if (in()) len = __ldg(lengths + b);
        }
    }
};

// Which elements the dropout keeps: zeros where not, whatever was there.  thr < 65536.  The octets
// g, g + step, ... (32-bit numbers) go through the rounds together, which share their keys; the
// first two rounds' products that do not depend on the octet are left to the compiler to hoist.
struct Dropper {
    DropoutRng R;
    uint32_t thr16;  // threshold in the upper half of a word
    __device__ __forceinline__ void start(const unsigned long long *rng, uint32_t thr) {
        R.load(rng);
        thr16 = thr << 16;
    }
    template <int NO> __device__ __forceinline__ void apply(uint32_t g, uint32_t step, float2 (&x)[NO][4]) const {
        uint4 w[NO];
        R.blocks<NO>(g, step, w);
#pragma unroll
        for (int j = 0; j < NO; ++j) {
            const uint32_t q[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[j][i].x = (q[i] << 16) < thr16 ? 0.f : x[j][i].x;
                x[j][i].y = q[i] < thr16 ? 0.f : x[j][i].y;
            }
        }
    }
};

// Sum over the TPR threads of a row (8, 16 or 32 lanes of a warp, or a whole block of TPR), the
// same in all of them.  Blocks: `red` holds 2 x TPR/32 values; `flip` alternates its halves, so
// one barrier per sum is enough.
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
        if (threadIdx.x % 32 == 0) half[threadIdx.x / 32] = v;
        __syncthreads();
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
