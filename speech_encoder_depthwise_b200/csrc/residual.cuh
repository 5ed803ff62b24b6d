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
