// Host-side argument handling shared by the translation units of the C ABI (api.cu,
// api_residual.cu and dw_noalloc.cu): status mapping, size and pointer checks, and the checks
// of the weight/bias gradient.
#pragma once

#include <initializer_list>

#include "dw_internal.h"
#include "dwconv.h"

namespace dwapi {

// DW_OK for cudaSuccess; otherwise records the error for dw_last_cuda_error and returns DW_ERR_CUDA.
dw_status_t cuda_status(cudaError_t e);

inline size_t dtype_size(dw_dtype_t t) { return t == DW_F32 ? 4 : 2; }

inline bool valid_dtype(dw_dtype_t t) { return t == DW_F32 || t == DW_BF16 || t == DW_F16; }

// n = a*b*c without overflow of int64 (all >= 0)
inline bool mul3(int64_t a, int64_t b, int64_t c, int64_t *n) {
    __int128 p = static_cast<__int128>(a) * b * c;
    if (p > static_cast<__int128>(INT64_MAX / 4)) return false;
    *n = static_cast<int64_t>(p);
    return true;
}

inline bool overlaps(const void *a, size_t na, const void *b, size_t nb) {
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
    return pa < pb + nb && pb < pa + na;
}

inline bool aligned(const void *p, size_t n) { return p == nullptr || reinterpret_cast<uintptr_t>(p) % n == 0; }

// Whether every pointer lies on a multiple of its elements' size (absent ones do): a load of one that does not
// would fault.
inline bool on_elements(size_t esize, std::initializer_list<const void *> ps) {
    for (const void *p : ps)
        if (!aligned(p, esize)) return false;
    return true;
}

// Channel counts beyond this are rejected: frame offsets are kept in 32 bits inside a run.
constexpr int64_t kMaxChannels = 1 << 22;

// Checks and argument set-up of the depthwise conv1d weight/bias gradient, everything except
// the memory of the partial rows: on DW_OK, *a holds every field but `partials` and `G`, and
// *n = B * T * C (0: nothing to read, dW and dbias are only zeroed).
dw_status_t bwd_dw_prepare(const void *x, const void *dy, float *dw, float *dbias, const int32_t *lengths,
                           int64_t B, int64_t T, int64_t C, int K, int pad_left, dw_dtype_t io_dtype,
                           dwk::DwArgs *a, int64_t *n);

}  // namespace dwapi
