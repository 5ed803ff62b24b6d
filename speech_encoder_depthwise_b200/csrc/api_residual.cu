// The C ABI of the residual path (include/dwconv.h): layer norm, dropout with the residual add,
// and the two in one pass.  Argument checks on the host before any CUDA call, then one launcher.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "api_internal.h"

namespace {

using dwapi::aligned;
using dwapi::cuda_status;
using dwapi::dtype_size;
using dwapi::mul3;
using dwapi::on_elements;
using dwapi::overlaps;

// The memory of one call: no output may overlap an input or another output.
struct Region {
    const void *p;
    size_t n;
};
bool disjoint(std::initializer_list<Region> outs, std::initializer_list<Region> ins) {
    for (auto o = outs.begin(); o != outs.end(); ++o) {
        if (o->p == nullptr) continue;
        for (const Region &i : ins)
            if (i.p != nullptr && overlaps(o->p, o->n, i.p, i.n)) return false;
        for (auto q = o + 1; q != outs.end(); ++q)
            if (q->p != nullptr && overlaps(o->p, o->n, q->p, q->n)) return false;
    }
    return true;
}

// How many elements past a boundary of 8 every activation lies, the same for all; -1 where they differ.
int oct_phase(dw_dtype_t dt, std::initializer_list<const void *> acts) {
    int phase = -1;
    for (const void *p : acts) {
        if (p == nullptr) continue;
        const int k = static_cast<int>(reinterpret_cast<uintptr_t>(p) / dtype_size(dt) % 8);
        if (phase >= 0 && k != phase) return -1;
        phase = k;
    }
    return phase;
}

dw_status_t check_sizes(int64_t B, int64_t T, int64_t C, dw_dtype_t dt, int64_t *n) {
    if (!dwapi::valid_dtype(dt) || B < 0 || T < 0 || C < 1) return DW_ERR_INVALID_ARG;
    if (C > dwapi::kMaxChannels) return DW_ERR_UNSUPPORTED;
    return mul3(B, T, C, n) ? DW_OK : DW_ERR_INVALID_ARG;
}

// The drop threshold of p and the factor of a kept element.
dw_status_t set_dropout(const uint64_t *rng, double p, double alpha, int64_t n, dwk::ResidualArgs *a) {
    if (!(p >= 0.0 && p <= 1.0) || !isfinite(alpha)) return DW_ERR_INVALID_ARG;
    a->thr = static_cast<uint32_t>(floor(p * 65536.0 + 0.5));
    a->mult = a->thr < 65536u ? static_cast<float>(alpha * 65536.0 / (65536.0 - a->thr)) : 0.f;
    if (!isfinite(a->mult)) return DW_ERR_INVALID_ARG;
    a->rng = reinterpret_cast<const unsigned long long *>(rng);
    if (n > 0 && a->thr > 0 && (rng == nullptr || !aligned(rng, 8))) return DW_ERR_INVALID_ARG;
    return DW_OK;
}

// The generator's state where the call reads it.
const void *drawn(const dwk::ResidualArgs *a) { return a->thr > 0 ? a->rng : nullptr; }

void set_sizes(dwk::ResidualArgs *a, const int32_t *lengths, int64_t B, int64_t T, int64_t C, dw_dtype_t dt) {
    a->lengths = lengths;
    a->B = B; a->T = T; a->C = C;
    a->dtype = static_cast<int>(dt);
}

dw_status_t norm_fwd(dwk::ResidualArgs *a, int64_t n, float eps, dw_dtype_t dt, dw_stream_t stream) {
    if (!(eps >= 0.f) || !isfinite(eps)) return DW_ERR_INVALID_ARG;
    if (n == 0) return DW_OK;
    if (a->x == nullptr || a->y == nullptr) return DW_ERR_INVALID_ARG;
    if (!on_elements(dtype_size(dt), {a->x, a->res, a->y, a->h}) ||
        !on_elements(4, {a->gamma, a->beta, a->mean, a->rstd, a->lengths}))
        return DW_ERR_INVALID_ARG;
    const size_t act = static_cast<size_t>(n) * dtype_size(dt), row = static_cast<size_t>(a->B * a->T) * sizeof(float),
                 par = static_cast<size_t>(a->C) * sizeof(float);
    if (!disjoint({{a->y, act}, {a->h, act}, {a->mean, row}, {a->rstd, row}},
                  {{a->x, act}, {a->res, act}, {a->gamma, par}, {a->beta, par}, {drawn(a), 16},
                   {a->lengths, static_cast<size_t>(a->B) * sizeof(int32_t)}}))
        return DW_ERR_INVALID_ARG;
    a->eps = eps;
    a->phase = oct_phase(dt, {a->x, a->res, a->y, a->h});
    return cuda_status(dwk::layernorm_fwd_launch(*a, static_cast<cudaStream_t>(stream)));
}

dw_status_t norm_bwd(dwk::ResidualArgs *a, int64_t n, dw_dtype_t dt, void *workspace, size_t workspace_bytes,
                     dw_stream_t stream) {
    const bool params = a->dgamma != nullptr || a->dbeta != nullptr;
    const size_t act = static_cast<size_t>(n) * dtype_size(dt), row = static_cast<size_t>(a->B * a->T) * sizeof(float),
                 par = static_cast<size_t>(a->C) * sizeof(float);
    size_t need = 0;
    if (!on_elements(4, {a->dgamma, a->dbeta})) return DW_ERR_INVALID_ARG;
    if (n > 0) {
        if (a->x == nullptr || a->dy == nullptr || a->mean == nullptr || a->rstd == nullptr || a->dx == nullptr)
            return DW_ERR_INVALID_ARG;
        if (!on_elements(dtype_size(dt), {a->x, a->dy, a->dh, a->dx, a->dres}) ||
            !on_elements(4, {a->gamma, a->mean, a->rstd, a->lengths}))
            return DW_ERR_INVALID_ARG;
        if (params) {
            need = dwk::layernorm_bwd_workspace_bytes(a->B, a->T, a->C);
            if (workspace == nullptr || workspace_bytes < need || !aligned(workspace, 16)) return DW_ERR_WORKSPACE;
            a->partials = static_cast<float *>(workspace);
        }
        a->G = dwk::layernorm_bwd_partial_rows(a->B, a->T, a->C);
        a->phase = oct_phase(dt, {a->x, a->dy, a->dh, a->dx, a->dres});
    }
    if (n == 0 && !params) return DW_OK;
    // with no rows only dgamma and dbeta are touched
    const auto in = [&](const void *p) { return n > 0 ? p : nullptr; };
    if (!disjoint({{in(a->dx), act}, {in(a->dres), act}, {a->dgamma, par}, {a->dbeta, par}, {a->partials, need}},
                  {{in(a->x), act}, {in(a->dy), act}, {in(a->dh), act}, {in(a->gamma), par}, {in(a->mean), row},
                   {in(a->rstd), row}, {in(drawn(a)), 16},
                   {in(a->lengths), static_cast<size_t>(a->B) * sizeof(int32_t)}}))
        return DW_ERR_INVALID_ARG;
    return cuda_status(dwk::layernorm_bwd_launch(*a, static_cast<cudaStream_t>(stream)));
}

dw_status_t dropout_add(dwk::ResidualArgs *a, int64_t n, dw_dtype_t dt, dw_stream_t stream) {
    if (n == 0) return DW_OK;
    if (a->x == nullptr || a->y == nullptr) return DW_ERR_INVALID_ARG;
    if (!on_elements(dtype_size(dt), {a->x, a->res, a->y}) || !on_elements(4, {a->lengths})) return DW_ERR_INVALID_ARG;
    const size_t act = static_cast<size_t>(n) * dtype_size(dt);
    if (!disjoint({{a->y, act}}, {{a->x, act}, {a->res, act}, {drawn(a), 16},
                                  {a->lengths, static_cast<size_t>(a->B) * sizeof(int32_t)}}))
        return DW_ERR_INVALID_ARG;
    a->phase = oct_phase(dt, {a->x, a->res, a->y});
    return cuda_status(dwk::dropout_add_launch(*a, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

dw_status_t dw_layernorm_fwd(const void *x, const float *gamma, const float *beta, void *y, float *mean,
                             float *rstd, const int32_t *lengths, int64_t B, int64_t T, int64_t C, float eps,
                             dw_dtype_t io_dtype, dw_stream_t stream) {
    int64_t n = 0;
    const dw_status_t st = check_sizes(B, T, C, io_dtype, &n);
    if (st != DW_OK) return st;
    dwk::ResidualArgs a;
    set_sizes(&a, lengths, B, T, C, io_dtype);
    a.x = x; a.gamma = gamma; a.beta = beta; a.y = y; a.mean = mean; a.rstd = rstd;
    return norm_fwd(&a, n, eps, io_dtype, stream);
}

size_t dw_layernorm_bwd_workspace_size(int64_t B, int64_t T, int64_t C) {
    int64_t n = 0;
    if (check_sizes(B, T, C, DW_F32, &n) != DW_OK || n == 0) return 0;
    return dwk::layernorm_bwd_workspace_bytes(B, T, C);
}

dw_status_t dw_layernorm_bwd(const void *x, const void *dy, const float *gamma, const float *mean,
                             const float *rstd, void *dx, float *dgamma, float *dbeta, const int32_t *lengths,
                             int64_t B, int64_t T, int64_t C, dw_dtype_t io_dtype, void *workspace,
                             size_t workspace_bytes, dw_stream_t stream) {
    int64_t n = 0;
    const dw_status_t st = check_sizes(B, T, C, io_dtype, &n);
    if (st != DW_OK) return st;
    dwk::ResidualArgs a;
    set_sizes(&a, lengths, B, T, C, io_dtype);
    a.x = x; a.dy = dy; a.gamma = gamma;
    a.mean = const_cast<float *>(mean); a.rstd = const_cast<float *>(rstd);
    a.dx = dx; a.dgamma = dgamma; a.dbeta = dbeta;
    return norm_bwd(&a, n, io_dtype, workspace, workspace_bytes, stream);
}

dw_status_t dw_dropout_add_fwd(const void *x, const void *residual, void *y, const uint64_t *rng, double p,
                               double alpha, const int32_t *lengths, int64_t B, int64_t T, int64_t C,
                               dw_dtype_t io_dtype, dw_stream_t stream) {
    int64_t n = 0;
    dwk::ResidualArgs a;
    dw_status_t st = check_sizes(B, T, C, io_dtype, &n);
    if (st == DW_OK) st = set_dropout(rng, p, alpha, n, &a);
    if (st != DW_OK) return st;
    set_sizes(&a, lengths, B, T, C, io_dtype);
    a.x = x; a.res = residual; a.y = y;
    return dropout_add(&a, n, io_dtype, stream);
}

dw_status_t dw_dropout_add_bwd(const void *dy, void *dx, const uint64_t *rng, double p, double alpha,
                               const int32_t *lengths, int64_t B, int64_t T, int64_t C, dw_dtype_t io_dtype,
                               dw_stream_t stream) {
    return dw_dropout_add_fwd(dy, nullptr, dx, rng, p, alpha, lengths, B, T, C, io_dtype, stream);
}

dw_status_t dw_dropout_add_layernorm_fwd(const void *x, const void *residual, const uint64_t *rng, double p,
                                         double alpha, const float *gamma, const float *beta, void *h, void *y,
                                         float *mean, float *rstd, const int32_t *lengths, int64_t B, int64_t T,
                                         int64_t C, float eps, dw_dtype_t io_dtype, dw_stream_t stream) {
    int64_t n = 0;
    dwk::ResidualArgs a;
    dw_status_t st = check_sizes(B, T, C, io_dtype, &n);
    if (st == DW_OK) st = set_dropout(rng, p, alpha, n, &a);
    if (st != DW_OK) return st;
    set_sizes(&a, lengths, B, T, C, io_dtype);
    a.x = x; a.res = residual; a.gamma = gamma; a.beta = beta;
    a.h = h; a.y = y; a.mean = mean; a.rstd = rstd;
    return norm_fwd(&a, n, eps, io_dtype, stream);
}

dw_status_t dw_dropout_add_layernorm_bwd(const void *dy, const void *dh, const void *h, const float *gamma,
                                         const float *mean, const float *rstd, const uint64_t *rng, double p,
                                         double alpha, void *dx, void *dresidual, float *dgamma, float *dbeta,
                                         const int32_t *lengths, int64_t B, int64_t T, int64_t C,
                                         dw_dtype_t io_dtype, void *workspace, size_t workspace_bytes,
                                         dw_stream_t stream) {
    int64_t n = 0;
    dwk::ResidualArgs a;
    dw_status_t st = check_sizes(B, T, C, io_dtype, &n);
    if (st == DW_OK) st = set_dropout(rng, p, alpha, n, &a);
    if (st != DW_OK) return st;
    set_sizes(&a, lengths, B, T, C, io_dtype);
    a.x = h; a.dy = dy; a.dh = dh; a.gamma = gamma;
    a.mean = const_cast<float *>(mean); a.rstd = const_cast<float *>(rstd);
    a.dx = dx; a.dres = dresidual; a.dgamma = dgamma; a.dbeta = dbeta;
    return norm_bwd(&a, n, io_dtype, workspace, workspace_bytes, stream);
}

}  // extern "C"
