// The row kernel of layer norm backward (alone, or with the gradients of dropout and the residual
// add) and its dispatch; instantiated per element type in layernorm_bwd_{bf16,f16,f32}.cu.
#pragma once

#include "dw_internal.h"
#include "residual.cuh"

namespace dwk {
namespace lnb {

enum Mode { kPlain, kFused, kFusedDrop };  // layer norm alone; with residual add; with dropout too

// Threads of a block, one block on an SM: as many as the registers of NO octets (dgamma, dbeta, xh and g:
// 32 registers an octet) and float32's staging area leave room for, a multiple of 128 so that the four
// partitions of an SM hold the same number of warps, and of TPR.  Spills (-Xptxas -v) are at most 32 bytes stored
// and 40 loaded a thread: 16-bit <32, 4> plain with edges and with dropout without them, bf16 <16, 2> with dropout
// and edges, float32 <16, 2> with the residual and edges and <32, 3> with dropout.  `heavy`: four octets
// with the residual, where either edges are held too (dropout+add+ln 32x1500x1023 bf16 95 us with 256 threads,
// 112 with 384 and spills) or no mask is drawn, so that memory is the bound and fewer rows at once suffice
// (32x1500x2048 bf16 150 us with 256, 174 with 384; with dropout 163 and 156).
constexpr bool heavy(bool SHIFT, int mode) { return mode == kFused || (SHIFT && mode == kFusedDrop); }
template <typename T> constexpr int threads_for(int TPR, int NO, bool four256) {
    constexpr bool f32 = sizeof(T) == 4;
    const int most = NO == 1   ? 768
                     : NO == 2 ? 512
                     : NO == 3 ? (f32 && TPR > 32 ? 256 : 384)
                               : (f32 || four256 ? 256 : 384);
    return most / TPR * TPR;
}

// Registers of a thread: what leaves room on every partition for one warp of 32 registers, so that the
// finalize kernel's blocks wait on the same SMs and start at once (4.4 -> 1.6 us behind 1024 channels).
template <typename T> constexpr int regs_for(int TPR, int NO, bool four256) {
    return (16384 - 1024) * 4 / threads_for<T>(TPR, NO, four256) / 8 * 8;
}

// A thread's own octets on their way from global to shared memory (cp.async): it waits for its own
// copies only and reads what it copied itself, so no barrier is involved.
template <typename T> __device__ __forceinline__ void stage_octet(void *dst, const T *src) {
    const uint32_t d = smem_addr(dst);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
    if constexpr (sizeof(T) == 4)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d + 16), "l"(src + 4) : "memory");
}
__device__ __forceinline__ void stage_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void stage_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The same for one element e of a 16-bit tensor of n elements, by way of the aligned 4 bytes it lies in (cp.async
// moves no fewer), or by itself where half of them lie outside the tensor.  Edges held in registers two
// rows ahead instead made a row wait for their loads (dropout+add+ln 32x1500x1023 bf16 111 us, staged 95; 777
// channels 104 / 87); float32 is faster with registers (32x1500x1023 104 us, staged 107).
template <typename T> constexpr bool kStageEdges = sizeof(T) == 2;
template <typename T> __device__ __forceinline__ int odd_half(const T *p) {
    return static_cast<int>(reinterpret_cast<uintptr_t>(p) / 2 & 1);
}
template <typename T> __device__ __forceinline__ void stage_edge(uint32_t *dst, const T *t, int64_t e, int64_t n) {
    const int half = odd_half(t + e);
    if (e >= half && e - half + 2 <= n)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(dst)), "l"(t + e - half) : "memory");
    else
        reinterpret_cast<T *>(dst)[half] = t[e];
}
template <typename T> __device__ __forceinline__ float staged_edge(const uint32_t *src, const T *t, int64_t e) {
    return load1(reinterpret_cast<const T *>(src) + odd_half(t + e));
}

// Thread-block clusters: all blocks arrived, and a float of another block's shared memory.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive;\n\tbarrier.cluster.wait;" ::: "memory");
}
__device__ __forceinline__ float cluster_load(const float *p, uint32_t rank) {
    uint32_t at;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}
constexpr int kCluster = 8;

// TPR threads hold a row's NO octets each, staged in shared memory two rows ahead of their use.
// Every thread keeps its channels from row to row, so dgamma and dbeta add up in registers over all
// its rows; the block's groups are then added in a fixed order through shared memory into the
// block's partial row.  `few` rows: the grid is one cluster of 8 blocks, which adds its blocks' rows
// itself (in order, through distributed shared memory) and writes dgamma and dbeta.  SHIFT: C or the
// tensors' address not a multiple of 8 elements, or gamma missing or misaligned.
//
// Bound by HBM for long batches; staged copies cost no registers, which dgamma and dbeta take (rows
// of 2048 bf16, 32x1500: 82 us, 196 with a block of 256 loading one row at a time).  Measured (graph
// replay, cold inputs, finalize included; fraction of the measured copy bandwidth): 32x1500x2048
// bf16 82.0 us (0.92), with dropout and residual 32x1500x1024 bf16 75.1 us (0.85) and 16x1500x512
// bf16 22.7 us (0.70), 16x1500x512 bf16 15.6 us (0.60), 8x733x519 float32 12.4 us (0.37).  The
// small ones pay about 3 us for the two sums after the last row (block 1.2 us, finalize 1.6 us)
// beside launch and first load, and for a last round of rows that few groups have: rows of 512 go 2368 at
// a time, so 24000 take 11 rounds for 10.1 and 5864 take 3 for 2.5.
template <typename T, int TPR, int NO, bool SHIFT, int MODE>
__global__ void __maxnreg__(regs_for<T>(TPR, NO, heavy(SHIFT, MODE)))
layernorm_bwd_rows_kernel(const ResidualArgs a, const int few) {
    constexpr int kThreads = threads_for<T>(TPR, NO, heavy(SHIFT, MODE)), GPB = kThreads / TPR;
    constexpr int kTensors = MODE == kPlain ? 2 : 3, kStages = 2;
    constexpr int kUnits = TPR < 32 && !SHIFT ? kThreads / 32 : GPB;
    static_assert(TPR <= 32 || GPB <= 15, "a named barrier per group, numbers 1 to 15");
    __shared__ float2 red_all[GPB][2 * (TPR > 32 ? TPR / 32 : 1)];
    extern __shared__ __align__(128) unsigned char smem[];
    launch_dependents();
    const int g = threadIdx.x / TPR, grid = gridDim.x, rows = static_cast<int>(a.B * a.T);
    const T *x = static_cast<const T *>(a.x), *dy = static_cast<const T *>(a.dy);
    const T *dh = MODE == kPlain ? nullptr : static_cast<const T *>(a.dh);
    T *dx = static_cast<T *>(a.dx), *dres = MODE == kPlain ? nullptr : static_cast<T *>(a.dres);
    float2 *red = red_all[g];
    const int first = blockIdx.x + grid * g;
    Channels<T, TPR, NO, SHIFT> ch;
    ch.start(static_cast<int>(a.C), first, a.phase);
    const int Q = shifted_q(ch.C);
    int off[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) off[i] = shifted_at(ch.head + i, Q) + ch.lane;
    // stages [kStages][kTensors][NO][kThreads] octets | gamma; at the end the units' dgamma, dbeta
    Oct<T> *stage = reinterpret_cast<Oct<T> *>(smem) + threadIdx.x;
    constexpr int kTensorStep = NO * kThreads, kStageStep = kTensors * kTensorStep;
    float *sp = reinterpret_cast<float *>(smem + static_cast<size_t>(kStages) * kStageStep * sizeof(Oct<T>));
    constexpr bool kEdgeStage = SHIFT && kStageEdges<T>;
    uint32_t *edge_stage = reinterpret_cast<uint32_t *>(sp + 8 * Q) + threadIdx.x;  // [kStages][kTensors][kThreads]
    const int64_t elements = static_cast<int64_t>(rows) * ch.C;
    float gamma_e = 0.f;
    grid_dependency_wait();

    // rows on their way: pipe.r is the next to request
    RowWalk pipe;
    pipe.start(a.lengths, first, grid * GPB, rows, static_cast<int>(a.T));
    uint32_t valid = 0;  // bit i: row i from the one at hand is valid
    float mean_q[kStages] = {}, rstd_q[kStages] = {};
    float xe_q[kStages] = {}, ge_q[kStages] = {}, he_q[kStages] = {};
    // buf: stage; slot: place in the queues and in valid.  Nothing is staged for a masked row: its copies,
    // which nobody waits for, could land after the next ones into the same stage.
    const auto request = [&](int buf, int slot) {
        if (pipe.in() && pipe.valid()) {
            valid |= 1u << slot;
            const int64_t e = ch.at(pipe.r);
            Oct<T> *st = stage + buf * kStageStep;
#pragma unroll
            for (int j = 0; j < NO; ++j) {
                if (!ch.any(j)) continue;
                stage_octet(st + j * kThreads, x + e + 8 * j * TPR);
                stage_octet(st + kTensorStep + j * kThreads, dy + e + 8 * j * TPR);
                if constexpr (MODE != kPlain)
                    if (dh) stage_octet(st + 2 * kTensorStep + j * kThreads, dh + e + 8 * j * TPR);
            }
            mean_q[slot] = a.mean[pipe.r];
            rstd_q[slot] = a.rstd[pipe.r];
            if (kEdgeStage && ch.edge()) {
                uint32_t *se = edge_stage + buf * (kTensors * kThreads);
                stage_edge(se, x, ch.edge_at(pipe.r), elements);
                stage_edge(se + kThreads, dy, ch.edge_at(pipe.r), elements);
                if (MODE != kPlain && dh) stage_edge(se + 2 * kThreads, dh, ch.edge_at(pipe.r), elements);
            } else if (ch.edge()) {
                xe_q[slot] = load1(x + ch.edge_at(pipe.r));
                ge_q[slot] = load1(dy + ch.edge_at(pipe.r));
                if (MODE != kPlain && dh) he_q[slot] = load1(dh + ch.edge_at(pipe.r));
            }
        }
        stage_commit();
        pipe.next();
    };
#pragma unroll
    for (int i = 0; i < kStages; ++i) request(i, i);
    // gamma from L1 for up to 1024 channels, from shared memory beyond (4096: 85 us instead of 91) and
    // with edges
    constexpr bool kShared = SHIFT || TPR > 32;
    if constexpr (kShared) {
        for (int c = threadIdx.x; c < ch.C; c += kThreads)
            sp[SHIFT ? shifted_at(c, Q) : halves_at(c, Q)] = a.gamma ? load_global(a.gamma + c) : 1.f;
        __syncthreads();
        if (ch.edge()) gamma_e = sp[shifted_at(ch.ce, Q)];
    }
    Dropper D;
    if constexpr (MODE == kFusedDrop) D.start(a.rng, a.thr);
    const float inv = 1.f / static_cast<float>(ch.C);
    int flip = 0, buf = 0, r = first;
    float2 ag[NO][4] = {}, ab[NO][4] = {};
    float age = 0.f, abe = 0.f;
    // groups of one warp walk together (their sums share its shuffles): until the first one is done
    int lead = TPR < 32 ? blockIdx.x + grid * (threadIdx.x / 32 * (32 / TPR)) : first;
    for (; lead < rows; lead += grid * GPB) {
        const bool live = valid & 1u;
        const int64_t e = ch.at(r);
        if (r < rows && !live) {
            ch.store_zeros(dx, r);
            if (dres) ch.store_zeros(dres, r);
        }
        if (TPR < 32 || live) {
            const float mean = mean_q[0], rstd = rstd_q[0];
            stage_wait<kStages - 1>();
            const Oct<T> *st = stage + buf * kStageStep;
            float2 s1 = make_float2(0.f, 0.f), s2 = s1;
            // xh of three and more octets is computed again from the staged x: registers for more warps
            constexpr bool kKeep = NO <= 2;
            float2 gg[NO][4], xh[kKeep ? NO : 1][4];
            float ge = 0.f, xhe = 0.f;
#pragma unroll
            for (int j = 0; j < NO; ++j) {
                // nothing was staged for a masked row or behind the row: zeros
                const bool on = TPR < 32 ? live && ch.any(j) : ch.any(j);
                Oct<T> xo, go;
                xo.zero();
                go.zero();
                if (on) {
                    xo = st[j * kThreads];
                    go = st[kTensorStep + j * kThreads];
                }
                float2(&h)[4] = xh[kKeep ? j : 0];
                xo.get(h);
                go.get(gg[j]);
                float2 ga[4];
                if constexpr (SHIFT) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        ga[i] = ch.any(j) ? make_float2(sp[off[2 * i] + j * TPR], sp[off[2 * i + 1] + j * TPR])
                                          : make_float2(0.f, 0.f);
                } else if constexpr (!kShared) {
                    load_params8(a.gamma + (ch.any(j) ? ch.c0(j) : 0), ga);
                } else {
                    const int v = ch.any(j) ? j * TPR + ch.lane : 0;
                    const float4 p = reinterpret_cast<const float4 *>(sp)[v];
                    const float4 q = reinterpret_cast<const float4 *>(sp)[Q + v];
                    ga[0] = make_float2(p.x, p.y); ga[1] = make_float2(p.z, p.w);
                    ga[2] = make_float2(q.x, q.y); ga[3] = make_float2(q.z, q.w);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    h[i] = fmul2(fadd2(h[i], both(-mean)), both(rstd));
                    ag[j][i] = ffma2(gg[j][i], h[i], ag[j][i]);
                    ab[j][i] = fadd2(ab[j][i], gg[j][i]);
                    gg[j][i] = fmul2(gg[j][i], ga[i]);
                    s1 = fadd2(s1, gg[j][i]);
                    s2 = ffma2(gg[j][i], h[i], s2);
                }
            }
            if constexpr (SHIFT) {
                if (kEdgeStage && ch.edge() && live) {
                    const uint32_t *se = edge_stage + buf * (kTensors * kThreads);
                    xe_q[0] = staged_edge(se, x, ch.edge_at(r));
                    ge_q[0] = staged_edge(se + kThreads, x, ch.edge_at(r));
                    if (MODE != kPlain && dh) he_q[0] = staged_edge(se + 2 * kThreads, x, ch.edge_at(r));
                }
                if (ch.edge() && live) {
                    xhe = (xe_q[0] - mean) * rstd;
                    age = fmaf(ge_q[0], xhe, age);
                    abe += ge_q[0];
                    ge = ge_q[0] * gamma_e;
                    s1.x += ge;
                    s2.x = fmaf(ge, xhe, s2.x);
                }
            }
            const float2 sum = row_sum<TPR>(make_float2(s1.x + s1.y, s2.x + s2.y), red, flip);
            const float c1 = sum.x * inv, c2 = sum.y * inv;
            if (live) {
#pragma unroll
                for (int j = 0; j < NO; ++j) {
                    float2 d[4] = {};
                    if constexpr (MODE != kPlain)
                        if (dh && ch.any(j)) st[2 * kTensorStep + j * kThreads].get(d);
                    float2(&h)[4] = xh[kKeep ? j : 0];
                    if constexpr (!kKeep) {
                        st[j * kThreads].get(h);
#pragma unroll
                        for (int i = 0; i < 4; ++i) h[i] = fmul2(fadd2(h[i], both(-mean)), both(rstd));
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 t = fadd2(gg[j][i], ffma2(h[i], both(-c2), both(-c1)));
                        gg[j][i] = MODE == kPlain ? fmul2(both(rstd), t) : ffma2(both(rstd), t, d[i]);
                    }
                }
                float de = 0.f;
                if constexpr (SHIFT) de = fmaf(rstd, ge - fmaf(xhe, c2, c1), MODE == kPlain ? 0.f : he_q[0]);
                if constexpr (MODE != kPlain) {
                    if (dres) {
                        ch.store_row(dres, e, gg);
                        if (ch.edge()) store1(dres + ch.edge_at(r), de);
                    }
                    if constexpr (MODE == kFusedDrop) {
                        if constexpr (SHIFT) D.apply(static_cast<uint32_t>(e >> 3), TPR, gg, ch.edge_at(r), de);
                        else D.apply(static_cast<uint32_t>(e >> 3), TPR, gg);
                    }
#pragma unroll
                    for (int j = 0; j < NO; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) gg[j][i] = fmul2(gg[j][i], both(a.mult));
                    de *= a.mult;
                }
                ch.store_row(dx, e, gg);
                if (ch.edge()) store1(dx + ch.edge_at(r), de);
            }
        }
        r += grid * GPB;
        valid >>= 1;
#pragma unroll
        for (int i = 0; i + 1 < kStages; ++i) {
            mean_q[i] = mean_q[i + 1];
            rstd_q[i] = rstd_q[i + 1];
            if constexpr (!kEdgeStage) {
                xe_q[i] = xe_q[i + 1];
                ge_q[i] = ge_q[i + 1];
                he_q[i] = he_q[i + 1];
            }
        }
        request(buf, kStages - 1);
        buf = buf + 1 == kStages ? 0 : buf + 1;
    }
    if (!a.dgamma && !a.dbeta) return;
    // the units' sums by channel: dgamma at slot[at], dbeta at slot[8 Q + at].  A unit is a group, or without
    // edges the groups of one warp, which hold the same channels and are added by shuffles.  Then the
    // units are added in order.
    const int64_t Cp = (a.C + 3) / 4 * 4;
    float *pg = a.partials + static_cast<int64_t>(blockIdx.x) * 2 * Cp;
    float *slots = reinterpret_cast<float *>(smem);  // the stages are done with
    if constexpr (TPR < 32 && !SHIFT) {
#pragma unroll
        for (int o = TPR; o < 32; o <<= 1)
#pragma unroll
            for (int j = 0; j < NO; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    ag[j][i] = plus(ag[j][i], shfl_xor(ag[j][i], o));
                    ab[j][i] = plus(ab[j][i], shfl_xor(ab[j][i], o));
                }
    }
    float *slot = slots + (TPR < 32 && !SHIFT ? static_cast<int>(threadIdx.x) / 32 : g) * 16 * Q;
    stage_wait<0>();
    __syncthreads();
    if (TPR >= 32 || SHIFT || static_cast<int>(threadIdx.x % 32) < TPR) {
#pragma unroll
        for (int j = 0; j < NO; ++j) {
            if (!ch.any(j)) continue;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                slot[off[i] + j * TPR] = i % 2 ? ag[j][i / 2].y : ag[j][i / 2].x;
                slot[8 * Q + off[i] + j * TPR] = i % 2 ? ab[j][i / 2].y : ab[j][i / 2].x;
            }
        }
        if (ch.edge()) {
            slot[shifted_at(ch.ce, Q)] = age;
            slot[8 * Q + shifted_at(ch.ce, Q)] = abe;
        }
    }
    __syncthreads();
    float *total = slots + kUnits * 16 * Q;  // few: this block's sums, [2][C]
    for (int c = threadIdx.x; c < 2 * ch.C; c += kThreads) {
        const int which = c >= ch.C, k = which ? c - ch.C : c;
        const float *p = slots + which * 8 * Q + shifted_at(k, Q);
        float t = p[0];
#pragma unroll
        for (int q = 1; q < kUnits; ++q) t += p[q * 16 * Q];
        if (few) total[c] = t;
        else pg[which * Cp + k] = t;
    }
    if (!few) return;
    cluster_sync();
    for (int c = blockIdx.x * kThreads + threadIdx.x; c < 2 * ch.C; c += kCluster * kThreads) {
        float t[kCluster];
#pragma unroll
        for (int q = 0; q < kCluster; ++q) t[q] = cluster_load(total + c, q);
#pragma unroll
        for (int q = 1; q < kCluster; ++q) t[0] += t[q];
        float *out = c < ch.C ? a.dgamma : a.dbeta;
        if (out) out[c < ch.C ? c : c - ch.C] = t[0];
    }
    cluster_sync();  // nobody leaves while its sums are read
}

template <typename T, int TPR, int NO, bool SHIFT, int MODE>
cudaError_t launch(const ResidualArgs &a, int *G, cudaStream_t s) {
    constexpr int kThreads = threads_for<T>(TPR, NO, heavy(SHIFT, MODE)), GPB = kThreads / TPR;
    constexpr int kTensors = MODE == kPlain ? 2 : 3;
    constexpr int kUnits = TPR < 32 && !SHIFT ? kThreads / 32 : GPB;
    const auto kern = layernorm_bwd_rows_kernel<T, TPR, NO, SHIFT, MODE>;
    const size_t words = 8 * static_cast<size_t>(shifted_q(static_cast<int>(a.C)));
    const size_t stages = 2 * static_cast<size_t>(kTensors) * NO * kThreads * sizeof(Oct<T>);
    const size_t edges = SHIFT && kStageEdges<T> ? 2 * kTensors * kThreads * sizeof(uint32_t) : 0;
    const size_t during = stages + words * sizeof(float) + edges, after = (kUnits + 1) * 2 * words * sizeof(float);
    const size_t smem = during > after ? during : after;
    if (smem > 226 * 1024) return cudaErrorNotSupported;
    // a carve-out with room for a finalize block beside this one (519 float32 channels: 5.0 us for 148 rows
    // instead of 7.6), the rest left to L1
    const size_t all = smem + sizeof(float2) * GPB * 2 * (TPR > 32 ? TPR / 32 : 1) + 4096;
    const int share = static_cast<int>(all * 100 / (228 * 1024)) + 1;
    static SmemGrant grant;
    const cudaError_t e =
        grant(reinterpret_cast<const void *>(kern), static_cast<int>(smem), share < 100 ? share : 100);
    if (e != cudaSuccess) return e;
    const int64_t rows = a.B * a.T;
    // one launch instead of two where half of one cluster's groups hold every row: the same time on the GPU
    // (64 rows of 512 bf16: 3.8 us either way; 256 rows: 4.9 us against 4.1) and 2.5 us less on the host
    if (rows <= kCluster * GPB / 2) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(kCluster);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        cudaLaunchAttribute at[2];
        at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[0].val.programmaticStreamSerializationAllowed = 1;
        at[1].id = cudaLaunchAttributeClusterDimension;
        at[1].val.clusterDim = {kCluster, 1, 1};
        cfg.attrs = at;
        cfg.numAttrs = 2;
        *G = 0;
        return cudaLaunchKernelEx(&cfg, kern, a, 1);
    }
    int64_t grid = sm_count();
    if (grid > a.G) grid = a.G;
    if (SHIFT && rows > grid * GPB) {  // more than one row a group: keep them a multiple of 8 apart
        constexpr int kMult = GPB % 8 == 0 ? 1 : (GPB % 4 == 0 ? 2 : (GPB % 2 == 0 ? 4 : 8));
        if (grid < kMult) return cudaErrorNotSupported;
        grid = grid / kMult * kMult;
    }
    *G = static_cast<int>(grid);
    return launch_programmatic(kern, dim3(static_cast<unsigned>(grid)), dim3(kThreads), smem, s, a, 0);
}

template <typename T, int TPR, int NO, bool SHIFT>
cudaError_t launch(const ResidualArgs &a, int *G, cudaStream_t s) {
    if (a.thr) return launch<T, TPR, NO, SHIFT, kFusedDrop>(a, G, s);
    if (a.dh || a.dres || a.mult != 1.f) return launch<T, TPR, NO, SHIFT, kFused>(a, G, s);
    return launch<T, TPR, NO, SHIFT, kPlain>(a, G, s);
}

// n: the octets of a row, C / 8 rounded down (edges need 16 lanes).
template <typename T, bool SHIFT>
cudaError_t launch_octets(const ResidualArgs &a, int64_t n, int *G, cudaStream_t s) {
    if constexpr (!SHIFT) {
        if (n <= 8) return launch<T, 8, 1, SHIFT>(a, G, s);
        if (n <= 16) return launch<T, 8, 2, SHIFT>(a, G, s);
    } else if (n <= 16) {
        return launch<T, 16, 1, SHIFT>(a, G, s);
    }
    if (n <= 32) return launch<T, 16, 2, SHIFT>(a, G, s);
    if (n <= 64) return launch<T, 32, 2, SHIFT>(a, G, s);
    if (n <= 96) return launch<T, 32, 3, SHIFT>(a, G, s);
    if (n <= 128) return launch<T, 32, 4, SHIFT>(a, G, s);
    if (n <= 192) return launch<T, 64, 3, SHIFT>(a, G, s);
    if (n <= 256) return launch<T, 64, 4, SHIFT>(a, G, s);
    if (n <= 384) return launch<T, 128, 3, SHIFT>(a, G, s);
    if (n <= 512) return launch<T, 128, 4, SHIFT>(a, G, s);
    if (n <= 768) return launch<T, 256, 3, SHIFT>(a, G, s);
    if (n <= 1024) return launch<T, 256, 4, SHIFT>(a, G, s);
    return cudaErrorNotSupported;
}

// cudaErrorNotSupported: no row kernel for these sizes or this alignment.
template <typename T>
cudaError_t launch_rows(const ResidualArgs &a, int *G, cudaStream_t s) {
    if (!row_kernels_serve(a)) return cudaErrorNotSupported;
    if (a.C % 8 == 0 && a.phase == 0 && a.gamma && reinterpret_cast<uintptr_t>(a.gamma) % 32 == 0)
        return launch_octets<T, false>(a, a.C / 8, G, s);
    return launch_octets<T, true>(a, a.C / 8, G, s);
}

}  // namespace lnb
}  // namespace dwk
