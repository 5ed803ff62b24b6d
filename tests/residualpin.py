"""Error bounds of the residual-path kernels, element by element, from their arithmetic.

u = 2^-24 is float32's half step.  A stored output adds half a step of its type,
``finfo(t).eps / 2`` relative to the value (at least that times the smallest normal number, the
half step of the subnormal numbers).  Sums of C float32 terms have a depth (the longest chain of additions) of
at most K = C / 256 + 64 in every kernel (a block of 256 threads, or a warp holding up to 32
elements a lane, then trees), so they are off by at most K u times the sum of the absolute terms.
"""
import numpy as np
import torch

U = 2.0 ** -24
TD = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def depth(C):
    return C / 256 + 64


def store(dtype, v, err):
    """The bound of a stored value: its float32 error and half a step of the stored one."""
    f = torch.finfo(TD[dtype])
    half = 0.0 if dtype == "f32" else f.eps / 2  # a float32 store rounds nothing further
    return err + half * np.maximum(np.abs(v) + err, f.tiny)


def sum_err(s, keep_mx):
    """s = res + m x by one fused multiply-add, m rounded: u (|m x| + |s|)."""
    return U * (np.abs(keep_mx) + np.abs(s))


def layernorm_fwd_err(s, y, mean, rstd, gamma, beta, ds):
    """(y, mean, rstd) errors; ds: the error of s."""
    C = s.shape[-1]
    K = depth(C)
    ga, be = (1.0 if gamma is None else np.abs(gamma)), (0.0 if beta is None else np.abs(beta))
    dsm = ds.max(-1, keepdims=True)
    m, r = mean[..., None], rstd[..., None]
    e_mean = (K + 2) * U * np.abs(s).mean(-1, keepdims=True) + dsm
    d = np.abs(s - m)
    # the variance: centred terms off by u |d| + e_mean + ds, their squares summed in K steps; second-order
    # terms doubled in.  rstd halves its relative error; sqrt and the division add at most 4 u
    sd = 1.0 / np.maximum(r, 1e-30)
    e_d = U * d + e_mean + ds
    e_var = 2 * (d * e_d).mean(-1, keepdims=True) + (e_d ** 2).mean(-1, keepdims=True) + (K + 4) * U * sd ** 2
    rel_r = 0.5 * e_var / sd ** 2 + 4 * U
    e_y = ga * r * e_d + (np.abs(y) + be) * (rel_r + 4 * U)
    return 1.05 * e_y, 1.05 * e_mean[..., 0], 1.05 * (rel_r * r)[..., 0]


def layernorm_bwd_err(h, dy, gamma, mean, rstd, dh):
    C = h.shape[-1]
    K = depth(C)
    r = rstd[..., None]
    xh = np.abs(h - mean[..., None]) * r
    g = np.abs(dy * (1.0 if gamma is None else gamma))
    A, Bm = g.mean(-1, keepdims=True), (g * xh).mean(-1, keepdims=True)
    e = U * r * (6 * (g + A + xh * Bm) + (K + 2) * A + xh * (K + 6) * Bm)
    return e + (U * (np.abs(dh) + r * (g + A + xh * Bm)) if dh is not None else 0.0)


def param_err(h, dy, mean, rstd, valid, rows_per_block, G):
    """dgamma, dbeta: rows in a chain, the block's warps and the partial rows after it."""
    D = rows_per_block + G / 8 + 40
    v = valid[..., None]
    xh = np.abs(h - mean[..., None]) * rstd[..., None]
    return U * (D + 3) * (np.abs(dy) * xh * v).sum((0, 1)), U * D * (np.abs(dy) * v).sum((0, 1))


def assert_within(name, got, ref, bound):
    got = np.asarray(got, np.float64)
    bad = ~(np.abs(got - ref) <= bound)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.abs(got - ref) / np.maximum(bound, 1e-300), 0)), got.shape)
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.size} beyond the bound, worst at {i}: got {got[i]!r} "
                             f"want {ref[i]!r} bound {np.broadcast_to(bound, got.shape)[i]:.3g}")
