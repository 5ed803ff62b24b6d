"""CPU oracle of the residual path (fp64, plain loops): layer norm, dropout with the residual
add, and the two in sequence, forward and backward.

TEST INFRASTRUCTURE ONLY, like the rest of this package.  The arithmetic lives in
``residual_oracle.c``; pinned by ``tests/test_oracle_residual_pins.py``.
"""
from __future__ import annotations

import ctypes
import os
import threading

import numpy as np

from . import _D, _I, _L, _dp, _f64, _HERE, _ip, _lens
from . import build as _build

_SRC = os.path.join(_HERE, "residual_oracle.c")
_LIB_PATH = os.path.join(_HERE, "_build", "libresidual_oracle.so")
_lock = threading.Lock()
_lib = None
_U8 = ctypes.POINTER(ctypes.c_uint8)
_U32 = ctypes.POINTER(ctypes.c_uint32)
_F = ctypes.c_double


def build(force: bool = False) -> str:
    return _build(force, _SRC, _LIB_PATH)


def lib():
    global _lib
    with _lock:
        if _lib is None:
            h = ctypes.CDLL(build())
            h.oracle_philox4x32.argtypes = [_U32, _U32, _U32]
            h.oracle_dropout_kept.argtypes = [_L, _L, ctypes.c_uint64, ctypes.c_uint64, ctypes.c_uint32, _U8]
            h.oracle_dropout_add.argtypes = [_D, _D, _U8, _F, _I, _L, _L, _L, _D]
            h.oracle_layernorm_fwd.argtypes = [_D, _D, _D, _I, _L, _L, _L, _F, _D, _D, _D]
            h.oracle_layernorm_bwd.argtypes = [_D, _D, _D, _D, _D, _D, _I, _L, _L, _L, _D, _D, _D]
            for f in ("oracle_philox4x32", "oracle_dropout_kept", "oracle_dropout_add", "oracle_layernorm_fwd",
                      "oracle_layernorm_bwd"):
                getattr(h, f).restype = None
            _lib = h
    return _lib


def _opt(a):
    return None if a is None else _f64(a)


def philox4x32(counter, key):
    c, k, o = np.array(counter, np.uint32), np.array(key, np.uint32), np.zeros(4, np.uint32)
    lib().oracle_philox4x32(*(a.ctypes.data_as(_U32) for a in (c, k, o)))
    return o


def threshold(p) -> int:
    return int(np.floor(p * 65536.0 + 0.5))


def multiplier(p, alpha) -> float:
    """The factor of a kept element."""
    thr = threshold(p)
    return alpha * 65536.0 / (65536.0 - thr) if thr < 65536 else 0.0


def kept(shape, seed, offset, p, first=0):
    """Truth values: which elements of a [B, T, C] tensor (from flat index ``first`` on) the dropout
    keeps."""
    out = np.zeros(int(np.prod(shape)), np.uint8)
    lib().oracle_dropout_kept(int(first), out.size, int(seed) % 2 ** 64, int(offset) % 2 ** 64, threshold(p),
                              out.ctypes.data_as(_U8))
    return out.reshape(shape).astype(bool)


def dropout_add(x, residual, seed, offset, p, alpha, lengths):
    """s = [t < len_b] (residual + [kept] m x); residual may be None."""
    x, residual = _f64(x), _opt(residual)
    B, T, C = x.shape
    keep = np.ascontiguousarray(kept(x.shape, seed, offset, p), np.uint8) if threshold(p) else None
    s = np.empty_like(x)
    lib().oracle_dropout_add(_dp(x), _dp(residual), keep.ctypes.data_as(_U8) if keep is not None else None,
                             multiplier(p, alpha), _ip(_lens(lengths, B)), B, T, C, _dp(s))
    return s


def layernorm_fwd(x, gamma, beta, lengths, eps):
    """(y, mean, rstd)."""
    x, gamma, beta = _f64(x), _opt(gamma), _opt(beta)
    B, T, C = x.shape
    y, mean, rstd = np.empty_like(x), np.empty((B, T)), np.empty((B, T))
    lib().oracle_layernorm_fwd(_dp(x), _dp(gamma), _dp(beta), _ip(_lens(lengths, B)), B, T, C, eps, _dp(y), _dp(mean),
                               _dp(rstd))
    return y, mean, rstd


def layernorm_bwd(x, dy, gamma, mean, rstd, lengths, dh=None):
    """(dx, dgamma, dbeta); ``dh`` is added to dx on the valid frames."""
    x, dy, gamma, mean, rstd, dh = _f64(x), _f64(dy), _opt(gamma), _f64(mean), _f64(rstd), _opt(dh)
    B, T, C = x.shape
    dx, dgamma, dbeta = np.empty_like(x), np.empty(C), np.empty(C)
    lib().oracle_layernorm_bwd(_dp(x), _dp(dy), _dp(dh), _dp(gamma), _dp(mean), _dp(rstd), _ip(_lens(lengths, B)), B,
                               T, C, _dp(dx), _dp(dgamma), _dp(dbeta))
    return dx, dgamma, dbeta


def dropout_add_layernorm_fwd(x, residual, seed, offset, p, alpha, gamma, beta, lengths, eps):
    """(s, y, mean, rstd)."""
    s = dropout_add(x, residual, seed, offset, p, alpha, lengths)
    return (s, *layernorm_fwd(s, gamma, beta, lengths, eps))


def dropout_add_layernorm_bwd(dy, dh, h, gamma, mean, rstd, seed, offset, p, alpha, lengths):
    """(dx, dresidual, dgamma, dbeta)."""
    ds, dgamma, dbeta = layernorm_bwd(h, dy, gamma, mean, rstd, lengths, dh)
    return dropout_add(ds, None, seed, offset, p, alpha, lengths), ds, dgamma, dbeta
