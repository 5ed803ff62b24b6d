"""Pointers that are no multiple of their element's size: every entry point refuses them on the host
(a kernel's load or store there would fault).  Pointers are fake addresses that are never dereferenced."""
import pytest

import speech_encoder_depthwise_b200 as dw
from speech_encoder_depthwise_b200 import build as dwbuild

B, T, F, C, K = 2, 16, 8, 8, 3
ACT, PARAM = "activation", "float32 or int32"
A = iter(range(0x10000000, 0x7fffffff0000, 0x10000000))


def ptrs(kind, *names):
    return [(n, kind, next(A)) for n in names]


def sizes(*values):
    return [(None, None, v) for v in values]


DT = [("dt", None, dw.DW_BF16)]
ST = sizes(None)


def ws(n):
    return [(None, None, next(A)), (None, None, n)]


BIG = 1 << 26
CALLS = {
    "dwconv1d_fwd": [*ptrs(ACT, "x"), *ptrs(PARAM, "w", "bias"), *ptrs(ACT, "y"), *ptrs(PARAM, "lengths"),
                     *sizes(B, T, C, K, 1), *DT, *ST],
    "dwconv1d_bwd_dx": [*ptrs(ACT, "dy"), *ptrs(PARAM, "w"), *ptrs(ACT, "dx"), *ptrs(PARAM, "lengths"),
                        *sizes(B, T, C, K, 1), *DT, *ST],
    "dwconv1d_bwd": [*ptrs(ACT, "x", "dy"), *ptrs(PARAM, "w"), *ptrs(ACT, "dx"), *ptrs(PARAM, "dw", "dbias", "lengths"),
                     *sizes(B, T, C, K, 1), *DT, *ws(BIG), *ST],
    "dwconv1d_bwd_dw": [*ptrs(ACT, "x", "dy"), *ptrs(PARAM, "dw", "dbias", "lengths"), *sizes(B, T, C, K, 1), *DT, *ws(BIG),
                        *ST],
    "dwconv1d_bwd_dw_noalloc": [*ptrs(ACT, "x", "dy"), *ptrs(PARAM, "dw", "dbias", "lengths"), *sizes(B, T, C, K, 1), *DT,
                                *ST],
    "dwconv1d_fwd_packed": [*ptrs(ACT, "x"), *ptrs(PARAM, "w", "bias"), *ptrs(ACT, "y"), *ptrs(PARAM, "offsets"),
                            *sizes(B, T, C, K, 1), *DT, *ST],
    "dwconv1d_bwd_dx_packed": [*ptrs(ACT, "dy"), *ptrs(PARAM, "w"), *ptrs(ACT, "dx"), *ptrs(PARAM, "offsets"),
                               *sizes(B, T, C, K, 1), *DT, *ST],
    "dwconv1d_bwd_dw_packed": [*ptrs(ACT, "x", "dy"), *ptrs(PARAM, "dw", "dbias", "offsets"), *sizes(B, T, C, K, 1), *DT,
                               *ws(BIG), *ST],
    "dwconv1d_stream_fwd": [*ptrs(ACT, "x"), *ptrs(PARAM, "w", "bias"), *ptrs(ACT, "y", "cache"), *ptrs(PARAM, "lengths"),
                            *sizes(B, T, C, K), *DT, *ST],
    "dw_subsample_fwd": [*ptrs(PARAM, "mel", "w0", "b0", "w1", "b1"), *ptrs(ACT, "out"),
                         *ptrs(PARAM, "lengths", "out_lengths"), *sizes(B, T, F, C, 0), *DT, *ST],
    "dw_subsample_fwd_simt": [*ptrs(PARAM, "mel", "w0", "b0", "w1", "b1"), *ptrs(ACT, "out"),
                              *ptrs(PARAM, "lengths", "out_lengths"), *sizes(B, T, F, C, 0), *DT, *ST],
    "dw_subsample_bwd": [*ptrs(PARAM, "mel", "w0", "b0", "w1"), *ptrs(ACT, "dout"),
                         *ptrs(PARAM, "lengths", "dw0", "db0", "dw1", "db1"), *sizes(B, T, F, C, 0), *DT, *ws(BIG), *ST],
    "dwconv2d_fwd": [*ptrs(ACT, "x"), *ptrs(PARAM, "w", "bias"), *ptrs(ACT, "y"), *ptrs(PARAM, "lengths", "out_lengths"),
                     *sizes(B, T, F, C, 3, 3, 2, 2, 1, 1, 1), *DT, *ST],
    "dwconv2d_bwd_dx": [*ptrs(ACT, "dy"), *ptrs(PARAM, "w"), *ptrs(ACT, "dx"), *ptrs(PARAM, "lengths"),
                        *sizes(B, T, F, C, 3, 3, 2, 2, 1, 1, 1), *DT, *ST],
    "dwconv2d_bwd_dw": [*ptrs(ACT, "x", "dy"), *ptrs(PARAM, "dw", "dbias", "lengths"),
                        *sizes(B, T, F, C, 3, 3, 2, 2, 1, 1, 1), *DT, *ws(BIG), *ST],
    "dw_layernorm_fwd": [*ptrs(ACT, "x"), *ptrs(PARAM, "gamma", "beta"), *ptrs(ACT, "y"),
                         *ptrs(PARAM, "mean", "rstd", "lengths"), *sizes(B, T, C, 1e-5), *DT, *ST],
    "dw_layernorm_bwd": [*ptrs(ACT, "x", "dy"), *ptrs(PARAM, "gamma", "mean", "rstd"), *ptrs(ACT, "dx"),
                         *ptrs(PARAM, "dgamma", "dbeta", "lengths"), *sizes(B, T, C), *DT, *ws(BIG), *ST],
    "dw_dropout_add_fwd": [*ptrs(ACT, "x", "residual", "y"), *ptrs(PARAM, "rng"), *sizes(0.1, 1.0), *ptrs(PARAM, "lengths"),
                           *sizes(B, T, C), *DT, *ST],
    "dw_dropout_add_bwd": [*ptrs(ACT, "dy", "dx"), *ptrs(PARAM, "rng"), *sizes(0.1, 1.0), *ptrs(PARAM, "lengths"),
                           *sizes(B, T, C), *DT, *ST],
    "dw_dropout_add_layernorm_fwd": [*ptrs(ACT, "x", "residual"), *ptrs(PARAM, "rng"), *sizes(0.1, 1.0),
                                     *ptrs(PARAM, "gamma", "beta"), *ptrs(ACT, "h", "y"),
                                     *ptrs(PARAM, "mean", "rstd", "lengths"), *sizes(B, T, C, 1e-5), *DT, *ST],
    "dw_dropout_add_layernorm_bwd": [*ptrs(ACT, "dy", "dh", "h"), *ptrs(PARAM, "gamma", "mean", "rstd", "rng"),
                                     *sizes(0.1, 1.0), *ptrs(ACT, "dx", "dresidual"),
                                     *ptrs(PARAM, "dgamma", "dbeta", "lengths"), *sizes(B, T, C), *DT, *ws(BIG), *ST],
    "dw_selftest_wait_timeout": [*ptrs(PARAM, "done"), *ST],
}


@pytest.fixture(scope="module")
def lib():
    dwbuild.build()
    return dw.lib()


def test_every_entry_point_with_pointers_is_here():
    with_pointers = {n for n, (_, args) in dw.SIGNATURES.items() if dw._vp in args}
    assert set(CALLS) == with_pointers
    for n, call in CALLS.items():
        assert len(call) == len(dw.SIGNATURES[n][1]), n


@pytest.mark.parametrize("fn", list(CALLS))
@pytest.mark.parametrize("dtype", [dw.DW_F32, dw.DW_BF16, dw.DW_F16])
def test_pointers_between_elements_are_refused(lib, fn, dtype):
    values = [dtype if name == "dt" else v for name, _, v in CALLS[fn]]
    for i, (name, kind, p) in enumerate(CALLS[fn]):
        if kind is None:
            continue
        size = 2 if kind == ACT and dtype != dw.DW_F32 else 4
        for off in range(1, size):
            args = list(values)
            args[i] = p + off
            assert getattr(lib, fn)(*args) == dw.DW_ERR_INVALID_ARG, (name, off)
