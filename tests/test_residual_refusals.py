"""Argument checks of the residual path's C entry points: found on the host before any CUDA
call, so they run without a device.  Pointers are fake addresses that are never dereferenced."""
import pytest

import speech_encoder_depthwise_b200 as dw
from speech_encoder_depthwise_b200 import build as dwbuild

X, RES, Y, H, DY, DH, DX, DS = (0x10000000 * i for i in range(1, 9))
GA, BE, MEAN, RSTD, DGA, DBE, RNG, LN, WS = (0x100000000 + 0x1000000 * i for i in range(9))
B, T, C = 2, 10, 8


@pytest.fixture(scope="module")
def lib():
    dwbuild.build()
    return dw.lib()


FORMS = {
    "dw_layernorm_fwd": dict(x=X, gamma=GA, beta=BE, y=Y, mean=MEAN, rstd=RSTD, lengths=LN, B=B, T=T, C=C, eps=1e-5,
                             dt=dw.DW_BF16, stream=None),
    "dw_layernorm_bwd": dict(x=X, dy=DY, gamma=GA, mean=MEAN, rstd=RSTD, dx=DX, dgamma=DGA, dbeta=DBE, lengths=LN, B=B,
                             T=T, C=C, dt=dw.DW_BF16, ws=WS, wsn=1 << 20, stream=None),
    "dw_dropout_add_fwd": dict(x=X, res=RES, y=Y, rng=RNG, p=0.1, alpha=1.0, lengths=LN, B=B, T=T, C=C, dt=dw.DW_BF16,
                               stream=None),
    "dw_dropout_add_bwd": dict(dy=DY, dx=DX, rng=RNG, p=0.1, alpha=1.0, lengths=LN, B=B, T=T, C=C, dt=dw.DW_BF16,
                               stream=None),
    "dw_dropout_add_layernorm_fwd": dict(x=X, res=RES, rng=RNG, p=0.1, alpha=1.0, gamma=GA, beta=BE, h=H, y=Y,
                                         mean=MEAN, rstd=RSTD, lengths=LN, B=B, T=T, C=C, eps=1e-5, dt=dw.DW_BF16,
                                         stream=None),
    "dw_dropout_add_layernorm_bwd": dict(dy=DY, dh=DH, h=H, gamma=GA, mean=MEAN, rstd=RSTD, rng=RNG, p=0.1, alpha=1.0,
                                         dx=DX, dres=DS, dgamma=DGA, dbeta=DBE, lengths=LN, B=B, T=T, C=C,
                                         dt=dw.DW_BF16, ws=WS, wsn=1 << 20, stream=None),
}
NAN = float("nan")


def call(lib, fn, **kw):
    a = dict(FORMS[fn])
    a.update(kw)
    assert set(a) == set(FORMS[fn])
    return getattr(lib, fn)(*a.values())


@pytest.mark.parametrize("fn", list(FORMS))
def test_sizes_and_types(lib, fn):
    for kw in (dict(B=-1), dict(T=-1), dict(C=0), dict(dt=3), dict(dt=-1), dict(B=1 << 40, T=1 << 40)):
        assert call(lib, fn, **kw) == dw.DW_ERR_INVALID_ARG, kw
    assert call(lib, fn, C=(1 << 22) + 1) == dw.DW_ERR_UNSUPPORTED


@pytest.mark.parametrize("fn,required", [
    ("dw_layernorm_fwd", ["x", "y"]), ("dw_layernorm_bwd", ["x", "dy", "mean", "rstd", "dx"]),
    ("dw_dropout_add_fwd", ["x", "y", "rng"]), ("dw_dropout_add_bwd", ["dy", "dx", "rng"]),
    ("dw_dropout_add_layernorm_fwd", ["x", "y", "rng"]),
    ("dw_dropout_add_layernorm_bwd", ["dy", "h", "mean", "rstd", "rng", "dx"])])
def test_required_pointers(lib, fn, required):
    for name in required:
        assert call(lib, fn, **{name: None}) == dw.DW_ERR_INVALID_ARG, name


@pytest.mark.parametrize("fn", [f for f in FORMS if "dropout" in f])
def test_dropout_arguments(lib, fn):
    for kw in (dict(p=-0.01), dict(p=1.01), dict(p=NAN), dict(alpha=NAN), dict(alpha=float("inf")), dict(rng=RNG + 4),
               dict(alpha=1e300)):
        assert call(lib, fn, **kw) == dw.DW_ERR_INVALID_ARG, kw
    # checked for empty batches too
    assert call(lib, fn, B=0, p=2.0) == dw.DW_ERR_INVALID_ARG


@pytest.mark.parametrize("fn", [f for f in FORMS if "layernorm_fwd" in f])
def test_eps(lib, fn):
    for e in (-1e-5, NAN, float("inf")):
        assert call(lib, fn, eps=e) == dw.DW_ERR_INVALID_ARG


OUTS = {"y", "h", "dx", "dres", "mean", "rstd", "dgamma", "dbeta"}
INS = {"x", "res", "dy", "dh", "gamma", "beta", "rng", "lengths"}


@pytest.mark.parametrize("fn", list(FORMS))
def test_outputs_overlap_nothing(lib, fn):
    form = FORMS[fn]
    back = fn.endswith("bwd")
    outs = [n for n in form if n in OUTS and not (back and n in ("mean", "rstd", "h"))]
    ins = [n for n in form if n in INS or (back and n in ("mean", "rstd", "h"))]
    for i, o in enumerate(outs):
        for other in ins + outs[:i]:
            assert call(lib, fn, **{o: form[other]}) == dw.DW_ERR_INVALID_ARG, (o, other)
            assert call(lib, fn, **{o: form[other] + 4}) == dw.DW_ERR_INVALID_ARG, (o, other)
    if back and "ws" in form:
        for o in outs + ins:
            assert call(lib, fn, ws=form[o]) == dw.DW_ERR_INVALID_ARG, o


@pytest.mark.parametrize("fn", ["dw_layernorm_bwd", "dw_dropout_add_layernorm_bwd"])
def test_workspace(lib, fn):
    n = dw.dw_layernorm_bwd_workspace_size(B, T, C)
    assert n > 0 and n % 16 == 0
    for kw in (dict(ws=None), dict(wsn=n - 1), dict(ws=WS + 8), dict(ws=None, dgamma=None)):
        assert call(lib, fn, **kw) == dw.DW_ERR_WORKSPACE, kw
    assert dw.dw_layernorm_bwd_workspace_size(0, T, C) == 0
    assert dw.dw_layernorm_bwd_workspace_size(B, T, 0) == 0
    assert dw.dw_layernorm_bwd_workspace_size(1 << 40, 1 << 40, 8) == 0
    # bounded however wide the rows are
    assert 0 < dw.dw_layernorm_bwd_workspace_size(64, 3000, 1 << 22) <= 64 << 20
    assert dw.dw_layernorm_bwd_workspace_size(64, 3000, 1024) <= 64 << 20


@pytest.mark.parametrize("fn", list(FORMS))
def test_empty_batches_touch_no_device(lib, fn):
    none = {n: None for n in FORMS[fn] if n in OUTS | INS | {"ws", "h"}}
    if "wsn" in FORMS[fn]:
        none["wsn"] = 0
    assert call(lib, fn, B=0, **none) == dw.DW_OK
    assert call(lib, fn, T=0, **none) == dw.DW_OK
