"""The fused forward and backward as a pair (GPU), against the fp64 gradients of the exact function."""
import numpy as np
import pytest
import torch

import speech_encoder_depthwise_b200 as dw
from gpuhelp import dev
from oracle import residual as orc
from residualpin import TD, assert_within, layernorm_bwd_err, layernorm_fwd_err, param_err, store, sum_err
from test_parity_residual import EPS, Case, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    from speech_encoder_depthwise_b200 import build
    build.build()
    dw.lib()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("B,T,C", [(4, 300, 512), (3, 400, 519), (2, 150, 2048), (2, 20, 8200)])
@pytest.mark.parametrize("mean", [0.0, 30.0])
@pytest.mark.parametrize("p", [0.0, 0.2])
def test_forward_and_backward_as_a_pair(B, T, C, dtype, mean, p):
    """The gradients of the exact function at the forward's inputs.  The backward rebuilds xh from the stored h and
    the float32 statistics, so xh is off by (half a step of h + the mean's error) rstd + its share of rstd's error:
    the bound follows that through the formula.  mean: the residual stream's, in deviations of a row."""
    c = Case(B, T, C, dtype, lengths=[T] + [T // 2] * (B - 1), seed=C)
    f = torch.finfo(TD[dtype])
    c.res = torch.from_numpy(c.res + np.float32(mean)).to(TD[dtype]).float().numpy()
    alpha, mult, rng = 0.5, orc.multiplier(p, 0.5), c.rng if p else None
    h, y, dx, ds = (c.out() for _ in range(4))
    m, r = torch.empty(B, T, device="cuda"), torch.empty(B, T, device="cuda")
    dg, db = torch.empty(C, device="cuda"), torch.empty(C, device="cuda")
    ws, G, per = workspace(c)
    dw.dw_dropout_add_layernorm_fwd(c.act(c.x), c.act(c.res), rng, p, alpha, dev(c.gamma), dev(c.beta), h.t, y.t, m, r, c.ln,
                                    EPS)
    dw.dw_dropout_add_layernorm_bwd(c.act(c.dy), c.act(c.dh), h.t, dev(c.gamma), m, r, rng, p, alpha, dx.t, ds.t, dg, db,
                                    c.ln, ws.t)
    got = c.done(dx=dx, ds=ds)

    v = c.valid[..., None].astype(np.float64)
    s, ry, rm, rr = orc.dropout_add_layernorm_fwd(c.x, c.res, c.seed, c.off, p, alpha, c.gamma, c.beta, c.lengths, EPS)
    rdx, rds, rdg, rdb = orc.dropout_add_layernorm_bwd(c.dy, c.dh, s, c.gamma, rm, rr, c.seed, c.off, p, alpha, c.lengths)
    es = sum_err(s, mult * c.x * v)
    _, em, er = layernorm_fwd_err(s, ry, rm, rr, c.gamma, c.beta, es)
    half = 0.0 if dtype == "f32" else f.eps / 2 * np.maximum(np.abs(s) + es, f.tiny)
    R = rr[..., None]
    rel = er[..., None] / np.maximum(R, 1e-30)
    xh, g = (s - rm[..., None]) * R, c.dy * c.gamma * v
    d = (1 + rel) * R * (half + es + em[..., None]) + np.abs(xh) * rel
    c2 = (g * xh).mean(-1, keepdims=True)
    t = g - g.mean(-1, keepdims=True) - xh * c2
    gd = (np.abs(g) * d).mean(-1, keepdims=True)
    e = R * (1 + rel) * (d * np.abs(c2) + np.abs(xh) * gd + d * gd) + np.abs(t) * R * rel
    # the arithmetic's own error, at the magnitudes that xh has with its error
    stored = rm[..., None] + np.sign(xh) * (np.abs(xh) + d) / np.maximum(R, 1e-30)
    e = (e + 1.01 * layernorm_bwd_err(stored, c.dy, c.gamma, rm, rr, c.dh)) * v
    assert_within("dresidual", got["ds"], rds, store(dtype, rds, e))
    assert_within("dx", got["dx"], rdx, store(dtype, rdx, (mult * e + 2.0 ** -23 * np.abs(rdx)) * (rdx != 0)))
    eg, eb = param_err(stored, c.dy, rm, rr, c.valid, per, G)
    assert_within("dgamma", dg.cpu().numpy(), rdg, 1.01 * eg + (np.abs(c.dy) * d * v).sum((0, 1)) + 1e-30)
    assert_within("dbeta", db.cpu().numpy(), rdb, eb + 1e-30)


def test_generator_state_that_is_not_read_may_lie_anywhere():
    """p = 0 draws nothing: rng may then be memory that the call writes."""
    x = torch.randn(1, 4, 8, device="cuda")
    y, h, dx = (torch.empty_like(x) for _ in range(3))
    m, r = torch.empty(1, 4, device="cuda"), torch.empty(1, 4, device="cuda")

    def inside(t):
        return t.view(-1)[4:8].view(torch.int64)
    dw.dw_dropout_add_fwd(x, None, y, inside(y), 0.0, 1.0, None)
    assert torch.equal(y, x)
    dw.dw_dropout_add_layernorm_fwd(x, None, inside(h), 0.0, 1.0, None, None, h, y, m, r, None)
    assert torch.equal(h, x)
    dw.dw_dropout_add_layernorm_bwd(y, y, x, None, m, r, inside(dx), 0.0, 1.0, dx, None, None, None, None, None)
    torch.cuda.synchronize()
    assert torch.isfinite(dx).all()
    with pytest.raises(dw.DwError):  # read: refused
        dw.dw_dropout_add_fwd(x, None, y, inside(y), 0.5, 1.0, None)
