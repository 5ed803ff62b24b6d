"""GPU parity of the residual path (layer norm, dropout with the residual add, the two in one
pass; forward and backward) against the fp64 oracle, with element-wise bounds derived from the
arithmetic (residualpin).  Masked frames of every input hold NaN and must not matter; every
output lies between guard bands."""
import numpy as np
import pytest
import torch

import speech_encoder_depthwise_b200 as dw
from gpuhelp import Guarded, assert_masked_zero, dev
from oracle import residual as orc
from residualpin import (TD, assert_within, layernorm_bwd_err, layernorm_fwd_err, param_err, store, sum_err)
from synth import bf16_round, f16_round

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    from speech_encoder_depthwise_b200 import build
    build.build()
    dw.lib()


def rounded(a, dtype):
    a = np.ascontiguousarray(a, np.float32)
    return bf16_round(a) if dtype == "bf16" else f16_round(a) if dtype == "f16" else a


class Case:
    """Inputs of one size: activations rounded to the type, masked frames of the device copies NaN."""

    def __init__(self, B, T, C, dtype, lengths=None, seed=0, offset=0, scale=1.0, shift=0.5):
        r = np.random.default_rng(seed)
        self.B, self.T, self.C, self.dtype, self.offset = B, T, C, dtype, offset
        chan = shift * r.standard_normal(C)
        self.x = rounded(scale * (r.standard_normal((B, T, C)) + chan), dtype)
        self.res = rounded(scale * (r.standard_normal((B, T, C)) + chan), dtype)
        self.dy = rounded(r.standard_normal((B, T, C)), dtype)
        self.dh = rounded(r.standard_normal((B, T, C)), dtype)
        self.gamma = (1 + 0.2 * r.standard_normal(C)).astype(np.float32)
        self.beta = (0.2 * r.standard_normal(C)).astype(np.float32)
        self.seed, self.off = (int(v) for v in r.integers(0, 2 ** 63 - 1, 2))
        self.lengths = None if lengths is None else np.asarray(lengths, np.int32)
        L = np.full(B, T) if lengths is None else np.clip(self.lengths, 0, T)
        self.valid = np.arange(T)[None] < L[:, None]
        self.rng = torch.tensor([self.seed, self.off], dtype=torch.int64, device="cuda")
        self.ln = dev(self.lengths)

    def act(self, a):
        """Device copy at the case's element offset from 16-byte alignment, masked frames NaN."""
        g = Guarded(a.shape, TD[self.dtype], offset=self.offset)
        g.t.copy_(torch.from_numpy(np.where(self.valid[..., None], a, np.float32("nan"))).to(TD[self.dtype]))
        return g.t

    def out(self):
        return Guarded((self.B, self.T, self.C), TD[self.dtype], offset=self.offset)

    def done(self, **outs):
        torch.cuda.synchronize()
        r = {}
        for k, g in outs.items():
            if g is None:
                continue
            g.check_slack()
            r[k] = g.numpy()
            if r[k].ndim >= 2:
                assert_masked_zero(r[k], self.lengths, self.T)
        return r


def f32g(*shape):
    return Guarded(shape, torch.float32)


def run_ln_fwd(c, gamma=True, beta=True, stats=True, eps=EPS):
    ga, be = (c.gamma if gamma else None), (c.beta if beta else None)
    y, mean, rstd = c.out(), f32g(c.B, c.T) if stats else None, f32g(c.B, c.T) if stats else None
    dw.dw_layernorm_fwd(c.act(c.x), dev(ga), dev(be), y.t, mean.t if stats else None, rstd.t if stats else None, c.ln,
                        eps)
    got = c.done(y=y, mean=mean, rstd=rstd)
    ry, rm, rr = orc.layernorm_fwd(c.x, ga, be, c.lengths, eps)
    s = c.x * c.valid[..., None].astype(np.float64)
    ey, em, er = layernorm_fwd_err(s, ry, rm, rr, ga, be, np.zeros(c.x.shape))
    assert_within("y", got["y"], ry, store(c.dtype, ry, ey))
    if stats:
        assert_within("mean", got["mean"], rm, em)
        assert_within("rstd", got["rstd"], rr, er)


def backward_inputs(c):
    """mean and rstd of x in float32, as a forward pass keeps them."""
    _, m, r = orc.layernorm_fwd(c.x, None, None, c.lengths, EPS)
    m, r = m.astype(np.float32), r.astype(np.float32)
    nan = np.float32("nan")
    return m, r, dev(np.where(c.valid, m, nan)), dev(np.where(c.valid, r, nan))


def workspace(c):
    n = dw.dw_layernorm_bwd_workspace_size(c.B, c.T, c.C)
    g = Guarded((max(n, 16) // 4,), torch.float32)
    G = n // (8 * ((c.C + 3) // 4 * 4))
    return g, G, c.B * c.T / G


def check_params(c, got, ref, m, r, G, per):
    eg, eb = param_err(c.x, c.dy, m, r, c.valid, per, G)
    if "dgamma" in got:
        assert_within("dgamma", got["dgamma"], ref[-2], eg + 1e-30)
    if "dbeta" in got:
        assert_within("dbeta", got["dbeta"], ref[-1], eb + 1e-30)


def run_ln_bwd(c, gamma=True, dgamma=True, dbeta=True):
    ga = c.gamma if gamma else None
    m, r, mt, rt = backward_inputs(c)
    dx, dg, db = c.out(), f32g(c.C) if dgamma else None, f32g(c.C) if dbeta else None
    ws, G, per = workspace(c)
    dw.dw_layernorm_bwd(c.act(c.x), c.act(c.dy), dev(ga), mt, rt, dx.t, dg.t if dg else None, db.t if db else None,
                        c.ln, ws.t if dg or db else None)
    got = c.done(dx=dx, dgamma=dg, dbeta=db)
    ws.check_slack()
    ref = orc.layernorm_bwd(c.x, c.dy, ga, m, r, c.lengths)
    assert_within("dx", got["dx"], ref[0], store(c.dtype, ref[0], layernorm_bwd_err(c.x, c.dy, ga, m, r, None)))
    check_params(c, got, ref, m, r, G, per)


def run_drop(c, p, alpha, residual=True):
    res = c.res if residual else None
    y, dx = c.out(), c.out()
    dw.dw_dropout_add_fwd(c.act(c.x), c.act(c.res) if residual else None, y.t, c.rng, p, alpha, c.ln)
    dw.dw_dropout_add_bwd(c.act(c.dy), dx.t, c.rng, p, alpha, c.ln)
    got = c.done(y=y, dx=dx)
    ry = orc.dropout_add(c.x, res, c.seed, c.off, p, alpha, c.lengths)
    rdx = orc.dropout_add(c.dy, None, c.seed, c.off, p, alpha, c.lengths)
    assert_within("y", got["y"], ry, store(c.dtype, ry, sum_err(ry, orc.multiplier(p, alpha) * c.x)))
    assert_within("dx", got["dx"], rdx, store(c.dtype, rdx, sum_err(rdx, rdx)))
    # the mask itself, exactly: a dropped gradient is +0
    keep = orc.kept(c.dy.shape, c.seed, c.off, p) & c.valid[..., None]
    assert (got["dx"][~keep] == 0).all()
    if orc.multiplier(p, alpha) and c.dtype != "f16":
        assert (got["dx"][keep & (c.dy != 0)] != 0).all()


def run_dal_fwd(c, p, alpha, residual=True, h=True, stats=True, gamma=True, beta=True):
    res, ga, be = (c.res if residual else None), (c.gamma if gamma else None), (c.beta if beta else None)
    hg, y = c.out() if h else None, c.out()
    mean, rstd = (f32g(c.B, c.T), f32g(c.B, c.T)) if stats else (None, None)
    dw.dw_dropout_add_layernorm_fwd(c.act(c.x), c.act(c.res) if residual else None, c.rng if p else None, p, alpha,
                                    dev(ga), dev(be), hg.t if h else None, y.t, mean.t if stats else None,
                                    rstd.t if stats else None, c.ln, EPS)
    got = c.done(h=hg, y=y, mean=mean, rstd=rstd)
    s, ry, rm, rr = orc.dropout_add_layernorm_fwd(c.x, res, c.seed, c.off, p, alpha, ga, be, c.lengths, EPS)
    es = sum_err(s, orc.multiplier(p, alpha) * c.x * c.valid[..., None])
    ey, em, er = layernorm_fwd_err(s, ry, rm, rr, ga, be, es)
    if h:
        assert_within("h", got["h"], s, store(c.dtype, s, es))
    assert_within("y", got["y"], ry, store(c.dtype, ry, ey))
    if stats:
        assert_within("mean", got["mean"], rm, em)
        assert_within("rstd", got["rstd"], rr, er)


def run_dal_bwd(c, p, alpha, dh=True, dres=True, gamma=True, dgamma=True, dbeta=True):
    ga = c.gamma if gamma else None
    m, r, mt, rt = backward_inputs(c)
    dx, ds = c.out(), c.out() if dres else None
    dg, db = f32g(c.C) if dgamma else None, f32g(c.C) if dbeta else None
    ws, G, per = workspace(c)
    dw.dw_dropout_add_layernorm_bwd(c.act(c.dy), c.act(c.dh) if dh else None, c.act(c.x), dev(ga), mt, rt,
                                    c.rng if p else None, p, alpha, dx.t, ds.t if dres else None,
                                    dg.t if dg else None, db.t if db else None, c.ln, ws.t)
    got = c.done(dx=dx, dres=ds, dgamma=dg, dbeta=db)
    ws.check_slack()
    ref = orc.dropout_add_layernorm_bwd(c.dy, c.dh if dh else None, c.x, ga, m, r, c.seed, c.off, p, alpha, c.lengths)
    es = layernorm_bwd_err(c.x, c.dy, ga, m, r, c.dh if dh else None)
    if dres:
        assert_within("dresidual", got["dres"], ref[1], store(c.dtype, ref[1], es))
    mult = orc.multiplier(p, alpha)
    assert_within("dx", got["dx"], ref[0], store(c.dtype, ref[0], (mult * es + 2.0 ** -23 * np.abs(ref[0])) * (ref[0] != 0)))
    check_params(c, got, ref, m, r, G, per)


def run_all(c, p=0.1, alpha=0.5):
    run_ln_fwd(c)
    run_ln_bwd(c)
    run_drop(c, p, alpha)
    run_dal_fwd(c, p, alpha)
    run_dal_bwd(c, p, alpha)


DTYPES = ["bf16", "f16", "f32"]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("C", [1, 2, 7, 8, 31, 64, 80, 127, 130, 256, 257, 512, 519, 520, 768, 1023, 1024, 1025, 1500,
                               2047, 2048, 3001, 4096, 4100])
def test_channel_counts(C, dtype):
    """Rows on and off 16-byte boundaries, every width of the kernels, lengths with an empty item."""
    run_all(Case(4, 13, C, dtype, lengths=[13, 0, 7, 1], seed=C))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("C", [5000, 8191, 8192, 8200, 12345, 20000])
def test_wide_rows(C, dtype):
    run_all(Case(2, 5, C, dtype, lengths=[5, 2], seed=C))


@pytest.mark.parametrize("offset", [1, 3, 4])
@pytest.mark.parametrize("dtype", DTYPES)
def test_misaligned_buffers(dtype, offset):
    for C in (64, 333):
        run_all(Case(3, 9, C, dtype, lengths=[9, 4, 6], seed=offset, offset=offset))


@pytest.mark.parametrize("B,T,C", [(1, 1, 512), (64, 1, 512), (64, 1, 1024), (1, 1, 1), (1, 700, 65), (7, 1, 2048),
                                   (300, 2, 8), (1000, 1, 3)])
def test_few_and_single_frames(B, T, C):
    for dtype in ("bf16", "f32"):
        run_all(Case(B, T, C, dtype, seed=B + T), p=0.25, alpha=1.0)


@pytest.mark.parametrize("dtype", DTYPES)
def test_conformer_batch(dtype):
    rng = np.random.default_rng(4)
    run_all(Case(16, 1500, 512, dtype, lengths=rng.integers(750, 1501, 16), seed=4))


def test_odd_batch_long_enough_for_every_warp():
    """More rows than the grid holds at once, rows off 16-byte boundaries: every residue of the row start."""
    rng = np.random.default_rng(5)
    for dtype, C in (("bf16", 131), ("f32", 33), ("f16", 1023)):
        run_all(Case(5, 2900 if C < 1000 else 900, C, dtype, lengths=rng.integers(0, 2901 if C < 1000 else 901, 5), seed=C))


@pytest.mark.parametrize("lengths", [[0, 0, 0], [-5, 99, 4], [6, 6, 6]])
def test_length_values(lengths):
    """No valid frame at all; lengths outside [0, T] are clamped."""
    run_all(Case(3, 6, 72, "bf16", lengths=lengths, seed=2))


@pytest.mark.parametrize("p", [0.0, 1e-6, 2.0 ** -16, 0.5, 0.9999, 1.0 - 1e-7, 1.0])
@pytest.mark.parametrize("C", [64, 37])
def test_drop_probabilities(p, C):
    c = Case(2, 40, C, "bf16", lengths=[40, 17], seed=8)
    run_drop(c, p, 1.0)
    run_drop(c, p, 0.5, residual=False)
    run_dal_fwd(c, p, 1.0)
    run_dal_bwd(c, p, 1.0)


@pytest.mark.parametrize("C", [96, 45, 2000])
def test_optional_operands(C):
    c = Case(2, 11, C, "f16", lengths=[11, 5], seed=3)
    run_ln_fwd(c, gamma=False)
    run_ln_fwd(c, beta=False, stats=False)
    run_ln_fwd(c, gamma=False, beta=False)
    run_ln_bwd(c, gamma=False)
    run_ln_bwd(c, dgamma=False)
    run_ln_bwd(c, dbeta=False)
    run_ln_bwd(c, dgamma=False, dbeta=False)
    run_dal_fwd(c, 0.2, 1.0, residual=False)
    run_dal_fwd(c, 0.2, 1.0, h=False, stats=False)
    run_dal_fwd(c, 0.0, 1.0, gamma=False, beta=False)
    run_dal_bwd(c, 0.2, 0.5, dh=False)
    run_dal_bwd(c, 0.2, 0.5, dres=False, gamma=False)
    run_dal_bwd(c, 0.0, 1.0, dgamma=False)


def test_large_mean_keeps_the_variance():
    """Rows with a mean of 1000 deviations: the variance comes from centred values."""
    c = Case(2, 9, 512, "f32", seed=6, shift=0.0)
    c.x = (c.x + np.float32(1000)).astype(np.float32)
    run_ln_fwd(c)


def test_nan_and_infinity_stay_in_their_rows():
    c = Case(2, 8, 256, "bf16", seed=7)
    x = c.x.copy()
    x[0, 3, 5], x[1, 2, 9] = np.nan, np.inf
    y = c.out()
    dw.dw_layernorm_fwd(c.act(x), dev(c.gamma), dev(c.beta), y.t, None, None, None, EPS)
    torch.cuda.synchronize()
    bad = np.isnan(y.numpy()).any(-1)
    want = np.zeros((2, 8), bool)
    want[0, 3] = want[1, 2] = True
    assert np.array_equal(bad, want)
    # a dropped NaN counts as zero
    keep = orc.kept(c.x.shape, c.seed, c.off, 0.5)
    dx = c.out()
    dw.dw_dropout_add_bwd(c.act(np.where(keep, c.dy, np.float32("nan"))), dx.t, c.rng, 0.5, 1.0, None)
    torch.cuda.synchronize()
    assert np.isfinite(dx.numpy()).all()


def test_empty_gradients_are_zeros():
    for B, T in ((0, 5), (3, 0)):
        e = torch.empty(B, T, 40, dtype=torch.bfloat16, device="cuda")
        m = torch.empty(B, T, device="cuda")
        dg, db = f32g(40), f32g(40)
        dw.dw_layernorm_bwd(e, e, None, m, m, e, dg.t, db.t, None, None)
        dw.dw_layernorm_fwd(e, None, None, e, m, m, None)
        dw.dw_dropout_add_fwd(e, None, e, None, 0.5, 1.0, None)
        torch.cuda.synchronize()
        dg.check_slack()
        assert (dg.numpy() == 0).all() and (db.numpy() == 0).all()


@pytest.mark.parametrize("C", [256, 101])
def test_packed_rows_equal_padded_rows(C):
    """B = 1, T = N with lengths at the last offset: the padded batch's valid rows, bit for bit."""
    lens = np.array([17, 0, 30, 5], np.int32)
    c = Case(4, 30, C, "bf16", lengths=lens, seed=1)
    x = c.act(c.x)
    y, mean, rstd = torch.empty_like(x), torch.empty(4, 30, device="cuda"), torch.empty(4, 30, device="cuda")
    dw.dw_layernorm_fwd(x, dev(c.gamma), dev(c.beta), y, mean, rstd, c.ln)
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    N = int(off[-1]) + 6
    xp = torch.full((1, N, C), float("nan"), dtype=torch.bfloat16, device="cuda")
    for b in range(4):
        xp[0, off[b]:off[b + 1]] = x[b, :lens[b]]
    yp, mp, rp = torch.empty_like(xp), torch.empty(1, N, device="cuda"), torch.empty(1, N, device="cuda")
    offsets = dev(off)
    dw.dw_layernorm_fwd(xp, dev(c.gamma), dev(c.beta), yp, mp, rp, offsets[-1:])
    torch.cuda.synchronize()
    for b in range(4):
        assert torch.equal(yp[0, off[b]:off[b + 1]], y[b, :lens[b]])
        assert torch.equal(mp[0, off[b]:off[b + 1]], mean[b, :lens[b]])
    assert (yp[0, off[-1]:] == 0).all() and (rp[0, off[-1]:] == 0).all()


@pytest.mark.parametrize("B,T,C,dtype", [(16, 700, 512, "bf16"), (3, 911, 77, "f32"), (2, 300, 2100, "f16")])
def test_gradients_are_reproducible(B, T, C, dtype):
    c = Case(B, T, C, dtype, seed=12)
    _, _, mt, rt = backward_inputs(c)
    x, dy = c.act(c.x), c.act(c.dy)
    outs = []
    for fill in (0, 255):
        dx, dg, db = torch.empty_like(x), torch.empty(C, device="cuda"), torch.empty(C, device="cuda")
        ws = torch.full((dw.dw_layernorm_bwd_workspace_size(B, T, C),), fill, dtype=torch.uint8, device="cuda")
        dw.dw_layernorm_bwd(x, dy, dev(c.gamma), mt, rt, dx, dg, db, None, ws)
        outs.append((dx, dg, db))
    torch.cuda.synchronize()
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_other_stream_and_explicit_stream():
    c = Case(4, 50, 512, "bf16", seed=13)
    want = torch.empty(4, 50, 512, dtype=torch.bfloat16, device="cuda")
    x, ga = c.act(c.x), dev(c.gamma)
    dw.dw_layernorm_fwd(x, ga, None, want, None, None, None)
    s = torch.cuda.Stream()
    got, got2 = torch.zeros_like(want), torch.zeros_like(want)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        dw.dw_layernorm_fwd(x, ga, None, got, None, None, None)
    dw.dw_layernorm_fwd(x, ga, None, got2, None, None, None, stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(got2, want)


def test_binding_refusals(cuda_device):
    x = torch.zeros(2, 3, 8, dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(x)
    rng = torch.zeros(2, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError):
        dw.dw_layernorm_fwd(x[0], None, None, y[0], None, None, None)          # not [B, T, C]
    with pytest.raises(ValueError):
        dw.dw_layernorm_fwd(x[:, :, ::2], None, None, y[:, :, :4].contiguous(), None, None, None)
    with pytest.raises(ValueError):
        dw.dw_layernorm_fwd(x, torch.ones(8), None, y, None, None, None)       # gamma on the host
    with pytest.raises(TypeError):
        dw.dw_layernorm_fwd(x, torch.ones(8, dtype=torch.float16, device="cuda"), None, y, None, None, None)
    with pytest.raises(TypeError):
        dw.dw_layernorm_fwd(x, None, None, y.float(), None, None, None)
    with pytest.raises(TypeError):
        dw.dw_dropout_add_fwd(x, None, y, rng.int(), 0.5, 1.0, None)
    with pytest.raises(ValueError):
        dw.dw_dropout_add_fwd(x, None, y, rng[:1], 0.5, 1.0, None)
    for bad in (lambda: dw.dw_dropout_add_fwd(x, None, y, None, 0.5, 1.0, None),
                lambda: dw.dw_dropout_add_fwd(x, None, x, rng, 0.5, 1.0, None),
                lambda: dw.dw_layernorm_fwd(x, None, None, None, None, None, None)):
        with pytest.raises(dw.DwError) as e:
            bad()
        assert e.value.status == dw.DW_ERR_INVALID_ARG
    torch.cuda.synchronize()
