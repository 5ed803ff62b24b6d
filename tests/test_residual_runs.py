"""Runs of the residual path as programs make them (GPU): a conformer conv module's chain forward and
backward with the depthwise conv, a captured training step whose mask changes between replays,
calls on two streams, rows past 32-bit offsets, and every row kernel with several rows per thread
group."""
import numpy as np
import pytest
import torch

import oracle
import speech_encoder_depthwise_b200 as dw
from gpuhelp import assert_bf16_close, assert_masked_zero, dev, max_abs, rms
from oracle import residual as orc
from residualpin import assert_within, layernorm_bwd_err, layernorm_fwd_err, param_err, store, sum_err
from synth import bf16_round
from test_parity_residual import Case, run_dal_bwd, run_dal_fwd, run_ln_bwd, run_ln_fwd

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    from speech_encoder_depthwise_b200 import build
    build.build()
    dw.lib()


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("C", [512, 519])
def test_conv_module_chain(C):
    """norm -> depthwise conv -> dropout, residual add, next norm; then back through all of it.  Queued
    without a host synchronization into buffers that held other values; each stage is checked
    against the oracle on the GPU's own input to it."""
    B, T, K, pl, p, alpha = 6, 500, 9, 4, 0.15, 0.5
    r = np.random.default_rng(21)
    lens = np.array([500, 0, 333, 1, 499, 250], np.int32)
    valid = np.arange(T)[None] < lens[:, None]
    nan = np.float32("nan")

    def act():
        return dev(np.where(valid[..., None], bf16_round(r.standard_normal((B, T, C)).astype(np.float32)), nan), BF)

    def fill(*shape, dt=BF):
        return torch.full(shape, 1000.0, dtype=dt, device="cuda")
    h0, dy1, dh1 = act(), act(), act()
    ga = [dev((1 + 0.1 * r.standard_normal(C)).astype(np.float32)) for _ in range(2)]
    be = [dev((0.1 * r.standard_normal(C)).astype(np.float32)) for _ in range(2)]
    w = dev((r.standard_normal((K, C)) / 3).astype(np.float32))
    bias = dev(r.standard_normal(C).astype(np.float32))
    ln = dev(lens)
    seed, off = 77, 5
    rng = torch.tensor([seed, off], dtype=torch.int64, device="cuda")
    y0, u, h1, y1, du, ds, dy0, dh0 = (fill(B, T, C) for _ in range(8))
    m0, r0, m1, r1 = (fill(B, T, dt=torch.float32) for _ in range(4))
    dg0, db0, dg1, db1, gb = (fill(C, dt=torch.float32) for _ in range(5))
    gw = fill(K, C, dt=torch.float32)
    ws = torch.empty(dw.dw_layernorm_bwd_workspace_size(B, T, C), dtype=torch.uint8, device="cuda")
    wsc = torch.empty(max(16, dw.dwconv1d_bwd_dw_workspace_size(B, T, C, K)), dtype=torch.uint8, device="cuda")

    dw.dw_layernorm_fwd(h0, ga[0], be[0], y0, m0, r0, ln)
    dw.dwconv1d_fwd(y0, w, bias, u, ln, pl)
    dw.dw_dropout_add_layernorm_fwd(u, h0, rng, p, alpha, ga[1], be[1], h1, y1, m1, r1, ln)
    dw.dw_dropout_add_layernorm_bwd(dy1, dh1, h1, ga[1], m1, r1, rng, p, alpha, du, ds, dg1, db1, ln, ws)
    dw.dwconv1d_bwd_dw(y0, du, gw, gb, ln, pl, wsc)
    dw.dwconv1d_bwd_dx(du, w, dy0, ln, pl)
    # the residual's gradient joins the first norm's: no dropout here, the same workspace again
    dw.dw_dropout_add_layernorm_bwd(dy0, ds, h0, ga[0], m0, r0, None, 0.0, 1.0, dh0, None, dg0, db0, ln, ws)
    torch.cuda.synchronize()

    g = [(ga[i].cpu().numpy().astype(np.float64), be[i].cpu().numpy().astype(np.float64)) for i in range(2)]
    vm = valid[..., None]
    h0n = np.where(vm, f64(h0), 0)
    ry, rm, rr = orc.layernorm_fwd(h0n, *g[0], lens, EPS)
    ey, em, er = layernorm_fwd_err(h0n, ry, rm, rr, *g[0], np.zeros(h0n.shape))
    assert_within("y0", f64(y0), ry, store("bf16", ry, ey))
    assert_within("mean0", f64(m0), rm, em)
    assert_within("rstd0", f64(r0), rr, er)
    wn, bn = f64(w), f64(bias)
    assert_bf16_close(f64(u), oracle.dwconv1d_fwd(f64(y0), wn, bn, lens, pl))
    un = np.where(vm, f64(u), 0)
    s, ry, rm, rr = orc.dropout_add_layernorm_fwd(un, h0n, seed, off, p, alpha, *g[1], lens, EPS)
    es = sum_err(s, orc.multiplier(p, alpha) * un)
    ey, em, er = layernorm_fwd_err(s, ry, rm, rr, *g[1], es)
    assert_within("h1", f64(h1), s, store("bf16", s, es))
    assert_within("y1", f64(y1), ry, store("bf16", ry, ey))
    dyn, dhn = np.where(vm, f64(dy1), 0), np.where(vm, f64(dh1), 0)
    rdu, rds, rg, rb = orc.dropout_add_layernorm_bwd(dyn, dhn, f64(h1), g[1][0], f64(m1), f64(r1), seed, off, p, alpha, lens)
    es = layernorm_bwd_err(f64(h1), dyn, g[1][0], f64(m1), f64(r1), dhn)
    assert_within("ds", f64(ds), rds, store("bf16", rds, es))
    assert_within("du", f64(du), rdu, store("bf16", rdu, (orc.multiplier(p, alpha) * es + 2.0 ** -23 * np.abs(rdu)) * (rdu != 0)))
    G = 296
    eg, eb = param_err(f64(h1), dyn, f64(m1), f64(r1), valid, B * T / 148, G)
    assert_within("dgamma1", f64(dg1), rg, eg + 1e-30)
    assert_within("dbeta1", f64(db1), rb, eb + 1e-30)
    rgw, rgb = oracle.dwconv1d_bwd_dw(f64(y0), f64(du), K, lens, pl)
    for a, b in ((gw, rgw), (gb, rgb)):
        assert max_abs(f64(a), b) <= 1e-5 * max(rms(b), 1e-6)
    assert_bf16_close(f64(dy0), oracle.dwconv1d_bwd_dx(f64(du), wn, lens, pl))
    rdh, _, rg, rb = orc.dropout_add_layernorm_bwd(f64(dy0), f64(ds), h0n, g[0][0], f64(m0), f64(r0), 0, 0, 0.0, 1.0, lens)
    es = layernorm_bwd_err(h0n, f64(dy0), g[0][0], f64(m0), f64(r0), f64(ds))
    assert_within("dh0", f64(dh0), rdh, store("bf16", rdh, es + 2.0 ** -24 * np.abs(rdh)))
    eg, eb = param_err(h0n, f64(dy0), f64(m0), f64(r0), valid, B * T / 148, G)
    assert_within("dgamma0", f64(dg0), rg, eg + 1e-30)
    assert_within("dbeta0", f64(db0), rb, eb + 1e-30)
    for t in (y0, u, h1, y1, du, ds, dy0, dh0):
        assert_masked_zero(f64(t), lens, T)


@pytest.mark.parametrize("C", [640, 1277])
def test_captured_step_draws_a_new_mask_per_replay(C):
    """A step captured before any other call of its size; the program advances rng on the device."""
    B, T, p = 3, 40, 0.3
    x, res, dy = (torch.randn(B, T, C, device="cuda").to(BF) for _ in range(3))
    ga, be = torch.rand(C, device="cuda") + 0.5, torch.randn(C, device="cuda")
    ln = torch.tensor([40, 11, 0], dtype=torch.int32, device="cuda")
    ws = torch.empty(dw.dw_layernorm_bwd_workspace_size(B, T, C), dtype=torch.uint8, device="cuda")

    def buffers():
        a = lambda: torch.zeros(B, T, C, dtype=BF, device="cuda")
        v = lambda *s: torch.zeros(*s, device="cuda")
        return dict(h=a(), y=a(), m=v(B, T), r=v(B, T), dx=a(), ds=a(), dg=v(C), db=v(C), z=a())

    def step(o, rng):
        dw.dw_dropout_add_layernorm_fwd(x, res, rng, p, 1.0, ga, be, o["h"], o["y"], o["m"], o["r"], ln)
        dw.dw_dropout_add_layernorm_bwd(dy, None, o["h"], ga, o["m"], o["r"], rng, p, 1.0, o["dx"], o["ds"], o["dg"],
                                        o["db"], ln, ws)
        dw.dw_dropout_add_fwd(o["dx"], res, o["z"], rng, p, 0.5, ln)
    rng = torch.tensor([9, 100], dtype=torch.int64, device="cuda")
    one = torch.tensor([0, 1], dtype=torch.int64, device="cuda")
    got = buffers()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(got, rng)
        rng += one
    masks = []
    for k in range(3):
        graph.replay()
        torch.cuda.synchronize()
        want = buffers()
        step(want, torch.tensor([9, 100 + k], dtype=torch.int64, device="cuda"))
        torch.cuda.synchronize()
        for name in want:
            assert torch.equal(got[name], want[name]), (k, name)
        masks.append(got["dx"].clone())
    assert not torch.equal(masks[0], masks[1]) and int(rng[1]) == 103


def test_two_streams_at_once():
    """Concurrent backward calls with a workspace each give the results of calls one at a time."""
    B, T, C = 8, 400, 520
    args, want = [], []
    for i in range(2):
        x, dy = (torch.randn(B, T, C, device="cuda").to(BF) for _ in range(2))
        m, r = x.float().mean(-1), torch.rsqrt(x.float().var(-1, unbiased=False) + EPS)
        args.append((x, dy, torch.rand(C, device="cuda"), m.contiguous(), r.contiguous()))

    def call(i, out, stream=None):
        dw.dw_layernorm_bwd(*args[i], *out[:3], None, out[3], stream=stream)

    def outs():
        return (torch.zeros(B, T, C, dtype=BF, device="cuda"), torch.zeros(C, device="cuda"), torch.zeros(C, device="cuda"),
                torch.empty(dw.dw_layernorm_bwd_workspace_size(B, T, C), dtype=torch.uint8, device="cuda"))
    for i in range(2):
        want.append(outs())
        call(i, want[i])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [outs() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for i in range(2):
            call(i, got[i], streams[i])
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for a, b in zip(g[:3], w[:3]):
            assert torch.equal(a, b)


def test_flat_indices_past_32_bits():
    """2.2e9 elements: a tile of rows repeated, so every repetition's norm and gradient must be the
    first one's; the mask at the far end against the oracle."""
    C, tile, reps = 1032, 4096, 513
    T = tile * reps
    xt, gt = torch.randn(tile, C, device="cuda").half(), torch.randn(tile, C, device="cuda").half()
    x = xt.repeat(reps, 1)[None]
    ga, be = torch.rand(C, device="cuda") + 0.5, torch.randn(C, device="cuda")
    y, m, r = torch.empty_like(x), torch.empty(1, T, device="cuda"), torch.empty(1, T, device="cuda")
    dw.dw_layernorm_fwd(x, ga, be, y, m, r, None)
    small = [torch.empty(1, tile, C, dtype=torch.float16, device="cuda"), torch.empty(1, tile, device="cuda"),
             torch.empty(1, tile, device="cuda")]
    dw.dw_layernorm_fwd(xt[None], ga, be, *small, None)
    torch.cuda.synchronize()
    assert bool((y.view(reps, tile, C) == small[0]).all()) and bool((m.view(reps, tile) == small[1]).all())
    # backward: dx repeats too; dbeta is reps times the tile's, up to float32 sums
    dy = gt.repeat(reps, 1)[None]
    dg, db = torch.empty(C, device="cuda"), torch.empty(C, device="cuda")
    ws = torch.empty(dw.dw_layernorm_bwd_workspace_size(1, T, C), dtype=torch.uint8, device="cuda")
    dw.dw_layernorm_bwd(x, dy, ga, m, r, y, dg, db, None, ws)
    dxt = torch.empty_like(small[0])
    dw.dw_layernorm_bwd(xt[None], gt[None], ga, small[1], small[2], dxt, torch.empty_like(dg), torch.empty_like(db), None, ws)
    torch.cuda.synchronize()
    assert bool((y.view(reps, tile, C) == dxt).all())
    ref, mag = gt.double().sum(0) * reps, gt.double().abs().sum(0) * reps
    # a chain of at most T / 148 / 8 rows, then the block's units and the partial rows: u times the magnitude each
    assert bool(((db.double() - ref).abs() <= (T / 1184 + 64) * 2.0 ** -24 * mag).all())
    # dropout: y = x where kept, 0 where not, at both sides of 2^31 and at the end
    rng = torch.tensor([3, 4], dtype=torch.int64, device="cuda")
    dw.dw_dropout_add_fwd(x, None, y, rng, 0.5, 0.5, None)
    torch.cuda.synchronize()
    flat, fx = y.view(-1), x.view(-1)
    for first in (0, 2 ** 31 - 4096, T * C - 8192):
        keep = orc.kept((8192,), 3, 4, 0.5, first=first)
        got, src = flat[first:first + 8192].cpu().numpy(), fx[first:first + 8192].cpu().numpy()
        assert np.array_equal(got, np.where(keep, src, np.float16(0)))
    # the same mask from the row kernel (p = 1/2, alpha = 1/2: the kept sum is x itself)
    h = dy
    dw.dw_dropout_add_layernorm_fwd(x, None, rng, 0.5, 0.5, ga, be, h, torch.empty_like(y), None, None, None)
    torch.cuda.synchronize()
    assert bool((h == y).all())


# one size per row kernel, forward and backward, without and with edges: octets, rows for more than one
# per thread group
SIZES = [(8, 15000), (16, 15000), (24, 9000), (32, 9000), (48, 6000), (64, 6000), (80, 6000), (96, 3000), (128, 3000),
         (192, 1700), (256, 1700), (383, 900), (512, 900), (768, 480), (1024, 480)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("extra", [0, 5])
@pytest.mark.parametrize("octets,rows", SIZES)
def test_every_row_kernel_with_several_rows_a_group(octets, rows, extra, dtype):
    c = Case(2, rows // 2, 8 * octets + extra, dtype, lengths=[rows // 2, rows // 3], seed=octets + extra)
    run_ln_fwd(c)
    run_ln_bwd(c)
    run_dal_fwd(c, 0.2, 0.5)
    run_dal_bwd(c, 0.2, 0.5)


@pytest.mark.parametrize("C", [64, 512, 2048, 8200])
def test_parameters_off_their_boundary(C):
    """gamma and beta that start 4 bytes after a 32-byte boundary, and no gamma at all."""
    c = Case(3, 50, C, "bf16", lengths=[50, 20, 0], seed=C)
    buf = torch.zeros(2, C + 1, device="cuda")
    buf[0, 1:] = dev(c.gamma)
    buf[1, 1:] = dev(c.beta)
    x, y, want = c.act(c.x), torch.empty(3, 50, C, dtype=BF, device="cuda"), torch.empty(3, 50, C, dtype=BF, device="cuda")
    m, r = torch.empty(3, 50, device="cuda"), torch.empty(3, 50, device="cuda")
    dw.dw_layernorm_fwd(x, buf[0, 1:], buf[1, 1:], y, m, r, c.ln)
    dw.dw_layernorm_fwd(x, dev(c.gamma), dev(c.beta), want, None, None, c.ln)
    torch.cuda.synchronize()
    ry, rm, rr = orc.layernorm_fwd(c.x, c.gamma, c.beta, c.lengths, EPS)
    s = c.x * c.valid[..., None].astype(np.float64)
    ey, _, _ = layernorm_fwd_err(s, ry, rm, rr, c.gamma, c.beta, np.zeros(s.shape))
    for t in (y, want):
        assert_within("y", f64(t), ry, store("bf16", ry, ey))
    run_ln_bwd(c, gamma=False)
    dx, dg, db = torch.empty_like(x), torch.empty(C, device="cuda"), torch.empty(C, device="cuda")
    dx2, dg2, db2 = torch.empty_like(x), torch.empty(C, device="cuda"), torch.empty(C, device="cuda")
    ws = torch.empty(dw.dw_layernorm_bwd_workspace_size(3, 50, C), dtype=torch.uint8, device="cuda")
    dy = c.act(c.dy)
    dw.dw_layernorm_bwd(x, dy, buf[0, 1:], m, r, dx, dg, db, c.ln, ws)
    dw.dw_layernorm_bwd(x, dy, dev(c.gamma), m, r, dx2, dg2, db2, c.ln, ws)
    torch.cuda.synchronize()
    mn, rn = f64(m), f64(r)
    rdx, rg, rb = orc.layernorm_bwd(c.x, c.dy, c.gamma, mn, rn, c.lengths)
    e = layernorm_bwd_err(c.x, c.dy, c.gamma, mn, rn, None)
    for t in (dx, dx2):
        assert_within("dx", f64(t), rdx, store("bf16", rdx, e))
    eg, eb = param_err(c.x, c.dy, mn, rn, c.valid, 2, 148)
    for t, q, b in ((dg, rg, eg), (dg2, rg, eg), (db, rb, eb), (db2, rb, eb)):
        assert_within("dparam", f64(t), q, b + 1e-30)


def test_more_rows_than_32_bit_row_kernels_take():
    """2^30 + 7 rows of two channels go through the general kernels."""
    T = 2 ** 30 + 7
    x = torch.zeros(1, T, 2, dtype=torch.float16, device="cuda")
    x[0, -1000:] = torch.randn(1000, 2, device="cuda").half()
    y, m = torch.empty_like(x), torch.empty(1, T, device="cuda")
    lengths = torch.tensor([T - 3], dtype=torch.int32, device="cuda")
    dw.dw_layernorm_fwd(x, None, None, y, m, None, lengths, 1e-3)
    torch.cuda.synchronize()
    xs = x[0, -1000:].double().cpu().numpy()[None]
    ry, rm, rr = orc.layernorm_fwd(xs, None, None, [997], 1e-3)
    ey, em, _ = layernorm_fwd_err(xs * (np.arange(1000) < 997)[None, :, None], ry, rm, rr, None, None, np.zeros(xs.shape))
    assert_within("y", f64(y[:, -1000:]), ry, store("f16", ry, ey))
    assert_within("mean", f64(m[:, -1000:]), rm, em)
    assert bool((y[0, :2 ** 20] == 0).all()) and bool((y[0, -3:] == 0).all())


@pytest.mark.parametrize("C", [64, 333])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_activations_at_different_alignments(C, dtype):
    """Inputs and outputs that lie differently past 16-byte boundaries take the general kernels."""
    c = Case(2, 21, C, dtype, lengths=[21, 8], seed=C)
    acts = c.act
    for i in range(2):
        c.act = lambda a: (setattr(c, "offset", 1 if i == 0 else 5), acts(a), setattr(c, "offset", 0))[1]
        c.offset = 0
        run_ln_fwd(c)
        run_ln_bwd(c)
        run_dal_fwd(c, 0.2, 0.5)
        run_dal_bwd(c, 0.2, 0.5)


@pytest.mark.parametrize("offset", range(8))
def test_every_phase_of_the_tensors(offset):
    """All tensors the same number of elements past a boundary: the row kernels with edges, several rows
    a thread group (with dropout, the general kernels)."""
    for dtype, C in (("f16", 256), ("f32", 130), ("bf16", 1021)):
        c = Case(2, 1500, C, dtype, lengths=[1500, 700], seed=offset, offset=offset)
        run_ln_fwd(c)
        run_ln_bwd(c)
        run_dal_fwd(c, 0.0, 0.5)
        run_dal_bwd(c, 0.0, 0.5)
    run_dal_bwd(Case(2, 30, 200, "bf16", lengths=[30, 7], seed=offset, offset=offset), 0.2, 0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("C,rows", [(8200, 700), (12288, 400), (25600, 310), (25608, 6), (51200, 6), (51208, 6)])
def test_rows_beyond_the_register_kernels(C, rows, dtype):
    """Rows in shared memory (forward to 51200 channels, backward to 25600) and past it."""
    c = Case(2, rows // 2, C, dtype, lengths=[rows // 2, rows // 3], seed=C)
    run_ln_fwd(c)
    run_ln_fwd(c, gamma=False)
    run_ln_bwd(c)
    run_dal_fwd(c, 0.2, 0.5)
    run_dal_fwd(c, 0.2, 0.5, residual=False, h=False)
    run_dal_bwd(c, 0.2, 0.5)
    run_dal_bwd(c, 0.0, 1.0, dh=False, gamma=False, dbeta=False)


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("rows,C", [(24, 512), (600, 512), (600, 519), (5000, 256), (300, 2048), (200, 8200), (40, 8201)])
def test_steps_that_hand_each_other_their_buffers(rows, C, dtype):
    """Thirty steps in one graph, each launch reading what the one before it has just written into
    memory that the step before also used (kernels start before their predecessors end): bit for
    bit the results of the same calls with a synchronization after each."""
    steps, z = 30, "cuda"
    torch.manual_seed(9)
    src = torch.randn(1, rows, C, device=z).to(dtype)
    ga, be = torch.randn(C, device=z), torch.randn(C, device=z)
    rng = torch.stack([torch.full((steps,), 3), torch.arange(steps)], 1).to(z)
    ws = torch.empty(dw.dw_layernorm_bwd_workspace_size(1, rows, C), dtype=torch.uint8, device=z)
    x, y = torch.empty_like(src), torch.empty_like(src)
    mean, rstd = torch.empty(1, rows, device=z), torch.empty(1, rows, device=z)
    dx = torch.empty(steps, 1, rows, C, dtype=dtype, device=z)
    dg, db = torch.empty(steps, C, device=z), torch.empty(steps, C, device=z)

    def run(after):
        for i in range(steps):
            dw.dw_dropout_add_fwd(src, None, x, rng[i], 0.25, 1.0, None)
            after()
            dw.dw_layernorm_fwd(x, ga, be, y, mean, rstd, None, EPS)
            after()
            dw.dw_layernorm_bwd(x, y, ga, mean, rstd, dx[i], dg[i], db[i], None, ws)
            after()
    run(torch.cuda.synchronize)
    want = [t.clone() for t in (dx, dg, db)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(lambda: None)
    for _ in range(5):
        for t in (dx, dg, db, x, y, mean, rstd):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for got, ref in zip((dx, dg, db), want):
            assert torch.equal(got, ref)
