"""Stream order of the residual path (GPU): calls that read what the call before them wrote, on the
kernels' less used ways (items that end inside an octet, odd channel counts, tensors off a boundary), in
buffers that the steps hand each other.  Each graph of calls gives, bit for bit, what the same
calls give with a synchronization after each."""
import pytest
import torch

import speech_encoder_depthwise_b200 as dw

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    from speech_encoder_depthwise_b200 import build
    build.build()
    dw.lib()


def off_boundary(shape, dtype, offset):
    """A tensor that starts ``offset`` elements past its allocation's boundary."""
    n = 1
    for s in shape:
        n *= s
    return torch.empty(n + offset, dtype=dtype, device="cuda")[offset:].view(shape)


def check_graph(run, outs, state):
    """``run(after)`` makes the calls; ``state``: (buffer, its value before the first call)."""
    def reset():
        for t, v in state:
            t.copy_(v)
        for t in outs:
            t.fill_(float("nan"))
    reset()
    run(torch.cuda.synchronize)
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(lambda: None)
    for _ in range(5):
        reset()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for got, ref in zip(outs, want):
            assert not torch.isnan(ref).any() and torch.equal(got, ref)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("lens,T,C,offset", [([37, 0, 20], 37, 131, 0), ([200, 77], 200, 1023, 0), ([4999], 5001, 33, 0),
                                             ([1, 0, 1, 1], 1, 519, 0), ([50, 9, 33], 50, 64, 1), ([300, 299], 300, 517, 3)])
def test_dropout_reads_what_the_call_before_wrote(lens, T, C, offset, dtype):
    """norm -> dropout + add -> dropout into the next step's residual stream, thirty steps."""
    B, steps = len(lens), 30
    torch.manual_seed(C)
    shape = (B, T, C)
    src = torch.randn(shape, device="cuda").to(dtype)
    ga, be = 0.5 * torch.rand(C, device="cuda"), 0.1 * torch.randn(C, device="cuda")
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    rng = torch.stack([torch.full((steps,), 5), torch.arange(steps)], 1).cuda()
    h, y = off_boundary(shape, dtype, offset), off_boundary(shape, dtype, offset)
    z = [off_boundary(shape, dtype, offset) for _ in range(steps)]

    def run(after):
        for i in range(steps):
            dw.dw_layernorm_fwd(h, ga, be, y, None, None, ln, EPS)
            after()
            dw.dw_dropout_add_fwd(y, h, z[i], rng[i], 0.25, 0.5, ln)
            after()
            dw.dw_dropout_add_bwd(z[i], h, rng[i], 0.125, 0.5, ln)
            after()
    check_graph(run, z, [(h, src)])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,C", [(40, 512), (40, 519), (600, 64), (9, 2048), (5, 8200), (5, 8201)])
def test_parameters_and_lengths_that_the_call_before_wrote(T, C, dtype):
    """gamma, beta, the generator's state and the lengths of a call are what the call before it (dgamma and dbeta, the
    out_lengths of a subsampler) or a copy between two calls wrote over other values."""
    B, steps, F = 3, 20, 8
    torch.manual_seed(C + T)
    x, dy = (torch.randn(B, T, C, device="cuda").to(dtype) for _ in range(2))
    mel = torch.randn(B, 4 * T, F, device="cuda")
    w = [torch.randn(s, device="cuda") for s in ((3, 3, 8), (8,), (3, 3, 8), (8,))]
    sub = torch.empty((B,) + dw.subsample_out_shape(4 * T, F) + (8,), device="cuda")
    assert sub.shape[1] == T
    frames = torch.randint(0, 4 * T + 1, (steps, B), dtype=torch.int32, device="cuda")
    frames[:, 0] = 4 * T
    rngs = torch.stack([torch.full((steps,), 7), torch.arange(steps)], 1).cuda()
    m, r = x.float().mean(-1), torch.rsqrt(x.float().var(-1, unbiased=False) + EPS)
    ln, rng = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda")
    dx, h = torch.empty_like(x), torch.empty_like(x)
    ga, be = torch.empty(C, device="cuda"), torch.empty(C, device="cuda")
    ws = torch.empty(dw.dw_layernorm_bwd_workspace_size(B, T, C), dtype=torch.uint8, device="cuda")
    y, z = (torch.empty(steps, B, T, C, dtype=dtype, device="cuda") for _ in range(2))
    gamma, beta = torch.rand(C, device="cuda"), torch.rand(C, device="cuda")

    def run(after):
        for i in range(steps):
            rng.copy_(rngs[i])
            dw.dw_dropout_add_layernorm_fwd(x, None, rng, 0.25, 1.0, ga, be, h, z[i], None, None, ln, EPS)
            after()
            dw.dw_subsample_fwd(mel, *w, sub, frames[i], ln, False)
            after()
            dw.dw_layernorm_bwd(h, dy, None, m, r, dx, ga, be, ln, ws)
            after()
            dw.dw_layernorm_fwd(x, ga, be, y[i], None, None, ln, EPS)
            after()
            dw.dw_subsample_fwd(mel, *w, sub, frames[steps - 1 - i], ln, False)
            after()
            dw.dw_dropout_add_fwd(y[i], x, h, rng, 0.5, 1.0, ln)
            after()
    check_graph(run, [y, z], [(ga, gamma), (be, beta), (ln, torch.full_like(ln, T)), (h, x), (dx, x)])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,C,K,offset", [(1, 512, 9, 0), (16, 512, 31, 0), (40, 519, 9, 0), (300, 64, 9, 0), (33, 130, 40, 1)])
def test_convs_read_what_the_norm_before_wrote(T, C, K, offset, dtype):
    """norm -> streaming conv -> conv -> its gradients, thirty steps through the same buffers, workspace and cache."""
    B, steps = 8, 30
    torch.manual_seed(C + K)
    shape = (B, T, C)
    src = torch.randn(steps, *shape, device="cuda").to(dtype)
    w, bias = torch.randn(K, C, device="cuda") / K, torch.randn(C, device="cuda")
    x, u, v, dx = (off_boundary(shape, dtype, offset) for _ in range(4))
    cache = off_boundary((B, K - 1, C), dtype, offset)
    m, r = torch.empty(B, T, device="cuda"), torch.empty(B, T, device="cuda")
    ln = torch.tensor([T, T // 2, T, 0, 1, T, T, T], dtype=torch.int32, device="cuda")
    ws = torch.empty(max(16, dw.dwconv1d_bwd_dw_workspace_size(B, T, C, K)), dtype=torch.uint8, device="cuda")
    gw, gb = torch.empty(steps, K, C, device="cuda"), torch.empty(steps, C, device="cuda")
    y = torch.empty(steps, *shape, dtype=dtype, device="cuda")

    def run(after):
        for i in range(steps):
            dw.dw_layernorm_fwd(src[i], None, None, x, m, r, ln, EPS)
            after()
            dw.dwconv1d_stream_fwd(x, w, bias, u, cache, ln)
            after()
            dw.dwconv1d_fwd(u, w, bias, v, ln, K // 2)
            after()
            dw.dwconv1d_bwd_dx(v, w, dx, ln, K // 2)
            after()
            dw.dwconv1d_bwd_dw(v, dx, gw[i], gb[i], ln, K // 2, ws)
            after()
            dw.dw_layernorm_fwd(dx, None, gb[i], y[i], None, None, ln, EPS)
            after()
    check_graph(run, [gw, gb, y], [(cache, torch.zeros_like(cache))])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("C,k,stride,offset", [(64, 3, 2, 0), (63, 3, 2, 0), (64, 5, 1, 0), (64, 3, 1, 1)])
def test_conv2d_and_subsampler_read_what_the_norm_before_wrote(C, k, stride, offset, dtype):
    """norm -> conv2d -> its gradients, and norm -> subsampler backward, twenty steps through the same buffers."""
    B, T, F, steps = 2, 40, 10, 20
    torch.manual_seed(C + k)
    st, pads = (stride, stride), (k // 2,) * 3
    To, Fo = dw.conv2d_out_shape(T, F, k, k, st, pads)
    src = torch.randn(steps, B, T, F * C, device="cuda").to(dtype)
    w, bias = torch.randn(k, k, C, device="cuda") / k, torch.randn(C, device="cuda")
    x, dx = (off_boundary((B, T, F, C), dtype, offset) for _ in range(2))
    v = off_boundary((B, To, Fo, C), dtype, offset)
    ln, ol = torch.tensor([T, 17], dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
    ws = torch.empty(max(16, dw.dwconv2d_bwd_dw_workspace_size(B, T, F, C, k, k, st, pads)), dtype=torch.uint8, device="cuda")
    gw, gb = torch.empty(steps, k, k, C, device="cuda"), torch.empty(steps, C, device="cuda")
    mel, w0, b0, w1 = (torch.randn(s, device="cuda") for s in ((B, 4 * T, 4 * F), (3, 3, C), (C,), (3, 3, C)))
    assert dw.subsample_out_shape(4 * T, 4 * F) == (T, F)
    wsb = torch.empty(dw.dw_subsample_bwd_workspace_size(B, 4 * T, 4 * F, C), dtype=torch.uint8, device="cuda")
    mln = torch.tensor([4 * T, 71], dtype=torch.int32, device="cuda")
    g = [[torch.empty_like(t) for t in (w0, b0, w1, b0)] for _ in range(steps)]

    def run(after):
        for i in range(steps):
            dw.dw_layernorm_fwd(src[i], None, None, x.view(B, T, F * C), None, None, ln, EPS)
            after()
            dw.dwconv2d_fwd(x, w, bias, v, ln, ol, st, pads)
            after()
            dw.dwconv2d_bwd_dx(v, w, dx, ln, st, pads)
            after()
            dw.dwconv2d_bwd_dw(dx, v, gw[i], gb[i], ln, st, pads, ws)
            after()
            dw.dw_subsample_bwd(mel, w0, b0, w1, x, mln, *g[i], False, wsb)
            after()
    check_graph(run, [gw, gb] + [t for s in g for t in s], [])


@pytest.mark.parametrize("C", [512, 136, 519, 8200])
@pytest.mark.parametrize("act,par", [(0, 0), (0, 1), (3, 0), (None, 0)])
def test_reproducible_at_equal_alignment(C, act, par):
    """The same values at other addresses with the same remainder modulo 32 bytes: every result bit for bit.
    (act: elements past a boundary, None for inputs and outputs that differ; par: gamma's.)"""
    B, T, dtype = 3, 700, torch.bfloat16
    torch.manual_seed(C)
    vx, vdy = (torch.randn(B, T, C, device="cuda").to(dtype) for _ in range(2))
    vga, ln = torch.rand(C, device="cuda") + 0.5, torch.tensor([700, 211, 0], dtype=torch.int32, device="cuda")
    m, r = vx.float().mean(-1), torch.rsqrt(vx.float().var(-1, unbiased=False) + EPS)
    got, kept = [], []
    for shift in (0, 16, 32):  # multiples of 32 bytes for both types
        i, o = (act, act) if act is not None else (0, 1)
        x, dy = (off_boundary((B, T, C), dtype, i + 2 * shift) for _ in range(2))
        dx, ga = off_boundary((B, T, C), dtype, o + 2 * shift), off_boundary((C,), torch.float32, par + shift)
        dg, db = (off_boundary((C,), torch.float32, shift) for _ in range(2))
        ws = torch.empty(dw.dw_layernorm_bwd_workspace_size(B, T, C), dtype=torch.uint8, device="cuda")
        for t, v in ((x, vx), (dy, vdy), (ga, vga)):
            t.copy_(v)
        dw.dw_layernorm_bwd(x, dy, ga, m, r, dx, dg, db, ln, ws)
        got.append((dx, dg, db))
        kept.append((x, dy, ga, ws))  # nothing is freed, so that no address comes back
    torch.cuda.synchronize()
    for other in got[1:]:
        for a, b in zip(got[0], other):
            assert torch.equal(a, b)
