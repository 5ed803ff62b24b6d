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
