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
