"""GPU parity of the residual path's less used modes, against the fp64 oracle with derived bounds: every
row kernel with several rows a thread group, without a mask and in fp16."""
import pytest

import speech_encoder_depthwise_b200 as dw
from test_parity_residual import Case, run_dal_bwd, run_dal_fwd, run_drop, run_ln_bwd, run_ln_fwd
from test_residual_runs import SIZES

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    from speech_encoder_depthwise_b200 import build
    build.build()
    dw.lib()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("extra", [0, 5])
@pytest.mark.parametrize("octets,rows", SIZES)
def test_every_row_kernel_without_a_mask(octets, rows, extra, dtype):
    """Residual add without dropout: a group's second and later rows reuse its stages and registers."""
    c = Case(2, rows // 2, 8 * octets + extra, dtype, lengths=[rows // 2, rows // 3], seed=octets + extra)
    run_dal_fwd(c, 0.0, 0.5)
    run_dal_bwd(c, 0.0, 0.5)


@pytest.mark.parametrize("extra", [0, 5])
@pytest.mark.parametrize("octets,rows", SIZES)
def test_every_row_kernel_in_fp16(octets, rows, extra):
    c = Case(2, rows // 2, 8 * octets + extra, "f16", lengths=[rows // 2, rows // 3], seed=octets + extra)
    run_ln_fwd(c)
    run_ln_bwd(c)
    run_drop(c, 0.2, 0.5)
    run_dal_fwd(c, 0.2, 0.5)
    run_dal_bwd(c, 0.2, 0.5)
