"""Which loads the kernels' sources use.  Kernels start while their predecessor in the stream still
runs (programmatic dependent launch), so what an earlier call writes is not read-only for as long
as they are resident: it must not be read by the read-only path, neither by name nor through a
``const ... *__restrict__`` parameter, which lets the compiler choose it.  A violation is a race that
shows only now and then, so the sources are looked at."""
import os
import re

import pytest

from speech_encoder_depthwise_b200 import build

READ_ONLY = r"__ldg\s*\(|\bld\.global[\w.:]*\.nc\b|const\s+[\w ]+\*\s*__restrict__"


def code(name):
    """A source without its comments."""
    with open(os.path.join(build.CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def function(text, name):
    """The body of the first function of that name."""
    at = text.index("{", text.index(name + "("))
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at:i + 1]


@pytest.mark.parametrize("name", ["dropout.cu", "dropout.cuh", "residual.cuh", "layernorm_fwd.cu", "layernorm_fwd.cuh",
                                  "layernorm_bwd.cu", "layernorm_bwd.cuh"])
def test_residual_path_reads_nothing_as_read_only(name):
    """Activations, parameters, lengths, generator state and partial rows."""
    assert re.findall(READ_ONLY, code(name)) == []


def test_lengths_are_not_read_as_read_only():
    """An earlier call may write them: dw_subsample_fwd and dwconv2d_fwd do (out_lengths)."""
    assert re.findall(READ_ONLY, function(code("dw_common.cuh"), "clamp_len")) == []
