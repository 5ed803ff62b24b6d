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


@pytest.mark.parametrize("name", sorted(n for n in os.listdir(build.CSRC) if n.endswith((".cu", ".cuh"))))
def test_kernels_read_nothing_as_read_only(name):
    """Activations, parameters, lengths, generator state and partial rows: an earlier call may have written any of
    them (out_lengths, weight gradients, a finalize kernel's partial rows)."""
    assert re.findall(READ_ONLY, code(name)) == []
