"""Which loads the kernels' sources use.  Kernels start while their predecessor in the stream still
runs (programmatic dependent launch), so what an earlier call writes is not read-only for as long
as they are resident: it must not be read by the read-only path, neither by name nor through a
``const ... *__restrict__`` parameter, which lets the compiler choose it.  A violation is a race that
shows only now and then, so the sources are looked at."""
import os
import re

import pytest

from speech_encoder_depthwise_b200 import build

RESTRICT = r"const\s+[\w ]+\*\s*__restrict__\s*(\w+)"


def code(name):
    """A source without its comments."""
    with open(os.path.join(build.CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


@pytest.mark.parametrize("name", ["dropout.cu"])
def test_no_activation_is_declared_read_only(name):
    params = re.findall(RESTRICT, code(name))
    assert not [p for p in params if p in ("x", "res")]
