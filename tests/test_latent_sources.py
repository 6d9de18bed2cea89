"""What the sources of the latent-attention and page kernels must not hold, on the CPU."""
import glob
import os
import re

import pytest

from linear_attention_serving_02_gb300 import build

SOURCES = sorted(glob.glob(os.path.join(build.CSRC, "*.cu")) + glob.glob(os.path.join(build.CSRC, "*.cuh")))


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_no_multicast(path):
    """The library runs on every rank of a sharded program: a block fetches its tiles for itself."""
    assert not re.search(r"multicast\s*::\s*cluster", open(path).read())
