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


EARLY = [p for p in SOURCES if re.search("latent|pages", os.path.basename(p))]


@pytest.mark.parametrize("path", EARLY, ids=os.path.basename)
def test_no_read_only_loads_in_kernels_launched_early(path):
    """These kernels come onto the GPU before the previous one has ended, so what they read is not
    constant for their lifetime: no load may claim that it is, nor a pointer that nothing else writes."""
    code = re.sub(r"//[^\n]*", "", open(path).read())
    assert "pdl_wait" in code or path.endswith(".cuh")
    assert not re.search(r"__ldg\b|ld\.global\.nc|__restrict__|__builtin_nontemporal_load", code)
