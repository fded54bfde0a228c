"""What the serving kernels' sources must not contain (no GPU)."""
import os
import re

import pytest

from dynamic_sparse_attention_minf_b200 import build as bld

EARLY = ["rope.cu", "kv_cache.cu", "tree_attn.cu", "tree_attn.cuh", "tree_wide.cu", "serve_device.cuh"]


@pytest.mark.parametrize("name", EARLY)
def test_kernels_launched_early_use_no_read_only_loads(name):
    """A kernel that lives while its predecessor still writes may not read through ld.global.nc, nor promise the
    compiler that nobody writes (const __restrict__), which lets it do the same."""
    with open(os.path.join(bld.CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert not re.search(r"__ldg\b|\.nc\b|__restrict__|__ldlu\b", code)
