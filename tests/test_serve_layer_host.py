"""The serving part of layer.py on the host: what it refuses, and where its calls
would run (no GPU; nothing is launched)."""
import contextlib
import types

import pytest
import torch

from dynamic_sparse_attention_minf_b200 import build as bld
from dynamic_sparse_attention_minf_b200 import layer, minf
from dynamic_sparse_attention_minf_b200 import workloads as wl

BF = dict(dtype=torch.bfloat16)


@pytest.fixture(scope="module")
def sp():
    bld.build()
    w = wl.small(Hq=4, Hkv=2, N=128, d=64, seed=1, patterns=[wl.PAT_A] * 4, n_sink=0, n_local=128)
    w.B = 2
    return layer.make_serve_plan(w, 160, page=16, device="cpu", max_tokens=4)


@pytest.mark.parametrize("kw", [
    dict(N=127), dict(N=256), dict(B=1), dict(B=3), dict(C=8 * 64 - 1), dict(C=4 * 64), dict(dtype=torch.float32),
    dict(o=torch.zeros(2, 4, 127, 64, **BF)), dict(o=torch.zeros(2, 4, 128, 64)), dict(o=torch.zeros(2, 4, 64, 128, **BF).transpose(2, 3)),
    dict(lse=torch.zeros(2, 4, 64)), dict(lse=torch.zeros(2, 4, 128, dtype=torch.float64))])
def test_prompt_of_other_sizes_is_refused(sp, kw):
    """A shorter batch of rows would be read behind its end by the layer's calls, and a smaller output written."""
    qkv = torch.zeros(kw.get("B", 2), kw.get("N", 128), kw.get("C", 8 * 64), dtype=kw.get("dtype", torch.bfloat16))
    with pytest.raises(minf.MinfError, match="serve_prompt"):
        layer.serve_prompt(sp, qkv, o=kw.get("o"), lse=kw.get("lse"))
