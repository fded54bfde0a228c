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


# -------------------------------------------- the plan's device, where it is not the current one
class _Now:
    """Stands in for torch.cuda's current device and stream, and for the calls; keeps what each call ran on."""

    def __init__(self, monkeypatch):
        self.now, self.calls = (0, "default"), []

        @contextlib.contextmanager
        def on(what):
            was, self.now = self.now, what
            yield
            self.now = was

        monkeypatch.setattr(torch.cuda, "device", lambda d: on((torch.device(d).index, "default")))
        monkeypatch.setattr(torch.cuda, "stream", lambda s: on(self.now if s is None else (s.device.index, s.name)))

        def call(name, result=None):
            # one with a `stream` argument of its own goes there, or to its tensors' device's current stream
            def f(*a, stream=None, **kw):
                self.calls.append((name, self.now if stream is None else (stream.device.index, stream.name)))
                return result
            return f
        t = torch.zeros(2, 2, 4, 64, **BF)
        monkeypatch.setattr(minf, "minf_qkv_norm_rope", call("rope", (t, t, t)))
        monkeypatch.setattr(minf, "minf_kv_write", call("write"))
        monkeypatch.setattr(minf, "minf_tree_attn", call("attn", (t, t)))
        monkeypatch.setattr(layer, "run_layer", call("layer"))


class _Dev1(torch.Tensor):
    """A host tensor that says it lies on the second GPU."""
    device = property(lambda self: torch.device("cuda", 1))


def _on_dev1(sp):
    p = types.SimpleNamespace(**vars(sp))
    p.lens = sp.lens.clone().as_subclass(_Dev1)
    return p


@pytest.mark.parametrize("stream", [None, "side"])
def test_calls_run_on_the_plans_device(sp, monkeypatch, stream):
    """The current device is 0, the plan lies on device 1: every call of a step, and run_layer's bare pointers above
    all, is made with device 1 current, on its default stream or on the given one."""
    now = _Now(monkeypatch)
    p = _on_dev1(sp)
    st = types.SimpleNamespace(device=torch.device("cuda", 1), name="side") if stream else None
    monkeypatch.setattr(torch, "arange", lambda *a, **kw: torch.tensor([0, 1, 2, 3], dtype=torch.int32))
    layer.serve_prompt(p, torch.zeros(2, 128, 8 * 64, **BF).as_subclass(_Dev1), stream=st)
    layer.serve_tokens(p, torch.zeros(2, 4, 8 * 64, **BF).as_subclass(_Dev1), stream=st)
    layer.keep_tokens(p, torch.zeros(2, 2, 4, 64, **BF), torch.zeros(2, 2, 4, 64, **BF), torch.ones(2, dtype=torch.int32),
                      rows=torch.zeros(2, 3, dtype=torch.int32), stream=st)
    assert {n for n, _ in now.calls} == {"rope", "write", "attn", "layer"}
    assert [c for c in now.calls[1:] if c[1] != (1, stream or "default")] == []
    assert now.calls[0][0] == "rope" and now.now == (0, "default")


def test_stream_of_another_device_is_refused(sp, monkeypatch):
    now = _Now(monkeypatch)
    p = _on_dev1(sp)
    st = types.SimpleNamespace(device=torch.device("cuda", 0), name="side")
    x = torch.zeros(2, 4, 8 * 64, **BF).as_subclass(_Dev1)
    for call in (lambda: layer.serve_tokens(p, x, stream=st), lambda: layer.keep_tokens(p, x, x, torch.ones(2), stream=st)):
        with pytest.raises(minf.MinfError, match="stream"):
            call()
    assert now.calls == []


# ------------------------------------------------------------------ what keep_tokens keeps
@pytest.mark.parametrize("with_rows", [False, True])
@pytest.mark.parametrize("count,n_draft,kept", [
    ([0, 4], None, [0, 4]), ([5, 2], None, [4, 2]), ([-1, 1 << 30], None, [0, 4]), ([-2147483648, 2147483647], None, [0, 4]),
    ([3, 3], [2, 4], [2, 3]), ([4, -1], [0, 0], [0, 0]), ([4, 4], [-2, 9], [0, 4])])
def test_kept_counts_are_bounded(sp, monkeypatch, with_rows, count, n_draft, kept):
    """The cached lengths move by no more than the step's tokens, and what is moved in the cache goes with them."""
    i32 = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    wrote = []
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(minf, "minf_kv_write", lambda *a, count=None, **kw: wrote.append(count.tolist()))
    p = types.SimpleNamespace(**vars(sp))
    p.lens = i32([130, 100])
    k = torch.zeros(2, 2, 4, 64, **BF)
    rows = torch.zeros(2, 4, dtype=torch.int32) if with_rows else None
    layer.keep_tokens(p, k, k, i32(count), rows=rows, n_draft=None if n_draft is None else i32(n_draft))
    assert p.lens.tolist() == [130 + kept[0], 100 + kept[1]] and p.lens.dtype == torch.int32
    assert wrote == ([kept] if with_rows else [])


def test_kept_tokens_stay_within_the_pages(sp, monkeypatch):
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    p = types.SimpleNamespace(**vars(sp))                        # 160 positions a sequence
    p.lens = torch.tensor([158, 160], dtype=torch.int32)
    for _ in range(3):
        layer.keep_tokens(p, None, None, torch.tensor([2, 1], dtype=torch.int32))
    assert p.lens.tolist() == [160, 160]
