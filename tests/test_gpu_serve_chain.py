"""Serving calls in a row with no other kernel between them, each over what the
one before has just written: every one may begin before its predecessor is over."""
import pytest
import torch

from dynamic_sparse_attention_minf_b200 import minf

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    minf.lib()


def cache(seed, rows, Hkv, d, page, e4m3):
    n = -(-rows // page)
    g = torch.Generator(device="cuda").manual_seed(seed)
    return minf.KVCache.empty(n, Hkv, page, d, e4m3), torch.randperm(n, generator=g, device="cuda").to(torch.int32)[None].contiguous()


def run(calls, graph):
    """The calls in order, eagerly or captured and replayed twice; their outputs."""
    if not graph:
        outs = [c() for c in calls]
    else:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=side):
            outs = [c() for c in calls]
        gr.replay()
        gr.replay()
    torch.cuda.synchronize()
    return [o for o in outs if o is not None]


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("rows", [3, 400, 5000])
def test_read_write_read(rows, e4m3, graph):
    """Read, written over, read again, several times on the same pages: each read gives what was written last."""
    Hkv, d = 3, 128
    c, pages = cache(rows, rows, Hkv, d, 32, e4m3)
    ws = minf.status_workspace()
    start, lens = torch.zeros(1, **I32), torch.full((1,), rows, **I32)
    g = torch.Generator(device="cuda").manual_seed(rows)
    # values that both element types hold exactly, of another power of two each time
    kv = [torch.randint(-8, 9, (2, 1, Hkv, rows, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(6)]
    for i, x in enumerate(kv):
        x[..., 0] = 448
        x *= 2.0 ** i
    k, v = ([torch.empty(1, Hkv, rows, d, dtype=torch.bfloat16, device="cuda") for _ in kv] for _ in "kv")
    calls = []
    for i, x in enumerate(kv):
        calls.append(lambda x=x: minf.minf_kv_write(x[0], x[1], c, pages, start, ws=ws))
        calls.append(lambda i=i: minf.minf_kv_read(c, pages, lens, rows, k=k[i], v=v[i], ws=ws))
    run(calls, graph)
    assert minf.minf_get_device_status(ws) == 0
    for i, x in enumerate(kv):
        assert torch.equal(k[i], x[0]) and torch.equal(v[i], x[1]), i


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("T,e4m3", [(1, True), (1, False), (8, True), (40, False), (40, True)])
def test_rope_write_attention_twice(T, e4m3, graph):
    """Steps of rotation, write and attention over the same positions and buffers, with other rows each time, give
    what each step gives alone."""
    Hq, Hkv, d, ctx = 8, 2, 128, 700
    H = Hq + 2 * Hkv
    c, pages = cache(T, ctx + T, Hkv, d, 64, e4m3)
    ws = minf.tree_attn_workspace(1, Hq, Hkv, T, d)
    g = torch.Generator(device="cuda").manual_seed(T)
    pre = torch.randn(2, 1, Hkv, ctx, d, generator=g, device="cuda").to(torch.bfloat16)
    minf.minf_kv_write(pre[0], pre[1], c, pages, torch.zeros(1, **I32), ws=ws)
    f = 500000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64, device="cuda") / d)
    pos = torch.arange(ctx, ctx + T, **I32)[None].contiguous()
    lens = torch.full((1,), ctx, **I32)
    q = torch.empty(1, Hq, T, d, dtype=torch.bfloat16, device="cuda")
    k, v = (torch.empty(1, Hkv, T, d, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    xs = [torch.randn(1, T, H * d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(5)]
    os = [torch.empty_like(q) for _ in xs]
    ls = [torch.empty(1, Hq, T, device="cuda") for _ in xs]

    def step(i):
        return [lambda: minf.minf_qkv_norm_rope(xs[i], Hq, Hkv, pos=pos, inv_freq=f, q=q, k=k, v=v) and None,
                lambda: minf.minf_kv_write(k, v, c, pages, lens, ws=ws),
                lambda: minf.minf_tree_attn(q, c, pages, lens, o=os[i], lse=ls[i], ws=ws) and None]

    alone = []
    for i in range(len(xs)):
        for call in step(i):
            call()
            torch.cuda.synchronize()
        alone.append((os[i].clone(), ls[i].clone()))
    run([call for i in range(len(xs)) for call in step(i)], graph)
    assert minf.minf_get_device_status(ws) == 0
    for i, (o, l) in enumerate(alone):
        assert torch.equal(os[i], o) and torch.equal(ls[i], l), i
