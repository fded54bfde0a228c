"""Attention over the cache where keys weigh very differently and so do their
values: rows of one channel, of zeros and of tiny numbers, beside a long context
whose tiles all fall to one block (its running reference and sums see every one
of them).

Tolerances are those of test_gpu_serve.py (u = 2^-8; a score is off by e_s), and
2^-17 for the log-sum-exp: with values' powers of two down to 2^-80 its three
32-bit sums of numbers up to 128 round by 2^-18 each, in powers of two.
"""
import math

import pytest
import torch

from dynamic_sparse_attention_minf_b200 import minf

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
I32 = dict(dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    minf.lib()


def exact(q, k, v, ctx, scale):
    """Float64 form of a chain: q [Hq, T, d] over one KV head's k, v [ctx + T, d]: O, LSE, sum p|v|, p."""
    T = q.shape[1]
    j = torch.arange(ctx + T, device=q.device)
    s = (q.double() @ k.double().T * scale).masked_fill(j[None] > ctx + torch.arange(T, device=q.device)[:, None], -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[..., None])
    return p @ v.double(), lse, p @ v.double().abs(), p


def one_block(rows, d, e4m3, nats, where, edit, seed=0, L=8192, B=150):
    """B sequences that share one cached sequence of L context keys, of scores within a nat or two of each other
    except for the key at `where`, `nats` above; edit(v, where) makes the values.  More sequences than blocks, so
    that a block takes the tiles of a whole sequence in a row.  Returns what check() looks at."""
    G = 4
    T = rows // G
    g = torch.Generator(device="cuda").manual_seed(seed)
    scale = d ** -0.5
    k, v, q = (torch.randn(1, h, n, d, generator=g, device="cuda") for h, n in ((1, L + T), (1, L + T), (G, T)))
    k *= 0.5
    q[..., 0], k[..., 0] = 16.0, 0.0
    k[0, 0, where] = 0
    k[0, 0, where, 0] = nats / (16 * scale)
    v = 1 + 0.3 * v
    edit(v[0, 0], where)
    q, k, v = (t.to(torch.bfloat16) for t in (q, k, v))
    n = -(-(L + T) // 64)
    c = minf.KVCache.empty(n, 1, 64, d, e4m3)
    pages = torch.randperm(n, generator=g, device="cuda").to(torch.int32)[None].contiguous()
    ws = minf.tree_attn_workspace(B, G, 1, T, d)
    minf.minf_kv_write(k, v, c, pages, torch.zeros(1, **I32), ws=ws)
    kd, vd = minf.minf_kv_read(c, pages, torch.full((1,), L + T, **I32), L + T, ws=ws)
    o, lse = minf.minf_tree_attn(q.expand(B, -1, -1, -1).contiguous(), c, pages.expand(B, -1).contiguous(),
                                 torch.full((B,), L, **I32), ws=ws)
    assert minf.minf_get_device_status(ws) == 0
    exps = c.v_exp[pages[0].long()].flatten()[:L + T].double() - 127 if e4m3 else None
    return q[0], kd[0, 0], vd[0, 0], L, scale, o, lse, exps


def check(q, k, v, ctx, scale, o, lse, exps, floor=0.0):
    """`floor`: 8-bit weights, times their values' powers of two, may be off by this part of the row's largest."""
    O, L, A, p = exact(q, k, v, ctx, scale)
    k64, q64 = k.double(), q.double()
    es = scale * (2.0 ** -17 * q64.norm(dim=-1) * k64.norm(dim=-1).max()
                  + (2.0 ** -18 * q64.abs().amax(-1) * k64.abs().sum(-1).max() if exps is not None else 0.0))
    tol = U * O.abs() + (U + 2 * es[..., None]) * A + 2.0 ** -120
    if floor:
        live = (v != 0).any(-1)
        top = (p * torch.exp2(exps) * live).amax(-1, keepdim=True)
        tol = tol + floor * top * (v.double().abs() * torch.exp2(-exps)[:, None]).sum(0)
    err = (o.double() - O).abs()
    assert (err <= tol).all(), ((err / tol).max().item(), err.max().item())
    err = (lse.double() - L).abs()
    assert (err <= es + 2.0 ** -20 * (1 + L.abs()) + 2.0 ** -17).all(), err.max().item()


ROWS = [4, 32, 64, 256]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("nats", [8, 40])
def test_sums_of_tiny_values_outlive_a_move(rows, nats, e4m3):
    """A context of values near 1e-24, then, in a later tile, a key 8 nats above it with values near 200: the sums
    before it are most of the total, although weight times value moves by 2^90.  And one 40 nats above it with tiny
    values too: its weight overflows against the reference of the tiles before it."""
    def tiny(v, where):
        v *= 1e-24
        if nats == 8:
            v[where] *= 2e26
    check(*one_block(rows, 128, e4m3, nats, 6000, tiny))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("nats,where", [(8, 0), (10, 0), (12, 5000), (14, 0), (16, 8190)])
def test_zero_row_beside_far_scores(rows, nats, where, e4m3):
    """A key whose values are all zero (a sink, a padding row) far above the others, which still hold a good part
    of the sum: it adds nothing, and takes nothing from the others' bits."""
    def zero(v, where):
        v[where] = 0
    check(*one_block(rows, 128 if nats != 12 else 64, e4m3, nats, where, zero))


@pytest.mark.parametrize("rows", ROWS)
def test_zero_rows_among_large_ones(rows):
    """Rows of zeros and rows that share their stored exponent (largest value in (224, 448]), in every tile and in
    the last, part-filled one; only zeros; and a pool of zeros that was never written."""
    def mixed(v, where):
        v *= 250
        v[::5] = 0
        v[1::7, 1:] = 0                                          # zero but for one channel
    check(*one_block(rows, 128, True, 9, 1000, mixed, L=2077))
    check(*one_block(rows, 64, True, 9, 100, lambda v, where: v.zero_(), L=1000))
    c = minf.KVCache.empty(3, 1, 64, 128, True)
    q = torch.randn(1, 4, rows // 4, 128, device="cuda").to(torch.bfloat16)
    ws = minf.tree_attn_workspace(1, 4, 1, rows // 4, 128)
    o, lse = minf.minf_tree_attn(q, c, torch.arange(3, **I32)[None], torch.full((1,), 100, **I32), ws=ws)
    assert minf.minf_get_device_status(ws) == 0 and (o == 0).all()
    want = torch.log(101.0 + torch.arange(rows // 4, device="cuda"))
    assert ((lse - want).abs() <= 2.0 ** -16).all()              # 2^-17, and that log's own rounding


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("nats,where,size", [(8, 0, 3.0), (10, 5000, 3.0), (12, 0, 3.0), (12, 300, 300.0), (14, 0, 3.0),
                                             (16, 8190, 3.0), (16, 0, 300.0)])
def test_one_channel_row_beside_far_scores(rows, nats, where, size, e4m3):
    """A key far above the others whose values are zero but for one channel: the other channels are what the other
    keys give, with the bits that the header promises."""
    def channel(v, where):
        v[where] = 0
        v[where, 5] = size
    floor = (2.0 ** -29 if rows <= 64 else 2.0 ** -27) if e4m3 else 0.0
    check(*one_block(rows, 128 if nats != 14 else 64, e4m3, nats, where, channel), floor=floor)


def small_cache(e4m3, L, d=128, page=32, seed=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = -(-L // page)
    c = minf.KVCache.empty(n, 2, page, d, e4m3)
    pages = torch.randperm(n, generator=g, device="cuda").to(torch.int32)[None].contiguous()
    k, v = (torch.randn(1, 2, L, d, generator=g, device="cuda").to(torch.bfloat16) for _ in "kv")
    return c, pages, k, v, g


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T,Hq", [(3, 4), (10, 4), (20, 4), (40, 8)])
def test_non_finite_rows_reach_who_sees_them(T, Hq, e4m3):
    """A NaN key or value of the context makes every row of its KV head NaN (with 16-bit values, in its channel
    only); a NaN key of a drafted token makes the rows NaN that see it, and no other row changes."""
    ctx, d, G = 300, 128, Hq // 2
    c, pages, k, v, g = small_cache(e4m3, ctx + T)
    q = torch.randn(1, Hq, T, d, generator=g, device="cuda").to(torch.bfloat16)
    see = torch.rand(T, T, generator=g, device="cuda") < 0.5
    see[:, 1] = torch.arange(T, device="cuda") % 2 == 0           # who sees drafted token 1
    mask = (see.long() << torch.arange(T, device="cuda")).sum(-1)[None].contiguous()
    ws = minf.tree_attn_workspace(1, Hq, 2, T, d)
    zero, lens = torch.zeros(1, **I32), torch.full((1,), ctx, **I32)

    def attend(k, v):
        minf.minf_kv_write(k, v, c, pages, zero, ws=ws)
        r = minf.minf_tree_attn(q, c, pages, lens, tree_mask=mask, ws=ws)
        assert minf.minf_get_device_status(ws) == 0
        return r

    o, lse = attend(k, v)
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    bad = k.clone()
    bad[0, 0, 7, 3] = math.nan
    o1, l1 = attend(bad, v)
    assert torch.isnan(o1[0, :G]).all() and torch.isnan(l1[0, :G]).all()
    assert torch.equal(o1[0, G:], o[0, G:]) and torch.equal(l1[0, G:], lse[0, G:])
    bad = v.clone()
    bad[0, 1, 150, 9] = math.nan
    o1, l1 = attend(k, bad)
    nan = torch.isnan(o1[0, G:])
    assert nan.all() if e4m3 else (nan[..., 9].all() and nan.sum() == nan[..., 9].numel())
    assert torch.equal(o1[0, :G], o[0, :G]) and torch.equal(l1[0, :G], lse[0, :G])
    bad = k.clone()
    bad[0, 0, ctx + 1] = math.nan
    o1, l1 = attend(bad, v)
    sees = see[:, 1]
    assert torch.isnan(o1[0, :G, sees]).all() and torch.isnan(l1[0, :G, sees]).all()
    assert torch.equal(o1[0, :G, ~sees], o[0, :G, ~sees]) and torch.equal(l1[0, :G, ~sees], lse[0, :G, ~sees])
    assert torch.equal(o1[0, G:], o[0, G:])


def test_eager_calls_beside_a_replayed_graph():
    """The same cache, read by a replayed graph and by eager calls on another stream, each with a workspace of its
    own: both sides give what they give alone."""
    c, pages, k, v, g = small_cache(True, 3000)
    lens = torch.tensor([2990], **I32)
    minf.minf_kv_write(k, v, c, pages, torch.zeros(1, **I32))
    qs = [torch.randn(1, 8, T, 128, generator=g, device="cuda").to(torch.bfloat16) for T in (1, 6)]
    ws = [minf.tree_attn_workspace(1, 8, 2, 6, 128) for _ in qs]
    alone = [minf.minf_tree_attn(q, c, pages, lens, ws=w) for q, w in zip(qs, ws)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = minf.minf_tree_attn(qs[0], c, pages, lens, ws=ws[0])
    torch.cuda.synchronize()
    eager, replayed = [], []
    for _ in range(30):
        with torch.cuda.stream(side):
            graph.replay()
            replayed.append(tuple(t.clone() for t in got))
        eager.append(minf.minf_tree_attn(qs[1], c, pages, lens, ws=ws[1]))
    torch.cuda.synchronize()
    for outs, want, w in ((replayed, alone[0], ws[0]), (eager, alone[1], ws[1])):
        assert minf.minf_get_device_status(w) == 0
        for o, lse in outs:
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
