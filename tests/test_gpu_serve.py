"""The serving operators on the GPU against their float64 forms: head norm and
rotation, the paged cache written and read back, attention of new tokens over
it, and a run of them together.

Tolerances count roundings (u = 2^-8 is half a bf16 step relative to the value):
 * rotation: one bf16 rounding of the result, and 2^-18 of the pair's size for
   the 32-bit sums, root, sine and products (a few roundings of 2^-24 each,
   d/2 of them in the sum of squares, which enters under a root);
 * the cache: exact;
 * attention: u |o| for the result, u sum p|v| for the weights held in 8 bits or
   more, and e_s sum p|v| for a score off by e_s, where e_s bounds the 32-bit
   products (2^-17 |q||k| scale) and, for 8-bit keys, a query held in two 4-bit
   parts per element, off by at most 2^-18 of the row's largest.
"""
import math

import numpy as np
import pytest
import torch

from dynamic_sparse_attention_minf_b200 import layer, minf
from dynamic_sparse_attention_minf_b200 import workloads as wl
from oracle import serve_oracle as so

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
BOUNDS = 6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    minf.lib()


def f64(t):
    return t.detach().double().cpu().numpy()


def bf(x):
    return torch.as_tensor(np.asarray(x)).to(torch.bfloat16).cuda()


def i32(x):
    return torch.as_tensor(np.asarray(x)).to(torch.int32).cuda().contiguous()


# ------------------------------------------------------------- norm and rotation
@pytest.mark.parametrize("B,N,Hq,Hkv,d,rot,inter,norm", [
    (1, 1, 32, 8, 128, 128, False, True),      # one token
    (3, 7, 6, 2, 128, 64, False, True),        # odd counts, half of each head turned
    (2, 33, 4, 2, 64, 64, True, False),
    (5, 130, 2, 1, 64, 32, True, True),
    (1, 700, 4, 4, 128, 16, False, False),     # several tokens per block
    (2, 601, 3, 3, 64, 48, False, True),
    (2, 5, 4, 2, 128, 0, False, True),         # norm only
    (2, 5, 4, 2, 128, 0, False, False),        # layout only
])
def test_norm_rope(B, N, Hq, Hkv, d, rot, inter, norm):
    g = torch.Generator().manual_seed(B * 1000 + N)
    H = Hq + 2 * Hkv
    # rows inside wider ones: a batch stride and a row stride of their own
    wide = torch.randn(B, N + 2, H * d + 24, generator=g).to(torch.bfloat16).cuda()
    x = wide[:, 1:N + 1, 8:8 + H * d]
    pos = i32(torch.randint(0, 1 << 20, (B, N), generator=g))
    f = (500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).cuda() if rot else None
    qw, kw = ((1 + 0.3 * torch.randn(d, generator=g)).to(torch.bfloat16).cuda() if norm else None for _ in "qk")
    q, k, v = minf.minf_qkv_norm_rope(x, Hq, Hkv, pos=pos, inv_freq=f, q_weight=qw, k_weight=kw, eps=1e-5,
                                      interleaved=inter)
    got = np.concatenate([f64(t) for t in (q, k, v)], axis=1)
    xn, fn = f64(x).reshape(B, N, H, d), None if f is None else f64(f)
    for b in range(B):
        for h in range(H):
            turned = h < Hq + Hkv
            w = (qw if h < Hq else kw) if turned else None
            ref = so.norm_rope(xn[b, :, h], f64(pos)[b], fn if turned else None, None if w is None else f64(w), 1e-5, inter)
            before = so.norm_rope(xn[b, :, h], f64(pos)[b], None, None if w is None else f64(w), 1e-5)
            if not turned or (w is None and f is None):
                assert np.array_equal(got[b, h], ref)
                continue
            size = np.abs(before).max(axis=1, keepdims=True) * 2
            assert (np.abs(got[b, h] - ref) <= U * np.abs(ref) + 2.0 ** -18 * size).all(), (b, h)
    # without the value heads, into given outputs
    q2, k2, none = minf.minf_qkv_norm_rope(x, Hq, Hkv, pos=pos, inv_freq=f, q_weight=qw, k_weight=kw, eps=1e-5,
                                           interleaved=inter, want_v=False, q=torch.zeros_like(q), k=torch.zeros_like(k))
    assert none is None and torch.equal(q, q2) and torch.equal(k, k2)


def test_norm_rope_default_positions_and_empty():
    x = torch.randn(2, 9, 3 * 64, device="cuda", dtype=torch.bfloat16)
    f = (10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)).cuda()
    pos = torch.arange(9, dtype=torch.int32, device="cuda").repeat(2, 1)
    for a, b in zip(minf.minf_qkv_norm_rope(x, 1, 1, inv_freq=f), minf.minf_qkv_norm_rope(x, 1, 1, pos=pos, inv_freq=f)):
        assert torch.equal(a, b)
    q, k, v = minf.minf_qkv_norm_rope(x[:, :0], 1, 1, inv_freq=f)
    assert q.shape == k.shape == v.shape == (2, 1, 0, 64)
    # a row of zeros and one with a NaN
    x[0, 0] = 0
    x[0, 1, 5] = float("nan")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    q, k, _ = minf.minf_qkv_norm_rope(x, 1, 1, inv_freq=f, q_weight=w, k_weight=w)
    assert (q[0, 0, 0] == 0).all() and torch.isnan(q[0, 0, 1]).all() and torch.isfinite(k[0]).all()


# -------------------------------------------------------------------------- cache
def random_cache(seed, B, rows, Hkv, page, d, e4m3, spare=2, fill=True):
    """(cache, pages [B, P] over a scattered pool); with `fill` every unused byte is a NaN."""
    g = torch.Generator().manual_seed(seed)
    P = max(1, -(-rows // page))
    n = B * P + spare
    c = minf.KVCache.empty(n, Hkv, page, d, e4m3)
    if fill:
        for t in (c.k, c.v):
            t.view(torch.uint8).fill_(0x7f)
            if not e4m3:
                t.fill_(float("nan"))
        for t in (c.k_exp, c.v_exp) if e4m3 else ():
            t.fill_(255)
    pages = i32(torch.randperm(n, generator=g)[:B * P].view(B, P))
    return c, pages


def edge_rows(B, H, M, d, seed):
    """Rows with zeros, tiny, huge, NaN and infinite entries among ordinary ones."""
    x = torch.randn(B, H, M, d, generator=torch.Generator().manual_seed(seed))
    x *= torch.exp(2 * torch.randn(B, H, M, 1, generator=torch.Generator().manual_seed(seed + 1)))
    special = [0.0, 1e-38, 3e38, 1e-25, 448.0, 1.75, 1.7578125, math.nan, math.inf]
    for i, s in enumerate(special):
        if i < M:
            x[0, 0, i] *= 0 if s == 0 else (1e-6 if i in (1, 3) else 1)
            x[0, 0, i, i % d] = s
            if s in (448.0, 1.75, 1.7578125):
                x[0, 0, i] = x[0, 0, i].clamp(-s, s)
    return x.to(torch.bfloat16)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("B,M,Hkv,d,page", [(1, 1, 1, 64, 16), (3, 45, 2, 128, 16), (2, 130, 3, 64, 32),
                                            (4, 9, 8, 128, 64), (1, 300, 2, 128, 128)])
def test_cache_write_and_read(B, M, Hkv, d, page, e4m3):
    c, pages = random_cache(M, B, 2 * M + 40, Hkv, page, d, e4m3, fill=False)
    k, v = edge_rows(B, Hkv, M, d, 3 * M), edge_rows(B, Hkv, M, d, 5 * M)
    rng = np.random.default_rng(M)
    start = rng.integers(0, M + 40, B)
    count = rng.integers(0, M + 1, B)
    count[0] = M
    # K as [B, M, H, d] (strided heads), V dense
    ks = k.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    ws = minf.status_workspace()
    before = [t.clone() for t in (c.k.view(torch.uint8), c.v.view(torch.uint8))]
    minf.minf_kv_write(ks, v.cuda(), c, pages, i32(start), count=i32(count), ws=ws)
    assert minf.minf_get_device_status(ws) == 0
    pg = pages.cpu().numpy()
    want = {}
    for name, src in (("k", k), ("v", v)):
        pool = f64(getattr(c, name).float())
        exps = getattr(c, name + "_exp").cpu().numpy() if e4m3 else None
        touched = np.zeros(pool.shape[0] * page, bool).reshape(-1, page)
        dense = np.zeros((B, Hkv, 2 * M + 40, d))
        for b in range(B):
            for i in range(count[b]):
                at = start[b] + i
                pid, row = pg[b, at // page], at % page
                touched[pid, row] = True
                for h in range(Hkv):
                    x = f64(src[b, h, i])
                    if e4m3:
                        q, e = so.quantise(x)
                        assert exps[pid, h, row] == e
                        assert np.array_equal(pool[pid, h, row], q, equal_nan=True), (name, b, h, i)
                        x = q * (math.nan if e == 255 else 2.0 ** (e - 127))
                    else:
                        assert np.array_equal(pool[pid, h, row], x, equal_nan=True)
                    dense[b, h, at] = x
        want[name] = dense
        raw = getattr(c, name).view(torch.uint8).cpu().numpy()
        old = before["kv".index(name)].cpu().numpy()
        assert np.array_equal(raw.transpose(0, 2, 1, 3)[~touched], old.transpose(0, 2, 1, 3)[~touched])
    lens = start + count
    lens[-1] = -3 if B > 1 else lens[-1]
    N = 2 * M + 37
    rk, rv = minf.minf_kv_read(c, pages, i32(lens), N, ws=ws)
    assert minf.minf_get_device_status(ws) == 0
    for got, name in ((f64(rk), "k"), (f64(rv), "v")):
        for b in range(B):
            n = min(max(lens[b], 0), N)
            assert np.array_equal(got[b, :, :n], want[name][b, :, :n], equal_nan=True)
            assert (got[b, :, n:] == 0).all()


def test_cache_write_by_rows_and_again():
    """Accepted tokens of a tree: rows gathered, some of them twice, over what the tree had written."""
    c, pages = random_cache(0, 2, 64, 2, 16, 128, True)
    k, v = (edge_rows(2, 2, 12, 128, s).cuda() for s in (1, 2))
    start = i32([30, 7])
    minf.minf_kv_write(k, v, c, pages, start)
    rows = i32([[0, 3, 3, 9], [11, 5, 0, 0]])
    minf.minf_kv_write(k, v, c, pages, start, count=i32([4, 2]), rows=rows)
    ref, pr = random_cache(0, 2, 64, 2, 16, 128, True)
    gk, gv = (torch.stack([t[b, :, rows[b].long()] for b in range(2)]) for t in (k, v))
    minf.minf_kv_write(k, v, ref, pr, start)
    minf.minf_kv_write(gk.contiguous(), gv.contiguous(), ref, pr, start, count=i32([4, 2]))
    for a, b in ((c.k, ref.k), (c.v, ref.v), (c.k_exp, ref.k_exp), (c.v_exp, ref.v_exp)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_cache_calls_report_bad_ids_and_go_on():
    c, pages = random_cache(0, 2, 64, 1, 16, 64, False, fill=False)
    k = torch.ones(2, 1, 4, 64, dtype=torch.bfloat16, device="cuda")
    ws = minf.status_workspace()
    bad = pages.clone()
    bad[0, 1] = c.n_pages
    for kw in (dict(pages=bad, start=i32([14, 0])),                    # rows 16, 17 in a page outside the pool
               dict(pages=pages, start=i32([62, 0])),                  # behind the table's end
               dict(pages=pages, start=i32([-1, 0])),
               dict(pages=pages, start=i32([0, 0]), count=i32([5, 4])),
               dict(pages=pages, start=i32([0, 0]), count=i32([-1, 4])),
               dict(pages=pages, start=i32([0, 0]), rows=i32([[0, 4], [0, 1]])),
               dict(pages=pages, start=i32([0, 0]), rows=i32([[-1, 2], [0, 1]]))):
        c.k.zero_()
        minf.minf_kv_write(k, k, c, kw["pages"], kw["start"], count=kw.get("count"), rows=kw.get("rows"), ws=ws)
        assert minf.minf_get_device_status(ws) == BOUNDS
        rk, _ = minf.minf_kv_read(c, pages, i32([0, 2]), 2, ws=ws)      # the other sequence was written
        assert minf.minf_get_device_status(ws) == 0
        assert (rk[1] == 1).all()
    minf.minf_kv_read(c, bad, i32([17, 0]), 64, ws=ws)
    assert minf.minf_get_device_status(ws) == BOUNDS
    minf.minf_kv_read(c, bad, i32([16, 64]), 64, ws=ws)                # entries behind the end are not read
    assert minf.minf_get_device_status(ws) == 0
    minf.minf_kv_read(c, pages, i32([65, 0]), 66, ws=ws)               # longer than the table
    assert minf.minf_get_device_status(ws) == BOUNDS


# ---------------------------------------------------------------------- attention
def random_tree(rng, T):
    """[T, T] ancestors-and-self matrix of a random tree."""
    see = np.zeros((T, T), bool)
    for t in range(T):
        if t:
            see[t] = see[rng.integers(0, t)] if rng.random() < 0.9 else False
        see[t, t] = True
    return see


def words(see):
    w = (see.astype(object) * np.array([1 << u for u in range(see.shape[1])], object)).sum(1)
    return [int(x) - (1 << 64) if int(x) >> 63 else int(x) for x in w]


def check_tree(q, kd, vd, ctx, nd, see, scale, o, lse, e4m3, o0=None, lse0=None):
    """Rows of o, lse against the float64 form on the cache's own values kd, vd [B, Hkv, L, d]."""
    B, Hq, T, d = q.shape
    g = Hq // kd.shape[1]
    for b in range(B):
        n, c = int(nd[b]), int(ctx[b])
        for h in range(Hq):
            k, v = kd[b, h // g, :c + n], vd[b, h // g, :c + n]
            O, L, A = so.tree_attention(q[b, h, :n], k, v, c, see[b][:n, :n], scale)
            if len(k):
                kn, k1 = np.sqrt((k * k).sum(1)).max(), np.abs(k).sum(1).max()
                qn, qm = np.sqrt((q[b, h, :n] ** 2).sum(1)), np.abs(q[b, h, :n]).max(1, initial=0.0)
                es = scale * (2.0 ** -17 * qn * kn + (2.0 ** -18 * qm * k1 if e4m3 else 0.0))
            else:
                es = np.zeros(n)
            tol = U * np.abs(O) + (U + 2 * es[:, None]) * A + 2.0 ** -120
            err = np.abs(o[b, h, :n] - O)
            assert (err <= tol).all(), (b, h, np.unravel_index((err - tol).argmax(), err.shape), (err / tol).max())
            fin = np.isfinite(L)
            assert np.array_equal(fin, np.isfinite(lse[b, h, :n]))
            assert (np.abs(lse[b, h, :n][fin] - L[fin]) <= es[fin] + 2.0 ** -20 * (1 + np.abs(L[fin]))).all()
        if o0 is not None:                                              # rows behind the last token
            assert np.array_equal(o[b, :, n:], o0[b, :, n:]) and np.array_equal(lse[b, :, n:], lse0[b, :, n:])


def run_tree(seed, B, Hq, Hkv, d, T, ctx, nd, page, e4m3, mask, scale=0.0, spike=None):
    rng = np.random.default_rng(seed)
    ctx, nd = np.asarray(ctx), np.asarray(nd)
    L = int((ctx + nd).max())
    c, pages = random_cache(seed, B, max(L, 1), Hkv, page, d, e4m3)     # whatever is not written is a NaN
    g = torch.Generator().manual_seed(seed)
    k = torch.randn(B, Hkv, max(L, 1), d, generator=g)
    v = torch.randn(B, Hkv, max(L, 1), d, generator=g) * torch.exp(torch.randn(B, Hkv, max(L, 1), 1, generator=g))
    q = torch.randn(B, Hq, T, d, generator=g)
    if spike is not None:
        spike(q, k, v)
    q, k, v = (t.to(torch.bfloat16).cuda() for t in (q, k, v))
    ws = minf.status_workspace()
    minf.minf_kv_write(k, v, c, pages, i32(np.zeros(B)), count=i32(ctx + nd), ws=ws)
    kd, vd = minf.minf_kv_read(c, pages, i32(ctx + nd), max(L, 1), ws=ws)
    assert minf.minf_get_device_status(ws) == 0
    if mask == "chain":
        see, tm = [np.tril(np.ones((T, T), bool))] * B, None
    else:
        see = [random_tree(rng, T) if mask == "tree" else rng.random((T, T)) < 0.3 for _ in range(B)]
        tm = torch.tensor([words(s) for s in see], dtype=torch.int64, device="cuda")
    ws = minf.tree_attn_workspace(B, Hq, Hkv, T, d)
    o = torch.full((B, Hq, T, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, Hq, T), 7.0, device="cuda")
    o0, lse0 = f64(o), f64(lse)
    minf.minf_tree_attn(q, c, pages, i32(ctx), n_draft=i32(nd), tree_mask=tm, o=o, lse=lse, scale=scale, ws=ws)
    assert minf.minf_get_device_status(ws) == 0
    check_tree(f64(q), f64(kd), f64(vd), ctx, nd, see, scale or 1 / math.sqrt(d), f64(o), f64(lse), e4m3, o0, lse0)
    return dict(q=q, c=c, pages=pages, ctx=i32(ctx), nd=i32(nd), tm=tm, o=o, lse=lse, ws=ws, scale=scale)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("B,Hq,Hkv,d,T,ctx,nd,page,mask", [
    (1, 4, 1, 128, 1, [0], [1], 16, "chain"),                            # nothing but the token itself
    (1, 1, 1, 64, 1, [1], [1], 64, "chain"),
    (2, 4, 2, 128, 1, [126, 127], [1, 1], 16, "chain"),                  # the token ends a tile / begins one
    (2, 8, 2, 64, 1, [128, 255], [1, 1], 128, "chain"),
    (3, 32, 8, 128, 1, [5, 700, 0], [1, 1, 1], 32, "chain"),
    (2, 6, 2, 128, 5, [300, 61], [5, 3], 64, "tree"),                    # padded batch, rows left as they were
    (4, 4, 2, 64, 13, [0, 17, 130, 1000], [13, 0, 1, 12], 32, "tree"),   # one sequence without new tokens
    (1, 8, 2, 128, 8, [120], [8], 16, "tree"),                           # 32 rows; the tree ends exactly a tile
    (1, 4, 2, 128, 24, [123], [24], 64, "random"),                       # rows that see nothing of the tree
    (2, 4, 2, 64, 20, [0, 0], [20, 7], 16, "random"),                    # no context: rows that see nothing at all
    (1, 4, 1, 128, 64, [385], [64], 128, "tree"),                        # 256 rows
    (2, 7, 1, 64, 40, [77, 200], [40, 33], 32, "tree"),                  # 280 rows of 7 heads
    (1, 3, 3, 128, 64, [64], [64], 64, "chain"),
    (1, 2, 2, 128, 33, [2500], [33], 16, "tree"),
    (6, 2, 1, 128, 2, [900, 3, 0, 4100, 64, 1], [2, 2, 2, 2, 1, 0], 16, "chain"),
])
def test_tree_attention(B, Hq, Hkv, d, T, ctx, nd, page, mask, e4m3):
    run_tree(sum(ctx) + T + Hq, B, Hq, Hkv, d, T, ctx, nd, page, e4m3, mask)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("where", [0, 200, 1500])
def test_tree_attention_late_maximum(where, e4m3):
    """A key that outweighs all before it by far, values of very different size: the running maximum moves."""
    def spike(q, k, v):
        k[:, :, where] = 6 * q[:, :k.shape[1], 0]
        v[:, :, :where] *= 1e-3
        v[:, :, where + 1:] *= 30.0
    run_tree(where, 1, 2, 2, 128, 3, [1700], [3], 64, e4m3, "chain", spike=spike)


@pytest.mark.parametrize("e4m3", [False, True])
def test_tree_attention_scale_and_flat_scores(e4m3):
    run_tree(5, 1, 4, 2, 64, 2, [3000], [2], 32, e4m3, "chain", scale=0.5)
    run_tree(6, 1, 4, 2, 64, 2, [3000], [2], 32, e4m3, "chain", scale=1e-4)     # every key counts the same

    def zero(q, k, v):
        q.zero_()
        v[:, :, 5:9] = 0
    run_tree(7, 1, 4, 2, 64, 2, [257], [2], 32, e4m3, "chain", spike=zero)


def test_tree_attention_bad_lengths_are_reported():
    r = run_tree(1, 2, 4, 2, 64, 2, [100, 20], [2, 2], 16, False, "chain")
    ws = r["ws"]
    for ctx, nd in (([100, -1], [2, 2]), ([100, 20], [2, 3]), ([100, 20], [2, -1]), ([100, 1 << 30], [2, 2]),
                    ([100, 2147483647], [2, 2])):
        o, lse = torch.full_like(r["o"], 5.0), torch.full_like(r["lse"], 5.0)
        minf.minf_tree_attn(r["q"], r["c"], r["pages"], i32(ctx), n_draft=i32(nd), o=o, lse=lse, ws=ws)
        assert minf.minf_get_device_status(ws) == BOUNDS
        assert torch.equal(o[0], r["o"][0]) and (o[1] == 5.0).all() and (lse[1] == 5.0).all()
    bad = r["pages"].clone()
    bad[1, 0] = -1
    minf.minf_tree_attn(r["q"], r["c"], bad, r["ctx"], ws=ws)
    assert minf.minf_get_device_status(ws) == BOUNDS
    o, lse = minf.minf_tree_attn(r["q"], r["c"], r["pages"], r["ctx"], ws=ws)
    assert minf.minf_get_device_status(ws) == 0 and torch.equal(o, r["o"]) and torch.equal(lse, r["lse"])


def test_tree_attention_same_bits_every_time_and_without_lse():
    r = run_tree(3, 3, 8, 2, 128, 4, [5000, 130, 2222], [4, 4, 2], 64, True, "tree")
    for _ in range(3):
        o, lse = torch.full_like(r["o"], 7.0), torch.full_like(r["lse"], 7.0)
        minf.minf_tree_attn(r["q"], r["c"], r["pages"], r["ctx"], n_draft=r["nd"], tree_mask=r["tm"], o=o, lse=lse, ws=r["ws"])
        assert torch.equal(o, r["o"]) and torch.equal(lse, r["lse"])
    o = torch.full_like(r["o"], 7.0)
    _, none = minf.minf_tree_attn(r["q"], r["c"], r["pages"], r["ctx"], n_draft=r["nd"], tree_mask=r["tm"], o=o,
                                  want_lse=False, ws=r["ws"])
    assert none is None and torch.equal(o, r["o"])


def test_non_finite_cache_rows():
    """A NaN row of the context reaches every row of its sequence and no other; an infinite score gives NaN."""
    for e4m3 in (False, True):
        r = run_tree(4, 2, 4, 2, 128, 2, [300, 300], [2, 2], 32, e4m3, "chain")
        k = torch.randn(2, 2, 1, 128, device="cuda").to(torch.bfloat16)
        k[0, 0, 0, 3] = float("inf")
        minf.minf_kv_write(k, torch.zeros_like(k), r["c"], r["pages"], i32([7, 301]), count=i32([1, 0]))
        o, lse = minf.minf_tree_attn(r["q"], r["c"], r["pages"], r["ctx"], ws=r["ws"])
        if e4m3:
            assert torch.isnan(o[0, :2]).all() and torch.isnan(lse[0, :2]).all()
        assert torch.isfinite(o[0, 2:]).all() and torch.equal(o[1], r["o"][1]) and torch.equal(lse[1], r["lse"][1])


# ------------------------------------------------- streams, graphs, calls together
def test_serving_step_in_a_graph_follows_its_lengths():
    """Norm and rotation, cache write and attention, captured once and replayed on a side stream while
    the positions, the inputs and the lengths move on; another call with its own workspace runs meanwhile."""
    B, Hq, Hkv, d, page = 2, 4, 2, 128, 16
    H = Hq + 2 * Hkv
    g = torch.Generator(device="cuda").manual_seed(0)
    c, pages = random_cache(0, B, 400, Hkv, page, d, True)
    f = (500000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64, device="cuda") / d))
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    x = torch.empty(B, 1, H * d, dtype=torch.bfloat16, device="cuda")
    ctx, pos = i32([0, 0]), i32([[0], [0]])
    q = torch.empty(B, Hq, 1, d, dtype=torch.bfloat16, device="cuda")
    k, v = (torch.empty(B, Hkv, 1, d, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    o, lse = torch.empty_like(q), torch.empty(B, Hq, 1, device="cuda")
    ws, ws2 = minf.tree_attn_workspace(B, Hq, Hkv, 1, d), minf.tree_attn_workspace(B, Hq, Hkv, 1, d)

    def step(ws=ws):
        minf.minf_qkv_norm_rope(x, Hq, Hkv, pos=pos, inv_freq=f, q_weight=w, k_weight=w, q=q, k=k, v=v)
        minf.minf_kv_write(k, v, c, pages, ctx, ws=ws)
        minf.minf_tree_attn(q, c, pages, ctx, o=o, lse=lse, ws=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        x.normal_(generator=g)
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    xs, got = [], []
    for i in range(150):
        xi = torch.randn(B, 1, H * d, device="cuda", generator=g).to(torch.bfloat16)
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.current_stream())
            x.copy_(xi)
            ctx.copy_(i32([i, i + 200]))
            pos.copy_(i32([[i], [i + 200]]))
            if i == 0:                                                  # a prefix for the second sequence
                pre = torch.randn(B, Hkv, 200, d, device="cuda", generator=g).to(torch.bfloat16)
                minf.minf_kv_write(pre, pre, c, pages, i32([0, 0]), count=i32([0, 200]), ws=ws)
            graph.replay()
            xs.append(xi)
            got.append((o.clone(), lse.clone()))
        if i % 50 == 7:                                                 # the same call, eagerly, at the same time
            minf.minf_tree_attn(q, c, pages, i32([1, 200]), ws=ws2)
    torch.cuda.synchronize()
    assert minf.minf_get_device_status(ws) == 0 and minf.minf_get_device_status(ws2) == 0
    kd, vd = (f64(t) for t in minf.minf_kv_read(c, pages, i32([150, 350]), 350))
    for i in (0, 1, 63, 149):
        qi = f64(minf.minf_qkv_norm_rope(xs[i], Hq, Hkv, pos=i32([[i], [i + 200]]), inv_freq=f, q_weight=w, k_weight=w)[0])
        check_tree(qi, kd, vd, [i, i + 200], [1, 1], [np.ones((1, 1), bool)] * 2, d ** -0.5, f64(got[i][0]), f64(got[i][1]),
                   True)


def test_given_stream_and_other_device():
    r = run_tree(9, 1, 4, 2, 64, 3, [500], [3], 64, False, "chain")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o, lse = minf.minf_tree_attn(r["q"], r["c"], r["pages"], r["ctx"], ws=r["ws"], stream=s)
    s.synchronize()
    assert torch.equal(o, r["o"]) and torch.equal(lse, r["lse"])
    if torch.cuda.device_count() > 1:
        with torch.cuda.device(1):
            o, lse = minf.minf_tree_attn(r["q"], r["c"], r["pages"], r["ctx"], ws=r["ws"])
        assert o.device == r["q"].device and torch.equal(o, r["o"])


@pytest.mark.parametrize("e4m3", [False, True])
def test_read_back_prefix_feeds_pre_fill(e4m3):
    """Cached rows read back dense give the dense pre-fill attention whose last row the cache attention gives too."""
    g = torch.Generator(device="cuda").manual_seed(2)
    N, Hq, Hkv, d = 512, 4, 2, 128
    c, pages = random_cache(1, 1, N, Hkv, 64, d, e4m3)
    q = torch.randn(1, Hq, N, d, generator=g, device="cuda").to(torch.bfloat16)
    k, v = (torch.randn(1, Hkv, N, d, generator=g, device="cuda").to(torch.bfloat16) for _ in "kv")
    minf.minf_kv_write(k, v, c, pages, i32([0]))
    kd, vd = minf.minf_kv_read(c, pages, i32([N]), N)
    if not e4m3:
        assert torch.equal(kd, k) and torch.equal(vd, v)
    o, lse = minf.minf_dense_attn(q, kd, vd)
    T = 8
    o2, lse2 = minf.minf_tree_attn(q[:, :, N - T:].contiguous(), c, pages, i32([N - T]))
    # both are within one rounding of the weights and one of the result of the same sums
    a = torch.nn.functional.scaled_dot_product_attention(q.double(), kd.double(), vd.double().abs(), is_causal=True,
                                                         enable_gqa=True)[:, :, N - T:]
    tol = 2 * (U * o2.double().abs() + (U + 2.0 ** -10) * a)
    assert ((o[:, :, N - T:].double() - o2.double()).abs() <= tol).all()
    assert ((lse[:, :, N - T:] - lse2).abs() <= 2.0 ** -10).all()


# ------------------------------------------------------------------ all together
@pytest.mark.parametrize("e4m3,stream", [(False, False), (True, True)])
def test_prompt_then_tree_then_tokens(e4m3, stream):
    """A layer served end to end: prompt rows through the pre-fill (window over all keys), a drafted tree, its
    accepted path kept, a chain, a generated token.  Every step against the float64 form on the cached values of
    the final sequence, whose positions carry the rotations of their final places."""
    B, Hq, Hkv, N, d, T = 2, 4, 2, 256, 128, 9
    w = wl.small(Hq=Hq, Hkv=Hkv, N=N, d=d, seed=3, patterns=[wl.PAT_A] * Hq, n_sink=0, n_local=N)
    w.B = B
    g = torch.Generator(device="cuda").manual_seed(5)
    C = (Hq + 2 * Hkv) * d
    f = 500000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64, device="cuda") / d)
    qw, kw = ((1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16) for _ in "qk")
    sp = layer.make_serve_plan(w, N + 40, page=16, e4m3=e4m3, inv_freq=f, q_weight=qw, k_weight=kw, max_tokens=T)
    perm = torch.randperm(sp.pages.numel(), generator=g, device="cuda").to(torch.int32)
    sp.pages.copy_(perm.view_as(sp.pages))
    rows = lambda n: torch.randn(B, n, C, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    st = torch.cuda.Stream() if stream else None
    sync = torch.cuda.synchronize

    x0 = rows(N)
    sync()
    o0 = layer.serve_prompt(sp, x0, stream=st)
    sync()
    # tree: 0 -> 1, 2; 1 -> 3, 4; 2 -> 5; 4 -> 6, 7; 5 -> 8
    parent = [-1, 0, 0, 1, 1, 2, 4, 4, 5]
    see, depth = np.zeros((T, T), bool), []
    for t, p in enumerate(parent):
        if p >= 0:
            see[t] = see[p]
        see[t, t] = True
        depth.append(0 if p < 0 else depth[p] + 1)
    x1 = rows(T)
    mask = torch.tensor([words(see)] * B, dtype=torch.int64, device="cuda")
    sync()
    o1, l1, k1, v1 = layer.serve_tokens(sp, x1, depth=i32(depth), tree_mask=mask, stream=st)
    path = [[0, 1, 4, 7], [0, 2, 5, 5]]           # sequence 1 keeps three
    kept = [4, 3]
    layer.keep_tokens(sp, k1, v1, i32(kept), rows=i32(path), stream=st)
    x2 = rows(2)
    sync()
    o2, l2, k2, v2 = layer.serve_tokens(sp, x2, stream=st)
    layer.keep_tokens(sp, k2, v2, i32([2, 2]), stream=st)
    x3 = rows(1)
    sync()
    o3, l3, k3, v3 = layer.serve_tokens(sp, x3, stream=st)
    layer.keep_tokens(sp, k3, v3, i32([1, 1]), stream=st)
    sync()
    assert layer.serve_status(sp) == 0
    assert sp.lens.tolist() == [N + 7, N + 6]
    kd, vd = layer.cached_prefix(sp, N + 8, stream=st)
    sync()
    assert (kd[0, :, N + 7:] == 0).all() and (vd[1, :, N + 6:] == 0).all()
    # the cache holds what rotating the final sequence's rows at their places gives
    for b in range(B):
        xb = torch.cat([x0[b], x1[b, path[b][:kept[b]]], x2[b], x3[b]])[None].contiguous()
        qb, kb, vb = minf.minf_qkv_norm_rope(xb, Hq, Hkv, inv_freq=f, q_weight=qw, k_weight=kw)
        n = xb.shape[1]
        if e4m3:
            ref = minf.KVCache.empty(-(-n // 16), Hkv, 16, d, True)
            table = torch.arange(-(-n // 16), dtype=torch.int32, device="cuda")[None]
            minf.minf_kv_write(kb, vb, ref, table, i32([0]))
            kb, vb = minf.minf_kv_read(ref, table, i32([n]), n)
        assert torch.equal(kd[b, :, :n], kb[0]) and torch.equal(vd[b, :, :n], vb[0])
        # prompt rows, on the unquantised keys and values
        qn = f64(minf.minf_qkv_norm_rope(x0[b:b + 1], Hq, Hkv, inv_freq=f, q_weight=qw, k_weight=kw)[0])
        kp, vp = (f64(t) for t in minf.minf_qkv_norm_rope(x0[b:b + 1], Hq, Hkv, inv_freq=f, q_weight=qw, k_weight=kw)[1:])
        for h in range(Hq):
            t0 = N - 3
            O, _, _ = so.tree_attention(qn[0, h, t0:], kp[0, h // 2], vp[0, h // 2], t0, np.tril(np.ones((3, 3), bool)),
                                        d ** -0.5)
            assert np.abs(f64(o0)[b, h, t0:] - O).max() <= 2e-2
        # steps 2 and 3, rows of the final sequence
        Kn, Vn, Q = f64(kd)[b:b + 1], f64(vd)[b:b + 1], f64(qb)
        at = N + kept[b]
        check_tree(Q[:, :, at:at + 2], Kn, Vn, [at], [2], [np.tril(np.ones((2, 2), bool))], d ** -0.5, f64(o2)[b:b + 1],
                   f64(l2)[b:b + 1], e4m3)
        check_tree(Q[:, :, at + 2:at + 3], Kn, Vn, [at + 2], [1], [np.ones((1, 1), bool)], d ** -0.5, f64(o3)[b:b + 1],
                   f64(l3)[b:b + 1], e4m3)
        # the accepted path's rows of the tree step are those of a chain over the final sequence
        for i in range(kept[b]):
            check_tree(Q[:, :, N + i:N + i + 1], Kn, Vn, [N + i], [1], [np.ones((1, 1), bool)], d ** -0.5,
                       f64(o1)[b:b + 1, :, path[b][i]:path[b][i] + 1], f64(l1)[b:b + 1, :, path[b][i]:path[b][i] + 1], e4m3)


def test_withheld_tiles_time_out_and_the_call_works_again():
    """While the status block's hook is set, the first block loads no tiles: its bounded waits run out, the call
    returns, and the status says so; afterwards the same workspace serves again."""
    r = run_tree(8, 1, 4, 2, 128, 3, [700], [3], 64, True, "chain")
    ws = r["ws"]
    ws[24:28].view(torch.int32).fill_(1)
    minf.minf_tree_attn(r["q"], r["c"], r["pages"], r["ctx"], ws=ws)
    assert minf.minf_get_device_status(ws) == 5
    ws[24:28].view(torch.int32).fill_(0)
    o, lse = minf.minf_tree_attn(r["q"], r["c"], r["pages"], r["ctx"], ws=ws)
    assert minf.minf_get_device_status(ws) == 0
    assert torch.equal(o, r["o"]) and torch.equal(lse, r["lse"])


@pytest.mark.parametrize("e4m3", [False, True])
def test_tree_attention_many_sequences(e4m3):
    """More sequences and heads than blocks (runs over several sequences), with empty ones among them, and a
    batch beyond one warp's look at the lengths."""
    rng = np.random.default_rng(4)
    B = 75
    ctx = rng.integers(0, 420, B)
    nd = rng.integers(0, 3, B)
    run_tree(11, B, 6, 3, 64, 2, ctx, nd, 16, e4m3, "chain")
    ctx = np.zeros(40, int)
    ctx[7] = 3000                                              # one long sequence among tiny ones
    run_tree(12, 40, 2, 1, 128, 2, ctx, np.full(40, 2), 32, e4m3, "chain")


@pytest.mark.parametrize("e4m3", [False, True])
def test_offsets_beyond_32_bits(e4m3):
    """Pages at the end of a pool of more than 4 GiB."""
    Hkv, page, d, L = 2, 64, 128, 150
    n = 140000 if not e4m3 else 270000                          # 4.6 / 4.4 GB of keys
    c = minf.KVCache.empty(n, Hkv, page, d, e4m3)
    pages = i32([[n - 1, n - 3, n - 2]])
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(1, Hkv, L, d, generator=g).to(torch.bfloat16).cuda() for _ in "kv")
    q = torch.randn(1, 4, 2, d, generator=g).to(torch.bfloat16).cuda()
    ws = minf.tree_attn_workspace(1, 4, Hkv, 2, d)
    minf.minf_kv_write(k, v, c, pages, i32([0]), ws=ws)
    kd, vd = minf.minf_kv_read(c, pages, i32([L]), L, ws=ws)
    if not e4m3:
        assert torch.equal(kd, k) and torch.equal(vd, v)
    o, lse = minf.minf_tree_attn(q, c, pages, i32([L - 2]), ws=ws)
    assert minf.minf_get_device_status(ws) == 0
    check_tree(f64(q), f64(kd), f64(vd), [L - 2], [2], [np.tril(np.ones((2, 2), bool))], d ** -0.5, f64(o), f64(lse), e4m3)


@pytest.mark.parametrize("T", [1, 30])
def test_infinite_scores(T):
    """A score of +infinity makes its rows NaN, wherever its key lies; -infinity weighs nothing."""
    for at in (3, 290):
        r = run_tree(21, 1, 4, 1, 64, T, [300], [T], 16, False, "chain")
        k, v = minf.minf_kv_read(r["c"], r["pages"], i32([300 + T]), 300 + T)
        k[0, 0, at] = 0
        k[0, 0, at, 0] = float("inf")
        q = r["q"].clone()
        q[..., 0] = q[..., 0].abs() + 1
        q[0, 0, :, 0] *= -1                                      # head 0: -infinity
        minf.minf_kv_write(k, v, r["c"], r["pages"], i32([0]))
        o, lse = minf.minf_tree_attn(q, r["c"], r["pages"], r["ctx"], ws=r["ws"])
        assert torch.isnan(o[0, 1:]).all() and torch.isnan(lse[0, 1:]).all()
        keep = [j for j in range(300 + T) if j != at]
        see = np.tril(np.ones((T, T), bool))
        O, L, A = so.tree_attention(f64(q)[0, 0], f64(k)[0, 0, keep], f64(v)[0, 0, keep], 299, see, 64 ** -0.5)
        assert (np.abs(f64(o)[0, 0] - O) <= U * np.abs(O) + (U + 2.0 ** -10) * A).all()
        assert np.abs(f64(lse)[0, 0] - L).max() <= 2.0 ** -10


def test_wide_rows_time_out_and_work_again():
    r = run_tree(31, 1, 8, 2, 128, 40, [700], [40], 64, True, "tree")
    ws = r["ws"]
    ws[24:28].view(torch.int32).fill_(1)
    minf.minf_tree_attn(r["q"], r["c"], r["pages"], r["ctx"], tree_mask=r["tm"], ws=ws)
    assert minf.minf_get_device_status(ws) == 5
    ws[24:28].view(torch.int32).fill_(0)
    o, lse = minf.minf_tree_attn(r["q"], r["c"], r["pages"], r["ctx"], tree_mask=r["tm"], ws=ws)
    assert minf.minf_get_device_status(ws) == 0
    assert torch.equal(o, r["o"]) and torch.equal(lse, r["lse"])


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv", [(64, 4, 2), (64, 2, 2), (20, 4, 1), (32, 4, 1)])
def test_wide_and_narrow_rows_late_maximum(T, Hq, Hkv, e4m3):
    """64 to 128 rows: a key beyond all others late in the context, values of very different size, and several
    blocks to a sequence; drafted keys fill the last tile."""
    def spike(q, k, v):
        k[:, :, 1400] = 5 * q[:, :Hkv, 3]
        v[:, :, :1400] *= 1e-3
    run_tree(T, 1, Hq, Hkv, 128, T, [128 * 14 - T], [T], 32, e4m3, "tree", spike=spike)
    run_tree(T + 1, 2, Hq, Hkv, 64, T, [1200, 0], [T, 5], 16, e4m3, "random")


def test_calls_on_two_streams_at_once():
    """The same cache read by two streams, each with its own workspace."""
    a = run_tree(41, 2, 8, 2, 128, 4, [3000, 1500], [4, 4], 64, True, "chain")
    ws = [a["ws"], minf.tree_attn_workspace(2, 8, 2, 4, 128)]
    ss = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    torch.cuda.synchronize()
    for i in range(20):
        for s in (0, 1):
            outs[s].append(minf.minf_tree_attn(a["q"], a["c"], a["pages"], a["ctx"], ws=ws[s], stream=ss[s]))
    torch.cuda.synchronize()
    for s in (0, 1):
        assert minf.minf_get_device_status(ws[s]) == 0
        for o, lse in outs[s]:
            assert torch.equal(o, a["o"]) and torch.equal(lse, a["lse"])


@pytest.mark.parametrize("e4m3", [False, True])
def test_many_row_groups(e4m3):
    """One KV head for all queries: 2048 rows in 16 groups, some of a shorter sequence's groups without rows."""
    run_tree(51, 2, 32, 1, 64, 64, [500, 3], [64, 9], 64, e4m3, "tree")
    run_tree(52, 1, 12, 1, 128, 64, [300], [33], 16, e4m3, "chain")


def test_head_counts_and_single_rows():
    for Hq, Hkv, T in ((5, 5, 1), (10, 2, 3), (16, 1, 1), (17, 1, 1), (33, 1, 2), (64, 1, 1), (65, 1, 1), (128, 1, 1)):
        run_tree(Hq, 1, Hq, Hkv, 64, T, [190], [T], 32, Hq % 2 == 0, "chain")


@pytest.mark.parametrize("T,e4m3", [(1, True), (40, False)])
def test_attention_follows_what_comes_before_it(T, e4m3):
    """The attention may begin before its predecessor in the stream is over, and must not read early: behind a
    kernel, a copy and a fill that change its inputs, in a row and captured into a graph."""
    a = run_tree(61, 1, 8, 2, 128, T, [2100], [T], 64, e4m3, "chain")
    b = run_tree(62, 1, 8, 2, 128, T, [900], [T], 64, e4m3, "chain")
    n = max(a["pages"].shape[1], b["pages"].shape[1])
    wide = lambda r: torch.cat([r["pages"], r["pages"][:, :1].expand(1, n - r["pages"].shape[1])], 1).contiguous()  # noqa: E731
    q, ctx, pages = a["q"].clone(), a["ctx"].clone(), wide(a)
    o, lse = torch.empty_like(a["o"]), torch.empty_like(a["lse"])
    pa, pb = wide(a), wide(b)
    big = torch.empty(64 << 20, device="cuda")
    flat = minf.KVCache.empty(a["c"].n_pages + b["c"].n_pages, 2, 64, 128, e4m3)   # both caches' pages in one pool
    for name in ("k", "v") + (("k_exp", "v_exp") if e4m3 else ()):
        t = getattr(flat, name)
        both = torch.cat([getattr(r["c"], name).view(torch.uint8).flatten() for r in (a, b)])
        t.view(torch.uint8).copy_(both.view(t.view(torch.uint8).shape))
    pb = pb + a["c"].n_pages
    ws = a["ws"]

    def step(r, p, slow):
        if slow:
            big.normal_()                                        # a long kernel before the changes
        q.copy_(r["q"])
        pages.copy_(p)
        ctx.fill_(0)
        ctx.add_(int(r["ctx"][0]) if not torch.cuda.is_current_stream_capturing() else r["len"])
        minf.minf_tree_attn(q, flat, pages, ctx, o=o, lse=lse, ws=ws)

    a["len"], b["len"] = 2100, 900
    for i in range(6):
        r, p = ((a, pa), (b, pb))[i % 2]
        step(r, p, i % 3 == 0)
        assert torch.equal(o, r["o"]) and torch.equal(lse, r["lse"])
    # calls in a row, each over the other's lengths, without a look between them
    got = []
    for i in range(8):
        r, p = ((a, pa), (b, pb))[i % 2]
        ctx.copy_(r["ctx"])
        pages.copy_(p)
        got.append(minf.minf_tree_attn(r["q"], flat, pages, ctx, ws=ws))
    for i, (oi, li) in enumerate(got):
        r = (a, b)[i % 2]
        assert torch.equal(oi, r["o"]) and torch.equal(li, r["lse"])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    outs = []
    with torch.cuda.graph(graph):
        for r, p in ((a, pa), (b, pb), (a, pa)):
            step(r, p, False)
            outs.append((o.clone(), lse.clone()))
        lse.zero_()
        minf.minf_tree_attn(q, flat, pages, ctx, o=o, lse=lse, ws=ws)
    for _ in range(3):
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for r, (oi, li) in zip((a, b, a), outs):
            assert torch.equal(oi, r["o"]) and torch.equal(li, r["lse"])
        assert torch.equal(o, a["o"]) and torch.equal(lse, a["lse"])
    assert minf.minf_get_device_status(ws) == 0


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("B,Hkv,T,longest,d", [(20, 8, 5, 4241, 128), (24, 8, 8, 2600, 128), (32, 8, 1, 939, 128),
                                               (16, 8, 16, 700, 128), (20, 4, 5, 4241, 64), (6, 4, 40, 1500, 128)])
def test_value_tiles_that_come_late(B, Hkv, T, longest, d, e4m3):
    """Batches of many last tiles (part keys, part rows to be cleared) whose values are still on their way, some of
    them from memory, when their scores are done: right, and the same bits every time."""
    rng = np.random.default_rng(longest)
    ctx = np.full(B, longest)
    ctx[::3] = rng.integers(1, longest, len(ctx[::3]))
    r = run_tree(71, B, 4 * Hkv, Hkv, d, T, ctx, np.full(B, T), 64, e4m3, "tree")
    fill = torch.empty(64 << 20, device="cuda")
    for i in range(24):
        if i % 2:
            fill.zero_()                                         # 256 MB: the cache is read from memory again
        o, lse = minf.minf_tree_attn(r["q"], r["c"], r["pages"], r["ctx"], tree_mask=r["tm"], ws=r["ws"])
        assert torch.equal(o, r["o"]) and torch.equal(lse, r["lse"]), i
    assert minf.minf_get_device_status(r["ws"]) == 0
