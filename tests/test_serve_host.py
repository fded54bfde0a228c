"""The serving entry points on the host: the oracle's own pins, and every
refusal of the C ABI and of the binding, before anything is launched (no GPU)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from dynamic_sparse_attention_minf_b200 import build as bld
from dynamic_sparse_attention_minf_b200 import minf
from oracle import serve_oracle as so


@pytest.fixture(scope="module")
def L():
    bld.build()
    return minf.lib()


# ------------------------------------------------------------------ oracle pins
def test_e4m3_round_is_nearest_even_over_all_bytes():
    vals = np.array([so.e4m3_value(b) for b in range(256)])
    fin = np.unique(vals[np.isfinite(vals)])
    assert fin.max() == 448.0 and np.array_equal(so.e4m3_round(fin), fin)
    mid = (fin[1:] + fin[:-1]) / 2
    got = so.e4m3_round(mid)
    torch_got = torch.from_numpy(mid).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(got, torch_got)
    x = np.random.default_rng(0).uniform(-448, 448, 4000)
    assert np.array_equal(so.e4m3_round(x), fin[np.abs(fin[None] - x[:, None]).argmin(1)])


def test_row_exponent():
    assert so.row_exponent([0.0, -448.0]) == 0
    assert so.row_exponent([448.5]) == 1
    assert so.row_exponent([0.0, 0.0]) == 0
    assert so.row_exponent([1e-38]) == -80
    assert so.row_exponent([1.0, math.inf]) is None and so.quantise([math.nan, 1.0])[1] == 255
    assert so.quantise([3.0, 448.0 * 8])[1] == 130


def test_rope_oracle_against_complex_numbers():
    rng = np.random.default_rng(1)
    x, pos, f = rng.standard_normal((5, 8)), np.array([0, 3, 7, 100, 12345]), np.array([1.0, 0.01])
    got = so.norm_rope(x, pos, f)
    z = (x[:, :2] + 1j * x[:, 2:4]) * np.exp(1j * pos[:, None] * f)
    assert np.allclose(got[:, :2], z.real) and np.allclose(got[:, 2:4], z.imag) and np.array_equal(got[:, 4:], x[:, 4:])
    z = (x[:, 0:4:2] + 1j * x[:, 1:4:2]) * np.exp(1j * pos[:, None] * f)
    got = so.norm_rope(x, pos, f, interleaved=True)
    assert np.allclose(got[:, 0:4:2], z.real) and np.allclose(got[:, 1:4:2], z.imag)
    n = so.norm_rope(x, pos, weight=np.full(8, 2.0), eps=0.0)
    assert np.allclose((n * n).mean(1), 4.0)


def test_tree_oracle_against_torch_attention():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((3, 4)), rng.standard_normal((8, 4)), rng.standard_normal((8, 4))
    see = np.tril(np.ones((3, 3), bool))
    o, lse, _ = so.tree_attention(q, k, v, 5, see, 0.5)
    mask = torch.cat([torch.ones(3, 5, dtype=torch.bool), torch.from_numpy(see)], 1)
    t = [torch.from_numpy(x)[None, None] for x in (q, k, v)]
    ref = torch.nn.functional.scaled_dot_product_attention(*t, attn_mask=mask, scale=0.5)[0, 0].numpy()
    assert np.allclose(o, ref)
    o, lse, _ = so.tree_attention(q, k[:3], v[:3], 0, np.zeros((3, 3), bool), 0.5)
    assert (o == 0).all() and np.isneginf(lse).all()


# --------------------------------------------------------------- C ABI refusals
FAKE = 1 << 20


def _cache(**kw):
    f = dict(k=FAKE, v=FAKE, k_exp=FAKE, v_exp=FAKE, n_pages=4, Hkv=2, page=16, d=128, type=1)
    f.update(kw)
    return ctypes.byref(minf._KVCacheC(*(f[n] for n, _ in minf._KVCacheC._fields_)))


BAD_CACHE = [(dict(k=None), 1), (dict(v=None), 1), (dict(k=FAKE + 8), 1), (dict(k_exp=None), 1), (dict(v_exp=FAKE + 4), 1),
             (dict(n_pages=0), 1), (dict(Hkv=0), 1), (dict(page=8), 2), (dict(page=48), 2), (dict(page=256), 2),
             (dict(d=96), 2), (dict(type=2), 2), (dict(n_pages=1 << 27), 2)]


def _rope(L, **kw):
    a = dict(X=FAKE, B=1, N=4, Hq=4, Hkv=2, d=128, sb=0, sn=1024, pos=FAKE, f=FAKE, rot=128, inter=0, qw=None, kw=None,
             eps=1e-6, Q=FAKE, K=FAKE, V=FAKE)
    a.update(kw)
    return L.minf_qkv_norm_rope(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(X=None), 1), (dict(Q=None), 1), (dict(K=None), 1), (dict(B=0), 1), (dict(N=-1), 1), (dict(Hq=3), 1),
    (dict(Hkv=0), 1), (dict(d=96), 2), (dict(sn=1023), 1), (dict(sn=1016), 1), (dict(sn=1025), 1), (dict(sb=4), 1),
    (dict(sb=-8), 1), (dict(rot=0), 1), (dict(rot=144), 1), (dict(rot=24), 2), (dict(X=FAKE + 2), 1), (dict(Q=FAKE + 8), 1),
    (dict(V=FAKE + 8), 1), (dict(qw=FAKE + 2), 1), (dict(f=FAKE + 4), 1), (dict(eps=-1.0), 1), (dict(eps=math.nan), 1),
    (dict(N=1 << 30), 2), (dict(N=0, X=None, Q=None, K=None, V=None), 0)])
def test_norm_rope_refusals(L, kw, code):
    assert _rope(L, **kw) == code


def _write(L, cache=None, **kw):
    s = (ctypes.c_int64 * 3)(4096, 2048, 128)
    a = dict(K=FAKE, V=FAKE, B=1, N=4, M=4, ks=s, vs=s, pages=FAKE, mp=2, start=FAKE, count=None, rows=None, ws=FAKE,
             wb=256)
    a.update(kw)
    return L.minf_kv_write(cache or _cache(), *a.values(), None)


def _read(L, cache=None, **kw):
    a = dict(pages=FAKE, B=1, mp=2, lens=FAKE, N=4, K=FAKE, V=FAKE, ws=FAKE, wb=256)
    a.update(kw)
    return L.minf_kv_read(cache or _cache(), *a.values(), None)


def _tree(L, cache=None, **kw):
    a = dict(Q=FAKE, B=1, Hq=4, T=4, scale=0.0, pages=FAKE, mp=2, ctx=FAKE, nd=None, mask=None, O=FAKE, lse=None, ws=FAKE,
             wb=1 << 40)
    a.update(kw)
    return L.minf_tree_attn(cache or _cache(), *a.values(), None)


@pytest.mark.parametrize("kw,code", BAD_CACHE)
def test_cache_refusals(L, kw, code):
    for call in (_write, _read, _tree):
        assert call(L, cache=_cache(**kw)) == code


def test_cache_call_refusals(L):
    odd = (ctypes.c_int64 * 3)(4096, 2048, 132)
    neg = (ctypes.c_int64 * 3)(-4096, 2048, 128)
    for kw, code in [(dict(K=None), 1), (dict(V=None), 1), (dict(pages=None), 1), (dict(mp=0), 1), (dict(start=None), 1),
                     (dict(B=0), 1), (dict(N=-1), 1), (dict(M=3), 1), (dict(ks=None), 1), (dict(ks=odd), 1),
                     (dict(vs=neg), 1), (dict(K=FAKE + 8), 1), (dict(ws=None), 1), (dict(wb=255), 4), (dict(mp=1 << 28), 2),
                     (dict(N=1 << 30, M=1 << 30, B=2), 2), (dict(N=0, M=0, K=None, V=None), 0)]:
        assert _write(L, **kw) == code, kw
    for kw, code in [(dict(K=None), 1), (dict(V=FAKE + 8), 1), (dict(lens=None), 1), (dict(N=-1), 1), (dict(wb=0), 4),
                     (dict(ws=FAKE + 8), 1), (dict(N=1 << 30), 2), (dict(N=0, K=None, V=None), 0)]:
        assert _read(L, **kw) == code, kw
    need = L.minf_tree_attn_workspace(1, 4, 2, 4, 128)
    assert need >= 256
    for kw, code in [(dict(Q=None), 1), (dict(O=None), 1), (dict(ctx=None), 1), (dict(T=0), 1), (dict(T=65), 2),
                     (dict(Hq=3), 1), (dict(Hq=0), 1), (dict(mask=FAKE + 4), 1), (dict(O=FAKE + 8), 1),
                     (dict(wb=need - 1), 4), (dict(ws=None), 1), (dict(B=1 << 24, Hq=64), 2)]:
        assert _tree(L, **kw) == code, kw
    for bad in [(0, 4, 2, 4, 128), (1, 3, 2, 4, 128), (1, 4, 2, 0, 128), (1, 4, 2, 65, 128), (1, 4, 2, 4, 96)]:
        assert L.minf_tree_attn_workspace(*bad) == 0


# --------------------------------------------------------------- binding refusals
OWN = r"^(?!serving call)"   # refused for what the case has wrong, not for lying on the CPU


def test_binding_refuses_mismatched_tensors():
    bf = dict(dtype=torch.bfloat16)
    with pytest.raises(minf.MinfError, match=OWN):
        minf.KVCache(torch.zeros(2, 1, 16, 64, **bf), torch.zeros(2, 1, 16, 128, **bf))
    with pytest.raises(minf.MinfError, match=OWN):
        minf.KVCache(torch.zeros(2, 1, 16, 64), torch.zeros(2, 1, 16, 64))
    with pytest.raises(minf.MinfError, match=OWN):                       # exponents missing
        k = torch.zeros(2, 1, 16, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
        minf.KVCache(k, k.clone())
    with pytest.raises(minf.MinfError, match=OWN):                       # exponents without an 8-bit cache
        e = torch.zeros(2, 1, 16, dtype=torch.uint8)
        minf.KVCache(torch.zeros(2, 1, 16, 64, **bf), torch.zeros(2, 1, 16, 64, **bf), e, e)
    c = minf.KVCache.empty(2, 1, 16, 64, device="cpu")
    pages = torch.zeros(1, 2, dtype=torch.int32)
    i1 = torch.zeros(1, dtype=torch.int32)
    k = torch.zeros(1, 1, 4, 64, **bf)
    for kw in (dict(k=k.float()), dict(k=k[..., :32]), dict(k=k.transpose(2, 3).contiguous().transpose(2, 3)),
               dict(pages=pages.long()), dict(pages=pages[0]), dict(start=i1.long()), dict(start=torch.zeros(2, dtype=torch.int32)),
               dict(count=i1.float()), dict(rows=i1)):
        a = dict(k=k, v=k, pages=pages, start=i1)
        a.update(kw)
        with pytest.raises(minf.MinfError, match=OWN):
            minf.minf_kv_write(a["k"], a["v"], c, a["pages"], a["start"], count=a.get("count"), rows=a.get("rows"))
    q = torch.zeros(1, 2, 3, 64, **bf)
    for kw in (dict(q=q.half()), dict(q=q.transpose(1, 2)), dict(q=q[..., :32]), dict(ctx=i1.long()),
               dict(mask=torch.zeros(1, 3, dtype=torch.int32)), dict(mask=torch.zeros(1, 2, dtype=torch.int64)),
               dict(nd=torch.zeros(2, dtype=torch.int32))):
        a = dict(q=q, ctx=i1)
        a.update(kw)
        with pytest.raises(minf.MinfError, match=OWN):
            minf.minf_tree_attn(a["q"], c, pages, a["ctx"], n_draft=a.get("nd"), tree_mask=a.get("mask"))
    with pytest.raises(minf.MinfError, match=OWN):
        minf.minf_kv_read(c, pages, i1.long(), 4)
    x = torch.zeros(1, 3, 4 * 64, **bf)
    for kw in (dict(qkv=x.float()), dict(qkv=x[0]), dict(qkv=x[..., :102]), dict(pos=torch.zeros(1, 3, dtype=torch.int64)),
               dict(pos=torch.zeros(3, dtype=torch.int32)), dict(inv_freq=torch.zeros(32)), dict(q_weight=torch.zeros(64)),
               dict(k_weight=torch.zeros(32, **bf))):
        a = dict(qkv=x)
        a.update(kw)
        with pytest.raises(minf.MinfError, match=OWN):
            minf.minf_qkv_norm_rope(Hq=2, Hkv=1, **a)


def test_binding_refuses_host_memory():
    x = torch.zeros(1, 3, 4 * 64, dtype=torch.bfloat16)
    with pytest.raises(minf.MinfError, match="device memory"):
        minf.minf_qkv_norm_rope(x, 2, 1)
    c = minf.KVCache.empty(2, 1, 16, 64, device="cpu")
    with pytest.raises(minf.MinfError, match="device memory"):
        minf.minf_kv_read(c, torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), 4)
