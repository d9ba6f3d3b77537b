"""Host-side refusals of the 8-bit key-value cache's entry points: the documented
status before anything touches the GPU (these run on a machine without one)."""
import ctypes

import pytest
import torch

from libutil import ensure_built

NULL, SHAPE, ALIGN, DTYPE, ALIAS, WORKSPACE = 1, 2, 4, 5, 7, 10
# addresses that are never followed, far from one another
K, V, KS, VS, Q, OUT, T, L, C, W = ((i + 1) << 36 for i in range(10))


@pytest.fixture(scope="module")
def w4():
    ensure_built()
    import int4_weight_only_repack_gb300 as mod
    return mod


def cache(w4, **change):
    f = dict(k=K, v=V, k_scale=KS, v_scale=VS, num_pages=10, page_size=64, kv_heads=8, head_dim=128)
    f.update(change)
    return w4._KV8CacheStruct(**f)


BAD_CACHES = [
    (dict(head_dim=96), SHAPE), (dict(head_dim=256), SHAPE), (dict(page_size=8), SHAPE),
    (dict(page_size=48), SHAPE), (dict(kv_heads=0), SHAPE), (dict(num_pages=0), SHAPE),
    (dict(num_pages=1 << 22), SHAPE),  # 2^31 rows
    (dict(k=None), NULL), (dict(v_scale=None), NULL), (dict(v=V + 8), ALIGN), (dict(k_scale=KS + 4), ALIGN),
]


def append(w4, c, **change):
    a = dict(k=Q, v=OUT, ks=1024, vs=1024, c=c, t=T, ts=4, l=L, cu=C, b=3, n=7, m=5, dt=1)
    a.update(change)
    ref = ctypes.addressof(a["c"]) if a["c"] is not None else None
    return w4.lib().w4_kv8_append(a["k"], a["v"], a["ks"], a["vs"], ref, a["t"], a["ts"], a["l"],
                                  a["cu"], a["b"], a["n"], a["m"], a["dt"], None)


def attend(w4, c, **change):
    a = dict(q=Q, qs=4096, c=c, t=T, ts=4, l=L, cu=C, o=OUT, b=3, n=7, m=5, kv=200, h=32, s=0.1, ca=1,
             dt=1, w=W, wb=1 << 30)
    a.update(change)
    ref = ctypes.addressof(a["c"]) if a["c"] is not None else None
    how = w4._KV8HeadsStruct(a["h"] or 0, a["ca"], a["s"])
    return w4.lib().w4_kv8_attention(a["q"], a["qs"], ref, a["t"], a["ts"], a["l"], a["cu"], a["o"],
                                     a["b"], a["n"], a["m"], a["kv"],
                                     None if a["h"] is None else ctypes.addressof(how), a["dt"],
                                     a["w"], a["wb"], None)


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_bad_caches(w4, change, status):
    c = cache(w4, **change)
    assert append(w4, c) == status
    assert attend(w4, c) == status
    assert w4.lib().w4_kv8_copy_pages(ctypes.addressof(c), T, L, 3, None) == status


def test_cache_missing(w4):
    assert append(w4, None) == NULL and attend(w4, None) == NULL
    assert w4.lib().w4_kv8_copy_pages(None, T, L, 3, None) == NULL


@pytest.mark.parametrize("change,status", [
    (dict(dt=2), DTYPE), (dict(b=-1), SHAPE), (dict(n=-1), SHAPE), (dict(m=-1), SHAPE),
    (dict(ts=0), SHAPE), (dict(ks=1016), SHAPE), (dict(vs=1028), SHAPE), (dict(t=None), NULL),
    (dict(l=None), NULL), (dict(cu=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL),
    (dict(k=Q + 8), ALIGN), (dict(t=T + 2), ALIGN), (dict(k=K + 64), ALIAS), (dict(v=KS), ALIAS),
    (dict(t=V + 4096), ALIAS), (dict(b=0, t=None, l=None, cu=None), 0), (dict(n=0), 0), (dict(m=0), 0),
])
def test_append_refusals(w4, change, status):
    assert append(w4, cache(w4), **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(dt=-1), DTYPE), (dict(b=-1), SHAPE), (dict(h=20), SHAPE), (dict(h=0), SHAPE),
    (dict(h=2048), SHAPE), (dict(h=None), NULL), (dict(ca=2), SHAPE), (dict(kv=-1), SHAPE), (dict(qs=4088), SHAPE), (dict(qs=4100), SHAPE),
    (dict(s=float("nan")), SHAPE), (dict(s=float("inf")), SHAPE), (dict(q=None), NULL),
    (dict(o=None), NULL), (dict(l=None), NULL), (dict(o=OUT + 2), ALIGN), (dict(l=L + 1), ALIGN),
    (dict(w=W + 8), ALIGN), (dict(o=Q + 4096), ALIAS), (dict(o=K), ALIAS), (dict(o=T), ALIAS),
    (dict(b=0, t=None, l=None, cu=None), 0), (dict(n=0), 0), (dict(m=0), 0),
])
def test_attention_refusals(w4, change, status):
    assert attend(w4, cache(w4), **change) == status


def test_attention_workspace(w4):
    size = w4.w4_kv8_attention_workspace_size(2, 2, 1, 100000, 32, 8, 128)
    if size:
        c = cache(w4, num_pages=4000)
        change = dict(b=2, n=2, m=1, kv=100000, ts=2000)
        assert attend(w4, c, w=None, wb=0, **change) == WORKSPACE
        assert attend(w4, c, wb=size - 1, **change) == WORKSPACE
        assert attend(w4, c, w=OUT, **change) == ALIAS
    assert w4.w4_kv8_attention_workspace_size(2, 2, 1, 100000, 30, 8, 128) == 0


def test_pool_refusals(w4):
    lib, ws = w4.lib(), w4.w4_kv8_pages_workspace_size(100, 6)
    assert ws >= 4 * (100 + 6)
    ok = (K, 100, T, 4, L, 6)
    reserve = lambda *a: lib.w4_kv8_reserve(*a, None)  # noqa: E731
    assert reserve(None, 100, T, 4, L, 6, Q, 64, None, W, ws) == NULL
    assert reserve(K, 0, T, 4, L, 6, Q, 64, None, W, ws) == SHAPE
    assert reserve(*ok, Q, 20, None, W, ws) == SHAPE
    assert reserve(*ok, None, 64, None, W, ws) == NULL
    assert reserve(*ok, Q, 64, None, W, ws - 1) == WORKSPACE
    assert reserve(*ok, Q, 64, None, None, ws) == WORKSPACE
    assert reserve(*ok, Q, 64, None, W + 4, ws) == ALIGN
    assert reserve(*ok, L, 64, None, W, ws) == ALIAS
    assert reserve(*ok, Q, 64, K + 8, W, ws) == ALIAS
    fork = lambda *a: lib.w4_kv8_fork(*a, None)  # noqa: E731
    assert fork(*ok, Q, V, 7, 64, KS, VS, None, W, ws) == SHAPE  # more targets than sequences
    assert fork(*ok, Q, None, 2, 64, KS, VS, None, W, ws) == NULL
    assert fork(*ok, Q, V, 2, 64, KS, KS + 4, None, W, ws) == ALIAS
    assert fork(*ok, Q, V, 2, 64, KS, Q, None, W, ws) == ALIAS
    free = lambda *a: lib.w4_kv8_free(*a, None)  # noqa: E731
    assert free(*ok, None, 2, 64, None) == NULL
    assert free(*ok, Q, -1, 64, None) == SHAPE
    assert free(*ok, T + 8, 2, 64, None) == ALIAS
    compact = lambda *a: lib.w4_kv8_compact(*a, None)  # noqa: E731
    assert compact(K, 100, T, 4, 6, None, VS, W, ws) == NULL
    assert compact(K, 100, T, 4, 6, KS, VS, W, 16) == WORKSPACE
    assert compact(K, 100, T, 4, 6, KS, KS + 396, W, ws) == ALIAS
    assert lib.w4_kv8_copy_pages(ctypes.addressof(cache(w4)), K, L, 3, None) == ALIAS
    assert lib.w4_kv8_copy_pages(ctypes.addressof(cache(w4)), None, L, 3, None) == NULL
    assert lib.w4_kv8_copy_pages(ctypes.addressof(cache(w4)), T, L, 0, None) == 0
    assert w4.w4_kv8_pages_workspace_size(0, 5) == 0


def test_status_strings(w4):
    for s, word in ((14, "PAGE"), (15, "NO_PAGES"), (16, "SEQ")):
        assert word in w4.w4_status_string(s)


def test_binding_refusals(w4):
    f8 = torch.zeros((4, 2, 16, 64), dtype=torch.uint8).view(torch.float8_e4m3fn)
    sc = torch.ones((4, 2))
    with pytest.raises(ValueError):
        w4.KV8Cache(f8.view(torch.uint8), f8, sc, sc)
    with pytest.raises(ValueError):
        w4.KV8Cache(f8, f8, sc[:3], sc)
    with pytest.raises(ValueError):
        w4.KV8Cache(f8.transpose(0, 1), f8.transpose(0, 1), sc.T, sc.T)
    c = w4.KV8Cache(f8, f8.clone(), sc, sc.clone())
    t, n, cu = (torch.zeros(s, dtype=torch.int32) for s in ((2, 4), (2,), (3,)))
    x = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        w4.kv8_attention(x[:, :, ::2], c, t, n, cu, 1, 16)        # dim 32
    with pytest.raises(ValueError):
        w4.kv8_attention(x.transpose(0, 1).contiguous().transpose(0, 1), c, t, n, cu, 1, 16)
    with pytest.raises(ValueError):
        w4.kv8_attention(x, c, t, n, cu[:2], 1, 16)
    with pytest.raises(ValueError):
        w4.kv8_attention(x, c, t.long(), n, cu, 1, 16)
    with pytest.raises(ValueError):
        w4.kv8_attention(x, c, t, n, cu, 1, 16, out=torch.empty(2, 4, 64))
    with pytest.raises(ValueError):
        w4.kv8_attention(x.float(), c, t, n, cu, 1, 16)           # fp32 queries
    with pytest.raises(w4.W4Error):
        w4.kv8_attention(torch.zeros((2, 3, 64), dtype=torch.bfloat16), c, t, n, cu, 1, 16)
    with pytest.raises(ValueError):
        w4.kv8_append(x, x, c, t, n, cu, 1)                       # 4 heads, not 2
    with pytest.raises(ValueError):
        w4.kv8_append(x[:, :2], x[:, :2].half(), c, t, n, cu, 1)
    with pytest.raises(ValueError):
        w4.KV8Pool(n, t, torch.zeros(3, dtype=torch.int32), 16)


def test_tokens_past_every_cache(w4):
    """Token positions, rounded up to a tile, have to stay inside 32 bits."""
    c = cache(w4)
    assert attend(w4, c, kv=(1 << 30) + 1) == SHAPE
    assert w4.w4_kv8_attention_workspace_size(2, 2, 1, (1 << 30) + 1, 32, 8, 128) == 0
