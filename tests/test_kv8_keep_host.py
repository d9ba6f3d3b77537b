"""Host-side refusals of w4_kv8_keep and w4_kv8_shorten, and of their binding (no GPU)."""
import ctypes

import pytest
import torch

from libutil import ensure_built
from test_kv8_binding import On, cache as small_cache, fake, ints  # noqa: F401
from test_kv8_host import ALIAS, ALIGN, BAD_CACHES, C, K, KS, L, NULL, OUT, Q, SHAPE, T, V, cache


@pytest.fixture(scope="module")
def w4():
    ensure_built()
    import int4_weight_only_repack_gb300 as mod
    return mod


def keep(w4, c, **change):
    a = dict(t=T, ts=4, l=L, cu=C, p=Q, b=3, n=7, m=5)
    a.update(change)
    return w4.lib().w4_kv8_keep(ctypes.addressof(c) if c is not None else None, a["t"], a["ts"], a["l"], a["cu"],
                                a["p"], a["b"], a["n"], a["m"], None)


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_bad_caches(w4, change, status):
    assert keep(w4, cache(w4, **change)) == status


@pytest.mark.parametrize("change,status", [
    (dict(b=-1), SHAPE), (dict(n=-1), SHAPE), (dict(m=-1), SHAPE), (dict(m=65), SHAPE), (dict(ts=0), SHAPE),
    (dict(t=None), NULL), (dict(l=None), NULL), (dict(cu=None), NULL), (dict(p=None), NULL),
    (dict(p=Q + 2), ALIGN), (dict(t=T + 1), ALIGN), (dict(p=K + 64), ALIAS), (dict(t=V), ALIAS), (dict(l=KS + 8), ALIAS),
    (dict(b=0, t=None, l=None, cu=None), 0), (dict(n=0, p=None), 0), (dict(m=0, p=None), 0),
])
def test_keep_refusals(w4, change, status):
    assert keep(w4, cache(w4), **change) == status


def test_keep_needs_a_cache(w4):
    assert keep(w4, None) == NULL
    assert keep(w4, cache(w4, v=K + 4096)) == ALIAS  # its own parts overlap


@pytest.mark.parametrize("change,status", [
    (dict(refs=None), NULL), (dict(table=None), NULL), (dict(lens=None), NULL), (dict(drop=None), NULL),
    (dict(pages=0), SHAPE), (dict(stride=0), SHAPE), (dict(seqs=-1), SHAPE), (dict(size=20), SHAPE),
    (dict(refs=K + 2), ALIGN), (dict(drop=Q + 1), ALIGN), (dict(status=OUT + 2), ALIGN),
    (dict(drop=L), ALIAS), (dict(drop=T + 8), ALIAS), (dict(drop=K + 396), ALIAS), (dict(status=L + 4), ALIAS),
    (dict(status=Q), ALIAS), (dict(lens=T + 92), ALIAS),
])
def test_shorten_refusals(w4, change, status):
    a = dict(refs=K, pages=100, table=T, stride=4, lens=L, seqs=6, drop=Q, size=64, status=None)
    a.update(change)
    assert w4.lib().w4_kv8_shorten(*a.values(), None) == status


def test_binding(w4, fake, monkeypatch):
    c, pool = small_cache(), w4.KV8Pool(ints(0, 0), torch.zeros((3, 4), dtype=torch.int32), ints(0, 0, 0), 16)
    table, lens, cu, path = torch.zeros((3, 4), dtype=torch.int32), ints(1, 1, 1), ints(0, 1, 2, 3), ints(0, 0, 0)
    for call in (lambda: w4.kv8_keep(c, table, lens, cu, path, 1), lambda: w4.kv8_shorten(pool, lens)):
        with pytest.raises(ValueError):  # on the CPU
            call()
    monkeypatch.setattr(w4, "_CURRENT_DEVICE", lambda: 0)
    monkeypatch.setattr(w4, "_on", lambda *_: None)
    c._device = pool._device = 0
    gpu = [On(t) for t in (table, lens, cu, path)]
    w4.kv8_keep(c, *gpu, 1)
    w4.kv8_shorten(pool, gpu[1])
    got = fake.seen["w4_kv8_keep"][0]
    assert got[1:9] == (table.data_ptr(), 4, lens.data_ptr(), cu.data_ptr(), path.data_ptr(), 3, 3, 1)
    assert fake.seen["w4_kv8_shorten"][0][6:8] == (lens.data_ptr(), 16)
    for i in range(4):
        with pytest.raises(ValueError):
            w4.kv8_keep(c, *[On(t.x, 1 if i == j else 0) for j, t in enumerate(gpu)], 1)
    for bad in (path.long(), torch.zeros((3, 2), dtype=torch.int32)[:, 0]):
        with pytest.raises(ValueError):
            w4.kv8_keep(c, *gpu[:3], On(bad), 1)
        with pytest.raises(ValueError):
            w4.kv8_shorten(pool, On(bad))
    with pytest.raises(ValueError):
        w4.kv8_shorten(pool, On(ints(0, 0)))
