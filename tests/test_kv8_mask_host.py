"""Host-side refusals of masked attention over the 8-bit cache, and what the binding
hands over (no GPU needed)."""
import ctypes

import pytest
import torch

from libutil import ensure_built
from test_kv8_host import ALIAS, ALIGN, C, DTYPE, L, NULL, OUT, Q, SHAPE, T, W, WORKSPACE, cache
from test_kv8_binding import cache as small_cache, fake, ints  # noqa: F401

TREE = 11 << 36


@pytest.fixture(scope="module")
def w4():
    ensure_built()
    import int4_weight_only_repack_gb300 as mod
    return mod


def attend(w4, **change):
    a = dict(q=Q, qs=4096, t=T, ts=4, l=L, cu=C, o=OUT, b=3, n=7, m=5, kv=200, h=32, s=0.1, ca=1, dt=1, w=W,
             wb=1 << 30, win=100, sinks=4, tree=None, mask=True)
    a.update(change)
    c = cache(w4)
    how = w4._KV8HeadsStruct(a["h"] or 0, a["ca"], a["s"])
    mask = w4._KV8MaskStruct(a["win"], a["sinks"], a["tree"])
    return w4.lib().w4_kv8_attention_masked(
        a["q"], a["qs"], ctypes.addressof(c), a["t"], a["ts"], a["l"], a["cu"], a["o"], a["b"], a["n"],
        a["m"], a["kv"], None if a["h"] is None else ctypes.addressof(how),
        ctypes.addressof(mask) if a["mask"] else None, a["dt"], a["w"], a["wb"], None)


@pytest.mark.parametrize("change,status", [
    (dict(mask=False), NULL), (dict(win=0, sinks=0), NULL), (dict(win=0, sinks=4), NULL),
    (dict(win=0, sinks=4, tree=TREE), SHAPE), (dict(win=-1), SHAPE), (dict(sinks=-1), SHAPE),
    (dict(sinks=(1 << 30) + 1), SHAPE), (dict(ca=0), SHAPE), (dict(ca=2), SHAPE), (dict(tree=TREE, m=65), SHAPE),
    (dict(tree=TREE + 4), ALIGN), (dict(tree=OUT + 8), ALIAS), (dict(tree=OUT - 8), ALIAS),
    (dict(tree=W + 64, m=5, kv=100000), ALIAS),
    # and what the call without a mask refuses
    (dict(h=None), NULL), (dict(dt=-1), DTYPE), (dict(b=-1), SHAPE), (dict(h=20), SHAPE), (dict(kv=-1), SHAPE),
    (dict(qs=4088), SHAPE), (dict(s=float("nan")), SHAPE), (dict(q=None), NULL), (dict(o=None), NULL),
    (dict(o=OUT + 2), ALIGN), (dict(o=Q + 4096), ALIAS), (dict(o=T), ALIAS), (dict(kv=100000, w=None), WORKSPACE),
    (dict(b=0, t=None, l=None, cu=None), 0), (dict(n=0), 0), (dict(m=0), 0),
    (dict(n=0, tree=TREE), 0),
])
def test_refusals(w4, change, status):
    assert attend(w4, **change) == status


def test_binding(w4, fake, monkeypatch):
    """The mask that the library gets, and that calls without one are as they were."""
    got = []

    def masked(*args):
        m = w4._KV8MaskStruct.from_address(args[13])
        got.append((m.window, m.sinks, m.tree))
        return 0

    monkeypatch.setattr(w4, "_one_gpu", lambda *_: None)
    monkeypatch.setattr(fake, "w4_kv8_attention_masked", masked, raising=False)
    c, x = small_cache(), torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    args = (x, c, torch.zeros((3, 4), dtype=torch.int32), ints(1, 1, 1), ints(0, 1, 2, 3), 1, 16)
    room = torch.zeros(512, dtype=torch.uint8)
    call = lambda **how: w4.kv8_attention(*args, workspace=room, **how)  # noqa: E731
    call()
    assert not got and len(fake.seen["w4_kv8_attention"]) == 1
    tree = torch.ones(3, dtype=torch.int64)
    for how in (dict(window=7), dict(window=7, sinks=3), dict(tree=tree), dict(window=2 ** 40, sinks=2 ** 35, tree=tree)):
        call(**how)
    assert got == [(7, 0, None), (7, 3, None), (0, 0, tree.data_ptr()), (2 ** 30, 2 ** 30, tree.data_ptr())]
    for how in (dict(sinks=3), dict(sinks=3, tree=tree), dict(window=0), dict(window=-5), dict(window=4, sinks=-1),
                dict(window=4, causal=False), dict(tree=tree, causal=False), dict(tree=tree[:2]),
                dict(tree=tree.int()), dict(tree=torch.ones(6, dtype=torch.int64)[::2])):
        with pytest.raises(ValueError):
            call(**how)
    assert len(got) == 4


def test_a_tree_on_the_cpu_is_refused(w4):
    c, x = small_cache(), torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        w4.kv8_attention(x, c, torch.zeros((3, 4), dtype=torch.int32), ints(1, 1, 1), ints(0, 1, 2, 3), 1, 16,
                         tree=torch.ones(3, dtype=torch.int64))
