"""Masked attention where offsets fall: the sequence that falls is left out, and no other,
whichever kernel takes the call and however its blocks are dealt."""
import numpy as np
import pytest
import torch

import kv8mask as mask
import kv8util as ref
from test_gpu_kv8 import queries, w4  # noqa: F401

pytestmark = pytest.mark.gpu


def definition(q, cache, table, lens, cu, max_q, window, sinks, dtype):
    """(out, tolerance, number of sequences that claim the row); a row that several claim has
    the first one's, a row that none claims NaN. Too many queries give zeros."""
    total = q.shape[0]
    out = torch.full(q.shape, float("nan"), dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    claims = torch.zeros(total, dtype=torch.int32, device="cuda")
    for b in reversed(range(len(lens))):
        q0, end = cu[b], cu[b + 1]
        if not 0 <= q0 <= end <= total:
            continue
        claims[q0:end] += 1
        if end - q0 > max_q:
            out[q0:end], tol[q0:end] = 0, 0
        elif end > q0:
            n, m = lens[b], end - q0
            out[q0:end], tol[q0:end] = mask.attention(
                q[q0:end], cache, table[b:b + 1], [n], [m], lambda _: mask.window_sees(n, m, window, sinks),
                q.shape[2] ** -0.5, dtype)
    return out, tol, claims


def setting(lens, total, heads, kv_heads, dim, dtype, page, seed):
    pages = sum(-(-n // page) for n in lens)
    cache = ref.random_cache(w4_module(), pages, kv_heads, page, dim, seed=seed)
    return queries(total, heads, dim, dtype, seed + 1).contiguous(), cache, ref.scattered_table(lens, page, pages, seed=seed + 2)


def w4_module():
    import int4_weight_only_repack_gb300 as mod
    return mod


def holds(out, want, tol, rows):
    """Equal within the tolerance in these rows, NaN where and only where nothing is due."""
    got, want, tol = out[rows].double(), want[rows], tol[rows]
    assert torch.equal(got.isnan(), want.isnan())
    assert ((got - want).abs().nan_to_num(0) <= tol).all()


@pytest.mark.parametrize("heads,kv_heads,dim,dtype", [(8, 2, 64, "bf16"), (4, 4, 128, "fp16"), (5, 1, 128, "bf16")])
@pytest.mark.parametrize("again", [1, 5, 12])
def test_sequences_behind_rows_that_are_claimed_again(w4, heads, kv_heads, dim, dtype, again):
    """700 rows claimed `again` times more, and single tokens behind them that only one
    sequence claims: those are all there."""
    long, singles, batch = 700, 25, 60
    cu = [0, long] + [0, long] * again + [long + i + 1 for i in range(singles)]
    cu += [cu[-1]] * (batch + 1 - len(cu))
    rng = np.random.default_rng(again)
    lens = [int(rng.integers(1, 900)) for _ in range(batch)]
    total = long + singles
    q, cache, table = setting(lens, total + 3, heads, kv_heads, dim, dtype, 32, 100)
    want, tol, claims = definition(q[:total], cache, table, lens, cu, long, 90, 2, dtype)
    assert (claims[long:] == 1).all() and (claims[:long] == again + 1).all()
    out = torch.full_like(q, float("nan"))
    w4.kv8_attention(q, cache, table, ref.ints(lens), ref.ints(cu), long, 900, out=out, window=90, sinks=2)
    assert w4.w4_device_status(clear=True) == 14
    holds(out, want, tol, slice(long, total))
    assert torch.isfinite(out[:long]).all() and out[total:].isnan().all()
    # one below the bound: zeros instead, in those rows alone
    w4.kv8_attention(q, cache, table, ref.ints(lens), ref.ints(cu), long - 1, 900, out=out, window=90, sinks=2)
    assert w4.w4_device_status(clear=True) == 14
    holds(out, want, tol, slice(long, total))
    assert not out[:long].any() and out[total:].isnan().all()


@pytest.mark.parametrize("heads,kv_heads,dim,dtype", [(8, 2, 64, "fp16"), (3, 3, 128, "bf16"), (5, 1, 64, "bf16")])
@pytest.mark.parametrize("batch,seed", [(3, 1), (9, 2), (33, 3), (40, 4), (64, 5), (70, 6), (150, 7), (40, 8)])
def test_offsets_that_fall(w4, heads, kv_heads, dim, dtype, batch, seed):
    """Anywhere and to anywhere: each row has its sequence's result, and rows that several
    claim the first one's, as blocks for the rows that there are go to it."""
    rng = np.random.default_rng(seed)
    counts = [int(rng.integers(0, 3)) for _ in range(batch)]
    counts[int(rng.integers(0, batch))] = 900
    cu = np.concatenate([[0], np.cumsum(counts)])
    total = int(cu[-1])
    for _ in range(int(rng.integers(1, 5))):
        cu[int(rng.integers(1, batch + 1))] = int(rng.integers(0, total + 1))
    cu, lens = cu.tolist(), [int(rng.integers(1, 1500)) for _ in range(batch)]
    q, cache, table = setting(lens, total, heads, kv_heads, dim, dtype, 16, 110)
    window = int(rng.integers(1, 400))
    for max_q in (900, 300):
        want, tol, claims = definition(q, cache, table, lens, cu, max_q, window, 3, dtype)
        out = torch.full_like(q, float("nan"))
        w4.kv8_attention(q, cache, table, ref.ints(lens), ref.ints(cu), max_q, 1500, out=out, window=window, sinks=3)
        w4.w4_device_status(clear=True)
        rows = -(-max_q * (heads // kv_heads) // 256)
        packed = 2 * (total * (heads // kv_heads) // 256 + batch) <= rows * batch
        holds(out, want, tol, claims >= 0 if packed else claims <= 1)


@pytest.mark.parametrize("seed", range(6))
def test_offsets_that_leave_the_rows(w4, seed):
    """Below zero, past the last row, and falling: what is written is right, what no
    sequence claims is not written."""
    rng = np.random.default_rng(20 + seed)
    batch, heads, kv_heads, dim = 40, 8, 2, 64
    counts = [int(rng.integers(0, 3)) for _ in range(batch)]
    counts[int(rng.integers(0, batch))] = 700
    cu = np.concatenate([[0], np.cumsum(counts)])
    total = int(cu[-1])
    for _ in range(6):
        cu[int(rng.integers(0, batch + 1))] = int(rng.choice([-1, -2 ** 31, total + 1, 2 ** 31 - 1, int(rng.integers(0, total))]))
    cu, lens = cu.tolist(), [int(rng.integers(1, 900)) for _ in range(batch)]
    q, cache, table = setting(lens, total, heads, kv_heads, dim, "bf16", 32, 120)
    want, tol, claims = definition(q, cache, table, lens, cu, 700, 100, 4, "bf16")
    out = torch.full_like(q, float("nan"))
    w4.kv8_attention(q, cache, table, ref.ints(lens), ref.ints(cu), 700, 900, out=out, window=100, sinks=4)
    assert w4.w4_device_status(clear=True) == 14
    assert out[claims == 0].isnan().all()
    there = (claims == 1) & ~out.isnan().flatten(1).any(1)
    assert out[(claims == 1) & ~there].isnan().all()
    holds(out, want, tol, there)


def test_a_graph_replayed_on_offsets_that_fall(w4):
    """Blocks dealt anew in every replay: good offsets, bad ones, good ones again."""
    counts = [1, 700, 2, 0, 40, 1] + [1] * 34
    lens = [300, 750, 90, 5, 400, 33] + [64 + b for b in range(34)]
    total, heads, kv_heads = sum(counts), 8, 2
    q, cache, table = setting(lens, total, heads, kv_heads, 128, "fp16", 32, 130)
    n, good = ref.ints(lens), ref.bounds(counts)
    cu, out = good.clone(), torch.zeros_like(q)
    call = lambda: w4.kv8_attention(q, cache, table, n, cu, 700, 800, out=out, window=90, sinks=2)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for at, to in ((None, 0), (5, 0), (None, 0), (3, 1), (30, 0), (None, 0)):
        cu.copy_(good)
        if at is not None:
            cu[at] = to
        out.fill_(float("nan"))
        graph.replay()
        want, tol, _ = definition(q, cache, table, lens, cu.tolist(), 700, 90, 2, "fp16")
        holds(out, want, tol, slice(None))
        assert w4.w4_device_status(clear=True) == (0 if at is None else 14)


@pytest.mark.parametrize("batch,long,heads,kv_heads,dim,window", [
    (900, 150, 8, 2, 64, 40), (900, 1500, 8, 2, 64, 40), (1500, 2500, 5, 1, 128, 70), (5000, 700, 4, 1, 64, 20)])
def test_a_chunk_beside_many_sequences(w4, batch, long, heads, kv_heads, dim, window):
    """Whether blocks are found by the offsets or counted by number, which both happen here."""
    rng = np.random.default_rng(batch + long)
    counts = [int(rng.integers(0, 2)) for _ in range(batch)]
    counts[batch // 3] = long
    lens = [max(1, c) + int(rng.integers(0, 60)) for c in counts]
    cu = np.concatenate([[0], np.cumsum(counts)]).tolist()
    q, cache, table = setting(lens, cu[-1] + 5, heads, kv_heads, dim, "bf16", 16, 140)
    total = cu[-1]
    out = torch.full_like(q, float("nan"))
    w4.kv8_attention(q, cache, table, ref.ints(lens), ref.ints(cu), long, max(lens), out=out, window=window, sinks=3)
    assert w4.w4_device_status() == 0 and out[total:].isnan().all()
    sees = lambda b: mask.window_sees(lens[b], counts[b], window, 3)  # noqa: E731
    want, tol = mask.attention(q[:total], cache, table, lens, counts, sees, dim ** -0.5, "bf16")
    holds(out, want, tol, slice(0, total))
