"""Attention over the 8-bit cache with a window and sinks, and of trees of drafts,
against the definition in 64 bits (kv8mask)."""
import numpy as np
import pytest
import torch

import kv8mask as mask
import kv8util as ref
from test_gpu_kv8 import queries, w4  # noqa: F401

pytestmark = pytest.mark.gpu

HEADS = [(8, 8, 128), (16, 2, 128), (14, 2, 64), (5, 1, 128), (71, 1, 64), (40, 1, 128)]


def check(w4, q, cache, table, lens, counts, dtype, window=None, sinks=0, trees=None, slack=0, spare=0):
    """One call against the definition; `spare` rows behind the last sequence stay."""
    total = sum(counts)
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    tree = None
    if trees is not None:
        tree = mask.words_tensor(sum(trees, []) + [-1 & (1 << 64) - 1] * spare)
    w4.kv8_attention(q, cache, table, ref.ints(lens), ref.bounds(counts), max(max(counts), 1) + slack,
                     max(max(lens), 1) + slack, out=out, window=window, sinks=sinks, tree=tree)

    def sees(b):
        if trees is not None:
            return mask.tree_sees(lens[b], counts[b], trees[b], window, sinks)
        return mask.window_sees(lens[b], counts[b], window, sinks)

    want, tol = mask.attention(q[:total], cache, table, lens, counts, sees, q.shape[2] ** -0.5, dtype)
    assert torch.isfinite(out[:total]).all()
    worst = ((out[:total].double() - want).abs() / tol.clamp_min(1e-30)).max().item() if total else 0.0
    assert worst <= 1, worst
    assert out[total:].isnan().all()
    assert w4.w4_device_status() == 0
    return out[:total]


# --------------------------------------------------------------------------- #
# windows                                                                       #
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("heads,kv_heads,dim", HEADS)
@pytest.mark.parametrize("page,dtype,window,sinks", [
    (16, "bf16", 1, 0), (32, "fp16", 7, 1), (64, "bf16", 32, 4), (128, "fp16", 33, 40),
    (16, "fp16", 300, 16), (64, "bf16", 600, 0), (32, "bf16", 5000, 3)])
@pytest.mark.parametrize("slack", [0, 600])
def test_decode(w4, heads, kv_heads, dim, page, dtype, window, sinks, slack):
    """slack: the bound of the lengths, by which an item is a CTA's or is split."""
    lens = [1, 15, 16, 17, 0, 31, 33, 64, 65, 127, 128, 129, 300, 1031 if slack else 500]
    cache = ref.random_cache(w4, 200, kv_heads, page, dim, seed=1)
    table = ref.scattered_table(lens, page, 200, seed=2)
    q = queries(len(lens) + 3, heads, dim, dtype, 3, pad=2)
    out = check(w4, q, cache, table, lens, [1] * len(lens), dtype, window, sinks, slack=slack, spare=3)
    assert torch.count_nonzero(out[4]) == 0  # nothing to see


@pytest.mark.parametrize("heads,kv_heads,dim", HEADS)
@pytest.mark.parametrize("window,sinks,page,dtype", [
    (1, 0, 16, "fp16"), (1, 2, 64, "bf16"), (3, 5, 16, "bf16"), (40, 0, 64, "fp16"), (63, 64, 16, "fp16"),
    (130, 4, 32, "bf16"), (1000, 1, 128, "bf16")])
def test_ragged_rows(w4, heads, kv_heads, dim, window, sinks, page, dtype):
    """Some sequences have more new tokens than tokens: their first see nothing."""
    counts = [3, 1, 0, 17, 64, 5, 130, 9, 33]
    lens = [3, 77, 40, 17, 200, 0, 260, 4, 33]
    cache = ref.random_cache(w4, 120, kv_heads, page, dim, seed=4, scales="any")
    table = ref.scattered_table(lens, page, 120, seed=5)
    q = queries(sum(counts), heads, dim, dtype, 6)
    check(w4, q, cache, table, lens, counts, dtype, window, sinks, slack=11)


@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 4, 128), (14, 2, 64), (12, 1, 128), (4, 2, 64)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (6, 9), (64, 3), (700, 500)])
def test_few_rows_over_many_tokens(w4, heads, kv_heads, dim, window, sinks):
    counts = [5, 1, 3, 4]
    lens = [2500, 3333, 1200, 4]
    cache = ref.random_cache(w4, 300, kv_heads, 32, dim, seed=7)
    table = ref.scattered_table(lens, 32, 300, seed=8)
    q = queries(sum(counts), heads, dim, "bf16", 9)
    check(w4, q, cache, table, lens, counts, "bf16", window, sinks)


@pytest.mark.parametrize("heads,kv_heads,dim,n,m,page,window,sinks,dtype", [
    (8, 2, 128, 1000, 1000, 64, 100, 4, "bf16"),
    (4, 4, 128, 1777, 515, 16, 1, 0, "fp16"),
    (4, 4, 128, 1777, 515, 16, 127, 130, "fp16"),
    (9, 3, 64, 2290, 257, 128, 300, 0, "bf16"),
    (4, 1, 64, 4611, 300, 32, 1024, 16, "fp16"),
    (10, 1, 128, 2100, 131, 64, 129, 1, "bf16"),
    (2, 2, 64, 900, 900, 16, 5, 300, "bf16"),
])
def test_prompts(w4, heads, kv_heads, dim, n, m, page, window, sinks, dtype):
    lens, counts = [n, n // 3, n - 1], [m, min(m, n // 3), 1]
    pages = 3 * (n // page + 1)
    cache = ref.random_cache(w4, pages, kv_heads, page, dim, seed=10)
    table = ref.scattered_table(lens, page, pages, seed=11)
    q = queries(sum(counts), heads, dim, dtype, 12, pad=2 * kv_heads)
    check(w4, q, cache, table, lens, counts, dtype, window, sinks)


@pytest.mark.parametrize("heads,kv_heads,dim,n,m,window,sinks", [
    (8, 1, 128, 40000, 1, 20000, 100), (8, 1, 128, 40000, 1, 300, 100), (4, 2, 64, 30011, 33, 25000, 2000),
    (8, 1, 128, 20000, 40, 9000, 3000), (4, 4, 64, 9001, 200, 5000, 0)])
def test_long_axes(w4, heads, kv_heads, dim, n, m, window, sinks):
    """Split along the tokens, sinks and window in different parts, and joined."""
    cache = ref.random_cache(w4, n // 64 + 1, kv_heads, 64, dim, seed=13)
    table = ref.scattered_table([n], 64, n // 64 + 1, seed=14)
    check(w4, queries(m, heads, dim, "fp16", 15), cache, table, [n], [m], "fp16", window, sinks)


@pytest.mark.parametrize("m,heads", [(1, 4), (1, 12), (6, 8), (300, 4), (40, 8)])
@pytest.mark.parametrize("slack", [0, 3000])
def test_a_wide_window_is_none(w4, m, heads, slack):
    """Bit for bit what the call without one gives, up to the largest numbers."""
    lens = [700, 350, 1]
    counts = [m, min(m, 350), 1]
    cache = ref.random_cache(w4, 60, 2, 32, 128, seed=16)
    table = ref.scattered_table(lens, 32, 60, seed=17)
    q = queries(sum(counts), heads, 128, "bf16", 18)
    args = (q, cache, table, ref.ints(lens), ref.bounds(counts), m, 700 + slack)
    want = w4.kv8_attention(*args)
    for window, sinks in ((2 ** 30, 0), (2 ** 30, 2 ** 30), (2 ** 40, 5), (10 ** 6, 2 ** 33), (700, 0), (1, 2 ** 30)):
        assert torch.equal(w4.kv8_attention(*args, window=window, sinks=sinks), want) or window < 2 ** 20
        got = w4.kv8_attention(*args, window=window, sinks=sinks)
        assert (got.float() - want.float()).abs().max() <= 2.0 ** -6 * want.float().abs().max()


# --------------------------------------------------------------------------- #
# trees                                                                         #
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("heads,kv_heads,dim", HEADS)
@pytest.mark.parametrize("kind", ["tree", "any"])
@pytest.mark.parametrize("page,dtype,window,sinks", [
    (16, "bf16", None, 0), (64, "fp16", None, 0), (32, "bf16", 20, 3), (128, "fp16", 1, 0)])
def test_trees(w4, heads, kv_heads, dim, kind, page, dtype, window, sinks):
    """Small enough for the few-row kernel in some of the heads; one sequence has more
    drafts than tokens, one no draft, one nothing but drafts."""
    counts = [5, 1, 0, 8, 7, 3, 9, 2]
    lens = [205, 77, 40, 8, 400, 0, 4, 130]
    rng = np.random.default_rng(19)
    trees = [mask.random_tree(m, rng, kind) for m in counts]
    cache = ref.random_cache(w4, 100, kv_heads, page, dim, seed=20, scales="any")
    table = ref.scattered_table(lens, page, 100, seed=21)
    q = queries(sum(counts) + 2, heads, dim, dtype, 22)
    for slack in (0, 55):
        check(w4, q, cache, table, lens, counts, dtype, window, sinks, trees, slack if max(counts) + slack <= 64 else 0,
              spare=2)


@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 1, 128), (14, 2, 64), (2, 2, 128), (1, 1, 64)])
@pytest.mark.parametrize("kind", ["tree", "any"])
@pytest.mark.parametrize("window,sinks", [(None, 0), (50, 70), (1000, 0)])
def test_wide_trees(w4, heads, kv_heads, dim, kind, window, sinks):
    """64 drafts, at every place of a page and a step."""
    counts = [64, 63, 33, 64, 64, 61]
    lens = [64, 1000, 33 + 95, 64 + 127, 64 + 1300, 3000]
    rng = np.random.default_rng(23)
    trees = [mask.random_tree(m, rng, kind) for m in counts]
    cache = ref.random_cache(w4, 200, kv_heads, 32, dim, seed=24)
    table = ref.scattered_table(lens, 32, 200, seed=25)
    q = queries(sum(counts), heads, dim, "bf16", 26)
    check(w4, q, cache, table, lens, counts, "bf16", window, sinks, trees)


@pytest.mark.parametrize("n,m,heads", [(30000, 60, 4), (9000, 64, 8), (20000, 7, 8)])
def test_trees_over_long_caches(w4, n, m, heads):
    rng = np.random.default_rng(27)
    cache = ref.random_cache(w4, n // 64 + 1, 1, 64, 128, seed=28)
    table = ref.scattered_table([n], 64, n // 64 + 1, seed=29)
    q = queries(m, heads, 128, "fp16", 30)
    check(w4, q, cache, table, [n], [m], "fp16", None, 0, [mask.random_tree(m, rng, "tree")])


@pytest.mark.parametrize("m,heads,n", [(1, 4, 900), (6, 8, 2000), (16, 2, 300), (60, 4, 1900), (64, 8, 64)])
def test_a_chain_is_no_tree(w4, m, heads, n):
    """Drafts in a row: bit for bit the call without a tree."""
    lens, counts = [n, n - 5 if n > 70 else n], [m, m]
    cache = ref.random_cache(w4, 80, 2, 64, 64, seed=31)
    table = ref.scattered_table(lens, 64, 80, seed=32)
    q = queries(2 * m, heads, 64, "bf16", 33)
    args = (q, cache, table, ref.ints(lens), ref.bounds(counts), m, n)
    chain = mask.words_tensor(2 * mask.random_tree(m, None, "chain"))
    assert torch.equal(w4.kv8_attention(*args, tree=chain), w4.kv8_attention(*args))


# --------------------------------------------------------------------------- #
# both                                                                          #
# --------------------------------------------------------------------------- #
def cases():
    """(name, counts, heads, window, sinks, tree?) of one and of many rows."""
    return [("decode", [1, 1], 8, 200, 5, False), ("drafts", [4, 2], 8, 200, 5, True),
            ("chunk", [150, 90], 4, 200, 5, False), ("wide tree", [60, 33], 8, 200, 5, True)]


@pytest.mark.parametrize("name,counts,heads,window,sinks,tree", cases())
@pytest.mark.parametrize("slack", [0, 3000])
def test_unseen_tokens_do_not_matter(w4, name, counts, heads, window, sinks, tree, slack):
    """NaN codes in every token that no query sees, of the sequence or of others."""
    lens, page = [1000, 777], 32
    rng = np.random.default_rng(34)
    trees = [mask.random_tree(m, rng, "tree") for m in counts] if tree else None
    cache = ref.random_cache(w4, 80, 2, page, 128, seed=35)
    table = ref.scattered_table(lens, page, 80, seed=36)
    q = queries(sum(counts), heads, 128, "bf16", 37)
    want = check(w4, q, cache, table, lens, counts, "bf16", window, sinks, trees, slack if not tree else 0).clone()
    seen = torch.zeros(80, page, dtype=torch.bool, device="cuda")
    near = torch.zeros(80, dtype=torch.bool, device="cuda")
    for b, (n, m) in enumerate(zip(lens, counts)):
        some = (mask.tree_sees(n, m, trees[b], window, sinks) if tree
                else mask.window_sees(n, m, window, sinks)).any(0).tolist()
        for j in range(n):
            seen[table[b, j // page].long(), j % page] |= some[j]
            if any(some[max(0, j - 256):j + 257]):
                near[table[b, j // page].long()] = True
    assert not seen.all() and not near.all()
    for codes, sc in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        raw = codes.view(torch.uint8)
        raw.copy_(torch.where(seen[:, None, :, None], raw, torch.full_like(raw, 0x7F)))
        sc.copy_(torch.where(near[:, None], sc, torch.full_like(sc, float("nan"))))
    got = check(w4, q, cache, table, lens, counts, "bf16", window, sinks, trees, slack if not tree else 0)
    assert torch.equal(got, want)


@pytest.mark.parametrize("name,counts,heads,window,sinks,tree", cases())
def test_nan_reaches_those_who_see_it(w4, name, counts, heads, window, sinks, tree):
    lens, page = [1000, 777], 64
    rng = np.random.default_rng(38)
    trees = [mask.random_tree(m, rng, "tree") for m in counts] if tree else None
    cache = ref.random_cache(w4, 40, 1, page, 64, seed=39)
    table = ref.scattered_table(lens, page, 40, seed=40)
    q = queries(sum(counts), heads, 64, "fp16", 41)
    sees = [mask.tree_sees(n, m, trees[b], window, sinks) if tree else mask.window_sees(n, m, window, sinks)
            for b, (n, m) in enumerate(zip(lens, counts))]
    how = dict(window=window, sinks=sinks, tree=mask.words_tensor(sum(trees, [])) if tree else None)
    args = (q, cache, table, ref.ints(lens), ref.bounds(counts), max(counts), 1000)
    clean = w4.kv8_attention(*args, **how)
    spots = [2, 4, 5, 60, 1000 - window - 1, 1000 - window, 1000 - window + 3, 999 - counts[0] // 2, 999]
    for spot in spots:
        for codes in (cache.k, cache.v):
            raw, at = codes.view(torch.uint8), (table[0, spot // page].long(), 0, spot % page, 7)
            keep = raw[at].clone()
            raw[at] = 0x7F
            got = w4.kv8_attention(*args, **how)
            raw[at] = keep
            hit = torch.cat((sees[0][:, spot], torch.zeros(counts[1], dtype=torch.bool, device="cuda")))
            if codes is cache.k:
                assert got[hit].isnan().all()
            else:  # (only its column of a value)
                assert got[hit][..., 7].isnan().all()
            assert torch.equal(got[~hit], clean[~hit])


@pytest.mark.parametrize("heads,max_q,max_kv", [(4, 1, 200), (4, 1, 3000), (16, 3, 200), (16, 3, 3000),
                                                (8, 33, 200), (8, 33, 3000)])
@pytest.mark.parametrize("tree", [False, True])
def test_more_new_tokens_than_the_bound_give_zeros(w4, heads, max_q, max_kv, tree):
    lens, counts = [100, 200, 150], [1, 300, max_q]
    cache = ref.random_cache(w4, 20, 2, 32, 64, seed=42)
    table = ref.scattered_table(lens, 32, 20, seed=43)
    q = queries(sum(counts), heads, 64, "bf16", 44)
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    words = [(1 << i % 64 + 1) - 1 for m in counts for i in range(m)]
    w4.kv8_attention(q, cache, table, ref.ints(lens), ref.bounds(counts), max_q, max_kv, out=out, window=70,
                     sinks=3, tree=mask.words_tensor(words) if tree else None)
    assert w4.w4_device_status(clear=True) == 14
    assert torch.count_nonzero(out[1:301]) == 0
    sees = lambda b: mask.window_sees([100, 0, 150][b], counts[b], 70, 3)  # noqa: E731
    want, tol = mask.attention(q, cache, table, [100, 0, 150], counts, sees, 64 ** -0.5, "bf16")
    keep = [0] + list(range(301, sum(counts)))
    assert ((out.double() - want).abs()[keep] <= tol[keep]).all()


@pytest.mark.parametrize("name,counts,heads,window,sinks,tree", cases())
def test_graphs(w4, name, counts, heads, window, sinks, tree):
    """Captured once, replayed on other lengths, trees and queries."""
    lens, page = [1000, 777], 64
    rng = np.random.default_rng(45)
    cache = ref.random_cache(w4, 60, 2, page, 64, seed=46)
    table = ref.scattered_table([1200, 1200], page, 60, seed=47)
    q = queries(sum(counts), heads, 64, "fp16", 48).contiguous()
    n, words = ref.ints(lens), None
    if tree:
        words = mask.words_tensor(sum((mask.random_tree(m, rng, "tree") for m in counts), []))
    call = lambda: w4.kv8_attention(q, cache, table, n, ref_cu, max(counts), 1200, window=window,  # noqa: E731
                                    sinks=sinks, tree=words)
    ref_cu = ref.bounds(counts)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for step in range(3):
        n.add_(61)
        q.copy_(queries(sum(counts), heads, 64, "fp16", 49 + step))
        if tree:
            words.copy_(mask.words_tensor(sum((mask.random_tree(m, rng, "any") for m in counts), [])))
        graph.replay()
        assert torch.equal(out, call())


def test_streams(w4):
    """Two streams at once, each with its own kept workspace."""
    lens, counts = [9000, 700], [3, 3]
    cache = ref.random_cache(w4, 400, 2, 32, 128, seed=52)
    table = ref.scattered_table(lens, 32, 400, seed=53)
    q = queries(6, 16, 128, "bf16", 54)
    args = (q, cache, table, ref.ints(lens), ref.bounds(counts), 3, 9000)
    want = [w4.kv8_attention(*args, window=w, sinks=4) for w in (8000, 90)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(20):
        got.append([w4.kv8_attention(*args, window=w, sinks=4, stream=s) for w, s in zip((8000, 90), streams)])
    torch.cuda.synchronize()
    for pair in got:
        assert torch.equal(pair[0], want[0]) and torch.equal(pair[1], want[1])


@pytest.mark.parametrize("tree", [False, True])
def test_more_sequences_than_a_split_call_takes(w4, tree):
    """Thousands of sequences, some longer than the window."""
    batch = 2100
    rng = np.random.default_rng(55)
    lens = [int(rng.integers(0, 40)) if b % 50 else 700 + b // 50 for b in range(batch)]
    counts = [min(2, n) for n in lens]
    trees = [mask.random_tree(m, rng, "any") for m in counts] if tree else None
    pages = sum(-(-n // 16) for n in lens)
    cache = ref.random_cache(w4, pages, 1, 16, 64, seed=56)
    table = ref.scattered_table(lens, 16, pages, seed=57)
    q = queries(sum(counts), 3, 64, "bf16", 58)
    check(w4, q, cache, table, lens, counts, "bf16", 600, 2, trees)


@pytest.mark.parametrize("counts,heads", [([1, 1], 4), ([30, 50], 4)])
def test_pages_past_32_bits(w4, counts, heads):
    """Codes that lie beyond 2^32 bytes."""
    lens, page, pages = [900, 333], 128, 40000  # 5.2 GB a side
    cache = w4.kv8_cache(pages, 8, page, 128)
    small = ref.random_cache(w4, 12, 8, page, 128, seed=59)
    near = ref.scattered_table(lens, page, 12, seed=60)
    for big, little in ((cache.k, small.k), (cache.v, small.v)):
        big.view(torch.uint8)[-12:].copy_(little.view(torch.uint8))
    cache.k_scale[-12:], cache.v_scale[-12:] = small.k_scale, small.v_scale
    far = torch.where(near >= 0, near + pages - 12, -1).to(torch.int32)
    q = queries(sum(counts), 8 * heads, 128, "fp16", 61)
    rng = np.random.default_rng(62)
    words = mask.words_tensor(sum((mask.random_tree(m, rng, "tree") for m in counts), []))
    for how in (dict(window=200, sinks=5), dict(tree=words), dict(window=100, tree=words)):
        args = ref.ints(lens), ref.bounds(counts), max(counts), 900
        assert torch.equal(w4.kv8_attention(q, cache, far, *args, **how), w4.kv8_attention(q, small, near, *args, **how))


def test_a_sequence_past_its_bounds(w4):
    """Longer than max_kv_len or its table row: zeros, and its neighbours are not touched."""
    lens, counts = [100, 200, 150], [2, 2, 2]
    cache = ref.random_cache(w4, 30, 2, 16, 64, seed=63)
    table = ref.scattered_table(lens, 16, 30, seed=64)
    q = queries(6, 4, 64, "bf16", 65)
    words = mask.words_tensor([1, 3] * 3)
    for n, most in (([100, 200, 150], 180), ([100, 16 * table.shape[1] + 1, 150], 1000), ([100, -1, 150], 1000)):
        for how in (dict(window=50, sinks=1), dict(tree=words)):
            out = w4.kv8_attention(q, cache, table, ref.ints(n), ref.bounds(counts), 2, most, **how)
            assert w4.w4_device_status(clear=True) == 14
            assert not out[2:4].any()
            rest = [0, 1, 4, 5]
            sees = lambda b: (mask.window_sees([100, 0, 150][b], 2, 50, 1) if "window" in how  # noqa: E731
                              else mask.tree_sees([100, 0, 150][b], 2, [1, 3]))
            want, tol = mask.attention(q, cache, table, [100, 0, 150], counts, sees, 64 ** -0.5, "bf16")
            assert ((out.double() - want).abs()[rest] <= tol[rest]).all()


def test_a_bad_page_counts_as_one_without_tokens(w4):
    lens, counts = [300], [4]
    cache = ref.random_cache(w4, 30, 1, 16, 64, seed=66)
    table = ref.scattered_table(lens, 16, 30, seed=67)
    q = queries(4, 4, 64, "bf16", 68)
    args = ref.ints(lens), ref.bounds(counts), 4, 300
    words = mask.words_tensor(mask.random_tree(4, None, "chain"))
    for bad in (30, -1, 2 ** 31 - 1, -2 ** 31):
        for how, spot in ((dict(window=100, sinks=20), 15), (dict(window=100, sinks=20), 1), (dict(tree=words), 7)):
            broken = table.clone()
            broken[0, spot] = bad
            out = w4.kv8_attention(q, cache, broken, *args, **how)
            assert w4.w4_device_status(clear=True) == 14

            def sees(b):
                s = mask.window_sees(300, 4, 100, 20) if "window" in how else mask.tree_sees(300, 4, [1, 3, 7, 15])
                s[:, 16 * spot:16 * spot + 16] = False
                return s

            want, tol = mask.attention(q, cache, table, lens, counts, sees, 64 ** -0.5, "bf16")
            assert ((out.double() - want).abs() <= tol).all()
    # one that no query sees is not looked at
    broken = table.clone()
    broken[0, 8] = 30
    w4.kv8_attention(q, cache, broken, *args, window=100, sinks=20)
    assert w4.w4_device_status() == 0


@pytest.mark.parametrize("batch,heads,kv_heads,window,tree", [
    (20, 16, 8, 1500, False), (20, 16, 8, 1500, True), (40, 8, 8, 2100, False), (33, 4, 2, 900, False)])
def test_many_windows_of_few_rows(w4, batch, heads, kv_heads, window, tree):
    """Items that a CTA has whole though they are long, and as many as are split again."""
    rng = np.random.default_rng(70)
    lens = [int(rng.integers(3, 4000)) for _ in range(batch)]
    counts = [int(rng.integers(1, 4)) for _ in range(batch)]
    trees = [mask.random_tree(m, rng, "tree") for m in counts] if tree else None
    pages = sum(-(-n // 64) for n in lens)
    cache = ref.random_cache(w4, pages, kv_heads, 64, 64, seed=71)
    table = ref.scattered_table(lens, 64, pages, seed=72)
    check(w4, queries(sum(counts), heads, 64, "fp16", 73), cache, table, lens, counts, "fp16", window, 4, trees)


@pytest.mark.parametrize("counts,lens,heads,kv_heads,dim,window,sinks,page,tree", [
    ([70], [3000], 4, 1, 128, 300, 4, 64, False), ([130, 33], [2500, 90], 2, 2, 64, 513, 0, 16, False),
    ([257], [2100], 4, 4, 128, 900, 40, 32, False), ([200, 300, 1], [2049, 300, 2000], 8, 2, 128, 1100, 1, 64, False),
    ([60], [5000], 8, 1, 64, 700, 9, 128, True), ([64, 40], [2300, 40], 8, 2, 128, 1500, 0, 64, True),
    ([150], [2700], 64, 32, 64, 1800, 5, 64, False)])
def test_prompts_with_short_windows_in_parts(w4, counts, lens, heads, kv_heads, dim, window, sinks, page, tree):
    """Items of a few steps that several CTAs share, two to eight of them, some without a token."""
    rng = np.random.default_rng(80)
    trees = [mask.random_tree(m, rng, "tree") for m in counts] if tree else None
    pages = sum(-(-n // page) for n in lens)
    cache = ref.random_cache(w4, pages, kv_heads, page, dim, seed=81)
    table = ref.scattered_table(lens, page, pages, seed=82)
    check(w4, queries(sum(counts), heads, dim, "bf16", 83), cache, table, lens, counts, "bf16", window, sinks, trees)


def mixed(batch, long, rng):
    """Mostly single tokens, some sequences without one, and few long ones."""
    counts = [int(rng.integers(0, 3)) for _ in range(batch)]
    for b, n in long.items():
        counts[b] = n
    return counts, [n + int(rng.integers(0, 700)) for n in counts]


@pytest.mark.parametrize("batch,long,heads,kv_heads,dim,window,sinks,spare", [
    (3, {1: 2000}, 2, 2, 128, 100, 4, 0), (40, {0: 600, 39: 257}, 8, 2, 128, 300, 0, 0),
    (33, {32: 900}, 4, 4, 64, 1000, 33, 7), (65, {2: 513, 40: 512, 64: 1}, 5, 1, 128, 64, 0, 0),
    (300, {7: 700, 250: 300}, 16, 2, 64, 50, 1, 90)])
def test_mixed_lengths(w4, batch, long, heads, kv_heads, dim, window, sinks, spare):
    """Blocks only for the rows that there are, and a graph replayed on other lengths."""
    rng = np.random.default_rng(90)
    counts, lens = mixed(batch, long, rng)
    lens = [max(n, 1) for n in lens]
    pages = sum(-(-n // 32) for n in lens)
    cache = ref.random_cache(w4, pages, kv_heads, 32, dim, seed=91)
    table = ref.scattered_table(lens, 32, pages, seed=92)
    q = queries(sum(counts) + spare, heads, dim, "bf16", 93).contiguous()
    check(w4, q, cache, table, lens, counts, "bf16", window, sinks)
    n, cu = ref.ints(lens), ref.bounds(counts)
    call = lambda: w4.kv8_attention(q, cache, table, n, cu, max(counts), max(lens), window=window,  # noqa: E731
                                    sinks=sinks, out=out)
    out = torch.zeros_like(q)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    turned = counts[::-1] if max(counts[::-1][b] - lens[b] for b in range(batch)) <= 0 else \
        [min(c, m) for c, m in zip(counts[::-1], lens)]
    cu.copy_(ref.bounds(turned))
    out.fill_(float("nan"))
    graph.replay()
    sees = lambda b: mask.window_sees(lens[b], turned[b], window, sinks)  # noqa: E731
    total = sum(turned)
    want, tol = mask.attention(q[:total], cache, table, lens, turned, sees, dim ** -0.5, "bf16")
    assert ((out[:total].double() - want).abs() <= tol).all()
    assert out[total:].isnan().all()
    assert w4.w4_device_status() == 0


def test_mixed_lengths_past_the_bounds(w4):
    """Too many queries give zeros; offsets that fall leave out their sequence, and those
    before it are done."""
    counts, lens = [1, 700, 2, 0, 40, 1] + [1] * 20, [300, 750, 90, 5, 400, 33] + [64] * 20
    pages = sum(-(-n // 32) for n in lens)
    cache = ref.random_cache(w4, pages, 2, 32, 128, seed=94)
    table = ref.scattered_table(lens, 32, pages, seed=95)
    q = queries(sum(counts), 8, 128, "fp16", 96)
    sees = lambda b: mask.window_sees(lens[b], counts[b], 90, 2)  # noqa: E731
    want, tol = mask.attention(q, cache, table, lens, counts, sees, 128 ** -0.5, "fp16")
    out = w4.kv8_attention(q, cache, table, ref.ints(lens), ref.bounds(counts), 699, 800, window=90, sinks=2)
    assert w4.w4_device_status(clear=True) == 14
    assert not out[1:701].any()
    rest = [0] + list(range(701, sum(counts)))
    assert ((out.double() - want).abs()[rest] <= tol[rest]).all()
    cu = ref.bounds(counts)
    cu[5] = 0  # of sequences 4 and 5: the one falls, the other has the rows of those before it
    out = torch.zeros_like(q)
    w4.kv8_attention(q, cache, table, ref.ints(lens), cu, 700, 800, out=out, window=90, sinks=2)
    assert w4.w4_device_status(clear=True) == 14
    assert ((out.double() - want).abs()[701:703] <= tol[701:703]).all()
