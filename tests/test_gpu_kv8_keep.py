"""Keeping the accepted drafts of a tree in the 8-bit cache, and shortening sequences,
against their definitions (exactly), and the operators around the cache together."""
import numpy as np
import pytest
import torch

import kv8mask as mask
import kv8util as ref
from test_gpu_kv8 import agrees, book_of, cache_state, queries, same, w4  # noqa: F401

pytestmark = pytest.mark.gpu


def keep(state, table, lens, counts, paths, page):
    """state: [k, v, k_scale, v_scale] float64 arrays, changed in place."""
    old = [x.copy() for x in state]
    for b, (n, m) in enumerate(zip(lens, counts)):
        base = n - m
        moves = [(base + i, base + d) for i, d in enumerate(paths[b]) if i != d]
        stays = [base + i for i, d in enumerate(paths[b]) if i == d]
        for col in sorted({to // page for to, _ in moves}):
            p = table[b][col]
            here = [(to, of) for to, of in moves if to // page == col]
            fixed = list(range(col * page, base)) + [j for j in stays if j // page == col]
            for i in (0, 1):
                for h in range(state[0].shape[1]):
                    now = max([old[2 + i][table[b][of // page], h] for _, of in here]
                              + [old[2 + i][p, h]] * bool(fixed))
                    for to, of in [(j, j) for j in fixed] + here:
                        source = table[b][of // page]
                        ratio = np.float32(old[2 + i][source, h]) / np.float32(now)
                        code = old[i][source, h, of % page]
                        x = (code.astype(np.float32) * ratio).astype(np.float64)
                        state[i][p, h, to % page] = code if ratio == 1 else np.where(
                            np.isnan(x), x, ref.round_e4m3(np.where(np.isnan(x), 0, x)))
                    state[2 + i][p, h] = now


def as_arrays(cache):
    return [x.double().cpu().numpy() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale)]


def packed(paths, counts):
    return ref.ints(sum((list(p) + [-1] * (m - len(p)) for p, m in zip(paths, counts)), []))


def random_paths(counts, rng):
    out = []
    for m in counts:
        k = int(rng.integers(0, m + 1)) if rng.random() < 0.7 else min(m, 2)
        out.append(sorted(rng.choice(m, k, replace=False).tolist()) if m else [])
    return out


def check(w4, page, dim, kv_heads, lens, counts, paths, seed, scales="pow2", slack=0):
    pages = sum(-(-n // page) for n in lens) + 3
    cache = ref.random_cache(w4, pages, kv_heads, page, dim, seed=seed, scales=scales)
    table = ref.scattered_table(lens, page, pages, seed=seed + 1)
    want = as_arrays(cache)
    keep(want, table.tolist(), lens, counts, paths, page)
    w4.kv8_keep(cache, table, ref.ints(lens), ref.bounds(counts), packed(paths, counts), max(counts) + slack)
    assert w4.w4_device_status() == 0
    for got, exact in zip(as_arrays(cache), want):
        assert np.array_equal(got, exact, equal_nan=True)
    return cache


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dim,kv_heads,scales", [(64, 3, "pow2"), (128, 2, "pow2"), (128, 1, "any")])
@pytest.mark.parametrize("seed", [1, 2, 3])
def test_against_the_definition(w4, page, dim, kv_heads, scales, seed):
    """With scales of any kind a code is off its definition only where fp32 and float64
    round the product to different sides of a tie: this compares with fp32's product."""
    rng = np.random.default_rng(seed)
    counts = [1, 0, 64, 2, 33, 17, 64, 5, 64, 40]
    lens = [m + int(rng.integers(0, 150)) for m in counts]
    lens[2], lens[1], lens[7] = 64, 0, 5  # nothing but drafts; an empty slot
    check(w4, page, dim, kv_heads, lens, counts, random_paths(counts, rng), 10 * seed, scales)


@pytest.mark.parametrize("page", [16, 64])
def test_particular_paths(w4, page):
    """All, none, a prefix, the last alone, every second, one that ends where a page ends."""
    counts = [20, 20, 20, 20, 64, 64, 16, 1]
    paths = [list(range(20)), [], [0, 1, 2], [19], list(range(0, 64, 2)), list(range(1, 33)), [0, 15], [0]]
    lens = [100, 37, 20, 64, 64 + 7, 64 + 25, 16, 1]
    cache = check(w4, page, 128, 2, lens, counts, paths, 40, slack=0)
    before = cache_state(cache)
    # what moves nothing changes nothing
    table = ref.scattered_table([100, 37], page, 20, seed=41)
    w4.kv8_keep(cache, table, ref.ints([100, 37]), ref.bounds([20, 20]), packed([range(20), []], [20, 20]), 64)
    assert same(cache_state(cache), before)


def test_loud_and_quiet_pages(w4):
    """Codes below the new scale's range are rounded, and to zero; NaN codes move as NaN."""
    page, lens, counts = 16, [40, 50], [30, 20]
    cache = ref.random_cache(w4, 12, 2, page, 64, seed=42)
    table = ref.scattered_table(lens, page, 12, seed=43)
    for sc in (cache.k_scale, cache.v_scale):
        sc.copy_(torch.exp2(-torch.arange(24, dtype=torch.float32, device="cuda").view(12, 2) * 0.75).exp2().log2())
    cache.k.view(torch.uint8)[table[0, 2].long(), 1, 3, 5] = 0x7F
    cache.v.view(torch.uint8)[table[1, 3].long(), 0, 1, 7] = 0xFF
    paths = [[2, 9, 25], [0, 7, 19]]
    want = as_arrays(cache)
    keep(want, table.tolist(), lens, counts, paths, page)
    w4.kv8_keep(cache, table, ref.ints(lens), ref.bounds(counts), packed(paths, counts), 30)
    for got, exact in zip(as_arrays(cache), want):
        assert np.array_equal(got, exact, equal_nan=True)
    assert np.isnan(want[0]).sum() == 2 and np.isnan(want[1]).sum() >= 1


@pytest.mark.parametrize("row", [[0, 0, -1, -1, -1], [1, 0, -1, -1, -1], [0, 2, 2, -1, -1], [5, -1, -1, -1, -1],
                                 [0, -1, 2, -1, -1], [-1, 0, -1, -1, -1], [0, 1, 2, 3, 2 ** 31 - 1]])
def test_what_is_no_path_is_left_alone(w4, row):
    page, lens, counts = 16, [40, 33, 50], [7, 5, 6]
    cache = ref.random_cache(w4, 12, 2, page, 64, seed=44)
    table = ref.scattered_table(lens, page, 12, seed=45)
    want = as_arrays(cache)
    keep(want, table.tolist(), lens, counts, [[0, 6], [], [1]], page)
    path = ref.ints([0, 6, -1, -1, -1, -1, -1] + row + [1, -1, -2, -2 ** 31, -1, -1])
    w4.kv8_keep(cache, table, ref.ints(lens), ref.bounds(counts), path, 7)
    assert w4.w4_device_status(clear=True) == 14
    for got, exact in zip(as_arrays(cache), want):
        assert np.array_equal(got, exact)


@pytest.mark.parametrize("how", ["page", "length", "many", "offsets", "short"])
def test_bad_sequences_are_left_alone(w4, how):
    page, lens, counts = 16, [40, 33, 50], [7, 5, 6]
    cache = ref.random_cache(w4, 12, 2, page, 64, seed=46)
    table = ref.scattered_table(lens, page, 12, seed=47)
    n, cu = ref.ints(lens), ref.bounds(counts)
    paths = [[0, 6], [2, 4], [1]]
    want, alone = as_arrays(cache), 1
    most = 7
    if how == "page":
        table[1, 1] = 12  # (drafts 28 to 32, of pages 1 and 2)
    elif how == "length":
        n[1] = 16 * table.shape[1] + 1
    elif how == "short":
        n[1] = 4
    elif how == "many":
        most, alone = 6, 0
    else:
        cu[1], alone = 19, None
    rows = table.tolist()
    good = [p if b != alone else [] for b, p in enumerate(paths)]
    if alone is None:  # sequences 0 and 1 have no rows of their own
        good[0], good[1] = [], []
    keep(want, rows, lens, counts, good, page)
    w4.kv8_keep(cache, table, n, cu, packed(paths, counts), most)
    assert w4.w4_device_status(clear=True) == 14
    for got, exact in zip(as_arrays(cache), want):
        assert np.array_equal(got, exact)


# --------------------------------------------------------------------------- #
# shorten                                                                       #
# --------------------------------------------------------------------------- #
def shorten(book, drop):
    for s, d in enumerate(drop):
        for j in range(book.pages(book.lens[s] - d), book.pages(book.lens[s])):
            book.refs[book.table[s][j]] -= 1
            book.table[s][j] = -1
        book.lens[s] -= d


@pytest.mark.parametrize("seqs,most", [(1, 50), (5, 64), (33, 200), (700, 90), (2500, 40)])
@pytest.mark.parametrize("page", [16, 64])
def test_shorten(w4, seqs, most, page):
    rng = np.random.default_rng(seqs)
    new = [int(rng.integers(0, most + 1)) for _ in range(seqs)]
    pool = w4.kv8_pool(sum(-(-n // page) for n in new) + 2, seqs, most, page)
    w4.kv8_reserve(pool, ref.ints(new))
    book = book_of(pool)
    for step in range(3):
        drop = [int(rng.choice([0, min(1, n), n, int(rng.integers(0, n + 1))])) for n in book.lens]
        w4.kv8_shorten(pool, ref.ints(drop))
        shorten(book, drop)
        assert int(pool.status) == 0 and agrees(pool, book)
    assert w4.w4_device_status() == 0


def test_a_long_sequence_is_shortened_by_many_pages(w4):
    pool = w4.kv8_pool(70000, 3, 16 * 65000, 16)
    w4.kv8_reserve(pool, ref.ints([100, 16 * 65000 - 3, 777]))
    book = book_of(pool)
    drop = [0, 16 * 64000, 776]
    w4.kv8_shorten(pool, ref.ints(drop))
    shorten(book, drop)
    assert int(pool.status) == 0 and agrees(pool, book)


def test_shared_pages_stay_with_the_other(w4):
    """A fork's child that is shortened into what it shares, and its parent then."""
    pool = w4.kv8_pool(20, 3, 64, 16)
    w4.kv8_reserve(pool, ref.ints([50, 0, 0]))
    w4.kv8_fork(pool, ref.ints([0, 0]), ref.ints([1, 2]))
    book = book_of(pool)
    for drop in ([0, 30, 0], [50, 0, 2], [0, 20, 48]):
        w4.kv8_shorten(pool, ref.ints(drop))
        shorten(book, drop)
        assert int(pool.status) == 0 and agrees(pool, book)
    assert not any(book.refs)


@pytest.mark.parametrize("drop,change", [
    ([0, 21, 0], None), ([0, -1, 5], None), ([0, 2 ** 31 - 1, 5], None), ([-2 ** 31, 0, 5], None), ([9, 20, 5], "page"),
    ([9, 20, 5], "free"), ([9, 20, 5], "long"), ([9, 20, 5], "negative")])
def test_a_failed_shorten_changes_nothing(w4, drop, change):
    pool = w4.kv8_pool(20, 3, 64, 16)
    w4.kv8_reserve(pool, ref.ints([40, 20, 33]))
    if change == "page":
        pool.table[1, 1] = 20
    elif change == "free":
        pool.refs[pool.table[1, 0].long()] = 0
    elif change == "long":
        pool.lens[1] = 65
    elif change == "negative":
        pool.lens[1] = -5
    book = book_of(pool)
    w4.kv8_shorten(pool, ref.ints(drop))
    assert int(pool.status) == 14 and agrees(pool, book)
    bare = w4.KV8Pool(pool.refs, pool.table, pool.lens, 16)  # without a status of its own
    w4.kv8_shorten(bare, ref.ints(drop))
    assert w4.w4_device_status(clear=True) == 14 and agrees(pool, book)


def test_a_page_named_too_often_stays_free(w4):
    pool = w4.kv8_pool(20, 2, 64, 16)
    w4.kv8_reserve(pool, ref.ints([20, 20]))
    pool.table[1, 1] = pool.table[0, 1]
    pool.refs[3] = 0
    w4.kv8_shorten(pool, ref.ints([10, 10]))
    assert int(pool.status) == 14 and pool.refs[:4].tolist() == [1, 0, 1, 0]


# --------------------------------------------------------------------------- #
# together                                                                      #
# --------------------------------------------------------------------------- #
class Layer:
    """What a layer has of keys: a norm's weights and the rotations. Every key and value
    has one element of the same size, so that every page has the same scale."""

    def __init__(self, w4, heads, kv_heads, dim, dtype, seed, window):
        self.w4, self.heads, self.kv_heads, self.dim, self.window = w4, heads, kv_heads, dim, window
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.weights = [1 + 0.2 * torch.randn(dim, device="cuda", generator=g) for _ in range(2)]
        self.table = w4.rope_table(4096, dim // 2)
        self.weights[1][-1] = 30.0
        self.dtype = dtype

    def step(self, pool, cache, qkv, positions, cu, m, most, tree=None):
        q, k, v = qkv.split((self.heads, self.kv_heads, self.kv_heads), 1)
        how = dict(window=self.window, sinks=2) if self.window else {}
        q, k = self.w4.qk_norm_rope(q, k, positions, self.table, *self.weights)
        self.w4.kv8_append(k, v, cache, pool.table, pool.lens, cu, m)
        return self.w4.kv8_attention(q, cache, pool.table, pool.lens, cu, m, most, tree=tree, **how)


def projection(tokens, heads, kv_heads, dim, dtype, seed):
    x = queries(tokens, heads + 2 * kv_heads, dim, dtype, seed)
    x[:, heads:, -1] = 3.0  # keys' last element is the loudest after the norm, values' too
    x[:, heads + kv_heads:, :-1] *= 0.1
    return x


@pytest.mark.parametrize("window", [None, 48])
@pytest.mark.parametrize("heads,kv_heads,dim,dtype,page", [
    (8, 2, 64, "bf16", 16), (32, 2, 128, "fp16", 64), (4, 4, 128, "bf16", 32)])
@pytest.mark.parametrize("graph", [False, True])
def test_a_tree_is_its_branches(w4, heads, kv_heads, dim, dtype, page, window, graph):
    """Two sequences read prompts, then a tree of drafts each; one branch is kept. The
    same branch read in order, one token a step, gives the same cache, the same
    lengths, pages and counts, and attention within both calls' tolerances."""
    prompt, counts, most = [70, 131], [9, 21], 200
    rng = np.random.default_rng(5)
    trees = [mask.random_tree(m, rng, "tree") for m in counts]
    paths = [[d for d in range(m) if max(t, key=lambda w: bin(w).count("1")) >> d & 1]
             for m, t in zip(counts, trees)]
    layer = Layer(w4, heads, kv_heads, dim, dtype, 6, window)
    first = projection(sum(prompt), heads, kv_heads, dim, dtype, 7)
    drafts = projection(sum(counts), heads, kv_heads, dim, dtype, 8)

    def start():
        pool = w4.kv8_pool(40, 2, most, page)
        cache = w4.kv8_cache(40, kv_heads, page, dim)
        w4.kv8_reserve(pool, ref.ints(prompt))
        pos = ref.ints(list(range(prompt[0])) + list(range(prompt[1])))
        layer.step(pool, cache, first, pos, ref.bounds(prompt), max(prompt), most)
        return pool, cache

    # the tree
    pool, cache = start()
    depth = [bin(w).count("1") - 1 for t in trees for w in t]
    pos = ref.ints([prompt[i >= counts[0]] + d for i, d in enumerate(depth)])
    cu, words, path = ref.bounds(counts), mask.words_tensor(sum(trees, [])), packed(paths, counts)
    more, drop = ref.ints(counts), ref.ints([m - len(p) for m, p in zip(counts, paths)])

    def verify():
        w4.kv8_reserve(pool, more)
        out = layer.step(pool, cache, drafts, pos, cu, max(counts), most, words)
        w4.kv8_keep(cache, pool.table, pool.lens, cu, path, max(counts))
        w4.kv8_shorten(pool, drop)
        return out

    if graph:
        parts = [x.view(torch.uint8) for x in (pool.refs, pool.table, pool.lens, cache.k, cache.v, cache.k_scale,
                                               cache.v_scale)]
        state = [x.clone() for x in parts]
        verify()  # (warms up; what it changed is put back)
        for x, y in zip(parts, state):
            x.copy_(y)
        torch.cuda.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            got = verify()
        captured.replay()
    else:
        got = verify()
    assert int(pool.status) == 0 and w4.w4_device_status() == 0

    # the branch
    other, plain = start()
    at = [0, counts[0]]
    for step in range(max(map(len, paths))):
        live = [b for b in (0, 1) if step < len(paths[b])]
        rows = [at[b] + paths[b][step] for b in live]
        new = [int(b in live) for b in (0, 1)]
        w4.kv8_reserve(other, ref.ints(new))
        out = layer.step(other, plain, drafts[rows], ref.ints([prompt[b] + step for b in live]),
                         ref.bounds(new), 1, most)
        err = (out.float() - got[rows].float()).abs().max()
        # roundings of the outputs (half an ulp each), of P (2^-10 each) and of the scores
        assert err <= (2 * ref.UNIT[dtype] + 2.0 ** -8) * got.float().abs().max()
    assert pool.lens.tolist() == other.lens.tolist() == [n + len(p) for n, p in zip(prompt, paths)]
    for b, n in enumerate(pool.lens.tolist()):
        for j in range(n):
            p, o = (x.table[b, j // page].long() for x in (pool, other))
            for mine, its in ((cache.k, plain.k), (cache.v, plain.v)):
                assert torch.equal(mine[p, :, j % page].view(torch.uint8), its[o, :, j % page].view(torch.uint8))
            assert torch.equal(cache.k_scale[p], plain.k_scale[o]) and torch.equal(cache.v_scale[p], plain.v_scale[o])
    held = sum(-(-n // page) for n in pool.lens.tolist())
    assert int((pool.refs > 0).sum()) == held and bool((pool.refs <= 1).all())


def test_a_fork_after_shortening_into_a_shared_page(w4):
    """The page is still the other's: the fork copies it, and new tokens go to the copy."""
    page, dim = 16, 64
    pool, cache = w4.kv8_pool(20, 3, 64, page), w4.kv8_cache(20, 1, page, dim)
    w4.kv8_reserve(pool, ref.ints([40, 0, 0]))
    x = queries(40, 1, dim, "bf16", 9)
    w4.kv8_append(x, x, cache, pool.table, pool.lens, ref.bounds([40, 0, 0]), 40)
    w4.kv8_copy_pages(cache, *w4.kv8_fork(pool, ref.ints([0]), ref.ints([1])))
    w4.kv8_shorten(pool, ref.ints([0, 20, 0]))  # 20 tokens: the second page is the parent's too
    before = [y[pool.table[0, :3].long()].clone() for y in cache_state_tensors(cache)]
    moves = w4.kv8_fork(pool, ref.ints([1]), ref.ints([2]))
    w4.kv8_copy_pages(cache, *moves)
    assert moves[0].tolist() == [int(pool.table[0, 1])] and int(pool.table[2, 1]) == int(moves[1])
    w4.kv8_reserve(pool, ref.ints([0, 0, 5]))
    y = queries(5, 1, dim, "bf16", 10)
    w4.kv8_append(y, y, cache, pool.table, pool.lens, ref.bounds([0, 0, 5]), 5)
    assert int(pool.status) == 0
    for now, was in zip(cache_state_tensors(cache), before):
        assert torch.equal(now[pool.table[0, :3].long()], was)


def cache_state_tensors(cache):
    return [cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale, cache.v_scale]


def test_keep_on_pages_past_32_bits(w4):
    page, pages, lens, counts, paths = 128, 40000, [300, 131], [60, 9], [list(range(5, 60, 3)), [0, 8]]
    cache = w4.kv8_cache(pages, 8, page, 128)  # 5.2 GB a side
    small = ref.random_cache(w4, 6, 8, page, 128, seed=50)
    near = ref.scattered_table(lens, page, 6, seed=51)
    for big, little in ((cache.k, small.k), (cache.v, small.v)):
        big.view(torch.uint8)[-6:].copy_(little.view(torch.uint8))
    cache.k_scale[-6:], cache.v_scale[-6:] = small.k_scale, small.v_scale
    far = torch.where(near >= 0, near + pages - 6, -1).to(torch.int32)
    for c, t in ((cache, far), (small, near)):
        w4.kv8_keep(c, t, ref.ints(lens), ref.bounds(counts), packed(paths, counts), 64)
    assert w4.w4_device_status() == 0
    for big, little in zip(cache_state_tensors(cache), cache_state_tensors(small)):
        assert torch.equal(big[-6:], little) and not (big[:-6] if big.dim() == 4 else big[:-6] - 1).any()


def test_many_sequences_are_shortened(w4):
    seqs = 50000
    pool = w4.kv8_pool(2 * seqs, seqs, 32, 16)
    w4.kv8_reserve(pool, torch.full((seqs,), 20, dtype=torch.int32, device="cuda"))
    drop = torch.arange(seqs, dtype=torch.int32, device="cuda") % 3 * 10
    w4.kv8_shorten(pool, drop)
    assert int(pool.status) == 0 and torch.equal(pool.lens, 20 - drop)
    held = (pool.lens + 15) // 16
    assert torch.equal((pool.table >= 0).sum(1).int(), held) and int(pool.refs.sum()) == int(held.sum())
    assert bool((pool.refs[pool.table[pool.table >= 0].long()] == 1).all())
    drop[seqs - 1] = 21  # one that cannot be: nothing happens to any
    before = [x.clone() for x in (pool.refs, pool.table, pool.lens)]
    w4.kv8_shorten(pool, drop)
    assert int(pool.status) == 14
    assert all(torch.equal(x, y) for x, y in zip(before, (pool.refs, pool.table, pool.lens)))
