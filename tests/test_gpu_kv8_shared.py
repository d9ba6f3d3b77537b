"""Sequences that end within a page which others hold too: they do not grow there."""
import numpy as np
import pytest
import torch

import kv8util as ref
from test_gpu_kv8 import agrees, book_of, queries, w4  # noqa: F401
from test_gpu_kv8_keep import cache_state_tensors

SHARED = 18


def test_the_error_has_a_name():
    import int4_weight_only_repack_gb300 as lib
    from libutil import ensure_built
    ensure_built()
    assert "W4_ERR_SHARED" in lib.w4_status_string(SHARED)


@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("who", [0, 1])
def test_a_sequence_does_not_grow_in_a_shared_page(w4, page, who):
    """A fork's child shortened into what it shares, or its parent: a common prefix, or a
    conversation that goes back. All or nothing: the call changes no other sequence either."""
    pool = w4.kv8_pool(40, 4, 8 * page, page)
    w4.kv8_reserve(pool, ref.ints([3 * page, 0, 7, 0]))
    w4.kv8_fork(pool, ref.ints([0]), ref.ints([1]))
    drop = [0] * 4
    drop[who] = page + 3
    w4.kv8_shorten(pool, ref.ints(drop))
    book = book_of(pool)
    for more in (1, page, 3):
        add = [0, 0, 5, page]
        add[who] = more
        w4.kv8_reserve(pool, ref.ints(add))
        assert int(pool.status) == SHARED and agrees(pool, book)
    bare = w4.KV8Pool(pool.refs, pool.table, pool.lens, page)  # without a status of its own
    w4.kv8_reserve(bare, ref.ints(add))
    assert w4.w4_device_status(clear=True) == SHARED and agrees(pool, book)
    # the other grows, and so do all while this one stays
    add = [4, 4, 9, 2 * page + 1]
    add[who] = 0
    w4.kv8_reserve(pool, ref.ints(add))
    assert int(pool.status) == 0
    # once the other has let the page go
    w4.kv8_free(pool, ref.ints([1 - who]))
    add = [0] * 4
    add[who] = 5
    w4.kv8_reserve(pool, ref.ints(add))
    assert int(pool.status) == 0 and int(pool.lens[who]) == 2 * page - 3 + 5


@pytest.mark.gpu
def test_a_shared_page_that_is_full_is_no_hindrance(w4):
    """Nor is a partial one that gets nothing, or that a fork has copied."""
    page = 16
    pool = w4.kv8_pool(40, 3, 128, page)
    w4.kv8_reserve(pool, ref.ints([48, 0, 0]))
    w4.kv8_fork(pool, ref.ints([0]), ref.ints([1]))
    w4.kv8_shorten(pool, ref.ints([0, 16, 0]))
    w4.kv8_reserve(pool, ref.ints([1, 1, 0]))
    assert int(pool.status) == 0 and pool.refs[:5].tolist() == [2, 2, 1, 1, 1]
    w4.kv8_shorten(pool, ref.ints([0, 10, 0]))  # 23 tokens: into the second page
    w4.kv8_reserve(pool, ref.ints([3, 0, 0]))
    assert int(pool.status) == 0
    w4.kv8_fork(pool, ref.ints([1]), ref.ints([2]))
    w4.kv8_reserve(pool, ref.ints([0, 0, 40]))
    assert int(pool.status) == 0 and pool.lens.tolist() == [52, 23, 63]


@pytest.mark.gpu
@pytest.mark.parametrize("graph", [False, True])
def test_the_other_sequence_keeps_its_tokens(w4, graph):
    """The whole way: fork, shorten, reserve, append. What the parent reads stays the same."""
    page, dim = 16, 64
    pool, cache = w4.kv8_pool(20, 2, 64, page), w4.kv8_cache(20, 1, page, dim)
    w4.kv8_reserve(pool, ref.ints([40, 0]))
    x = queries(40, 1, dim, "bf16", 9)
    w4.kv8_append(x, x, cache, pool.table, pool.lens, ref.bounds([40, 0]), 40)
    w4.kv8_copy_pages(cache, *w4.kv8_fork(pool, ref.ints([0]), ref.ints([1])))
    w4.kv8_shorten(pool, ref.ints([0, 20]))
    before = [y[pool.table[0, :3].long()].clone() for y in cache_state_tensors(cache)]
    more = ref.ints([0, 5])
    if graph:
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            w4.kv8_reserve(pool, more)
        captured.replay()
    else:
        w4.kv8_reserve(pool, more)
    if int(pool.status) == 0:
        y = queries(5, 1, dim, "bf16", 10) * 100
        w4.kv8_append(y, y, cache, pool.table, pool.lens, ref.bounds([0, 5]), 5)
    for now, was in zip(cache_state_tensors(cache), before):
        assert torch.equal(now[pool.table[0, :3].long()], was)
    assert int(pool.status) == SHARED and pool.lens.tolist() == [40, 20]


@pytest.mark.gpu
@pytest.mark.parametrize("seqs", [40, 1500])
def test_one_among_many(w4, seqs):
    """Whichever thread has it: the call is refused, and does what it says without it."""
    page = 16
    rng = np.random.default_rng(seqs)
    lens = [int(rng.integers(1, 60)) for _ in range(seqs)] + [0]
    pool = w4.kv8_pool(5 * seqs + 40, seqs + 1, 96, page)
    w4.kv8_reserve(pool, ref.ints(lens))
    for who in (0, seqs // 2, seqs - 1):
        if lens[who] < 20:
            w4.kv8_reserve(pool, ref.ints([20 * (s == who) for s in range(seqs)] + [0]))
        w4.kv8_fork(pool, ref.ints([who]), ref.ints([seqs]))
        n = int(pool.lens[who])
        w4.kv8_shorten(pool, ref.ints([0] * seqs + [n - 9]))
        book = book_of(pool)
        w4.kv8_reserve(pool, ref.ints([int(rng.integers(0, 3)) for _ in range(seqs)] + [1]))
        assert int(pool.status) == SHARED and agrees(pool, book)
        w4.kv8_reserve(pool, ref.ints([0] * (seqs + 1)))
        assert int(pool.status) == 0 and agrees(pool, book)
        w4.kv8_free(pool, ref.ints([seqs]))


@pytest.mark.gpu
def test_a_bad_page_number_is_not_followed(w4):
    """Neither below zero nor past the pool; a wrong length is still the length's error."""
    pool = w4.kv8_pool(20, 3, 64, 16)
    w4.kv8_reserve(pool, ref.ints([20, 20, 20]))
    for bad in (-1, -2 ** 31, 20, 2 ** 31 - 1):
        pool.table[1, 1] = bad
        w4.kv8_reserve(pool, ref.ints([0, 1, 0]))
        assert int(pool.status) == 0
    w4.kv8_reserve(pool, ref.ints([0, 0, 1000]))
    assert int(pool.status) == 14
