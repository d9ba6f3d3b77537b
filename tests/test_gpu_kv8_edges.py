"""The 8-bit key-value cache's operators where they can go wrong: calls that fail
half-way, sequences past a bound, chained forks, one token with nearly all of the
weight, loud pages beside quiet ones."""
import math
import threading

import numpy as np
import pytest
import torch

import kv8util as ref
from test_gpu_kv8 import agrees, book_of, cache_state, check, queries, same, w4  # noqa: F401

pytestmark = pytest.mark.gpu


# --------------------------------------------------------------------------- #
# pages                                                                         #
# --------------------------------------------------------------------------- #
def raw_fork(w4, pool, src, dst, copy_src, copy_dst):
    """The C call, with lists of the caller's."""
    ws = torch.empty(w4.w4_kv8_pages_workspace_size(pool.refs.shape[0], len(src)), dtype=torch.uint8,
                     device="cuda")
    a, b = ref.ints(src), ref.ints(dst)
    status = w4.lib().w4_kv8_fork(
        pool.refs.data_ptr(), pool.refs.shape[0], pool.table.data_ptr(), pool.table.shape[1],
        pool.lens.data_ptr(), pool.lens.shape[0], a.data_ptr(), b.data_ptr(), len(src),
        pool.page_size, copy_src.data_ptr(), copy_dst.data_ptr(), pool.status.data_ptr(),
        ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert status == 0
    torch.cuda.synchronize()


@pytest.mark.parametrize("src,dst,status", [
    ([0, 1, 0], [3, 4, 5], 15),          # three partial pages, two free ones
    ([0, 1], [3, 3], 16), ([0, 1], [3, 1], 16), ([0, 9], [3, 4], 16)])
def test_a_failed_fork_copies_nothing(w4, src, dst, status):
    """Its lists name no page, whatever they held: copying by them is a no-op."""
    pool = w4.kv8_pool(7, 6, 64, 16)
    cache = ref.random_cache(w4, 7, 2, 16, 64, seed=1)
    w4.kv8_reserve(pool, ref.ints([40, 20, 0, 0, 0, 0]))
    book, before = book_of(pool), cache_state(cache)
    stale = [ref.ints([0, 1, 2][:len(src)]), ref.ints([4, 3, 5][:len(src)])]
    raw_fork(w4, pool, src, dst, *stale)
    assert int(pool.status) == status and agrees(pool, book)
    w4.kv8_copy_pages(cache, *stale)
    assert same(cache_state(cache), before)
    assert all((x == -1).all() for x in stale)
    assert w4.w4_device_status() == 0


@pytest.mark.parametrize("tokens", [32, 37])
def test_forks_in_a_chain(w4, tokens):
    """Pairs take effect in order: a target may be a later pair's source."""
    pool = w4.kv8_pool(20, 7, 64, 16)
    cache = ref.random_cache(w4, 20, 2, 16, 64, seed=2)
    w4.kv8_reserve(pool, ref.ints([0, tokens, 5, 0, 0, 0, 0]))
    # 3 and 4 through 0, before 0's own pair nothing: 5 stays empty, and so does 6
    src, dst = [3, 1, 0, 4, 6], [5, 0, 4, 3, 6]
    moves = w4.kv8_fork(pool, ref.ints(src), ref.ints(dst))
    assert int(pool.status) == 0
    w4.kv8_copy_pages(cache, *moves)
    assert pool.lens.tolist() == [tokens, tokens, 5, tokens, tokens, 0, 0]
    full, part = divmod(tokens, 16)
    table = pool.table.tolist()
    want = [1] * full + [-1] * (4 - full)
    for s in (0, 3, 4):
        assert table[s][:full] == table[1][:full] and table[s][full + (part > 0):] == [-1] * (4 - full - (part > 0))
    assert table[5] == table[6] == [-1] * 4
    refs = [0] * 20
    for row in table:
        for p in row:
            if p >= 0:
                refs[p] += 1
    assert pool.refs.tolist() == refs and [refs[p] for p in table[1][:full]] == [4] * full
    if part:
        last = [table[s][full] for s in (1, 2 - 2, 3, 4)]
        assert len(set(last)) == 4 and all(refs[p] == 1 for p in last)
        for p in last[1:]:
            assert torch.equal(cache.k[p, :, :part].view(torch.uint8), cache.k[last[0], :, :part].view(torch.uint8))
            assert torch.equal(cache.v_scale[p], cache.v_scale[last[0]])


def fork_in_order(book, src, dst):
    """Pair by pair. Returns the moves; a chain's copies all read its first page."""
    first, moves = {}, []
    for s, d in zip(src, dst):
        full, part = divmod(book.lens[s], book.page)
        row, move = book.table[s][:full], (-1, -1)
        if part:
            move = (first.get(s, book.table[s][full]), book.lowest(1)[0])
            row.append(move[1])
            first[d] = move[0]
        for p in row:
            book.refs[p] += 1
        book.table[d], book.lens[d] = row + [-1] * (len(book.table[d]) - len(row)), book.lens[s]
        moves.append(move)
    return moves


@pytest.mark.parametrize("seqs", [40, 700])
def test_random_chains_of_forks(w4, seqs):
    rng = np.random.default_rng(seqs)
    pool = w4.kv8_pool(12 * seqs, seqs, 160, 16)
    new = [int(rng.integers(1, 161)) if s < seqs // 5 else 0 for s in range(seqs)]
    w4.kv8_reserve(pool, ref.ints(new))
    book = book_of(pool)
    dst = (rng.permutation(seqs - seqs // 5)[:seqs // 2] + seqs // 5).tolist()
    src = [int(rng.choice(dst[:i + 1] if rng.random() < 0.8 else range(seqs))) for i in range(len(dst))]
    a, b = w4.kv8_fork(pool, ref.ints(src), ref.ints(dst))
    moves = fork_in_order(book, src, dst)
    assert int(pool.status) == 0 and agrees(pool, book)
    assert list(zip(a.tolist(), b.tolist())) == moves


def test_a_fork_from_a_length_below_zero(w4):
    pool = w4.kv8_pool(10, 4, 64, 16)
    w4.kv8_reserve(pool, ref.ints([40, 0, 0, 0]))
    for bad in (-1, -2, -3, -2 ** 31):
        pool.lens[0] = bad
        book = book_of(pool)
        w4.kv8_fork(pool, ref.ints([0, 3]), ref.ints([2, 1]))
        assert int(pool.status) == 14 and agrees(pool, book)
        w4.kv8_fork(pool, ref.ints([3, 1]), ref.ints([0, 2]))  # nor is it an empty target
        assert int(pool.status) == 16 and agrees(pool, book)


@pytest.mark.parametrize("seqs,each", [(1 << 20, 2049), (1 << 20, 4097)])
def test_needs_past_32_bits(w4, seqs, each):
    """A million sequences that ask for 2^31 pages and more, or 2^32, are refused."""
    table = torch.empty((seqs, each), dtype=torch.int32, device="cuda")
    pool = w4.KV8Pool(ref.ints([0] * 1000), table, torch.zeros(seqs, dtype=torch.int32, device="cuda"), 16,
                      ref.ints([0]))
    table[5, :3] = 77
    new = torch.full((seqs,), 16 * each, dtype=torch.int32, device="cuda")
    w4.kv8_reserve(pool, new)
    assert int(pool.status) == 15 and not pool.refs.any() and not pool.lens.any()
    new.zero_()
    new[5] = 40
    w4.kv8_reserve(pool, new)
    assert int(pool.status) == 0 and pool.refs[:4].tolist() == [1, 1, 1, 0]
    assert table[5, :3].tolist() == [0, 1, 2] and int(pool.lens[5]) == 40


def test_lengths_past_32_bits(w4):
    table = torch.empty((1, 1 << 27), dtype=torch.int32, device="cuda")
    pool = w4.KV8Pool(ref.ints([0] * 1000), table, ref.ints([2 ** 30]), 16, ref.ints([0]))
    for new in (1, 2 ** 30, 2 ** 31 - 1):  # (the sums are 2^30 and up to 2^31 + 2^30)
        w4.kv8_reserve(pool, ref.ints([new]))
        assert int(pool.status) == 14 and int(pool.lens) == 2 ** 30 and not pool.refs.any()


def test_a_sequence_of_a_bad_length_is_left_alone_by_free(w4):
    pool = w4.kv8_pool(10, 3, 64, 16)
    w4.kv8_reserve(pool, ref.ints([40, 20, 0]))
    for bad in (65, -3):
        pool.lens[0] = bad
        book = book_of(pool)
        w4.kv8_free(pool, ref.ints([0]))
        assert int(pool.status) == 14 and agrees(pool, book)


# --------------------------------------------------------------------------- #
# attention                                                                     #
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("heads,kv_heads,max_q,max_kv", [
    (4, 2, 1, 200), (4, 2, 1, 3000), (16, 2, 3, 200), (16, 2, 3, 3000),  # few rows: items, runs
    (4, 1, 33, 200), (4, 1, 33, 3000)])                                  # many: tiles, split tiles
def test_more_new_tokens_than_the_bound_give_zeros(w4, heads, kv_heads, max_q, max_kv):
    lens, counts = [100, 200, 150], [1, 300, max_q]
    cache = ref.random_cache(w4, 20, kv_heads, 32, 64, seed=3)
    table = ref.scattered_table(lens, 32, 20, seed=4)
    q = queries(sum(counts), heads, 64, "bf16", 5)
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    w4.kv8_attention(q, cache, table, ref.ints(lens), ref.bounds(counts), max_q, max_kv, out=out)
    assert w4.w4_device_status(clear=True) == 14
    assert torch.count_nonzero(out[1:301]) == 0
    want, tol = ref.attention(q, cache, table, [100, 0, 150], counts, 64 ** -0.5, True, "bf16")
    keep = [0] + list(range(301, sum(counts)))
    assert ((out.double() - want).abs()[keep] <= tol[keep]).all()


@pytest.mark.parametrize("m", [1, 100])
def test_columns_of_a_wider_table(w4, m):
    """A row ends where its columns end, whatever lies beside them."""
    lens, page = [130, 60, 200], 16
    cache = ref.random_cache(w4, 40, 2, page, 64, seed=14)
    table = ref.scattered_table(lens, page, 40, seed=15)
    wide = ref.ints([[0] * 30] * 3)
    part = wide[:, 30 - table.shape[1]:]  # the last row's end is the buffer's
    part.copy_(table)
    q = queries(3 * m, 4, 64, "bf16", 16)
    check(w4, q, cache, part, lens, [m] * 3, True, "bf16")
    side = torch.cuda.Stream()
    args = ref.ints([130, 60, 209]), ref.bounds([m] * 3), m, 1000
    for stream in (None, side, side.cuda_stream):
        out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
        side.wait_stream(torch.cuda.current_stream())
        w4.kv8_attention(q, cache, part, *args, out=out, stream=stream)
        torch.cuda.synchronize()
        assert w4.w4_device_status(clear=True) == 14  # one token past the columns
        assert torch.count_nonzero(out[2 * m:]) == 0 and torch.count_nonzero(out[:m]) > 0
    if m == 1:
        k = queries(3, 2, 64, "bf16", 17)
        before = cache_state(cache)
        w4.kv8_append(k, k, cache, part, ref.ints([0, 0, 209]), ref.ints([0, 0, 0, 1]), 1)
        assert w4.w4_device_status(clear=True) == 14 and same(cache_state(cache), before)
        w4.kv8_append(k, k, cache, part, ref.ints([0, 0, 200]), ref.ints([0, 0, 0, 1]), 1)
        assert w4.w4_device_status() == 0 and not same(cache_state(cache), before)


@pytest.mark.parametrize("m,n", [(1, 3000), (50, 2900)])
def test_a_graph_outlives_the_growth_of_its_workspace(w4, m, n):
    """A captured split call, then a call on the same stream that needs more: the
    graph's workspace is not given to anyone else."""
    page, dim = 64, 128
    cache = ref.random_cache(w4, 600, 1, page, dim, seed=18)
    table = ref.scattered_table([n, 20000], page, 600, seed=19)
    q = queries(m, 8, dim, "bf16", 20)
    small = (cache, table[:1], ref.ints([n]), ref.bounds([m]), m, n)
    big_m = 300
    big = (cache, table[1:], ref.ints([20000]), ref.bounds([big_m]), big_m, 20000)
    size = w4.w4_kv8_attention_workspace_size(1, m, m, n, 8, 1, dim)
    more = w4.w4_kv8_attention_workspace_size(1, big_m, big_m, 20000, 8, 1, dim)
    assert 0 < size < more
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph, big_q = torch.cuda.CUDAGraph(), queries(big_m, 8, dim, "bf16", 21)
    with torch.cuda.stream(side):
        want = w4.kv8_attention(q, *small)
        out = torch.empty_like(want)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            w4.kv8_attention(q, *small, out=out)
        w4.kv8_attention(big_q, *big)
        others = [torch.full((size,), 7, dtype=torch.uint8, device="cuda") for _ in range(8)]
        out.zero_()
        graph.replay()
    side.synchronize()
    assert torch.equal(out, want) and all((x == 7).all() for x in others)


@pytest.mark.parametrize("what", ["rows", "tiles", "linear", "linear_fp8"])
def test_a_thread_that_has_not_used_the_gpu(w4, what):
    """Its first CUDA call may be this library's."""
    cache = ref.random_cache(w4, 5, 1, 64, 128, seed=22)
    table = ref.scattered_table([300], 64, 5, seed=23)
    K, N = 256, 128
    scales = torch.full((K // 128, N), 0.01, device="cuda", dtype=torch.bfloat16)
    layer = w4.repack_awq(ref.ints([[7] * (N // 8)] * K), ref.ints([[5] * (N // 8)] * (K // 128)), scales, K, N,
                          128, torch.bfloat16)
    x = torch.ones((200, K), device="cuda", dtype=torch.bfloat16)
    m = 200 if what == "tiles" else 1
    q = queries(m, 4, 128, "bf16", 24)
    args = (cache, table, ref.ints([300]), ref.bounds([m]), m, 300)
    call = {"linear": lambda: w4.linear(x, layer), "linear_fp8": lambda: w4.linear_fp8(x, layer)}.get(
        what, lambda: w4.kv8_attention(q, *args))
    want, got = call(), []
    torch.cuda.synchronize()
    thread = threading.Thread(target=lambda: got.append(call()))
    thread.start()
    thread.join()
    assert len(got) == 1 and torch.equal(got[0], want)


def test_threads_that_share_a_stream(w4):
    """Calls of several host threads on one stream, all with the stream's workspace."""
    page, dim, rounds = 64, 128, 150
    cache = ref.random_cache(w4, 300, 1, page, dim, seed=22)
    table = ref.scattered_table([2900, 9000], page, 300, seed=23)
    K, N = 4096, 1024
    g = torch.Generator(device="cuda").manual_seed(24)
    words = lambda *shape: torch.randint(-2 ** 31, 2 ** 31 - 1, shape, device="cuda", generator=g,  # noqa: E731
                                         dtype=torch.int32)
    scales = torch.full((K // 128, N), 0.01, device="cuda", dtype=torch.bfloat16)
    layer = w4.repack_awq(words(K, N // 8), words(K // 128, N // 8), scales, K, N, 128, torch.bfloat16)
    assert w4.w4a16_gemm_workspace_size(128, N, K, 128, torch.bfloat16, False) > 0  # splits K

    def attend(m, row, n, heads):
        q = queries(m, heads, dim, "bf16", 25 + m)
        args = (cache, table[row:row + 1], ref.ints([n]), ref.bounds([m]), m, n)
        return lambda: w4.kv8_attention(q, *args)

    x = torch.randn((128, K), device="cuda", generator=g).bfloat16()
    work = [attend(1, 0, 2900, 4), attend(1, 1, 9000, 8), attend(50, 0, 2800, 8), attend(2, 1, 8000, 8),
            lambda: w4.linear(x, layer), lambda: w4.linear_fp8(x, layer)]
    want = [f() for f in work]
    torch.cuda.synchronize()
    start, right = threading.Barrier(len(work)), []

    def run(f, expected):
        start.wait()
        got = [f() for _ in range(rounds)]
        right.extend(1 for y in got if torch.equal(y, expected))

    threads = [threading.Thread(target=run, args=a) for a in zip(work, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(right) == len(work) * rounds and w4.w4_device_status() == 0


@pytest.mark.parametrize("kv_heads,dim,page", [(3, 64, 32), (3, 64, 16), (2, 128, 64)])
def test_codes_are_not_replaced_before_they_are_read(w4, kv_heads, dim, page):
    """Many ragged sequences of a few steps each, all scores equal: every call gives
    the same, the mean of the values that a row sees."""
    rng = np.random.default_rng(dim + page)
    lens = [int(x) for x in rng.integers(130, 521, 70)]
    counts = [int(x) for x in rng.integers(20, 59, 70)]
    pages = sum(-(-n // page) for n in lens)
    cache = ref.random_cache(w4, pages, kv_heads, page, dim, seed=33, scales="any")
    table = ref.scattered_table(lens, page, pages, seed=34)
    q = queries(sum(counts), 16 * kv_heads, dim, "fp16", 35)
    want = check(w4, q, cache, table, lens, counts, True, "fp16", scale=0.0)
    args = (cache, table, ref.ints(lens), ref.bounds(counts), max(counts), max(lens))
    outs = [torch.empty_like(want) for _ in range(20)]
    for _ in range(20):
        for out in outs:
            w4.kv8_attention(q, *args, scale=0.0, out=out)
        assert all(torch.equal(out, want) for out in outs)


@pytest.mark.parametrize("batch,heads,dim,page", [(64, 8, 128, 64), (64, 16, 64, 16), (3, 8, 128, 128)])
def test_units_are_not_replaced_before_they_are_read(w4, batch, heads, dim, page):
    """The same for few rows, split among warps."""
    rng = np.random.default_rng(batch + dim)
    lens = [int(x) for x in rng.integers(30, 120000 // batch, batch)]
    pages = sum(-(-n // page) for n in lens)
    cache = ref.random_cache(w4, pages, 2, page, dim, seed=36, scales="any")
    table = ref.scattered_table(lens, page, pages, seed=37)
    q = queries(batch, 2 * heads, dim, "bf16", 38)
    want = check(w4, q, cache, table, lens, [1] * batch, True, "bf16", scale=0.0)
    args = (cache, table, ref.ints(lens), ref.bounds([1] * batch), 1, max(lens))
    outs = [torch.empty_like(want) for _ in range(20)]
    for _ in range(20):
        for out in outs:
            w4.kv8_attention(q, *args, scale=0.0, out=out)
        assert all(torch.equal(out, want) for out in outs)


def test_outputs_of_a_call_on_another_stream(w4):
    """The current stream still works on a block of the output's size that it let go
    of, and the output is used on both streams and let go of in turn."""
    n, m = 500, 64
    cache = ref.random_cache(w4, 10, 2, 64, 128, seed=39)
    table = ref.scattered_table([n], 64, 10, seed=40)
    q = queries(m, 8, 128, "bf16", 41)
    args = (cache, table, ref.ints([n]), ref.bounds([m]), m, n)
    want = w4.kv8_attention(q, *args)
    side, a = torch.cuda.Stream(), torch.randn((4096, 4096), device="cuda").bfloat16()
    torch.cuda.synchronize()
    for _ in range(5):
        for _ in range(20):
            a @ a
        block = torch.empty_like(want)
        block.fill_(7)
        del block
        out = w4.kv8_attention(q, *args, stream=side)
        with torch.cuda.stream(side):
            mine = out.clone()
        torch.cuda.current_stream().wait_stream(side)
        yours = out.clone()
        del out
        other = w4.kv8_attention(q, *args, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(mine, want) and torch.equal(yours, want) and torch.equal(other, want)


LOW = 2.0 ** -33  # of a row's largest p_j times its value scale: what the kernels may lose of one


def exact_row(cache, table, q, n, scale):
    """One query head over n tokens of kv head 0, in float64: (out, tolerance).

    Of a token's p, times its value scale, the kernels keep fp16's eleven bits, and
    of what is small at least LOW of the row's largest. Scores here are small, so
    their own rounding is below 2^-16 of p; sums take n / 16 fp32 additions."""
    ids = table[0].long()
    k = ref.values(cache.k, cache.k_scale, ids, 0, n)
    code = cache.v[ids, 0].double().reshape(-1, cache.head_dim)[:n]
    vs = cache.v_scale[ids, 0].double().repeat_interleave(cache.page_size)[:n, None]
    s = (k @ q.double())[:, None] * scale
    p = torch.exp(s - s.max())
    out = (p * vs * code).sum(0) / p.sum()
    tol = ((p * vs * code.abs()).sum(0) * (2.0 ** -11 + 2.0 ** -16 + n * 2.0 ** -27)
           + LOW * (p * vs).max() * code.abs().sum(0)) / p.sum()
    return out, tol + 2.0 ** -11 * out.abs() + 2.0 ** -25


@pytest.mark.parametrize("m", [1, 2, 40])
@pytest.mark.parametrize("dim,page", [(128, 64), (64, 16)])
@pytest.mark.parametrize("at", [0, 70001])
def test_one_token_with_nearly_all_of_the_weight(w4, m, dim, page, at):
    """Every other token has 2^-26 of its weight; together they have 0.2 %, and the
    whole output, since its own value is zero."""
    n, heads = 131072, 4
    cache = w4.kv8_cache(n // page, 1, page, dim)
    g = torch.Generator(device="cuda").manual_seed(6)
    v = torch.randn((n, dim), device="cuda", generator=g) + 100
    v[at] = 0
    cache.v.view(torch.uint8).copy_(v.to(ref.F8).view(torch.uint8).view(cache.v.shape))
    k = torch.zeros((n, dim), device="cuda")
    k[at, 3] = 26
    cache.k.view(torch.uint8).copy_(k.to(ref.F8).view(torch.uint8).view(cache.k.shape))
    table = ref.ints(list(range(n // page))).view(1, -1)
    q = torch.zeros((m, heads, dim), dtype=torch.float16, device="cuda")
    q[:, :, 3] = 1
    out = w4.kv8_attention(q, cache, table, ref.ints([n]), ref.bounds([m]), m, n, scale=math.log(2),
                           causal=False)
    want, tol = exact_row(cache, table, q[0, 0], n, math.log(2))
    assert (tol < 0.05 * want.abs()).all()  # that the test can see what it looks for
    assert ((out.double() - want).abs() <= tol).all(), (out[0, 0, :4], want[:4])


@pytest.mark.parametrize("m", [1, 2, 70])
@pytest.mark.parametrize("up", [18, 26])
@pytest.mark.parametrize("spread", [0.0, 0.3])
def test_a_loud_page_beside_quiet_ones(w4, m, up, spread):
    """One page's values stand 2^up above the others', but not in the even columns:
    there the quiet pages are the result."""
    n, page, dim, heads = 1024, 64, 128, 4
    cache = ref.random_cache(w4, n // page, 1, page, dim, seed=7)
    cache.v_scale.fill_(2.0 ** -9)
    cache.v_scale[5] = 2.0 ** (up - 9)
    cache.v.view(torch.uint8)[5, :, :, ::2] = 0
    cache.v.view(torch.uint8)[5, :, :, 1::2] = torch.full((), 1.0).to(ref.F8).view(torch.uint8).item()
    raw = cache.v.view(torch.uint8)
    raw &= 0x7F  # of one sign, so that nothing cancels
    cache.k_scale.fill_(2.0 ** -6)
    table = ref.ints(list(range(n // page))).view(1, -1)
    q = queries(m, heads, dim, "fp16", 8) * spread
    out = w4.kv8_attention(q, cache, table, ref.ints([n]), ref.bounds([m]), m, n, causal=False)
    for i, h in ((0, 0), (m - 1, heads - 1)):
        want, tol = exact_row(cache, table, q[i, h], n, dim ** -0.5)
        assert (tol[::2] < 0.05 * want[::2].abs()).all()
        bad = (out[i, h].double() - want).abs() > tol
        assert not bad[::2].any() and not (bad & (want.abs() < 60000)).any()


@pytest.mark.parametrize("m,mag", [(1, 2.0 ** 21), (70, 2.0 ** 21), (1, 2.0 ** 24), (70, 2.0 ** 24), (1, 2.0 ** 30)])
def test_scores_that_round_by_more_than_they_differ(w4, m, mag):
    """Whichever token wins, the result is an average of values. (Scores of up to 14
    times mag, in steps of 2^-24 of them.)"""
    n, page, dim, heads = 1000, 64, 128, 4
    cache = ref.random_cache(w4, n // page + 1, 1, page, dim, seed=30)
    table = ref.scattered_table([n], page, cache.num_pages, seed=31)
    q = queries(m, heads, dim, "bf16", 32)
    out = w4.kv8_attention(q, cache, table, ref.ints([n]), ref.bounds([m]), m, n, causal=False, scale=mag / 10)
    v = ref.values(cache.v, cache.v_scale, table[0].long(), 0, n)
    lo, hi = v.amin(0), v.amax(0)
    edge = 2.0 ** -7 * torch.maximum(lo.abs(), hi.abs())
    assert torch.isfinite(out).all()
    assert ((out.double() >= lo - edge) & (out.double() <= hi + edge)).all()


@pytest.mark.parametrize("batch,max_kv", [(300, 900), (2100, 900), (2100, 100)])
def test_many_sequences(w4, batch, max_kv):
    """More sequences than a thread block has threads, and than a split call takes."""
    rng = np.random.default_rng(batch)
    lens = [int(x) for x in rng.integers(0, 40, batch)]
    lens[3], lens[batch - 2] = max_kv, max_kv - 1
    counts = [int(x) for x in rng.integers(0, 3, batch)]
    counts[3] = 2
    page = 32
    pages = sum(-(-n // page) for n in lens)
    cache = ref.random_cache(w4, pages, 2, page, 64, seed=9)
    table = ref.scattered_table(lens, page, pages, seed=10)
    q = queries(sum(counts), 4, 64, "bf16", 11)
    check(w4, q, cache, table, lens, counts, True, "bf16")


# --------------------------------------------------------------------------- #
# append                                                                        #
# --------------------------------------------------------------------------- #
def test_append_reports_bad_offsets(w4):
    """Offsets that fall, and lengths past what any cache may hold."""
    cache = w4.kv8_cache(8, 1, 16, 64)
    table = ref.ints([[0, 1], [2, 3], [4, 5]])
    x = torch.ones((6, 1, 64), dtype=torch.bfloat16, device="cuda")
    before = cache_state(cache)
    w4.kv8_append(x, x, cache, table, ref.ints([0, 9, 0]), ref.ints([4, 4, 2, 2]), 4)
    assert w4.w4_device_status(clear=True) == 14 and same(cache_state(cache), before)
    # a row of 2^27 pages: the page that ends at token 2^31 has no 32-bit end
    longest = torch.zeros((1, 1 << 27), dtype=torch.int32, device="cuda")
    longest[0, -1] = 3
    w4.kv8_append(x, x, cache, longest, ref.ints([2 ** 31 - 1]), ref.ints([0, 1]), 1)
    assert w4.w4_device_status(clear=True) == 14 and same(cache_state(cache), before)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64)])
def test_append_to_scales_that_are_no_powers_of_two(w4, dtype, dim, page):
    """Pages written by another program: old scales that stay, and that grow."""
    held, new = [3, page - 2, 1, 7], [2, 2, page - 1, 1]
    lens = [a + b for a, b in zip(held, new)]
    cache = ref.random_cache(w4, 4, 2, page, dim, seed=12, scales="any")
    for sc in (cache.k_scale, cache.v_scale):
        sc[:] = ref.ints([1, 3, 5, 7]).float()[:, None] / 3 * ref.ints([1, 2]).float() / 1024
        sc[2] *= 1e4  # stays
    state = cache_state(cache)
    table = ref.ints([0, 1, 2, 3]).view(4, 1)
    x = torch.from_numpy(np.random.default_rng(13).standard_normal((sum(new), 4, dim))).cuda().to(ref.DTYPES[dtype])
    k, v = x[:, :2], x[:, 2:]
    w4.kv8_append(k, v, cache, table, ref.ints(lens), ref.bounds(new), max(new))
    ref.append(state, k.double().cpu().numpy(), v.double().cpu().numpy(), table.cpu().numpy(), lens, new, page)
    assert same(cache_state(cache), state)
    assert w4.w4_device_status() == 0
