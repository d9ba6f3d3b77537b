"""The 8-bit key-value cache operators against plain 64-bit forms (kv8util):
attention over it within a tolerance derived from its roundings, append, fork,
reserve, free, compact and copy exactly."""
import numpy as np
import pytest
import torch

import kv8util as ref
from libutil import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_built()
    import int4_weight_only_repack_gb300 as mod
    mod.w4_device_status(clear=True)
    return mod


def queries(n, heads, dim, dtype, seed, pad=0):
    """[n, heads, dim] rows of a buffer `pad` heads wider."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((n, heads + pad, dim), device="cuda", generator=g) * 1.3
    return x.to(ref.DTYPES[dtype])[:, :heads]


def check(w4, q, cache, table, lens, counts, causal, dtype, scale=None, slack=0):
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    got = w4.kv8_attention(q, cache, table, ref.ints(lens), ref.bounds(counts),
                           max(max(counts), 1) + slack, max(max(lens), 1) + slack, scale=scale,
                           causal=causal, out=out)
    assert got is out
    want, tol = ref.attention(q, cache, table, lens, counts,
                              q.shape[2] ** -0.5 if scale is None else scale, causal, dtype)
    # past the type's range the answer is infinite, within the tolerance of it either is
    edge = torch.finfo(q.dtype).max * (1 + ref.UNIT[dtype])
    inf = out.double() == want.sign() * float("inf")
    assert inf[want.abs() - tol > edge].all()
    err = torch.where(inf & (want.abs() + tol >= edge), 0.0, (out.double() - want).abs())
    assert torch.isfinite(err).all()
    worst = (err / tol.clamp_min(1e-30)).max().item() if err.numel() else 0.0
    assert worst <= 1, worst
    assert w4.w4_device_status() == 0
    return out


HEADS = [(8, 8, 128), (16, 2, 128), (14, 2, 64), (5, 1, 128), (71, 1, 64), (6, 3, 64), (40, 1, 128)]


@pytest.mark.parametrize("heads,kv_heads,dim", HEADS)
@pytest.mark.parametrize("page,dtype", [(16, "bf16"), (32, "fp16"), (64, "bf16"), (128, "fp16")])
def test_decode(w4, heads, kv_heads, dim, page, dtype):
    lens = [1, 15, 16, 17, 0, 31, 33, 64, 65, 127, 128, 129, 300, 1031]
    cache = ref.random_cache(w4, 200, kv_heads, page, dim, seed=1)
    table = ref.scattered_table(lens, page, 200, seed=2)
    q = queries(len(lens), heads, dim, dtype, 3, pad=2)
    out = check(w4, q, cache, table, lens, [1] * len(lens), True, dtype)
    assert torch.count_nonzero(out[4]) == 0  # nothing to see


@pytest.mark.parametrize("heads,kv_heads,dim", HEADS)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("page,dtype", [(16, "fp16"), (64, "bf16")])
def test_ragged_rows(w4, heads, kv_heads, dim, causal, page, dtype):
    counts = [3, 1, 0, 17, 64, 5, 130, 9, 33]
    lens = [3, 77, 40, 17, 200, 0, 260, 4, 33]
    cache = ref.random_cache(w4, 120, kv_heads, page, dim, seed=4, scales="any")
    table = ref.scattered_table(lens, page, 120, seed=5)
    q = queries(sum(counts), heads, dim, dtype, 6)
    # causal: 5 queries over no token, and 9 over 4: their first see nothing
    check(w4, q, cache, table, lens, counts, causal, dtype, slack=11)


@pytest.mark.parametrize("heads,kv_heads,dim,n,m,page,causal,dtype", [
    (8, 2, 128, 1000, 1000, 64, True, "bf16"),
    (4, 4, 128, 777, 515, 16, True, "fp16"),
    (9, 3, 64, 1290, 257, 128, True, "bf16"),
    (4, 4, 64, 611, 300, 32, False, "fp16"),
    (10, 1, 128, 2100, 131, 64, False, "bf16"),
])
def test_prompts(w4, heads, kv_heads, dim, n, m, page, causal, dtype):
    lens, counts = [n, n // 3, n - 1], [m, min(m, n // 3), 1]
    pages = 3 * (n // page + 1)
    cache = ref.random_cache(w4, pages, kv_heads, page, dim, seed=7)
    table = ref.scattered_table(lens, page, pages, seed=8)
    q = queries(sum(counts), heads, dim, dtype, 9, pad=2 * kv_heads)
    check(w4, q, cache, table, lens, counts, causal, dtype)


@pytest.mark.parametrize("batch,n,heads,kv_heads,dim,page", [
    (1, 20011, 8, 1, 128, 64), (3, 9000, 16, 4, 64, 16), (1, 40000, 5, 5, 128, 128)])
def test_long_decode(w4, batch, n, heads, kv_heads, dim, page):
    """One axis split over many thread blocks and joined."""
    lens = [n - 977 * b for b in range(batch)]
    pages = batch * (n // page + 1)
    cache = ref.random_cache(w4, pages, kv_heads, page, dim, seed=10)
    table = ref.scattered_table(lens, page, pages, seed=11)
    q = queries(batch, heads, dim, "fp16", 12)
    check(w4, q, cache, table, lens, [1] * batch, True, "fp16")


@pytest.mark.parametrize("m", [1, 3, 200])
def test_slots_without_tokens_do_not_matter(w4, m):
    """NaN codes and scales of unused slots, pages and table entries stay out."""
    page, dim, kv_heads = 32, 128, 2
    lens, counts = [45, 200, 321], [min(m, 45), m, m]
    cache = ref.random_cache(w4, 40, kv_heads, page, dim, seed=13)
    table = ref.scattered_table(lens, page, 40, seed=14, width=20)
    q = queries(sum(counts), 6, dim, "bf16", 15)
    want = check(w4, q, cache, table, lens, counts, True, "bf16").clone()
    used = torch.zeros(40, page, dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        for j in range(n):
            used[table[b, j // page].long(), j % page] = True
    for codes, sc in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        raw = codes.view(torch.uint8)
        raw.copy_(torch.where(used[:, None, :, None], raw, torch.full_like(raw, 0x7F)))
        sc.copy_(torch.where(used.any(1)[:, None], sc, torch.full_like(sc, float("nan"))))
    table[table < 0] = 2 ** 30  # never followed
    got = check(w4, q, cache, table, lens, counts, True, "bf16")
    assert torch.equal(got, want)


@pytest.mark.parametrize("m", [1, 40, 300])
def test_nan_reaches_only_rows_that_see_it(w4, m):
    """A NaN key or value in a token later than a query leaves the query alone."""
    page, dim, n = 64, 128, 320
    cache = ref.random_cache(w4, 8, 1, page, dim, seed=16)
    table = ref.scattered_table([n], page, 8, seed=17)
    q = queries(m, 4, dim, "fp16", 18)
    args = (cache, table, ref.ints([n]), ref.bounds([m]), m, n)
    clean = w4.kv8_attention(q, *args)
    spot = n - 1 - m // 2  # seen by the second half of the queries
    for codes in (cache.k, cache.v):
        raw = codes.view(torch.uint8)
        at = (table[0, spot // page].long(), 0, spot % page, 5)
        keep = raw[at].clone()
        raw[at] = 0x7F
        got = w4.kv8_attention(q, *args)
        raw[at] = keep
        sees = torch.arange(m, device="cuda") >= spot - (n - m)
        assert torch.equal(got[~sees], clean[~sees])
        assert torch.isnan(got[sees]).any(-1).all()


@pytest.mark.parametrize("m", [1, 200])
def test_extreme_scores(w4, m):
    """Rows whose scores span thousands (one token takes all), tiny and huge
    queries, value scales from 2^-40 to 2^20 in one sequence."""
    page, dim, n = 16, 128, 400
    lens, counts = [n], [m]
    cache = ref.random_cache(w4, 30, 1, page, dim, seed=19)
    cache.v_scale.copy_(torch.exp2(torch.linspace(-40, 20, 30, device="cuda").round())[:, None])
    table = ref.scattered_table(lens, page, 30, seed=20)
    for mag in (1e-6, 1.0, 300.0):
        q = (queries(m, 4, dim, "fp16", 21).float() * mag).half()
        check(w4, q, cache, table, lens, counts, False, "fp16", scale=1.0 if mag > 1 else 0.1)
    zero = torch.zeros_like(q)
    check(w4, zero, cache, table, lens, counts, True, "fp16")


def test_bf16_queries_beyond_fp16(w4):
    cache = ref.random_cache(w4, 30, 2, 32, 128, seed=22)
    table = ref.scattered_table([300, 500], 32, 30, seed=23)
    q = (queries(2, 8, 128, "bf16", 24).float() * 2.0 ** 40).bfloat16()
    check(w4, q, cache, table, [300, 500], [1, 1], True, "bf16", scale=2.0 ** -43)
    q = (queries(2, 8, 128, "bf16", 24).float() * 2.0 ** -60).bfloat16()
    check(w4, q, cache, table, [300, 500], [1, 1], True, "bf16", scale=2.0 ** 57)


def test_offsets_past_32_bits(w4):
    """A cache of 5 GB a side, with the sequences' pages at its end."""
    page, dim, kv_heads = 128, 128, 8
    pages = 40000
    cache = w4.kv8_cache(pages, kv_heads, page, dim)
    small = ref.random_cache(w4, 60, kv_heads, page, dim, seed=25)
    for big, part in ((cache.k, small.k), (cache.v, small.v)):
        big.view(torch.uint8)[-60:] = part.view(torch.uint8)
    cache.k_scale[-60:], cache.v_scale[-60:] = small.k_scale, small.v_scale
    lens = [1500, 2000, 700]
    table = ref.scattered_table(lens, page, 60, seed=26) + (pages - 60)
    for counts in ([1, 1, 1], [200, 150, 90]):
        q = queries(sum(counts), 16, dim, "bf16", 27)
        check(w4, q, cache, table, lens, counts, True, "bf16")
    new = torch.randn((3, kv_heads, dim), device="cuda").bfloat16()
    w4.kv8_append(new, new, cache, table, ref.ints(lens), ref.bounds([1, 1, 1]), 1)
    for b, n in enumerate(lens):
        p = int(table[b, (n - 1) // page])
        x = cache.v[p, :, (n - 1) % page].double() * cache.v_scale[p].double()[:, None]
        assert ((x - new[b].double()).abs() <= 2.0 ** -4 * new[b].double().abs() + 1e-2).all()
    w4.kv8_copy_pages(cache, ref.ints([pages - 1]), ref.ints([3]))
    assert torch.equal(cache.k.view(torch.uint8)[3], cache.k.view(torch.uint8)[pages - 1])
    assert w4.w4_device_status() == 0


def test_streams_graphs_and_determinism(w4):
    lens, counts = [700, 3000, 64], [1, 1, 1]
    cache = ref.random_cache(w4, 60, 4, 64, 128, seed=28)
    table = ref.scattered_table(lens, 64, 60, seed=29)
    q = queries(3, 16, 128, "bf16", 30)
    args = (cache, table, ref.ints(lens), ref.bounds(counts), 1, 3000)
    want = w4.kv8_attention(q, *args)
    for _ in range(5):
        assert torch.equal(w4.kv8_attention(q, *args), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(want)
    w4.kv8_attention(q, *args, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        w4.kv8_attention(q, *args, out=out)
    side.synchronize()
    with torch.cuda.graph(graph, stream=side):
        w4.kv8_attention(q, *args, out=out)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_bad_device_values_are_skipped(w4):
    W4_ERR_PAGE = 14
    lens, page = [100, 200, 150], 32
    cache = ref.random_cache(w4, 20, 2, page, 128, seed=31)
    table = ref.scattered_table(lens, page, 20, seed=32)
    q = queries(3, 4, 128, "bf16", 33)
    cu = ref.bounds([1, 1, 1])
    good = w4.kv8_attention(q, cache, table, ref.ints(lens), cu, 1, 200)
    bad = table.clone()
    bad[1, 2] = 20
    got = w4.kv8_attention(q, cache, bad, ref.ints(lens), cu, 1, 200)
    assert w4.w4_device_status(clear=True) == W4_ERR_PAGE
    assert torch.equal(got[[0, 2]], good[[0, 2]]) and torch.isfinite(got).all()
    got = w4.kv8_attention(q, cache, table, ref.ints([100, 200000, 150]), cu, 1, 200)
    assert w4.w4_device_status(clear=True) == W4_ERR_PAGE
    assert torch.equal(got[[0, 2]], good[[0, 2]]) and torch.count_nonzero(got[1]) == 0
    new = q[:, :2].contiguous()
    for t, n in ((bad, [100, 96 - 10, 150]), (table, [100, -3, 150]), (table, [0, 200000, 0])):
        w4.kv8_append(new, new, cache, t, ref.ints(n), cu, 1)
        w4.w4_device_status(clear=True)
    bad[:, :] = 99
    w4.kv8_append(new, new, cache, bad, ref.ints(lens), cu, 1)
    assert w4.w4_device_status(clear=True) == W4_ERR_PAGE


# --------------------------------------------------------------------------- #
# append                                                                        #
# --------------------------------------------------------------------------- #
def cache_state(c):
    return [c.k.double().cpu().numpy(), c.v.double().cpu().numpy(),
            c.k_scale.double().cpu().numpy(), c.v_scale.double().cpu().numpy()]


def same(a, b):
    return all(np.array_equal(x, y, equal_nan=True) for x, y in zip(a, b))


@pytest.mark.parametrize("kv_heads,dim,page,dtype", [
    (3, 128, 16, "bf16"), (2, 64, 32, "fp16"), (1, 128, 64, "fp16"), (5, 64, 128, "bf16"),
    (2, 128, 128, "bf16")])
def test_append(w4, kv_heads, dim, page, dtype):
    """Three calls of growing, shrinking and ragged counts: pages are begun, filled
    and continued, scales grow and stay."""
    rng = np.random.default_rng(40)
    total = [page + 5, 1, 2 * page, 0, 3 * page + 1, 7]
    cache = ref.random_cache(w4, 20, kv_heads, page, dim, seed=41)
    table = ref.scattered_table(total, page, 20, seed=42)
    state = cache_state(cache)
    done = [0] * len(total)
    for call, mag in enumerate((0.01, 30.0, 1.0)):
        counts = [t - d if call == 2 else int(rng.integers(0, t - d + 1)) for t, d in zip(total, done)]
        done = [d + c for d, c in zip(done, counts)]
        x = torch.from_numpy(rng.standard_normal((sum(counts), 2 * kv_heads + 1, dim)) * mag).cuda()
        x = x.to(ref.DTYPES[dtype])
        k, v = x[:, :kv_heads], x[:, kv_heads:2 * kv_heads]
        w4.kv8_append(k, v, cache, table, ref.ints(done), ref.bounds(counts), max(max(counts), 1) + call)
        ref.append(state, k.double().cpu().numpy(), v.double().cpu().numpy(), table.cpu().numpy(),
                   done, counts, page)
        assert same(cache_state(cache), state)
    assert w4.w4_device_status() == 0


def test_append_scales_at_their_edges(w4):
    """Largest magnitudes at 448 * 2^n and next to it, zeros, infinities, NaN."""
    page, dim = 16, 64
    peaks = [448.0, 447.0, 450.0, 1.75, 1.7578125, 1.7421875, 2.0 ** -30, 2.0 ** -60, 0.0, 65504.0,
             float("inf"), float("nan"), 3e38]
    cache = ref.random_cache(w4, len(peaks), 1, page, dim, seed=43)
    state = cache_state(cache)
    x = torch.zeros((len(peaks), 1, dim), dtype=torch.bfloat16, device="cuda")
    for i, p in enumerate(peaks):
        x[i, 0, i] = p
        x[i, 0, 40] = -1.0 if np.isnan(p) or np.isinf(p) else -p / 3
    table = ref.ints(list(range(len(peaks)))).view(-1, 1)
    lens = [1] * len(peaks)
    w4.kv8_append(x, x, cache, table, ref.ints(lens), ref.bounds(lens), 1)
    n = x.double().cpu().numpy()
    ref.append(state, n, n, table.cpu().numpy(), lens, lens, page)
    assert same(cache_state(cache), state)


def test_append_then_attend_at_once(w4):
    """The whole serving order on one stream, with nothing waited for between."""
    page, dim, kv_heads, heads = 16, 128, 2, 8
    cache = w4.kv8_cache(40, kv_heads, page, dim)
    lens = [70, 33, 100]
    table = ref.scattered_table(lens, page, 40, seed=44)
    x = torch.randn((sum(lens), heads + 2 * kv_heads, dim), device="cuda").bfloat16()
    q, k, v = x.split([heads, kv_heads, kv_heads], dim=1)
    cu, kv = ref.bounds(lens), ref.ints(lens)
    w4.kv8_append(k, v, cache, table, kv, cu, 100)
    out = w4.kv8_attention(q, cache, table, kv, cu, 100, 100)
    want, tol = ref.attention(q, cache, table, lens, lens, dim ** -0.5, True, "bf16")
    assert ((out.double() - want).abs() <= tol).all()
    # and near the unquantised attention: e4m3 keeps 4 bits
    at = 0
    for n in lens:
        kk = k[at:at + n].double().repeat_interleave(heads // kv_heads, 1)
        vv = v[at:at + n].double().repeat_interleave(heads // kv_heads, 1)
        s = torch.einsum("ihd,jhd->hij", q[at:at + n].double(), kk) * dim ** -0.5
        s += torch.full((n, n), -float("inf"), device="cuda", dtype=torch.float64).triu(1)
        o = torch.einsum("hij,jhd->ihd", s.softmax(-1), vv)
        assert (out[at:at + n].double() - o).norm() <= 0.06 * o.norm()
        at += n


# --------------------------------------------------------------------------- #
# pages                                                                         #
# --------------------------------------------------------------------------- #
def book_of(pool):
    return ref.Book(pool.refs.tolist(), pool.table.tolist(), pool.lens.tolist(), pool.page_size)


def agrees(pool, book):
    return (pool.refs.tolist() == book.refs and pool.lens.tolist() == book.lens
            and pool.table.tolist() == book.table)


@pytest.mark.parametrize("pages,seqs,page", [(7, 3, 16), (300, 40, 32), (5000, 700, 16), (40001, 65, 64)])
def test_pool_life(w4, pages, seqs, page):
    """Random reserves, forks, frees and compactions, each against the plain one."""
    rng = np.random.default_rng(pages)
    longest = max(2, min(pages * page // seqs, 40 * page))
    pool = w4.kv8_pool(pages, seqs, longest, page)
    book = book_of(pool)
    for step in range(12):
        new = [int(rng.integers(0, max(1, (longest - n) // 2 + 1))) if rng.random() < 0.5 else 0
               for n in book.lens]
        w4.kv8_reserve(pool, ref.ints(new))
        assert book.reserve(new) == (int(pool.status) == 0)
        assert int(pool.status) in (0, 15) and agrees(pool, book)
        empty = [s for s, n in enumerate(book.lens) if n == 0]
        if empty:
            dst = rng.permutation(empty)[:int(rng.integers(1, len(empty) + 1))].tolist()
            src = [int(rng.integers(0, seqs)) for _ in dst]
            src = [s for s in src if s not in dst] or [next(iter(set(range(seqs)) - set(dst)), dst[0])]
            dst = dst[:len(src)]
            src = src[:len(dst)]
            a, b = w4.kv8_fork(pool, ref.ints(src), ref.ints(dst))
            moves = book.fork(src, dst)
            assert (moves is not None) == (int(pool.status) == 0) and agrees(pool, book)
            if moves is not None:
                assert list(zip(a.tolist(), b.tolist())) == moves
        gone = rng.integers(0, seqs, max(1, seqs // 3)).tolist()  # some twice
        w4.kv8_free(pool, ref.ints(gone))
        book.free(dict.fromkeys(gone))
        assert int(pool.status) == 0 and agrees(pool, book)
        if step % 3 == 2:
            a, b = w4.kv8_compact(pool)
            moves = book.compact()
            assert agrees(pool, book)
            assert list(zip(a.tolist(), b.tolist()))[:len(moves)] == moves
            assert (a[len(moves):] == -1).all() and (b[len(moves):] == -1).all()


def test_pool_extremes(w4):
    pool = w4.kv8_pool(9, 3, 9 * 16, 16)
    w4.kv8_reserve(pool, ref.ints([9 * 16, 0, 0]))         # every page
    assert int(pool.status) == 0 and pool.refs.tolist() == [1] * 9
    a, _ = w4.kv8_compact(pool)                            # full: nothing moves
    assert (a == -1).all() and pool.table[0].tolist() == list(range(9))
    w4.kv8_reserve(pool, ref.ints([0, 1, 0]))
    assert int(pool.status) == 15 and pool.lens.tolist() == [144, 0, 0]
    w4.kv8_fork(pool, ref.ints([0]), ref.ints([2]))        # nothing partial: shares all
    assert int(pool.status) == 0 and pool.refs.tolist() == [2] * 9
    w4.kv8_free(pool, ref.ints([0, 2, 2, 1]))
    assert pool.refs.tolist() == [0] * 9 and pool.lens.tolist() == [0, 0, 0]
    a, _ = w4.kv8_compact(pool)                            # empty
    assert (a == -1).all()


def test_pool_errors_change_nothing(w4):
    pool = w4.kv8_pool(50, 6, 160, 16)
    w4.kv8_reserve(pool, ref.ints([40, 17, 0, 0, 0, 0]))
    book = book_of(pool)
    for src, dst, status in (([0, 1], [2, 2], 16), ([0], [1], 16), ([0], [6], 16), ([-1], [3], 16),
                             ([0, 1, 0], [3, 4, 1], 16)):
        w4.kv8_fork(pool, ref.ints(src), ref.ints(dst))
        assert int(pool.status) == status and agrees(pool, book)
    for new in ([121, 0, 0, 0, 0, 0], [0, -1, 0, 0, 0, 0]):
        w4.kv8_reserve(pool, ref.ints(new))
        assert int(pool.status) == 14 and agrees(pool, book)
    w4.kv8_free(pool, ref.ints([9]))
    assert int(pool.status) == 16 and agrees(pool, book)
    quiet = w4.KV8Pool(pool.refs, pool.table, pool.lens, 16)  # no status of its own
    w4.kv8_free(quiet, ref.ints([-2]))
    assert w4.w4_device_status(clear=True) == 16 and agrees(pool, book)


@pytest.mark.parametrize("kv_heads,dim,page", [(1, 64, 16), (3, 128, 16), (8, 128, 64), (5, 64, 128)])
def test_copy_pages(w4, kv_heads, dim, page):
    cache = ref.random_cache(w4, 31, kv_heads, page, dim, seed=50, scales="any")
    before = [x.clone() for x in (cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale,
                                  cache.v_scale)]
    src, dst = [3, 30, -1, 3, 7, -1], [0, 1, -1, 29, 2, 12]
    w4.kv8_copy_pages(cache, ref.ints(src), ref.ints(dst))
    for was, now in zip(before, (cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale,
                                 cache.v_scale)):
        want = was.clone()
        for s, d in zip(src, dst):
            if s >= 0:
                want[d] = was[s]
        assert torch.equal(now, want)
    w4.kv8_copy_pages(cache, ref.ints([31]), ref.ints([0]))
    assert w4.w4_device_status(clear=True) == 14


def test_fork_compact_keep_what_sequences_hold(w4):
    """Attention over a sequence, its fork and both after a compaction agree."""
    page, dim = 16, 64
    pool = w4.kv8_pool(60, 5, 320, page)
    cache = ref.random_cache(w4, 60, 2, page, dim, seed=51)
    w4.kv8_reserve(pool, ref.ints([100, 57, 0, 33, 0]))
    q = queries(5, 4, dim, "bf16", 52)
    q[2], q[4] = q[0], q[1]
    one = ref.bounds([1] * 5)

    def attend():
        return w4.kv8_attention(q, cache, pool.table, pool.lens, one, 1, 320)

    was = attend()
    w4.kv8_copy_pages(cache, *w4.kv8_fork(pool, ref.ints([0, 1]), ref.ints([2, 4])))
    now = attend()
    assert torch.equal(now[[0, 1, 3]], was[[0, 1, 3]]) and torch.equal(now[[2, 4]], was[[0, 1]])
    w4.kv8_free(pool, ref.ints([0, 3]))
    w4.kv8_copy_pages(cache, *w4.kv8_compact(pool))
    after = attend()
    assert torch.equal(after[[1, 2, 4]], now[[1, 2, 4]])
    assert torch.count_nonzero(after[[0, 3]]) == 0
    assert w4.w4_device_status() == 0


def test_workspace_contents_do_not_matter(w4):
    lens = [5000, 700, 2100, 33, 0]
    cache = ref.random_cache(w4, 300, 4, 32, 128, seed=60)
    table = ref.scattered_table(lens, 32, 300, seed=61)
    size = w4.w4_kv8_attention_workspace_size(5, 5, 1, 5000, 8, 4, 128)
    q = queries(5, 8, 128, "bf16", 62)
    want = check(w4, q, cache, table, lens, [1] * 5, True, "bf16")
    for fill in (0, 0x7F, 0xFF):
        ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
        got = w4.kv8_attention(q, cache, table, ref.ints(lens), ref.bounds([1] * 5), 1, 5000,
                               workspace=ws)
        assert torch.equal(got, want)


@pytest.mark.parametrize("heads,kv_heads,dim,n,m,page,causal", [
    (8, 1, 128, 5000, 60, 64, True), (16, 2, 64, 3001, 40, 16, True), (9, 1, 64, 2000, 131, 128, False),
    (70, 1, 128, 2500, 1, 32, True), (4, 1, 128, 300, 300, 64, True)])
def test_few_tiles_over_a_long_axis(w4, heads, kv_heads, dim, n, m, page, causal):
    """Few tiles of many rows: their steps are split over thread blocks and joined.
    One sequence is short, so that some parts of it are empty; one has no token."""
    lens, counts = [n, 130, 0], [m, min(m, 130), 2]
    pages = 2 * (n // page + 3)
    cache = ref.random_cache(w4, pages, kv_heads, page, dim, seed=70, scales="any")
    table = ref.scattered_table(lens, page, pages, seed=71)
    q = queries(sum(counts), heads, dim, "bf16", 72)
    check(w4, q, cache, table, lens, counts, causal, "bf16")
    need = w4.w4_kv8_attention_workspace_size(3, sum(counts), m, n, heads, kv_heads, dim)
    assert (need > 0) == (n > 15 * 128)


def test_several_items_for_every_sm(w4):
    """More tiles than the GPU holds at once, of one and of two halves."""
    n, heads, kv_heads, dim, page = 300, 320, 160, 64, 64
    cache = ref.random_cache(w4, 8, kv_heads, page, dim, seed=73)
    table = ref.scattered_table([n], page, 8, seed=74)
    q = queries(n, heads, dim, "fp16", 75)
    check(w4, q, cache, table, [n], [n], True, "fp16")


def split_case(w4, seed, dim=128, page=64, n=2900, m=50):
    """A call whose tiles are split along the tokens, and a workspace of its size."""
    lens, counts = [n, 2100], [m, 7]
    cache = ref.random_cache(w4, 2 * (n // page + 1), 1, page, dim, seed=seed, scales="any")
    table = ref.scattered_table(lens, page, cache.num_pages, seed=seed + 1)
    q = queries(sum(counts), 8, dim, "fp16", seed + 2)
    size = w4.w4_kv8_attention_workspace_size(2, sum(counts), m, n, 8, 1, dim)
    assert size > 0
    return lens, counts, cache, table, q, size


def test_split_tiles_workspace_contents_do_not_matter(w4):
    lens, counts, cache, table, q, size = split_case(w4, 80)
    want = check(w4, q, cache, table, lens, counts, True, "fp16")
    for fill in (0, 0x7F, 0xFF):
        ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
        got = w4.kv8_attention(q, cache, table, ref.ints(lens), ref.bounds(counts), max(counts),
                               max(lens), workspace=ws)
        assert torch.equal(got, want)
    with pytest.raises(w4.W4Error):
        w4.kv8_attention(q, cache, table, ref.ints(lens), ref.bounds(counts), max(counts),
                         max(lens), workspace=ws[:size - 1])


@pytest.mark.parametrize("page", [16, 64])
def test_split_tiles_nan_reaches_only_rows_that_see_it(w4, page):
    """In the last tokens, where rows differ in what they see, and in the first."""
    m, n = 50, 2900
    lens, counts, cache, table, q, _ = split_case(w4, 90, page=page, n=n, m=m)
    args = (cache, table, ref.ints(lens), ref.bounds(counts), m, n)
    clean = w4.kv8_attention(q, *args)
    for spot in (n - 1 - m // 2, 3):
        for codes in (cache.k, cache.v):
            raw = codes.view(torch.uint8)
            at = (table[0, spot // page].long(), 0, spot % page, 5)
            keep = raw[at].clone()
            raw[at] = 0x7F
            got = w4.kv8_attention(q, *args)
            raw[at] = keep
            sees = torch.arange(sum(counts), device="cuda") >= spot - (n - m)
            sees[m:] = False  # the other sequence
            assert torch.equal(got[~sees], clean[~sees])
            assert torch.isnan(got[sees]).any(-1).all()


def test_split_tiles_extreme_scores(w4):
    """The parts' bases differ by thousands, their value scales by 2^60."""
    lens, counts, cache, table, q, _ = split_case(w4, 100, page=16)
    cache.v_scale.copy_(torch.exp2(torch.linspace(-40, 20, cache.num_pages, device="cuda").round())[:, None])
    for mag in (1e-6, 1.0, 300.0):
        check(w4, (q.float() * mag).half(), cache, table, lens, counts, False, "fp16",
              scale=1.0 if mag > 1 else 0.1)
    check(w4, torch.zeros_like(q), cache, table, lens, counts, True, "fp16")
