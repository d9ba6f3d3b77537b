"""Masks that hide nothing, against the call without a mask: bit for bit where both deal
the tokens to blocks alike, and everywhere within the tolerance of the definition. A call
deals them alike unless a prompt's items are split over blocks (fewer than half as many
items as SMs, 16 steps of 128 tokens at least), or the bound of the lengths lets the
window hide tokens."""
import pytest
import torch

import kv8mask as mask
import kv8util as ref
from test_gpu_kv8 import queries, w4  # noqa: F401

pytestmark = pytest.mark.gpu


def near(got, want, tol):
    worst = ((got.double() - want).abs() / tol.clamp_min(1e-30)).max().item()
    assert torch.isfinite(got).all() and worst <= 1, worst


@pytest.mark.parametrize("m,heads", [(1, 4), (1, 12), (6, 8), (300, 4), (40, 8)])
@pytest.mark.parametrize("slack", [0, 3000])
@pytest.mark.parametrize("dim,dtype", [(128, "bf16"), (64, "fp16")])
def test_windows_that_hide_nothing(w4, m, heads, slack, dim, dtype):
    """Equal whenever the window or the sinks reach the bound of the lengths, the bound
    itself among them."""
    lens, counts, most = [700, 350, 1], [m, min(m, 350), 1], 700 + slack
    cache = ref.random_cache(w4, 60, 2, 32, dim, seed=16)
    table = ref.scattered_table(lens, 32, 60, seed=17)
    q = queries(sum(counts), heads, dim, dtype, 18)
    args = (q, cache, table, ref.ints(lens), ref.bounds(counts), m, most)
    want = w4.kv8_attention(*args)
    exact, tol = mask.attention(q, cache, table, lens, counts, lambda b: mask.window_sees(lens[b], counts[b], 2 ** 31, 0),
                                dim ** -0.5, dtype)
    near(want, exact, tol)
    split = -(-m * heads // 2 // 256) * 2 * 3 <= 76 and most > 15 * 128 and m * heads // 2 > 64
    for window, sinks in ((2 ** 30, 0), (2 ** 30, 2 ** 30), (2 ** 40, 5), (10 ** 6, 2 ** 33), (most, 0), (most, 7),
                          (1, 2 ** 30), (1, most), (700, 0), (701, 0), (1, 700), (350, 350)):
        got = w4.kv8_attention(*args, window=window, sinks=sinks)
        if max(window, sinks) >= most and not split:
            assert torch.equal(got, want), (window, sinks)
        near(got, exact, tol)
    assert w4.w4_device_status() == 0


@pytest.mark.parametrize("heads,kv_heads,dim,m", [(32, 8, 128, 61), (16, 8, 64, 64), (8, 1, 64, 40)])
@pytest.mark.parametrize("n", [6000, 4500, 2200, 4097, 300])
def test_split_prompts(w4, heads, kv_heads, dim, m, n):
    """A chain of drafts, a wide window and neither, under a bound of 6000: the parts are
    not the same for every length, the results are within the definition's tolerance."""
    cache = ref.random_cache(w4, 100, kv_heads, 64, dim, seed=22)
    table = ref.scattered_table([n], 64, 100, seed=23, width=94)
    q = queries(m, heads, dim, "fp16", 24)
    args = (q, cache, table, ref.ints([n]), ref.bounds([m]), m, 6000)
    exact, tol = mask.attention(q, cache, table, [n], [m], lambda b: mask.window_sees(n, m, 2 ** 31, 0), dim ** -0.5,
                                "fp16")
    chain = mask.words_tensor(mask.random_tree(m, None, "chain"))
    for how in (dict(), dict(tree=chain), dict(window=6000), dict(window=2 ** 30, sinks=3), dict(window=6000, tree=chain)):
        near(w4.kv8_attention(*args, **how), exact, tol)


@pytest.mark.parametrize("m,heads,lens,most", [
    (6, 8, [2000, 1995], 6000), (16, 2, [300, 295], 300), (64, 4, [1900, 64], 1900), (60, 16, [1000, 700], 1900),
    (64, 8, [2300, 900, 70, 64, 1500, 2299, 64, 100, 333, 1000], 2300)])
def test_chains_where_nothing_is_split(w4, m, heads, lens, most):
    """Few rows, short bounds, or items enough: bit for bit the call without a tree."""
    kv_heads = 2 if len(lens) < 5 else 8
    pages = sum(-(-n // 64) for n in lens)
    cache = ref.random_cache(w4, pages, kv_heads, 64, 64, seed=31)
    table = ref.scattered_table(lens, 64, pages, seed=32)
    q = queries(len(lens) * m, heads * kv_heads // 2, 64, "bf16", 33)
    args = (q, cache, table, ref.ints(lens), ref.bounds([m] * len(lens)), m, most)
    chain = mask.words_tensor(len(lens) * mask.random_tree(m, None, "chain"))
    want = w4.kv8_attention(*args)
    for how in (dict(tree=chain), dict(window=most), dict(window=most, sinks=9), dict(window=most + 64, tree=chain)):
        assert torch.equal(w4.kv8_attention(*args, **how), want)
