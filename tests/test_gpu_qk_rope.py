"""Norms of query and key heads with the rotation by position, against the formulas in
64 bits. In fp32 a normed element y is off by less than 2^-19 of itself (20 additions of
the squares, 2^-24 of their sum each and half of that in the root; rsqrtf 2^-22; three
products), the cosines and sines are inputs, and a turned element a c - b s by that much
of |a c| + |b s|. One rounding to the type follows (at least 2^-25 in fp16)."""
import pytest
import torch

import kv8util as ref
from libutil import ensure_built

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def w4():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_built()
    import int4_weight_only_repack_gb300 as mod
    mod.w4_device_status(clear=True)
    return mod


def formula(x, weight, positions, table, interleaved, eps=EPS):
    """(out, tolerance) in float64; a padded token's rows are NaN."""
    y = x.double()
    if weight is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * weight.double()
    err = 2.0 ** -19 * y.abs()
    out = y.clone()
    if table is not None:
        rot = table.shape[1]
        cs = table.double()[positions.clamp_min(0).long()][:, None]
        c, s = cs[..., :rot // 2], cs[..., rot // 2:]
        first = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
        second = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
        a, b = y[..., first], y[..., second]
        out[..., first], out[..., second] = a * c - b * s, b * c + a * s
        err[..., first] = 2.0 ** -19 * ((a * c).abs() + (b * s).abs())
        err[..., second] = 2.0 ** -19 * ((b * c).abs() + (a * s).abs())
    u = torch.finfo(x.dtype).eps / 2
    if positions is not None:
        out[positions < 0] = float("nan")
    return out, err + u * (out.abs() + err) + 2.0 ** -25 * (x.dtype is torch.float16)


def check(got, want, tol):
    """Equal within the tolerance; NaN where the formula has NaN, and only there."""
    assert torch.equal(got.isnan(), want.isnan())
    off = torch.where(want.isnan(), 0.0, (got.double() - want).abs() - tol)
    assert (off <= 0).all(), off.max()


def projection(tokens, heads, dim, dtype, seed, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((tokens, heads, dim), device="cuda", generator=g)
    x *= torch.exp(spread * torch.randn((tokens, heads, 1), device="cuda", generator=g))
    return x.to(ref.DTYPES[dtype])


def weights(dim, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [1 + 0.4 * torch.randn(dim, device="cuda", generator=g) for _ in range(2)]


HEADS = [(1, 1, 64), (7, 1, 128), (28, 4, 64), (32, 8, 128), (3, 5, 64), (71, 1, 64), (64, 8, 128)]


@pytest.mark.parametrize("heads,kv_heads,dim", HEADS)
@pytest.mark.parametrize("tokens,dtype", [(1, "bf16"), (2, "fp16"), (333, "bf16"), (1030, "fp16")])
@pytest.mark.parametrize("rot,interleaved", [(1, False), (1, True), (2, False), (2, True)])
def test_against_the_formula(w4, heads, kv_heads, dim, tokens, dtype, rot, interleaved):
    """Whole heads and half of them turned, pairs of both kinds."""
    table = w4.rope_table(5000, dim // rot)
    x = projection(tokens, heads + 2 * kv_heads, dim, dtype, 1)
    q, k, _ = x.split((heads, kv_heads, kv_heads), 1)
    g = torch.Generator(device="cuda").manual_seed(2)
    pos = torch.randint(0, 5000, (tokens,), device="cuda", generator=g, dtype=torch.int32)
    wq, wk = weights(dim, 3)
    got = w4.qk_norm_rope(q, k, pos, table, wq, wk, EPS, interleaved)
    for y, z, w in zip(got, (q, k), (wq, wk)):
        assert y.shape == z.shape and y.is_contiguous()
        check(y, *formula(z, w, pos, table, interleaved))
    assert w4.w4_device_status() == 0


@pytest.mark.parametrize("dim,rots", [(64, (16, 32, 48, 64)), (128, (16, 80, 96, 112, 128))])
@pytest.mark.parametrize("norms", [(True, True), (True, False), (False, True), (False, False)])
def test_parts_of_a_head_and_sides_without_a_norm(w4, dim, rots, norms):
    x = projection(19, 7, dim, "bf16", 4)
    pos = ref.ints(list(range(100, 119)))
    wq, wk = (w if n else None for w, n in zip(weights(dim, 5), norms))
    for rot in rots:
        for interleaved in (False, True):
            table = w4.rope_table(200, rot, 5e5)
            got = w4.qk_norm_rope(x[:, :5], x[:, 5:], pos, table, wq, wk, EPS, interleaved)
            for y, z, w in zip(got, (x[:, :5], x[:, 5:]), (wq, wk)):
                check(y, *formula(z, w, pos, table, interleaved))
                if w is None and rot < dim:  # what neither norm nor rotation touches
                    assert torch.equal(y[..., rot:], z[..., rot:])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_norms_alone_and_one_side(w4, dtype):
    x = projection(37, 9, 128, dtype, 6)
    wq, wk = weights(128, 7)
    for pos in (None, ref.ints([5] * 37)):
        q, k = w4.qk_norm_rope(x[:, :6], x[:, 6:], pos, None, wq, wk, 1e-3)
        check(q, *formula(x[:, :6], wq, None, None, False, 1e-3))
        check(k, *formula(x[:, 6:], wk, None, None, False, 1e-3))
    table, pos = w4.rope_table(50, 128), ref.ints(list(range(37)))
    q, k = w4.qk_norm_rope(x, None, pos, table, wq)
    assert k is None
    check(q, *formula(x, wq, pos, table, False))
    q, k = w4.qk_norm_rope(None, x, pos, table, None, wk)
    assert q is None
    check(k, *formula(x, wk, pos, table, False))


@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_in_a_projection_s_rows(w4, interleaved):
    """Queries and keys are turned where they lie; the values beside them stay."""
    x = projection(65, 20, 64, "bf16", 8)
    before = x.clone()
    table, pos = w4.rope_table(100, 64), ref.ints(list(range(65)))
    wq, wk = weights(64, 9)
    q, k, v = x.split((12, 4, 4), 1)
    got = w4.qk_norm_rope(q, k, pos, table, wq, wk, EPS, interleaved, q, k)
    assert got[0] is q and got[1] is k
    check(q, *formula(before[:, :12], wq, pos, table, interleaved))
    check(k, *formula(before[:, 12:16], wk, pos, table, interleaved))
    assert torch.equal(v, before[:, 16:])
    apart = w4.qk_norm_rope(before[:, :12], before[:, 12:16], pos, table, wq, wk, EPS, interleaved)
    assert torch.equal(apart[0], q) and torch.equal(apart[1], k)


def test_padded_tokens_and_positions_past_the_table(w4):
    """Neither is written; the second is an error, and the others are done all the same."""
    x = projection(8, 5, 128, "fp16", 10)
    table, (wq, wk) = w4.rope_table(30, 128), weights(128, 11)
    pos = ref.ints([3, -1, 0, 29, -2 ** 31, 7, 7, 7])
    out = [torch.full((8, h, 128), 9.0, dtype=x.dtype, device="cuda") for h in (4, 1)]
    w4.qk_norm_rope(x[:, :4], x[:, 4:], pos, table, wq, wk, q_out=out[0], k_out=out[1])
    assert w4.w4_device_status() == 0
    for y, z, w in zip(out, (x[:, :4], x[:, 4:]), (wq, wk)):
        want, tol = formula(z, w, pos, table, False)
        assert (y[[1, 4]] == 9).all()
        check(torch.where(want.isnan(), want.to(y.dtype), y), want, tol)
    for bad in (30, 2 ** 31 - 1):
        pos[2] = bad
        again = [torch.full_like(y, 9.0) for y in out]
        w4.qk_norm_rope(x[:, :4], x[:, 4:], pos, table, wq, wk, q_out=again[0], k_out=again[1])
        assert w4.w4_device_status(clear=True) == 17
        for y, z in zip(again, out):
            assert (y[2] == 9).all() and torch.equal(y[[0, 3, 5, 6, 7]], z[[0, 3, 5, 6, 7]])
    only = torch.full_like(out[0], 9.0)  # norms alone: padding counts, a large position does not
    w4.qk_norm_rope(x[:, :4], None, pos, None, wq, q_out=only)
    assert w4.w4_device_status() == 0
    assert (only[[1, 4]] == 9).all() and (only[2] != 9).any()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_infinities_and_nan_stay_in_their_heads(w4, dtype):
    x = projection(6, 6, 64, dtype, 12)
    table, pos, (wq, wk) = w4.rope_table(10, 64), ref.ints([0, 1, 2, 3, 4, 5]), weights(64, 13)
    clean = w4.qk_norm_rope(x[:, :4], x[:, 4:], pos, table, wq, wk)
    x[1, 2, 5], x[3, 4, 63] = float("nan"), float("inf")
    got = w4.qk_norm_rope(x[:, :4], x[:, 4:], pos, table, wq, wk)
    assert got[0][1, 2].isnan().all() and got[1][3, 0, [31, 63]].isnan().all()
    for y, z, at in zip(got, clean, ((1, 2), (3, 0))):
        keep = torch.ones(y.shape[:2], dtype=torch.bool, device="cuda")
        keep[at] = False
        assert torch.equal(y[keep], z[keep])


def test_loud_and_quiet_heads(w4):
    """The squares of bf16 elements up to 2^60 and of the smallest are summed in fp32."""
    table, pos, (w, _) = w4.rope_table(4, 128), ref.ints([0, 1, 2, 3]), weights(128, 14)
    x = projection(4, 3, 128, "bf16", 15, spread=0)
    for scale in (2.0 ** 57, 1.0, 2.0 ** -40):
        y = (x.float() * scale).to(x.dtype)
        got, _ = w4.qk_norm_rope(y, None, pos, table, w)
        check(got, *formula(y, w, pos, table, False))
    zero, _ = w4.qk_norm_rope(torch.zeros_like(x), None, pos, table, w)
    assert not zero.any()


def test_the_table(w4):
    """Cosines and sines of far positions are those of the exact angle."""
    table = w4.rope_table(131072, 32, 1e4).double().cpu()
    at = torch.arange(131072, dtype=torch.float64)[:, None]
    angle = at * 1e4 ** (-torch.arange(16, dtype=torch.float64) / 16)
    want = torch.cat((angle.cos(), angle.sin()), 1)
    # 2^-25 of the rounding to fp32, and the angles' own roundings: 2^17 * 2^-52
    assert ((table - want).abs() <= 2.0 ** -25 + 2.0 ** -33).all()


def test_streams_and_graphs(w4):
    """On a side stream, and captured and replayed on new contents."""
    x = projection(40, 10, 128, "bf16", 16)
    table, (wq, wk) = w4.rope_table(500, 128), weights(128, 17)
    pos = ref.ints(list(range(40)))
    want = w4.qk_norm_rope(x[:, :8], x[:, 8:], pos, table, wq, wk)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        got = w4.qk_norm_rope(x[:, :8], x[:, 8:], pos, table, wq, wk, stream=stream)
        side.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = w4.qk_norm_rope(x[:, :8], x[:, 8:], pos, table, wq, wk)
    for step in range(3):
        x.copy_(projection(40, 10, 128, "bf16", 18 + step))
        pos += 40
        graph.replay()
        again = w4.qk_norm_rope(x[:, :8], x[:, 8:], pos, table, wq, wk)
        assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


def test_many_tokens(w4):
    """More heads than one wave of blocks holds, an odd number of tokens."""
    x = projection(20011, 10, 64, "fp16", 21)
    table, (wq, wk) = w4.rope_table(20011, 64), weights(64, 22)
    pos = torch.arange(20011, dtype=torch.int32, device="cuda")
    got = w4.qk_norm_rope(x[:, :8], x[:, 8:], pos, table, wq, wk)
    for y, z, w in zip(got, (x[:, :8], x[:, 8:]), (wq, wk)):
        check(y, *formula(z, w, pos, table, False))


def test_no_tokens(w4):
    x = projection(0, 3, 64, "bf16", 23)
    got = w4.qk_norm_rope(x[:, :2], x[:, 2:], ref.ints([]), w4.rope_table(4, 64), *weights(64, 24))
    assert got[0].shape == (0, 2, 64) and got[1].shape == (0, 1, 64)


def test_rows_past_32_bits(w4):
    """Token rows a megabyte and more apart, offsets beyond 2^32 bytes."""
    wide = torch.empty((2500, 1 << 20), dtype=torch.bfloat16, device="cuda")
    src = projection(2500, 3, 128, "bf16", 25)
    rows = wide[:, :3 * 128].view(2500, 3, 128)
    rows.copy_(src)
    table, (wq, wk) = w4.rope_table(2500, 128), weights(128, 26)
    pos = torch.arange(2500, dtype=torch.int32, device="cuda")
    want = w4.qk_norm_rope(src[:, :2], src[:, 2:], pos, table, wq, wk)
    got = w4.qk_norm_rope(rows[:, :2], rows[:, 2:], pos, table, wq, wk, q_out=rows[:, :2], k_out=rows[:, 2:])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("heads,kv_heads", [(1024, 1024), (1, 1024), (1024, 3)])
def test_most_heads(w4, heads, kv_heads):
    x = projection(3, heads + kv_heads, 64, "fp16", 27)
    table, (wq, wk), pos = w4.rope_table(9, 64), weights(64, 28), ref.ints([9, 0, 8, 4])[1:]  # 4-byte alignment
    got = w4.qk_norm_rope(x[:, :heads], x[:, heads:], pos, table, wq, wk)
    for y, z, w in zip(got, (x[:, :heads], x[:, heads:]), (wq, wk)):
        check(y, *formula(z, w, pos, table, False))


def test_calls_from_several_threads(w4):
    import threading
    x, table = projection(50, 6, 128, "bf16", 29), w4.rope_table(100, 128)
    pos, (wq, wk) = ref.ints(list(range(50))), weights(128, 30)
    want = w4.qk_norm_rope(x[:, :4], x[:, 4:], pos, table, wq, wk)
    wrong = []

    def work():
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.default_stream())
        for _ in range(50):
            got = w4.qk_norm_rope(x[:, :4], x[:, 4:], pos, table, wq, wk, stream=stream)
            stream.synchronize()
            if not (torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])):
                wrong.append(got)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
