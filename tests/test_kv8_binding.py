"""What the 8-bit cache's binding hands to the library, and what it refuses, with a
stand-in for the library (no GPU)."""
import contextlib
import ctypes
import weakref

import pytest
import torch

import int4_weight_only_repack_gb300 as w4

F8 = torch.float8_e4m3fn


class Calls:
    """Takes any call, remembers the arguments by entry point, returns `status`."""

    def __init__(self, status=0):
        self.seen, self.status = {}, status

    def __getattr__(self, name):
        def call(*args):
            self.seen.setdefault(name, []).append(args)
            return 512 if name.endswith("_size") else self.status
        return call


@pytest.fixture
def fake(monkeypatch):
    calls = Calls()
    monkeypatch.setattr(w4, "_LIB", calls)
    monkeypatch.setattr(w4, "_KV8_SIZES", {})  # (its sizes are not the library's)
    monkeypatch.setattr(w4, "_KV8_SPACES", {})
    return calls


def cache(pages=8, heads=2, page=16, dim=64):
    codes = lambda: torch.zeros((pages, heads, page, dim), dtype=torch.uint8).view(F8)  # noqa: E731
    return w4.KV8Cache(codes(), codes(), torch.ones(pages, heads), torch.ones(pages, heads))


def ints(*x):
    return torch.tensor(x, dtype=torch.int32)


@pytest.mark.parametrize("table", [
    torch.zeros((3, 9), dtype=torch.int32)[:, :4], torch.zeros((3, 9), dtype=torch.int32)[:, 5:],
    torch.zeros((3, 9), dtype=torch.int32)[:, :1], torch.zeros((4, 3), dtype=torch.int32).t(),
    torch.zeros((1, 4), dtype=torch.int32).expand(3, 4)])
def test_a_pool_refuses_a_part_of_a_table(fake, table):
    """Its kernels write whole rows: they would write past the columns given."""
    with pytest.raises(ValueError):
        w4.KV8Pool(torch.zeros(8, dtype=torch.int32), table, ints(0, 0, 0), 16)
    w4.KV8Pool(torch.zeros(8, dtype=torch.int32), table.contiguous(), ints(0, 0, 0), 16)


@pytest.mark.parametrize("cut", [slice(0, 4), slice(5, 9), slice(3, 4)])
def test_columns_of_a_table_are_handed_over_as_rows_of_their_length(fake, monkeypatch, cut):
    """append and attention must not look past the columns given."""
    rows = []

    def keep(table, stride, batch):
        rows.append((list((ctypes.c_int * (batch * stride)).from_address(table)), stride))

    wide = torch.arange(27, dtype=torch.int32).view(3, 9)
    monkeypatch.setattr(fake, "w4_kv8_append", lambda *a: keep(a[5], a[6], 3) or 0, raising=False)
    monkeypatch.setattr(fake, "w4_kv8_attention", lambda *a: keep(a[3], a[4], 3) or 0, raising=False)
    monkeypatch.setattr(w4, "_one_gpu", lambda *_: None)  # the addresses are read here
    c, x = cache(), torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    args = (c, wide[:, cut], ints(1, 1, 1), ints(0, 1, 2, 3), 1)
    w4.kv8_append(x, x, *args)
    w4.kv8_attention(x, *args, 16, workspace=torch.zeros(512, dtype=torch.uint8))
    want = (wide[:, cut].reshape(-1).tolist(), wide[:, cut].shape[1])
    assert rows == [want, want]


def test_a_replaced_workspace_stays(monkeypatch):
    """A captured graph may hold its address. What is kept stays within a bound."""
    made = []

    def empty(n, dtype, device):
        made.append((weakref.ref(t := torch.zeros(n, dtype=dtype)), n))
        return t

    monkeypatch.setattr(w4, "_WORKSPACES", {})
    monkeypatch.setattr(w4, "_KV8_SPACES", {})
    monkeypatch.setattr(torch, "empty", empty)
    first = w4._space(1000, 0, None, None)
    assert first[1] >= 1000 and w4._space(900, 0, None, None) == first
    for n in range(1100, 40000, 100):
        address, size = w4._space(n, 0, None, None)
        assert size >= n
        w4.gemm_workspace(n, torch.device("cuda", 0))
    assert all(ref() is not None for ref, _ in made)
    assert sum(n for _, n in made) <= 3 * made[-1][1]
    assert address == made[-1][0]().data_ptr()


class On:
    """A tensor that says it is on GPU `index`."""

    def __init__(self, x, index=0):
        self.x, self.index = x, index

    def get_device(self):
        return self.index

    def __getattr__(self, name):
        return getattr(self.x, name)


def calls(c, pool, x, table, lens, cu, more=None):
    """Every call of the binding that hands tensors over, by its tensors' names."""
    return [lambda: w4.kv8_append(x, x, c, table, lens, cu, 1),
            lambda: w4.kv8_attention(x, c, table, lens, cu, 1, 16, out=x, workspace=more),
            lambda: w4.kv8_reserve(pool, lens), lambda: w4.kv8_fork(pool, lens, lens),
            lambda: w4.kv8_free(pool, lens), lambda: w4.kv8_copy_pages(c, lens, lens)]


def test_tensors_that_are_not_on_the_gpu_are_refused(fake, monkeypatch):
    """Their addresses would be followed on the GPU."""
    monkeypatch.setattr(w4, "_CURRENT_DEVICE", lambda: 0)
    monkeypatch.setattr(w4, "_on", lambda *_: None)
    monkeypatch.setattr(w4, "_space", lambda *_: (0, 1 << 30))
    c, pool = cache(), w4.KV8Pool(ints(0, 0), torch.zeros((3, 4), dtype=torch.int32), ints(0, 0, 0), 16)
    x, table = torch.zeros((3, 2, 64), dtype=torch.bfloat16), torch.zeros((3, 4), dtype=torch.int32)
    lens, cu, ws = ints(1, 1, 1), ints(0, 1, 2, 3), torch.zeros(512, dtype=torch.uint8)
    for call in calls(c, pool, x, table, lens, cu, ws) + [lambda: w4.kv8_compact(pool)]:  # all on the CPU
        with pytest.raises(ValueError):
            call()
    c._device = pool._device = 0
    gpu = [On(t) for t in (x, table, lens, cu, ws)]
    for call in calls(c, pool, *gpu):
        call()
    assert len([name for name in fake.seen if not name.endswith("_size")]) == 6
    for wrong in (-1, 1):
        for i in range(5):
            args = [On(t.x, wrong if i == j else 0) for j, t in enumerate(gpu)]
            uses = {0: (0, 1), 1: (0, 1), 2: range(6), 3: (0, 1), 4: (1,)}[i]
            for j, call in enumerate(calls(c, pool, *args)):
                if j in uses:
                    with pytest.raises(ValueError):
                        call()
    monkeypatch.setattr(w4, "_CURRENT_DEVICE", lambda: 1)  # the launch would go to GPU 1
    for call in calls(c, pool, *gpu):
        with pytest.raises(ValueError):
            call()


def test_a_handle_s_tensors_are_on_one_device(fake):
    c = cache()
    meta = torch.empty(c.k_scale.shape, device="meta")
    with pytest.raises(ValueError):
        w4.KV8Cache(c.k, c.v, c.k_scale, meta)
    table = torch.zeros((3, 4), dtype=torch.int32)
    with pytest.raises(ValueError):
        w4.KV8Pool(ints(0), table, ints(0, 0, 0), 16, torch.empty(1, dtype=torch.int32, device="meta"))
    with pytest.raises(ValueError):
        w4.KV8Pool(ints(0), table, torch.empty(3, dtype=torch.int32, device="meta"), 16)


def test_a_handle_s_attributes_cannot_be_set(fake):
    """Its addresses stay those of the tensors it was made of."""
    c = cache()
    pool = w4.KV8Pool(ints(0, 0), torch.zeros((3, 4), dtype=torch.int32), ints(0, 0, 0), 16)
    for handle, names in ((c, "k v k_scale v_scale num_pages page_size kv_heads head_dim"),
                          (pool, "refs table lens status page_size")):
        for name in names.split():
            was = getattr(handle, name)
            with pytest.raises(AttributeError):
                setattr(handle, name, was)
            assert getattr(handle, name) is was
    pool.lens[0], c.k_scale[1] = 5, 2.0  # their contents can
    c.layer = 7
    assert c.layer == 7


def test_a_workspace_with_holes_is_refused(fake, monkeypatch):
    """Its bytes are counted as if they were adjacent."""
    monkeypatch.setattr(w4, "_one_gpu", lambda *_: None)
    x, table = torch.zeros((3, 2, 64), dtype=torch.bfloat16), torch.zeros((3, 4), dtype=torch.int32)
    room = torch.zeros(1, dtype=torch.uint8).expand(1 << 20)
    with pytest.raises(ValueError):
        w4.kv8_attention(x, cache(), table, ints(1, 1, 1), ints(0, 1, 2, 3), 1, 16, workspace=room)


def test_a_call_s_outputs_are_made_on_its_stream(fake, monkeypatch):
    """On the current stream they could be memory that work still running there uses."""
    where, made, recorded = [None], [], []

    @contextlib.contextmanager
    def on_stream(stream, index):
        where.append(stream)
        yield
        where.pop()

    def make(real):
        def call(*args, **kw):
            made.append(where[-1])
            return real(*args, **kw)
        return call

    monkeypatch.setattr(w4, "_on_stream", on_stream)
    monkeypatch.setattr(w4, "_one_gpu", lambda *_: None)
    monkeypatch.setattr(w4, "_on", lambda *_: None)
    monkeypatch.setattr(w4, "_space", lambda *_: (0, 1 << 30))
    monkeypatch.setattr(torch, "empty", make(torch.empty))
    monkeypatch.setattr(torch, "empty_like", make(torch.empty_like))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *_: "current")
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda x, s: recorded.append(s))
    c, pool = cache(), w4.KV8Pool(ints(0, 0), torch.zeros((3, 4), dtype=torch.int32), ints(0, 0, 0), 16)
    x, table = torch.zeros((3, 2, 64), dtype=torch.bfloat16), torch.zeros((3, 4), dtype=torch.int32)
    for stream in (None, "side"):
        w4.kv8_attention(x, c, table, ints(1, 1, 1), ints(0, 1, 2, 3), 1, 16, stream=stream)
        w4.kv8_fork(pool, ints(0), ints(1), stream=stream)
        w4.kv8_compact(pool, stream=stream)
    assert made == [None] * 3 + ["side"] * 3 and recorded == ["current"] * 3
