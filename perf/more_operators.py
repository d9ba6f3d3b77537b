"""Cases, plain forms and calls of the operators around the 8-bit cache's attention.

  norm    the norm of every query and key head and the rotation by its position,
          in one pass: what stands between a layer's projection and the cache
  window  attention over the cache where a query sees the last `window` tokens and
          the first `sinks`
  tree    attention of a tree of drafted tokens: a query sees all that was there
          before the drafts, and of the drafts those that its bits name
  keep    after such a tree was checked: the drafts that were accepted move together
          in the cache's pages, and the sequences become shorter by the others

The cache is that of perf/operators.py: e4m3 codes [pages][kv_heads][page][dim], a
fp32 scale for each page and head, value = code * scale; sequence b's token j lies in
page table[b][j // page], slot j % page.

`run` computes them in elementary torch operations in 32 bits where `own` is false,
and through this package where it is true; `exact` in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
F8 = torch.float8_e4m3fn
F8_MAX = 448.0


# --------------------------------------------------------------------------- #
# Cases                                                                         #
# --------------------------------------------------------------------------- #
def listed():
    return [
        # one user's decode step: 40 heads of one token, where latency counts
        dict(name="norm: one token", kind="norm", tokens=1, heads=32, kv_heads=8, dim=128, rot=128,
             rows=4096, interleaved=False, weights=True, dtype="bf16", mix=1),
        # a server's decode step, every sequence at a position of its own, far ones among them
        dict(name="norm: decode batch", kind="norm", tokens=64, heads=64, kv_heads=8, dim=128,
             rot=128, rows=131072, interleaved=False, weights=True, dtype="bf16", mix=2),
        # a model that rotates half of each head, in neighbouring pairs; odd counts
        dict(name="norm: half of a head", kind="norm", tokens=333, heads=28, kv_heads=4, dim=64,
             rot=32, rows=8192, interleaved=True, weights=True, dtype="fp16", mix=3),
        # a prompt: bound by memory
        dict(name="norm: prompt", kind="norm", tokens=8000, heads=32, kv_heads=8, dim=128, rot=128,
             rows=8192, interleaved=False, weights=True, dtype="bf16", mix=4),
        # one chat that has grown past its window
        dict(name="window: one short decode", kind="window", batch=1, q_min=1, q_max=1, kv_min=1500,
             kv_max=1500, heads=32, kv_heads=32, dim=128, page=16, window=512, sinks=4,
             dtype="bf16", mix=5),
        # a server's decode step over long conversations, most of them beyond the window
        dict(name="window: decode batch", kind="window", batch=64, q_min=1, q_max=1, kv_min=500,
             kv_max=32768, heads=64, kv_heads=8, dim=128, page=64, window=4096, sinks=4,
             dtype="bf16", mix=6),
        # pieces of several prompts over what they have cached so far
        dict(name="window: prompt chunks", kind="window", batch=4, q_min=100, q_max=2000,
             kv_min=2000, kv_max=12001, heads=40, kv_heads=40, dim=128, page=32, window=1000,
             sinks=16, dtype="fp16", mix=7),
        # a prompt read in one piece by a layer with a window and no sinks
        dict(name="window: prompt", kind="window", batch=1, q_min=8000, q_max=8000, kv_min=8000,
             kv_max=8000, heads=32, kv_heads=8, dim=128, page=64, window=1024, sinks=0,
             dtype="bf16", mix=8),
        # one user, a wide tree of drafts checked at once over a long conversation
        dict(name="tree: one user", kind="tree", batch=1, q_min=61, q_max=61, kv_min=6000,
             kv_max=6000, heads=32, kv_heads=8, dim=128, page=64, window=0, sinks=0, dtype="bf16",
             mix=9),
        # a batch of small trees: odd group of 7 heads, small dim, ragged
        dict(name="tree: batch", kind="tree", batch=24, q_min=3, q_max=9, kv_min=35, kv_max=3001,
             heads=28, kv_heads=4, dim=64, page=32, window=0, sinks=0, dtype="fp16", mix=10),
        # what follows the one user's tree
        dict(name="keep: one user", kind="keep", batch=1, q_min=61, q_max=61, kv_min=600, kv_max=600,
             kv_heads=8, dim=128, page=64, mix=13),
        # what follows a batch's trees, some of whose pages are given back
        dict(name="keep: batch", kind="keep", batch=64, q_min=9, q_max=33, kv_min=40, kv_max=900,
             kv_heads=8, dim=128, page=16, mix=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["norm", "norm", "window", "window", "window", "chunks", "tree", "tree", "keep"])
    heads, kv_heads, dim = rng.choice([(32, 32, 128), (64, 8, 128), (32, 8, 128), (40, 40, 128),
                                       (28, 4, 64), (20, 20, 64), (16, 1, 128), (14, 2, 64),
                                       (24, 3, 128), (6, 6, 64)])
    page, mix = rng.choice([16, 32, 64, 128]), rng.randrange(1 << 20)
    share = min(1.0, 128 * 8 / (kv_heads * dim))  # a wider cache gets fewer tokens
    dtype = rng.choice(["bf16", "fp16"])
    if kind == "norm":
        # norm and rotation, the rotation alone, the norm alone
        weights, rot = rng.choice([(True, dim), (True, dim), (True, dim // 2), (True, dim // 4 * 3),
                                   (False, dim), (True, 0)])
        tokens = _log_int(rng, 1, 8000 * 40 * 128 // ((heads + kv_heads) * dim))
        return dict(kind="norm", tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim, rot=rot,
                    rows=_log_int(rng, max(tokens, 2000), 131072), weights=weights,
                    interleaved=rng.choice([False, True]), dtype=dtype, mix=mix)
    c = dict(kind=kind, page=page, kv_heads=kv_heads, dim=dim, mix=mix)
    if kind == "keep":
        c["batch"], c["q_max"] = _log_int(rng, 1, 64), rng.randint(2, 64)
        c["q_min"] = rng.randint(1, c["q_max"])
        c["kv_max"] = rng.randint(c["q_max"], max(c["q_max"] + 1, int(900 * share)))
        c["kv_min"] = c["q_max"]
        return c
    c.update(heads=heads, dtype=dtype, kind="window", window=_log_int(rng, 1, 4096),
             sinks=rng.choice([0, 1, 4, 4, 16, 100]))
    if kind == "window":
        c["batch"] = _log_int(rng, 1, 64)
        c["q_min"], c["q_max"] = 1, rng.choice([1, 1, 5])
        c["kv_max"] = _log_int(rng, 17, max(17, int(32768 * 24 * share / c["batch"])))
        c["kv_min"] = rng.randint(1, c["kv_max"])
        c["window"] = min(c["window"], int(180000 * share / c["batch"]))
    elif kind == "chunks":
        c["batch"], c["q_max"] = rng.randint(1, 4), _log_int(rng, 20, 2000)
        c["q_min"] = rng.randint(1, c["q_max"])
        c["kv_max"] = _log_int(rng, c["q_max"], max(c["q_max"], int(12000 * share)))
        c["kv_min"] = rng.randint(c["q_max"], c["kv_max"])
        rows = c["batch"] * c["q_max"] * heads * dim
        c["window"] = max(1, min(c["window"], int(3e10 / rows) - c["sinks"]))
    else:
        c["kind"] = "tree"
        c["batch"], c["q_max"] = _log_int(rng, 1, 32), rng.randint(2, 64)
        c["q_min"] = rng.randint(1, c["q_max"])
        c["kv_max"] = _log_int(rng, 64, max(64, int(65536 * share / c["batch"])))
        c["kv_min"] = rng.randint(64, c["kv_max"])
        if rng.random() < 0.7:  # most trees are checked by layers without a window
            c["window"] = c["sinks"] = 0
    return c


def _lengths(case):
    """(new tokens, tokens with them) of every sequence: made from the case alone,
    log-uniform, the extremes among them."""
    rng = random.Random(case["mix"])
    got = []
    for b in range(case["batch"]):
        q = case["q_max"] if b == 0 else rng.randint(case["q_min"], case["q_max"])
        kv = case["kv_max"] if b == 0 else _log_int(rng, case["kv_min"], case["kv_max"])
        got.append((min(q, kv), kv))
    return got


def _trees(case):
    """For every sequence the bits of its drafts: a draft sees itself and those before it
    on its branch; its parent is any earlier draft, later ones more often."""
    rng = random.Random(case["mix"] + 1)
    out = []
    for n, _ in _lengths(case):
        bits = []
        for i in range(n):
            parent = max(rng.randrange(i), rng.randrange(i)) if i else -1
            bits.append((bits[parent] if i else 0) | 1 << i)
        out.append(bits)
    return out


def _paths(case):
    """For every sequence the drafts that are kept: the first and some that follow, seldom
    none at all."""
    rng = random.Random(case["mix"] + 2)
    out = []
    for n, _ in _lengths(case):
        kept = min(n, _log_int(rng, 2, max(2, n // 2)))
        path = [0] + sorted(rng.sample(range(1, n), kept - 1))
        out.append([] if rng.random() < 0.05 else path)
    return out


def _pages_of(tokens, page):
    return -(-tokens // page)


def work(case):
    kind = case["kind"]
    if kind == "norm":
        elements = case["tokens"] * (case["heads"] + case["kv_heads"]) * case["dim"]
        extra = 4 * case["tokens"] * (case["rot"] + 1) + (8 * case["dim"] if case["weights"] else 0)
        return {"bytes": 4.0 * elements + extra, "flops": 8.0 * elements}
    row = 2 * case["kv_heads"] * case["dim"]  # a token's keys and values, one byte each
    page, lens = case["page"], _lengths(case)
    if kind == "keep":
        moved = pages = left = 0
        for path, (n, kv) in zip(_paths(case), lens):
            at = [(kv - n + i, kv - n + j) for i, j in enumerate(path) if i != j]
            moved += len(at)
            pages += len({j // page for pair in at for j in pair})
            left += _pages_of(kv, page) - _pages_of(kv - n + len(path), page)
        return {"bytes": 2.0 * moved * row + pages * (8.0 * case["kv_heads"] + 4) + 8.0 * left
                + 8.0 * len(lens), "flops": 0.0}
    w, sinks = case["window"] or 1 << 40, case["sinks"]
    held = pages = pairs = 0
    for b, (n, kv) in enumerate(lens):
        base = kv - n
        if kind == "tree":
            for bits in _trees(case)[b]:
                lo = max(0, base + bin(bits).count("1") - w)
                pairs += base - lo + min(sinks, lo) + bin(bits).count("1")
            first = max(0, base + 1 - w)
        else:
            for i in range(n):
                lo = max(0, base + i + 1 - w)
                pairs += base + i + 1 - lo + min(sinks, lo)
            first = max(0, base + 1 - w)
        held += kv - first + min(sinks, first)
        pages += _pages_of(kv, page) - first // page + _pages_of(min(sinks, first // page * page), page)
    new = sum(n for n, _ in lens)
    nbytes = held * row + pages * (8.0 * case["kv_heads"] + 4) + 4.0 * new * case["heads"] * case["dim"]
    return {"bytes": nbytes + (8.0 * new if kind == "tree" else 0.0),
            "flops": 4.0 * pairs * case["heads"] * case["dim"]}


# --------------------------------------------------------------------------- #
# Inputs                                                                        #
# --------------------------------------------------------------------------- #
def _fitting(amax):
    """A power of two in which amax stays within e4m3's 448."""
    return torch.exp2(torch.ceil(torch.log2(amax.clamp_min(2.0 ** -30) / F8_MAX)))


def _fill_cache(k, v, ks, vs, gen):
    """Codes and scales of a pool that has been in use: keys with strong channels,
    values with quiet and loud tokens, in every page."""
    pages, kv_heads, page, dim = k.shape
    dev = k.device
    for what, codes, scales in (("k", k, ks), ("v", v, vs)):
        x = torch.randn((pages, kv_heads, page, dim), generator=gen, device=dev)
        if what == "k":
            x *= 1 + 3 * (torch.rand((kv_heads, 1, dim), generator=gen, device=dev) > 0.95)
        else:
            x *= 0.3 * torch.exp(0.5 * torch.randn((pages, kv_heads, page, 1), generator=gen,
                                                   device=dev))
        s = _fitting(x.abs().amax((-2, -1)))
        x /= s[:, :, None, None]
        codes.copy_(x.clamp_(-F8_MAX, F8_MAX).to(F8))
        scales.copy_(s)
        del x


def _cache_in(buf, pages, kv_heads, page, dim):
    """k, v, k_scale, v_scale as parts of one buffer (made if None), and the buffer."""
    codes, scales = pages * kv_heads * page * dim, (pages * kv_heads * 4 + 15) // 16 * 16
    if buf is None:
        buf = torch.zeros(2 * codes + 2 * scales, dtype=torch.uint8, device="cuda")
    parts = torch.split(buf, [codes, codes, scales, scales])
    k, v = (x.view(F8).view(pages, kv_heads, page, dim) for x in parts[:2])
    ks, vs = (x[:pages * kv_heads * 4].view(torch.float32).view(pages, kv_heads) for x in parts[2:])
    return k, v, ks, vs, buf


def _rotations(rows, rot, dev):
    """cos and sin of every position's angles, [rows, rot], made once for a model: the
    angle of pair j is position * 10000 ** (-2 j / rot), far positions and all in 64 bits."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
    angle = torch.arange(rows, dtype=torch.float64, device=dev)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 1000003 + case["mix"])
    rng = random.Random(seed * 7919 + case["mix"])
    kind, dim, kv_heads = case["kind"], case["dim"], case["kv_heads"]
    st = dict(kind=kind)
    if kind == "norm":
        _prepare_norm(case, st, gen, rng, dev)
        return st
    page = st["page"] = case["page"]
    order = list(range(case["batch"]))
    rng.shuffle(order)
    lens = [_lengths(case)[b] for b in order]
    kv = [n for _, n in lens]
    cu = np.cumsum([0] + [q for q, _ in lens]).astype(np.int32)
    need = sum(_pages_of(n, page) for n in kv)
    pages, width = need + need // 8 + 1, _pages_of(max(kv), page)
    numbers = rng.sample(range(pages), need)  # the sequences' pages lie scattered over the pool
    table, at = np.full((len(kv), width), -1, np.int32), 0
    for b, n in enumerate(kv):
        m = _pages_of(n, page)
        table[b, :m] = numbers[at:at + m]
        at += m
    table = torch.from_numpy(table).to(dev)
    st["k"], st["v"], st["k_scale"], st["v_scale"], buf = _cache_in(None, pages, kv_heads, page, dim)
    _fill_cache(st["k"], st["v"], st["k_scale"], st["v_scale"], gen)
    st["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device=dev)
    st["cu_q"] = torch.from_numpy(cu).to(dev)
    st["max_q"], st["max_kv"] = max(q for q, _ in lens), max(kv)
    if kind == "keep":
        # a pass changes the cache and the bookkeeping, so it begins with copies of both
        st["held"] = buf
        st["k"], st["v"], st["k_scale"], st["v_scale"], st["buf"] = _cache_in(
            buf.clone(), pages, kv_heads, page, dim)
        refs = torch.zeros(pages, dtype=torch.int32, device=dev)
        refs[torch.tensor(numbers, device=dev)] = 1
        st["book"] = torch.cat([refs, st["kv_lens"], table.reshape(-1)])
        st["table"], st["pages"], st["slots"], st["width"] = table, pages, len(kv), width
        paths = [_paths(case)[b] for b in order]
        rows = [p + [-1] * (q - len(p)) for p, (q, _) in zip(paths, lens)]
        st["path"] = torch.tensor(sum(rows, []), dtype=torch.int32, device=dev)
        st["drop"] = torch.tensor([q - len(p) for p, (q, _) in zip(paths, lens)], dtype=torch.int32,
                                  device=dev)
    else:
        st["table"] = table
        # what the fused projection of a layer gives: queries, keys and values side by side
        qkv = torch.randn((int(cu[-1]), case["heads"] + 2 * kv_heads, dim), generator=gen, device=dev)
        st["q"] = (1.5 * qkv).to(DT[case["dtype"]])[:, :case["heads"]]
        st["scale"], st["window"], st["sinks"] = 1.0 / math.sqrt(dim), case["window"], case["sinks"]
        if kind == "tree":
            bits = sum((_trees(case)[b] for b in order), [])
            st["tree"] = torch.from_numpy(np.array(bits, np.uint64).view(np.int64)).to(dev)
    st["cache"] = _handle(st)
    return st


def _prepare_norm(case, st, gen, rng, dev):
    n, h, hk, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
    # a projection's output: heads of different loudness, a few strong channels
    qkv = torch.randn((n, h + 2 * hk, d), generator=gen, device=dev)
    qkv *= torch.exp(torch.randn((1, h + 2 * hk, 1), generator=gen, device=dev))
    qkv *= 1 + 5 * (torch.rand((1, h + 2 * hk, d), generator=gen, device=dev) > 0.95)
    st["q"], st["k"], _ = torch.split(qkv.to(DT[case["dtype"]]), [h, hk, hk], dim=1)
    st["q_weight"], st["k_weight"] = (
        (1 + 0.3 * torch.randn(d, generator=gen, device=dev) if case["weights"] else None)
        for _ in range(2))
    if n > case["rows"] // 4:  # a prompt, its tokens one after the other
        start = rng.randint(0, case["rows"] - n)
        at = list(range(start, start + n))
    else:
        at = [rng.randrange(case["rows"]) for _ in range(n)]
    st["positions"] = torch.tensor(at, dtype=torch.int32, device=dev)
    st["rotations"] = _rotations(case["rows"], case["rot"], dev) if case["rot"] else None
    st["interleaved"], st["eps"] = case["interleaved"], 1e-6


def _handle(st):
    """The cache as a program keeps it: the framework's object over the four buffers."""
    if not own:
        return None
    import int4_weight_only_repack_gb300 as w4
    return w4.KV8Cache(st["k"], st["v"], st["k_scale"], st["v_scale"])


# --------------------------------------------------------------------------- #
# One pass                                                                      #
# --------------------------------------------------------------------------- #
def run(state):
    if own:
        return _run_own(state)
    return {"norm": _plain_norm, "window": _plain_attend, "tree": _plain_attend,
            "keep": _plain_keep}[state["kind"]](state)


def _run_own(st):
    import int4_weight_only_repack_gb300 as w4
    if st["kind"] == "norm":
        return w4.qk_norm_rope(st["q"], st["k"], st["positions"], st["rotations"], st["q_weight"],
                               st["k_weight"], eps=st["eps"], interleaved=st["interleaved"])
    if st["kind"] == "keep":
        refs, lens, table = _begin(st)
        w4.kv8_keep(st["cache"], table, lens, st["cu_q"], st["path"], st["max_q"])
        w4.kv8_shorten(w4.KV8Pool(refs, table, lens, st["page"]), st["drop"])
        return [refs, lens, table, st["k"], st["v"], st["k_scale"], st["v_scale"]]
    how = dict(window=st["window"], sinks=st["sinks"]) if st["window"] else {}
    if st["kind"] == "tree":
        how["tree"] = st["tree"]
    return w4.kv8_attention(st["q"], st["cache"], st["table"], st["kv_lens"], st["cu_q"],
                            st["max_q"], st["max_kv"], scale=st["scale"], **how)


def _begin(st):
    """Puts the cache back and returns refs, lengths and table of a copy of the bookkeeping."""
    st["buf"].copy_(st["held"])
    book = st["book"].clone()
    p, s = st["pages"], st["slots"]
    return book[:p], book[p:p + s], book[p + s:].view(s, st["width"])


def _plain_norm(st):
    out = []
    for x, w in ((st["q"], st["q_weight"]), (st["k"], st["k_weight"])):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + st["eps"]) * w
        if st["rotations"] is not None:
            cs = st["rotations"][st["positions"].long()][:, None]
            rot = cs.shape[-1]
            c, s = cs[..., :rot // 2], cs[..., rot // 2:]
            if st["interleaved"]:
                a, b = y[..., 0:rot:2], y[..., 1:rot:2]
                turned = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
            else:
                a, b = y[..., :rot // 2], y[..., rot // 2:rot]
                turned = torch.cat([a * c - b * s, b * c + a * s], -1)
            y = torch.cat([turned, y[..., rot:]], -1)
        out.append(y.to(x.dtype))
    return out


def _plain_attend(st):
    q, lens, cu, page = st["q"], st["kv_lens"].long(), st["cu_q"].long(), st["page"]
    b, heads, d = lens.shape[0], q.shape[1], q.shape[2]
    hk = st["k"].shape[1]
    group = heads // hk
    row = torch.arange(st["max_q"], device=q.device)
    n = (cu[1:] - cu[:-1])[:, None]
    base = lens[:, None] - n
    real = row < n
    tok = (cu[:-1, None] + row).clamp_max(max(q.shape[0] - 1, 0))
    # the tokens that some query of a sequence sees: the sinks, then the window of the first
    sinks = st["sinks"]
    window = st["window"] or st["max_kv"] + st["max_q"]
    first = (base + 1 - window).clamp_min(0)
    length = min(st["max_kv"], sinks + window + st["max_q"])
    at = torch.arange(length, device=q.device).expand(b, length)
    j = torch.where(at < torch.minimum(first, torch.full_like(first, sinks)), at,
                    at + (first - sinks).clamp_min(0))
    held = j < lens[:, None]
    j0 = torch.where(held, j, 0)
    p = st["table"].long().gather(1, j0 // page).clamp_min(0)
    k, v = ((codes.view(torch.uint8)[p, :, j0 % page].view(F8).float() * scales[p][..., None])
            .permute(0, 2, 1, 3) for codes, scales in ((st["k"], st["k_scale"]),
                                                       (st["v"], st["v_scale"])))
    x = q[tok].float().view(b, -1, hk, group, d).permute(0, 2, 3, 1, 4).reshape(b, hk, -1, d)
    s = torch.matmul(x, k.transpose(2, 3)).view(b, hk, group, -1, length) * st["scale"]
    # what query i sees: seen [batch, query, token]
    j, base = j[:, None], base[:, :, None]
    if st["kind"] == "tree":
        bits = st["tree"][tok]
        count = (bits[:, :, None] >> torch.arange(64, device=q.device) & 1).sum(-1, keepdim=True)
        low = count + base - window
        draft = (bits[:, :, None] >> (j - base).clamp(0, 63) & 1).bool()
        seen = torch.where(j < base, (j >= low) | (j < sinks), draft)
    else:
        last = base + row[None, :, None]
        seen = (j <= last) & ((j > last - window) | (j < sinks))
    seen = (seen & held[:, None] & real[:, :, None])[:, None, None]
    s = torch.where(seen, s, -math.inf)
    top = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(torch.isinf(top), 0.0, top))
    total = e.sum(-1, keepdim=True)
    v = torch.where(held[:, None, :, None], v, 0.0)
    o = torch.matmul(e.view(b, hk, -1, length), v).view(b, hk, group, -1, d)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(b, -1, heads, d)
    out = torch.zeros((q.shape[0] + 1, heads, d), device=q.device)
    out[torch.where(real, tok, q.shape[0])] = o  # rows past a sequence's own go to a spare row
    return out[:-1].to(q.dtype)


def _plain_keep(st):
    refs, lens, table = _begin(st)
    page, cu, path = st["page"], st["cu_q"].long(), st["path"].long()
    t = torch.arange(path.shape[0], device=path.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    i = t - cu[b]
    base = lens.long()[b] - (cu[b + 1] - cu[b])
    # moves of tokens; a page that gets some keeps its scale only if other tokens stay in it
    move = torch.nonzero((path >= 0) & (path != i))[:, 0]
    stay = torch.nonzero(path == i)[:, 0]
    from_j, to_j = base[move] + path[move], base[move] + i[move]
    from_p = table[b[move], from_j // page].long()
    to_p = table[b[move], to_j // page].long()
    stay_p = table[b[stay], (base[stay] + i[stay]) // page].long()
    partly = base[move] > to_j // page * page  # it holds tokens from before the drafts
    kept = torch.zeros(st["pages"], dtype=torch.bool, device=path.device)
    kept[stay_p] = True
    kept[to_p[partly]] = True
    gets = torch.zeros_like(kept)
    gets[to_p] = True
    # the slots of those pages whose tokens stay: those before the drafts, and unmoved drafts
    slot = torch.arange(page, device=path.device)
    fixed = torch.zeros((st["pages"], page), dtype=torch.bool, device=path.device)
    fixed[to_p] = slot < (base[move] - to_j // page * page)[:, None]
    fixed[stay_p, (base[stay] + i[stay]) % page] = True
    fixed &= gets[:, None]
    for codes, scales in ((st["k"], st["k_scale"]), (st["v"], st["v_scale"])):
        now = torch.where(gets[:, None] & ~kept[:, None], 0.0, scales)
        now.index_reduce_(0, to_p, scales[from_p], "amax")
        raw = codes.view(torch.uint8)
        moved = raw[from_p, :, from_j % page].view(F8).float()
        moved = (moved * (scales[from_p] / now[to_p])[..., None]).to(F8)
        again = (codes.float() * (scales / now)[:, :, None, None]).to(F8).view(torch.uint8)
        raw.copy_(torch.where(fixed[:, None, :, None], again, raw))
        raw[to_p, :, to_j % page] = moved.view(torch.uint8)
        scales.copy_(now)
    # the sequences get shorter; pages beyond their ends lose a reference
    col = torch.arange(st["width"], device=path.device)
    have = (lens + page - 1) // page
    lens -= st["drop"]
    want = (lens + page - 1) // page
    gone = (col >= want[:, None]) & (col < have[:, None])
    refs.index_add_(0, torch.where(gone, table, 0).long().reshape(-1),
                    -gone.to(torch.int32).reshape(-1))
    table.copy_(torch.where(gone, -1, table))
    return [refs, lens, table, st["k"], st["v"], st["k_scale"], st["v_scale"]]


# --------------------------------------------------------------------------- #
# The definitions in 64 bits                                                    #
# --------------------------------------------------------------------------- #
def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _exact_norm, "window": _exact_attend, "tree": _exact_attend,
            "keep": _exact_keep}[case["kind"]](st)


def _exact_norm(st):
    out = []
    for x, w in ((st["q"], st["q_weight"]), (st["k"], st["k_weight"])):
        y = x.double()
        if w is not None:
            y = y / torch.sqrt(y.square().sum(-1, keepdim=True) / y.shape[-1] + st["eps"]) * w.double()
        if st["rotations"] is not None:
            cs = st["rotations"].double()[st["positions"].long()]
            half = cs.shape[1] // 2
            turn = torch.complex(cs[:, :half], cs[:, half:])[:, None]
            first = (torch.arange(half, device=x.device) * 2 if st["interleaved"]
                     else torch.arange(half, device=x.device))
            second = first + (1 if st["interleaved"] else half)
            z = torch.complex(y[..., first], y[..., second]) * turn
            y = y.index_copy(-1, first, z.real).index_copy(-1, second, z.imag)
        out.append(y)
    return out


def _exact_attend(st):
    q, page = st["q"].double(), st["page"]
    group = q.shape[1] // st["k"].shape[1]
    out = torch.zeros_like(q)
    cu, lens = st["cu_q"].tolist(), st["kv_lens"].tolist()
    for b, n in enumerate(lens):
        ids, m = st["table"][b, :_pages_of(n, page)].long(), cu[b + 1] - cu[b]
        j, p = torch.arange(n, device=q.device), torch.arange(n - m, n, device=q.device)[:, None]
        if st["kind"] == "tree":
            sees = torch.zeros((m, n), dtype=torch.bool, device=q.device)
            for i, bits in enumerate(st["tree"][cu[b]:cu[b + 1]].tolist()):
                on = [d for d in range(m) if bits >> d & 1]
                low = n - m + len(on) - st["window"] if st["window"] else 0
                sees[i, :min(st["sinks"], n - m)] = True
                sees[i, min(max(0, low), n - m):n - m] = True
                sees[i, [n - m + d for d in on]] = True
        else:
            sees = (j <= p) & ((j > p - st["window"]) | (j < st["sinks"]))
        for g in range(st["k"].shape[1]):
            k, v = ((c.view(torch.uint8)[ids, g].view(F8).double() * s[ids, g].double()[:, None, None])
                    .reshape(-1, q.shape[2])[:n] for c, s in ((st["k"], st["k_scale"]),
                                                             (st["v"], st["v_scale"])))
            for h in range(g * group, (g + 1) * group):
                s = (q[cu[b]:cu[b + 1], h] @ k.T) * st["scale"]
                out[cu[b]:cu[b + 1], h] = torch.softmax(s.masked_fill_(~sees, -math.inf), -1) @ v
    return out


def _round_e4m3(x):
    """The e4m3 value nearest to each element, ties to the even code, saturated at 448."""
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -60))).clamp_min(-6)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-F8_MAX, F8_MAX)


def _exact_keep(st):
    """Draft by draft, page by page, as the definition says."""
    page, cu, path = st["page"], st["cu_q"].tolist(), st["path"].tolist()
    lens, table, drop = st["kv_lens"].tolist(), st["table"].tolist(), st["drop"].tolist()
    got = []
    for codes, scales in ((st["k"], st["k_scale"]), (st["v"], st["v_scale"])):
        new, now = codes.double(), scales.double()
        for b, n in enumerate(lens):
            base = n - (cu[b + 1] - cu[b])
            pairs = [(base + i, base + d) for i, d in enumerate(path[cu[b]:cu[b + 1]]) if d >= 0]
            for col in sorted({to // page for to, of in pairs if to != of}):
                p, here = table[b][col], [(to, of) for to, of in pairs if to // page == col]
                stays = list(range(col * page, base)) + [to for to, of in here if to == of]
                come = [(to, of) for to, of in here if to != of]
                s = [scales[table[b][of // page]] for _, of in come] + [scales[p]] * bool(stays)
                now[p] = torch.stack(s).amax(0).double()
                for to, of in [(j, j) for j in stays] + come:
                    source = table[b][of // page]
                    ratio = scales[source].double() / now[p]
                    new[p, :, to % page] = _round_e4m3(codes[source, :, of % page].double() * ratio[:, None])
        got.append((new, now))
    refs, left = st["book"][:st["pages"]].tolist(), [n - d for n, d in zip(lens, drop)]
    for b, n in enumerate(lens):
        for col in range(_pages_of(left[b], page), _pages_of(n, page)):
            refs[table[b][col]] -= 1
            table[b][col] = -1
    whole = [torch.tensor(x, dtype=torch.int32) for x in (refs, left, table)]
    return whole + [got[0][0], got[1][0], got[0][1], got[1][1]]
