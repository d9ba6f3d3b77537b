"""Cases, plain forms and calls of the 8-bit key-value cache operators.

A cache holds keys and values as e4m3 codes in pages of `page` tokens,
[pages][kv_heads][page][dim], with one fp32 scale for each page and head
([pages][kv_heads], keys and values apart): value = code * scale. Sequence b's
token j lives in page table[b][j // page], slot j % page. Three operators:

  attend  softmax(scale * q . k) v of new tokens over their sequence's cache
  append  quantise new keys and values into the cache
  pages   the cache's bookkeeping: fork sequences (sharing full pages, copying
          the last partial one), compact the live pages to the front, free
          sequences and reserve pages for new tokens

`run` computes them in elementary torch operations in 32 bits where `own` is
false, and through this package where it is true; `exact` in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
F8 = torch.float8_e4m3fn
F8_MAX = 448.0
MIN_EXP = -40  # smallest page scale an append gives: 2^-40


# --------------------------------------------------------------------------- #
# Cases                                                                         #
# --------------------------------------------------------------------------- #
def listed():
    return [
        # one user's chat turn being decoded: the shortest call, where latency counts
        dict(name="attend: one short decode", kind="attend", batch=1, q_min=1, q_max=1, kv_min=137,
             kv_max=137, heads=32, kv_heads=32, dim=128, page=16, causal=True, dtype="bf16", idle=0,
             mix=1),
        # a server's decode step: ragged lengths, grouped heads, two slots idle
        dict(name="attend: decode batch", kind="attend", batch=64, q_min=1, q_max=1, kv_min=60,
             kv_max=4096, heads=64, kv_heads=8, dim=128, page=64, causal=True, dtype="bf16", idle=2,
             mix=2),
        # two users with a whole book in the context: few rows, a very long axis
        dict(name="attend: long decode", kind="attend", batch=2, q_min=1, q_max=1, kv_min=130001,
             kv_max=131072, heads=64, kv_heads=8, dim=128, page=64, causal=True, dtype="fp16",
             idle=0, mix=3),
        # a few drafted tokens verified at once: odd group of 7 heads, small dim, ragged
        dict(name="attend: drafted tokens", kind="attend", batch=24, q_min=1, q_max=6, kv_min=35,
             kv_max=3001, heads=28, kv_heads=4, dim=64, page=32, causal=True, dtype="fp16", idle=1,
             mix=4),
        # a prompt read in one piece: bound by the products
        dict(name="attend: prompt", kind="attend", batch=1, q_min=8000, q_max=8000, kv_min=8000,
             kv_max=8000, heads=32, kv_heads=8, dim=128, page=64, causal=True, dtype="bf16", idle=0,
             mix=5),
        # chunks of several prompts over what they have cached so far
        dict(name="attend: prompt chunks", kind="attend", batch=6, q_min=100, q_max=777, kv_min=800,
             kv_max=6001, heads=40, kv_heads=40, dim=128, page=64, causal=True, dtype="fp16", idle=0,
             mix=6),
        # a decoder's prompts attending to encoder states of another length, no causal mask
        dict(name="attend: encoder states", kind="attend", batch=8, q_min=30, q_max=200, kv_min=400,
             kv_max=1500, heads=20, kv_heads=20, dim=64, page=128, causal=False, dtype="bf16",
             idle=1, mix=7),
        # the same decode step's new token of every sequence
        dict(name="append: decode batch", kind="append", batch=64, q_min=1, q_max=1, kv_min=60,
             kv_max=4096, heads=64, kv_heads=8, dim=128, page=64, dtype="bf16", idle=2, mix=8),
        # whole prompts and prompt chunks written at once, ragged, starting inside pages
        dict(name="append: prompts", kind="append", batch=8, q_min=1000, q_max=8192, kv_min=1000,
             kv_max=12000, heads=32, kv_heads=8, dim=128, page=64, dtype="bf16", idle=0, mix=9),
        # sixteen sequences each continued in four ways
        dict(name="pages: fork", kind="fork", batch=16, children=64, kv_min=50, kv_max=2000,
             kv_heads=8, dim=128, page=64, pages=1024, mix=10),
        # sequences end and others grow: the bookkeeping of a step alone
        dict(name="pages: free and reserve", kind="turnover", batch=512, leave=37, grow=1, kv_min=30,
             kv_max=4000, page=64, pages=32768, mix=11),
        # a pool that has become scattered is moved to the front: bound by the copy
        dict(name="pages: compact", kind="compact", batch=100, kv_min=500, kv_max=4000, kv_heads=8,
             dim=128, page=64, pages=8000, mix=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["decode", "decode", "draft", "prompt", "chunks", "encoder", "append",
                       "append", "fork", "compact", "turnover"])
    heads, kv_heads, dim = rng.choice([(32, 32, 128), (64, 8, 128), (32, 8, 128), (40, 40, 128),
                                       (28, 4, 64), (20, 20, 64), (16, 1, 128), (14, 2, 64),
                                       (24, 3, 128), (6, 6, 64)])
    page = rng.choice([16, 32, 64, 128])
    c = dict(kind="attend", heads=heads, kv_heads=kv_heads, dim=dim, page=page, causal=True,
             dtype=rng.choice(["bf16", "fp16"]), idle=rng.choice([0, 0, 1, 3]),
             mix=rng.randrange(1 << 20))
    top = 128 * 8  # kv_heads * dim of the listed cases: a wider cache gets fewer tokens
    share = min(1.0, top / (kv_heads * dim))
    if kind == "decode":
        c["batch"] = _log_int(rng, 1, 256)
        c["kv_max"] = _log_int(rng, 1, max(1, int(131072 * 2 * share / c["batch"])))
        c["kv_min"] = _log_int(rng, 1, c["kv_max"])
        c["q_min"] = c["q_max"] = 1
    elif kind == "draft":
        c["batch"], c["q_min"], c["q_max"] = _log_int(rng, 1, 64), 1, rng.randint(2, 16)
        c["kv_max"] = _log_int(rng, 17, max(17, int(65536 * share / c["batch"])))
        c["kv_min"] = rng.randint(17, c["kv_max"])
    elif kind == "prompt":
        c["batch"] = 1
        c["q_max"] = c["kv_max"] = _log_int(rng, 17, min(8000, int(8000 * math.sqrt(32 / heads))))
        c["q_min"] = c["kv_min"] = c["q_max"]
    elif kind == "chunks":
        c["batch"], c["q_max"] = rng.randint(2, 8), _log_int(rng, 20, 900)
        c["kv_max"] = _log_int(rng, c["q_max"], max(c["q_max"], 6001 * 6 // c["batch"]))
        c["q_min"] = rng.randint(1, c["q_max"])
        c["kv_min"] = rng.randint(c["q_max"], c["kv_max"])
    elif kind == "encoder":
        c["causal"] = False
        c["batch"], c["q_max"] = rng.randint(1, 16), _log_int(rng, 1, 300)
        c["q_min"] = rng.randint(1, c["q_max"])
        c["kv_max"] = _log_int(rng, 1, 1500)
        c["kv_min"] = rng.randint(1, c["kv_max"])
    elif kind == "append":
        c["kind"] = "append"
        c["batch"] = _log_int(rng, 1, 128)
        c["q_max"] = _log_int(rng, 1, max(1, int(30000 * share / c["batch"])))
        c["q_min"] = rng.randint(1, c["q_max"])
        c["kv_max"] = max(c["q_max"], _log_int(rng, 1, max(1, int(100000 * share / c["batch"]))))
        c["kv_min"] = c["q_max"]
        del c["causal"]
    else:
        c = dict(kind=kind, page=page, mix=c["mix"], pages=_log_int(rng, 300, 8000))
        c["batch"] = _log_int(rng, 1, 64)
        c["pages"] = max(c["pages"], 16 * c["batch"])
        c["kv_max"] = max(2, int(0.4 * c["pages"] // c["batch"] * page))
        c["kv_min"] = rng.randint(1, c["kv_max"])
        if kind == "turnover":
            c["leave"], c["grow"] = rng.randint(0, c["batch"]), rng.choice([1, 3, 2 * page + 1])
            return c
        while kv_heads * dim * page * c["pages"] > 8 * 128 * 64 * 8000:
            page //= 2
            c["page"] = page
            c["kv_max"] = max(2, c["kv_max"] // 2)
            c["kv_min"] = min(c["kv_min"], c["kv_max"])
        c["kv_heads"], c["dim"] = kv_heads, dim
        if kind == "fork":
            c["children"] = min(_log_int(rng, 1, 128), int(0.4 * c["pages"]))
    return c


def _lengths(case):
    """(new tokens, tokens with them) of every sequence of an attend or append
    case: made from the case alone, log-uniform, the extremes among them."""
    rng = random.Random(case["mix"])
    got = []
    for b in range(case["batch"]):
        q = case["q_max"] if b == 0 else rng.randint(case["q_min"], case["q_max"])
        kv = case["kv_max"] if b == 0 else _log_int(rng, case["kv_min"], case["kv_max"])
        if case["kind"] == "append" or case["causal"]:
            q = min(q, kv)
        got.append((q, kv))
    for _ in range(case["idle"]):  # a slot without a sequence: a row, but nothing to attend to
        got.append((0 if case["kind"] == "append" else 1, 0))
    return got


def _kv_lens(case, rng):
    """The lengths of the sequences of a bookkeeping case."""
    return [case["kv_max"] if b == 0 else _log_int(rng, case["kv_min"], case["kv_max"])
            for b in range(case["batch"])]


def _pages_of(tokens, page):
    return -(-tokens // page)


def work(case):
    kind = case["kind"]
    if kind == "turnover":
        rows = case["leave"] + case["batch"]
        width = _pages_of(case["kv_max"] + case["grow"], case["page"])
        return {"bytes": 4.0 * (case["pages"] + rows + 2 * case["leave"] * width), "flops": 0.0}
    row = 2 * case["kv_heads"] * case["dim"]  # a token's keys and values, one byte each
    if kind == "fork":
        whole = case["page"] * row + 8 * case["kv_heads"]
        width = _pages_of(case["kv_max"], case["page"])
        return {"bytes": 2.0 * case["children"] * whole + 4.0 * (case["pages"] + 2 * case["children"] * width),
                "flops": 0.0}
    if kind == "compact":
        live = sum(_pages_of(n, case["page"]) for n in _kv_lens(case, random.Random(case["mix"])))
        moved = live * (1 - live / case["pages"])  # the mean over where the live pages lie
        whole = case["page"] * row + 8 * case["kv_heads"]
        return {"bytes": 2.0 * moved * whole + 4.0 * (2 * case["pages"] + 2 * live), "flops": 0.0}
    lens = _lengths(case)
    new, held = sum(q for q, _ in lens), sum(kv for _, kv in lens)
    npages = sum(_pages_of(kv, case["page"]) for _, kv in lens)
    if kind == "append":
        touched = sum(_pages_of(kv, case["page"]) - (kv - q) // case["page"] for q, kv in lens)
        return {"bytes": 3.0 * new * row + touched * (8.0 * case["kv_heads"] + 4), "flops": 2.0 * new * row}
    pairs = 0
    for q, kv in lens:
        pairs += q * (kv - q) + q * (q + 1) // 2 if case["causal"] and kv else q * kv
    nbytes = held * row + npages * (8.0 * case["kv_heads"] + 4) + 4.0 * new * case["heads"] * case["dim"]
    return {"bytes": nbytes, "flops": 4.0 * pairs * case["heads"] * case["dim"]}


# --------------------------------------------------------------------------- #
# Inputs                                                                        #
# --------------------------------------------------------------------------- #
def _fitting(amax):
    """The smallest power of two, 2^-40 at least, in which amax stays within e4m3's 448:
    amax = m 2^e with m in [0.5, 1), and 448 = 0.875 * 2^9."""
    m, e = torch.frexp(amax)
    need = e - 9 + (m > 0.875).to(e.dtype)
    need = torch.where(amax > 0, need, torch.full_like(need, MIN_EXP)).clamp_min(MIN_EXP)
    return torch.ldexp(torch.ones_like(amax), need)


def _random_cache(pages, kv_heads, page, dim, gen, dev):
    """Codes and scales of a pool that has been in use: keys with strong channels,
    values with quiet and loud tokens, in every page."""
    out = []
    for what in ("k", "v"):
        x = torch.randn((pages, kv_heads, page, dim), generator=gen, device=dev)
        if what == "k":
            x *= 1 + 3 * (torch.rand((kv_heads, 1, dim), generator=gen, device=dev) > 0.95)
        else:
            x *= 0.3 * torch.exp(0.5 * torch.randn((pages, kv_heads, page, 1), generator=gen,
                                                   device=dev))
        s = _fitting(x.abs().amax((-2, -1)))
        out.append(((x / s[:, :, None, None]).clamp_(-F8_MAX, F8_MAX).to(F8), s))
        del x
    (k, ks), (v, vs) = out
    return k, v, ks, vs


def _tables(lens, page, pages, width, rng, dev):
    """A table whose sequences' pages lie scattered over the pool, -1 where there is none."""
    order = rng.sample(range(pages), sum(_pages_of(n, page) for n in lens))
    table = np.full((len(lens), max(1, width)), -1, np.int32)
    at = 0
    for b, n in enumerate(lens):
        m = _pages_of(n, page)
        table[b, :m] = order[at:at + m]
        at += m
    return torch.from_numpy(table).to(dev), order


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 1000003 + case["mix"])
    rng = random.Random(seed * 7919 + case["mix"])
    kind, page = case["kind"], case["page"]
    st = dict(kind=kind, page=page)
    if kind in ("attend", "append"):
        lens = _lengths(case)
        rng.shuffle(lens)
        kv = [n for _, n in lens]
        cu = np.cumsum([0] + [q for q, _ in lens]).astype(np.int32)
        need = sum(_pages_of(n, page) for n in kv)
        st["table"], _ = _tables(kv, page, need + need // 8 + 1, _pages_of(max(kv), page), rng, dev)
        st["k"], st["v"], st["k_scale"], st["v_scale"] = _random_cache(
            need + need // 8 + 1, case["kv_heads"], page, case["dim"], gen, dev)
        st["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device=dev)
        st["cu_q"] = torch.from_numpy(cu).to(dev)
        st["max_q"], st["max_kv"] = max(q for q, _ in lens), max(kv)
        # what the fused projection of a layer gives: queries, keys and values side by side
        qkv = torch.randn((int(cu[-1]), case["heads"] + 2 * case["kv_heads"], case["dim"]),
                          generator=gen, device=dev)
        qkv[:, :case["heads"]] *= 1.5
        qkv = qkv.to(DT[case["dtype"]])
        st["q"], st["k_new"], st["v_new"] = torch.split(
            qkv, [case["heads"], case["kv_heads"], case["kv_heads"]], dim=1)
        if kind == "attend":
            st["causal"], st["scale"] = case["causal"], 1.0 / math.sqrt(case["dim"])
        st["cache"] = _handle(st)
        return st
    if kind != "turnover":
        st["k"], st["v"], st["k_scale"], st["v_scale"] = _random_cache(
            case["pages"], case["kv_heads"], page, case["dim"], gen, dev)
        st["cache"] = _handle(st)
    lens = _kv_lens(case, random.Random(case["mix"]))
    rng.shuffle(lens)
    width = _pages_of(case["kv_max"] + case.get("grow", 0), page)
    slots = len(lens) + case.get("children", 0)
    table, used = _tables(lens + [0] * (slots - len(lens)), page, case["pages"], width, rng, dev)
    refs = torch.zeros(case["pages"], dtype=torch.int32, device=dev)
    refs[torch.tensor(used, device=dev)] = 1
    held = torch.tensor(lens + [0] * (slots - len(lens)), dtype=torch.int32, device=dev)
    # refs, lengths and table in one buffer: a pass changes them, so it begins with a copy of it
    st["book"] = torch.cat([refs, held, table.reshape(-1)])
    st["pages"], st["slots"], st["width"] = case["pages"], slots, table.shape[1]
    if kind == "fork":
        src = [rng.randrange(len(lens)) for _ in range(case["children"])]
        st["src"] = torch.tensor(src, dtype=torch.int32, device=dev)
        st["dst"] = torch.arange(len(lens), slots, dtype=torch.int32, device=dev)
    if kind == "turnover":
        gone = sorted(rng.sample(range(len(lens)), case["leave"]))
        st["gone"] = torch.tensor(gone, dtype=torch.int32, device=dev)
        new = [0 if b in set(gone) else rng.randint(1, case["grow"]) for b in range(len(lens))]
        st["new"] = torch.tensor(new, dtype=torch.int32, device=dev)
    return st


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
    return {"attend": _plain_attend, "append": _plain_append, "fork": _plain_fork,
            "turnover": _plain_turnover, "compact": _plain_compact}[state["kind"]](state)


def _run_own(st):
    import int4_weight_only_repack_gb300 as w4
    kind = st["kind"]
    if kind == "attend":
        return w4.kv8_attention(st["q"], st["cache"], st["table"], st["kv_lens"], st["cu_q"],
                                st["max_q"], st["max_kv"], scale=st["scale"], causal=st["causal"])
    if kind == "append":
        w4.kv8_append(st["k_new"], st["v_new"], st["cache"], st["table"], st["kv_lens"], st["cu_q"],
                      st["max_q"])
        return [st["k"], st["v"], st["k_scale"], st["v_scale"]]
    refs, lens, table = _book(st)
    pool = w4.KV8Pool(refs, table, lens, st["page"])
    if kind == "turnover":
        w4.kv8_free(pool, st["gone"])
        w4.kv8_reserve(pool, st["new"])
        return [refs, lens, table]
    if kind == "fork":
        src, dst = w4.kv8_fork(pool, st["src"], st["dst"])
    else:
        src, dst = w4.kv8_compact(pool)
    w4.kv8_copy_pages(st["cache"], src, dst)
    return [refs, lens, table, src, dst, st["k"], st["v"], st["k_scale"], st["v_scale"]]


def _book(st):
    """refs, lengths and table of a copy of the bookkeeping, for a pass to change."""
    book = st["book"].clone()
    p, s = st["pages"], st["slots"]
    return book[:p], book[p:p + s], book[p + s:].view(s, st["width"])


def _gather(codes, scales, table):
    """[batch, kv_heads, tokens, dim] fp32 values of the table's pages (page 0's for -1)."""
    at = table.clamp_min(0).long()
    x = codes.view(torch.uint8)[at].view(F8).float() * scales[at][..., None, None]
    b, n, h, p, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(b, h, n * p, d)


def _plain_attend(st):
    q, lens, cu = st["q"], st["kv_lens"].long(), st["cu_q"].long()
    k = _gather(st["k"], st["k_scale"], st["table"])
    v = _gather(st["v"], st["v_scale"], st["table"])
    b, hk, length, d = k.shape
    heads, group = q.shape[1], q.shape[1] // hk
    row = torch.arange(st["max_q"], device=q.device)
    n = (cu[1:] - cu[:-1])[:, None]
    real = row < n
    tok = (cu[:-1, None] + row).clamp_max(max(q.shape[0] - 1, 0))
    x = q[tok].float().view(b, -1, hk, group, d).permute(0, 2, 3, 1, 4).reshape(b, hk, -1, d)
    s = torch.matmul(x, k.transpose(2, 3)).view(b, hk, group, -1, length) * st["scale"]
    col = torch.arange(length, device=q.device)
    seen = (col < lens[:, None])[:, None, :] & real[:, :, None]
    if st["causal"]:
        seen = seen & (col <= (lens[:, None] - n + row)[:, :, None])
    seen = seen[:, None, None]
    s = torch.where(seen, s, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(-1, keepdim=True)
    v = torch.where((col < lens[:, None])[:, None, :, None], v, 0.0)
    o = torch.matmul(p.view(b, hk, -1, length), v).view(b, hk, group, -1, d)
    o = torch.where(total > 0, o / total, 0.0)
    o = o.permute(0, 3, 1, 2, 4).reshape(b, -1, heads, d)
    out = torch.zeros((q.shape[0] + 1, heads, d), device=q.device)
    out[torch.where(real, tok, q.shape[0])] = o  # rows past a sequence's own go to a spare row
    return out[:-1].to(q.dtype)


def _plain_append(st):
    page, lens, cu = st["page"], st["kv_lens"].long(), st["cu_q"].long()
    t = torch.arange(st["k_new"].shape[0], device=lens.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    pos = lens[b] - (cu[b + 1] - t)
    where, slot = st["table"][b, pos // page].long(), pos % page
    count = cu[1:] - cu[:-1]
    first = lens - count  # each sequence's tokens before the call
    # pages that held tokens and get more: at most one of each sequence
    part = torch.nonzero((count > 0) & (first % page > 0))[:, 0]
    shared = st["table"][part, first[part] // page].long()
    held = torch.arange(page, device=t.device) < (first[part] % page)[:, None]
    for codes, scales, new in ((st["k"], st["k_scale"], st["k_new"]),
                               (st["v"], st["v_scale"], st["v_new"])):
        x = new.float()
        amax = torch.zeros_like(scales).index_reduce_(0, where, x.abs().amax(-1), "amax")
        now = _fitting(amax)
        now[shared] = torch.maximum(now[shared], scales[shared])
        flat = codes.view(torch.uint8)
        # codes already in a page whose scale grows are stored again in the new one
        old = flat[shared].view(F8).float()
        again = (old * (scales[shared] / now[shared])[:, :, None, None]).to(F8)
        flat[shared] = torch.where(held[:, None, :, None], again.view(torch.uint8), flat[shared])
        code = (x / now[where][:, :, None]).clamp(-F8_MAX, F8_MAX).to(F8)
        flat[where, :, slot] = code.view(torch.uint8)
        scales[where] = now[where]
    return [st["k"], st["v"], st["k_scale"], st["v_scale"]]


def _free_pages(refs):
    """Every page's number, the free ones first, each kind in ascending order."""
    return torch.argsort((refs > 0).to(torch.int8), stable=True)


def _plain_fork(st):
    refs, lens, table = _book(st)
    src, dst, page = st["src"].long(), st["dst"].long(), st["page"]
    n = lens[src].long()
    col = torch.arange(st["width"], device=refs.device)
    full, part = n // page, (n % page > 0).long()
    rank = torch.cumsum(part, 0) - part
    fresh = _free_pages(refs)[rank]
    rows = table[src]
    last = rows.gather(1, full.clamp_max(st["width"] - 1)[:, None])[:, 0]
    copy_src = torch.where(part > 0, last, -1).to(torch.int32)
    copy_dst = torch.where(part > 0, fresh, -1).to(torch.int32)
    child = torch.where(col < full[:, None], rows, -1)
    child = torch.where((col == full[:, None]) & (part[:, None] > 0), copy_dst[:, None], child)
    one = (child >= 0).to(torch.int32)
    refs.index_add_(0, child.clamp_min(0).long().reshape(-1), one.reshape(-1))
    table[dst] = child
    lens[dst] = lens[src]
    return _plain_copied(st, refs, lens, table, copy_src, copy_dst)


def _plain_copied(st, refs, lens, table, src, dst):
    """Copies the pages src to dst (pairs of -1: none) and returns a pass's outputs."""
    keep = src >= 0
    s, d = src[keep].long(), dst[keep].long()
    for x in (st["k"], st["v"]):
        x.view(torch.uint8)[d] = x.view(torch.uint8)[s]
    for x in (st["k_scale"], st["v_scale"]):
        x[d] = x[s]
    return [refs, lens, table, src, dst, st["k"], st["v"], st["k_scale"], st["v_scale"]]


def _plain_turnover(st):
    refs, lens, table = _book(st)
    page, gone = st["page"], st["gone"].long()
    col = torch.arange(st["width"], device=refs.device)
    rows = table[gone]
    held = col < ((lens[gone] + page - 1) // page)[:, None]
    refs.index_add_(0, torch.where(held, rows, 0).long().reshape(-1),
                    -held.to(torch.int32).reshape(-1))
    table[gone] = -1
    lens[gone] = 0
    have = (lens + page - 1) // page
    lens += st["new"]
    want = (lens + page - 1) // page
    need = (want - have).long()
    rank = (torch.cumsum(need, 0) - need)[:, None] + col - have[:, None]
    fresh = (col >= have[:, None]) & (col < want[:, None])
    free = _free_pages(refs)
    table.copy_(torch.where(fresh, free[rank.clamp(0, st["pages"] - 1)].to(torch.int32), table))
    at = torch.arange(st["pages"], device=refs.device)
    refs[free] += (at < need.sum()).to(torch.int32)
    return [refs, lens, table]


def _plain_compact(st):
    refs, lens, table = _book(st)
    n = st["pages"]
    at = torch.arange(n, device=refs.device)
    live = refs > 0
    count = live.sum()
    hole, mover = ~live & (at < count), live & (at >= count)
    src = torch.argsort((~mover).to(torch.int8), stable=True)
    dst = torch.argsort((~hole).to(torch.int8), stable=True)
    moved = at < mover.sum()
    copy_src = torch.where(moved, src, -1).to(torch.int32)
    copy_dst = torch.where(moved, dst, -1).to(torch.int32)
    to = at.clone()
    to[src] = torch.where(moved, dst, src)
    table.copy_(torch.where(table >= 0, to[table.clamp_min(0).long()].to(torch.int32), table))
    old = refs.clone()
    refs.copy_(torch.where(mover, 0, refs))
    refs[dst] = torch.where(moved, old[src], refs[dst])
    return _plain_copied(st, refs, lens, table, copy_src, copy_dst)


# --------------------------------------------------------------------------- #
# The definitions in 64 bits                                                    #
# --------------------------------------------------------------------------- #
def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] == "attend":
        return _exact_attend(st)
    if case["kind"] == "append":
        return _exact_append(st)
    return _exact_pages(st)


def _exact_attend(st):
    q, page = st["q"].double(), st["page"]
    group = q.shape[1] // st["k"].shape[1]
    out = torch.zeros_like(q)
    cu, lens = st["cu_q"].tolist(), st["kv_lens"].tolist()
    for b, n in enumerate(lens):
        if n == 0 or cu[b] == cu[b + 1]:
            continue
        ids = st["table"][b, :_pages_of(n, page)].long()
        for h in range(q.shape[1]):
            g = h // group
            k, v = ((c.view(torch.uint8)[ids, g].view(F8).double() * s[ids, g].double()[:, None, None])
                    .reshape(-1, q.shape[2])[:n] for c, s in ((st["k"], st["k_scale"]),
                                                             (st["v"], st["v_scale"])))
            m = cu[b + 1] - cu[b]
            s = (q[cu[b]:cu[b + 1], h] @ k.T) * st["scale"]
            if st["causal"]:
                i = torch.arange(m, device=q.device)[:, None]
                s.masked_fill_(torch.arange(n, device=q.device) > n - m + i, -math.inf)
            out[cu[b]:cu[b + 1], h] = torch.softmax(s, -1) @ v
    return out


def _round_e4m3(x):
    """The e4m3 value nearest to each element, ties to the even code, saturated at 448."""
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -60))).clamp_min(-6)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-F8_MAX, F8_MAX)


def _exact_append(st):
    page, cu, lens = st["page"], st["cu_q"].tolist(), st["kv_lens"].tolist()
    table = st["table"].tolist()
    got = [st["k"].double(), st["v"].double(), st["k_scale"].double(), st["v_scale"].double()]
    for codes, scales, new in ((got[0], got[2], st["k_new"]), (got[1], got[3], st["v_new"])):
        for b, n in enumerate(lens):
            j = n - (cu[b + 1] - cu[b])
            while j < n:  # page by page
                end, before = min(n, (j // page + 1) * page), j % page
                p = table[b][j // page]
                x = new[cu[b + 1] - (n - j):cu[b + 1] - (n - end)].double().transpose(0, 1)
                amax = x.abs().amax((1, 2))
                fit = torch.exp2(torch.floor(torch.log2(amax.clamp_min(2.0 ** -60))) - 8)
                fit = torch.where(amax > F8_MAX * fit, 2 * fit, fit).clamp_min(2.0 ** MIN_EXP)
                now = torch.maximum(fit, scales[p]) if before else fit
                if before:
                    codes[p, :, :before] = _round_e4m3(
                        codes[p, :, :before] * (scales[p] / now)[:, None, None])
                codes[p, :, before:before + end - j] = _round_e4m3(x / now[:, None, None])
                scales[p] = now
                j = end
    return got


def _exact_pages(st):
    refs, lens, table = (x.cpu().numpy().copy() for x in _book(st))
    page = st["page"]
    src, dst = [], []
    if st["kind"] == "turnover":
        for b in st["gone"].tolist():
            for p in table[b, :_pages_of(int(lens[b]), page)]:
                refs[p] -= 1
            table[b], lens[b] = -1, 0
        free = iter(np.flatnonzero(refs == 0).tolist())
        for b, n in enumerate(st["new"].tolist()):
            have = _pages_of(int(lens[b]), page)
            lens[b] += n
            for j in range(have, _pages_of(int(lens[b]), page)):
                table[b, j] = next(free)
                refs[table[b, j]] = 1
        return [torch.from_numpy(x) for x in (refs, lens, table)]
    if st["kind"] == "fork":
        free = iter(np.flatnonzero(refs == 0).tolist())
        for a, b in zip(st["src"].tolist(), st["dst"].tolist()):
            full, part = divmod(int(lens[a]), page)
            table[b], lens[b] = -1, lens[a]
            table[b, :full] = table[a, :full]
            if part:
                table[b, full] = next(free)
            for p in table[b, :full + (part > 0)]:
                refs[p] += 1
            src.append(int(table[a, full]) if part else -1)
            dst.append(int(table[b, full]) if part else -1)
    else:
        live = np.flatnonzero(refs > 0)
        src = [p for p in live.tolist() if p >= len(live)]
        dst = np.flatnonzero(refs[:len(live)] == 0).tolist()
        to = dict(zip(src, dst))
        for b in range(len(lens)):
            for j in range(st["width"]):
                table[b, j] = to.get(int(table[b, j]), table[b, j])
        for a, b in to.items():
            refs[a], refs[b] = 0, refs[a]
        src += [-1] * (st["pages"] - len(src))
        dst += [-1] * (st["pages"] - len(dst))
    src, dst = (torch.tensor(x, dtype=torch.int32) for x in (src, dst))
    keep = src >= 0
    s, d = src[keep].long().cuda(), dst[keep].long().cuda()
    moved = []
    for x in (st["k"], st["v"], st["k_scale"], st["v_scale"]):
        x = x.double()
        x[d] = x[s]
        moved.append(x)
    return [torch.from_numpy(x) for x in (refs, lens, table)] + [src, dst] + moved
