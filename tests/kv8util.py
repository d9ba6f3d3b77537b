"""Plain 64-bit forms of the 8-bit key-value cache operators, for the tests."""
import math

import numpy as np
import torch

F8 = torch.float8_e4m3fn
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
UNIT = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}  # half an ulp, relative


def codes_of(x):
    """float64 values of e4m3 codes."""
    return x.double()


def as_f8(values):
    return values.float().to(F8)


def random_cache(w4, pages, heads, page, dim, seed, scales="pow2"):
    """A cache of random codes; scales: powers of two, or any positive fp32."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = dict(device="cuda", generator=g)
    c = w4.kv8_cache(pages, heads, page, dim)
    for codes, sc in ((c.k, c.k_scale), (c.v, c.v_scale)):
        x = torch.randn((pages, heads, page, dim), **dev) * 100
        codes.view(torch.uint8).copy_(x.clamp(-448, 448).to(F8).view(torch.uint8))
        e = torch.randint(-10, -4, (pages, heads), **dev).float()
        sc.copy_(torch.exp2(e) if scales == "pow2" else torch.exp2(e + torch.rand((pages, heads), **dev)))
    return c


def scattered_table(lens, page, pages, seed, width=None):
    """Every sequence's pages at random places; -1 past its own."""
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    order = rng.permutation(pages)
    assert sum(need) <= pages
    t = np.full((len(lens), width or max(1, max(need, default=1))), -1, np.int32)
    at = 0
    for b, m in enumerate(need):
        t[b, :m] = order[at:at + m]
        at += m
    return torch.from_numpy(t).cuda()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def bounds(counts):
    return ints(np.concatenate([[0], np.cumsum(counts)]).tolist())


def values(codes, scale, ids, head, n):
    """[n, dim] float64 values of one sequence and head."""
    x = codes[ids, head].double() * scale[ids, head].double()[:, None, None]
    return x.reshape(-1, codes.shape[-1])[:n]


def attention(q, cache, table, lens, counts, scale, causal, dtype):
    """(out, tolerance) in float64.

    The tolerance per element, with u the output type's half ulp, A = sum p |v| /
    sum p, n tokens, S = the largest scale * sum |q_d k_d|, and V the largest value
    a code can stand for: p is rounded to fp16 once (2^-11 of it, or 2^-25 below
    fp16's normal range, where 1 is the largest p times its value scale), the
    score's fp32 sum and scaling err by at most 2^-20 (S + 8) in the exponent (which
    enters the numerator and the sum), and n / 16 fp32 additions by 2^-24 each.
        tol = u |out| + A (2^-10 + 2^-19 (S + 8) + n 2^-26) + n 2^-24 V
    """
    page, dim = cache.page_size, cache.head_dim
    group = q.shape[1] // cache.kv_heads
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    at = 0
    for b, (n, m) in enumerate(zip(lens, counts)):
        ids = table[b, :-(-n // page)].long()
        for h in range(q.shape[1]):
            if n == 0 or m == 0:
                continue
            k = values(cache.k, cache.k_scale, ids, h // group, n)
            v = values(cache.v, cache.v_scale, ids, h // group, n)
            x = q[at:at + m, h].double()
            s = x @ k.T * scale
            big = (x.abs() @ k.abs().T * abs(scale)).amax(1, keepdim=True)
            if causal:
                i = torch.arange(m, device=q.device)[:, None]
                s = s.masked_fill(torch.arange(n, device=q.device) > n - m + i, -math.inf)
            top = s.amax(1, keepdim=True)
            p = torch.exp(s - torch.where(torch.isinf(top), 0.0, top))
            total = p.sum(1, keepdim=True)
            w = torch.where(total > 0, p / total.clamp_min(1e-300), 0.0)
            o = w @ v
            vmax = 448 * cache.v_scale[ids, h // group].double().amax()
            out[at:at + m, h] = o
            tol[at:at + m, h] = (UNIT[dtype] * o.abs()
                                 + (w @ v.abs()) * (2.0 ** -10 + 2.0 ** -19 * (big + 8) + n * 2.0 ** -26)
                                 + n * 2.0 ** -24 * vmax * (total > 0))
        at += m
    return out, tol


def round_e4m3(x):
    """The e4m3 value nearest to each element (ties to the even code), saturated."""
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -60)))
    step = 2.0 ** (np.maximum(e, -6) - 3)
    return np.clip(np.round(x / step) * step, -448, 448)


def fit(amax):
    """The smallest power of two >= 2^-40 with amax <= 448 of it."""
    s = 2.0 ** -40
    while amax > 448 * s:
        s *= 2
    return s


def append(state, new_k, new_v, table, lens, counts, page):
    """state: [k, v, k_scale, v_scale] float64 arrays, changed in place."""
    at = 0
    for b, (n, m) in enumerate(zip(lens, counts)):
        for j in range(n - m, n):
            if j > n - m and j % page:
                continue  # one turn per page
            end, p, held = min(n, (j // page + 1) * page), table[b][j // page], j % page
            for i, new in ((0, new_k), (1, new_v)):
                x = new[at + j - (n - m):at + end - (n - m)]
                for h in range(x.shape[1]):
                    now = fit(np.abs(np.where(np.isfinite(x[:, h]), x[:, h], 0)).max())
                    old = state[2 + i][p, h]
                    if held:
                        now = max(now, old)
                        if now > old:
                            state[i][p, h, :held] = round_e4m3(state[i][p, h, :held] * (old / now))
                    y = np.clip(x[:, h] / now, -1e6, 1e6)
                    state[i][p, h, held:held + end - j] = np.where(np.isnan(y), np.nan, round_e4m3(y))
                    state[2 + i][p, h] = now
        at += m


class Book:
    """A pool's bookkeeping, step by step."""

    def __init__(self, refs, table, lens, page):
        self.refs, self.table, self.lens, self.page = list(refs), [list(r) for r in table], list(lens), page

    def pages(self, n):
        return -(-n // self.page)

    def lowest(self, count):
        free = [p for p, r in enumerate(self.refs) if r == 0]
        return free[:count] if count <= len(free) else None

    def reserve(self, new):
        need = [self.pages(n + a) - self.pages(n) for n, a in zip(self.lens, new)]
        got = self.lowest(sum(need))
        if got is None:
            return False
        for s, (m, a) in enumerate(zip(need, new)):
            at = self.pages(self.lens[s])
            for j in range(m):
                p = got.pop(0)
                self.table[s][at + j], self.refs[p] = p, 1
            self.lens[s] += a
        return True

    def fork(self, src, dst):
        part = [self.lens[s] % self.page != 0 for s in src]
        got = self.lowest(sum(part))
        if got is None:
            return None
        moves = []
        for s, d, has in zip(src, dst, part):
            n = self.lens[s]
            full = n // self.page
            row = self.table[s][:full] + [-1] * (len(self.table[s]) - full)
            move = (-1, -1)
            if has:
                move = (self.table[s][full], got.pop(0))
                row[full] = move[1]
            for p in row[:self.pages(n)]:
                self.refs[p] += 1
            self.table[d], self.lens[d] = row, n
            moves.append(move)
        return moves

    def free(self, seqs):
        for s in seqs:
            for j in range(self.pages(self.lens[s])):
                self.refs[self.table[s][j]] -= 1
            if self.lens[s]:
                self.table[s] = [-1] * len(self.table[s])
            self.lens[s] = 0

    def compact(self):
        used = sum(r > 0 for r in self.refs)
        src = [p for p, r in enumerate(self.refs) if r > 0 and p >= used]
        dst = [p for p, r in enumerate(self.refs) if r == 0 and p < used]
        to = dict(zip(src, dst))
        self.table = [[to.get(p, p) for p in row] for row in self.table]
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
        return list(zip(src, dst))
