"""Plain 64-bit forms of masked attention over the 8-bit cache, for the tests."""
import math

import numpy as np
import torch

import kv8util as ref


def window_sees(n, m, window, sinks, device="cuda"):
    """[m, n]: what the last m of n tokens see through a window beside the sinks."""
    p = torch.arange(n - m, n, device=device)[:, None]
    j = torch.arange(n, device=device)
    return (j <= p) & ((j > p - window) | (j < sinks))


def tree_sees(n, m, words, window=None, sinks=0, device="cuda"):
    """[m, n]: what m drafts see by their words, after n - m other tokens (which may be
    less than none: then the first drafts do not exist)."""
    base = n - m
    sees = np.zeros((m, max(n, 0)), bool)
    j = np.arange(max(base, 0))
    for i, word in enumerate(words):
        on = [d for d in range(m) if word >> d & 1]
        sees[i, :len(j)] = True if window is None else (j < sinks) | (j >= base + len(on) - window)
        sees[i, [base + d for d in on if base + d >= 0]] = True
    return torch.from_numpy(sees).to(device)


def attention(q, cache, table, lens, counts, sees, scale, dtype):
    """(out, tolerance) in float64, the tolerance being kv8util.attention's, with the
    tokens that a query sees for n. sees(b): [queries, tokens] of sequence b."""
    page, dim = cache.page_size, cache.head_dim
    group = q.shape[1] // cache.kv_heads
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    at = 0
    for b, (n, m) in enumerate(zip(lens, counts)):
        if n and m:
            ids, seen = table[b, :-(-n // page)].long(), sees(b)
            some = seen.any(0)  # (codes and scales of the others may be anything)
            count = seen.sum(1)[:, None]
            k, v = ((c[ids].double() * sc[ids].double()[..., None, None]).transpose(0, 1)
                    .reshape(cache.kv_heads, -1, dim)[:, :n].masked_fill(~some[:, None], 0)
                    for c, sc in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
            x = q[at:at + m].double().view(m, cache.kv_heads, group, dim).permute(1, 2, 0, 3)
            k, v = k[:, None], v[:, None]  # [kv heads, group, tokens, dim]
            s = (x @ k.transpose(2, 3) * scale).masked_fill(~seen, -math.inf)
            big = (x.abs() @ k.abs().transpose(2, 3) * abs(scale)).masked_fill(~seen, 0).amax(-1, keepdim=True)
            top = s.amax(-1, keepdim=True)
            p = torch.exp(s - torch.where(torch.isinf(top), 0.0, top))
            total = p.sum(-1, keepdim=True)
            w = torch.where(total > 0, p / total.clamp_min(1e-300), 0.0)
            o = w @ v
            loud = cache.v_scale[ids].double().t().repeat_interleave(page, 1)[:, :n]
            vmax = 448 * loud.masked_fill(~some, 0).amax(1)[:, None, None, None]
            t = (ref.UNIT[dtype] * o.abs()
                 + (w @ v.abs()) * (2.0 ** -10 + 2.0 ** -19 * (big + 8) + count * 2.0 ** -26)
                 + count * 2.0 ** -24 * vmax * (total > 0))
            for to, y in ((out, o), (tol, t)):
                to[at:at + m] = y.permute(2, 0, 1, 3).reshape(m, -1, dim)
        at += m
    return out, tol


def random_tree(n, rng, kind):
    """Words of n drafts: 'tree' (a draft sees its branch), 'chain' (all before it), or
    'any' (any bits, none and those past n among them)."""
    words = []
    for i in range(n):
        if kind == "tree":
            parent = int(rng.integers(-1, i)) if i else -1
            words.append((words[parent] if parent >= 0 else 0) | 1 << i)
        elif kind == "chain":
            words.append((1 << i + 1) - 1)
        else:
            words.append(int(rng.integers(0, 1 << 62)) << 2 | int(rng.integers(0, 4)) if rng.random() > 0.2 else 0)
    return words


def words_tensor(words):
    """int64 on the GPU, bit 63 its sign."""
    return torch.tensor([w - (1 << 64) if w >> 63 else w for w in words], dtype=torch.int64, device="cuda")
