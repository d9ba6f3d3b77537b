"""Speculative decoding with 4-bit weights and an 8-bit key-value cache, in one small decoder.

Every layer norms its query and key heads and turns them by their positions; the lower
layers see a sliding window with two sinks. Each step the first layer alone guesses a
tree of tokens, the whole decoder checks all of them in one pass, the branch that it
agrees with is kept in every layer's cache, and the sequences give back the rest.
The weights are random; what counts is which calls are made, and in what order.

    python examples/draft_kv8.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import int4_weight_only_repack_gb300 as w4  # noqa: E402


class Decoder:
    """Attention blocks (no feed-forward part) with AWQ weights."""

    def __init__(self, layers=3, heads=8, kv_heads=2, dim=64, vocab=500, window=48, max_len=512,
                 dtype=torch.bfloat16, seed=0):
        self.heads, self.kv_heads, self.dim, self.max_len = heads, kv_heads, dim, max_len
        g = torch.Generator(device="cuda").manual_seed(seed)
        hidden = heads * dim
        self.embedding, self.head = (torch.randn(vocab, hidden, device="cuda", generator=g).to(dtype)
                                     for _ in range(2))
        self.rotations = w4.rope_table(max_len, dim)

        def layer(K, N):
            words = lambda *shape: torch.randint(-2 ** 31, 2 ** 31 - 1, shape, device="cuda",
                                                 generator=g, dtype=torch.int32)
            scales = torch.full((K // 128, N), 0.1 * K ** -0.5, device="cuda", dtype=dtype)
            return w4.repack_awq(words(K, N // 8), words(K // 128, N // 8), scales, K, N, 128, dtype)

        # the last layer sees everything, the others a window
        self.blocks = [(layer(hidden, (heads + 2 * kv_heads) * dim), layer(hidden, hidden),
                        *(1 + 0.1 * torch.randn(dim, device="cuda", generator=g) for _ in range(2)),
                        dict(window=window, sinks=2) if n < layers - 1 else {}) for n in range(layers)]

    def caches(self, num_pages, page_size):
        return [w4.kv8_cache(num_pages, self.kv_heads, page_size, self.dim) for _ in self.blocks]

    def __call__(self, tokens, positions, caches, pool, cu_q, max_q_len, tree=None, layers=None):
        """Logits of new tokens; pool.lens counts them already."""
        x = self.embedding[tokens]
        for (qkv, out, q_norm, k_norm, sees), cache in list(zip(self.blocks, caches))[:layers]:
            y = w4.linear(torch.nn.functional.rms_norm(x, x.shape[1:]), qkv)
            q, k, v = y.unflatten(1, (-1, self.dim)).split((self.heads, self.kv_heads, self.kv_heads), 1)
            w4.qk_norm_rope(q, k, positions, self.rotations, q_norm, k_norm, q_out=q, k_out=k)
            w4.kv8_append(k, v, cache, pool.table, pool.lens, cu_q, max_q_len)
            a = w4.kv8_attention(q, cache, pool.table, pool.lens, cu_q, max_q_len, self.max_len,
                                 tree=tree, **sees)
            x = x + w4.linear(a.flatten(1), out)
        return torch.nn.functional.rms_norm(x.float(), x.shape[1:]) @ self.head.float().t()


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def check(pool):
    status = int(pool.status) or w4.w4_device_status()
    if status:
        raise RuntimeError(w4.w4_status_string(status))


def tree_of(width, depth):
    """(parents, bits) of the root and `depth` levels of drafts, each draft of a level but
    the last one's root having `width` children."""
    parents, level = [-1], [0]
    for _ in range(depth):
        first = len(parents)
        parents += [p for p in level for _ in range(width)]
        level = range(first, len(parents))
    bits = []
    for i, p in enumerate(parents):
        bits.append((bits[p] if p >= 0 else 0) | 1 << i)
    return parents, bits


def generate(lengths=(70, 33, 120), new_tokens=24, width=2, depth=3, page_size=16, seed=0):
    """Returns (each sequence's new tokens, accepted drafts, steps, pool)."""
    model = Decoder(seed=seed)
    n, parents_bits = len(lengths), tree_of(width, depth)
    parents, bits = parents_bits
    m = len(parents)
    pages = n * -(-(max(lengths) + new_tokens + 2 * m) // page_size)
    pool = w4.kv8_pool(pages, n, model.max_len, page_size)
    caches = model.caches(pages, page_size)

    g = torch.Generator(device="cuda").manual_seed(seed)
    prompt = torch.randint(0, model.embedding.shape[0], (sum(lengths),), device="cuda", generator=g)
    w4.kv8_reserve(pool, ints(lengths))
    cu_q = ints([0] + torch.tensor(lengths).cumsum(0).tolist())
    positions = ints([i for length in lengths for i in range(length)])
    logits = model(prompt, positions, caches, pool, cu_q, max(lengths))
    root = logits[cu_q[1:].long() - 1].argmax(1)
    check(pool)

    # what does not change from step to step
    cu_tree = ints([m * b for b in range(n + 1)])
    tree = torch.tensor(bits, dtype=torch.int64, device="cuda").repeat(n)
    deep = torch.tensor([bin(b).count("1") - 1 for b in bits], device="cuda")
    up = torch.tensor(parents, device="cuda")
    all_drafts = ints([m] * n)
    text, accepted, steps = [[int(t)] for t in root], 0, 0

    while min(map(len, text)) < new_tokens:
        # the first layer guesses the tree, level by level, into its own cache; every level
        # is written anew with the ones before it (the drafts' slots are reserved once)
        base = pool.lens.clone()
        w4.kv8_reserve(pool, all_drafts)
        positions = (base[:, None] + deep).to(torch.int32).flatten()
        tokens = root[:, None].expand(n, m).clone()
        for level in range(1, depth + 1):
            guess = model(tokens.flatten(), positions, caches, pool, cu_tree, m, tree, layers=1)
            best = guess.view(n, m, -1).topk(width, 2).indices
            for i in (deep == level).nonzero().flatten().tolist():
                p = parents[i]
                tokens[:, i] = best[:, p, parents[:i].count(p)]
        # the decoder checks all of them at once
        choice = model(tokens.flatten(), positions, caches, pool, cu_tree, m, tree).argmax(1).view(n, m)
        # the longest branch whose every draft is what the decoder chose after its parent
        right = torch.ones(n, m, dtype=torch.bool, device="cuda")
        right[:, 1:] = tokens[:, 1:] == choice.gather(1, up[1:].expand(n, -1))
        for i in range(1, m):
            right[:, i] &= right[:, parents[i]]
        last = torch.where(right, deep * m - torch.arange(m, device="cuda"), -m).argmax(1)  # the first of the deepest
        path = torch.full((n, m), -1, dtype=torch.int32)
        for b, i in enumerate(last.tolist()):
            branch = [d for d in range(m) if bits[i] >> d & 1]
            path[b, :len(branch)] = torch.tensor(branch, dtype=torch.int32)
            text[b] += tokens[b, branch[1:]].tolist() + [int(choice[b, i])]
            accepted += len(branch) - 1
        root = choice.gather(1, last[:, None]).flatten()
        drop = (path < 0).sum(1).to(torch.int32).cuda()
        path = path.flatten().cuda()
        for cache in caches:
            w4.kv8_keep(cache, pool.table, pool.lens, cu_tree, path, m)
        w4.kv8_shorten(pool, drop)
        check(pool)
        steps += 1
    return text, accepted, steps, pool


if __name__ == "__main__":
    text, accepted, steps, pool = generate()
    for b, tokens in enumerate(text):
        print(f"sequence {b}: {len(tokens)} tokens {tokens}")
    print(f"{steps} steps, {accepted} drafts accepted")
