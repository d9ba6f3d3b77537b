"""Serving with 4-bit weights and an 8-bit key-value cache, in one small decoder.

Prompts of different lengths are read in one ragged batch, every sequence is
forked into alternatives that share the prompt's pages, and all of them decode
together, a step being one replayed CUDA graph: pages reserved on the device,
linear layers, keys and values quantised into the cache, attention. Halfway the
less likely alternatives are freed and the pool is compacted. The weights are
random; what counts is which calls are made, and in what order.

    python examples/serve_kv8.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import int4_weight_only_repack_gb300 as w4  # noqa: E402


class Decoder:
    """Attention blocks (no feed-forward part) with AWQ weights."""

    def __init__(self, layers=2, heads=8, kv_heads=2, dim=64, vocab=1000, dtype=torch.bfloat16,
                 seed=0):
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        g = torch.Generator(device="cuda").manual_seed(seed)
        hidden = heads * dim
        self.embedding, self.head = (torch.randn(vocab, hidden, device="cuda", generator=g).to(dtype)
                                     for _ in range(2))

        def layer(K, N):
            words = lambda *shape: torch.randint(-2 ** 31, 2 ** 31 - 1, shape, device="cuda",
                                                 generator=g, dtype=torch.int32)
            scales = torch.full((K // 128, N), 0.3 * K ** -0.5, device="cuda", dtype=dtype)
            return w4.repack_awq(words(K, N // 8), words(K // 128, N // 8), scales, K, N, 128, dtype)

        self.blocks = [(layer(hidden, (heads + 2 * kv_heads) * dim), layer(hidden, hidden))
                       for _ in range(layers)]

    def caches(self, num_pages, page_size):
        return [w4.kv8_cache(num_pages, self.kv_heads, page_size, self.dim) for _ in self.blocks]

    def __call__(self, tokens, caches, pool, cu_q, max_q_len, max_kv_len):
        """Hidden states of new tokens; pool.lens counts them already."""
        x = self.embedding[tokens]
        for (qkv, out), cache in zip(self.blocks, caches):
            y = w4.linear(torch.nn.functional.rms_norm(x, x.shape[1:]), qkv)
            y = y.unflatten(1, (-1, self.dim))  # the three below are views of it
            q, k, v = y.split((self.heads, self.kv_heads, self.kv_heads), 1)
            w4.kv8_append(k, v, cache, pool.table, pool.lens, cu_q, max_q_len)
            a = w4.kv8_attention(q, cache, pool.table, pool.lens, cu_q, max_q_len, max_kv_len)
            x = x + w4.linear(a.flatten(1), out)
        return x

    def logits(self, x):
        return torch.nn.functional.rms_norm(x.float(), x.shape[1:]) @ self.head.float().t()


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def check(pool):
    status = int(pool.status)
    if status:
        raise RuntimeError(w4.w4_status_string(status))


def decode(model, caches, pool, live, tokens, steps, max_len, graph):
    """steps tokens for each of the live sequences, and their summed log-probability."""
    slots = pool.lens.shape[0]
    new = torch.zeros(slots, dtype=torch.int32)
    new[live] = 1
    cu_q = ints([0] + new.cumsum(0).tolist())
    new, tokens = new.cuda(), tokens.clone()
    score = torch.zeros(len(live), device="cuda")

    def step():
        w4.kv8_reserve(pool, new)
        logp = model.logits(model(tokens, caches, pool, cu_q, 1, max_len)).log_softmax(1)
        best, token = logp.max(1)
        score.add_(best)
        tokens.copy_(token)

    out, replay = [], None
    for _ in range(steps):
        if graph and replay is None and out:  # the first step warmed everything up
            replay = torch.cuda.CUDAGraph()
            with torch.cuda.graph(replay):
                step()
        replay.replay() if replay is not None else step()
        out.append(tokens.clone())
    check(pool)
    return torch.stack(out, 1), score


def serve(lengths=(70, 200, 33), forks=3, steps=24, page_size=16, graph=True, compact=True,
          distinct=True, seed=0):
    """Returns ({slot: its tokens}, pool). distinct: the alternatives of a prompt
    start with its likeliest tokens, one each; else all with the likeliest."""
    model = Decoder(seed=seed)
    slots, max_len = len(lengths) * forks, max(lengths) + steps
    per_seq = -(-max_len // page_size)
    pool = w4.kv8_pool(slots * per_seq, slots, max_len, page_size)
    caches = model.caches(slots * per_seq, page_size)

    # the prompts, in slots 0, forks, 2 * forks, ...; the other slots are empty
    n = torch.zeros(slots, dtype=torch.int32)
    n[::forks] = torch.tensor(lengths, dtype=torch.int32)
    prompt = torch.randint(0, model.embedding.shape[0], (sum(lengths),), device="cuda",
                           generator=torch.Generator(device="cuda").manual_seed(seed))
    w4.kv8_reserve(pool, n.cuda())
    check(pool)
    cu_q = ints([0] + n.cumsum(0).tolist())
    x = model(prompt, caches, pool, cu_q, max(lengths), max_len)
    last = model.logits(x[cu_q[1:][::forks].long() - 1])
    first = last.topk(forks, 1).indices if distinct else last.topk(1, 1).indices.expand(-1, forks)

    # alternatives share the prompt's full pages; each gets the last partial one
    pairs = [(s - s % forks, s) for s in range(slots) if s % forks]
    if pairs:
        moves = w4.kv8_fork(pool, ints([a for a, _ in pairs]), ints([b for _, b in pairs]))
        check(pool)
        for cache in caches:
            w4.kv8_copy_pages(cache, *moves)

    tokens = first.reshape(-1)
    half, score = decode(model, caches, pool, list(range(slots)), tokens, steps // 2, max_len, graph)
    text = {s: [int(tokens[s])] + half[s].tolist() for s in range(slots)}

    # keep the likeliest alternative of each prompt
    keep = [forks * i + int(score[forks * i:forks * (i + 1)].argmax()) for i in range(len(lengths))]
    drop = [s for s in range(slots) if s not in keep]
    if drop:
        w4.kv8_free(pool, ints(drop))
        check(pool)
    if compact:
        moves = w4.kv8_compact(pool)
        for cache in caches:
            w4.kv8_copy_pages(cache, *moves)
    rest, _ = decode(model, caches, pool, keep, half[keep, -1], steps - steps // 2, max_len, graph)
    for s, more in zip(keep, rest.tolist()):
        text[s] += more
    return text, pool


if __name__ == "__main__":
    text, pool = serve()
    for slot, tokens in text.items():
        print(f"slot {slot}: {len(tokens)} tokens {tokens}")
    used = pool.refs.nonzero().flatten()
    print(f"{used.numel()} pages in use, the highest {int(used.max())}")
    w4.kv8_free(pool, pool.lens.nonzero().flatten().int())
    check(pool)
    print(f"{int(pool.refs.sum())} after the end")
