"""A tree of drafts against the branch of it that is kept, read token by token, with a
tolerance for each element that a wrong mask exceeds: a draft that saw its siblings, or
missed its own branch, shows."""
import numpy as np
import pytest
import torch

import kv8mask as mask
import kv8util as ref
from test_gpu_kv8 import w4  # noqa: F401
from test_gpu_kv8_keep import Layer, packed, projection

pytestmark = pytest.mark.gpu


class Step(Layer):
    """The layer's step, which keeps the queries that the attention got."""

    def step(self, pool, cache, qkv, positions, cu, m, most, tree=None):
        q, k, v = qkv.split((self.heads, self.kv_heads, self.kv_heads), 1)
        how = dict(window=self.window, sinks=2) if self.window else {}
        self.q, k = self.w4.qk_norm_rope(q, k, positions, self.table, *self.weights)
        self.w4.kv8_append(k, v, cache, pool.table, pool.lens, cu, m)
        return self.w4.kv8_attention(self.q, cache, pool.table, pool.lens, cu, m, most, tree=tree, **how)


@pytest.mark.parametrize("window", [None, 48])
@pytest.mark.parametrize("heads,kv_heads,dim,dtype,page", [
    (8, 2, 64, "bf16", 16), (32, 2, 128, "fp16", 64), (4, 4, 128, "bf16", 32), (16, 2, 128, "bf16", 64)])
@pytest.mark.parametrize("prompt,counts", [([70, 131], [9, 21]), ([2600, 131], [5, 3]), ([2600, 40], [64, 33])])
def test_a_tree_is_its_branches_element_by_element(w4, heads, kv_heads, dim, dtype, page, window, prompt, counts):
    most = max(p + c for p, c in zip(prompt, counts)) + 5
    rng = np.random.default_rng(5)
    trees = [mask.random_tree(m, rng, "tree") for m in counts]
    paths = [[d for d in range(m) if max(t, key=lambda w: bin(w).count("1")) >> d & 1]
             for m, t in zip(counts, trees)]
    layer = Step(w4, heads, kv_heads, dim, dtype, 6, window)
    first = projection(sum(prompt), heads, kv_heads, dim, dtype, 7)
    drafts = projection(sum(counts), heads, kv_heads, dim, dtype, 8)
    pages, scale = sum(-(-(p + c) // page) for p, c in zip(prompt, counts)) + 3, dim ** -0.5

    def start():
        pool = w4.kv8_pool(pages, 2, most, page)
        cache = w4.kv8_cache(pages, kv_heads, page, dim)
        w4.kv8_reserve(pool, ref.ints(prompt))
        pos = ref.ints(list(range(prompt[0])) + list(range(prompt[1])))
        layer.step(pool, cache, first, pos, ref.bounds(prompt), max(prompt), most)
        return pool, cache

    def definition(pool, cache, q, new, sees):
        return mask.attention(q, cache, pool.table, pool.lens.tolist(), new, sees, scale, dtype)

    def near(got, want, tol):
        worst = ((got.double() - want).abs() / tol.clamp_min(1e-30)).max().item()
        assert worst <= 1, worst

    # the tree
    pool, cache = start()
    depth = [bin(w).count("1") - 1 for t in trees for w in t]
    pos = ref.ints([prompt[i >= counts[0]] + d for i, d in enumerate(depth)])
    cu, path = ref.bounds(counts), packed(paths, counts)
    w4.kv8_reserve(pool, ref.ints(counts))
    got = layer.step(pool, cache, drafts, pos, cu, max(counts), most, mask.words_tensor(sum(trees, [])))
    queries, lens = layer.q, pool.lens.tolist()
    sinks = 2 if window else 0
    want, tol = definition(pool, cache, queries, counts,
                           lambda b: mask.tree_sees(lens[b], counts[b], trees[b], window, sinks))
    near(got, want, tol)
    # What two wrong masks would give is off by more, in every draft that they are wrong for. (One
    # draft of n tokens moves the result by about 1 / n of sum p |v|, of which the two tolerances
    # are 2^-9 at least: it shows among 2^7 tokens, and cannot among 2600 without a window.)
    own = [[1 << d for d in range(m)] for m in counts]
    causal = [mask.random_tree(m, None, "chain") for m in counts]
    for other in (own, causal) if window or max(prompt) < 2 ** 8 else ():
        def sees(b):  # the tree's sight of the tokens before the drafts, other's of the drafts
            s = mask.tree_sees(lens[b], counts[b], trees[b], window, sinks)
            s[:, prompt[b]:] = mask.tree_sees(lens[b], counts[b], other[b])[:, prompt[b]:]  # noqa: B023
            return s

        bad, loose = definition(pool, cache, queries, counts, sees)
        wrong = torch.tensor([x != y for t, o in zip(trees, other) for x, y in zip(t, o)], device="cuda")
        assert wrong.any()
        assert ((bad - want).abs() > 2 * (tol + loose)).flatten(1).any(1)[wrong].all()
    w4.kv8_keep(cache, pool.table, pool.lens, cu, path, max(counts))
    w4.kv8_shorten(pool, ref.ints([m - len(p) for m, p in zip(counts, paths)]))
    assert int(pool.status) == 0 and w4.w4_device_status() == 0

    # the branch
    plain, other = start()
    at = [0, counts[0]]
    for step in range(max(map(len, paths))):
        live = [b for b in (0, 1) if step < len(paths[b])]
        rows = [at[b] + paths[b][step] for b in live]
        new = [int(b in live) for b in (0, 1)]
        w4.kv8_reserve(plain, ref.ints(new))
        out = layer.step(plain, other, drafts[rows], ref.ints([prompt[b] + step for b in live]), ref.bounds(new), 1, most)
        assert torch.equal(layer.q, queries[rows])
        n = plain.lens.tolist()
        exact, near_by = definition(plain, other, layer.q, new,
                                    lambda b: mask.window_sees(n[b], new[b], window or 2 ** 31, sinks))  # noqa: B023
        near(out, exact, near_by)
        near(out, got[rows].double(), near_by + tol[rows])  # and each other
    assert pool.lens.tolist() == plain.lens.tolist() == [p + len(x) for p, x in zip(prompt, paths)]
