"""The example that decodes by trees of drafts: it runs, and its bookkeeping is right
(what the operators compute is tested elsewhere)."""
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("draft_kv8", os.path.join(ROOT, "examples", "draft_kv8.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_trees(example):
    assert example.tree_of(2, 2) == ([-1, 0, 0, 1, 1, 2, 2], [1, 3, 5, 11, 19, 37, 69])
    assert len(example.tree_of(2, 5)[0]) == 63 and len(example.tree_of(1, 3)[0]) == 4


@pytest.mark.parametrize("width,depth,page_size", [(2, 3, 16), (1, 4, 64), (3, 2, 32)])
def test_it_runs(example, width, depth, page_size):
    lengths = (70, 33, 120)
    text, accepted, steps, pool = example.generate(lengths, 20, width, depth, page_size)
    # a step adds the kept drafts and the token after them; that one is not in the cache yet
    assert pool.lens.tolist() == [n + len(t) - 1 for n, t in zip(lengths, text)]
    assert sum(map(len, text)) == len(lengths) * (steps + 1) + accepted
    pages = int(((pool.lens + page_size - 1) // page_size).sum())
    assert int((pool.refs > 0).sum()) == pages and bool((pool.refs <= 1).all())
    assert bool(((pool.table >= 0).sum(1) == (pool.lens + page_size - 1) // page_size).all())
