"""The 8-bit cache's operators and the linear layers together, as a server runs
them. No sequence is longer than 512 tokens, so an item's result does not depend
on the batch around it, and every comparison here is exact."""
import importlib.util
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def serve():
    spec = importlib.util.spec_from_file_location("serve_kv8",
                                                  os.path.join(ROOT, "examples", "serve_kv8.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module.serve


def test_equal_starts_stay_equal(serve):
    """Forks that decode the same token read the same cache, whatever their pages."""
    text, _ = serve(lengths=(70, 129), forks=3, steps=20, distinct=False, graph=False)
    for prompt in (0, 3):
        half = [text[prompt + i][:11] for i in range(3)]
        assert half[0] == half[1] == half[2]


@pytest.mark.parametrize("page_size", [16, 64])
def test_graphs_and_compaction_change_nothing(serve, page_size):
    args = dict(lengths=(70, 200, 1), forks=2, steps=30, page_size=page_size)
    plain, _ = serve(graph=False, compact=False, **args)
    captured, _ = serve(graph=True, compact=False, **args)
    moved, pool = serve(graph=True, compact=True, **args)
    assert plain == captured == moved
    held = pool.lens[pool.lens > 0]
    pages = int(((held + page_size - 1) // page_size).sum())
    assert held.numel() == 3 and int((pool.refs > 0).sum()) == pages
    assert bool((pool.refs[:pages] == 1).all())  # the front of the pool, one owner each
    assert len({t for tokens in plain.values() for t in tokens}) > 20  # no fixed point
