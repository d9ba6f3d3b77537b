"""The barriers of the tcgen05 attention kernel in a masked call, by the model of
test_kv8_barriers: there the steps in which some row does not see every token, and in
which the keys are announced only after the values were looked at, may be any: a
window's first, its last, both, those of the sinks."""
import pytest

import test_kv8_barriers as model


def converter(steps, edges):
    for j in range(steps):
        stage, before = j % model.STAGES, j // model.STAGES - 1
        yield "wait", ("raw", 0), j
        yield "arrive", ("rawfree", 0)
        yield "wait", ("kfree", stage), before
        if j in edges:
            yield "wait", ("raw", 1), j
        yield "arrive", ("k", stage)
        yield "wait", ("raw", 1), j
        yield "arrive", ("rawfree", 1)
        yield "wait", ("vfree", stage), before
        yield "arrive", ("v", stage)


@pytest.mark.parametrize("n", [(n0, n1) for n0, n1 in model.CASES if max(n0, n1) <= 6])
def test_every_wait_ends(n, monkeypatch):
    monkeypatch.setattr(model, "converter", converter)
    steps = max(n)
    for edges in {(0,), (0, steps - 1), (1,), (1, 2), (0, 1, steps - 2, steps - 1), tuple(range(0, steps, 2)),
                  tuple(range(1, steps, 2))}:
        assert model.stuck(n, True, edges, True) == []
