"""The barriers of the tcgen05 attention kernel by the model of test_kv8_barriers, in the
order in which the kernel announces products: the end of a step's second product before
the scores issued behind it. Every wait ends, with and without a mask, and no row takes an
older product's end for that of its last one."""
import pytest

import test_kv8_barriers as model
import test_kv8_masked_barriers as masked


def issuer(n):
    steps = max(n)
    yield "wait", "q", 0
    yield "wait", ("k", 0), 0
    for i in (0, 1):
        if n[i]:
            yield "arrive", ("s", i)
    yield "arrive", ("kfree", 0)
    seen = -1
    for j in range(steps):
        for i in (0, 1):
            if j >= n[i]:
                continue
            if j != seen:
                if j + 1 < steps:
                    yield "wait", ("k", (j + 1) % model.STAGES), (j + 1) // model.STAGES
                else:
                    yield "wait", ("v", j % model.STAGES), j // model.STAGES
                seen = j
            yield "wait", ("p", i), j
            yield "arrive", ("o", i)
            if j + 1 < n[i]:
                yield "arrive", ("s", i)
            if i == 1 or j >= n[1]:
                yield "arrive", ("vfree", j % model.STAGES)
            if j + 1 < n[i] and (i == 1 or j + 1 >= n[1]):
                yield "arrive", ("kfree", (j + 1) % model.STAGES)


@pytest.mark.parametrize("n", model.CASES)
def test_the_two_orders_differ_in_that_alone(n):
    mine = list(issuer(n))
    assert mine == masked.issuer(n) and sorted(map(str, mine)) == sorted(map(str, model.issuer(n)))
    for at, op in enumerate(mine):
        if op[0] == "arrive" and op[1][0] == "o" and mine[at + 1:at + 2] == [("arrive", ("s", op[1][1]))]:
            break
    else:
        assert max(n) <= 1


@pytest.mark.parametrize("rescales", [False, True])
@pytest.mark.parametrize("n", model.CASES)
def test_every_wait_ends(n, rescales, monkeypatch):
    monkeypatch.setattr(model, "issuer", issuer)
    for edge in (0, max(n) - 1, 99):
        assert model.stuck(n, rescales, edge, True) == []


@pytest.mark.parametrize("rescales", [False, True])
@pytest.mark.parametrize("n", [(n0, n1) for n0, n1 in model.CASES if max(n0, n1) <= 6])
def test_every_wait_of_a_masked_call_ends(n, rescales, monkeypatch):
    monkeypatch.setattr(model, "issuer", issuer)
    monkeypatch.setattr(model, "converter", masked.converter)
    steps = max(n)
    for edges in {(0,), (0, steps - 1), (1,), (1, 2), (0, 1, steps - 2, steps - 1), tuple(range(0, steps, 2)),
                  tuple(range(1, steps, 2))}:
        assert model.stuck(n, rescales, edges, True) == []


def test_the_model_sees_a_lapped_waiter(monkeypatch):
    """Keys looked for when a step begins, which the kernel does not do."""
    monkeypatch.setattr(model, "issuer", issuer)
    assert model.stuck((4, 4), False, 99, False) != []


@pytest.mark.parametrize("n", [(n0, n1) for n0, n1 in model.CASES if 0 < max(n0, n1) <= 5])
def test_no_row_takes_an_older_product_for_its_last(n):
    assert not masked.early(n, list(issuer(n)))
