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


def issuer(n):
    """The kernel's order: a product's end is announced before the scores issued behind it."""
    ops = list(model.issuer(n))
    for i in range(1, len(ops)):
        if ops[i][:2] in (("arrive", ("o", 0)), ("arrive", ("o", 1))) and ops[i - 1] == ("arrive", ("s", ops[i][1][1])):
            ops[i - 1], ops[i] = ops[i], ops[i - 1]
    return ops


def early(n, issuer_ops):
    """Whether holding the role that issues the products up somewhere lets a row that does
    not rescale take an older product's end for that of its last one, which has not come."""
    found = False
    for held_at in range(len(issuer_ops)):
        bars = {"q": model.Barrier(4)}
        for x in range(2):
            for k, c in (("k", 3), ("v", 2), ("kfree", 1), ("vfree", 1), ("s", 1), ("p", 2), ("o", 1), ("raw", 1),
                         ("rawfree", 2)):
                bars[k, x] = model.Barrier(c)
        ops = [list(model.row_warp(i, n[i], False, True)) for i in (0, 0, 1, 1)]
        ops += [list(model.converter(max(n), 99)) for _ in range(2)] + [list(model.loader(max(n))), issuer_ops]
        at = [0] * len(ops)
        for held in (True, False):
            moved = True
            while moved:
                moved = False
                for r, o in enumerate(ops):
                    while at[r] < len(o) and not (held and r == 7 and at[r] == held_at):
                        if o[at[r]][0] == "arrive":
                            bars[o[at[r]][1]].arrive()
                        elif not bars[o[at[r]][1]].passed(o[at[r]][2]):
                            break
                        elif bars[o[at[r]][1]].phases <= o[at[r]][2]:
                            found = True
                        at[r] += 1
                        moved = True
    return found


@pytest.mark.parametrize("n", [(2, 2), (3, 3), (4, 5), (5, 0)])
def test_no_row_takes_an_older_product_for_its_last(n):
    assert not early(n, issuer(n))
    assert early(n, list(model.issuer(n)))  # announced after the scores: the model sees the difference
