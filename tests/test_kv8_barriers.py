"""The barriers of the tcgen05 attention kernel (kv8_prompt.cu), as a model on the
CPU: whichever warp is held up, wherever and for however long, every wait ends.

A barrier tells its last phase from the one before by a parity bit only, so a waiter
that looks after the phase following its own has completed waits for ever (in the
kernel: until its limit). The model's roles are lists of waits and arrivals in the
kernel's order; arrivals of the tensor cores follow their issue at once."""
import pytest

STAGES = 2


class Barrier:
    def __init__(self, count):
        self.count, self.pending, self.phases = count, count, 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.pending, self.phases = self.count, self.phases + 1

    def passed(self, phase):
        """Waits for phase number `phase`, by its parity alone."""
        return self.phases % 2 != phase % 2


def row_warp(tile, steps, rescales, keys_first):
    """keys_first: a step's keys are looked for before the hand-over that the step's
    products wait for; otherwise when the step begins."""
    if keys_first and steps:
        yield "wait", ("k", 0), 0
    yield "arrive", "q"
    for j in range(steps):
        if not keys_first:
            yield "wait", ("k", j % STAGES), j // STAGES
        yield "wait", ("s", tile), j
        if j > 0 and rescales:
            yield "wait", ("o", tile), j - 1
        if keys_first and j + 1 < steps:
            yield "wait", ("k", (j + 1) % STAGES), (j + 1) // STAGES
        yield "arrive", ("p", tile)
    if steps:
        yield "wait", ("o", tile), steps - 1


def converter(steps, edge):
    for j in range(steps):
        stage, before = j % STAGES, j // STAGES - 1  # the phase that freed the stage; -1: free
        yield "wait", ("raw", 0), j
        yield "arrive", ("rawfree", 0)
        yield "wait", ("kfree", stage), before
        if j >= edge:
            yield "wait", ("raw", 1), j
        yield "arrive", ("k", stage)
        yield "wait", ("raw", 1), j
        yield "arrive", ("rawfree", 1)
        yield "wait", ("vfree", stage), before
        yield "arrive", ("v", stage)


def loader(steps):
    for j in range(steps):
        yield "wait", ("rawfree", 0), j - 1
        yield "arrive", ("raw", 0)
        yield "arrive", ("k", j % STAGES)  # the scales
        yield "wait", ("rawfree", 1), j - 1
        yield "arrive", ("raw", 1)


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
                    yield "wait", ("k", (j + 1) % STAGES), (j + 1) // STAGES
                else:
                    yield "wait", ("v", j % STAGES), j // STAGES
                seen = j
            yield "wait", ("p", i), j
            if j + 1 < n[i]:
                yield "arrive", ("s", i)
            yield "arrive", ("o", i)
            if i == 1 or j >= n[1]:
                yield "arrive", ("vfree", j % STAGES)
            if j + 1 < n[i] and (i == 1 or j + 1 >= n[1]):
                yield "arrive", ("kfree", (j + 1) % STAGES)


def finishes(n, rescales, edge, keys_first, victim, held_at):
    """Runs everyone but `victim` (held before its operation `held_at`) as far as they
    get, then everyone. Whether all end, and whether the victim got that far."""
    steps = max(n)
    roles = [row_warp(i, n[i], rescales, keys_first) for i in (0, 0, 1, 1)]
    if steps:
        roles += [converter(steps, edge), converter(steps, edge), loader(steps), issuer(n)]
    counts = {"q": 4}
    for x in range(2):
        counts.update({("k", x): 3, ("v", x): 2, ("kfree", x): 1, ("vfree", x): 1, ("s", x): 1, ("p", x): 2,
                       ("o", x): 1, ("raw", x): 1, ("rawfree", x): 2})
    bars = {k: Barrier(c) for k, c in counts.items()}
    at, done = [0] * len(roles), [False] * len(roles)
    ops = [list(r) for r in roles]

    def run(held):
        moved = True
        while moved:
            moved = False
            for r in range(len(roles)):
                while at[r] < len(ops[r]) and not (held and r == victim and at[r] == held_at):
                    op = ops[r][at[r]]
                    if op[0] == "wait" and not bars[op[1]].passed(op[2]):
                        break
                    if op[0] == "arrive":
                        bars[op[1]].arrive()
                    at[r] += 1
                    moved = True
                done[r] = at[r] == len(ops[r])

    run(True)
    reached = at[victim] == held_at
    run(False)
    return all(done), reached, len(ops[victim])


CASES = [(n0, n1) for n1 in range(0, 8) for n0 in range(max(0, n1 - 2), n1 + 1)] + [(n, 0) for n in (1, 2, 5)]


def stuck(n, rescales, edge, keys_first):
    """(role, operation) at which holding a warp up makes some wait endless."""
    found = []
    for victim in range(8 if max(n) else 4):
        at, length = 0, 1
        while at < length:
            ok, _, length = finishes(n, rescales, edge, keys_first, victim, at)
            if not ok:
                found.append((victim, at))
            at += 1
    return found


@pytest.mark.parametrize("rescales", [False, True])
@pytest.mark.parametrize("n", CASES)
def test_every_wait_ends(n, rescales):
    for edge in (0, max(n) - 1, 99):
        assert stuck(n, rescales, edge, True) == []


def test_the_model_sees_a_lapped_waiter():
    """The order that the kernel does not use: keys looked for when a step begins."""
    assert stuck((4, 4), False, 99, False) != []
