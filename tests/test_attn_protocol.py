"""The order of events between the row warps and the products of the many-rows
attention kernel, checked over every interleaving (a model; no GPU).

Two warps hold the halves of a row's scores.  For each tile of keys they wait
for the scores, vote on raising the maximum, where a row has to raise it
exchange values and rescale the sums (each warp half of their columns), and
deliver their half's weights.  The products wait for the first half's weights,
add to all columns, wait for the second half's, add again, and announce the
sums, on which the next scores' use and rescaling wait.

A program is a list of instructions; a state holds every program's place and
register and the shared counters.  All states that any order of steps reaches
are visited.
"""
import pytest


def rows(half, tiles, raising, joined):
    """A row warp: `joined` tells whether the two meet again after rescaling."""
    code = []
    for i in range(tiles):
        code += [("wait", "score", i + 1), ("meet", "vote %d" % i)]
        if i in raising:
            code.append(("meet", "exchange %d" % i))
            if i > 0:
                code += [("wait", "sum", i), ("act", "rescale", half, i)]
                if joined:
                    code.append(("meet", "rescaled %d" % i))
        code.append(("add", "weight%d" % half))
    return code + [("wait", "sum", tiles), ("meet", "end")]


def products(tiles):
    code = [("add", "score")]
    for i in range(tiles):
        code += [("wait", "weight0", i + 1), ("act", "product", 0, i), ("wait", "weight1", i + 1), ("act", "product", 1, i),
                 ("add", "sum")]
        if i + 1 < tiles:
            code.append(("add", "score"))
    return code


def explore(programs, check):
    """Visits every reachable state.  check(done, event): `event` happens after the set `done` of events.  Returns the
    number of states; raises AssertionError where programs are left waiting for ever."""
    counters = ("score", "sum", "weight0", "weight1")
    start = (tuple(0 for _ in programs), (0,) * len(counters), frozenset())
    seen, todo = {start}, [start]
    while todo:
        at, count, done = todo.pop()
        nexts = []
        for n, code in enumerate(programs):
            if at[n] == len(code):
                continue
            step = code[at[n]]
            moved = at[:n] + (at[n] + 1,) + at[n + 1:]
            if step[0] == "wait" and count[counters.index(step[1])] >= step[2]:
                nexts.append((moved, count, done))
            elif step[0] == "add":
                k = counters.index(step[1])
                nexts.append((moved, count[:k] + (count[k] + 1,) + count[k + 1:], done))
            elif step[0] == "act":
                check(done, step[1:])
                nexts.append((moved, count, done | {step[1:]}))
            elif step[0] == "meet" and n == 0 and at[1] < len(programs[1]) and programs[1][at[1]] == step:
                nexts.append(((at[0] + 1, at[1] + 1) + at[2:], count, done))
        assert nexts or all(at[n] == len(code) for n, code in enumerate(programs)), ("left waiting", at)
        for s in nexts:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    return len(seen)


def rescaled_before_products(done, event):
    if event[0] == "rescale":
        assert ("product", 0, event[2]) not in done, "a product added to sums that were not yet rescaled"


@pytest.mark.parametrize("raising", [(), (0,), (1,), (0, 1, 2), (2,), (0, 2)])
def test_sums_are_rescaled_before_products_add_to_them(raising):
    explore([rows(0, 3, raising, True), rows(1, 3, raising, True), products(3)], rescaled_before_products)


def test_the_check_sees_a_missing_meeting():
    with pytest.raises(AssertionError, match="not yet rescaled"):
        explore([rows(0, 3, (1,), False), rows(1, 3, (1,), False), products(3)], rescaled_before_products)
