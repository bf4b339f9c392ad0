"""The order of events between the row warps and the products of the many-rows
attention kernel, checked over every interleaving (a model; no GPU).

Two warps hold the halves of a row's scores.  For each tile of keys they wait
for the scores, vote on raising the maximum, where a row has to raise it
exchange values and rescale the sums (each warp half of their columns), and
deliver their half's weights.  The products wait for the first half's weights,
add to all columns, wait for the second half's, add again, and announce the
sums, on which the next scores' use and rescaling wait.

Waits are bounded: any that is not yet fulfilled may run out, after which
nothing that is computed counts, but every program has to come to its end.

A program is a list of instructions; a state holds every program's place,
whether its waits have all been fulfilled, and the shared counters.  All states
that any order of steps reaches are visited.
"""
import pytest

COUNTERS = ("item", "score", "sum", "weight0", "weight1")


def rows(half, tiles, raising, joined=True, together=True):
    """A row warp on one item.  joined: the two meet again after rescaling.  together: one whose wait has run out
    leaves with the other; otherwise it leaves alone."""
    code = []

    def wait(counter, n):
        code.append(("wait", counter, n))
        if not together:
            code.append(("leave alone",))

    def meet(label):
        code.append(("both ok" if together else "meet", label))

    wait("item", 1)
    if together:
        meet("item")
    for i in range(tiles):
        wait("score", i + 1)
        code.append(("vote", "tile %d" % i, i in raising))       # its end: the next "deliver" unless any has voted
        meet("exchange %d" % i)
        if i > 0:
            code.append(("wait", "sum", i))
            code.append(("act", "rescale", half, i))
            if joined:
                meet("rescaled %d" % i)
        code.append(("deliver", "weight%d" % half))
    wait("sum", tiles)
    meet("end")
    return code


def products(tiles):
    code = [("add", "item"), ("add", "score")]
    for i in range(tiles):
        code += [("wait", "weight0", i + 1), ("act", "product", 0, i), ("wait", "weight1", i + 1), ("act", "product", 1, i),
                 ("add", "sum")]
        if i + 1 < tiles:
            code.append(("add", "score"))
    return code


def explore(programs, check=lambda done, event: None, expiry=False):
    """Visits every reachable state of (row warp, row warp, products).  check(done, event): `event` happens after the set
    `done` of events.  expiry: waits may run out.  Raises AssertionError where a program is left waiting for ever.
    Returns how many states end with every wait fulfilled, and how many otherwise."""
    start = ((0, 0, 0), (True, True, True), (0,) * len(COUNTERS), frozenset())
    seen, todo, ends = {start}, [start], [0, 0]
    while todo:
        at, ok, count, done = todo.pop()
        nexts = []

        def move(n, to, ok=ok, count=count, done=done):
            return at[:n] + (to,) + at[n + 1:], ok, count, done

        def failed(n):
            return ok[:n] + (False,) + ok[n + 1:]

        for n, code in enumerate(programs):
            pc = at[n]
            if pc == len(code):
                continue
            step = code[pc]
            if step[0] == "wait":
                if not ok[n]:
                    nexts.append(move(n, pc + 1 if n < 2 else len(code)))
                elif count[COUNTERS.index(step[1])] >= step[2]:
                    nexts.append(move(n, pc + 1))
                elif expiry:
                    nexts.append(move(n, pc + 1 if n < 2 else len(code), ok=failed(n)))
            elif step[0] == "leave alone":
                nexts.append(move(n, pc + 1 if ok[n] else len(code)))
            elif step[0] in ("add", "deliver"):
                k = COUNTERS.index(step[1])
                nexts.append(move(n, pc + 1, count=count[:k] + (count[k] + 1,) + count[k + 1:]))
            elif step[0] == "act":
                if ok[n]:
                    check(done, step[1:])
                nexts.append(move(n, pc + 1, done=done | {step[1:]} if ok[n] else done))
            elif n == 0 and at[1] < len(programs[1]):            # a meeting of the two row warps
                other = programs[1][at[1]]
                if other[0] not in ("vote", "meet", "both ok"):
                    continue
                assert other[:2] == step[:2], ("they meet at different places", step, other)
                to = []
                for m in (0, 1):
                    c, pc = programs[m], at[m]
                    to.append(pc + 1)
                    if step[0] == "vote" and not (step[2] or not ok[0] or not ok[1]):
                        to[m] = next(j for j in range(pc, len(c)) if c[j][0] == "deliver")
                    if step[0] == "both ok" and not (ok[0] and ok[1]):
                        to[m] = len(c)
                nexts.append((tuple(to) + at[2:], ok, count, done))
        if not nexts:
            assert all(at[n] == len(code) for n, code in enumerate(programs)), ("left waiting", at)
            ends[0 if all(ok) else 1] += 1
        for s in nexts:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    return ends


def rescaled_before_products(done, event):
    if event[0] == "rescale":
        assert ("product", 0, event[2]) not in done, "a product added to sums that were not yet rescaled"


RAISING = [(), (0,), (1,), (0, 1, 2), (2,), (0, 2)]


@pytest.mark.parametrize("raising", RAISING)
def test_sums_are_rescaled_before_products_add_to_them(raising):
    good, bad = explore([rows(0, 3, raising), rows(1, 3, raising), products(3)], rescaled_before_products)
    assert good == 1 and bad == 0


def test_the_check_sees_a_missing_meeting():
    with pytest.raises(AssertionError, match="not yet rescaled"):
        explore([rows(0, 3, (1,), joined=False), rows(1, 3, (1,), joined=False), products(3)], rescaled_before_products)


@pytest.mark.parametrize("raising", RAISING)
def test_all_come_to_their_end_when_waits_run_out(raising):
    good, bad = explore([rows(0, 3, raising), rows(1, 3, raising), products(3)], rescaled_before_products, expiry=True)
    assert good == 1 and bad > 0


def test_the_check_sees_a_warp_that_leaves_alone():
    with pytest.raises(AssertionError, match="left waiting"):
        explore([rows(0, 2, (1,), together=False), rows(1, 2, (1,), together=False), products(2)], expiry=True)


# ------------------------------------------------------------------ the few-rows kernels: lanes of one warp

def lane(chunks, together):
    """A lane that waits for each chunk's copy and then joins the warp's matrix instructions on it."""
    code = []
    for i in range(chunks):
        code += [("wait", "score", i + 1), ("both ok", "wait %d" % i) if together else ("leave alone",), ("meet", "products %d" % i)]
    return code


def copies(chunks):
    return [("add", "score")] * chunks


def test_lanes_of_a_warp_give_up_together():
    good, bad = explore([lane(3, True), lane(3, True), copies(3)], expiry=True)
    assert good == 1 and bad > 0


def test_the_check_sees_a_lane_that_leaves_alone():
    with pytest.raises(AssertionError, match="left waiting"):
        explore([lane(2, False), lane(2, False), copies(2)], expiry=True)
