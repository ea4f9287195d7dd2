"""The waits of the paged attention's tensor-core kernel for its P.V products,
as a model that goes through every order of events (no GPU).

The kernel's agents: the MMA warp issues S and P.V products, the tensor core
completes them in issue order, and softmax warps wait for S, write P, and wait
for P.V products before they rescale O, overwrite P or read the result.  An
mbarrier wait names a phase by its parity alone: it passes when the last phase
completed has that parity.  So a wait for a phase that is followed by another
before the waiting warp looks never passes, and one for a phase whose
predecessor is still open passes too early.  Both are faults.

Kinds, as in the kernel's header:
  one    one query tile: two S buffers, S(j+2) behind PV(j)
  sep    P in columns of its own: S(j+1) when the softmax has loaded S(j)
  place  P where S was: S(j+1) behind PV(j)
"""
import pytest

WARPS = 2


def _softmax(kind, segments, epilogue):
    """A softmax warp's events: ("s", t) waits for S(t), ("free", t) frees S(t)
    (sep), ("p", t) hands P(t) over, ("pv", t) waits for PV(t); "pv?" is a wait
    that depends on the scores."""
    ev, t = [], 0
    for n in segments:
        for j in range(n):
            ev.append(("s", t))
            if kind == "sep":
                ev.append(("free", t))
            if j > 0 and kind != "place":
                ev.append(("pv?", t - 1))
            if kind == "sep" and t > 0:
                ev.append(("pv", t - 1))
            ev.append(("p", t))
            t += 1
        ev += [("pv", t + d) for d in epilogue if t + d >= 0]
    return ev


def _mma(kind, segments):
    """The MMA warp's events: it waits for ("free", t) or ("p", t) of all
    warps and issues ("S", t) or ("PV", t)."""
    ev, t = [], 0
    for n in segments:
        def s(j):
            if kind == "sep" and j > 0:
                ev.append(("free", t + j - 1))
            ev.append(("S", t + j))
        s(0)
        if kind == "one" and n > 1:
            s(1)
        for j in range(n):
            if kind == "sep" and j + 1 < n:
                s(j + 1)
            ev.extend((("p", t + j), ("PV", t + j)))
            if kind == "place" and j + 1 < n:
                s(j + 1)
            if kind == "one" and j + 2 < n:
                s(j + 2)
        t += n
    return ev


def _faults(kind, segments, epilogue, pv_bars):
    """The faults that some order of events leads to."""
    soft, mma = _softmax(kind, segments, epilogue), _mma(kind, segments)
    s_bars = 2 if kind == "one" else 1
    issued_at = [i for i, e in enumerate(mma) if e[0] in "SPV" and e[0].isupper()]
    products = [mma[i] for i in issued_at]
    found, seen = set(), set()
    todo = [((0,) * WARPS, 0, 0)]  # places of the warps, of the MMA warp; products complete
    while todo:
        state = todo.pop()
        if state in seen:
            continue
        seen.add(state)
        warps, m, done = state
        complete = products[:done]

        def passes(what, t, bars):
            """A wait for phase t // bars of barrier t % bars."""
            phases = sum(1 for w, x in complete if w == what and x % bars == t % bars)
            ok = (phases - 1) % 2 == (t // bars) % 2
            if ok and (what, t) not in complete:
                found.add("early")
            return ok

        moved = False
        for w in range(WARPS):
            if warps[w] == len(soft):
                continue
            kind_of, t = soft[warps[w]]
            go = True
            if kind_of == "s":
                go = passes("S", t, s_bars)
            elif kind_of == "pv":
                go = passes("PV", t, pv_bars)
            after = warps[:w] + (warps[w] + 1,) + warps[w + 1:]
            if kind_of == "pv?":  # also without the wait
                todo.append((after, m, done))
                moved = True
                go = passes("PV", t, pv_bars)
            if go:
                todo.append((after, m, done))
                moved = True
        if m < len(mma):
            e = mma[m]
            if e[0].isupper() or all(e in soft[:p] for p in warps):
                todo.append((warps, m + 1, done))
                moved = True
        if done < sum(1 for i in issued_at if i < m):
            todo.append((warps, m, done + 1))
            moved = True
        if not moved and (m < len(mma) or any(p < len(soft) for p in warps)):
            found.add("stuck")
    return found


SEGMENTS = [(1,), (2,), (3, 1, 2), (4, 3), (1, 1, 5)]


@pytest.mark.parametrize("segments", SEGMENTS)
@pytest.mark.parametrize("kind,pv_bars", [("one", 2), ("sep", 1), ("place", 1)])
def test_waits_for_products_pass_when_they_are_complete(kind, pv_bars, segments):
    # the epilogue waits for the last product alone
    assert _faults(kind, segments, (-1,), pv_bars) == set()


@pytest.mark.parametrize("kind", ["one", "sep"])
def test_the_model_finds_waits_that_may_be_late_or_early(kind):
    # the last but one first: it may be over, with the last one complete too
    assert "stuck" in _faults(kind, (3, 2), (-2, -1), 1)
    # one barrier and the last product alone: passes on the phase before it
    if kind == "one":
        assert "early" in _faults(kind, (3, 2), (-1,), 1)
