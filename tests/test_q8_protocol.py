"""Model check of the barriers of the 8-bit attention kernel for many rows (host only).

A CTA's roles (converters, queries' copies, products of the two tiles, softmax warps of
one tile) and its asynchronous work (copies, each products warp's matrix products and
commits, in their order) go through the steps of some pieces.  A wait names the phase of
its barrier by parity alone: it means what it says only while the barrier has completed
that phase or is in it.  An arrival counts for whatever phase the barrier is in: it means
what it says only in its own.  The model runs every interleaving and reports each wait
and arrival that a role reaches in another state.

Which barriers exist once and which once for even and once for odd steps is taken from the
kernel's source, as are the stages of its ring; the rest restates it."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "paged_kv_cache_213_gb300", "csrc", "q8_prefill.cu")
SOFTMAX, CONVERTERS = 2, 2  # warps in the model (the kernel has four of each)


def _barrier(name, i, halves):
    """(barrier, phase) of step i where there is one for even and one for odd steps."""
    return (f"{name}{i & 1}", i >> 1) if halves else (name, i)


def _roles(pieces, stages, halves):
    """pieces: (steps, steps that rows of the tile attend).  Per role its ("wait", barrier, phase), ("may", barrier, phase) for a wait that some
    steps take, ("arrive", barrier, phase), ("issue", engine, (barrier, phase)); and the
    arrivals that complete a phase of each barrier."""
    counts = {}
    converter, copies, products, other, softmax = [], [], [], [], []
    f = done = pc = 0  # steps so far, those with rows of the tile, pieces with such
    for n, mine in pieces:
        if mine:
            if pc > 0:
                copies.append(("wait", "q_empty", pc - 1))
            copies.append(("issue", "tma", ("q_full", pc)))
        for i in range(f, f + n):
            s = i % stages
            if i >= stages:
                converter.append(("wait", f"empty{s}", i // stages - 1))
            converter.append(("arrive", f"full{s}", i // stages))
            counts[f"full{s}"], counts[f"empty{s}"] = CONVERTERS, 2
        for i in range(n + 2):
            if i >= 2:
                empty = (f"empty{(f + i - 2) % stages}", (f + i - 2) // stages)
                if i - 2 < mine:
                    sc = done + i - 2
                    if i == 2 and pc > 0:
                        products.append(("wait", "o_free", pc - 1))
                    products.append(("wait", *_barrier("p_ready", sc, halves["p_ready"])))
                    products.append(("issue", "mma", _barrier("pv_done", sc, halves["pv_done"])))
                products.append(("issue", "mma", empty))
                other.append(("issue", "mma2", empty))
            if i < n:
                products.append(("wait", f"full{(f + i) % stages}", (f + i) // stages))
                other.append(("wait", f"full{(f + i) % stages}", (f + i) // stages))
                if i < mine:
                    if i == 0:
                        products.append(("wait", "q_full", pc))
                    s_full = _barrier("s_full", done + i, halves["s_full"])
                    products.append(("issue", "mma", s_full))
                    products.append(("arrive", *s_full))
                    if i + 1 == mine:
                        products.append(("issue", "mma", ("q_empty", pc)))
        for sc in range(done, done + mine):
            softmax.append(("wait", *_barrier("s_full", sc, halves["s_full"])))
            if sc > done:
                softmax.append(("may", *_barrier("pv_done", sc - 1, halves["pv_done"])))
            softmax.append(("arrive", *_barrier("p_ready", sc, halves["p_ready"])))
        if mine:
            softmax.append(("wait", *_barrier("pv_done", done + mine - 1, halves["pv_done"])))
            softmax.append(("arrive", "o_free", pc))
        f, done, pc = f + n, done + mine, pc + (mine > 0)
    for name, count in (("s_full", 2), ("p_ready", SOFTMAX), ("pv_done", 1)):
        for b in (f"{name}0", f"{name}1", name):
            counts[b] = count
    counts.update(q_full=1, q_empty=1, o_free=SOFTMAX)
    roles = {"copies": copies, "products": products, "other": other}
    roles.update({f"softmax{i}": softmax for i in range(SOFTMAX)})
    roles.update({f"converter{i}": converter for i in range(CONVERTERS)})
    return roles, counts


def faults(pieces, stages, halves):
    """The kinds of steps (role, "wait" or "arrive", barrier) that some interleaving
    reaches in another phase than theirs."""
    named, counts = _roles(pieces, stages, halves)
    names, roles = list(named), list(named.values())
    engines = ("tma", "mma", "mma2")
    queued = [[x[2] for r in roles for x in r if x[0] == "issue" and x[1] == e] for e in engines]
    barriers = {b: i for i, b in enumerate(sorted(counts))}
    count = [counts[b] for b in barriers]
    # one tuple: places of the roles, issued and finished by each engine, arrivals at each barrier
    R, E = len(roles), len(engines)
    start = (0,) * (R + 2 * E + len(barriers))
    A = R + 2 * E
    seen, todo, found, ends = {start}, [start], set(), 0

    def arrive(state, b, phase, who):
        k = barriers[b]
        if state[A + k] // count[k] != phase:
            found.add((who, "arrive", b))
        state[A + k] += 1

    while todo:
        at = todo.pop()
        after = []
        for i, role in enumerate(roles):
            if at[i] == len(role):
                continue
            kind, what, phase = role[at[i]]
            new = list(at)
            new[i] += 1
            if kind in ("wait", "may"):
                k = barriers[what]
                behind = at[A + k] // count[k] - phase
                if kind == "may":
                    after.append(tuple(new))
                if behind not in (0, 1):
                    found.add((names[i], "wait", what))
                elif behind == 1 and kind == "wait":
                    after.append(tuple(new))
            elif kind == "arrive":
                arrive(new, what, phase, names[i])
                after.append(tuple(new))
            else:
                new[R + engines.index(what)] += 1
                after.append(tuple(new))
        for e in range(E):
            if at[R + E + e] < at[R + e]:
                new = list(at)
                arrive(new, *queued[e][at[R + E + e]], engines[e])
                new[R + E + e] += 1
                after.append(tuple(new))
        ends += all(at[i] == len(r) for i, r in enumerate(roles))
        for state in after:
            if state not in seen:
                seen.add(state)
                todo.append(state)
    assert found or ends, "no interleaving ends"
    return found


def _kernel():
    text = open(SOURCE).read()
    m = re.search(r"uint64_t ([^;]*s_full[^;]*);", text)
    assert m, "the barriers are not where they were"
    halves = {n: f"{n}[2][2]" in m.group(1) for n in ("s_full", "p_ready", "pv_done")}
    return int(re.search(r"constexpr int kStages = (\d+);", text).group(1)), halves


@pytest.mark.parametrize("pieces", [[(5, 5)], [(1, 1), (1, 1), (3, 3)], [(3, 3), (2, 2)],
                                    [(3, 1), (2, 0), (1, 1)], [(2, 0), (4, 3)]])
def test_every_wait_and_arrival_is_in_its_phase(pieces):
    stages, halves = _kernel()
    assert faults(pieces, stages, halves) == set()


@pytest.mark.parametrize("stages", [2, 3])
def test_shorter_rings(stages):
    assert faults([(3, 3), (1, 1)], stages, dict(s_full=True, p_ready=True, pv_done=True)) == set()


def test_the_model_finds_barriers_that_even_and_odd_steps_share():
    """With the scores two steps ahead: a warp of softmax that is a step ahead of the others
    arrives in their phase, and one that waits for the outputs of a step passes with the
    end of the step before."""
    every = dict(s_full=True, p_ready=True, pv_done=True)
    got = faults([(4, 4)], 4, dict(every, p_ready=False))
    assert any(x[0].startswith("softmax") and x[1:] == ("arrive", "p_ready") for x in got)
    got = faults([(4, 4)], 4, dict(every, pv_done=False))
    assert any(x[0].startswith("softmax") and x[1:] == ("wait", "pv_done") for x in got)
    got = faults([(4, 4)], 4, dict(every, s_full=False))
    assert any(x[1:] == ("wait", "s_full") for x in got)
