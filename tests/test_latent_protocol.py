"""Model check of the absorbed latent attention kernel's barriers (host only).

A CTA's roles (copies, scores, outputs' products, softmax) and its asynchronous
work (tile copies, both warps' products and what tells of their end, each in its own
order) go through the tiles of a piece.  A wait names the phase of its barrier by parity alone, so it
means what it says only while its barrier has completed that phase or is in it: a
wait one phase further behind passes at once, and one whose phase is followed by
another completed one never passes.  The model runs every interleaving and reports
each wait that a role reaches in such a state.

What the softmax waits for before it says that a tile's weights are ready is taken
from the kernel's source; the rest restates it."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "paged_kv_cache_213_gb300", "csrc", "latent_attention.cu")


def _roles(tiles, stages, halves, waits):
    """Per role a list of ("wait", barrier, phase), ("may", barrier, phase) for a wait
    that some tiles take (the softmax's, where the outputs follow a new reference),
    ("arrive", barrier) and ("issue", engine, barriers that its completion arrives on)."""
    copies, scores, products, softmax = [], [], [], []
    for g in range(tiles):
        s = g % stages
        if g >= stages:
            copies.append(("wait", f"empty{s}", g // stages - 1))
        copies.append(("issue", "tma", (f"full{s}",)))
        if g > 1:
            scores.append(("wait", f"p_ready{g & 1}", (g >> 1) - 1))
        scores.append(("wait", f"full{s}", g // stages))
        scores.append(("issue", "qk", (f"s_full{g & 1}",)))
        products.append(("wait", f"p_ready{g & 1}", g >> 1))
        # one barrier for all tiles, or one for the even and one for the odd ones
        products.append(("issue", "pv", (f"empty{s}",)))
        products.append(("issue", "pv", (f"pv_done{g & 1}" if halves else "pv_done",)))
        softmax.append(("wait", f"s_full{g & 1}", g >> 1))
        if g > 0:
            softmax.append(("may", f"pv_done{(g - 1) & 1}", (g - 1) >> 1) if halves else
                           ("may", "pv_done", g - 1))
        if waits and g > 1:
            softmax.append(("wait", f"pv_done{g & 1}", (g >> 1) - 1))
        softmax.append(("arrive", f"p_ready{g & 1}"))
    return copies, scores, products, softmax


def faults(tiles, stages, halves, waits):
    """The waits (role, step) that some interleaving reaches too early or too late."""
    roles = _roles(tiles, stages, halves, waits)
    engines = ("tma", "qk", "pv")
    names = sorted({x for r in roles for step in r for x in
                    (step[2] if step[0] == "issue" else (step[1],))})
    at = {n: i for i, n in enumerate(names)}
    queued = {e: [step[2] for r in roles for step in r if step[0] == "issue" and step[1] == e]
              for e in engines}
    start = ((0,) * len(roles), (0,) * len(engines), (0,) * len(engines), (0,) * len(names))
    seen, todo, found, ends = {start}, [start], set(), 0
    while todo:
        pcs, issued, finished, done = todo.pop()
        after = []
        for i, role in enumerate(roles):
            if pcs[i] == len(role):
                continue
            kind, *what = role[pcs[i]]
            p2 = pcs[:i] + (pcs[i] + 1,) + pcs[i + 1:]
            if kind == "may":
                after.append((p2, issued, finished, done))
            if kind in ("wait", "may"):
                behind = done[at[what[0]]] - what[1]  # 0: in the phase, 1: it is complete
                if behind not in (0, 1):
                    found.add((i, pcs[i]))
                elif behind == 1:
                    after.append((p2, issued, finished, done))
            elif kind == "arrive":
                k = at[what[0]]
                after.append((p2, issued, finished, done[:k] + (done[k] + 1,) + done[k + 1:]))
            else:
                e = engines.index(what[0])
                after.append((p2, issued[:e] + (issued[e] + 1,) + issued[e + 1:], finished, done))
        for e in range(len(engines)):
            if finished[e] < issued[e]:
                d = list(done)
                for n in queued[engines[e]][finished[e]]:
                    d[at[n]] += 1
                after.append((pcs, issued, finished[:e] + (finished[e] + 1,) + finished[e + 1:],
                              tuple(d)))
        ends += all(p == len(r) for p, r in zip(pcs, roles))
        for state in after:
            if state not in seen:
                seen.add(state)
                todo.append(state)
    assert found or ends, "no interleaving ends"
    return found


def _kernel(stages):
    """(halves, waits) of the kernel's form with this ring: whether even and odd tiles
    have a barrier each for the end of their products, and whether the softmax waits for
    the products of two tiles before ahead of its arrival on p_ready."""
    text = open(SOURCE).read()
    m = re.search(r"fence_proxy_async_smem\(\);\s*__syncwarp\(\);(.*?)"
                  r"mbar_arrive\(&sh\.p_ready\[g & 1\]\);", text, flags=re.S)
    assert m, "the arrival on p_ready is not where it was"
    wait = re.search(r"if \((C::STAGES > 2 && )?g > 1\)\s*wait_or_stop\(&sh\.pv_done\[g & 1\]",
                     m.group(1))
    return "pv_done[2]" in text, wait is not None and (stages > 2 or not wait.group(1))


@pytest.mark.parametrize("stages", [2, 4])
def test_every_wait_is_in_its_phase(stages):
    assert faults(9, stages, *_kernel(stages)) == set()


def test_the_model_finds_the_missing_wait():
    """Without the softmax's wait for earlier products a ring of four stages lets it
    run two tiles ahead of them: its own wait for them passes a phase early, and the
    products' wait for weights can be two phases late.  A ring of two does not, once
    even and odd tiles have a barrier each."""
    softmax, products = 3, 2
    for halves in (False, True):
        assert {role for role, _ in faults(9, 4, halves, False)} >= {softmax, products}
    assert {role for role, _ in faults(9, 2, False, False)} == {softmax}
    assert not faults(9, 2, True, False)
