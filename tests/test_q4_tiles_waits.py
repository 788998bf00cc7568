"""The waits of the 4-bit attention's tensor-core kernel on the products of a row tile, in every order of events (no GPU).

The kernel's waits on `o_done` (a tile's weighted values have been added) are read from its source, conditions, barriers
and parities; the rest of the protocol is written down here.  An mbarrier's parity tells a phase from the next only: a
wait that may come when the phase after the one it means has completed too never ends, and one that may come a phase
early ends at once.
"""
import os
import re

import pytest

from lattice_vq_weight_gb300 import build

NAME = "lq_attn_q4_tiles.cu"


def waits_of(text):
    """The kernel's waits on o_done, in their order, and the barrier that values arrive on: (condition, barrier, parity)."""
    text = re.sub(r"//[^\n]*", "", text)
    python = lambda c: re.sub(r"\(uint32_t\)\s*|\(int\)\s*", "", c).replace("&&", " and ").replace("||", " or ").strip()
    found = re.findall(r"if \(([^;{}]*?)\)\s*\{?\s*ok = (?:ok && |__all_sync\(0xffffffffu, )wait_on\(&o_done\[t\](?:\[(.*?)\])?, (.*?), timeout\)",
                       text)
    assert len(found) == text.count("wait_on(&o_done"), "a wait that this test does not understand"
    arrivals = re.findall(r"mma_commit\(&o_done\[t\](?:\[(.*?)\])?\);", text)
    assert len(arrivals) == 1
    waits = [tuple(python(x) or "0" for x in w) for w in found]
    # the products' warp waits before the scores, the softmax before it rescales and after its tiles
    return waits[0], waits[1], waits[2:], python(arrivals[0]) or "0"


def explore(waits, n, bufs, warps=2):
    """Run every order of the events of n tiles; raises where a wait ends too early or nothing can go on."""
    before_scores, before_rescale, at_end, values_on = waits
    buf_of = lambda j: j & 1 if bufs == 2 else 0
    parity_of = lambda j: (j >> 1 if bufs == 2 else j) & 1

    def value(expr, j):
        return int(eval(expr, {"j": j, "n": n, "B": bufs, "ok": True, "buf_of": buf_of, "parity_of": parity_of}))

    def wait(w, j, tile):
        return [("wait", ("o", value(w[1], j)), value(w[2], j), tile)] if value(w[0], j) else []

    def scores(j):
        return wait(before_scores, j, j - bufs) + [("issue", ("s", buf_of(j)), -1)] if j < n else []

    def values(j):
        return [("wait", ("p", buf_of(j)), parity_of(j), None), ("issue", ("o", value(values_on, j)), j)]

    issue = scores(0)
    for j in range(n):
        issue += scores(j + 1) + values(j) if bufs == 2 else values(j) + scores(j + 1)
    softmax = []
    for j in range(n):
        softmax.append(("wait", ("s", buf_of(j)), parity_of(j), None))
        if j > 0:
            softmax.append(("maybe", wait(before_rescale, j, j - 1)))
        softmax.append(("arrive", ("p", buf_of(j))))
    for w in at_end:
        softmax += wait(w, n - 1, None)
    softmax.append(("read", n - 1))                            # the outputs
    programs = [issue] + [softmax] * warps
    products = [op for op in issue if op[0] == "issue"]        # the tensor core ends them in their order
    # how often each barrier has completed, whatever the arrivals
    start = ((0,) * len(programs), 0, ())
    seen, todo = {start}, [start]
    while todo:
        at, ended, arrived = todo.pop()
        issued = sum(op[0] == "issue" for op in issue[:at[0]])
        done = [op[2] for op in products[:ended]]
        phases = {}
        for _, bar, _ in products[:ended]:
            phases[bar] = phases.get(bar, 0) + 1
        for bar in set(arrived):
            phases[bar] = phases.get(bar, 0) + arrived.count(bar) // warps

        def passes(op, who):
            if phases.get(op[1], 0) & 1 == op[2]:
                return False
            assert op[3] is None or op[3] in done, f"{who} goes on before the values of tile {op[3]}"
            return True

        after = [(at, ended + 1, arrived)] if ended < issued else []
        for i, program in enumerate(programs):
            if at[i] == len(program):
                continue
            op, step = program[at[i]], tuple(a + (k == i) for k, a in enumerate(at))
            if op[0] == "issue" or (op[0] == "wait" and passes(op, i)):
                after.append((step, ended, arrived))
            elif op[0] == "maybe":
                after.append((step, ended, arrived))           # (the maximum has not moved)
                if all(passes(w, i) for w in op[1]):
                    after.append((step, ended, arrived))
            elif op[0] == "arrive":
                after.append((step, ended, tuple(sorted(arrived + (op[1],)))))
            elif op[0] == "read":
                assert op[1] in done, "outputs are read before the last values are added"
                after.append((step, ended, arrived))
        finished = all(a == len(p) for a, p in zip(at, programs))
        assert after or finished, f"nothing goes on: products {ended} of {issued}, places {at}, phases {phases}"
        for s in after:
            if s not in seen:
                seen.add(s)
                todo.append(s)


@pytest.mark.parametrize("bufs", [1, 2])
@pytest.mark.parametrize("n", [1, 2, 3, 4, 5])
def test_every_wait_ends_and_none_too_early(bufs, n):
    explore(waits_of(open(os.path.join(build.CSRC, NAME)).read()), n, bufs)


def test_the_model_finds_a_wait_that_may_never_end():
    """One barrier for both buffers, and a wait for the tile before the last one after the last weights are announced."""
    once = ("j >= B", "0", "(j - B) & 1"), ("B == 2", "0", "(j - 1) & 1"), (("n > 0", "0", "(n - 1) & 1"),), "0"
    twice = once[:2] + ((("B == 2 and n > 1", "0", "n & 1"),) + once[2], "0")
    explore(once, 3, 1)
    with pytest.raises(AssertionError, match="nothing goes on"):
        explore(twice, 2, 2)
    with pytest.raises(AssertionError, match="before the last values"):
        explore(once, 2, 2)
