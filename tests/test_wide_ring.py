"""The batch product's rings (qc_int8_wide.cu) as a model on the CPU: loads that land in
any order, widening groups and matrix instructions that run whenever their waits allow.
A wait on an mbarrier tells a phase only from the one before it; with the kernel's ring
lengths no interleaving may let a wait pass on an older phase, and none may get stuck."""
from __future__ import annotations

import os
import random
import re

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                   "embedding_communication_codecs_gb300", "csrc", "qc_int8_wide.cu")


def constants():
    text = open(SRC).read()
    groups = int(re.search(r"kGroups = (\d+)", text).group(1))

    def of(name):
        text_of = re.search(name + r" = ((?:BT == \d+ \? \d+ : )+)(\d+);", text)
        lengths = {int(t): int(n) for t, n in re.findall(r"BT == (\d+) \? (\d+)", text_of.group(1))}
        return {t: lengths.get(t, int(text_of.group(2))) for t in (32, 48, 64, 96, 128)}
    return groups, of("kRing"), of("kStages")


def run(stages, ring, groups, steps, seed):
    rnd = random.Random(seed)
    full, empty, ready, freed = [0] * stages, [0] * stages, [0] * ring, [0] * ring
    issued, done, loading = 0, 0, []
    at, has_slot = list(range(groups)), [False] * groups

    def passes(phases, parity):     # mbarrier.try_wait.parity
        return (phases & 1) != parity
    while done < steps:
        can = []
        if issued < steps and passes(empty[issued % stages], ((issued // stages) & 1) ^ 1):
            can.append(("issue", None))
        can += [("land", i) for i in loading]
        for g, i in enumerate(at):
            if i < steps:
                if not has_slot[g]:
                    if passes(freed[i % ring], ((i // ring) & 1) ^ 1):
                        can.append(("slot", g))
                elif passes(full[i % stages], (i // stages) & 1):
                    can.append(("widen", g))
        if passes(ready[done % ring], (done // ring) & 1):
            can.append(("multiply", None))
        assert can, "stuck"
        what, x = rnd.choice(can)
        if what == "issue":
            assert empty[issued % stages] == issued // stages
            loading.append(issued)
            issued += 1
        elif what == "land":
            loading.remove(x)
            full[x % stages] += 1
        elif what == "slot":
            assert freed[at[x] % ring] == at[x] // ring, "a slot still in use was taken"
            has_slot[x] = True
        elif what == "widen":
            i = at[x]
            assert i < issued and i not in loading and full[i % stages] == i // stages + 1, "a stage was read early"
            empty[i % stages] += 1
            ready[i % ring] += 1
            at[x], has_slot[x] = i + groups, False
        else:
            assert ready[done % ring] == done // ring + 1
            freed[done % ring] += 1
            done += 1


@pytest.mark.parametrize("tokens", [32, 48, 64, 96, 128])
def test_no_wait_passes_on_an_older_phase(tokens):
    groups, ring, stages = constants()
    for seed in range(300):
        run(stages[tokens], ring[tokens], groups, 60, seed)


def test_the_model_sees_a_ring_that_is_too_short():
    groups, _, _ = constants()
    with pytest.raises(AssertionError):
        for seed in range(50):
            run(4, groups - 1, groups, 60, seed)
