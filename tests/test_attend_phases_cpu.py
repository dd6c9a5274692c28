"""The attention kernel's product barriers as a model, every interleaving of the
issuer and the two softmax groups over short lists of parts.

A wait knows a phase by its parity: for phase n it passes once the completions
differ from n in parity, which is right only with n + 1 of them.  The model finds
waits that pass early and waits that never end.
"""
import itertools

import pytest

MEETS = {"meet0": 2, "meet1": 2}  # arrivals that complete a phase, 1 for the others


def _programs(parts, count_only):
    """Steps of the issuer and the groups; a part is (two row tiles, key tiles)."""
    issuer, group = [], [[], []]
    steps, outs, meets = [0, 0], [0, 0], 0  # phases before this part
    for two, tiles in parts:
        mine = [tiles, tiles] if two else [(tiles + 1) // 2, tiles // 2]
        issuer += [("arrive", f"s{g}") for g in (0, 1) if mine[g]]
        for j in range(mine[0]):
            for g in (0, 1):
                if j < mine[g]:
                    issuer += [("wait", f"p{g}", steps[g] + j), ("arrive", f"s{g}" if j + 1 < mine[g] else f"o{g}")]
        for g in (0, 1):
            for j in range(mine[g]):
                group[g] += [("wait", f"s{g}", steps[g] + j), ("arrive", f"p{g}")]
            if two:
                group[g] += [("wait", f"o{g}", outs[g]), ("store",)]
                if not count_only:
                    group[g].append(("wait", f"o{1 - g}", outs[1 - g]))
            else:
                group[g] += [("wait", f"o{o}", outs[o]) for o in (0, 1) if mine[o]]
                for m in ("meet0", "meet1"):
                    group[g] += [("arrive", m), ("wait", m, meets)]
        for g in (0, 1):
            steps[g] += mine[g]
            outs[g] += mine[g] > 0
        meets += not two
    return [issuer, *group]


def _fault(parts, count_only):
    programs = _programs(parts, count_only)
    start = ((0, 0, 0), ())
    seen, todo = {start}, [start]
    while todo:
        at, arrivals = todo.pop()
        moved = False
        for k, program in enumerate(programs):
            if at[k] == len(program):
                continue
            op, now = program[at[k]], dict(arrivals)
            if op[0] == "arrive":
                now[op[1]] = now.get(op[1], 0) + 1
            elif op[0] == "wait":
                done = now.get(op[1], 0) // MEETS.get(op[1], 1)
                if done % 2 == op[2] % 2:
                    continue
                if done < op[2] + 1:
                    return "early", op
            moved = True
            state = (at[:k] + (at[k] + 1,) + at[k + 1:], tuple(sorted(now.items())))
            if state not in seen:
                seen.add(state)
                todo.append(state)
        if not moved and any(a < len(p) for a, p in zip(at, programs)):
            return "stuck", at
    return None


KINDS = [(two, tiles) for two in (True, False) for tiles in (1, 2, 3)]


@pytest.mark.parametrize("length", [1, 2, 3])
def test_no_wait_passes_early_or_never_ends(length):
    for parts in itertools.product(KINDS, repeat=length):
        assert _fault(parts, count_only=True) is None, parts


@pytest.mark.parametrize("after", [(True, 1), (False, 1), (False, 2)])
def test_model_finds_the_wait_that_comes_two_phases_late(after):
    assert _fault(((True, 2), after), count_only=False)[0] == "stuck"
