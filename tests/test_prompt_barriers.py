"""The hand-shake of the prompt attention's roles within an item, as a model whose every order of events is
walked through: a wait looks at one bit of its barrier's phase, so no barrier may complete twice before
everyone who waits for it has looked."""

import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_kv_cache_12_gb300", "csrc", "kv_prompt.cu")


def roles(passes, heard):
    """Each role as a list of steps ("wait" | "arrive", barrier, phase).  Barriers: S0, S1 scores of a tile, P0, P1 what
    their products wait for (`heard`: P1 also for the loader, which says so when it has seen S1), D values of a pass
    and keys of the next (two)."""
    loader, issuer, soft = [], [("arrive", "S0", 0), ("arrive", "S1", 0)], [[], []]
    for g in range(passes):
        if g:
            loader.append(("wait", "S1", g - 1))               # the stages of pass g - 2 are free
            if heard:
                loader.append(("arrive", "P1", g - 1))
        loader.append(("arrive", f"D{g % 2}", g // 2))
        for tile in (0, 1):
            if tile == 0:
                issuer.append(("wait", f"D{g % 2}", g // 2))
            issuer.append(("wait", f"P{tile}", g))
            if g + 1 < passes:
                issuer.append(("arrive", f"S{tile}", g + 1))
            soft[tile] += [("wait", f"S{tile}", g), ("arrive", f"P{tile}", g)]
    loader.append(("wait", "S1", passes - 1))
    if heard:
        loader.append(("arrive", "P1", passes - 1))
    return [loader, issuer, *soft]


def stuck(passes, heard):
    """Whether some order of events ends with a role that waits for ever."""
    steps = roles(passes, heard)
    need = {"P1": 1 + heard}                                   # arrivals that complete a phase
    seen, todo = set(), [(0,) * len(steps)]
    while todo:
        at = todo.pop()
        if at in seen:
            continue
        seen.add(at)
        came = {}
        for role, i in zip(steps, at):
            for kind, bar, _ in role[:i]:
                if kind == "arrive":
                    came[bar] = came.get(bar, 0) + 1
        moved = False
        for r, i in enumerate(at):
            if i == len(steps[r]):
                continue
            kind, bar, phase = steps[r][i]
            running = came.get(bar, 0) // need.get(bar, 1)     # the barrier's phase
            if kind == "arrive":
                assert running == phase                        # never for a phase that is not running
            elif running % 2 == phase % 2:                     # a wait sees one bit of it
                continue
            moved = True
            todo.append(at[:r] + (i + 1,) + at[r + 1:])
        if not moved and any(i < len(role) for i, role in zip(at, steps)):
            return True
    return False


def loader_is_heard():
    source = open(SOURCE, encoding="utf-8").read()
    count = re.search(r"mbar_init\(sh->bars \+ kGo \+ kRing \+ i, ([^)]*)\);", source).group(1)
    loader = source[source.index("bool load_item("):source.index("void load_tiles(")]
    says = "arrive(sh->bars + kGo + kRing + g % kRing)" in loader
    assert says == (sum(map(int, count.split("+"))) == 5)                        # four softmax warps, and the loader
    return says


@pytest.mark.parametrize("passes", [1, 2, 3, 6])
def test_no_order_of_events_leaves_a_role_behind(passes):
    assert not stuck(passes, loader_is_heard())


def test_a_loader_that_is_not_heard_can_be_left_behind():
    assert stuck(3, False)
