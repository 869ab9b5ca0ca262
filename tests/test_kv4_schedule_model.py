"""A model of the ring of tiles in attention over the 4-bit cache (no GPU needed): two loading warps take four tiles in turn,
groups of working warps take every n-th tile, and a stage's barriers tell apart only neighbouring phases. Every reachable
state of their progress is visited: no stage is filled again before its tile has been worked on, and no tile worked on before
it is there, for the numbers of stages and groups the kernel uses; with others that its static_assert refuses, some are."""
import os
import re
from collections import deque

import pytest

import routed_expert_ffn_softmax_gb300 as moe

SOURCE = os.path.join(os.path.dirname(moe.__file__), "csrc", "kv4_decode.cu")
TURN = 4


def search(stages, groups, tiles):
    """None, or what happens too early. A state is each loader's next tile and that of two warps of each group, a quick one and
    a slow one (others of the group are between them): a stage is free when both have worked on its tile."""
    start = (0, TURN) + tuple(range(groups)) * 2
    seen, queue = {start}, deque([start])

    def phases(t, through):  # completed phases of the barrier of t's stage
        return sum(through(u) for u in range(t % stages, t + 2 * stages + 1, stages))

    while queue:
        s = queue.popleft()
        loaded = lambda u: u < s[u // TURN % 2]  # noqa: E731
        worked = lambda u: u < min(s[2 + u % groups], s[2 + groups + u % groups])  # noqa: E731
        for i, t in enumerate(s):
            if t >= tiles:
                continue
            # a wait for the parity of a phase passes when the current phase has the other parity
            if i < 2:
                done = phases(t, worked)
                if done & 1 == (t // stages & 1) ^ 1:
                    continue
                if done != t // stages:
                    return "filled", t, s
                to = t + 1 if (t + 1) % TURN else t + 1 + TURN
            else:
                full = phases(t, loaded)
                if full & 1 == t // stages & 1:
                    continue
                if full != t // stages + 1:
                    return "worked on", t, s
                to = t + groups
            n = s[:i] + (to,) + s[i + 1:]
            if i >= 2 + groups and n[i] > n[i - groups]:  # the quick one first
                continue
            if n not in seen:
                seen.add(n)
                queue.append(n)
    assert any(min(s) >= tiles for s in seen), "the ring stands still"
    return None


def constant(name):
    with open(SOURCE, encoding="utf-8") as f:
        return re.search(rf"constexpr int {name} = ([^;]+);", f.read())[1]


def test_the_kernels_numbers():
    """The pairs below are the kernel's: its stages, and the tiles its working warps are at together (8 warps, 2 or 4 of a tile's
    8 chunks each)."""
    assert constant("kWarps") == "8" and constant("kUnit") == "2" and constant("kLongUnit") == "kNT == 1 ? 4 : 2"
    assert constant("kStages") == "kNT == 1 ? 9 : 7" and constant("kTurn") == str(TURN)


@pytest.mark.parametrize("stages,groups", [(9, 2), (9, 4), (7, 2)])
def test_nothing_is_early(stages, groups):
    assert TURN % groups == 0 and stages > TURN + groups
    assert search(stages, groups, 40 if groups < 4 else 28) is None


@pytest.mark.parametrize("stages,groups", [(5, 3), (8, 3), (7, 4), (4, 2)])
def test_the_model_finds_what_is_early(stages, groups):
    assert search(stages, groups, 28)[0] in ("filled", "worked on")
