"""A model of the ring of tiles in attention over the 4-bit cache (no GPU needed): two loading warps take four tiles in turn,
groups of working warps take every n-th tile, and a stage's barrier tells apart only neighbouring phases. Under random
interleavings no stage is filled again before its tile has been worked on, for the numbers of stages and groups the kernel
uses; with fewer stages than its static_assert asks for, the model shows one that is."""
import os
import random
import re

import pytest

import routed_expert_ffn_softmax_gb300 as moe

SOURCE = os.path.join(os.path.dirname(moe.__file__), "csrc", "kv4_decode.cu")
TURN = 4


def refilled_early(stages, groups, seed, tiles=60, steps=3000):
    """Whether a loader fills a stage whose tile is still worked on; one actor moves at a time, by weights that change now and
    then, so that some fall far behind."""
    rng = random.Random(seed)
    actors = range(2 + groups)
    pick = lambda: [rng.random() ** 4 + 1e-3 for _ in actors]  # noqa: E731
    weights = pick()
    done = [0] * stages   # completed phases of a stage's `empty` barrier
    held = {}             # stage -> the tile in it
    load = [0, TURN]      # each loader's next tile
    work = list(range(groups))
    for _ in range(steps):
        if rng.random() < 0.02:
            weights = pick()
        a = rng.choices(actors, weights)[0]
        if a < 2:
            t = load[a]
            st = t % stages
            # the wait for the parity of the phase that frees the stage passes when the current phase has the other parity
            if t < tiles and (done[st] & 1) != (((t // stages) & 1) ^ 1):
                if st in held or done[st] != t // stages:
                    return True
                held[st] = t
                load[a] = t + 1 if (t + 1) % TURN else t + 1 + TURN
        else:
            t = work[a - 2]
            st = t % stages
            if t < tiles and held.get(st) == t:
                del held[st]
                done[st] += 1
                work[a - 2] += groups
    return False


def constant(name):
    with open(SOURCE, encoding="utf-8") as f:
        m = re.search(rf"constexpr int {name} = ([^;]+);", f.read())
    return m[1]


def test_the_kernels_numbers():
    """The pairs below are the kernel's: its stages, and the tiles its working warps are at together."""
    assert constant("kWarps") == "8" and constant("kUnit") == "2" and constant("kLongUnit") == "kNT == 1 ? 4 : 2"
    assert constant("kStages") == "kNT == 1 ? 9 : 7" and constant("kTurn") == str(TURN)


@pytest.mark.parametrize("stages,groups", [(9, 2), (9, 4), (7, 2)])
def test_no_stage_is_filled_early(stages, groups):
    assert stages >= TURN + groups
    assert not any(refilled_early(stages, groups, seed) for seed in range(400))


def test_the_model_finds_too_few_stages():
    assert sum(refilled_early(5, 3, seed) for seed in range(50)) > 10
