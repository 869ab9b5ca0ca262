"""A model of the ring of tiles in attention over the 4-bit cache (no GPU needed): two loading warps take four tiles in turn,
groups of working warps take every n-th tile, and a stage's barriers tell apart only neighbouring phases. Every reachable
state of their progress is visited: no stage is filled again before its tile has been worked on, and no tile worked on before
it is there, for the numbers of stages and groups the kernel uses; with others that its static_assert refuses, some are. And a
model of how the list of tiles is shared out: every tile once, a cut segment's parts where they are looked for, counters apart."""
import os
import random
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


def _split(nts, h_kv, grid, segment, per_cta, together, whole, most_own):
    """The kernel's shares: (pieces of each CTA, a function that gives the first and last CTA of a segment and where the parts of
    a CTA of them are), every division as there."""
    segments, tiles = h_kv * sum(nt > 0 for nt in nts), h_kv * sum(nts)
    own = 0
    if segments <= grid and max(nts) <= whole:
        own = 1 << 20
    elif segments < grid:
        t = max(2, (tiles + grid - segments - 1) // (grid - segments))
        own = t if t <= most_own else 0
    pre, before, units = [0], 0, [0]
    for nt in nts:
        before += nt > 0
        pre.append(pre[-1] + nt)
        units.append(pre[-1] // own + before if own else pre[-1] + segment * before)
    ctas = h_kv * units[-1] if own else min(-(-tiles // together), grid)
    assert ctas <= grid
    if ctas == 0:
        return [], None
    extra = segment if not own and tiles >= per_cta * grid else 0
    n_units = h_kv * units[-1] if own or extra else tiles
    share, more = divmod(n_units, ctas)

    def units_of(b):
        return units[b + 1] - units[b] if own else nts[b] + extra

    def range_start(c):
        return c * share + min(c, more)

    def sequence_at(prefix, x):
        return max(b for b in range(len(nts)) if h_kv * prefix[b] <= x)

    def tile_at(x):
        if not own and not extra:
            return x
        if x >= h_kv * units[-1]:
            return tiles
        b = sequence_at(units, x)
        j, r = divmod(x - h_kv * units[b], units_of(b))
        return h_kv * pre[b] + j * nts[b] + (min(nts[b], r * own) if own else max(0, r - extra))

    def parts(b, j, seg0):
        unit0 = h_kv * units[b] + j * units_of(b) if own or extra else seg0

        def cta_of(i):
            big = more * (share + 1)
            return i // (share + 1) if i < big else more + (i - big) // share

        first = unit0 if own else cta_of(unit0 + extra)
        last = unit0 + (nts[b] - 1) // own if own else cta_of(unit0 + extra + nts[b] - 1)
        return [(c, 0 if range_start(c) >= unit0 else 1) for c in range(first, last + 1)]

    pieces = []
    for c in range(ctas):
        x, end = tile_at(range_start(c)), tile_at(range_start(c + 1))
        mine = []
        while x < end:
            b = sequence_at(pre, x)
            j, tl = divmod(x - h_kv * pre[b], nts[b])
            n = min(end - x, nts[b] - tl)
            mine.append((b, j, tl, n, x - tl))
            x += n
        pieces.append(mine)
    return pieces, parts


@pytest.mark.parametrize("segment", [0, 3])
def test_shares_cover_all_tiles_and_cut_segments_find_their_parts(segment):
    rng = random.Random(segment)
    for _ in range(1500):
        h_kv, grid = rng.randint(1, 5), rng.choice([rng.randint(1, 12), rng.randint(10, 150)])
        nts = [rng.choice([0, 1, 2, rng.randint(1, 40)]) for _ in range(rng.randint(1, 9))]
        if rng.random() < 0.2:
            nts = [nt % 9 for nt in nts]
        pieces, parts_of = _split(nts, h_kv, grid, segment, rng.randint(0, 4), rng.choice([2, 4]), rng.choice([0, 8, 40]),
                                  rng.choice([0, 6, 40]))
        seen, cut = {}, {}
        for c, mine in enumerate(pieces):
            for i, (b, j, tl, n, seg0) in enumerate(mine):
                for t in range(tl, tl + n):
                    assert seen.setdefault((b, j, t), c) == c
                if n < nts[b]:
                    cut.setdefault((b, j, seg0), []).append((c, 0 if i == 0 else 1))
        assert len(seen) == h_kv * sum(nts)
        most, used = rng.choice([2, 3, 8]), []
        for segment_at, parts in cut.items():
            assert parts == parts_of(*segment_at)
            # the counters: the first CTA's, or those of groups of more than one CTA and the second CTA's for the groups
            first, last = parts[0][0], parts[-1][0]
            if len(parts) > 2 * most:
                used += [lead for lead in range(first, last + 1, most) if lead < last] + [first + 1]
            else:
                used.append(first)
        assert len(used) == len(set(used))
