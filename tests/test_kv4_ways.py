"""Every way that attention over the 4-bit cache can share out and join its work is taken by a shape that the GPU tests run, and the
model of the shares holds with the kernel's own numbers (no GPU needed)."""
import random

import pytest

import kv4_shapes
from test_kv4_schedule_model import _split

GRIDS = (148, 152, 160)


@pytest.mark.parametrize("grid", GRIDS)
def test_every_way_has_a_shape(grid):
    taken = set().union(*(kv4_shapes.ways(s, grid) for s in kv4_shapes.SHAPES))
    missing = kv4_shapes.ways_there_are() - taken
    assert not missing, sorted(missing)
    unknown = {w for w in taken - kv4_shapes.ways_there_are() if "joined" in w}
    assert not unknown, sorted(unknown)


def test_shapes_are_told_apart():
    """A shape of each kind, counted by hand for 152 CTAs: 2048 tiles in 8 segments; 2 segments of 5 and 1 tiles; 41 * 4 of one."""
    def shares(**s):
        return {w for w in kv4_shapes.ways(dict(page=16, **s), 152) if w.endswith(("whole", "own", "even", "weighted", "chunks"))}
    assert shares(lens=[32768], h_q=32, h_kv=8) == {"1: weighted", "1: weighted, 4 chunks"}
    assert shares(lens=[32768], h_q=128, h_kv=8) == {"2: weighted", "2: weighted, 2 chunks"}
    assert shares(lens=[600, 0, 3], h_q=16, h_kv=1) == {"2: whole", "2: whole, 2 chunks"}
    assert shares(lens=[100] * 41, h_q=8, h_kv=4) == {"1: even", "1: even, 2 chunks"}
    assert shares(lens=[5000], h_q=8, h_kv=1) == {"1: own", "1: own, 2 chunks"}


@pytest.mark.parametrize("n,window,n_sink,want", [
    (0, 0, 0, (0, False, 0)), (-3, 0, 0, (0, False, 0)), (1, 0, 4, (1, False, 0)), (129, 0, 0, (2, False, 0)),
    (1000, 1000, 4, (8, False, 0)), (2049, 128, 130, (4, False, 2)), (300, 100, 4, (2, True, 0)), (2000, 1, 0, (1, False, 0))])
def test_tiles_of(n, window, n_sink, want):
    assert kv4_shapes.tiles_of(n, window, n_sink) == want


@pytest.mark.parametrize("eights", [1, 2])
def test_shares_with_the_kernels_numbers(eights):
    """As the test of many numbers in test_kv4_schedule_model.py does: every tile once, a cut segment's parts where they are looked
    for, counters apart, for batches of one to hundreds of sequences."""
    k = kv4_shapes.numbers(eights)
    rng = random.Random(eights)
    kinds = set()
    for _ in range(400):
        grid, h_kv = rng.choice(GRIDS), rng.choice([1, 2, 3, 4, 8])
        longest = rng.choice([1, 4, 12, 60, 400])
        nts = [rng.choice([0, 1, rng.randint(1, longest), rng.randint(1, longest)]) for _ in range(rng.choice([1, 3, 9, 40, 200]))]
        total, segments = h_kv * sum(nts), h_kv * sum(nt > 0 for nt in nts)
        own = (segments <= grid and max(nts) <= k["kWhole"]) or (
            segments < grid and max(2, -(-total // (grid - segments))) <= k["kOwn"])
        longs = not own and k["kLongUnit"] != k["kUnit"] and sum(nts) >= k["kLong"] * len(nts)
        together = k["kWarps"] * (k["kLongUnit"] if longs else k["kUnit"]) // 8
        pieces, parts_of = _split(nts, h_kv, grid, k["kSegment"], k["kSegmentFrom"], together, k["kWhole"], k["kOwn"])
        assert len(pieces) <= grid
        seen, cut = set(), {}
        for c, mine in enumerate(pieces):
            for i, (b, j, tl, n, seg0) in enumerate(mine):
                assert 0 <= tl and tl + n <= nts[b] and j < h_kv
                new = {(b, j, t) for t in range(tl, tl + n)}
                assert not new & seen
                seen |= new
                if n < nts[b]:
                    cut.setdefault((b, j, seg0), []).append((c, 0 if i == 0 else 1))
        assert len(seen) == total
        used = []
        for at, parts in cut.items():
            assert parts == parts_of(*at)
            first, last = parts[0][0], parts[-1][0]
            if len(parts) > 2 * k["kMost"]:
                used += [lead for lead in range(first, last + 1, k["kMost"]) if lead < last] + [first + 1]
                kinds.add("groups")
            else:
                used.append(first)
                kinds.add("batches" if len(parts) > k["kMost"] else "once")
        assert len(used) == len(set(used))
    assert kinds == {"once", "batches", "groups"}
