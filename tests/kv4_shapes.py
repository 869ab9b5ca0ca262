"""Shapes of attention over the 4-bit cache that take each of the kernel's ways to share out and join its work, and which way a
shape takes, by the kernel's own numbers."""
import os
import re

import routed_expert_ffn_softmax_gb300 as moe

SOURCE = os.path.join(os.path.dirname(moe.__file__), "csrc", "kv4_decode.cu")
KEYS, FOLD = 128, 16


def numbers(eights):
    """The constants of Split<eights> as they stand in the source."""
    with open(SOURCE, encoding="utf-8") as f:
        text = f.read()

    def value(name):
        e = re.search(rf"constexpr int {name} = ([^;]+);", text)[1].replace("kNT", str(eights))
        m = re.fullmatch(r"(\d+) == 1 \? (\d+) : (\d+)", e)
        return int(m[2] if m[1] == "1" else m[3]) if m else eval(e, {"kD": 128})

    n = {k: value(k) for k in ("kWarps", "kUnit", "kLongUnit", "kLong", "kSegment", "kSegmentFrom", "kWhole", "kOwn", "kRow")}
    assert re.search(r"kJoinFloats = kWarps \* 8 \* kNT \* kRow;", text)
    assert re.search(r"int kMost = kJoinFloats \* 4 / \(128 \+ 512 \* 8 \* kNT\);", text)
    n["kMost"] = n["kWarps"] * 8 * eights * n["kRow"] * 4 // (128 + 512 * 8 * eights)
    return n


def tiles_of(n, window, n_sink):
    """(key tiles of a query at the end of n keys, whether its sink keys are folded into the window's first tile, tiles of sinks)."""
    if n <= 0:
        return 0, False, 0
    lo = n - window if 0 < window <= n - 1 else 0
    sinks, w0 = min(n_sink, lo), lo // KEYS
    ns = min(-(-sinks // KEYS), w0)
    before = lo - w0 * KEYS
    fold = ns > 0 and sinks <= KEYS and -(-sinks // FOLD) <= before // FOLD
    ns = 0 if fold else ns
    return ns + -(-n // KEYS) - w0, fold, ns


def ways(s, grid):
    """What a shape takes with `grid` CTAs: a set of words, all with the eights of heads (1 or 2) in front."""
    from test_kv4_schedule_model import _split
    eights = 1 if s["h_q"] // s["h_kv"] <= 8 else 2
    k = numbers(eights)
    spans = [tiles_of(n, s.get("window", 0), s.get("n_sink", 0)) for n in s["lens"]]
    nts = [nt for nt, *_ in spans]
    h_kv, total = s["h_kv"], s["h_kv"] * sum(nts)
    segments = h_kv * sum(nt > 0 for nt in nts)
    if segments <= grid and max(nts) <= k["kWhole"]:
        share = "whole"
    elif segments < grid and max(2, -(-total // (grid - segments))) <= k["kOwn"]:
        share = "own"
    else:
        share = "weighted" if total >= k["kSegmentFrom"] * grid else "even"
    longs = share in ("weighted", "even") and k["kLongUnit"] != k["kUnit"] and sum(nts) >= k["kLong"] * len(nts)
    unit = k["kLongUnit"] if longs else k["kUnit"]
    got = {share, f"{share}, {unit} chunks"}
    pieces, parts_of = _split(nts, h_kv, grid, k["kSegment"], k["kSegmentFrom"], k["kWarps"] * unit // 8, k["kWhole"], k["kOwn"])
    for mine in pieces:
        for b, j, tl, n, seg0 in mine:
            if n < nts[b] and tl == 0:
                parts = len(parts_of(b, j, seg0))
                got.add(f"{share}, {unit} chunks, joined " + ("at once" if parts <= k["kMost"] else
                                                               "in batches" if parts <= 2 * k["kMost"] else "in groups"))
    if any(fold for _, fold, _ in spans):
        got.add(f"{unit} chunks, folded sinks")
    if any(ns for *_, ns in spans):
        got.add(f"{unit} chunks, tiles of sinks")
    if s.get("window", 0) and any((n - s["window"]) % KEYS for n in s["lens"] if n > s["window"]):
        got.add(f"{unit} chunks, window inside a tile")
    if s.get("bad"):
        got.add(f"{unit} chunks, bad pages of {'less' if s['page'] < KEYS else 'more'} than a tile")
    return {f"{eights}: {w}" for w in got}


# lens: keys of each sequence; bad: (sequence, page of it) whose table entry is out of range
SHAPES = [
    dict(name="one long context", lens=[32768], h_q=32, h_kv=8, page=64),
    dict(name="one long context of odd length, 16 heads a group", lens=[32701], h_q=64, h_kv=4, page=64),
    dict(name="long windows, few sinks", lens=[30000, 29999, 31, 30117, 30040], h_q=32, h_kv=8, page=16, window=4096, n_sink=4),
    dict(name="long windows, many sinks", lens=[30000, 29999, 30117, 30040], h_q=32, h_kv=8, page=512, window=4096, n_sink=130),
    dict(name="long windows, many sinks, 16 heads a group", lens=[30000, 29999, 30117], h_q=128, h_kv=8, page=16, window=4097,
         n_sink=130),
    dict(name="bad pages of long contexts", lens=[9000, 8000, 12001], h_q=16, h_kv=8, page=16,
         bad=[(0, 0), (0, 300), (1, 499), (1, 498), (2, 7), (2, 750)]),
    dict(name="bad long pages of long contexts", lens=[9000, 8000, 12001], h_q=16, h_kv=8, page=512,
         bad=[(0, 3), (1, 15), (2, 23), (2, 0)]),
    dict(name="bad pages, 16 heads a group", lens=[700, 90, 1500], h_q=32, h_kv=2, page=16, bad=[(0, 0), (1, 5), (2, 93)]),
    dict(name="bad long pages, 16 heads a group", lens=[700, 90, 1500], h_q=32, h_kv=2, page=512, bad=[(0, 0), (2, 2)]),
    dict(name="long contexts of several lengths", lens=[5000, 1, 0, 11111, 7000, 2500, 9001], h_q=12, h_kv=4, page=32),
    dict(name="as many long contexts as make whole segments", lens=[2600, 2700, 2800] * 15, h_q=8, h_kv=4, page=64),
    dict(name="two long contexts, one head", lens=[70000, 60001], h_q=1, h_kv=1, page=128),
    dict(name="a very long context between others", lens=[400, 130000, 333], h_q=8, h_kv=1, page=256),
    dict(name="short segments in equal shares", lens=[100] * 41, h_q=16, h_kv=4, page=16),
    dict(name="short segments in equal shares, 16 heads a group", lens=[100, 0, 129] * 21, h_q=64, h_kv=4, page=16),
    dict(name="equal shares that cut", lens=[120] * 60 + [140] * 55 + [4000, 1, 8000, 1, 1500], h_q=4, h_kv=1, page=64),
    dict(name="equal shares that cut, 16 heads a group", lens=[120] * 60 + [140] * 55 + [4000, 1, 8000, 1, 1500], h_q=16, h_kv=1, page=64),
    dict(name="many short segments", lens=[(37 * i) % 700 for i in range(120)], h_q=32, h_kv=4, page=16),
    dict(name="many short segments, 16 heads a group", lens=[(37 * i) % 700 for i in range(120)], h_q=64, h_kv=4, page=16),
    dict(name="windows over short segments", lens=[(91 * i) % 3000 for i in range(64)], h_q=64, h_kv=4, page=16, window=1000,
         n_sink=4),
    dict(name="windows over short segments, 8 heads a group", lens=[(91 * i) % 3000 for i in range(64)], h_q=32, h_kv=4, page=16,
         window=1000, n_sink=4),
    dict(name="sinks of their own tiles", lens=[1500, 700, 2049], h_q=8, h_kv=2, page=16, window=128, n_sink=130),
    dict(name="sinks of their own tiles, 16 heads a group", lens=[1500, 700, 2049], h_q=32, h_kv=2, page=16, window=128, n_sink=130),
    dict(name="whole short segments", lens=[1, 900, 128, 0, 515], h_q=8, h_kv=2, page=16, bad=[(1, 2)]),
    dict(name="whole short segments, long pages", lens=[1, 900, 128, 0, 515], h_q=8, h_kv=2, page=128, bad=[(1, 2)]),
    dict(name="few CTAs a segment", lens=[1300, 4000], h_q=8, h_kv=1, page=64),
    dict(name="few CTAs a segment, 16 heads a group", lens=[1300, 4000], h_q=16, h_kv=1, page=64),
    dict(name="a segment over many CTAs", lens=[5000, 3000], h_q=8, h_kv=1, page=64),
    dict(name="a segment over many CTAs, 16 heads a group", lens=[5000, 3000], h_q=16, h_kv=1, page=64),
    dict(name="one segment over most CTAs", lens=[40000], h_q=8, h_kv=1, page=64),
    dict(name="one segment over most CTAs, 16 heads a group", lens=[40000], h_q=16, h_kv=1, page=64),
    dict(name="long contexts of 16 heads a group", lens=[40000, 0, 2500, 30001, 17, 22000, 14000, 18000], h_q=64, h_kv=4, page=64),
    dict(name="a very long context, 16 heads a group", lens=[400, 150000], h_q=16, h_kv=1, page=256),
]


def ways_there_are():
    """Everything a shape may take; what no shape can is left out with the reason."""
    all_ways = set()
    for e in (1, 2):
        joins = ("at once", "in batches", "in groups")
        all_ways |= {f"{e}: whole, 2 chunks"}                                    # nothing is cut
        all_ways |= {f"{e}: own, 2 chunks, joined {j}" for j in joins}
        # equal shares have fewer than two tiles a CTA: at 20 tiles a sequence a segment has CTAs of its own instead
        all_ways |= {f"{e}: even, 2 chunks"} | {f"{e}: even, 2 chunks, joined {j}" for j in joins}
        all_ways |= {f"{e}: weighted, 2 chunks, joined at once"}
        all_ways |= {f"{e}: 2 chunks, {w}" for w in ("folded sinks", "tiles of sinks", "window inside a tile",
                                                       "bad pages of less than a tile", "bad pages of more than a tile")}
    all_ways |= {f"1: weighted, 4 chunks, joined {j}" for j in joins}
    all_ways |= {f"2: weighted, 2 chunks, joined {j}" for j in joins}
    all_ways |= {f"1: 4 chunks, {w}" for w in ("folded sinks", "tiles of sinks", "window inside a tile",
                                                "bad pages of less than a tile", "bad pages of more than a tile")}
    return all_ways
