"""A paged cache held in 4 bits on the GPU, through the binding, against plain 64-bit forms (needs a GPU)."""
import pytest
import torch

import paged_reference as ref
import routed_expert_ffn_softmax_gb300 as moe
import step_reference as step

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
D = 128
SCALE = D ** -0.5


@pytest.fixture(scope="module", autouse=True)
def _built():
    from routed_expert_ffn_softmax_gb300 import build
    build.build()
    moe.load()
    yield


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def randn(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).to(DEV)


# ---------------------------------------------------------------- norm, rotation, store
def head_inputs(N, h_q, h_kv, rot, axes, norm=True, pad=0, seed=0, far=4096, size=1.0):
    g = torch.Generator().manual_seed(seed)
    wide = (size * torch.randn(N, (h_q + 2 * h_kv) * D + pad, generator=g)).to(torch.bfloat16).to(DEV)
    s = dict(qkv=wide[:, :(h_q + 2 * h_kv) * D], inv=None, pair=None)
    s["w"] = [(1 + 0.2 * torch.randn(D, generator=g)).to(torch.bfloat16).to(DEV) if norm else None for _ in range(2)]
    if rot:
        s["inv"] = (1e6 ** (-torch.arange(0, rot, 2).double() / rot)).float().to(DEV)
    s["pos"] = torch.randint(0, far, (axes, N) if axes > 1 else (N,), generator=g, dtype=torch.int32).to(DEV)
    if axes > 1:
        s["pair"] = torch.randint(0, axes, (rot // 2,), generator=g, dtype=torch.int32).to(DEV)
    return s


def store_both(s, N, h_q, h_kv, page, num_pages, slots, interleaved):
    """The bf16 call's outputs and the 4-bit call's."""
    q16, q4 = (torch.full((N, h_q, D), -9.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    k, v = (torch.zeros(num_pages, h_kv, page, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    raw = torch.zeros(num_pages, h_kv, page // 16, step.BLOCK_BYTES, dtype=torch.uint8, device=DEV)
    args = (s["qkv"], *s["w"], 1e-6, s["inv"])
    if s["pair"] is None:
        moe.moe_qk_norm_rope(*args, s["pos"], slots, q16, k, v, interleaved=interleaved)
    else:
        moe.moe_qk_norm_mrope(*args, s["pair"], s["pos"], slots, q16, k, v, interleaved=interleaved)
    moe.moe_qk_norm_rope_kv4(*args, s["pair"], s["pos"], slots, q4, raw, interleaved=interleaved)
    torch.cuda.synchronize()
    return q16, k, v, q4, raw


def parts(raw, i):
    at = i * step.BLOCK_BYTES // 2
    codes = raw[..., at:at + 1024].unflatten(-1, (16, 64)).flatten(2, 3)
    scales = raw[..., at + 1024:at + 1152].contiguous().view(torch.bfloat16).unflatten(-1, (16, 4)).flatten(2, 3)
    return codes, scales


STORES = [
    # N, h_q, h_kv, page, rot, axes, norm, interleaved, pad
    (1, 16, 2, 16, 128, 1, True, False, 0),
    (1, 1, 1, 16, 0, 1, False, False, 0),
    (33, 32, 4, 16, 128, 1, True, False, 8),
    (70, 5, 1, 32, 128, 3, True, False, 0),
    (257, 6, 3, 64, 64, 1, True, False, 0),
    (65, 3, 3, 128, 32, 2, False, False, 16),
    (129, 32, 8, 1024, 128, 4, True, True, 0),
    (40, 7, 1, 16, 48, 1, True, True, 0),
    (2000, 64, 4, 16, 128, 1, True, False, 0),
    (500, 2, 5, 32, 16, 1, False, False, 0),
]


@pytest.mark.parametrize("N,h_q,h_kv,page,rot,axes,norm,interleaved,pad", STORES)
def test_store_holds_the_bf16_rows_in_4_bits(N, h_q, h_kv, page, rot, axes, norm, interleaved, pad):
    """The codes are exactly those of the rows that the bf16 call stores; other rows and a token without a slot are left."""
    s = head_inputs(N, h_q, h_kv, rot, axes, norm, pad, seed=N)
    num_pages = ref.up(N, page) + 2
    slots = torch.randperm(num_pages * page, generator=torch.Generator().manual_seed(N))[:N].to(torch.int32)
    if N > 20:
        slots[3], slots[17] = -1, num_pages * page
    q16, k, v, q4, raw = store_both(s, N, h_q, h_kv, page, num_pages, slots.to(DEV), interleaved)
    assert torch.equal(q16, q4)
    for i, rows in enumerate((k, v)):
        c, sc = step.quantise(rows)
        codes, scales = parts(raw, i)
        stored = torch.zeros(num_pages * page, dtype=torch.bool, device=DEV)
        ok = (slots >= 0) & (slots < num_pages * page)
        stored[slots[ok].long()] = True
        stored = stored.view(num_pages, 1, page).expand(-1, h_kv, -1)
        assert torch.equal(codes[stored], step.pack_rows(c)[stored])
        assert torch.equal(scales[stored], sc[stored])
        assert not codes[~stored].any() and not scales[~stored].any()


@pytest.mark.parametrize("size", [1e-39, 1e-30, 1e30])
def test_store_of_tiny_and_huge_values(size):
    s = head_inputs(40, 4, 2, 0, 1, norm=False, size=size)
    slots = torch.arange(40, dtype=torch.int32, device=DEV)
    _, k, v, _, raw = store_both(s, 40, 4, 2, 16, 3, slots, False)
    for i, rows in enumerate((k, v)):
        c, sc = step.quantise(rows)
        codes, scales = parts(raw, i)
        live = (torch.arange(48, device=DEV) < 40).view(3, 1, 16).expand(-1, 2, -1)
        assert torch.equal(codes[live], step.pack_rows(c)[live]) and torch.equal(scales[live], sc[live])


def test_store_halves_and_zeros():
    """Quotients that are halves go to even codes, a group of zeros has scale 0, a group with NaN or infinity reads as NaN."""
    x = torch.zeros(1, 3 * D)
    x[0, D:D + 32] = torch.tensor([7.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 3.5, 4.5, 5.5, 6.5, -6.5] + [0.0] * 20)  # scale 1
    x[0, D + 64:D + 96] = float("nan")
    x[0, 2 * D + 5], x[0, 2 * D + 40] = float("inf"), float("nan")
    s = dict(qkv=x.to(torch.bfloat16).to(DEV), w=(None, None), inv=None, pair=None, pos=i32([0]))
    *_, raw = store_both(s, 1, 1, 1, 16, 1, i32([2]), False)
    codes, scales = (p[0, 0, 2] for p in parts(raw, 0))
    assert step.unpack_rows(codes)[:12].tolist() == [7, 0, 2, 2, 0, -2, -2, 4, 4, 6, 6, -6]
    assert scales[0] == 1 and scales[1] == 0 and scales[2].isnan() and scales[3] == 0
    kb, vb = (torch.zeros(1, 1, 16, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ws = moe.alloc_paged_workspace(device=DEV)
    moe.moe_kv4_load(raw, i32([[0]]), i32([2]), i32([3]), kb, vb, i32([[0]]), ws)
    assert kb[0, 0, 2, 64:96].isnan().all() and not kb[0, 0, 2, 32:64].any() and kb[0, 0, 2, 7] == 4
    assert vb[0, 0, 2, :64].isnan().all() and not vb[0, 0, 2, 64:].any()


# ---------------------------------------------------------------- rows read back
@pytest.mark.parametrize("page,h_kv", [(16, 1), (16, 4), (32, 3), (128, 2), (1024, 1)])
def test_load(page, h_kv):
    lens = [0, 1, 15, 16, 17, 300, 1, 64, 2050]
    first = [0, 0, 3, 16, 16, 33, 1, 60, 0]
    c = step.Kv4(lens, h_kv, page, DEV, seed=page, codes_lo=-8)
    need = [ref.up(n, page) for n in lens]
    order = torch.randperm(sum(need) + 2, generator=torch.Generator().manual_seed(1)).tolist()
    dst = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
    for b, n in enumerate(need):
        for i in range(n):
            dst[b, i] = order.pop()
    for begins in (first, None):
        k, v = (torch.full((sum(need) + 2, h_kv, page, D), -3.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        want = [k.clone(), v.clone()]
        ws = moe.alloc_paged_workspace(device=DEV)
        moe.moe_kv4_load(c.raw, c.table, None if begins is None else i32(begins), i32(lens), k, v, dst.to(DEV), ws)
        torch.cuda.synchronize()
        assert moe.workspace_status(ws) == 0 and not ws.any()
        for b, n in enumerate(lens):
            for p in range(0 if begins is None else begins[b], n):
                for w, rows in zip(want, c.values(b)):
                    w[dst[b, p // page], :, p % page] = rows[p].to(torch.bfloat16)
        assert torch.equal(k, want[0]) and torch.equal(v, want[1])


def test_load_bad_pages_and_lengths():
    lens = [40, 40, 40, 16, 16, 20]
    c = step.Kv4(lens, 2, 16, DEV, extra=0)
    dst = torch.arange(18, dtype=torch.int32).view(6, 3)
    c.table[0, 1], dst[1, 2], dst[1, 0] = 1 << 29, 18, -1
    said = i32([40, 40, -1, 16, 49, 20])
    k, v = (torch.full((18, 2, 16, D), -3.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    want = k.clone(), v.clone()
    ws = moe.alloc_paged_workspace(device=DEV)
    moe.moe_kv4_load(c.raw, c.table, i32([0, 0, 0, -1, 0, 30]), said, k, v, dst.to(DEV), ws)
    torch.cuda.synchronize()
    assert moe.workspace_status(ws) == 6
    for w, kv in zip(want, (0, 1)):
        for b, rows in ((0, range(40)), (1, range(16, 32))):
            for p in rows:
                w[dst[b, p // 16], :, p % 16] = 0.0 if b == 0 and p // 16 == 1 else c.values(b)[kv][p].to(torch.bfloat16)
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])
    ws.zero_()
    moe.moe_kv4_load(c.raw, c.table[3:4], i32([0]), i32([99]), k, v, dst[3:4].to(DEV), ws)
    assert moe.workspace_status(ws) == 4


# ---------------------------------------------------------------- one token per sequence
def decode(c, lens, h_q, scale=SCALE, window=0, n_sink=0, seed=1, hide=True, ws=None, q=None, status=0):
    B = len(lens)
    q = randn(B, h_q, D, seed=seed) if q is None else q
    sees = []
    for b, n in enumerate(lens):
        key = torch.arange(max(n, 0), device=DEV)
        sees.append(ref.visible(n - 1, key, window, n_sink))
        if hide and n > 0:
            c.hide(b, ~sees[-1])
    out = torch.full((B, h_q, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    ws = moe.alloc_paged_workspace(B, B, h_q, c.h_kv, D, device=DEV) if ws is None else ws
    moe.moe_gqa_kv4_decode(q, c.raw, c.table, i32(lens), scale, out, ws, window=window, n_sink=n_sink)
    torch.cuda.synchronize()
    assert moe.workspace_status(ws) == status and not ws[4:4096].any()
    return q, out, sees


def check_decode(c, lens, q, out, sees, scale=SCALE, what=""):
    for b, n in enumerate(lens):
        k, v = c.values(b)
        step.check(out[b], *step.attend(q[b], k, v, sees[b], scale, c.rows[b][0][1]), max(n, 1), f"{what} sequence {b} of {n}")


LENS = [1, 0, 15, 16, 17, 127, 128, 129, 255, 700, 1, 2000]


@pytest.mark.parametrize("h_q,h_kv", [(1, 1), (2, 1), (12, 4), (7, 1), (8, 1), (16, 2), (9, 1), (32, 2), (30, 2), (40, 5)])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_decode(h_q, h_kv, page):
    c = step.Kv4(LENS, h_kv, page, DEV, seed=h_q, codes_lo=-8)
    check_decode(c, LENS, *decode(c, LENS, h_q))


@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 1), (16, 4), (100, 0), (100, 1), (128, 130), (513, 4), (5000, 4), (300, 17)])
@pytest.mark.parametrize("page", [16, 32, 128])
def test_decode_window(page, window, n_sink):
    lens = [1, 40, 128, 129, 700, 1500, 5, 2049]
    c = step.Kv4(lens, 2, page, DEV, seed=window)
    q, out, sees = decode(c, lens, 8, window=window, n_sink=n_sink)
    check_decode(c, lens, q, out, sees, what=f"window {window} sinks {n_sink}")


@pytest.mark.parametrize("h_q,h_kv,page,n", [(8, 1, 16, 40000), (16, 1, 64, 30001), (4, 4, 1024, 9000)])
def test_decode_long(h_q, h_kv, page, n):
    """One long sequence over all SMs, and a short one behind it."""
    c = step.Kv4([n, 3], h_kv, page, DEV)
    check_decode(c, [n, 3], *decode(c, [n, 3], h_q))


def test_decode_many_sequences():
    lens = torch.randint(0, 40, (2048,), generator=torch.Generator().manual_seed(3)).tolist()
    c = step.Kv4(lens, 1, 16, DEV)
    q, out, sees = decode(c, lens, 2, hide=False)
    for b in list(range(40)) + list(range(2008, 2048)):
        k, v = c.values(b)
        step.check(out[b], *step.attend(q[b], k, v, sees[b], SCALE, c.rows[b][0][1]), max(lens[b], 1), f"sequence {b}")


@pytest.mark.parametrize("scale", [0.0, -0.1, 3.0])
def test_decode_scales(scale):
    lens = [300, 17]
    c = step.Kv4(lens, 2, 16, DEV)
    check_decode(c, lens, *decode(c, lens, 8, scale=scale), scale=scale)


@pytest.mark.parametrize("spread", [0.5, 2.0])
def test_decode_scales_of_values_far_apart(spread):
    """Scales of keys and values over several powers of ten; the largest p s may belong to a key of little weight."""
    lens = [700, 90, 33]
    c = step.Kv4(lens, 2, 32, DEV, spread=spread)
    check_decode(c, lens, *decode(c, lens, 8, scale=SCALE / 10 ** spread), scale=SCALE / 10 ** spread)


@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("decades", [1, 3, 5])
def test_decode_value_scales_far_apart(decades, window):
    """Value scales over up to ten powers of ten beside ordinary scores: between keys, groups and sequences."""
    lens = [700, 90, 33, 3000]
    c = step.Kv4(lens, 2, 16, DEV, seed=decades)
    g = torch.Generator().manual_seed(decades)
    for b, n in enumerate(lens):
        k, (codes, s) = c.rows[b]
        s = (s.float() * 10 ** (decades * (2 * torch.rand(n, 2, 4, generator=g) - 1)).to(DEV)).to(torch.bfloat16)
        c.rows[b] = [k, (codes, s)]
        c.put(b, slice(0, n), *c.rows[b])
    check_decode(c, lens, *decode(c, lens, 16, window=window, n_sink=1))


@pytest.mark.parametrize("factor", [2.0 ** -60, 2.0 ** -20, 2.0 ** 20, 2.0 ** 60])
def test_decode_sizes_of_queries_and_values(factor):
    """Queries times a factor and the scale by its inverse change nothing; values times a factor only the output's size."""
    lens = [260, 31]
    c = step.Kv4(lens, 1, 16, DEV, seed=5)
    q, out, _ = decode(c, lens, 8, hide=False)
    _, same, _ = decode(c, lens, 8, hide=False, q=q * factor, scale=SCALE / factor)
    assert torch.equal(out, same)
    if abs(factor) <= 2.0 ** 60:
        scales = c.part(1, "scales")
        scales.copy_((scales.contiguous().view(torch.bfloat16) * factor).view(torch.uint8))
        c.rows = [[k, (v[0], v[1] * factor)] for k, v in c.rows]
        _, big, sees = decode(c, lens, 8, hide=False, q=q)
        for b, n in enumerate(lens):
            k, v = c.values(b)
            want = step.attend(q[b], k, v / factor, sees[b], SCALE, c.rows[b][0][1])
            step.check(big[b].double() / factor, *want, n, "values")


def test_decode_query_components_far_apart():
    """One component of a query head 2^10 times the others, beside codes of 0: the offset of the codes, which it is
    multiplied with all the same, leaves 2^-24 * 8 * 2^10 of a scale, far below the tolerance."""
    c = step.Kv4([50], 1, 16, DEV)
    codes, sc = c.rows[0][0]
    codes[:, :, 5] = 0
    c.put(0, slice(0, 50), (codes, sc), c.rows[0][1])
    q = randn(1, 4, D, seed=2)
    q[:, :, 5] = 2.0 ** 10
    check_decode(c, [50], *decode(c, [50], 4, hide=False, q=q))


def test_decode_nan_query_and_visible_nan():
    lens = [40, 40, 40]
    c = step.Kv4(lens, 2, 16, DEV)
    q = randn(3, 8, D)
    q[1, 2, 7] = float("nan")
    _, out, sees = decode(c, lens, 8, q=q, hide=False)
    assert out[1, 2].isnan().all() and torch.isfinite(out[1, [0, 1, 3, 4, 5, 6, 7]].float()).all()
    k, v = c.rows[2]
    s = v[1].clone()
    s[11, 1, 2] = float("nan")
    c.put(2, slice(0, 40), k, (v[0], s))
    _, out, _ = decode(c, lens, 8, q=randn(3, 8, D), hide=False)
    assert out[2, 4:, 64:96].isnan().all() and torch.isfinite(out[2, :4].float()).all() and torch.isfinite(out[0].float()).all()


def test_decode_bad_pages_and_lengths():
    """A visible page out of range reads as zeros (status 6), a bad length as an empty sequence (status 4 alone)."""
    lens = [70, 200, 33]
    c = step.Kv4(lens, 2, 16, DEV, extra=0)
    c.table[0, 2], c.table[1, 12] = c.raw.shape[0], -1
    q, out, sees = decode(c, lens, 8, hide=False, status=6)
    for b, rows in ((0, slice(32, 48)), (1, slice(192, 200))):
        k, v = c.values(b)
        k[rows], v[rows] = 0, 0
        step.check(out[b], *step.attend(q[b], k, v, sees[b], SCALE), lens[b], "bad page")
    k, v = c.values(2)
    step.check(out[2], *step.attend(q[2], k, v, sees[2], SCALE), 33, "other sequence")
    for bad in (-1, 13 * 16 + 1, 1 << 30):
        q, out, _ = decode(c, [bad, 0, 33], 8, hide=False, status=4)
        assert not out[:2].any()
        step.check(out[2], *step.attend(q[2], *c.values(2), sees[2], SCALE), 33, "beside a bad length")


def test_decode_bad_pages_of_many_tokens():
    """A page that spans several tiles, and one that ends inside a tile."""
    lens = [1500, 1100]
    c = step.Kv4(lens, 1, 512, DEV, extra=0)
    c.table[0, 1], c.table[1, 2] = -5, 1 << 30
    q, out, sees = decode(c, lens, 4, hide=False, status=6)
    for b, rows in ((0, slice(512, 1024)), (1, slice(1024, 1100))):
        k, v = c.values(b)
        k[rows], v[rows] = 0, 0
        step.check(out[b], *step.attend(q[b], k, v, sees[b], SCALE), lens[b], "bad page")


def test_decode_repeats_exactly_on_one_workspace():
    lens = [3000, 5, 900, 1]
    c = step.Kv4(lens, 2, 16, DEV)
    ws = moe.alloc_paged_workspace(4, 4, 32, 2, D, device=DEV)
    outs = [decode(c, lens, h, ws=ws, hide=False)[1] for h in (32, 4, 32, 4, 32)]
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[0], outs[4]) and torch.equal(outs[1], outs[3])


def test_decode_graph_and_streams():
    lens = [1000, 70]
    c = step.Kv4(lens, 2, 16, DEV)
    q, want, _ = decode(c, lens, 16, hide=False)
    out, ws = torch.zeros_like(want), moe.alloc_paged_workspace(2, 2, 16, 2, D, device=DEV)
    n = i32(lens)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            moe.moe_gqa_kv4_decode(q, c.raw, c.table, n, SCALE, out, ws)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    # two calls at once, each with its own workspace, one given its stream by the argument
    outs, wss = [torch.zeros_like(want) for _ in range(2)], [torch.zeros_like(ws) for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for o, w, s in zip(outs, wss, streams):
        for _ in range(5):
            moe.moe_gqa_kv4_decode(q, c.raw, c.table, n, SCALE, o, w, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


@pytest.mark.parametrize("h_q,h_kv,page,window", [(32, 4, 16, 0), (64, 4, 32, 300), (16, 16, 128, 0)])
def test_decode_ragged_batches_repeat_exactly(h_q, h_kv, page, window):
    """Many whole and cut pieces per CTA: checked once, then 30 more calls give the same bits."""
    g = torch.Generator().manual_seed(h_q)
    lens = torch.randint(0, 1200, (100,), generator=g).tolist()
    lens[7], lens[8] = 0, 9000
    c = step.Kv4(lens, h_kv, page, DEV, seed=h_q)
    q, out, sees = decode(c, lens, h_q, window=window, n_sink=5, hide=False)
    check_decode(c, lens, q, out, sees)
    ws, n, again = moe.alloc_paged_workspace(100, 100, h_q, h_kv, D, device=DEV), i32(lens), torch.empty_like(out)
    for _ in range(30):
        again.fill_(float("nan"))
        moe.moe_gqa_kv4_decode(q, c.raw, c.table, n, SCALE, again, ws, window=window, n_sink=5)
        assert torch.equal(again, out)
    assert moe.workspace_status(ws) == 0


@pytest.mark.parametrize("h_q", [8, 32])
def test_decode_short_and_empty_sequences_share_the_sms(h_q):
    """Runs of empty sequences in front, between and behind; segments of fewer tiles than a start counts for."""
    g = torch.Generator().manual_seed(h_q)
    lens = [0] * 60 + torch.randint(0, 300, (90,), generator=g).tolist() + [0] * 40 + [5000, 1, 0, 129] * 3 + [0] * 9
    c = step.Kv4(lens, 2, 16, DEV, seed=h_q)
    check_decode(c, lens, *decode(c, lens, h_q))


def test_decode_one_sequence_over_all_ctas():
    """More parts of a cut segment than are joined at once, for 1, 5, 8, 9 and 16 heads."""
    n = 128 * 152 * 2 + 77
    c = step.Kv4([n], 1, 64, DEV)
    for h_q in (1, 5, 8, 9, 16):
        check_decode(c, [n], *decode(c, [n], h_q, hide=False))


@pytest.mark.parametrize("h_q,h_kv", [(8, 1), (32, 2)])
def test_decode_joins_in_groups_repeat_exactly(h_q, h_kv):
    """Segments cut into more pieces than are joined at once, between shorter ones, on one workspace: the same bits every time."""
    lens = [40000, 0, 2500, 1, 30001, 17]
    c = step.Kv4(lens, h_kv, 64, DEV, seed=h_q)
    q, out, sees = decode(c, lens, h_q, hide=False)
    check_decode(c, lens, q, out, sees)
    ws = moe.alloc_paged_workspace(len(lens), len(lens), h_q, h_kv, D, device=DEV)
    full, first, again = i32(lens), [40000, 0, 0, 0, 0, 0], torch.empty_like(out)
    alone = decode(c, first, h_q, hide=False, q=q)[1]
    for _ in range(20):
        for n, want in ((full, out), (i32(first), alone)):
            again.fill_(float("nan"))
            moe.moe_gqa_kv4_decode(q, c.raw, c.table, n, SCALE, again, ws)
            assert torch.equal(again, want)
    assert moe.workspace_status(ws) == 0 and not ws[4:4096].any()


def test_calls_without_work():
    """No tokens, no sequences, sequences without keys."""
    raw = moe.alloc_kv4_cache(2, 2, 16, DEV)
    ws = moe.alloc_paged_workspace(4, 4, 8, 2, D, device=DEV)
    none = lambda *s, t=torch.bfloat16: torch.empty(*s, dtype=t, device=DEV)  # noqa: E731
    k, v = none(2, 2, 16, D), none(2, 2, 16, D)
    moe.moe_qk_norm_rope_kv4(none(0, 12 * D), None, None, 0.0, None, None, none(0, t=torch.int32), none(0, t=torch.int32),
                             none(0, 8, D), raw)
    moe.moe_qk_norm_mrope(none(0, 12 * D), None, None, 0.0, None, None, none(3, 0, t=torch.int32), none(0, t=torch.int32),
                          none(0, 8, D), k, v)
    moe.moe_kv4_load(raw, none(0, 2, t=torch.int32), None, none(0, t=torch.int32), k, v, none(0, 2, t=torch.int32), ws)
    moe.moe_gqa_kv4_decode(none(0, 8, D), raw, none(0, 2, t=torch.int32), none(0, t=torch.int32), SCALE, none(0, 8, D), ws)
    moe.moe_add_rms_norm(none(0, 256), none(0, 256), none(256), 1e-6, None, none(0, 256))
    out = torch.full((3, 8, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    table = i32([[1 << 30, -1]] * 3)
    moe.moe_gqa_kv4_decode(randn(3, 8, D), raw, table, i32([0, 0, 0]), SCALE, out, ws)
    before = k.clone()
    moe.moe_kv4_load(raw, table, i32([0, 5, 32]), i32([0, 5, 7]), k, v, table, ws)
    torch.cuda.synchronize()
    assert moe.workspace_status(ws) == 0 and not out.any() and torch.equal(before.view(torch.int16), k.view(torch.int16))


def test_a_captured_step_follows_its_inputs():
    """Norm, store, attention and norm again, captured once: replays with other inputs in place give the eager results."""
    B, h_q, h_kv, page, H = 5, 16, 2, 16, 256
    lens = [40, 17, 1, 300, 128]
    c = step.Kv4(lens, h_kv, page, DEV)
    ws = moe.alloc_paged_workspace(B, B, h_q, h_kv, D, device=DEV)
    n, pos = i32(lens), i32([x - 1 for x in lens])
    slots = i32([int(c.table[b, (x - 1) // page]) * page + (x - 1) % page for b, x in enumerate(lens)])
    inv = (1e6 ** (-torch.arange(0, D, 2).double() / D)).float().to(DEV)
    x, res, qkv = randn(B, H), randn(B, H, seed=1), randn(B, (h_q + 2 * h_kv) * D, seed=2)
    y, q, out = torch.empty_like(x), randn(B, h_q, D), randn(B, h_q, D)

    def run():
        moe.moe_add_rms_norm(x, res, None, 1e-6, res, y)
        moe.moe_qk_norm_rope_kv4(qkv, None, None, 0.0, inv, None, pos, slots, q, c.raw)
        moe.moe_gqa_kv4_decode(q, c.raw, c.table, n, SCALE, out, ws)

    saved = [t.clone() for t in (x, res, qkv)]
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        run()
    for seed in (10, 11, 12):
        news = [saved[0] * 0 + randn(B, H, seed=seed), randn(B, H, seed=seed + 100), randn(*qkv.shape, seed=seed + 200)]
        got = []
        for call in (g.replay, run):
            for t, v in zip((x, res, qkv), news):
                t.copy_(v)
            call()
            torch.cuda.synchronize()
            got.append([t.clone() for t in (res, y, q, out, c.raw)])
        assert all(torch.equal(a, b) for a, b in zip(*got))


def test_decode_cache_past_32_bits():
    page, h_kv = 1024, 2
    num_pages = (5 << 30) // (h_kv * page * 144)
    lens = [3000, 1025]
    c = step.Kv4(lens, h_kv, page, DEV, num_pages=num_pages)
    c.table[0, :3] = i32([num_pages - 1, num_pages - 2, num_pages - 3])
    c.table[1, :2] = i32([num_pages - 4, 0])
    for b in range(2):
        c.put(b, slice(0, lens[b]), *c.rows[b])
    check_decode(c, lens, *decode(c, lens, 16, hide=False))
    k, v = (torch.zeros(6, h_kv, page, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ws = moe.alloc_paged_workspace(device=DEV)
    moe.moe_kv4_load(c.raw, c.table, None, i32(lens), k, v, i32([[3, 1, 5], [0, 4, -1]]), ws)
    assert torch.equal(k[5, :, :952].transpose(0, 1), c.values(0)[0][2048:].to(torch.bfloat16))
    assert torch.equal(v[4, :, 0], c.values(1)[1][1024].to(torch.bfloat16))


# ---------------------------------------------------------------- a run of them
def test_a_serving_run():
    """Prompts and then single tokens: planned, normed, rotated, stored in 4 bits, read back for the prompts, attended."""
    h_q, h_kv, page, num_pages = 16, 2, 16, 64
    B, width = 3, 16
    ws = moe.alloc_paged_workspace(256, B, h_q, h_kv, D, device=DEV)
    raw = moe.alloc_kv4_cache(num_pages, h_kv, page, DEV).fill_(255)
    wide = [torch.full((num_pages, h_kv, page, D), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    dst = torch.arange(B * width, dtype=torch.int32, device=DEV).view(B, width)
    free, left = torch.randperm(num_pages).to(torch.int32).to(DEV), i32([num_pages])
    lens = i32([0] * B)
    inv = (1e6 ** (-torch.arange(0, D, 2).double() / D)).float().to(DEV)
    pair = (torch.arange(D // 2) % 3).to(torch.int32).to(DEV)
    w = [(1 + 0.1 * randn(D, seed=i)).contiguous() for i in range(2)]
    for n_step, new in enumerate(([40, 1, 100], [3, 30, 0], [1, 1, 1], [1, 1, 1])):
        N = sum(new)
        x = randn(N, h_q + 2 * h_kv, D, seed=10 + n_step)
        ctx, cu, pos, slots = lens.clone(), i32([0] * (B + 1)), i32([0] * N), i32([0] * N)
        moe.moe_paged_plan(ctx, i32(new), page, num_pages, free, left, table, lens, cu, pos, slots, left, ws)
        axes = torch.stack([pos, pos // 7, pos % 7]).contiguous()
        q, out = (torch.empty(N, h_q, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        moe.moe_qk_norm_rope_kv4(x.view(N, -1), *w, 1e-6, inv, pair, axes, slots, q, raw)
        moe.moe_kv4_load(raw, table, ctx, lens, *wide, dst, ws)  # the new rows alone
        if max(new) > 1:
            moe.moe_gqa_paged_prefill(q, cu, *wide, dst, lens, SCALE, out, ws)
        else:
            moe.moe_gqa_kv4_decode(q, raw, table, lens, SCALE, out, ws)
        torch.cuda.synchronize()
        assert moe.workspace_status(ws) == 0
        for b in range(B):
            n, c = int(lens[b]), int(ctx[b])
            rows = [t[dst[b].long()].transpose(1, 2).flatten(0, 1)[:n] for t in wide]
            at = slice(int(cu[b]), int(cu[b + 1]))
            key = torch.arange(n, device=DEV)
            see = ref.visible(torch.arange(c, n, device=DEV)[:, None], key[None, :], 0, 0)
            if n > c:
                if max(new) > 1:
                    ref.check(out[at], *ref.attend(q[at], *rows, see, SCALE), f"step {n_step} sequence {b}")
                else:
                    exact_rows = [raw_rows(raw, table[b], n, i) for i in range(2)]
                    assert all(torch.equal(r, e.to(torch.bfloat16)) for r, e in zip(rows, exact_rows))
                    step.check(out[at][0], *step.attend(q[at][0], *exact_rows, see[0], SCALE), n, f"step {n_step} sequence {b}")
                # what was read back is what the formulas give, to the step of 4 bits and the bf16 roundings
                exact, _ = norm_rope_axes(x[at, h_q:h_q + h_kv], w[1], 1e-6, axes[:, at], inv, pair)
                err = (rows[0][c:n].double() - exact).abs()
                half = exact.unflatten(-1, (4, 32)).abs().amax(-1, keepdim=True).expand(-1, -1, -1, 32).flatten(-2) / 14
                assert (err <= half * (1 + 2.0 ** -5) + 2.0 ** -6 * exact.abs() + 1e-6).all()


def raw_rows(raw, pages, n, i):
    """Keys (i = 0) or values of a sequence's n tokens in 64 bits, [n, h_kv, 128]."""
    codes, scales = (p[pages[:ref.up(n, raw.shape[2] * 16)].long()].transpose(1, 2).flatten(0, 1)[:n] for p in parts(raw, i))
    return step.unpack_rows(codes).double() * scales.double().repeat_interleave(32, -1)


def norm_rope_axes(x, weight, eps, positions, inv_freq, pair_axis, interleaved=False):
    """norm_rope with a position axis of its own for each pair: positions [axes, N]."""
    pos = positions.long()[pair_axis.long()].t().double()  # [N, pairs]
    live = torch.ones(x.shape[0], dtype=torch.double, device=x.device)
    out, size = ref.norm_rope(x, weight, eps, live * 0, inv_freq, interleaved)  # unrotated, for the shapes
    x = x.double()
    if weight is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double()
    rot = 2 * inv_freq.numel()
    first = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    second = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    angle = (pos * inv_freq.double())[:, None, :]
    a, b = x[..., first].clone(), x[..., second].clone()
    out[..., first], out[..., second] = a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()
    return out, size
