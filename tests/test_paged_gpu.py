"""The serving path over a paged key/value cache on the GPU, through the binding, against plain 64-bit forms
(needs a GPU)."""
import numpy as np
import pytest
import torch

import paged_reference as ref
import routed_expert_ffn_softmax_gb300 as moe

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


# ---------------------------------------------------------------- plan
def run_plan(ctx, new, page, num_pages, free, count, table, n_rows, alias=False, ws=None):
    B = len(ctx)
    ws = moe.alloc_paged_workspace(device=DEV) if ws is None else ws
    c, t, fc = i32(ctx), i32(table), i32([count])
    out = dict(seq_lens=c if alias else i32([-5] * B), cu=i32([-5] * (B + 1)), left=fc if alias else i32([-5]),
               positions=i32([-5] * n_rows), slots=i32([-5] * n_rows), table=t)
    moe.moe_paged_plan(c, i32(new), page, num_pages, i32(free), fc, t, out["seq_lens"], out["cu"], out["positions"],
                       out["slots"], out["left"], ws)
    torch.cuda.synchronize()
    got = {k: v.cpu().tolist() for k, v in out.items()}
    got["left"] = got["left"][0]
    got["status"] = moe.workspace_status(ws)
    assert not ws[4:4096].any(), "the workspace's control words must be left zero"
    return got


def table_for(ctx, page, width, order):
    rows = []
    for c in ctx:
        n = ref.up(max(c, 0), page)
        rows.append([order.pop() for _ in range(n)] + [-1] * (width - n))
    return rows


PLANS = {
    "one token each": ([5, 16, 31, 0], [1, 1, 1, 1], 16, 8, 64),
    "prompts": ([0, 0, 7], [100, 1, 40], 16, 16, 200),
    "nothing new": ([3, 0, 16], [0, 0, 0], 16, 4, 5),
    "one sequence": ([0], [1], 1024, 1, 1),
    "no token rows": ([4], [0], 16, 1, 0),
    "rows run out": ([0, 0, 0], [10, 20, 5], 16, 8, 25),
    "the table runs out": ([30, 2, 10], [4, 3, 40], 16, 2, 64),
    "bad lengths": ([-3, 5, 6], [2, -4, 7], 16, 4, 32),
}


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("name", PLANS)
def test_plan(name, alias):
    ctx, new, page, width, n_rows = PLANS[name]
    order = torch.randperm(200, generator=torch.Generator().manual_seed(len(name))).tolist()
    table = table_for(ctx, page, width, order)
    args = (ctx, new, page, 200, order, len(order) - 3, table, n_rows)
    assert run_plan(*args, alias=alias) == ref.plan(*args)


@pytest.mark.parametrize("count", [-1, 0, 1, 3, 4, 5, 9, 11])
def test_plan_free_list_runs_out(count):
    """Needs of 1, 3, 0, 2, 1 pages: sequences that need none are never left out."""
    ctx, new = [16, 0, 3, 30, 16], [1, 48, 5, 20, 2]
    table = table_for(ctx, 16, 5, list(range(20, 40)))
    args = (ctx, new, 16, 64, list(range(10)), count, table, 80)
    assert run_plan(*args) == ref.plan(*args)


def test_plan_bad_pages():
    args = ([5, 0], [20, 3], 16, 50, [50, 7, -2], 3, [[60, -1, -1], [-1, -1, -1]], 30)
    assert run_plan(*args) == ref.plan(*args)


@pytest.mark.parametrize("B,hi,page", [(2048, 40, 16), (700, 300, 64), (3, 20000, 32), (513, 2, 1024)])
def test_plan_many(B, hi, page):
    g = np.random.default_rng(B)
    ctx, new = g.integers(0, 500, B).tolist(), g.integers(0, hi, B).tolist()
    width = max(ref.up(c + n, page) for c, n in zip(ctx, new))
    total = sum(ref.up(c + n, page) for c, n in zip(ctx, new))
    order = g.permutation(total + 5).tolist()
    table = table_for(ctx, page, width, order)
    args = (ctx, new, page, total + 5, order, len(order), table, sum(new) + 17)
    assert run_plan(*args) == ref.plan(*args)


def test_plan_repeats_on_one_workspace():
    ws = moe.alloc_paged_workspace(device=DEV)
    args = ([5, 0], [20, 3], 16, 50, [4, 7, 9], 3, [[6, -1, -1], [-1, -1, -1]], 30)
    for _ in range(3):
        assert run_plan(*args, ws=ws) == ref.plan(*args)


# ---------------------------------------------------------------- norm, rotation, store
def run_qk(N, h_q, h_kv, page, rot, norm=True, interleaved=False, pad=0, seed=0, far=0, base=1e6, left_out=()):
    dev = DEV
    g = torch.Generator().manual_seed(seed)
    heads = h_q + 2 * h_kv
    wide = torch.randn(N, heads * D + pad, generator=g).to(torch.bfloat16).to(dev)
    qkv = wide[:, :heads * D]
    w = [(1 + 0.2 * torch.randn(D, generator=g)).to(torch.bfloat16).to(dev) if norm else None for _ in range(2)]
    inv = (base ** (-torch.arange(0, rot, 2).double() / rot)).float().to(dev) if rot else None
    pos = (far + torch.randint(0, 5000, (N,), generator=g)).to(torch.int32)
    pages = ref.up(N, page) + 2
    slots = torch.randperm(pages * page, generator=g)[:N].to(torch.int32)
    for i, s in left_out:
        slots[i] = s if s < 0 else pages * page + s
    k = torch.randn(pages, h_kv, page, D, generator=g).to(torch.bfloat16).to(dev)
    v = torch.randn(pages, h_kv, page, D, generator=g).to(torch.bfloat16).to(dev)
    k0, v0 = k.clone(), v.clone()
    q_out = torch.full((N, h_q, D), float("nan"), dtype=torch.bfloat16, device=dev)
    moe.moe_qk_norm_rope(qkv, *w, 1e-6, inv, pos.to(dev), slots.to(dev), q_out, k, v, interleaved=interleaved)
    torch.cuda.synchronize()
    x = qkv.reshape(N, heads, D)
    # fp32: a sum of 128 squares in 8 + 4 steps, 1/sqrt, two products, the angle (pi 2^-24), sin and cos, a fused
    # product-sum: below 32 half steps of 2^-24 in all, of |a| + |b|; then one rounding to bf16
    for what, got, (want, size) in (
            ("q", q_out, ref.norm_rope(x[:, :h_q], w[0], 1e-6, pos.to(dev), inv, interleaved)),
            ("k", None, ref.norm_rope(x[:, h_q:h_q + h_kv], w[1], 1e-6, pos.to(dev), inv, interleaved))):
        if what == "k":
            ok = (slots >= 0) & (slots < pages * page)
            at = slots[ok].long().to(dev)
            got, want, size = k[at // page, :, at % page], want[ok.to(dev)], size[ok.to(dev)]
            assert torch.equal(v[at // page, :, at % page], x[:, h_q + h_kv:][ok.to(dev)])
            k0[at // page, :, at % page], v0[at // page, :, at % page] = got, v[at // page, :, at % page]
            assert torch.equal(k, k0) and torch.equal(v, v0), "rows of other slots must stay as they were"
        over = (got.double() - want).abs() - (2.0 ** -8 * want.abs() + 2.0 ** -19 * size)
        assert torch.isfinite(got.float()).all() and over.max() <= 0, f"{what}: off by {over.max():.3g}"


@pytest.mark.parametrize("N,h_q,h_kv,page,rot,norm,interleaved", [
    (1, 16, 2, 16, 128, True, False), (1, 1, 1, 16, 128, True, True), (7, 32, 4, 16, 128, True, False),
    (33, 64, 4, 64, 64, True, False), (65, 32, 8, 32, 32, False, True), (129, 5, 5, 128, 16, True, False),
    (40, 12, 3, 1024, 128, False, False), (9, 3, 1, 256, 48, True, True), (5, 24, 2, 16, 112, True, False),
    (300, 32, 4, 16, 0, True, False), (20, 32, 4, 16, 0, False, False), (3001, 8, 2, 32, 128, True, False)])
def test_qk_norm_rope(N, h_q, h_kv, page, rot, norm, interleaved):
    run_qk(N, h_q, h_kv, page, rot, norm, interleaved, seed=N)


def test_qk_strided_rows_and_left_out_tokens():
    run_qk(50, 8, 2, 16, 128, pad=72, left_out=((0, -1), (17, 0), (49, 12345), (3, -2 ** 31)))


@pytest.mark.parametrize("far", [1_000_000, 2 ** 30, 2 ** 31 - 5000])
@pytest.mark.parametrize("base", [10.0, 1e6])
def test_qk_far_positions(far, base):
    run_qk(40, 8, 2, 16, 128, far=far, base=base)


# ---------------------------------------------------------------- decode
def run_decode(lens, h_q, h_kv, page, window=0, n_sink=0, seed=0, ws=None, scale=SCALE, cache=None, stream=None):
    B = len(lens)
    c = cache or ref.Cache(lens, h_kv, page, DEV, seed)
    q = randn(B, h_q, D, seed=seed + 1)
    want, size = [], []
    for b, n in enumerate(lens):
        see = ref.visible(torch.tensor([[n - 1]], device=DEV), torch.arange(n, device=DEV), window, n_sink)
        o, s = ref.attend(q[b:b + 1], *c.rows[b], see, scale)
        want.append(o)
        size.append(s)
        if n and not cache:
            c.hide(b, ~see.any(0))
    out = torch.full_like(q, float("nan"))
    ws = moe.alloc_paged_workspace(B, B, h_q, h_kv, D, device=DEV) if ws is None else ws
    moe.moe_gqa_paged_decode(q, c.k, c.v, c.table, i32(lens), scale, out, ws, window=window, n_sink=n_sink)
    torch.cuda.synchronize()
    assert moe.workspace_status(ws) == 0
    ref.check(out, torch.cat(want), torch.cat(size), f"{lens[:6]} {h_q}/{h_kv} page {page} window {window} sink {n_sink}")
    assert not ws[4:4096].any()
    return out


EDGES = (1, 127, 128, 129, 0, 255, 256, 257, 700)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256, 1024])
@pytest.mark.parametrize("h_q,h_kv", [(16, 2), (32, 8), (64, 4)])
def test_decode_pages(page, h_q, h_kv):
    run_decode(EDGES, h_q, h_kv, page, seed=page)


@pytest.mark.parametrize("h_q,h_kv", [(1, 1), (8, 8), (4, 2), (12, 4), (5, 1), (24, 2), (16, 1)])
def test_decode_groups(h_q, h_kv):
    run_decode((200, 1, 333), h_q, h_kv, 32, seed=h_q)


@pytest.mark.parametrize("page", [16, 64, 128, 512])
@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 1), (64, 4), (128, 0), (129, 130), (100, 128), (200, 300),
                                           (256, 16), (5000, 4), (1, 5000), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_decode_window_and_sinks(page, window, n_sink):
    run_decode(EDGES + (1500, 3001), 16, 2, page, window, n_sink, seed=window % 1000 + page)


def test_decode_one_long_sequence_over_all_ctas():
    run_decode((5, 20001, 130, 1), 8, 1, 16)
    run_decode((5, 20001, 130, 1), 8, 1, 16, window=9000, n_sink=700)


def test_decode_many_sequences():
    g = np.random.default_rng(3)
    run_decode(g.integers(0, 40, 2048).tolist(), 8, 1, 16)
    run_decode(g.integers(0, 600, 301).tolist(), 32, 4, 16, window=77, n_sink=3)


def test_decode_agrees_with_the_contiguous_cache():
    """The same rows through moe_gqa_decode's contiguous cache and through pages: both within their bound of the
    64-bit result, so within twice that of each other."""
    lens = (300, 17, 1025)
    c = ref.Cache(lens, 4, 64, DEV, seed=4)
    q = randn(3, 32, D, seed=5)
    flat = [torch.full((3, 4, 1088, D), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    for b, n in enumerate(lens):
        for f, r in zip(flat, c.rows[b]):
            f[b, :, :n] = r.transpose(0, 1)
    a, b = torch.empty_like(q), torch.empty_like(q)
    moe.moe_gqa_paged_decode(q, c.k, c.v, c.table, i32(lens), SCALE, a,
                             moe.alloc_paged_workspace(3, 3, 32, 4, D, device=DEV))
    moe.moe_gqa_decode(q, *flat, i32(lens), SCALE, b, moe.alloc_gqa_workspace(3, 32, 4, D, 1088, DEV))
    for i, n in enumerate(lens):
        want = ref.attend(q[i:i + 1], *c.rows[i], torch.ones(1, n, dtype=torch.bool, device=DEV), SCALE)
        ref.check(a[i:i + 1], *want, "paged")
        ref.check(b[i:i + 1], *want, "contiguous")


def test_decode_bad_length_and_bad_page():
    lens = (40, 300, 64)
    c = ref.Cache(lens, 2, 16, DEV, seed=1)
    q = randn(3, 16, D)
    out, ws = torch.empty_like(q), moe.alloc_paged_workspace(3, 3, 16, 2, D, device=DEV)
    for bad in (-1, c.table.shape[1] * 16 + 1, -2 ** 31, 2 ** 31 - 1):
        ws[:4] = 0
        moe.moe_gqa_paged_decode(q, c.k, c.v, c.table, i32([40, bad, 64]), SCALE, out, ws)
        assert moe.workspace_status(ws) == 4 and not out[1].any()
        for b in (0, 2):
            o, s = ref.attend(q[b:b + 1], *c.rows[b], torch.ones(1, lens[b], dtype=torch.bool, device=DEV), SCALE)
            ref.check(out[b:b + 1], o, s, "beside a bad length")
    ws[:4] = 0
    c.table[1, 3] = c.k.shape[0]
    moe.moe_gqa_paged_decode(q, c.k, c.v, c.table, i32(lens), SCALE, out, ws)
    assert moe.workspace_status(ws) == 6 and torch.isfinite(out.float()).all()


@pytest.mark.parametrize("kind", ["decode", "prefill", "prefix"])
def test_cache_larger_than_32_bit_offsets(kind):
    """Pages whose elements lie past 2^32 (and whose bytes past 2^33) in the cache."""
    h_kv, page = 8, 64
    pages = 2 ** 32 // (h_kv * page * D) + 40
    k, v = (torch.empty(pages, h_kv, page, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    n = 150
    far = [pages - 1, pages - 30, pages - 17]
    rows = [randn(n, h_kv, D, seed=s) for s in (1, 2)]
    pos = torch.arange(n, device=DEV)
    slots = i32(far)[pos // page] * page + (pos % page).to(torch.int32)
    qkv = torch.cat([randn(n, 16 * D, seed=3), rows[0].view(n, -1), rows[1].view(n, -1)], 1)
    q_out = torch.empty(n, 16, D, dtype=torch.bfloat16, device=DEV)
    moe.moe_qk_norm_rope(qkv, None, None, 0.0, None, pos.to(torch.int32), slots, q_out, k, v)
    assert torch.equal(q_out.view(n, -1), qkv[:, :16 * D])
    assert torch.equal(k[far[0], :, 5], rows[0][5]) and torch.equal(v[far[1], :, 7], rows[1][page + 7])
    ws = moe.alloc_paged_workspace(n, 1, 16, h_kv, D, n, device=DEV)
    if kind == "prefill":
        out = torch.empty_like(q_out)
        moe.moe_gqa_paged_prefill(q_out, i32([0, n]), k, v, i32([far]), i32([n]), SCALE, out, ws)
        see = ref.visible(pos[:, None], pos, 0, 0)
        want = ref.attend(q_out, *rows, see, SCALE)
    else:
        out = torch.empty(1, 16, D, dtype=torch.bfloat16, device=DEV)
        q = q_out[-1:].contiguous()
        if kind == "decode":
            moe.moe_gqa_paged_decode(q, k, v, i32([far]), i32([n]), SCALE, out, ws)
        else:
            moe.moe_gqa_prefix_decode(q, i32(far), n, k, v, i32([[0]]), i32([0]), SCALE, out, ws)
        want = ref.attend(q, *rows, torch.ones(1, n, dtype=torch.bool, device=DEV), SCALE)
    ref.check(out, *want, kind)
    del k, v
    torch.cuda.empty_cache()


# ---------------------------------------------------------------- many tokens per sequence
def run_prefill(lens, new, h_q, h_kv, page, window=0, n_sink=0, seed=0, tail=3, scale=SCALE, ws=None):
    B, N = len(lens), sum(new)
    c = ref.Cache(lens, h_kv, page, DEV, seed)
    q = randn(N + tail, h_q, D, seed=seed + 1)
    cu = [0]
    want, size = [], []
    for b, (n, m) in enumerate(zip(lens, new)):
        pos = torch.arange(n - m, n, device=DEV)[:, None]
        see = ref.visible(pos, torch.arange(n, device=DEV), window, n_sink)
        o, s = ref.attend(q[cu[-1]:cu[-1] + m], *c.rows[b], see, scale)
        want.append(o)
        size.append(s)
        cu.append(cu[-1] + m)
        if n and m:
            c.hide(b, ~see.any(0))
    out = torch.full_like(q, 7.0)
    ws = moe.alloc_paged_workspace(N + tail, B, h_q, h_kv, D, device=DEV) if ws is None else ws
    moe.moe_gqa_paged_prefill(q, i32(cu), c.k, c.v, c.table, i32(lens), scale, out, ws, window=window, n_sink=n_sink)
    torch.cuda.synchronize()
    assert moe.workspace_status(ws) == 0
    what = f"{lens[:6]} new {new[:6]} {h_q}/{h_kv} page {page} window {window} sink {n_sink}"
    ref.check(out[:N], torch.cat(want), torch.cat(size), what)
    assert (out[N:] == 7.0).all(), "rows behind the last sequence must stay as they were"
    assert not ws[4:4096].any()
    return out


LENS, NEW = (1, 130, 0, 257, 700, 64, 513), (1, 130, 0, 100, 3, 1, 513)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256, 1024])
@pytest.mark.parametrize("h_q,h_kv", [(16, 2), (32, 8), (64, 4)])
def test_prefill_pages(page, h_q, h_kv):
    run_prefill(LENS, NEW, h_q, h_kv, page, seed=page)


@pytest.mark.parametrize("h_q,h_kv", [(1, 1), (8, 8), (4, 2), (3, 1), (10, 2), (24, 2), (13, 1), (7, 1)])
def test_prefill_groups(h_q, h_kv):
    run_prefill((300, 1, 77), (300, 1, 20), h_q, h_kv, 32, seed=h_q)


@pytest.mark.parametrize("page", [16, 128, 512])
@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 1), (64, 4), (128, 0), (129, 130), (100, 128), (200, 300),
                                           (256, 16), (5000, 4), (1, 5000), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_prefill_window_and_sinks(page, window, n_sink):
    run_prefill(LENS + (1500,), NEW + (700,), 16, 2, page, window, n_sink, seed=window % 1000 + page)


@pytest.mark.parametrize("window,n_sink", [(0, 0), (3000, 4)])
def test_prefill_few_rows_behind_long_contexts(window, n_sink):
    """Few row blocks and many key tiles: blocks are cut between CTAs."""
    run_prefill((20000, 9000, 33), (5, 33, 2), 8, 1, 16, window, n_sink)


def test_prefill_long_prompt():
    run_prefill((4100,), (4100,), 16, 2, 64)
    run_prefill((4100, 50), (4100, 50), 16, 2, 64, window=1000, n_sink=4)


def test_prefill_many_sequences():
    g = np.random.default_rng(5)
    new = g.integers(0, 6, 2048).tolist()
    run_prefill([n + int(c) for n, c in zip(new, g.integers(0, 30, 2048))], new, 8, 1, 16)


def test_prefill_one_token_each_agrees_with_decode():
    lens = (300, 17, 1025)
    run_prefill(lens, (1, 1, 1), 32, 4, 64, tail=0)
    run_prefill(lens, (1, 1, 1), 32, 4, 64, window=100, n_sink=2, tail=0)


def test_prefill_more_queries_than_keys():
    """Queries before the sequence's first token see nothing."""
    c = ref.Cache((5, 0), 2, 16, DEV)
    q = randn(12, 16, D)
    out, ws = torch.full_like(q, 7.0), moe.alloc_paged_workspace(12, 2, 16, 2, D, device=DEV)
    moe.moe_gqa_paged_prefill(q, i32([0, 9, 12]), c.k, c.v, c.table, i32([5, 0]), SCALE, out, ws)
    assert not out[:4].any() and not out[9:].any() and moe.workspace_status(ws) == 0
    see = ref.visible(torch.arange(5, device=DEV)[:, None], torch.arange(5, device=DEV), 0, 0)
    ref.check(out[4:9], *ref.attend(q[4:9], *c.rows[0], see, SCALE), "queries with keys")


def test_prefill_bad_offsets_lengths_and_pages():
    c = ref.Cache((40, 300, 64), 2, 16, DEV)
    q = randn(30, 16, D)
    ws = moe.alloc_paged_workspace(30, 3, 16, 2, D, device=DEV)

    def go(cu, lens):
        ws[:4] = 0
        out = torch.full_like(q, 7.0)
        moe.moe_gqa_paged_prefill(q, i32(cu), c.k, c.v, c.table, i32(lens), SCALE, out, ws)
        return out, moe.workspace_status(ws)

    good, st = go([0, 10, 20, 30], [40, 300, 64])
    assert st == 0
    for bad in (-1, 2 ** 31 - 1):
        out, st = go([0, 10, 20, 30], [40, bad, 64])
        assert st == 4 and not out[10:20].any()
        assert torch.equal(out[:10], good[:10]) and torch.equal(out[20:], good[20:])
    out, st = go([0, 10, 31, 30], [40, 300, 64])  # leaves 0 .. N: sequences 1 and 2 are not written
    assert st == 4 and (out[10:] == 7).all()
    out, st = go([-3, 10, 20, 30], [40, 300, 64])
    assert st == 4 and (out[:10] == 7).all() and torch.equal(out[10:], good[10:])
    c.table[1, 3] = -1
    out, st = go([0, 10, 20, 30], [40, 300, 64])
    assert st == 6 and torch.isfinite(out.float()).all()
    ref_rows = [0, 9, 20, 29]
    assert torch.isfinite(out[ref_rows].float()).all()


# ---------------------------------------------------------------- shared prefix
def run_prefix(prefix, lens, h_q, h_kv, page, seed=0, ws=None, scale=SCALE):
    B = len(lens)
    c = ref.Cache([prefix] + list(lens), h_kv, page, DEV, seed)
    q = randn(B, h_q, D, seed=seed + 1)
    shared, own = c.table[0].contiguous(), c.table[1:].contiguous()
    out = torch.full_like(q, float("nan"))
    ws = moe.alloc_paged_workspace(B, B, h_q, h_kv, D, prefix, device=DEV) if ws is None else ws
    moe.moe_gqa_prefix_decode(q, shared, prefix, c.k, c.v, own, i32(lens), scale, out, ws)
    torch.cuda.synchronize()
    assert moe.workspace_status(ws) == 0
    for b, n in enumerate(lens):
        k, v = (torch.cat([c.rows[0][i], c.rows[b + 1][i]]) for i in (0, 1))
        see = torch.ones(1, prefix + n, dtype=torch.bool, device=DEV)
        ref.check(out[b:b + 1], *ref.attend(q[b:b + 1], k, v, see, scale), f"prefix {prefix} sequence {b} of {n}")
    assert not ws[4:4096].any()
    return out


@pytest.mark.parametrize("page", [16, 64, 128, 512])
@pytest.mark.parametrize("prefix", [0, 1, 127, 128, 129, 1000, 4097])
def test_prefix(prefix, page):
    run_prefix(prefix, EDGES, 32, 4, page, seed=prefix)


@pytest.mark.parametrize("h_q,h_kv", [(1, 1), (8, 8), (4, 2), (3, 1), (10, 2), (24, 2), (13, 1), (16, 1), (64, 4)])
@pytest.mark.parametrize("B", [1, 9, 40])
def test_prefix_groups(h_q, h_kv, B):
    run_prefix(700, [(37 * i) % 300 for i in range(B)], h_q, h_kv, 32, seed=h_q)


def test_prefix_many_sequences():
    run_prefix(3000, [(7 * i) % 50 for i in range(700)], 16, 2, 16)
    run_prefix(20000, [0] * 5, 8, 1, 16)
    run_prefix(300, [1] * 2048, 8, 8, 16)


def test_prefix_without_own_keys_or_prefix():
    assert not run_prefix(0, (0, 0), 16, 2, 16).any()
    run_prefix(500, (0, 0, 0), 16, 2, 16)


# ---------------------------------------------------------------- values, streams, graphs
def test_scores_far_apart():
    """A key that dwarfs the rest, late and early, takes all the weight: its value row comes back bit for bit."""
    lens = (700, 300)
    c = ref.Cache(lens, 2, 16, DEV)
    for rows in c.rows:
        rows[0][..., 5] = 0
    c.rows[0][0][433, 1, 5] = 4096
    c.rows[1][0][0, 0, 5] = 4096
    for b, n in enumerate(lens):
        c.put(b, slice(0, n), *c.rows[b])
    q = torch.zeros(2, 16, D, dtype=torch.bfloat16, device=DEV)
    q[:, :, 5] = 1
    ws = moe.alloc_paged_workspace(4, 2, 16, 2, D, 300, device=DEV)
    out = torch.empty_like(q)
    moe.moe_gqa_paged_decode(q, c.k, c.v, c.table, i32(lens), 1.0, out, ws)
    assert all(torch.equal(out[0, h], c.rows[0][1][433, 1]) for h in range(8, 16))
    assert all(torch.equal(out[1, h], c.rows[1][1][0, 0]) for h in range(8))
    moe.moe_gqa_paged_prefill(q, i32([0, 1, 2]), c.k, c.v, c.table, i32(lens), 1.0, out, ws)
    assert all(torch.equal(out[0, h], c.rows[0][1][433, 1]) for h in range(8, 16))
    assert all(torch.equal(out[1, h], c.rows[1][1][0, 0]) for h in range(8))
    moe.moe_gqa_prefix_decode(q, c.table[1].contiguous(), 300, c.k, c.v, c.table, i32([700, 0]), 1.0, out, ws)
    assert all(torch.equal(out[1, h], c.rows[1][1][0, 0]) for h in range(8))


@pytest.mark.parametrize("scale", [0.0, -0.05, 3.0, 40.0])
def test_scales(scale):
    run_decode((300, 17), 16, 2, 16, scale=scale)
    run_prefill((300, 17), (200, 17), 16, 2, 16, scale=scale)
    run_prefix(300, (17, 200), 16, 2, 16, scale=scale)


def step(s, ws, stream=None):
    moe.moe_paged_plan(s["ctx"], s["new"], s["page"], s["k"].shape[0], s["free"], s["count"], s["table"], s["lens"],
                       s["cu"], s["pos"], s["slots"], s["left"], ws, stream=stream)
    moe.moe_qk_norm_rope(s["qkv"], s["qw"], s["kw"], 1e-6, s["inv"], s["pos"], s["slots"], s["q"], s["k"], s["v"],
                         stream=stream)
    if s["prompt"]:
        moe.moe_gqa_paged_prefill(s["q"], s["cu"], s["k"], s["v"], s["table"], s["lens"], SCALE, s["out"], ws,
                                  window=s["window"], n_sink=s["n_sink"], stream=stream)
    else:
        moe.moe_gqa_paged_decode(s["q"], s["k"], s["v"], s["table"], s["lens"], SCALE, s["out"], ws,
                                 window=s["window"], n_sink=s["n_sink"], stream=stream)


def step_inputs(ctx, new, page, h_q, h_kv, k, v, table, free, window, n_sink, rows, seed):
    N, B = rows, len(ctx)
    g = torch.Generator().manual_seed(seed)
    w = lambda: (1 + 0.2 * torch.randn(D, generator=g)).to(torch.bfloat16).to(DEV)  # noqa: E731
    return dict(ctx=i32(ctx), new=i32(new), page=page, free=free, count=i32([free.numel()]), table=table,
                lens=i32([0] * B), cu=i32([0] * (B + 1)), pos=i32([0] * N), slots=i32([0] * N), left=i32([0]),
                qkv=randn(N, (h_q + 2 * h_kv) * D, seed=seed + 1), qw=w(), kw=w(),
                inv=(1e6 ** (-torch.arange(0, D, 2).double() / D)).float().to(DEV),
                q=torch.zeros(N, h_q, D, dtype=torch.bfloat16, device=DEV),
                out=torch.full((N, h_q, D), 7.0, dtype=torch.bfloat16, device=DEV), k=k, v=v, window=window,
                n_sink=n_sink, prompt=rows != B)


@pytest.mark.parametrize("window,n_sink", [(0, 0), (20, 3)])
def test_prompt_then_decode_steps_together(window, n_sink):
    """Prompts (with padding rows behind them), then decode steps, each planned, normed, rotated, stored and attended
    on the device; every output against attention over all the rows so far in 64 bits."""
    page, h_q, h_kv, B = 16, 16, 2, 4
    k = torch.full((40, h_kv, page, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    v = k.clone()
    table = torch.full((B, 10), -1, dtype=torch.int32, device=DEV)
    free = torch.randperm(40, generator=torch.Generator().manual_seed(1)).to(torch.int32).to(DEV)
    ws = moe.alloc_paged_workspace(200, B, h_q, h_kv, D, device=DEV)
    ctx, new, rows = [0] * B, [50, 1, 33, 100], 190
    qs = [[] for _ in range(B)]
    ks = [[] for _ in range(B)]
    for turn in range(4):
        s = step_inputs(ctx, new, page, h_q, h_kv, k, v, table, free, window, n_sink, rows, seed=10 * turn)
        step(s, ws)
        torch.cuda.synchronize()
        assert moe.workspace_status(ws) == 0
        free = free[:int(s["left"])].contiguous()
        cu = s["cu"].tolist()
        for b in range(B):
            x = s["qkv"][cu[b]:cu[b + 1]].view(-1, h_q + 2 * h_kv, D)
            pos = torch.arange(ctx[b], ctx[b] + new[b], device=DEV)
            # the attention is checked on the rounded queries and keys that the kernel stored
            pid, off = table[b].long()[pos // page], pos % page
            kn, _ = ref.norm_rope(x[:, h_q:h_q + h_kv], s["kw"], 1e-6, pos, s["inv"], False)
            assert (k[pid, :, off].double() - kn).abs().max() <= 2.0 ** -7 * kn.abs().max()
            ks[b].append((k[pid, :, off].clone(), x[:, h_q + h_kv:]))
            kk, vv = (torch.cat([t[i] for t in ks[b]]) for i in (0, 1))
            see = ref.visible(pos[:, None], torch.arange(ctx[b] + new[b], device=DEV), window, n_sink)
            ref.check(s["out"][cu[b]:cu[b + 1]], *ref.attend(s["q"][cu[b]:cu[b + 1]], kk, vv, see, SCALE),
                      f"turn {turn} sequence {b}")
        assert (s["out"][cu[B]:] == 7.0).all()
        ctx = [c + n for c, n in zip(ctx, new)]
        new, rows = [1] * B, B


def test_step_in_front_of_the_experts():
    """A decode step's attention output through the routed experts, twice on the same inputs: the same bits."""
    H, I, E, top_k, B = 2048, 256, 8, 2, 5
    k = torch.zeros((40, 2, 16, D), dtype=torch.bfloat16, device=DEV)
    table = torch.full((B, 4), -1, dtype=torch.int32, device=DEV)
    s = step_inputs([0] * B, [1] * B, 16, 16, 2, k, k.clone(), table, torch.arange(40, dtype=torch.int32, device=DEV),
                    0, 0, B, 3)
    ws, mws = moe.alloc_paged_workspace(B, B, 16, 2, D, device=DEV), moe.alloc_workspace(B, H, I, E, top_k, device=DEV)
    W = [randn(E, *sh, seed=i) * 0.02 for i, sh in enumerate(((I, H), (I, H), (H, I)))]
    logits = torch.randn(B, E, generator=torch.Generator().manual_seed(1)).to(DEV)
    got = []
    for _ in range(2):
        y = torch.empty(B, H, dtype=torch.bfloat16, device=DEV)
        step(s, ws)
        moe.moe_ffn_forward(s["out"].view(B, H), logits, *W, None, None, None, top_k, y, mws)
        got.append(y)
    # one key each: attention returns the value heads themselves
    vals = s["qkv"].view(B, 20, D)[:, 18:].repeat_interleave(8, dim=1)
    assert torch.equal(s["out"], vals)
    assert torch.equal(*got) and torch.isfinite(got[0].float()).all() and got[0].any()


@pytest.mark.parametrize("prompt", [False, True])
def test_step_captured_and_replayed_on_another_stream(prompt):
    B, rows = 3, (60 if prompt else 3)
    ctx, new = ([0, 5, 0], [30, 1, 20]) if prompt else ([40, 7, 300], [1, 1, 1])
    c = ref.Cache([max(x, 1) for x in ctx], 2, 16, DEV, spare=20, extra=8)
    free = torch.tensor(c.free, dtype=torch.int32, device=DEV)
    s = step_inputs(ctx, new, 16, 16, 2, c.k, c.v, c.table, free, 0, 0, rows, 5)
    ws = moe.alloc_paged_workspace(64, B, 16, 2, D, device=DEV)
    step(s, ws)
    torch.cuda.synchronize()
    names = ("table", "lens", "cu", "pos", "slots", "left", "q", "k", "v", "out")
    first = {n: s[n].clone() for n in names}
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(s, ws)
    for n in ("pos", "slots", "q", "lens"):
        s[n].zero_()
    s["out"].fill_(7.0)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(3):
            graph.replay()
    side.synchronize()
    for n in names:
        a, b = s[n], first[n]
        assert torch.equal(a.view(torch.int16) if a.dtype == torch.bfloat16 else a,
                           b.view(torch.int16) if b.dtype == torch.bfloat16 else b), n
    assert moe.workspace_status(ws) == 0


def test_two_streams_with_their_own_workspaces():
    lens = (3000, 200, 1500)
    c = ref.Cache(lens, 2, 16, DEV)
    q = [randn(3, 16, D, seed=i) for i in range(2)]
    ws = [moe.alloc_paged_workspace(3, 3, 16, 2, D, 3000, device=DEV) for _ in range(2)]
    lt, want = i32(lens), []
    for i in range(2):
        o = torch.empty_like(q[i])
        moe.moe_gqa_paged_decode(q[i], c.k, c.v, c.table, lt, SCALE, o, ws[i])
        want.append(o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.empty_like(q[0]) for _ in range(20)] for _ in range(2)]
    for r in range(20):
        for i in range(2):
            moe.moe_gqa_paged_decode(q[i], c.k, c.v, c.table, lt, SCALE, outs[i][r], ws[i], stream=streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i in range(2) for o in outs[i])


def test_results_repeat():
    a = [run_decode((3000, 17, 1500), 32, 4, 16, window=900, n_sink=4), run_prefill((3000, 17), (40, 17), 32, 4, 16),
         run_prefix(3000, (17, 100), 32, 4, 16)]
    b = [run_decode((3000, 17, 1500), 32, 4, 16, window=900, n_sink=4), run_prefill((3000, 17), (40, 17), 32, 4, 16),
         run_prefix(3000, (17, 100), 32, 4, 16)]
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_one_workspace_serves_smaller_calls():
    ws = moe.alloc_paged_workspace(1300, 16, 32, 4, D, 5000, device=DEV)
    for _ in range(2):
        run_prefix(4097, EDGES, 32, 4, 16, ws=ws)
        run_prefill(LENS, NEW, 32, 4, 16, ws=ws)
        run_decode(EDGES, 32, 4, 16, ws=ws)


def test_nothing_to_do():
    """No sequences, or no tokens: calls that do nothing, and calls whose sequences are all empty."""
    k = torch.full((4, 2, 16, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    ws = moe.alloc_paged_workspace(8, 4, 16, 2, D, 64, device=DEV)
    e = torch.empty(0, 16, D, dtype=torch.bfloat16, device=DEV)
    none, no_rows = i32([]).view(0, 3), i32([])
    moe.moe_paged_plan(no_rows, no_rows, 16, 4, i32([1]), i32([1]), none, no_rows, i32([0]), no_rows, no_rows, i32([9]), ws)
    moe.moe_qk_norm_rope(torch.empty(0, 20 * D, dtype=torch.bfloat16, device=DEV), None, None, 0.0, None, no_rows, no_rows,
                         e, k, k)
    moe.moe_gqa_paged_decode(e, k, k, none, no_rows, SCALE, e, ws)
    moe.moe_gqa_paged_prefill(e, i32([0]), k, k, none, no_rows, SCALE, e, ws)
    moe.moe_gqa_paged_prefill(e, i32([0, 0]), k, k, i32([[0]]), i32([5]), SCALE, e, ws)
    moe.moe_gqa_prefix_decode(e, i32([0]), 16, k, k, none, no_rows, SCALE, e, ws)
    # sequences without keys, their queries NaN; and packed rows that belong to no sequence
    q = torch.full((4, 16, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    table = i32([[-1, -1]] * 4)
    out = torch.full_like(q, 7.0)
    moe.moe_gqa_paged_prefill(q, i32([2] * 5), k, k, table, i32([0] * 4), SCALE, out, ws)
    torch.cuda.synchronize()
    assert (out == 7.0).all()
    moe.moe_gqa_paged_prefill(q, i32([0, 1, 2, 3, 4]), k, k, table, i32([0] * 4), SCALE, out, ws)
    torch.cuda.synchronize()
    assert not out.any()
    out.fill_(7.0)
    moe.moe_gqa_paged_decode(q, k, k, table, i32([0] * 4), SCALE, out, ws)
    torch.cuda.synchronize()
    assert not out.any() and moe.workspace_status(ws) == 0


def test_a_query_of_nan_stays_in_its_row():
    lens, new = (300, 70), (60, 70)
    c = ref.Cache(lens, 2, 16, DEV)
    clean = randn(130, 16, D, seed=2)
    bad = clean.clone()
    bad[33] = float("nan")
    ws = moe.alloc_paged_workspace(130, 130, 16, 2, D, 300, device=DEV)

    def prefill(q):
        out = torch.empty_like(q)
        moe.moe_gqa_paged_prefill(q, i32([0, 60, 130]), c.k, c.v, c.table, i32(lens), SCALE, out, ws)
        return out

    def behind(q):
        out = torch.empty_like(q)
        own = c.table[1:].expand(130, -1).contiguous()
        moe.moe_gqa_prefix_decode(q, c.table[0].contiguous(), 300, c.k, c.v, own, i32([70] * 130), SCALE, out, ws)
        return out

    for f in (prefill, behind):
        a, b = f(clean), f(bad)
        rest = torch.arange(130, device=DEV) != 33
        assert torch.equal(a[rest], b[rest]) and b[33].isnan().all()


def test_prefix_bad_page():
    c = ref.Cache((300, 40, 17), 2, 16, DEV)
    q = randn(2, 16, D)
    out, ws = torch.empty_like(q), moe.alloc_paged_workspace(2, 2, 16, 2, D, 300, device=DEV)
    for page in (-1, c.k.shape[0], 2 ** 31 - 1):
        ws[:4] = 0
        shared = c.table[0].clone()
        shared[7] = page
        moe.moe_gqa_prefix_decode(q, shared, 300, c.k, c.v, c.table[1:].contiguous(), i32([40, 17]), SCALE, out, ws)
        assert moe.workspace_status(ws) == 6
        # the page's keys and values read as zeros
        for b, n in enumerate((40, 17)):
            k, v = (torch.cat([c.rows[0][i], c.rows[b + 1][i]]) for i in (0, 1))
            k[7 * 16:8 * 16] = 0
            v[7 * 16:8 * 16] = 0
            see = torch.ones(1, 300 + n, dtype=torch.bool, device=DEV)
            ref.check(out[b:b + 1], *ref.attend(q[b:b + 1], k, v, see, SCALE), "a page of zeros")


def test_prefill_offsets_over_each_other():
    """Offsets that descend and start again would make more row blocks than the tokens do: the status word tells, and the
    workspace serves the next call."""
    lens = [100] * 9
    c = ref.Cache(lens, 2, 16, DEV)
    q, ws = randn(100, 16, D), moe.alloc_paged_workspace(100, 9, 16, 2, D, device=DEV)
    out = torch.empty_like(q)
    moe.moe_gqa_paged_prefill(q, i32([0, 100] * 5), c.k, c.v, c.table, i32(lens), SCALE, out, ws)
    torch.cuda.synchronize()
    assert moe.workspace_status(ws) == 4
    ws[:4] = 0
    run_prefill((300, 17), (83, 17), 16, 2, 16, tail=0, ws=ws)


def test_prefix_captured_between_writes_of_its_inputs():
    """The sequences' own keys are started before the prefix's kernels have finished: what runs in front of the call must
    have, in a stream and in a graph."""
    lens = (40, 0, 900, 17, 300) * 8
    c = ref.Cache((2500,) + lens, 2, 16, DEV)
    shared, own = c.table[0].contiguous(), c.table[1:].contiguous()
    qs = [randn(40, 16, D, seed=i) for i in range(3)]
    tables = [own, own.roll(5, 0), own.roll(10, 0)]
    ls = [i32(lens), i32(lens).roll(5, 0), i32(lens).roll(10, 0)]
    ws = moe.alloc_paged_workspace(40, 40, 16, 2, D, 2500, device=DEV)
    want = []
    for q, t, n in zip(qs, tables, ls):
        want.append(torch.empty_like(q))
        moe.moe_gqa_prefix_decode(q, shared, 2500, c.k, c.v, t, n, SCALE, want[-1], ws)
        torch.cuda.synchronize()
    q, t, n = qs[0].clone(), own.clone(), ls[0].clone()
    outs = [torch.empty_like(q) for _ in range(9)]

    def run():
        for i, o in enumerate(outs):
            q.copy_(qs[i % 3])
            t.copy_(tables[i % 3])
            n.copy_(ls[i % 3])
            moe.moe_gqa_prefix_decode(q, shared, 2500, c.k, c.v, t, n, SCALE, o, ws)

    run()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i % 3]) for i, o in enumerate(outs))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(5):
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, want[i % 3]) for i, o in enumerate(outs))
    assert moe.workspace_status(ws) == 0


def test_binding_refuses_shapes_and_types():
    c = ref.Cache((40, 300), 2, 16, DEV)
    q = randn(2, 16, D)
    ws = moe.alloc_paged_workspace(2, 2, 16, 2, D, 300, device=DEV)
    good = dict(q=q, k_cache=c.k, v_cache=c.v, block_table=c.table, seq_lens=i32([40, 300]), scale=SCALE,
                out=torch.empty_like(q), workspace=ws)
    moe.moe_gqa_paged_decode(**good)
    bad = [("q", q[:1], ValueError), ("q", q.view(32, D), ValueError), ("q", q.half(), TypeError), ("q", None, TypeError),
           ("q", randn(2, D, 16).transpose(1, 2), ValueError), ("v_cache", c.v[:-1], ValueError),
           ("k_cache", c.k[:, :, ::2], ValueError), ("block_table", c.table.long(), TypeError),
           ("block_table", c.table[0], ValueError), ("block_table", c.table[:, ::2], ValueError),
           ("seq_lens", i32([40]), ValueError), ("seq_lens", [40, 300], TypeError), ("out", torch.empty_like(q[:1]), ValueError),
           ("out", torch.empty_like(q, device="cpu"), ValueError), ("scale", "x", TypeError), ("scale", float("nan"), moe.MoeError),
           ("workspace", ws[:256], moe.MoeError), ("workspace", ws.int(), TypeError), ("workspace", ws[1:], moe.MoeError)]
    for name, value, kind in bad:
        with pytest.raises(kind):
            moe.moe_gqa_paged_decode(**{**good, name: value})
    for more in (dict(window=-1), dict(n_sink=-1)):
        with pytest.raises(moe.MoeError):
            moe.moe_gqa_paged_decode(**good, **more)
    for more in (dict(window=2 ** 31), dict(window=1 << 80)):
        with pytest.raises(OverflowError):
            moe.moe_gqa_paged_decode(**good, **more)
    for cu in (i32([0, 1]), i32([0, 1, 2, 2])):
        with pytest.raises(ValueError):
            moe.moe_gqa_paged_prefill(cu_q=cu, **good)
    shared = c.table[1].contiguous()
    moe.moe_gqa_prefix_decode(prefix_table=shared, prefix_len=300, **good)
    for table, n, kind in ((shared[:18], 300, ValueError), (None, 300, ValueError), (shared, -1, moe.MoeError),
                           (shared.view(1, -1), 300, ValueError), (shared.long(), 300, TypeError)):
        with pytest.raises(kind):
            moe.moe_gqa_prefix_decode(prefix_table=table, prefix_len=n, **good)
    qkv, pos = randn(2, 20 * D), i32([0, 1])
    qk = dict(qkv=qkv, q_weight=None, k_weight=None, eps=0.0, inv_freq=None, positions=pos, slots=i32([-1, -1]), q_out=q.clone(),
              k_cache=c.k, v_cache=c.v)
    moe.moe_qk_norm_rope(**qk)
    f = lambda n: torch.ones(n, device=DEV)  # noqa: E731
    for name, value, kind in [("qkv", qkv[:1], ValueError), ("qkv", qkv[:, :-1], ValueError), ("qkv", qkv[:1].expand(2, -1), moe.MoeError),
                              ("q_weight", f(D), TypeError), ("k_weight", qkv[0, :64], ValueError), ("inv_freq", f(65), moe.MoeError),
                              ("inv_freq", f(4), moe.MoeError), ("inv_freq", f((2, 32)), ValueError), ("eps", -1.0, moe.MoeError),
                              ("positions", pos[:1], ValueError), ("slots", pos.long(), TypeError), ("interleaved", 2, moe.MoeError)]:
        with pytest.raises(kind):
            moe.moe_qk_norm_rope(**{**qk, name: value})
    torch.cuda.synchronize()
    assert moe.workspace_status(ws) == 0


def test_prefill_more_blocks_and_sequences_than_one_search_step():
    """More than 32 x 32 row blocks of a sequence, and more sequences: sampled rows against 64 bits."""
    n, h_q = 20001, 16
    c = ref.Cache((n,), 1, 64, DEV)
    q = randn(n, h_q, D, seed=3)
    out, ws = torch.empty_like(q), moe.alloc_paged_workspace(n, 1, h_q, 1, D, device=DEV)
    moe.moe_gqa_paged_prefill(q, i32([0, n]), c.k, c.v, c.table, i32([n]), SCALE, out, ws, window=300, n_sink=5)
    rows = torch.cat([torch.arange(0, n, 97), torch.arange(n - 20, n)]).to(DEV)
    see = ref.visible(rows[:, None], torch.arange(n, device=DEV), 300, 5)
    ref.check(out[rows], *ref.attend(q[rows], *c.rows[0], see, SCALE), "sampled rows")
    assert moe.workspace_status(ws) == 0 and torch.isfinite(out.float()).all()
    g = np.random.default_rng(8)
    lens = g.integers(1, 60, 2048)
    run_prefill(lens.tolist(), [int(g.integers(0, m + 1)) for m in lens], 8, 1, 16)


def test_all_attention_calls_at_once_on_three_streams():
    lens = (3000, 200, 1500)
    c = ref.Cache(lens, 2, 16, DEV)
    lt, cu, shared = i32(lens), i32([0, 150, 151, 400]), c.table[0].contiguous()
    q, qp = randn(3, 16, D, seed=1), randn(400, 16, D, seed=2)
    ws = [moe.alloc_paged_workspace(400, 3, 16, 2, D, 3000, device=DEV) for _ in range(3)]
    calls = [lambda o, s: moe.moe_gqa_paged_decode(q, c.k, c.v, c.table, lt, SCALE, o, ws[0], window=900, n_sink=4, stream=s),
             lambda o, s: moe.moe_gqa_paged_prefill(qp, cu, c.k, c.v, c.table, lt, SCALE, o, ws[1], stream=s),
             lambda o, s: moe.moe_gqa_prefix_decode(q, shared, 3000, c.k, c.v, c.table, lt, SCALE, o, ws[2], stream=s)]
    like = [q, qp, q]
    want = [torch.empty_like(x) for x in like]
    for f, o in zip(calls, want):
        f(o, None)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [[torch.zeros_like(x) for x in like] for _ in range(20)]
    torch.cuda.synchronize()
    for r in range(20):
        for i in range(3):
            calls[i](outs[r][i], streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for row in outs for o, w in zip(row, want))
    assert all(moe.workspace_status(w) == 0 and not w[4:4096].any() for w in ws)
