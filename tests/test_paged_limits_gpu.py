"""The serving path over a paged key/value cache at the edges its header allows: the largest token row counts, large
frequencies at far positions, a scale of 0, bad pages, the precedence of the status word's codes (needs a GPU)."""
import pytest
import torch

import paged_reference as ref
import routed_expert_ffn_softmax_gb300 as moe
from test_paged_gpu import DEV, D, SCALE, i32, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from routed_expert_ffn_softmax_gb300 import build
    build.build()
    moe.load()
    yield


# ---------------------------------------------------------------- plan
def test_plan_with_as_many_token_rows_as_32_bits_count():
    """2^31 - 1 token rows, nearly all of them one sequence's: every row's position and slot, and the words around the
    rows as they were."""
    page, pages, n_rows, pad = 1024, 2 ** 21 - 1, 2 ** 31 - 1, 4096
    new = [3, 2 ** 31 - 6000]
    width = ref.up(new[1], page)
    ws = moe.alloc_paged_workspace(device=DEV)
    rows = [torch.full((n_rows + 2 * pad,), -5, dtype=torch.int32, device=DEV) for _ in range(2)]
    positions, slots = (r[pad:pad + n_rows] for r in rows)
    table, lens, cu, left = (torch.full(s, -1, dtype=torch.int32, device=DEV) for s in ((2, width), (2,), (3,), (1,)))
    free = torch.arange(pages, dtype=torch.int32, device=DEV)
    moe.moe_paged_plan(i32([0, 0]), i32(new), page, pages, free, i32([pages]), table, lens, cu, positions, slots, left, ws)
    torch.cuda.synchronize()
    assert moe.workspace_status(ws) == 0
    assert lens.tolist() == new and cu.tolist() == [0, 3, sum(new)] and left.tolist() == [pages - 1 - width]
    # pages come from the end of the list: sequence 0 has the last, sequence 1 those before it
    assert table[0, 0] == pages - 1 and torch.equal(table[1], pages - 2 - torch.arange(width, dtype=torch.int32, device=DEV))
    assert all((r[:pad] == -5).all() and (r[pad + n_rows:] == -5).all() for r in rows)
    for at in range(0, n_rows, 1 << 27):
        t = torch.arange(at, min(n_rows, at + (1 << 27)), device=DEV)
        pos = torch.where(t < 3, t, t - 3)
        slot = torch.where(t < 3, (pages - 1) * page + pos, (pages - 2 - pos // page) * page + pos % page)
        real = t < sum(new)
        assert torch.equal(positions[at:at + t.numel()], torch.where(real, pos, 0).to(torch.int32))
        assert torch.equal(slots[at:at + t.numel()], torch.where(real, slot, -1).to(torch.int32))


# ---------------------------------------------------------------- norm and rotation
def turns_per_position(inv_freq, bits=200):
    """inv_freq / (2 pi) modulo 1 of fp32 values, as whole numbers of 2^-bits turns (pi by Machin's formula)."""
    one = 1 << (bits + 400)

    def arctan_inverse(n):
        term, total, k = one // n, one // n, 1
        while term:
            term //= -n * n
            k += 2
            total += term // k
        return total

    two_pi = 8 * (4 * arctan_inverse(5) - arctan_inverse(239))
    out = []
    for f in inv_freq.tolist():
        num, den = f.as_integer_ratio()
        out.append((num * one * (one >> 400) // (den * two_pi)) % (1 << bits))
    return out


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("largest", [1.0, 7.0, 1000.0])
def test_the_angle_of_large_frequencies_at_far_positions(largest, interleaved):
    """Off by less than |pos| max(1, |inv_freq|) 2^-53 turns, against whole-number arithmetic; positive and negative
    frequencies, positions near 2^31 and below 0. (2^-19 of |a| + |b| for the fp32 sine, cosine and sums, as in run_qk; 1%
    for the square of the angle's error, which is below 2^-9.)"""
    g = torch.Generator().manual_seed(3)
    N, bits = 60, 200
    inv = (largest * torch.rand(D // 2, generator=g)).float() * (1 - 2 * (torch.arange(D // 2) % 2))
    pos = torch.cat([2 ** 31 - 1 - torch.randint(0, 10 ** 6, (N // 2,), generator=g), -torch.randint(1, 10 ** 9, (N // 2,), generator=g)])
    x = torch.randn(N, 3, D, generator=g).to(torch.bfloat16)
    q, k = torch.empty(N, 1, D, dtype=torch.bfloat16, device=DEV), torch.empty(4, 1, 16, D, dtype=torch.bfloat16, device=DEV)
    moe.moe_qk_norm_rope(x.view(N, -1).to(DEV), None, None, 0.0, inv.to(DEV), pos.to(torch.int32).to(DEV), i32([-1] * N), q, k,
                         k.clone(), interleaved=interleaved)
    turn = turns_per_position(inv, bits)
    angle = torch.tensor([[(t * p % (1 << bits)) / (1 << bits) for t in turn] for p in pos.tolist()], dtype=torch.float64)
    angle = angle * (2 * torch.pi)
    first, second = (slice(0, D, 2), slice(1, D, 2)) if interleaved else (slice(0, D // 2), slice(D // 2, D))
    a, b = x[:, 0, first].double(), x[:, 0, second].double()
    off = 2 * torch.pi * pos.abs().double()[:, None] * inv.abs().double().clamp(min=1.0) * 2.0 ** -53
    for at, want in ((first, a * angle.cos() - b * angle.sin()), (second, b * angle.cos() + a * angle.sin())):
        over = (q[:, 0, at].cpu().double() - want).abs() - (2.0 ** -8 * want.abs() + (2.0 ** -19 + 1.01 * off) * (a.abs() + b.abs()))
        assert over.max() <= 0, f"off by {over.max():.3g}"


@pytest.mark.parametrize("rot", [128, 32])
def test_rows_whose_squares_overflow_come_out_as_zero(rot):
    x = randn(3, 3 * D, seed=1)
    x[1] *= 2.0 ** 64
    w, inv = torch.ones(D, dtype=torch.bfloat16, device=DEV), torch.ones(rot // 2, device=DEV)
    q, k = torch.empty(3, 1, D, dtype=torch.bfloat16, device=DEV), torch.full((1, 1, 16, D), 7.0, dtype=torch.bfloat16, device=DEV)
    v = k.clone()
    moe.moe_qk_norm_rope(x, w, w, 1e-6, inv, i32([5, 6, 7]), i32([0, 1, 2]), q, k, v)
    assert not q[1].any() and not k[0, 0, 1].any() and torch.equal(v[0, 0, 1], x[1, 2 * D:])
    assert q[0].any() and q[2].any() and torch.isfinite(q.float()).all()


# ---------------------------------------------------------------- attention
@pytest.mark.parametrize("size", [1.0, 1e15])
def test_a_scale_of_zero_weighs_all_keys_alike(size):
    """Whatever the scores: with queries and keys of 1e15 they reach 1e31."""
    lens = (300, 70)
    c = ref.Cache(lens, 2, 16, DEV)
    for b, n in enumerate(lens):
        c.rows[b][0] = (c.rows[b][0].float() * size).to(torch.bfloat16)
        c.put(b, slice(0, n), *c.rows[b])
    q = (randn(130, 16, D, seed=2).float() * size).to(torch.bfloat16)
    ws = moe.alloc_paged_workspace(130, 130, 16, 2, D, 300, device=DEV)
    out = torch.empty_like(q)
    moe.moe_gqa_paged_prefill(q, i32([0, 60, 130]), c.k, c.v, c.table, i32(lens), 0.0, out, ws)
    for b, (rows, n) in enumerate(((slice(0, 60), 300), (slice(60, 130), 70))):
        pos = torch.arange(n - (rows.stop - rows.start), n, device=DEV)[:, None]
        see = ref.visible(pos, torch.arange(n, device=DEV), 0, 0)
        ref.check(out[rows], *ref.attend(q[rows], *c.rows[b], see, 0.0), f"prompt {b}")
    out = torch.empty_like(q[:2])
    moe.moe_gqa_paged_decode(q[:2], c.k, c.v, c.table, i32(lens), 0.0, out, ws)
    for b, n in enumerate(lens):
        ref.check(out[b:b + 1], *ref.attend(q[b:b + 1], *c.rows[b], torch.ones(1, n, dtype=torch.bool, device=DEV), 0.0), "one token")
    moe.moe_gqa_prefix_decode(q[:2], c.table[0].contiguous(), 300, c.k, c.v, c.table[1:].expand(2, -1).contiguous(),
                              i32([70, 0]), 0.0, out, ws)
    for b, n in enumerate((70, 0)):
        k, v = (torch.cat([c.rows[0][i], c.rows[1][i][:n]]) for i in (0, 1))
        see = torch.ones(1, 300 + n, dtype=torch.bool, device=DEV)
        ref.check(out[b:b + 1], *ref.attend(q[b:b + 1], k, v, see, 0.0), f"behind a prefix, {n} own keys")
    assert moe.workspace_status(ws) == 0


def zeroed(c, b, idx):
    """Sequence b's rows with those of its idx-th page zero."""
    rows = [r.clone() for r in c.rows[b]]
    for r in rows:
        r[idx * c.page:(idx + 1) * c.page] = 0
    return rows


# sequence 1 has 1000 keys; behind a window of 200 the first visible one of it is 800, 32 keys into a tile, so that up to 32
# sink keys are copied into the rows before it in boxes of 16
BAD_PAGES = [(16, 0, 0, 0), (16, 0, 0, 61), (64, 0, 0, 15), (1024, 0, 0, 0), (16, 200, 3, 0), (16, 200, 20, 1), (16, 200, 3, 50),
             (64, 200, 3, 0), (64, 200, 3, 12), (256, 200, 30, 0), (256, 200, 30, 3), (16, 200, 140, 8), (64, 200, 140, 2)]


@pytest.mark.parametrize("entry", [-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1])
@pytest.mark.parametrize("page,window,n_sink,idx", BAD_PAGES)
def test_a_bad_page_reads_as_zeros(page, window, n_sink, idx, entry):
    lens = (40, 1000, 64)
    c = ref.Cache(lens, 2, page, DEV, seed=idx)
    c.table[1, idx] = entry
    rows = [c.rows[0], zeroed(c, 1, idx), c.rows[2]]
    ws = moe.alloc_paged_workspace(90, 3, 16, 2, D, device=DEV)
    q = randn(90, 16, D, seed=1)
    out = torch.empty_like(q)
    for what, new in (("one token", (1, 1, 1)), ("prompt", (20, 50, 20))):
        ws[:4] = 0
        cu = [0, new[0], new[0] + new[1], sum(new)]
        if what == "prompt":
            moe.moe_gqa_paged_prefill(q, i32(cu), c.k, c.v, c.table, i32(lens), SCALE, out, ws, window=window, n_sink=n_sink)
        else:
            moe.moe_gqa_paged_decode(q[:3], c.k, c.v, c.table, i32(lens), SCALE, out[:3], ws, window=window, n_sink=n_sink)
        assert moe.workspace_status(ws) == 6, what
        for b, n in enumerate(lens):
            pos = torch.arange(n - new[b], n, device=DEV)[:, None]
            see = ref.visible(pos, torch.arange(n, device=DEV), window, n_sink)
            at = slice(cu[b], cu[b + 1])
            ref.check(out[at], *ref.attend(q[at], *rows[b], see, SCALE), f"{what}, sequence {b}")


# ---------------------------------------------------------------- the status word
@pytest.mark.parametrize("before", [0, 1, 2, 3, 4, 6, 7])
def test_the_status_word_keeps_the_code_that_matters_most(before):
    """1 to 3 stay whatever comes (the workspace is not fit for use); of the others the largest is kept."""
    c = ref.Cache((40, 300), 2, 16, DEV)
    q, qp = randn(2, 16, D), randn(30, 16, D)
    out, outp = torch.empty_like(q), torch.empty_like(qp)
    ws = moe.alloc_paged_workspace(30, 2, 16, 2, D, 40, device=DEV)
    bad_pages = c.table.clone()
    bad_pages[1, 3] = -1
    good, lt, bad = c.table, i32([40, 300]), i32([-1, 300])
    cu, one, rows = i32([0, 10, 30]), i32([1]), i32([0] * 4)
    plan = lambda ctx, free: moe.moe_paged_plan(  # noqa: E731
        i32([ctx]), one, 16, 50, i32([5]), i32([free]), i32([[3, 4]]), i32([0]), i32([0, 0]), rows, rows.clone(), i32([0]), ws)
    calls = {
        "one token, bad length": (4, lambda: moe.moe_gqa_paged_decode(q, c.k, c.v, good, bad, SCALE, out, ws)),
        "one token, bad page": (6, lambda: moe.moe_gqa_paged_decode(q, c.k, c.v, bad_pages, lt, SCALE, out, ws)),
        "prompt, bad length": (4, lambda: moe.moe_gqa_paged_prefill(qp, cu, c.k, c.v, good, bad, SCALE, outp, ws)),
        "prompt, bad page": (6, lambda: moe.moe_gqa_paged_prefill(qp, cu, c.k, c.v, bad_pages, lt, SCALE, outp, ws)),
        "prefix, bad page": (6, lambda: moe.moe_gqa_prefix_decode(q, i32([0, -1, 1]), 40, c.k, c.v, good, lt, SCALE, out, ws)),
        "plan, bad length": (4, lambda: plan(-1, 1)),
        "plan, no room": (7, lambda: plan(16, 0)),
    }
    for what, (code, call) in calls.items():
        ws[:4] = torch.tensor([before, 0, 0, 0], dtype=torch.uint8, device=DEV)
        call()
        torch.cuda.synchronize()
        assert moe.workspace_status(ws) == (before if 1 <= before <= 3 else max(before, code)), what
    assert not ws[4:4096].any()


def test_the_contiguous_cache_keeps_the_code_of_a_wait_too():
    ws = moe.alloc_gqa_workspace(1, 8, 1, D, 64, DEV)
    k = torch.zeros(1, 1, 64, D, dtype=torch.bfloat16, device=DEV)
    q = randn(1, 8, D)
    for before, after in ((0, 4), (1, 1), (3, 3), (4, 4)):
        ws[:4] = torch.tensor([before, 0, 0, 0], dtype=torch.uint8, device=DEV)
        moe.moe_gqa_decode(q, k, k, i32([65]), SCALE, torch.empty_like(q), ws)
        torch.cuda.synchronize()
        assert moe.workspace_status(ws) == after
