"""The layer step's calls at sizes where their grids take several turns, and the norm's 8-bit codes next to where rounding turns
(needs a GPU)."""
import numpy as np
import pytest
import torch

import paged_reference as ref
import routed_expert_ffn_softmax_gb300 as moe
import step_reference as step
from test_kv4_gpu import i32
from test_norm_gpu import D, DEV, EPS, check_norm, randn, run_norm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from routed_expert_ffn_softmax_gb300 import build
    build.build()
    moe.load()
    yield


# ---------------------------------------------------------------- rows read back
@pytest.mark.parametrize("page,h_kv,lens,first", [(16, 2, [60000, 0, 70001, 5, 31], [7, 0, 33, 5, 0]),
                                                  (256, 8, [40000, 3, 25001], None)])
def test_load_of_more_blocks_than_the_grid_takes_at_once(page, h_kv, lens, first):
    """Two to three turns of the grid's warps, 16 tokens of a head each."""
    warps = 6 * 8 * torch.cuda.get_device_properties(DEV).multi_processor_count
    assert sum(ref.up(n, 16) for n in lens) * h_kv > 2 * warps
    c = step.Kv4(lens, h_kv, page, DEV, seed=page, codes_lo=-8)
    need = [ref.up(n, page) for n in lens]
    order = torch.randperm(sum(need) + 2, generator=torch.Generator().manual_seed(1)).to(torch.int32)
    dst = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
    for b, n in enumerate(need):
        dst[b, :n], order = order[:n], order[n:]
    dst = dst.to(DEV)
    k, v = (torch.full((sum(need) + 2, h_kv, page, D), -3.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    want = [k.clone(), v.clone()]
    ws = moe.alloc_paged_workspace(device=DEV)
    moe.moe_kv4_load(c.raw, c.table, None if first is None else i32(first), i32(lens), k, v, dst, ws)
    torch.cuda.synchronize()
    assert moe.workspace_status(ws) == 0 and not ws.any()
    for b, n in enumerate(lens):
        pos = torch.arange(0 if first is None else first[b], n, device=DEV)
        for w, rows in zip(want, c.values(b)):
            w[dst[b].long()[pos // page], :, pos % page] = rows[pos].to(torch.bfloat16)
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])


# ---------------------------------------------------------------- several position axes
@pytest.mark.parametrize("rot,interleaved", [(128, False), (64, False), (128, True)])
@pytest.mark.parametrize("N,h_q,h_kv,axes", [(2433, 3, 1, 2), (4000, 32, 4, 3), (8000, 16, 2, 4)])
@pytest.mark.parametrize("four", [False, True])
def test_many_tokens_with_several_axes_are_as_few(rot, interleaved, N, h_q, h_kv, axes, four):
    """Whole tokens in rounds over the warps and the rest in shares: every token as in a call of 97, bit by bit, and its rows'
    rotation by the formula."""
    page, pages = 64, ref.up(N, 64)
    g = torch.Generator().manual_seed(N + rot)
    qkv, w = randn(N, (h_q + 2 * h_kv) * D, seed=N), [randn(D, seed=i) for i in (1, 2)]
    inv = (10000.0 ** (-torch.arange(rot // 2) * 2 / rot)).float().to(DEV)
    pair = torch.randint(0, axes, (rot // 2,), generator=g, dtype=torch.int32).to(DEV)
    positions = torch.randint(0, 1 << 20, (axes, N + 3), generator=g, dtype=torch.int32).to(DEV)[:, 1:N + 1]
    slots = torch.randperm(N, generator=g).to(torch.int32).to(DEV)
    outs = []
    for few in (N, 97):
        q = torch.full((N, h_q, D), -9.0, dtype=torch.bfloat16, device=DEV)
        if four:
            caches = (moe.alloc_kv4_cache(pages, h_kv, page).fill_(7),)
        else:
            caches = tuple(torch.full((pages, h_kv, page, D), -9.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        call = moe.moe_qk_norm_rope_kv4 if four else moe.moe_qk_norm_mrope
        for at in range(0, N, few):
            to = min(N, at + few)
            call(qkv[at:to], *w, EPS, inv, pair, positions[:, at:to], slots[at:to], q[at:to], *caches, interleaved=interleaved)
        outs.append((q, *caches))
    for a, b in zip(*outs):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    x = qkv.view(N, -1, D)[:, :h_q]
    for a in range(axes):
        want, size = ref.norm_rope(x, w[0], EPS, positions[a], inv, interleaved)
        mine = torch.zeros(D, dtype=torch.bool, device=DEV)
        of = (pair == a).nonzero().flatten()
        mine[2 * of if interleaved else of] = True
        mine[2 * of + 1 if interleaved else of + rot // 2] = True
        # one rounding to bf16 (2^-8), and 2^-19 of the pair's size for the fp32 norm, sine and cosine
        over = (outs[0][0].double() - want).abs() - (2.0 ** -8 * want.abs() + 2.0 ** -19 * size + 1e-30)
        assert (over[..., mine] <= 0).all()


# ---------------------------------------------------------------- 8-bit codes
def near_halves(tops, per):
    """For each T of `tops` (a product of two 8-bit significands) `per` pairs (a, b, k), 128 <= a, b < 256, whose
    127 a b 2^-k / T come as close to a half, 0.5 .. 126.5, as such products do."""
    a = np.arange(128, 256)
    products, first = np.unique(np.outer(a, a).ravel(), return_index=True)
    pairs = [(128 + i // 128, 128 + i % 128) for i in first]
    out = []
    for T in tops:
        found = []
        for half in [0.5, 1.5, 2.5, 3.5, 7.5, 13.5, 31.5, 62.5, 63.5, 100.5, 126.5]:
            for k in range(0, 10):
                target = half * T / 127 * 2.0 ** k
                if not products[0] <= target <= products[-1]:
                    continue
                i = int(np.searchsorted(products, target))
                for n in (i - 1, i):
                    if 0 <= n < len(products):
                        off = abs(products[n] * 127.0 / 2.0 ** k / T - half)
                        if products[n] <= T * 2.0 ** k:  # |t| <= T
                            found.append((off / half, *pairs[n], k))
        out.append([f[1:] for f in sorted(found)[:per]])
    return out


@pytest.mark.parametrize("H,calls", [(1024, 40), (32768, 2)])
def test_norm_codes_of_quotients_next_to_halves(H, calls):
    """Quotients of 16-bit products that are no halves but within 2^-23 of one where t is small next to T: a correctly rounded
    division tells them apart from halves at every magnitude."""
    rng = np.random.RandomState(H)
    for call in range(calls):
        groups = H // 128
        tops = rng.randint(128, 256, (groups, 2))
        found = near_halves([int(x) * int(y) for x, y in tops], 20)
        r, w = np.zeros((groups, 128)), np.ones((groups, 128))
        for g, pairs in enumerate(found):
            r[g, 0], w[g, 0] = tops[g]
            for i, (x, y, k) in enumerate(pairs):
                for side, s in ((0, 1.0), (1, -1.0)):
                    r[g, 1 + 2 * i + side], w[g, 1 + 2 * i + side] = s * x * 2.0 ** -k, y
        residual = torch.from_numpy(r.reshape(1, H)).to(torch.bfloat16).to(DEV)
        weight = torch.from_numpy(w.reshape(H)).to(torch.bfloat16).to(DEV)
        assert torch.equal(residual.double().cpu(), torch.from_numpy(r.reshape(1, H)))
        check_norm(run_norm(None, residual, weight, q=True), None, residual, weight)
