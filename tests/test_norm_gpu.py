"""The residual's addition with the root-mean-square norm, and the rotation over several position axes, on the GPU,
through the binding, against plain 64-bit forms (needs a GPU)."""
import pytest
import torch

import paged_reference as ref
import routed_expert_ffn_softmax_gb300 as moe
import step_reference as step

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
D = 128
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _built():
    from routed_expert_ffn_softmax_gb300 import build
    build.build()
    moe.load()
    yield


def randn(*shape, seed=0, size=1.0):
    return (size * torch.randn(*shape, generator=torch.Generator().manual_seed(seed))).to(torch.bfloat16).to(DEV)


# ---------------------------------------------------------------- residual and norm
def run_norm(x, residual, weight, y=True, q=False, in_place=False, eps=EPS, stream=None):
    N, H = residual.shape
    out = dict(r=residual if in_place else torch.full_like(residual, -9.0),
               y=torch.full((N, H), -9.0, dtype=torch.bfloat16, device=DEV) if y else None,
               q=torch.full((N, H), -99, dtype=torch.int8, device=DEV) if q else None,
               s=torch.full((N, H // 128), -9.0, device=DEV) if q else None)
    moe.moe_add_rms_norm(x, residual, weight, eps, out["r"], out["y"], out["q"], out["s"], stream=stream)
    return out


def check_norm(out, x, residual, weight, eps=EPS):
    """y is rounded once (2^-8); its factor comes from fp32 sums of at most 64 + 10 steps and one rsqrt, 2^-17 in all."""
    r, y, t, factor = step.add_norm(x, residual, weight, eps)
    assert torch.equal(out["r"], r)
    if out["y"] is not None:
        assert ((out["y"].double() - y).abs() <= (2.0 ** -8 + 2.0 ** -17) * y.abs() + 1e-38).all()
    if out["q"] is not None:
        codes, top = step.int8_codes(t)
        assert torch.equal(out["q"], codes)
        scale = torch.where(top > 0, top * factor / 127, 1.0)
        assert ((out["s"].double() - scale).abs() <= 2.0 ** -17 * scale).all()


SIZES = [(1, 8), (1, 128), (3, 256), (5, 1000), (64, 4096), (7, 4104), (513, 6144), (40, 7168), (2, 8192), (3, 16384), (2, 16392),
         (2, 32768), (1000, 128), (3000, 1024), (1, 7168)]


@pytest.mark.parametrize("N,H", SIZES)
@pytest.mark.parametrize("add", [True, False])
def test_norm(N, H, add):
    x, residual, w = randn(N, H) if add else None, randn(N, H, seed=1, size=3.0), randn(H, seed=2)
    out = run_norm(x, residual, w, q=H % 128 == 0)
    check_norm(out, x, residual, w)
    alone = run_norm(x, residual, w, y=H % 128 != 0, q=H % 128 == 0)
    assert all(torch.equal(v, out[k]) for k, v in alone.items() if v is not None)


@pytest.mark.parametrize("H", [128, 4096, 4104])
def test_norm_in_place_strided_and_without_weight(H):
    wide, residual = randn(9, H + 24, seed=3), randn(9, H, seed=4)
    x = wide[:, 8:8 + H]
    check_norm(run_norm(x, residual, None), x, residual, None)
    kept = residual.clone()
    check_norm(run_norm(x, residual, None, in_place=True), x, kept, None)
    a, kept = randn(9, H), residual.clone()
    b = a.clone()
    moe.moe_add_rms_norm(a, residual, None, EPS, None, y=a)  # over its own input; the sum is not stored
    assert torch.equal(residual, kept)
    check_norm(dict(r=step.add_norm(b, kept, None, EPS)[0], y=a, q=None, s=None), b, kept, None)


def test_norm_codes_at_halves():
    """127 t / T is a half for many pairs of 8-bit numbers: all of them, and their neighbours, are decided exactly."""
    t = torch.arange(-127, 128, dtype=torch.float32)
    rows = []
    for top in (127, 2, 254, 170, 129, 255, 131, 192):
        rows += [torch.cat([v, torch.tensor([float(top)])]) for v in t.clamp(-top, top).unfold(0, 127, 32)]
    residual = torch.stack(rows).to(torch.bfloat16).to(DEV)
    w = torch.full((128,), 0.75, dtype=torch.bfloat16, device=DEV)
    for weight in (None, w):
        check_norm(run_norm(None, residual, weight, q=True), None, residual, weight)
    g = torch.Generator().manual_seed(0)
    many = torch.randint(-255, 256, (4000, 512), generator=g).to(torch.bfloat16).to(DEV)
    weight = torch.randint(1, 256, (512,), generator=g).to(torch.bfloat16).to(DEV)
    check_norm(run_norm(None, many, weight, q=True), None, many, weight)


@pytest.mark.parametrize("size", [1e-30, 1e-15, 1e15])
def test_norm_sizes(size):
    residual, w = randn(5, 512, size=size), randn(512, seed=1)
    out = run_norm(None, residual, w, q=True, eps=0.0 if size > 1e-20 else EPS)
    check_norm(out, None, residual, w, eps=0.0 if size > 1e-20 else EPS)


def test_norm_zeros_and_what_is_not_finite():
    residual = randn(6, 256)
    residual[1] = 0
    residual[2, 130:] = 0
    residual[3, 7] = float("nan")
    residual[4, 200] = float("inf")
    kept = residual.clone()
    out = run_norm(None, residual, None, q=True)
    live = [0, 1, 2, 5]
    check_norm({k: v[live] for k, v in out.items()}, None, kept[live], None)
    assert not out["q"][1].any() and (out["s"][1] == 1).all()
    assert out["y"][3].isnan().all() and out["s"][3].isnan().all()
    assert not out["y"][4, :200].any() and out["y"][4, 200].isnan()
    check_norm({k: v[[5]] for k, v in out.items()}, None, kept[[5]], None)


def test_norm_graph_and_streams():
    x, residual, w = randn(64, 4096), randn(64, 4096, seed=1), randn(4096, seed=2)
    want = run_norm(x, residual, w, q=True)
    got = {k: torch.zeros_like(v) for k, v in want.items()}
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        moe.moe_add_rms_norm(x, residual, w, EPS, got["r"], got["y"], got["q"], got["s"])
    for _ in range(2):
        for v in got.values():
            v.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(got[k], want[k]) for k in want)
    torch.cuda.synchronize()
    other = run_norm(x, residual, w, q=True, stream=stream)
    stream.synchronize()
    assert all(torch.equal(other[k], want[k]) for k in want)


def test_norm_rows_past_32_bits():
    N, H = (1 << 16) + 3, 32768
    residual = torch.zeros(N, H, dtype=torch.bfloat16, device=DEV)
    residual[-1] = randn(H)
    q, s = torch.empty(N, H, dtype=torch.int8, device=DEV), torch.empty(N, H // 128, device=DEV)
    moe.moe_add_rms_norm(None, residual, None, EPS, None, None, q, s)
    check_norm(dict(r=residual[-1:], y=None, q=q[-1:], s=s[-1:]), None, residual[-1:], None)
    assert not q[-2].any() and (s[-2] == 1).all()


# ---------------------------------------------------------------- several position axes
def rotate(qkv, h_q, h_kv, w, positions, inv, pair, slots, page, num_pages, interleaved=False):
    N = qkv.shape[0]
    q = torch.full((N, h_q, D), -9.0, dtype=torch.bfloat16, device=DEV)
    k, v = (torch.full((num_pages, h_kv, page, D), -9.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    moe.moe_qk_norm_mrope(qkv, *w, EPS, inv, pair, positions, slots, q, k, v, interleaved=interleaved)
    torch.cuda.synchronize()
    return q, k, v


@pytest.mark.parametrize("rot", [16, 64, 96, 128])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("axes,N,h_q,h_kv", [(1, 5, 3, 1), (2, 1, 16, 2), (3, 70, 8, 1), (4, 33, 2, 3), (16, 300, 32, 4)])
def test_axes(rot, interleaved, axes, N, h_q, h_kv):
    """One rounding to bf16 (2^-8), and 2^-19 of the pair's size for the fp32 norm, sine and cosine."""
    g = torch.Generator().manual_seed(rot + axes)
    qkv = torch.randn(N, (h_q + 2 * h_kv) * D, generator=g).to(torch.bfloat16).to(DEV)
    w = [(1 + 0.2 * torch.randn(D, generator=g)).to(torch.bfloat16).to(DEV) for _ in range(2)]
    wide = torch.randint(-1000, 1 << 20, (axes, N + 5), generator=g, dtype=torch.int32).to(DEV)
    positions = wide[:, :N]  # rows apart
    inv = (1e4 ** (-torch.arange(0, rot, 2).double() / rot)).float().to(DEV)
    pair = torch.randint(0, axes, (rot // 2,), generator=g, dtype=torch.int32).to(DEV)
    page, num_pages = 32, ref.up(N, 32) + 1
    slots = torch.randperm(num_pages * page, generator=g)[:N].to(torch.int32).to(DEV)
    q, k, v = rotate(qkv, h_q, h_kv, w, positions, inv, pair, slots, page, num_pages, interleaved)
    x = qkv.view(N, -1, D)
    off = torch.arange(N, device=DEV)
    pid, row = slots.long() // page, slots.long() % page
    for got, part, weight in ((q, x[:, :h_q], w[0]), (k[pid, :, row], x[:, h_q:h_q + h_kv], w[1])):
        for a in range(axes):  # the pairs of one axis at a time, each against one list of positions
            want, size = ref.norm_rope(part, weight, EPS, positions[a], inv, interleaved)
            mine = torch.zeros(D, dtype=torch.bool, device=DEV)
            of = (pair == a).nonzero().flatten()
            mine[2 * of if interleaved else of] = True
            mine[2 * of + 1 if interleaved else of + rot // 2] = True
            if a == 0:
                mine[rot:] = True
            bound = 2.0 ** -8 * want.abs() + 2.0 ** -19 * size + 1e-30
            assert ((got.double() - want).abs() <= bound)[..., mine].all()
    assert torch.equal(v[pid, :, row], x[:, h_q + h_kv:])
    other = torch.ones(num_pages * page, dtype=torch.bool, device=DEV)
    other[slots.long()] = False
    assert (k.transpose(1, 2).reshape(num_pages * page, -1)[other] == -9).all() and off.numel() == N


@pytest.mark.parametrize("rot,interleaved", [(128, False), (128, True), (64, False)])
def test_one_axis_gives_the_one_axis_call(rot, interleaved):
    """Bit by bit, whether the one axis is chosen by every pair or the axes hold the same positions."""
    N, h_q, h_kv = 50, 8, 2
    qkv, w = randn(N, (h_q + 2 * h_kv) * D), [randn(D, seed=i) for i in (1, 2)]
    inv = (1e6 ** (-torch.arange(0, rot, 2).double() / rot)).float().to(DEV)
    pos = torch.randint(0, 1 << 30, (N,), dtype=torch.int32, device=DEV)
    slots = torch.arange(N, dtype=torch.int32, device=DEV)
    want = [torch.full((N, h_q, D), -9.0, dtype=torch.bfloat16, device=DEV)]
    want += [torch.full((4, h_kv, 16, D), -9.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    moe.moe_qk_norm_rope(qkv, *w, EPS, inv, pos, slots, *want, interleaved=interleaved)
    pairs = torch.arange(rot // 2, dtype=torch.int32, device=DEV)
    for positions, pair in ((pos, pairs * 0), (pos[None], pairs * 0), (pos[None].repeat(3, 1), pairs % 3),
                            (pos[None].expand(4, N), pairs % 4)):
        got = rotate(qkv, h_q, h_kv, w, positions, inv, pair, slots, 16, 4, interleaved)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_pairs_of_no_axis_do_not_turn():
    N, h_q, h_kv = 9, 4, 1
    for rot, interleaved in ((128, False), (64, False), (128, True)):
        qkv = randn(N, (h_q + 2 * h_kv) * D)
        inv = torch.ones(rot // 2, device=DEV)
        pair = torch.tensor([0, -1, 2, 1 << 30] * (rot // 8), dtype=torch.int32, device=DEV)
        pos = torch.full((2, N), 3, dtype=torch.int32, device=DEV)
        slots = torch.arange(N, dtype=torch.int32, device=DEV)
        q, k, _ = rotate(qkv, h_q, h_kv, (None, None), pos, inv, pair, slots, 16, 1, interleaved)
        still = torch.ones(D, dtype=torch.bool, device=DEV)
        of = (pair == 0).nonzero().flatten()
        still[2 * of if interleaved else of] = False
        still[2 * of + 1 if interleaved else of + rot // 2] = False
        x = qkv.view(N, -1, D)
        assert torch.equal(q[..., still], x[:, :h_q][..., still]) and not torch.equal(q, x[:, :h_q])


@pytest.mark.parametrize("rot,interleaved", [(128, False), (64, False), (128, True)])
@pytest.mark.parametrize("h_q,h_kv", [(32, 4), (3, 1), (20, 20)])
@pytest.mark.parametrize("four", [False, True])
def test_many_tokens_are_as_few(rot, interleaved, h_q, h_kv, four):
    """A call's work is shared out by its size; every token is as in a call of a few."""
    page, heads = 64, h_q + 2 * h_kv
    w = randn(D, seed=1)
    inv = (10000.0 ** (-torch.arange(rot // 2) * 2 / rot)).float().to(DEV)
    for N in (61, 500, 1217, 2000, 2433, 3649, 5000, 7400):
        qkv = randn(N, heads * D, seed=N)
        positions = torch.arange(N, dtype=torch.int32, device=DEV) * 7
        slots = torch.randperm(N, generator=torch.Generator().manual_seed(2)).to(torch.int32).to(DEV)
        outs = []
        for step_tokens in (N, 97):
            q = torch.full((N, h_q, D), -9.0, dtype=torch.bfloat16, device=DEV)
            if four:
                cache = (moe.alloc_kv4_cache((N + page - 1) // page, h_kv, page).fill_(7),)  # (rows behind N stay)
            else:
                cache = tuple(torch.full(((N + page - 1) // page, h_kv, page, D), -9.0, dtype=torch.bfloat16, device=DEV)
                              for _ in range(2))
            for at in range(0, N, step_tokens):
                to = min(N, at + step_tokens)
                part = (qkv[at:to], w, w, EPS, inv)
                if four:
                    moe.moe_qk_norm_rope_kv4(*part, None, positions[at:to], slots[at:to], q[at:to], *cache,
                                             interleaved=interleaved)
                else:
                    moe.moe_qk_norm_rope(*part, positions[at:to], slots[at:to], q[at:to], *cache, interleaved=interleaved)
            outs.append((q, *cache))
        for a, b in zip(*outs):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), N


# ---------------------------------------------------------------- around the experts
def test_a_layer_step_with_the_experts():
    """Residual and norm in front of the routed experts and behind them, as a layer runs them."""
    import moe_workloads as mw
    cfg = mw.CONFIGS["tiny"]
    L = {k: (v.to(DEV) if v is not None else None) for k, v in mw.make_layer(cfg).items()}
    T, H = 8, cfg.H
    _, logits = mw.make_tokens(cfg, T)
    attn, residual, w1, w2 = randn(T, H, seed=5), randn(T, H, seed=6, size=2.0), randn(H, seed=7), randn(H, seed=8)
    res0 = residual.clone()
    h, out, y = (torch.empty(T, H, dtype=torch.bfloat16, device=DEV) for _ in range(3))
    ws = moe.alloc_workspace(T, H, cfg.I, cfg.E, cfg.top_k, moe.MOE_W_BF16, DEV)
    moe.moe_add_rms_norm(attn, residual, w1, EPS, residual, h)
    moe.moe_ffn_forward(h, logits.to(DEV), L["W_gate"], L["W_up"], L["W_down"], None, None, None, cfg.top_k, out, ws)
    moe.moe_add_rms_norm(out, residual, w2, EPS, residual, y)
    torch.cuda.synchronize()
    assert moe.workspace_status(ws) == 0
    r1 = (attn.double() + res0.double()).to(torch.bfloat16)
    want, *_ = step.add_norm(out, r1, w2, EPS)
    assert torch.equal(residual, want)
    check_norm(dict(r=residual, y=y, q=None, s=None), out, r1, w2)
    import numpy as np
    import oracle
    ref_out = oracle.forward(h.cpu(), logits, *(L[n].cpu() for n in ("W_gate", "W_up", "W_down")), wtype="bf16", top_k=cfg.top_k)
    want = torch.from_numpy(oracle.bf16_bits_to_f32(ref_out["out"]).astype(np.float64))
    assert ((out.double().cpu() - want).abs() <= 1e-2 * want.abs().max() + 1e-3).all()
