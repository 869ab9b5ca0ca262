"""The serving path over a paged key/value cache: what its header declares is exported, bad calls are refused on the
host before any CUDA work, and the 64-bit plain forms the GPU tests use agree with libraries (no GPU needed)."""
import ctypes
import os
import re

import pytest
import torch

import paged_reference as ref
import routed_expert_ffn_softmax_gb300 as moe
from routed_expert_ffn_softmax_gb300 import build as moe_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "paged", "moe_paged.h")
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
F = 1 << 20  # an aligned non-null address; never dereferenced (the calls below fail first)


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return moe.load()


def test_header_and_exports(lib):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(moe_[a-z_0-9]+)\s*\(", src)))
    assert names == sorted(["moe_paged_workspace_size", "moe_paged_plan", "moe_qk_norm_rope", "moe_gqa_paged_decode",
                            "moe_gqa_paged_prefill", "moe_gqa_prefix_decode"])
    out = os.popen(f"nm -D --defined-only {moe_build.LIB}").read()
    for n in names:
        assert re.search(rf"\bT {n}$", out, flags=re.M) and n in moe.__all__, n


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "paged/moe_paged.h"\nint main(void) { return (int)sizeof(moe_status_t) == 0; }\n')
    assert os.system(f"gcc -std=c99 -Wall -Werror -I {ROOT}/include -c {src} -o {tmp_path}/t.o") == 0


def test_workspace_size(lib):
    ws = moe.moe_paged_workspace_size
    assert ws() > 0 and ws() % 256 == 0
    base = ws(64, 64, 32, 4, 128, 0)
    for bigger in (ws(5000, 64, 32, 4, 128, 0), ws(64, 64, 32, 4, 128, 8192), ws(2048, 2048, 32, 4, 128, 0)):
        assert bigger >= base
    # monotone in the tokens, the sequences and the prefix
    sizes = [ws(B, B, 64, 4, 128, p) for B in (1, 8, 9, 64, 300, 2048) for p in (0, 1, 129, 40000)]
    for i, B in enumerate((1, 8, 9, 64, 300, 2048)):
        row = sizes[4 * i:4 * i + 4]
        assert row == sorted(row)
        assert all(x <= y for x, y in zip(row, sizes[4 * i + 4:4 * i + 8]))
    for bad in ((-1, 1, 8, 1, 128, 0), (1, -1, 8, 1, 128, 0), (1, 1, 0, 1, 128, 0), (1, 1, 8, 3, 128, 0),
                (1, 1, 8, 1, 64, 0), (1, 1, 17, 1, 128, 0), (1, 2049, 8, 1, 128, 0), (1, 1, 8, 1, 128, -1)):
        assert ws(*bad) == 0
    with pytest.raises(ValueError):
        moe.alloc_paged_workspace(1, 1, 8, 3, device="cpu")


def plan(lib, **kw):
    a = dict(ctx=F, new=F, B=4, page=16, pages=100, free=F, n_free=10, count=F, table=F, width=8, lens=F, cu=F, pos=F,
             slots=F, rows=64, left=F, ws=F, ws_bytes=1 << 20)
    a.update(kw)
    return lib.moe_paged_plan(*a.values(), None)


def test_plan_refusals(lib):
    assert plan(lib, B=-1) == INVALID
    assert plan(lib, n_free=-1) == INVALID and plan(lib, rows=-1) == INVALID
    for page in (0, -16, 8, 24, 2048):
        assert plan(lib, page=page) == INVALID
    assert plan(lib, pages=0) == INVALID and plan(lib, width=0) == INVALID
    assert plan(lib, pages=1 << 27) == UNSUPPORTED          # 2^31 slots
    assert plan(lib, width=1 << 27) == UNSUPPORTED          # positions past 32 bits
    assert plan(lib, B=2049) == UNSUPPORTED
    for name in ("ctx", "new", "free", "count", "table", "lens", "cu", "pos", "slots", "left", "ws"):
        assert plan(lib, **{name: None}) == INVALID, name
        assert plan(lib, **{name: F + 2}) == INVALID, name
    assert plan(lib, ws=F + 128) == INVALID
    assert plan(lib, ws_bytes=1024) == WORKSPACE
    assert plan(lib, B=0, ctx=None, ws=None) == OK


def qk(lib, **kw):
    a = dict(qkv=F, stride=40 * 128, N=4, h_q=32, h_kv=4, d=128, qw=F, kw=F, eps=1e-6, inv=F, rot=128, inter=0, pos=F,
             slots=F, q=F, k=F, v=F, pages=100, page=16)
    a.update(kw)
    return lib.moe_qk_norm_rope(*a.values(), None)


def test_qk_refusals(lib):
    assert qk(lib, N=-1) == INVALID and qk(lib, h_q=0) == INVALID and qk(lib, h_kv=0) == INVALID
    assert qk(lib, d=64, rot=64) == UNSUPPORTED
    for rot in (-16, 8, 20, 144):
        assert qk(lib, rot=rot) == INVALID
    assert qk(lib, inter=2) == INVALID and qk(lib, inter=-1) == INVALID
    assert qk(lib, stride=40 * 128 - 8) == INVALID and qk(lib, stride=40 * 128 + 4) == INVALID
    assert qk(lib, eps=-1.0) == INVALID and qk(lib, eps=float("nan")) == INVALID
    assert qk(lib, page=48) == INVALID and qk(lib, pages=0) == INVALID
    assert qk(lib, pages=1 << 27) == UNSUPPORTED
    for name in ("qkv", "inv", "pos", "slots", "q", "k", "v"):
        assert qk(lib, **{name: None}) == INVALID, name
    for name in ("qkv", "qw", "kw", "q", "k", "v"):
        assert qk(lib, **{name: F + 8}) == INVALID, name
    for name in ("inv", "pos", "slots"):
        assert qk(lib, **{name: F + 2}) == INVALID, name
    assert qk(lib, N=0, qkv=None, q=None) == OK


def attn(lib, which, **kw):
    decode = dict(q=F, k=F, v=F, table=F, lens=F, B=2, h_q=32, h_kv=4, d=128, pages=100, page=16, width=8, scale=0.1,
                  window=0, sink=0, out=F, ws=F, ws_bytes=1 << 40)
    prefill = dict(q=F, cu=F, k=F, v=F, table=F, lens=F, N=64, B=2, h_q=32, h_kv=4, d=128, pages=100, page=16, width=8,
                   scale=0.1, window=0, sink=0, out=F, ws=F, ws_bytes=1 << 40)
    prefix = dict(q=F, ptable=F, prefix=500, k=F, v=F, table=F, lens=F, B=2, h_q=32, h_kv=4, d=128, pages=100, page=16,
                  width=8, scale=0.1, out=F, ws=F, ws_bytes=1 << 40)
    fn, a = {"decode": (lib.moe_gqa_paged_decode, decode), "prefill": (lib.moe_gqa_paged_prefill, prefill),
             "prefix": (lib.moe_gqa_prefix_decode, prefix)}[which]
    assert set(kw) <= set(a), kw
    a.update(kw)
    return fn(*a.values(), None)


@pytest.mark.parametrize("which", ["decode", "prefill", "prefix"])
def test_attention_refusals(lib, which):
    f = lambda **kw: attn(lib, which, **kw)  # noqa: E731
    assert f(B=-1) == INVALID and f(h_kv=3) == INVALID and f(h_q=0) == INVALID
    assert f(h_q=68) == UNSUPPORTED and f(d=64) == UNSUPPORTED and f(B=2049) == UNSUPPORTED
    assert f(page=20) == INVALID and f(page=2048) == INVALID and f(pages=0) == INVALID and f(width=0) == INVALID
    assert f(pages=1 << 27) == UNSUPPORTED and f(width=1 << 27) == UNSUPPORTED
    assert f(pages=1 << 20, page=1024, h_q=1 << 12, h_kv=1 << 12) == UNSUPPORTED  # num_pages * h_kv past 32 bits
    assert f(scale=float("inf")) == INVALID and f(scale=float("nan")) == INVALID
    names = ["q", "k", "v", "table", "lens", "out", "ws"] + {"prefill": ["cu"], "prefix": ["ptable"]}.get(which, [])
    for name in names:
        assert f(**{name: None}) == INVALID, name
        assert f(**{name: F + 2}) == INVALID, name
    assert f(ws=F + 128) == INVALID and f(q=F + 8) == INVALID
    assert f(ws_bytes=4096) == WORKSPACE
    assert f(B=0, q=None, out=None, ws=None) == OK
    if which != "prefix":
        assert f(window=-1) == INVALID and f(sink=-1) == INVALID
    else:
        assert f(prefix=-1) == INVALID
    if which == "prefill":
        assert f(N=-1) == INVALID and f(N=0, q=None) == OK
        assert f(N=1 << 27) == UNSUPPORTED           # N * h_q past 32 bits
    # key tiles are counted in 32 bits
    assert f(B=2048, h_q=64, h_kv=64, width=(1 << 30) // 16, **({"N": 2048} if which == "prefill" else {})) == UNSUPPORTED


def test_binding_refuses_before_the_call(lib):
    t = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)  # noqa: E731
    i = torch.int32
    ws = t(1 << 13, dt=torch.uint8)
    with pytest.raises(ValueError):  # host tensors
        moe.moe_gqa_paged_decode(t(2, 32, 128), t(9, 4, 16, 128), t(9, 4, 16, 128), t(2, 3, dt=i), t(2, dt=i), 0.1,
                                 t(2, 32, 128), ws)
    with pytest.raises(TypeError):   # fp16 queries
        moe.moe_gqa_paged_decode(t(2, 32, 128, dt=torch.float16), t(9, 4, 16, 128), t(9, 4, 16, 128), t(2, 3, dt=i),
                                 t(2, dt=i), 0.1, t(2, 32, 128), ws)
    with pytest.raises(TypeError):
        moe.moe_qk_norm_rope(t(2, 40 * 128), None, None, 0.0, None, t(2, dt=i), t(2, dt=i), t(2, 32, 128),
                             t(9, 4, 16, 128), t(9, 4, 16, 128))
    with pytest.raises(TypeError):   # 64-bit lengths
        moe.moe_paged_plan(t(2, dt=torch.int64), t(2, dt=i), 16, 9, t(9, dt=i), t(1, dt=i), t(2, 3, dt=i), t(2, dt=i),
                           t(3, dt=i), t(4, dt=i), t(4, dt=i), t(1, dt=i), ws)


def test_reference_attention_against_a_library():
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((9, 8, 16), (30, 2, 16), (30, 2, 16)))
    pos, key = torch.arange(21, 30)[:, None], torch.arange(30)
    for window, n_sink in ((0, 0), (5, 0), (5, 3), (1, 40)):
        see = ref.visible(pos, key, window, n_sink)
        got, size = ref.attend(q, k, v, see, 0.3)
        kk, vv = (x.repeat_interleave(4, 1).transpose(0, 1) for x in (k, v))
        want = torch.nn.functional.scaled_dot_product_attention(q.transpose(0, 1), kk, vv, attn_mask=see, scale=0.3)
        assert (got - want.transpose(0, 1)).abs().max() < 1e-12 and (size >= got.abs() - 1e-12).all()
    rows = [[int(j) for j in key if j <= p and (j > p - 5 or j < 3)] for p in range(21, 30)]
    see = ref.visible(pos, key, 5, 3)
    assert [see[i].nonzero().flatten().tolist() for i in range(9)] == rows
    o, _ = ref.attend(q[:1], k, v, torch.zeros(1, 30, dtype=torch.bool), 0.3)
    assert not o.any()


def test_reference_rotation_is_complex_multiplication():
    x = torch.randn(3, 2, 8, generator=torch.Generator().manual_seed(0), dtype=torch.float64)
    inv = torch.tensor([1.0, 0.1])
    pos = torch.tensor([0, 5, 100000])
    for inter in (False, True):
        y, _ = ref.norm_rope(x, None, 0.0, pos, inv, inter)
        pair = (lambda t, i: (t[..., 2 * i], t[..., 2 * i + 1])) if inter else (lambda t, i: (t[..., i], t[..., i + 2]))
        for i in range(2):
            turn = torch.polar(torch.ones(3, dtype=torch.float64), pos.double() * inv[i].double())[:, None]
            z = torch.complex(*pair(x, i)) * turn
            a, b = pair(y, i)
            assert (torch.complex(a, b) - z).abs().max() < 1e-12
        assert torch.equal(y[..., 4:], x[..., 4:])


def test_reference_plan_worked_example():
    """Pages of 16: sequence 0 has 20 tokens in pages 7, 3 and adds 14 (positions 20 .. 33: one new page); sequence 1
    starts with 3 tokens (one new page)."""
    r = ref.plan([20, 0], [14, 3], 16, 10, [4, 8, 5, 9], 3, [[7, 3, -1], [-1, -1, -1]], 20)
    assert r["table"] == [[7, 3, 5], [8, -1, -1]] and r["seq_lens"] == [34, 3] and r["cu"] == [0, 14, 17]
    assert r["slots"][:17] == [3 * 16 + i for i in range(4, 16)] + [80, 81] + [128, 129, 130]
    assert r["positions"][:17] == list(range(20, 34)) + [0, 1, 2] and r["slots"][17:] == [-1] * 3
    assert r["left"] == 1 and r["status"] == 0
