"""The norms, the several-axis rotation and the 4-bit cache: what their headers declare is exported, bad calls are refused on
the host before any CUDA work, and the plain forms of the GPU tests hold (no GPU needed)."""
import os
import re

import pytest
import torch

import routed_expert_ffn_softmax_gb300 as moe
import step_reference as step
from routed_expert_ffn_softmax_gb300 import build as moe_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
F = 1 << 20  # an aligned non-null address; never dereferenced (the calls below fail first)
WS = 1 << 30
DECLARED = {"moe_norm.h": ["moe_add_rms_norm", "moe_qk_norm_mrope"],
            "moe_kv4.h": ["moe_gqa_kv4_decode", "moe_kv4_load", "moe_qk_norm_rope_kv4"]}


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return moe.load()


@pytest.mark.parametrize("header", DECLARED)
def test_header_and_exports(lib, header, tmp_path):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "paged", header)).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(moe_[a-z_0-9]+)\s*\(", src)))
    assert names == DECLARED[header]
    out = os.popen(f"nm -D --defined-only {moe_build.LIB}").read()
    for n in names:
        assert re.search(rf"\bT {n}$", out, flags=re.M) and n in moe.__all__, n
    t = tmp_path / "t.c"
    t.write_text(f'#include "paged/{header}"\nint main(void) {{ return (int)sizeof(moe_status_t) == 0; }}\n')
    assert os.system(f"gcc -std=c99 -Wall -Werror -I {ROOT}/include -c {t} -o {tmp_path}/t.o") == 0


def changed(base, **kw):
    d = dict(base)
    assert set(kw) <= set(d)
    d.update(kw)
    return list(d.values())


NORM = dict(x=F, x_stride=256, residual=F, weight=F, eps=1e-6, N=4, H=256, residual_out=F, y=F, q=F, scales=F, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(N=0), OK), (dict(N=0, residual=None), OK), (dict(N=-1), INVALID), (dict(H=0), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(q=None), INVALID), (dict(scales=None), INVALID),
    (dict(y=None, q=None, scales=None), INVALID), (dict(H=264, x_stride=264), UNSUPPORTED),
    (dict(H=260, x_stride=264, q=None, scales=None), UNSUPPORTED), (dict(H=32896, x_stride=32896), UNSUPPORTED),
    (dict(x_stride=255), INVALID), (dict(x_stride=260), INVALID), (dict(x_stride=248), INVALID), (dict(residual=None), INVALID),
    (dict(x=F + 8), INVALID), (dict(residual=F + 2), INVALID), (dict(weight=F + 4), INVALID), (dict(residual_out=F + 8), INVALID),
    (dict(y=F + 8), INVALID), (dict(q=F + 8), INVALID), (dict(scales=F + 2), INVALID)])
def test_norm_refusals(lib, kw, want):
    assert lib.moe_add_rms_norm(*changed(NORM, **kw)) == want


ROPE = dict(qkv=F, row_stride=1280, N=4, h_q=8, h_kv=1, d=128, q_weight=F, k_weight=F, eps=1e-6, inv_freq=F, pair_axis=F,
            rot_dim=128, interleaved=0, positions=F, axis_stride=4, n_axes=3, slots=F, q_out=F, k_cache=F, v_cache=F, num_pages=4,
            page_size=16, stream=None)
ROPE4 = {("kv4_cache" if k == "k_cache" else k): v for k, v in ROPE.items() if k != "v_cache"}
ROPE_CASES = [
    (dict(N=0), OK), (dict(N=-1), INVALID), (dict(h_q=0), INVALID), (dict(h_kv=0), INVALID), (dict(d=64, rot_dim=64), UNSUPPORTED),
    (dict(rot_dim=8), INVALID), (dict(rot_dim=144), INVALID), (dict(interleaved=2), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(row_stride=1279), INVALID), (dict(row_stride=1284), INVALID), (dict(page_size=8), INVALID),
    (dict(page_size=48), INVALID), (dict(num_pages=0), INVALID), (dict(num_pages=1 << 27), UNSUPPORTED),
    (dict(n_axes=0), INVALID), (dict(n_axes=17), UNSUPPORTED), (dict(axis_stride=-1), INVALID), (dict(positions=None), INVALID),
    (dict(slots=None), INVALID), (dict(q_out=None), INVALID), (dict(inv_freq=None), INVALID), (dict(pair_axis=None), INVALID),
    (dict(pair_axis=F + 2), INVALID), (dict(positions=F + 1), INVALID), (dict(qkv=F + 8), INVALID), (dict(q_out=F + 8), INVALID),
    (dict(h_q=1 << 24, row_stride=1 << 40), UNSUPPORTED)]


@pytest.mark.parametrize("kw,want", ROPE_CASES + [(dict(k_cache=None), INVALID), (dict(v_cache=F + 8), INVALID)])
def test_mrope_refusals(lib, kw, want):
    assert lib.moe_qk_norm_mrope(*changed(ROPE, **kw)) == want


@pytest.mark.parametrize("kw,want", ROPE_CASES + [(dict(kv4_cache=None), INVALID), (dict(kv4_cache=F + 8), INVALID)])
def test_rope_kv4_refusals(lib, kw, want):
    assert lib.moe_qk_norm_rope_kv4(*changed(ROPE4, **kw)) == want


DECODE = dict(q=F, kv4_cache=F, block_table=F, seq_lens=F, B=4, h_q=16, h_kv=2, d=128, num_pages=64, page_size=16, max_pages=8,
              scale=0.1, window=0, n_sink=0, out=F, workspace=F, ws_bytes=WS, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), OK), (dict(B=-1), INVALID), (dict(B=2049), UNSUPPORTED), (dict(h_q=15), INVALID), (dict(h_q=34), UNSUPPORTED),
    (dict(d=64), UNSUPPORTED), (dict(num_pages=0), INVALID), (dict(page_size=24), INVALID), (dict(page_size=2048), INVALID),
    (dict(max_pages=0), INVALID), (dict(max_pages=1 << 27), UNSUPPORTED), (dict(scale=float("nan")), INVALID),
    (dict(window=-1), INVALID), (dict(n_sink=-1), INVALID), (dict(q=None), INVALID), (dict(kv4_cache=None), INVALID),
    (dict(kv4_cache=F + 8), INVALID), (dict(block_table=None), INVALID), (dict(seq_lens=F + 2), INVALID), (dict(out=F + 8), INVALID),
    (dict(workspace=F + 128), INVALID), (dict(ws_bytes=4096), WORKSPACE),
    (dict(B=2048, h_q=64, h_kv=16, max_pages=1 << 20, num_pages=1 << 20), UNSUPPORTED)])
def test_decode_refusals(lib, kw, want):
    assert lib.moe_gqa_kv4_decode(*changed(DECODE, **kw)) == want


LOAD = dict(kv4_cache=F, block_table=F, first=F, seq_lens=F, B=4, h_kv=2, d=128, num_pages=64, page_size=16, max_pages=8, k_cache=F,
            v_cache=F, dst_table=F, dst_pages=64, dst_max_pages=8, workspace=F, ws_bytes=4096, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), OK), (dict(B=-1), INVALID), (dict(B=2049), UNSUPPORTED), (dict(h_kv=0), INVALID), (dict(d=256), UNSUPPORTED),
    (dict(num_pages=0), INVALID), (dict(page_size=100), INVALID), (dict(max_pages=0), INVALID), (dict(dst_pages=0), INVALID),
    (dict(dst_max_pages=0), INVALID), (dict(kv4_cache=None), INVALID), (dict(block_table=None), INVALID),
    (dict(seq_lens=None), INVALID), (dict(k_cache=None), INVALID), (dict(v_cache=F + 8), INVALID), (dict(dst_table=None), INVALID),
    (dict(first=F + 2), INVALID), (dict(workspace=None), INVALID), (dict(workspace=F + 64), INVALID), (dict(ws_bytes=4095), WORKSPACE),
    (dict(B=2048, h_kv=64, max_pages=1 << 14), UNSUPPORTED), (dict(B=2048, h_kv=64, dst_max_pages=1 << 14), UNSUPPORTED)])
def test_load_refusals(lib, kw, want):
    assert lib.moe_kv4_load(*changed(LOAD, **kw)) == want


def test_binding_refusals():
    """The binding's checks raise before the library is called (tensors on the CPU, wrong shapes and types)."""
    moe_build.build()
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    ints = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="residual must be on a CUDA device"):
        moe.moe_add_rms_norm(None, bf(2, 128), None, 1e-6, None, bf(2, 128))
    with pytest.raises(TypeError, match="residual must be a tensor"):
        moe.moe_add_rms_norm(None, None, None, 1e-6, None, bf(2, 128))
    with pytest.raises(ValueError, match="residual must have 2 dimensions"):
        moe.moe_add_rms_norm(None, bf(128), None, 1e-6, None, bf(128))
    with pytest.raises(TypeError, match="residual has the wrong type"):
        moe.moe_add_rms_norm(None, torch.zeros(2, 128), None, 1e-6, None, bf(2, 128))
    raw = torch.zeros(4, 2, 1, 2304, dtype=torch.uint8)
    ws = torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(ValueError, match="q must be on a CUDA device"):
        moe.moe_gqa_kv4_decode(bf(1, 4, 128), raw, ints(1, 2), ints(1), 0.1, bf(1, 4, 128), ws)
    with pytest.raises(ValueError, match="kv4_cache must be on a CUDA device"):
        moe.moe_kv4_load(raw, ints(1, 2), None, ints(1), bf(4, 2, 16, 128), bf(4, 2, 16, 128), ints(1, 2), ws)
    for shape in ((4, 2, 1, 2304, 1), (4, 2, 2304)):
        with pytest.raises(ValueError, match="kv4_cache must have 4 dimensions"):
            moe.moe_kv4_load(torch.zeros(shape, dtype=torch.uint8), ints(1, 2), None, ints(1), bf(4, 2, 16, 128), bf(4, 2, 16, 128),
                             ints(1, 2), ws)
    with pytest.raises(TypeError, match="qkv must be a bf16 CUDA tensor"):
        moe.moe_qk_norm_rope_kv4(bf(3, 768), None, None, 0.0, None, None, ints(3), ints(3), bf(3, 2, 128), raw)
    with pytest.raises(TypeError, match="q_out must be a tensor|qkv must be"):
        moe.moe_qk_norm_mrope(bf(3, 768), None, None, 0.0, None, None, ints(3), ints(3), None, bf(4, 2, 16, 128), bf(4, 2, 16, 128))
    with pytest.raises(ValueError, match="page_size"):
        moe.alloc_kv4_cache(3, 2, 24, "cpu")
    assert moe.alloc_kv4_cache(3, 2, 64, "cpu").shape == (3, 2, 4, 2304)


# ---------------------------------------------------------------- the plain forms
def test_pack_and_unpack_are_inverse():
    c = torch.randint(-8, 8, (50, 128), generator=torch.Generator().manual_seed(0))
    raw = step.pack_rows(c)
    assert raw.shape == (50, 64) and torch.equal(step.unpack_rows(raw).long(), c)
    # word 4 g + w holds dimensions 32 w + 4 g .. + 3, the lowest in the lowest 4 bits
    words = raw.view(torch.uint16).long()
    for g, w in ((0, 0), (3, 2), (7, 3)):
        want = sum((c[:, 32 * w + 4 * g + i] + 8) << 4 * i for i in range(4))
        assert torch.equal(words[:, 4 * g + w], want)


def test_quantise_errs_by_half_a_scale_at_most():
    x = torch.randn(300, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    c, s = step.quantise(x)
    assert c.abs().max() == 7
    err = (c.unflatten(-1, (4, 32)) * s.double()[..., None] - x.double().unflatten(-1, (4, 32))).abs()
    assert (err <= s.double()[..., None] / 2 + 2.0 ** -8 * x.double().abs().unflatten(-1, (4, 32))).all()


def test_int8_codes_and_norm():
    x = torch.randn(5, 256, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    r, y, t, factor = step.add_norm(x, x, None, 1e-6)
    assert torch.equal(r, (2 * x.float()).to(torch.bfloat16))
    assert torch.allclose(y, torch.nn.functional.rms_norm(r.double(), (256,), eps=1e-6))
    q, top = step.int8_codes(t)
    assert q.abs().amax() == 127
    back = q.double().unflatten(-1, (2, 128)) * (top * factor / 127)[..., None]
    assert ((back.flatten(-2) - y).abs() <= (top * factor / 254).repeat_interleave(128, -1) * (1 + 1e-12)).all()


def test_attend_of_one_token():
    g = torch.Generator().manual_seed(3)
    q = torch.randn(4, 128, generator=g).to(torch.bfloat16)
    k, v = (torch.randn(30, 2, 128, generator=g).double() for _ in range(2))
    see = torch.arange(30) % 3 > 0
    out, size, top, _ = step.attend(q, k, v, see, 0.1)
    x = torch.nn.functional.scaled_dot_product_attention(
        q.double()[None, :, None], k[see].permute(1, 0, 2)[None], v[see].permute(1, 0, 2)[None], scale=0.1, enable_gqa=True)
    assert torch.allclose(out, x[0, :, 0]) and (size >= out.abs()).all() and (size >= top / 129).all()
