"""Attention over the 4-bit cache in every way that its work is shared out and joined, against plain 64-bit forms, and the same bits
every time on one workspace (needs a GPU)."""
import pytest
import torch

import kv4_shapes
import routed_expert_ffn_softmax_gb300 as moe
import step_reference as step
from test_kv4_gpu import D, DEV, SCALE, decode, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from routed_expert_ffn_softmax_gb300 import build
    build.build()
    moe.load()
    yield


def test_every_way_has_a_shape_on_this_gpu():
    grid = torch.cuda.get_device_properties(DEV).multi_processor_count
    assert not kv4_shapes.ways_there_are() - set().union(*(kv4_shapes.ways(s, grid) for s in kv4_shapes.SHAPES))


@pytest.mark.parametrize("s", kv4_shapes.SHAPES, ids=[s["name"].replace(" ", "-") for s in kv4_shapes.SHAPES])
def test_shape(s):
    lens, h_q, h_kv, page = s["lens"], s["h_q"], s["h_kv"], s["page"]
    masks = dict(window=s.get("window", 0), n_sink=s.get("n_sink", 0))
    c = step.Kv4(lens, h_kv, page, DEV, seed=len(s["name"]), codes_lo=-8)
    for i, (b, at) in enumerate(s.get("bad", ())):
        c.table[b, at] = -1 - i if i % 2 else c.raw.shape[0] + i
    ws = moe.alloc_paged_workspace(len(lens), len(lens), h_q, h_kv, D, device=DEV)
    status = 6 if s.get("bad") else 0
    q, out, sees = decode(c, lens, h_q, ws=ws, status=status, **masks)
    for b, n in enumerate(lens):
        k, v = c.values(b)
        for at in [at for seq, at in s.get("bad", ()) if seq == b]:
            k[at * page:(at + 1) * page] = 0
            v[at * page:(at + 1) * page] = 0
        step.check(out[b], *step.attend(q[b], k, v, sees[b], SCALE, c.rows[b][0][1]), max(n, 1), f"sequence {b} of {n}")
    again, n = torch.empty_like(out), i32(lens)
    for _ in range(10):
        again.fill_(float("nan"))
        moe.moe_gqa_kv4_decode(q, c.raw, c.table, n, SCALE, again, ws, **masks)
        assert torch.equal(again, out)
    assert moe.workspace_status(ws) == status and not ws[4:4096].any()
