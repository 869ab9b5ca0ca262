"""Failure detection in the waits of attention over the 4-bit cache: a producer that stops leaves the working warps without
tiles. Their waits and those of the warps that finish pieces run out (status 1 or 2; never 3, because copies under way are
waited for), each warp's once, and the kernel returns with the GPU usable: after the workspace is zeroed a normal call
matches the 64-bit result."""
import pytest
import torch

import routed_expert_ffn_softmax_gb300 as moe
from routed_expert_ffn_softmax_gb300 import build

DEV = "cuda:0"
D = 128
LIMIT_MS = 2100.0  # the longest that one wait takes to give up


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    moe.load()
    yield
    moe.moe_test_paged_give_up()


@pytest.mark.gpu
@pytest.mark.parametrize("tile", [0, 3, 17])
@pytest.mark.parametrize("h_q", [32, 64])
def test_producers_that_stop_end_the_call_within_a_few_limits(tile, h_q):
    """255 sequences of 300 keys with 4 key/value heads: some 20 tiles and 7 pieces a CTA, two of them cut, each with masked
    keys in its last tile. The working warps' waits run out a limit after the start, the finishing warps' with them or after."""
    from test_kv4_gpu import check_decode, decode, i32
    import step_reference as step
    B, h_kv = 255, 4
    pages = B * 5
    raw = torch.randint(0, 256, (pages, h_kv, 4, step.BLOCK_BYTES), dtype=torch.uint8, device=DEV)
    for at in (1024, 2176):
        raw[..., at:at + 128] = torch.full((64,), 0.5, dtype=torch.bfloat16, device=DEV).view(torch.uint8)
    q = torch.randn(B, h_q, D, device=DEV).to(torch.bfloat16)
    table, lens, out = i32(list(range(pages))).view(B, 5), i32([300] * B), torch.empty_like(q)
    ws = moe.alloc_paged_workspace(B, B, h_q, h_kv, D, device=DEV)
    call = lambda: moe.moe_gqa_kv4_decode(q, raw, table, lens, D ** -0.5, out, ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    assert moe.workspace_status(ws) == 0
    ends = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    moe.moe_test_paged_give_up(tile)
    try:
        ends[0].record()
        call()
        ends[1].record()
        torch.cuda.synchronize()
    finally:
        moe.moe_test_paged_give_up()
    ms = ends[0].elapsed_time(ends[1])
    assert ms < 3 * LIMIT_MS, f"{ms:.1f} ms"
    status = moe.workspace_status(ws)
    assert status in (1, 2), f"expected a wait timeout (1 or 2), got {status}"
    ws.zero_()
    some = [300, 17, 0, 1000]
    for window, n_sink in ((100, 3), (0, 0)):
        c = step.Kv4(some, h_kv, 16, DEV)
        check_decode(c, some, *decode(c, some, h_q, window=window, n_sink=n_sink, ws=ws))
