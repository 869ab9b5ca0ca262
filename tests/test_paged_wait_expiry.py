"""Failure detection in the attention kernels' own waits over a paged cache: prompts, the prefix a batch shares, one token
per sequence.

Producers that stop in the middle of a piece leave the other roles waiting for tiles that never come. Their waits run out
(status 1 or 2; never 3, because copies and products under way are waited for), each role waits at most once or twice, and
the kernel returns with the GPU usable: after the workspace is zeroed a normal call matches the 64-bit result."""
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


def test_the_hook_refuses_other_values():
    for bad in (-2, -2 ** 31):
        with pytest.raises(moe.MoeError):
            moe.moe_test_paged_give_up(bad)
    moe.moe_test_paged_give_up(0)
    moe.moe_test_paged_give_up()


def long_call(n, shared=False):
    """A call over one prompt of n tokens, or of 2000 queries behind n shared keys, in pages of 128 (random rows, whose result
    is not looked at)."""
    k, v = (torch.randn(-(-n // 128), 2, 128, D, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    q = torch.randn(2000 if shared else n, 16, D, device=DEV, dtype=torch.bfloat16)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    pages, out, scale = i32(list(range(k.shape[0]))), torch.empty_like(q), D ** -0.5
    if shared:
        own, none = i32([[0]] * 2000), i32([0] * 2000)
        return lambda ws: moe.moe_gqa_prefix_decode(q, pages, n, k, v, own, none, scale, out, ws)
    table, lens, cu = pages.view(1, -1), i32([n]), i32([0, n])
    return lambda ws: moe.moe_gqa_paged_prefill(q, cu, k, v, table, lens, scale, out, ws)


def timed(call, ws):
    ends = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    ends[0].record()
    call(ws)
    ends[1].record()
    torch.cuda.synchronize()
    return ends[0].elapsed_time(ends[1])


@pytest.mark.gpu
@pytest.mark.parametrize("shared,tile", [(False, 0), (False, 100), (True, 2)])
def test_producers_that_stop_end_the_call_within_a_few_limits(shared, tile):
    """Prompt: some 430 tiles a CTA, in pieces of up to 128, so that waits for every remaining tile of a piece would take
    minutes. The chain: the issuers' and the softmax's waits run out a limit after the producer stopped, the announcing
    warp's and the issuers' for the next piece another one later."""
    from test_paged_gpu import run_prefill, run_prefix
    call, ws = long_call(16384, shared), moe.alloc_paged_workspace(16384, 2000, 16, 2, D, 16384, device=DEV)
    call(ws)
    torch.cuda.synchronize()
    assert moe.workspace_status(ws) == 0
    moe.moe_test_paged_give_up(tile)
    try:
        ms = timed(call, ws)
    finally:
        moe.moe_test_paged_give_up()
    assert ms < 3 * LIMIT_MS, f"{ms:.1f} ms"
    status = moe.workspace_status(ws)
    assert status in (1, 2), f"expected a wait timeout (1 or 2), got {status}"
    ws.zero_()
    run_prefill((300, 17), (83, 17), 16, 2, 16, ws=ws)
    run_prefix(1000, (5, 0, 300), 16, 2, 16, ws=ws)


@pytest.mark.gpu
@pytest.mark.parametrize("tile", [0, 4])
def test_one_token_producers_that_stop_end_the_call_within_a_few_limits(tile):
    """255 sequences of 300 keys with 4 key/value heads: some 7 pieces a CTA, each with masked keys in its last tile. The
    issuer's and the softmax's waits run out together, the finisher's for the piece's product after them."""
    from test_paged_gpu import i32, run_decode
    B, pages = 255, 255 * 5
    k, v = (torch.randn(pages, 4, 64, D, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    q = torch.randn(B, 32, D, device=DEV, dtype=torch.bfloat16)
    table, lens, out = i32(list(range(pages))).view(B, 5), i32([300] * B), torch.empty_like(q)
    ws = moe.alloc_paged_workspace(B, B, 32, 4, D, device=DEV)
    call = lambda ws: moe.moe_gqa_paged_decode(q, k, v, table, lens, D ** -0.5, out, ws)  # noqa: E731
    call(ws)
    torch.cuda.synchronize()
    assert moe.workspace_status(ws) == 0
    moe.moe_test_paged_give_up(tile)
    try:
        ms = timed(call, ws)
    finally:
        moe.moe_test_paged_give_up()
    assert ms < 3 * LIMIT_MS, f"{ms:.1f} ms"
    status = moe.workspace_status(ws)
    assert status in (1, 2), f"expected a wait timeout (1 or 2), got {status}"
    ws.zero_()
    run_decode((300, 17, 0, 1000), 32, 4, 16, window=100, n_sink=3, ws=ws)
    run_decode((300, 17, 0, 1000), 32, 4, 16, ws=ws)
