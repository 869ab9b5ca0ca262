"""The README's calls for a prompt over the 4-bit cache, as they stand there, where the context was not all read back before:
after steps of single tokens, into bf16 pages that other layers use in between (needs a GPU)."""
import os
import re

import pytest
import torch

import paged_reference as ref
import routed_expert_ffn_softmax_gb300 as moe
from test_kv4_gpu import D, DEV, SCALE, i32, randn, raw_rows

pytestmark = pytest.mark.gpu
README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from routed_expert_ffn_softmax_gb300 import build
    build.build()
    moe.load()
    yield


def recipe():
    """The read-back and the attention over its rows."""
    with open(README, encoding="utf-8") as f:
        text = f.read()
    calls = re.findall(r"moe\.moe_kv4_load\([^)`]*\)|moe\.moe_gqa_paged_prefill\(q, cu_new, k_pages[^)`]*\)", text)
    assert len(calls) == 2 and calls[0].startswith("moe.moe_kv4_load")
    return calls


@pytest.mark.parametrize("steps", [([40, 1, 100], [1, 1, 1], [1, 1, 1], [3, 30, 20]),     # chunks behind single tokens
                                   ([70, 16, 5], [4, 4, 4], [1, 1, 1], [4, 4, 4])])      # drafted tokens, twice
def test_prompts_behind_single_tokens(steps):
    h_q, h_kv, page, num_pages = 16, 2, 16, 64
    B, width = 3, 16
    ws = moe.alloc_paged_workspace(256, B, h_q, h_kv, D, device=DEV)
    cache = moe.alloc_kv4_cache(num_pages, h_kv, page, DEV).fill_(255)
    block_table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    table = torch.arange(B * width, dtype=torch.int32, device=DEV).view(B, width)
    free, left = torch.randperm(num_pages, generator=torch.Generator().manual_seed(0)).to(torch.int32).to(DEV), i32([num_pages])
    seq_lens = i32([0] * B)
    inv = (1e6 ** (-torch.arange(0, D, 2).double() / D)).float().to(DEV)
    for n_step, new in enumerate(steps):
        N = sum(new)
        qkv = randn(N, (h_q + 2 * h_kv) * D, seed=n_step)
        ctx_lens, cu_new, positions, slots = seq_lens.clone(), i32([0] * (B + 1)), i32([0] * N), i32([0] * N)
        moe.moe_paged_plan(ctx_lens, i32(new), page, num_pages, free, left, block_table, seq_lens, cu_new, positions, slots, left, ws)
        q, out = (torch.empty(N, h_q, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        moe.moe_qk_norm_rope_kv4(qkv, None, None, 0.0, inv, None, positions, slots, q, cache)
        if max(new) == 1:
            moe.moe_gqa_kv4_decode(q, cache, block_table, seq_lens, SCALE, out, ws)
            torch.cuda.synchronize()
            continue
        # other layers' rows stand there
        k_pages, v_pages = (torch.full((B * width, h_kv, page, D), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        names = dict(moe=moe, kv4_cache=cache, block_table=block_table, ctx_lens=ctx_lens, seq_lens=seq_lens, k_pages=k_pages,
                     v_pages=v_pages, table=table, ws=ws, q=q, cu_new=cu_new, scale=SCALE, out=out)
        for call in recipe():
            exec(call, names)
        torch.cuda.synchronize()
        assert moe.workspace_status(ws) == 0
        for b in range(B):
            n, c = int(seq_lens[b]), int(ctx_lens[b])
            at = slice(int(cu_new[b]), int(cu_new[b + 1]))
            rows = [raw_rows(cache, block_table[b], n, i).to(torch.bfloat16) for i in range(2)]
            see = ref.visible(torch.arange(c, n, device=DEV)[:, None], torch.arange(n, device=DEV)[None, :], 0, 0)
            ref.check(out[at], *ref.attend(q[at], *rows, see, SCALE), f"step {n_step} sequence {b}")
