"""The residual's norm at the largest number of rows its header allows, on the GPU (needs a GPU)."""
import pytest
import torch

import routed_expert_ffn_softmax_gb300 as moe
from test_norm_gpu import DEV, EPS, check_norm, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from routed_expert_ffn_softmax_gb300 import build
    build.build()
    moe.load()
    yield
    torch.cuda.empty_cache()


def test_norm_of_as_many_rows_as_32_bits_count():
    """2^31 - 1 rows of 8, zeros but for the first and the last: those are normed, the others 0, and what stands around
    the rows is as it was."""
    N, H, some, pad = 2 ** 31 - 1, 8, 5000, 1 << 16
    residual = torch.zeros(N, H, dtype=torch.bfloat16, device=DEV)
    residual[:some], residual[-some:] = randn(some, H), randn(some, H, seed=1)
    around = torch.full((N * H + 2 * pad,), 7.0, dtype=torch.bfloat16, device=DEV)
    y = around[pad:-pad].view(N, H)
    moe.moe_add_rms_norm(None, residual, None, EPS, None, y)
    torch.cuda.synchronize()
    for at in (slice(0, some), slice(N - some, N)):
        check_norm(dict(r=residual[at], y=y[at], q=None, s=None), None, residual[at], None)
    assert (around[:pad] == 7).all() and (around[-pad:] == 7).all()
    for at in range(some, N - some, 1 << 28):
        assert not y[at:min(N - some, at + (1 << 28))].any()
