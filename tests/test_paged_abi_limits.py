"""Size limits that include/paged/moe_paged.h states, at the last size within and the first beyond (no GPU needed: the calls
that pass the size checks are refused for their workspace)."""
import pytest

from test_paged_abi import UNSUPPORTED, WORKSPACE, attn, lib  # noqa: F401


@pytest.mark.parametrize("which", ["decode", "prefill", "prefix"])
@pytest.mark.parametrize("h_q,h_kv", [(64, 4), (24, 8), (16, 16)])
def test_work_is_counted_in_32_bits(lib, which, h_q, h_kv):  # noqa: F811
    """(N / (2 (128 / G)) + B) * h_kv * (keys / 128 + 9) < 2^31 is served, the next power of two of keys is not."""
    B = N = 2048
    blocks = N // (2 * (128 // (h_q // h_kv))) + B
    served = [w for w in range(4, 26) if blocks * h_kv * ((1 << w) * 16 // 128 + 9) < 2 ** 31]
    more = dict(N=N) if which == "prefill" else {}
    call = lambda w: attn(lib, which, B=B, h_q=h_q, h_kv=h_kv, width=1 << w, ws_bytes=4096, **more)  # noqa: E731
    assert served and call(served[-1]) == WORKSPACE
    assert call(served[-1] + 1) == UNSUPPORTED
