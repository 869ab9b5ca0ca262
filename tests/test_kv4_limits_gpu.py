"""Attention over a paged cache held in 4 bits at the edges its header names: the least value scales, NaN scales (needs a GPU)."""
import math

import pytest
import torch

import routed_expert_ffn_softmax_gb300 as moe
import step_reference as step
from test_kv4_gpu import D, DEV, decode

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from routed_expert_ffn_softmax_gb300 import build
    build.build()
    moe.load()
    yield


def one_heavy_key(n, at, weight_log2, h_q, exponent, codes_seed=0):
    """A cache of one sequence of n keys, and queries and a scale under which the key `at` weighs 2^weight_log2 times each other:
    their first codes are 4 and -4 under scales of 1, the queries' first component alone is not 0."""
    c = step.Kv4([n], 1, 64, DEV, seed=codes_seed)
    (kc, ks), (vc, vs) = c.rows[0]
    kc[..., 0] = -4
    kc[at, :, 0] = 4
    vc = vc.abs().clamp(min=1)  # of one sign, so that nothing cancels
    c.rows[0] = [(kc, torch.ones_like(ks)), (vc, torch.full_like(vs, 2.0 ** exponent))]
    c.put(0, slice(0, n), *c.rows[0])
    q = torch.zeros(1, h_q, D, dtype=torch.bfloat16, device=DEV)
    q[..., 0] = 1.0
    return c, q, weight_log2 * math.log(2.0) / 8


@pytest.mark.parametrize("h_q", [4, 16])
@pytest.mark.parametrize("n", [900, 16385])
@pytest.mark.parametrize("exponent", [-80, -79, -70, -61, -60, 0, 60])
def test_light_keys_count_whatever_the_value_scales(exponent, n, h_q):
    """Keys of 2^-12 of the heaviest one's weight are more than it, taken together: their products with value scales of 2^-80,
    the least the header allows, are held as well as those with ordinary ones."""
    for at in (0, n // 2, n - 1):
        c, q, scale = one_heavy_key(n, at, 12.0, h_q, exponent)
        _, out, sees = decode(c, [n], h_q, scale=scale, hide=False, q=q)
        k, v = c.values(0)
        want = step.attend(q[0], k, v * 2.0 ** -exponent, sees[0], scale, c.rows[0][0][1])
        step.check(out[0].double() * 2.0 ** -exponent, *want, n, f"scales 2^{exponent}, heavy key {at}")


@pytest.mark.parametrize("h_q", [4, 16])
def test_values_that_are_all_zero(h_q):
    """Value scales of 0 count as the least where references are concerned: the sums of weights stay finite, the output is 0."""
    n = 30000
    c, q, scale = one_heavy_key(n, 700, 3.0, h_q, 0)
    c.rows[0][1] = (c.rows[0][1][0], torch.zeros_like(c.rows[0][1][1]))
    c.put(0, slice(0, n), *c.rows[0])
    _, out, _ = decode(c, [n], h_q, scale=scale, hide=False, q=q)
    assert not out.any()


@pytest.mark.parametrize("h_q", [4, 16])
@pytest.mark.parametrize("at", [37, 293])
@pytest.mark.parametrize("near", [0, 8, 16, 24, 100, None])
def test_a_nan_scale_of_values_leaves_the_other_dimensions_right(near, at, h_q):
    """Of key `at`, in a warp's first unit or behind others, the first group's value scale is 2^20 times the others', and of a key
    `near` it (in the same or another lane, unit or tile; None: of that key itself) the third group's is NaN. Dimensions 64 .. 95
    are NaN, all others as without it."""
    n = 400
    c = step.Kv4([n], 1, 16, DEV, seed=3)
    k, (vc, vs) = c.rows[0]
    vs = torch.ones_like(vs)
    vs[at, :, 0] = 2.0 ** 20
    c.rows[0] = [k, (vc, vs)]
    bad = vs.clone()
    bad[at if near is None else (at + near + (near == 0)) % n, :, 2] = float("nan")
    c.put(0, slice(0, n), k, (vc, bad))
    q, out, sees = decode(c, [n], h_q, hide=False)
    assert out[0, :, 64:96].isnan().all()
    kv = c.values(0)
    want = step.attend(q[0], *kv, sees[0], D ** -0.5, c.rows[0][0][1])
    live = [w.unflatten(-1, (4, 32))[:, [0, 1, 3]].flatten(1) for w in (out[0].float(), *want)]
    step.check(*live, n, f"NaN near {near}")


def test_a_nan_scale_of_keys_is_its_heads_alone():
    """A NaN scale of a visible key makes the outputs of that key/value head's queries NaN and leaves the others' right."""
    lens = [200, 700]
    c = step.Kv4(lens, 2, 16, DEV, seed=4)
    (kc, ks), v = c.rows[1]
    bad = ks.clone()
    bad[333, 0, 1] = float("nan")
    c.put(1, slice(0, 700), (kc, bad), v)
    q, out, sees = decode(c, lens, 8, hide=False)
    assert out[1, :4].isnan().all()
    for b, heads in ((0, slice(0, 8)), (1, slice(4, 8))):
        want = step.attend(q[b], *c.values(b), sees[b], D ** -0.5, c.rows[b][0][1])
        step.check(out[b, heads], *(w[heads] for w in want), lens[b], f"sequence {b}")
