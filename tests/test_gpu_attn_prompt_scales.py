"""Attention over whole prompts at scales that make its scores huge, against numpy in 64 bits.

Queries and keys are small whole numbers, so scores times 1/scale are exact in every step, and at these scales a key of a
lower score weighs nothing: a row's result is the average of the values of its highest keys.

Tolerance, with u = 2^-24, h half a unit of the rows' type relative to a value and V = max |v|: weights that are equal are
rounded to the type alike (h), sums over L keys and the division take (L/4 + 64) u, the output half a unit:
    |y - y64| <= (h + (L/4 + 64) u) V + h |y64| + 2^-25 (f16's smallest steps)."""
import numpy as np
import pytest
import torch

from tests.kv_util import HALF_UNIT, U, attention
from tests.test_gpu_attn_prompt import Prompt

pytestmark = pytest.mark.gpu


def check(p, y, scale, causal):
    q, k, v = (x.double().numpy() for x in (p.q, p.k, p.v))
    at_q = at_k = 0
    h = HALF_UNIT[p.xt]
    for n, L in zip(p.nq, p.nk):
        limits = [max(L - n + 1 + i, 0) if causal else L for i in range(n)]
        ref, V, _ = attention(q[at_q : at_q + n], k[at_k : at_k + L], v[at_k : at_k + L], float(np.float32(scale)), limits)
        got = y[at_q : at_q + n]
        assert np.isfinite(got).all()
        assert (np.abs(got - ref) <= (h + (L / 4 + 64) * U) * V + h * np.abs(ref) + 2.0 ** -25).all()
        at_q, at_k = at_q + n, at_k + L


def whole_numbers(nq, nk, D, xt, low, high, **kw):
    p = Prompt(nq, nk, 4, 2, D, xt, **kw)
    g = torch.Generator().manual_seed(D)
    for x, (a, b) in ((p.q, low), (p.k, high)):
        x.copy_(torch.randint(a, b + 1, x.shape, generator=g))
    return p


SCALES = [1e3, -1e4, 3e6, 1e8, -1e10, 1e16, -1e25, 1e31, -1e31, 2e35, -2e35]


@pytest.mark.parametrize("D,offset", [(16, 0), (64, 0), (80, 0), (128, 0), (128, 1), (256, 0), (256, 1)])
@pytest.mark.parametrize("scale", SCALES)
def test_scores_of_any_size(D, offset, scale):
    for xt, causal in (("bf16", True), ("f16", False)):
        p = whole_numbers([140, 1, 3], [300, 1, 2], D, xt, (-2, 2), (-2, 2), offset=offset)
        check(p, p.call(scale, causal), scale, causal)


@pytest.mark.parametrize("D,offset", [(64, 0), (128, 0), (128, 1), (256, 0)])
@pytest.mark.parametrize("scale", [1e4, 1e10, 1e31, -1e31])
def test_scores_that_are_all_low(D, offset, scale):
    """Every score far below 0, the first token's only one among them."""
    k = (-2, -1) if scale > 0 else (1, 2)
    p = whole_numbers([150], [150], D, "bf16", (1, 2), k, offset=offset)
    check(p, p.call(scale, True), scale, True)


@pytest.mark.parametrize("D,offset", [(64, 0), (128, 1), (256, 0)])
def test_no_scale_and_products_near_the_end_of_fp32(D, offset):
    """A scale of 0 weighs all keys alike, whatever their products."""
    p = Prompt([40], [200], 4, 2, D, "bf16", offset=offset)
    p.q.mul_(1e18)
    p.k.mul_(1e17)
    check(p, p.call(0.0, True), 0.0, True)
