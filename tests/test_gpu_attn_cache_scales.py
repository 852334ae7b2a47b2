"""Attention over the paged 8-bit cache at scales that make its scores huge, against numpy in 64 bits.

Queries are small whole numbers and keys whole numbers times a power of two, so products are exact, and at these scales a
token of a lower score weighs nothing: a row's result is the average of the values of its highest tokens.

Tolerance, with u = 2^-24: weights, which are equal, and the division take 64 u, sums over L tokens L/4 u of the largest |v|."""
import numpy as np
import pytest
import torch

from tests.gpu_util import DEV
from tests.kv_util import U, Cache, attention
from tests.test_gpu_attn_cache import call

pytestmark = pytest.mark.gpu


def run(scale, n_new, n_q, D, step, q_range=(-8, 8), codes=(-2, 2)):
    lens = [300, 1, 2, 5000]
    c = Cache(lens, 1, D, 16, fill=True)
    c.codes_host[0] = np.random.default_rng(D).integers(codes[0], codes[1] + 1, c.codes_host[0].shape)
    c.scale_host[0] = step
    c.upload()
    q = torch.randint(q_range[0], q_range[1] + 1, (c.B * n_new, n_q * D), generator=torch.Generator().manual_seed(D)).float()
    y = call(c, q.to(DEV), n_new, n_q, scale)
    torch.cuda.synchronize()
    q, y = (x.double().cpu().numpy().reshape(c.B, n_new, n_q, D) for x in (q, y))
    assert np.isfinite(y).all()
    for b, t in enumerate(lens):
        limits = [max(t - n_new + 1 + i, 0) for i in range(n_new)]
        ref, V, _ = attention(q[b], c.rows(b, t, 0), c.rows(b, t, 1), float(np.float32(scale)), limits)
        assert (np.abs(y[b] - ref) <= (t / 4 + 64) * U * V + U * np.abs(ref)).all()


SHAPES = [(1, 4, 64), (3, 8, 64), (1, 3, 128), (2, 10, 80), (1, 4, 256)]


@pytest.mark.parametrize("n_new,n_q,D", SHAPES)
@pytest.mark.parametrize("scale", [1e5, -1e7, 1e10, -1e16, 1e25, 1e31, -1e31, 2e34])
def test_scores_of_any_size(scale, n_new, n_q, D):
    run(scale, n_new, n_q, D, 1.0)


@pytest.mark.parametrize("n_new,n_q,D", SHAPES)
@pytest.mark.parametrize("scale", [2e38, -2e38, 1e37])
def test_scales_near_the_end_of_fp32(scale, n_new, n_q, D):
    """Products of up to 1: the scores are finite."""
    run(scale, n_new, n_q, D, 2.0 ** -12)


@pytest.mark.parametrize("n_new,n_q,D", SHAPES)
@pytest.mark.parametrize("scale", [1e10, 1e31, 2e34])
def test_scores_that_are_all_low(scale, n_new, n_q, D):
    run(scale, n_new, n_q, D, 1.0, (1, 8), (-2, -1))


def test_scores_at_the_lower_end_of_fp32():
    """One token, whose score is -3.2e38 in units of log 2."""
    c = Cache([1], 1, 16, 16, fill=True)
    c.codes_host[0], c.scale_host[0] = 0, 1.0
    c.codes_host[0, ..., 0] = 1
    c.upload()
    q = torch.zeros((1, 16))
    q[0, 0] = -1.125
    y = call(c, q.to(DEV), 1, 1, 1.97e38)
    torch.cuda.synchronize()
    want = c.rows(0, 1, 1)[0, 0]
    assert (np.abs(y.double().cpu().numpy()[0] - want) <= 64 * U * np.abs(want)).all()


@pytest.mark.parametrize("n_new,n_q,D", SHAPES)
def test_queries_below_the_normal_numbers(n_new, n_q, D):
    """Queries of some 1e-39 at a scale of 1e38.  Their products with the keys are as fp32 holds them there: beyond the relative
    errors of (D + 16) u, a block's scale times 2^-126 is off by 2^-150, and a product once more."""
    lens, scale = [300, 1, 40], 1e38
    c = Cache(lens, 1, D, 16, fill=True)
    q = torch.randn((c.B * n_new, n_q * D), generator=torch.Generator().manual_seed(D)) * 2e-39
    y = call(c, q.to(DEV), n_new, n_q, scale)
    torch.cuda.synchronize()
    q, y = (x.double().cpu().numpy().reshape(c.B, n_new, n_q, D) for x in (q, y))
    for b, t in enumerate(lens):
        limits = [max(t - n_new + 1 + i, 0) for i in range(n_new)]
        k = c.rows(b, t, 0)
        ref, V, S = attention(q[b], k, c.rows(b, t, 1), float(np.float32(scale)), limits)
        codes = (np.abs(q[b]) * 2.0 ** 126).sum(-1, keepdims=True) * 128
        E = (D + 16) * U * S + scale * (2.0 ** -150 * codes + 2.0 ** -149)
        assert (np.abs(y[b] - ref) <= (2 * E + (t / 4 + 64) * U) * V + U * np.abs(ref)).all()
