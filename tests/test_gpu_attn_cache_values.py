"""Attention over the paged 8-bit cache where the blocks of values differ in size by many orders, against numpy in 64 bits.

Tolerance: that of test_gpu_attn_cache.py, and for blocks of tiny scales what f16's smallest step leaves: weights times
scales are held times at most 2^126, each off by 2^-25 there, and a code is up to 2^7, so L tokens are off by L 2^-144 in all;
an output below 2^-126 is off by half of 2^-149 more."""
import numpy as np
import pytest
import torch

from tests.gpu_util import DEV
from tests.kv_util import U, Cache, attention
from tests.test_gpu_attn_cache import call
from tests.test_gpu_kv_cache import append

pytestmark = pytest.mark.gpu


def check(y, c, q, lens, n_new, n_q, scale):
    q = q.double().numpy().reshape(c.B, n_new, n_q, c.D)
    y = y.double().cpu().numpy().reshape(c.B, n_new, n_q, c.D)
    for b, t in enumerate(lens):
        limits = [max(t - n_new + 1 + i, 0) for i in range(n_new)]
        ref, V, S = attention(q[b], c.rows(b, t, 0), c.rows(b, t, 1), float(np.float32(scale)), limits)
        tol = (2 * (c.D + 16) * U * S + (t / 4 + 64) * U) * V + U * np.abs(ref) + t * 2.0 ** -144 + 2.0 ** -150
        assert np.isfinite(y[b]).all()
        bad = np.abs(y[b] - ref) > tol
        assert not bad.any(), (b, t, np.abs(y[b] - ref)[bad].max(), tol.max())


TINY = [1e-37, 3.7e-37, 3.8e-37, 3e-38, 3e-39, 1e-42, 2.0 ** -149]


@pytest.mark.parametrize("n_new,n_q,D", [(1, 4, 64), (1, 2, 128), (3, 8, 64), (1, 4, 256)])
@pytest.mark.parametrize("tiny", TINY)
def test_tiny_blocks_of_values(tiny, n_new, n_q, D):
    """Such blocks alone, before and behind ordinary ones and beside blocks of zeros."""
    orders = [[tiny] * 5, [tiny] * 4 + [1.0], [1.0] + [tiny] * 4, [0.0, tiny, 0.0, 0.5, tiny], [tiny, 0.0, 0.0, 0.0, 0.0]]
    lens = [16 * 5 - 3] * len(orders)
    c = Cache(lens, 1, D, 16, fill=True)
    for b, scales in enumerate(orders):
        c.scale_host[1, c.table_host[b, :5], 0] = np.float32(scales)
    c.upload()
    q = torch.randn((c.B * n_new, n_q * D), generator=torch.Generator().manual_seed(D)) * 4
    y = call(c, q.to(DEV), n_new, n_q, D ** -0.5)
    torch.cuda.synchronize()
    check(y, c, q, lens, n_new, n_q, D ** -0.5)


@pytest.mark.parametrize("size", [4e-35, 1e-36, 3e-37, 1e-38, 1e-40, 1e-45])
def test_tiny_values_appended(size):
    """A head whose values have decayed, through the append; then tokens of ordinary size."""
    n, D = 60, 64
    c = Cache([n], 1, D, 16)
    x = np.random.default_rng(0).standard_normal((n, 2 * D)).astype(np.float32)
    x[:40, D:] *= np.float32(size)
    q = torch.randn((1, 4 * D), generator=torch.Generator().manual_seed(1))
    for a, b in ((0, 40), (40, 60)):
        append(c, [b - a], [b], x=x[a:b])
        y = call(c, q.to(DEV), 1, 4, D ** -0.5)
        torch.cuda.synchronize()
        check(y, c, q, [b], 1, 4, D ** -0.5)


@pytest.mark.parametrize("n_new,n_q,D", [(1, 4, 64), (1, 2, 128), (3, 8, 64), (1, 4, 256)])
def test_values_near_the_end_of_fp32(n_new, n_q, D):
    """Values of one sign up to 3.3e38: their average is finite, their sum is not."""
    lens = [3, 700, 6000]
    c = Cache(lens, 1, D, 16, fill=True)
    c.codes_host[1] = c.codes_host[1] // 10 + 114
    c.scale_host[1] = 2.6e36
    c.upload()
    q = torch.randn((c.B * n_new, n_q * D), generator=torch.Generator().manual_seed(D))
    y = call(c, q.to(DEV), n_new, n_q, D ** -0.5)
    torch.cuda.synchronize()
    check(y, c, q, lens, n_new, n_q, D ** -0.5)
