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


def check_weighted(y, c, q, lens, n_new, n_q, scale):
    """As above with each token at its own weight P_j: the first line's V is sum P_j |v_j|, and weights times scales are held
    against a power of two that is at most four times the largest P_j of a row times its block's scale, off by 2^-32 of it
    each, with codes of up to 2^7: L 2^-23 of that largest one.  A weight below 2^-126 of the largest may count as 0."""
    q = q.double().numpy().reshape(c.B, n_new, n_q, c.D)
    y = y.double().cpu().numpy().reshape(c.B, n_new, n_q, c.D)
    assert np.isfinite(y).all()
    scale = float(np.float32(scale))
    for b, t in enumerate(lens):
        k, v = c.rows(b, t, 0), c.rows(b, t, 1)
        i = np.arange(t)
        vs = c.scale_host[1][c.table_host[b, i // c.page]].astype(np.float64)  # [t][n_kv]
        for n in range(n_new):
            L = max(t - n_new + 1 + n, 0)
            for h in range(n_q if L else 0):
                kv = h // (n_q // c.n_kv)
                s = k[:L, kv] @ q[b, n, h] * scale
                P = np.exp(s - s.max())
                P /= P.sum()
                S = (np.abs(k[:L, kv]) @ np.abs(q[b, n, h])).max() * abs(scale)
                ref, V = P @ v[:L, kv], P @ np.abs(v[:L, kv])
                tol = (2 * (c.D + 16) * U * S + (L / 4 + 64) * U) * V + L * 2.0 ** -23 * (P * vs[:L, kv]).max()
                tol = tol + U * np.abs(ref) + L * 2.0 ** -144 + 2.0 ** -125 * np.abs(v[:L, kv]).sum(0)
                bad = np.abs(y[b, n, h] - ref) > tol
                assert not bad.any(), (b, n, h, np.abs(y[b, n, h] - ref)[bad].max(), tol[bad].max(), ref[bad][:3])


@pytest.mark.parametrize("n_q,D", [(4, 64), (14, 64), (8, 128), (20, 128), (4, 256)])
@pytest.mark.parametrize("large", [2.0 ** 24, 1e12, 1e30])
def test_a_large_block_that_only_the_last_token_sees(large, n_q, D):
    """Drafts: the second one begins a page of large values, in the unit of the tokens that the first one sees."""
    lens = [17, 33, 16 * 7 + 1]
    c = Cache(lens, 1, D, 16, fill=True)
    for b, t in enumerate(lens):
        c.scale_host[1, c.table_host[b, (t - 1) // 16]] *= np.float32(large)
    c.upload()
    q = torch.randn((c.B * 2, n_q * D), generator=torch.Generator().manual_seed(D))
    y = call(c, q.to(DEV), 2, n_q, D ** -0.5)
    torch.cuda.synchronize()
    check_weighted(y, c, q, lens, 2, n_q, D ** -0.5)


@pytest.mark.parametrize("n_q,D", [(4, 64), (14, 64), (8, 128), (20, 128), (4, 256)])
@pytest.mark.parametrize("large", [1e12, 1e20, 1e30, 1e36])
@pytest.mark.parametrize("where", [[0], [3], [0, 5, 6]])
def test_a_large_block_that_weighs_next_to_nothing(where, large, n_q, D):
    """Its weights are some e^-55 of the others', so that its values count for nothing at 1e12 and for all at 1e30."""
    t = 16 * 7
    c = Cache([t], 1, D, 16, fill=True)
    c.scale_host[0] = 1.0 / 128
    for i in range(7):
        p = c.table_host[0, i]
        c.codes_host[0, p] = c.codes_host[0, p] // 16 - (110 if i in where else 0)
        c.scale_host[1, p] = 0.01 * (large if i in where else 1.0)
    c.upload()
    q = torch.rand((1, n_q * D), generator=torch.Generator().manual_seed(1)) + 0.5
    scale = 55 / (D * 110 / 128)
    y = call(c, q.to(DEV), 1, n_q, scale)
    torch.cuda.synchronize()
    check_weighted(y, c, q, [t], 1, n_q, scale)


@pytest.mark.parametrize("n_new,n_q,n_kv,D,page", [(1, 4, 1, 64, 16), (3, 6, 2, 128, 16), (2, 16, 1, 128, 32), (1, 8, 4, 256, 16), (5, 4, 1, 32, 64)])
@pytest.mark.parametrize("seed", [0, 1, 2])
def test_value_scales_over_the_whole_range(n_new, n_q, n_kv, D, page, seed):
    """Scales from 1e-42 to 1e36 in any order, zeros among them; long enough for shares and parts, too."""
    lens = [700, 5, 90, 6000]
    c = Cache(lens, n_kv, D, page, seed=seed, fill=True)
    g = np.random.default_rng(seed)
    e = g.integers(-42, 37, c.scale_host[1].shape)
    c.scale_host[1] = np.where(g.random(e.shape) < 0.1, 0.0, 10.0 ** e).astype(np.float32)
    c.upload()
    q = torch.randn((c.B * n_new, n_q * D), generator=torch.Generator().manual_seed(seed)) * 8
    y = call(c, q.to(DEV), n_new, n_q, D ** -0.5)
    torch.cuda.synchronize()
    check_weighted(y, c, q, lens, n_new, n_q, D ** -0.5)
