"""Attention over whole prompts against numpy in 64 bits.

Tolerance, with u = 2^-24, h half a unit of the rows' type relative to a value, S = |scale| * max_j sum_d |q_d k_d| and V = max |v|:
a score is off by (D + 16) u S, a weight relative to the others by twice that; rounding the weights takes h (f16, whose
smallest step is 2^-24: 2^-25 L more), exponential, division and the sums over L keys (64 + L/4) u:
    |y - y64| <= (2 (D + 16) u S + h + (L/4 + 64) u) V, and half a unit of the output."""
import numpy as np
import pytest
import torch

import gemv_quantize_q8_gb300 as kq
from tests.gpu_util import DEV
from tests.kv_util import HALF_UNIT, TYPES, U, attention, ints

pytestmark = pytest.mark.gpu


class Prompt:
    def __init__(self, n_q_tokens, n_k_tokens, Hq, Hk, D, xt, seed=0, amp=1.5, offset=0, pad=0, behind=0):
        g = torch.Generator().manual_seed(seed)
        self.nq, self.nk, self.Hq, self.Hk, self.D, self.xt = n_q_tokens, n_k_tokens, Hq, Hk, D, xt
        self.Tq, self.Tk, self.pad, self.offset, self.behind = sum(n_q_tokens), sum(n_k_tokens), pad, offset, behind
        t = TYPES[xt][1]
        self.q = (torch.randn((self.Tq, Hq, D), generator=g) * amp).to(t)
        self.k, self.v = (torch.randn((self.Tk, Hk, D), generator=g).to(t) for _ in range(2))

    def place(self, x):
        """x's rows in a buffer that starts `offset` elements behind a boundary, `pad` apart, with rows of NaN behind."""
        rows, width = x.shape[0], x.shape[1] * x.shape[2]
        ld = width + self.pad
        buf = torch.full(((rows + self.behind) * ld + 16,), float("nan"), dtype=x.dtype, device=DEV)
        view = buf[self.offset : self.offset + (rows + self.behind) * ld].view(rows + self.behind, ld)
        view[:rows, :width] = x.reshape(rows, width).to(DEV)
        return view, ld

    def call(self, scale, causal, in_place=False, stream=None, ws=None):
        q, ldq = self.place(self.q)
        k, ldk = self.place(self.k)
        v, ldv = self.place(self.v)
        y, ldy = (q, ldq) if in_place else self.place(torch.full_like(self.q, 7.0))
        cu_q, cu_k = (ints(np.concatenate([[0], np.cumsum(n)])) for n in (self.nq, self.nk))
        B, Tq, Tk = len(self.nq), self.Tq + self.behind, self.Tk + self.behind
        n = kq.kq_attn_prompt_workspace_bytes(B, Tq, self.Hq, self.Hk, self.D)
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV) if ws is None else ws
        torch.cuda.synchronize()
        kq.kq_attn_prompt(TYPES[self.xt][0], q, ldq, k, ldk, v, ldv, cu_q, cu_k, B, Tq, Tk, self.Hq, self.Hk, self.D, scale, int(causal), y,
                          ldy, ws, n, stream=stream)
        torch.cuda.synchronize()
        assert kq.kq_read_device_flag(ws) == 0
        width = self.Hq * self.D
        assert bool(y[self.Tq :].isnan().all()) and bool(y[: self.Tq, width:].isnan().all())
        return y[: self.Tq, :width].double().cpu().numpy().reshape(self.Tq, self.Hq, self.D)

    def check(self, y, scale, causal, rows=None):
        q, k, v = (x.double().numpy() for x in (self.q, self.k, self.v))
        at_q = at_k = 0
        h = HALF_UNIT[self.xt]
        g = np.random.default_rng(0)
        for n, L in zip(self.nq, self.nk):
            pick = np.arange(n) if rows is None or n <= rows else np.unique(np.concatenate([[0, n - 1], g.integers(0, n, rows)]))
            limits = [max(L - n + 1 + i, 0) if causal else L for i in pick]
            ref, V, S = attention(q[at_q + pick], k[at_k : at_k + L], v[at_k : at_k + L], float(np.float32(scale)), limits)
            tol = (2 * (self.D + 16) * U * S + h + (L / 4 + 64) * U + (L * 2.0 ** -25 if self.xt == "f16" else 0)) * V
            tol = tol + h * (np.abs(ref) + tol) + 2.0 ** -25
            got = y[at_q + pick]
            assert np.array_equal(np.isnan(got), np.isnan(ref))
            with np.errstate(invalid="ignore"):
                bad = np.abs(got - ref) > tol
            bad &= ~((got == ref) & np.isinf(ref))
            assert not bad.any(), (n, L, np.abs(got - ref)[bad].max(), tol.max(), np.argwhere(bad)[:4])
            at_q, at_k = at_q + n, at_k + L


def run(nq, nk, Hq, Hk, D, xt="bf16", causal=True, rows=None, scale=None, **kw):
    p = Prompt(nq, nk, Hq, Hk, D, xt, **kw)
    scale = D ** -0.5 if scale is None else scale
    y = p.call(scale, causal)
    p.check(y, scale, causal, rows)
    return p, y


SELF = [1, 0, 17, 64, 65, 128, 129, 3, 200]


@pytest.mark.parametrize("D", [8, 40, 64, 80, 96, 128, 136, 256])
@pytest.mark.parametrize("xt", ["f16", "bf16"])
@pytest.mark.parametrize("causal", [True, False])
def test_widths(D, xt, causal):
    run(SELF, SELF, 4, 2, D, xt, causal)


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (5, 5), (14, 2), (8, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_heads(Hq, Hk, D):
    run([130, 31], [130, 31], Hq, Hk, D)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128])
def test_cached_parts_and_empty_rows(causal, D):
    """More keys than queries; fewer (the first rows see nothing); none at all; queries that are not there."""
    run([20, 130, 1, 0, 50, 7, 300], [500, 131, 700, 9, 20, 0, 257], 4, 2, D, "f16", causal)


@pytest.mark.parametrize("D,xt", [(128, "bf16"), (64, "f16"), (80, "bf16")])
def test_long(D, xt):
    run([2500, 700], [2500, 700], 4, 2, D, xt, rows=40)
    run([300], [5000], 2, 1, D, xt, rows=40)


@pytest.mark.parametrize("D", [136, 192, 256])
@pytest.mark.parametrize("xt,causal", [("bf16", True), ("f16", False)])
@pytest.mark.parametrize("offset,pad", [(0, 0), (8, 8), (2, 0), (0, 4)])
def test_wide_heads(D, xt, causal, offset, pad):
    """Rows on 16 bytes and others; tiles that end inside, keys without queries' tiles and the other way round."""
    run([33, 64, 1, 200, 5, 0], [33, 100, 32, 170, 0, 7], 4, 2, D, xt, causal, offset=offset, pad=pad, behind=2)


@pytest.mark.parametrize("offset,pad", [(1, 0), (0, 3), (8, 8), (3, 5), (4, 4)])
@pytest.mark.parametrize("D", [64, 128])
def test_addresses_strides_and_rows_behind(offset, pad, D):
    run([70, 140], [70, 140], 2, 1, D, offset=offset, pad=pad, behind=3)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_in_place(D):
    p, y = run([150, 33], [150, 33], 4, 2, D)
    assert np.array_equal(p.call(D ** -0.5, True, in_place=True), y)


@pytest.mark.parametrize("amp,scale", [(20.0, 1.0), (1.0, 0.0), (5.0, -0.3), (1e-3, 1.0)])
@pytest.mark.parametrize("D", [64, 128])
def test_sizes_of_scores(amp, scale, D):
    run([300], [300], 2, 1, D, amp=amp, scale=scale)


def test_scores_that_rise_and_fall():
    """A maximum that grows with every tile, and one that the first key sets."""
    for order in (1.0, -1.0):
        p = Prompt([400], [400], 2, 1, 128, "bf16")
        p.q[:] = p.q.abs()
        p.k[:] = (torch.linspace(-6, 6, 400)[:, None, None] * order + 0.1 * p.k).to(p.k.dtype)
        for causal in (True, False):
            p.check(p.call(0.1, causal), 0.1, causal)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_what_a_token_does_not_see(D, bad):
    """Values and keys that are not finite reach the tokens that see them, and no others (of their sequence or another)."""
    for at in (0, 100, 131, 180, 299):
        p, _ = run([300, 140], [300, 140], 2, 1, D)
        p.v[at, 0, 3] = bad
        y = p.call(D ** -0.5, True)
        p.check(y, D ** -0.5, True)
        others = np.arange(D) != 3
        assert np.isfinite(y[:at]).all() and np.isfinite(y[300:]).all() and np.isfinite(y[..., others]).all()
        assert not np.isfinite(y[at:300, :, 3]).any()
        p.k[at, 0, 1] = bad
        y = p.call(D ** -0.5, True)
        p.check(y, D ** -0.5, True)
        assert np.isfinite(y[:at]).all() and np.isfinite(y[300:]).all()


def test_queries_that_are_not_finite():
    p, y = run([150], [150], 2, 1, 128)
    p.q[40, 1, 3], p.q[149, 0, 0] = float("nan"), float("inf")
    z = p.call(128 ** -0.5, True)
    hit = np.zeros((150, 2), bool)
    hit[40, 1] = hit[149, 0] = True
    assert np.isnan(z[hit]).all() and np.array_equal(z[~hit], y[~hit])


def test_many_sequences():
    g = np.random.default_rng(1)
    n = g.integers(0, 6, 500).tolist()
    run(n, n, 2, 1, 64)


def test_more_sequences_than_a_warp_finds_in_two_steps():
    g = np.random.default_rng(2)
    n = g.integers(0, 4, 2500).tolist()
    run(n, n, 6, 2, 64, "f16")


@pytest.mark.parametrize("offset", [0, 1])
def test_very_many_sequences_of_one_token(offset):
    """A token that sees itself alone gives its value."""
    n = [0 if b % 5 == 3 else 1 for b in range(70000)]
    p = Prompt(n, n, 1, 1, 8, "bf16", offset=offset)
    assert np.array_equal(p.call(0.3, True), p.v.double().numpy())


def test_two_calls_at_once():
    """Two streams, a workspace each; both take their pairs from a line of their own."""
    scale, work = 128 ** -0.5, []
    for seed, tokens in ((1, [1500, 800]), (2, [3000])):
        p = Prompt(tokens, tokens, 8, 2, 128, "bf16", seed=seed)
        q, k, v = (x.reshape(x.shape[0], -1).to(DEV) for x in (p.q, p.k, p.v))
        n = kq.kq_attn_prompt_workspace_bytes(len(tokens), p.Tq, 8, 2, 128)
        work.append((p, q, k, v, ints(np.cumsum([0] + tokens)), torch.zeros_like(q), torch.zeros(n, dtype=torch.uint8, device=DEV), n, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for p, q, k, v, cu, y, ws, n, stream in work:
            kq.kq_attn_prompt(kq.BF16, q, 1024, k, 256, v, 256, cu, cu, len(p.nq), p.Tq, p.Tk, 8, 2, 128, scale, 1, y, 1024, ws, n, stream=stream)
    torch.cuda.synchronize()
    for p, _, _, _, _, y, ws, _, _ in work:
        assert kq.kq_read_device_flag(ws) == 0
        p.check(y.double().cpu().numpy().reshape(p.Tq, 8, 128), scale, True, rows=40)


def test_repeatable_streams_and_graphs():
    p, y = run([500, 77], [500, 77], 4, 2, 128)
    assert np.array_equal(p.call(128 ** -0.5, True, stream=torch.cuda.Stream()), y)
    q, k, v = (x.reshape(x.shape[0], -1).to(DEV) for x in (p.q, p.k, p.v))
    out, cu = torch.zeros_like(q), ints([0, 500, 577])
    n = kq.kq_attn_prompt_workspace_bytes(2, 577, 4, 2, 128)
    ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kq.kq_attn_prompt(kq.BF16, q, 512, k, 256, v, 256, cu, cu, 2, 577, 577, 4, 2, 128, 128 ** -0.5, 1, out, 512, ws, n)
    for split in (500, 0, 311):
        cu.copy_(ints([0, split, 577]))
        graph.replay()
        torch.cuda.synchronize()
        p.nq = p.nk = [split, 577 - split]
        p.check(out.double().cpu().numpy().reshape(577, 4, 128), 128 ** -0.5, True, rows=60)
