"""Log probabilities, entropy and top alternatives against numpy in 64 bits.

Tolerance (fp32 arithmetic, u = 2^-24): S and sum e*d are sums of positive (negative) terms, each with a relative error of
a few u plus |d|*u from the rounding of d = x - m, added in chains of at most V/256 + 128 terms: relative error
(V/256 + 160)*u, times the mean |d| once more for the entropy's second sum.  A log probability adds the rounding of d."""
import numpy as np
import pytest
import torch

import gemv_quantize_q8_gb300 as kq
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"f32": (kq.F32, torch.float32), "f16": (kq.F16, torch.float16), "bf16": (kq.BF16, torch.bfloat16)}


def reference(x, t, k):
    """x: fp64 [M][V]."""
    M, V = x.shape
    out = {"lp": np.empty((M, t.shape[1])), "ent": np.empty(M), "ids": np.empty((M, k), np.int64), "top": np.empty((M, k)),
           "scale": np.empty(M)}
    for r in range(M):
        row = x[r]
        rank = np.where(np.isnan(row), -np.inf, row)
        ids = np.lexsort((np.arange(V), -rank))[:k]
        bad = np.isnan(row).any() or (row == np.inf).any()
        m = rank.max()
        if bad:
            lps, ent, mean = np.full(V, np.nan), np.nan, 0.0
        elif m == -np.inf:
            lps, ent, mean = np.full(V, -np.inf), 0.0, 0.0
        else:
            with np.errstate(all="ignore"):
                d = row - m
                e = np.exp(d)
                S = e.sum()
                lps = d - np.log(S)
                mean = (e[e > 0] * -d[e > 0]).sum() / S
                ent = np.log(S) + mean
        out["lp"][r] = [0.0 if j < 0 else np.nan if j >= V else lps[j] for j in t[r]]
        out["ent"][r], out["ids"][r], out["top"][r], out["scale"][r] = ent, ids, lps[ids], 1 + mean
    return out


def check(x, t, k, xt, offset=0, pad=0):
    M, V = x.shape
    T = t.shape[1]
    ld = V + pad
    buf = torch.full((M * ld + 8,), 3e4, dtype=TYPES[xt][1], device=DEV)
    buf[offset : offset + M * ld].view(M, ld)[:, :V] = x.to(DEV)
    view = buf[offset : offset + M * ld]
    lp, ent = torch.full((M, max(T, 1)), 7.0, device=DEV), torch.full((M,), 7.0, device=DEV)
    ids, top = torch.full((M, max(k, 1)), -7, dtype=torch.int32, device=DEV), torch.full((M, max(k, 1)), 7.0, device=DEV)
    dt = torch.from_numpy(t.astype(np.int32)).to(DEV)
    kq.kq_logprobs(TYPES[xt][0], view, ld, M, V, dt if T else None, T, lp if T else None, ent, k, ids if k else None,
                   top if k else None)
    torch.cuda.synchronize()
    want = reference(x.double().numpy(), t, k)
    rel = (V / 256 + 160) * U

    def near(got, ref, slack):
        got, ref = got.double().cpu().numpy(), np.asarray(ref)
        fine = np.isfinite(ref)
        assert np.array_equal(got[~fine], ref[~fine], equal_nan=True), (got[~fine], ref[~fine])
        off = np.abs(got[fine] - ref[fine])
        tol = np.broadcast_to(slack, ref.shape)[fine] + 4 * U * np.abs(ref[fine])
        assert (off <= tol).all(), (off.max(), tol[off.argmax()])

    scale = want["scale"]
    if T:
        near(lp, want["lp"], rel * scale[:, None])
    near(ent, want["ent"], 2 * rel * scale)
    if k:
        assert np.array_equal(ids.cpu().numpy(), want["ids"])
        near(top, want["top"], rel * scale[:, None])


def logits(g, M, V, xt, spread=2.5):
    return torch.from_numpy((g.standard_normal((M, V)) * spread).astype(np.float32)).to(TYPES[xt][1])


@pytest.mark.parametrize("M,V,T,k", [(1, 1, 1, 1), (1, 2, 1, 2), (2, 31, 3, 31), (3, 33, 1, 32), (1, 1000, 0, 5), (5, 4097, 2, 0),
                                     (1, 65536, 1, 5), (2, 131072, 1, 20), (40, 49999, 3, 8), (300, 5003, 1, 32), (700, 257, 1, 1)])
@pytest.mark.parametrize("xt", list(TYPES))
def test_against_64_bits(M, V, T, k, xt):
    g = np.random.default_rng(V + M)
    check(logits(g, M, V, xt), g.integers(0, V, (M, T)), k, xt, offset=V % 3, pad=M % 5)


@pytest.mark.parametrize("order", ["rising", "falling", "equal", "two values", "one far above"])
@pytest.mark.parametrize("V", [7, 300, 20001])
def test_orders_that_are_hard_for_a_selection(order, V):
    """Rows whose every element is a new best, or the same: all of them are candidates for the alternatives."""
    g = np.random.default_rng(3)
    base = {"rising": np.linspace(-8, 8, V), "falling": np.linspace(8, -8, V), "equal": np.full(V, 1.5),
            "two values": (np.arange(V) % 2) * 1.0, "one far above": np.where(np.arange(V) == V // 2, 60.0, 0.0)}[order]
    x = torch.from_numpy(np.stack([base, base[::-1].copy()]).astype(np.float32))
    for xt in ("f32", "bf16"):
        check(x.to(TYPES[xt][1]), g.integers(0, V, (2, 2)), min(V, 32), xt)


@pytest.mark.parametrize("M", [1, 200])
@pytest.mark.parametrize("xt", list(TYPES))
def test_masks(M, xt):
    """-inf in most places, in all but one, in all; the type's lowest value in the same; and rows of a single token."""
    g = np.random.default_rng(9)
    V = 3001
    x = logits(g, M * 6, V, xt)
    lowest = torch.finfo(TYPES[xt][1]).min
    mask = torch.from_numpy(g.random((M * 6, V)) < 0.99)
    kind = torch.arange(M * 6) % 6
    x = torch.where(mask & (kind == 0)[:, None], torch.tensor(float("-inf"), dtype=x.dtype), x)
    x = torch.where(mask & (kind == 1)[:, None], torch.tensor(lowest, dtype=x.dtype), x)
    x[kind == 2] = float("-inf")
    x[kind == 3] = float("-inf")
    x[kind == 3, V - 1] = 3.0
    x[kind == 4] = lowest
    x[kind == 5, : V - 2] = lowest
    check(x, g.integers(0, V, (M * 6, 2)), 20, xt)


@pytest.mark.parametrize("M", [1, 150])
def test_nan_and_infinity(M):
    g = np.random.default_rng(4)
    V = 5000
    x = logits(g, M * 4, V, "f32")
    kind = torch.arange(M * 4) % 4
    x[kind == 0, 17] = float("nan")
    x[kind == 1, V - 1] = float("inf")
    x[kind == 2, 3] = float("nan")
    x[kind == 2, 4:] = float("-inf")
    check(x, g.integers(0, V, (M * 4, 1)), 8, "f32")


def test_targets_that_are_no_tokens():
    g = np.random.default_rng(4)
    check(logits(g, 5, 100, "f32"), np.array([[-1, 0], [100, 99], [-2 ** 31, 5], [2 ** 31 - 1, 3], [7, 7]]), 0, "f32")


def test_large_values():
    """Logits of hundreds: the exponents' range, not their rounding, is what can go wrong."""
    g = np.random.default_rng(4)
    check(logits(g, 4, 2000, "f32", 300.0), g.integers(0, 2000, (4, 2)), 10, "f32")
    check(logits(g, 4, 2000, "f32", 1e37), g.integers(0, 2000, (4, 2)), 10, "f32")


def test_rows_of_many_rounds():
    """More rounds of a block over its row than the 32 bits that remember where the alternatives are."""
    M, V, k = 400, 270001, 20
    g = torch.Generator(device=DEV)
    g.manual_seed(0)
    x = (torch.randn((M, V), generator=g, device=DEV) * 2.5).to(torch.bfloat16)
    ent, ids, top = torch.empty(M, device=DEV), torch.empty((M, k), dtype=torch.int32, device=DEV), torch.empty((M, k), device=DEV)
    kq.kq_logprobs(kq.BF16, x, V, M, V, None, 0, None, ent, k, ids, top)
    for r in (0, 199, 399):
        want = reference(x[r : r + 1].double().cpu().numpy(), np.zeros((1, 0), int), k)
        assert np.array_equal(ids[r].cpu().numpy(), want["ids"][0])
        assert abs(ent[r].item() - want["ent"][0]) <= 2 * (V / 256 + 160) * U * want["scale"][0]
        assert np.abs(top[r].cpu().numpy() - want["top"][0]).max() <= (V / 256 + 160) * U * want["scale"][0]


def test_offsets_past_32_bits():
    M, V, ld = 3, 1000, 1_100_000_000
    g = np.random.default_rng(2)
    x = logits(g, M, V, "bf16")
    buf = torch.empty(M * ld, dtype=torch.bfloat16, device=DEV)
    buf.view(M, ld)[:, :V] = x.to(DEV)
    ent, ids, top = torch.empty(M, device=DEV), torch.empty((M, 4), dtype=torch.int32, device=DEV), torch.empty((M, 4), device=DEV)
    kq.kq_logprobs(kq.BF16, buf, ld, M, V, None, 0, None, ent, 4, ids, top)
    want = reference(x.double().numpy(), np.zeros((M, 0), int), 4)
    assert np.array_equal(ids.cpu().numpy(), want["ids"])
    assert np.allclose(ent.cpu().numpy(), want["ent"], rtol=0, atol=1e-4)


def test_again_gives_the_same_bits():
    g = np.random.default_rng(2)
    for M, V in ((1, 100003), (64, 30000), (2000, 999)):
        x = logits(g, M, V, "f32").to(DEV)
        outs = []
        for _ in range(3):
            ent, top = torch.empty(M, device=DEV), torch.empty((M, 5), device=DEV)
            kq.kq_logprobs(kq.F32, x, V, M, V, None, 0, None, ent, 5, torch.empty((M, 5), dtype=torch.int32, device=DEV), top)
            outs.append((ent.cpu(), top.cpu()))
        for e, t in outs[1:]:
            assert torch.equal(e, outs[0][0]) and torch.equal(t, outs[0][1])


@pytest.mark.parametrize("M", [2, 330])
@pytest.mark.parametrize("left", [0, 1, 19])
def test_few_tokens_left_and_many_targets(M, left):
    """Rows with fewer unmasked tokens than alternatives, whose list is filled up while the block's other warps still look
    targets up: several rounds of them for some warps, one fewer for others."""
    V, k, T = 5003, 20, 700
    g = np.random.default_rng(left)
    x = torch.full((M, V), float("-inf"))
    for r in range(M):
        x[r, torch.from_numpy(g.permutation(V)[:left])] = torch.from_numpy(g.standard_normal(left).astype(np.float32))
    x[0, 5] = float("nan")
    check(x, g.integers(0, V, (M, T)), k, "f32")


@pytest.mark.parametrize("k", [0, 3])
def test_more_rows_than_a_grid_holds(k):
    """Rows past the grid's 65535 come in a launch of their own, with their own targets and outputs."""
    M, V = 65541, 40
    g = np.random.default_rng(6)
    check(logits(g, M, V, "f32"), g.integers(0, V, (M, 2)), k, "f32")


def test_as_many_targets_as_tokens():
    """Every id of the vocabulary as a target of every row: the most that a call takes."""
    V = 700
    g = np.random.default_rng(8)
    check(logits(g, 3, V, "f32"), np.stack([g.permutation(V) for _ in range(3)]), 5, "f32")
