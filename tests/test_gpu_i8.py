"""The int8 products with scales per token and per channel, against whole-number sums in 64 bits.

The sum is exact and every later operation is one rounding of fp32, so the results are compared bit for bit."""
import numpy as np
import pytest
import torch

import gemv_quantize_q8_gb300 as kq
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu

TYPES = {"f32": (kq.F32, torch.float32), "f16": (kq.F16, torch.float16), "bf16": (kq.BF16, torch.bfloat16)}


def up16(k):
    return (k + 15) // 16 * 16


def codes(g, rows, K, pad=0, full=False):
    """Rows of int8 codes whose row ends hold bytes that must not count; full: also -128, the type's lowest."""
    a = g.integers(-128 if full else -127, 128, size=(rows, up16(K) + pad), dtype=np.int16).astype(np.int8)
    return a


def reference(q, sx, w, sw, bias, K, yt):
    """Exact sums, then one fp32 rounding for each operation of the definition."""
    acc = q[:, :K].astype(np.float64) @ w[:, :K].astype(np.float64).T   # below 2^53: exact
    with np.errstate(all="ignore"):
        y = (acc.astype(np.float32) * sx[:, None].astype(np.float32)) * sw[None].astype(np.float32)
        if bias is not None:
            y = y + bias[None].astype(np.float32)
    return torch.from_numpy(y).to(TYPES[yt][1])


def product(q, sx, w, sw, bias, K, yt, ldy_pad=0, stream=None):
    M, N = q.shape[0], w.shape[0]
    d = lambda a: None if a is None else torch.from_numpy(a).to(DEV)  # noqa: E731
    dq, dsx, dw, dsw, db = d(q), d(sx), d(w), d(sw), d(bias)
    y = torch.full((M, N + ldy_pad), 7.0, dtype=TYPES[yt][1], device=DEV)
    n = kq.kq_gemm_i8_workspace_bytes(M, N, K)
    ws = torch.full((n,), 0xAB, dtype=torch.uint8, device=DEV)
    kq.kq_gemm_i8(dq, q.shape[1], dsx, dw, w.shape[1], dsw, db, M, N, K, TYPES[yt][0], y, N + ldy_pad, ws, n)
    torch.cuda.synchronize()
    assert kq.kq_read_device_flag(ws) == 0
    y = y.cpu()
    assert bool((y[:, N:] == 7).all()), "written past the row"
    return y[:, :N]


def same(a, b):
    a, b = a.float().numpy(), b.float().numpy()
    ok = (a == b) | (np.isnan(a) & np.isnan(b))
    assert ok.all(), f"{(~ok).sum()} of {ok.size} differ, first at {np.argwhere(~ok)[0]}: {a[~ok][0]} for {b[~ok][0]}"


SHAPES = [(1, 1, 1), (1, 300, 17), (1, 1000, 2560), (2, 129, 4096), (3, 64, 100), (4, 17, 31), (5, 257, 1025), (7, 640, 513),
          (8, 96, 14336), (9, 1, 16), (9, 130, 1000), (13, 4099, 260), (16, 128, 1024), (17, 127, 1025), (31, 300, 4096),
          (33, 513, 2049), (64, 256, 64), (65, 255, 1040), (100, 1000, 333), (127, 129, 3000), (128, 128, 128), (129, 600, 1024),
          (200, 2560, 1500), (255, 384, 4111), (256, 512, 2048), (257, 257, 257), (300, 4096, 700), (777, 1030, 1030)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("yt", ["f32", "bf16"])
def test_product(M, N, K, yt):
    g = np.random.default_rng(M * 7919 + N * 31 + K)
    q, w = codes(g, M, K, 16 * (K % 3)), codes(g, N, K, 32 * (N % 2))
    sx, sw = (g.random(M) + 0.1).astype(np.float32) / 100, (g.random(N) + 0.1).astype(np.float32) / 1000
    bias = g.standard_normal(N).astype(np.float32) if (M + N) % 2 else None
    same(product(q, sx, w, sw, bias, K, yt, ldy_pad=K % 4), reference(q, sx, w, sw, bias, K, yt))


@pytest.mark.parametrize("M", [1, 6, 12, 70, 300])
@pytest.mark.parametrize("value", [(127, 127), (-128, -128), (-128, 127)])
def test_largest_sums(M, value):
    """Every code at the type's end: sums far past 2^24 stay exact."""
    K, N = 20000, 200
    q, w = np.full((M, up16(K)), value[0], np.int8), np.full((N, up16(K)), value[1], np.int8)
    q[:, ::7] -= np.sign(value[0])   # odd sums: they show a rounding
    one, ones = np.ones(M, np.float32), np.ones(N, np.float32)
    same(product(q, one, w, ones, None, K, "f32"), reference(q, one, w, ones, None, K, "f32"))


@pytest.mark.parametrize("M", [1, 8, 40, 260])
def test_longest_reduction(M):
    """K = 131071, the last length whose sums fit 32 bits, with every product at its largest."""
    K, N = 131071, 33
    q, w = np.full((M, 131072), -128, np.int8), np.full((N, 131072), -128, np.int8)
    w[::2] = 127
    one, ones = np.ones(M, np.float32), np.ones(N, np.float32)
    same(product(q, one, w, ones, None, K, "f32"), reference(q, one, w, ones, None, K, "f32"))


@pytest.mark.parametrize("yt", ["f16", "bf16", "f32"])
def test_scales_that_are_not_ordinary(yt):
    """Zero, infinite, NaN and subnormal scales, and results past the type's range, follow the formula."""
    g = np.random.default_rng(5)
    for M in (4, 40):
        q, w = codes(g, M, 64), codes(g, 70, 64)
        sx, sw = np.ones(M, np.float32), np.ones(70, np.float32)
        sx[:4] = [0.0, np.inf, np.nan, 1e-40]
        sw[:4] = [0.0, 1e-40, 1e30, -1.0]
        same(product(q, sx, w, sw, None, 64, yt), reference(q, sx, w, sw, None, 64, yt))


@pytest.mark.parametrize("M", [2, 20, 150, 400])
def test_rows_do_not_depend_on_the_batch(M):
    """A row's result is the same alone and in a batch, whatever kernel each size takes."""
    g = np.random.default_rng(M)
    q, w = codes(g, M, 1500), codes(g, 500, 1500)
    sx, sw = g.random(M).astype(np.float32), g.random(500).astype(np.float32)
    whole = product(q, sx, w, sw, None, 1500, "f32")
    for m in (0, M - 1):
        same(product(q[m : m + 1], sx[m : m + 1], w, sw, None, 1500, "f32"), whole[m : m + 1])


def quantise_reference(x):
    """Codes and scales from fp32 rows, one rounding for each operation."""
    x = x.astype(np.float32)
    with np.errstate(all="ignore"):
        amax = np.nanmax(np.where(np.isnan(x), 0, np.abs(x)), 1, keepdims=True).astype(np.float32)
        inv = np.float32(127) / amax
        zero = np.isinf(inv)
        v = x * np.where(zero, np.float32(0), inv).astype(np.float32)
        q = np.where(np.isnan(v), 0, np.rint(v)).astype(np.int8)
        return q, np.where(zero, np.float32(0), amax / np.float32(127))[:, 0]


def rows(g, M, K, xt, special=False):
    x = torch.from_numpy(g.standard_normal((M, K)).astype(np.float32))
    x = torch.where(torch.from_numpy(g.random((M, K)) < 0.01), x * 10, x)
    if special:
        x[0] = 0
        if M > 1:
            x[1, K // 2] = float("nan")
        if M > 2:
            x[2, K - 1] = float("inf")
        if M > 3:
            x[3] *= 1e-38
        if M > 4:
            x[4] = torch.round(x[4] * 3) / 2     # ties
            x[4, 0] = 127
    return x.to(TYPES[xt][1])


@pytest.mark.parametrize("M,K", [(1, 1), (1, 2560), (3, 17), (6, 1000), (8, 14336), (40, 4111), (300, 256), (5, 131071)])
@pytest.mark.parametrize("xt", list(TYPES))
@pytest.mark.parametrize("offset", [0, 1])
def test_quantise(M, K, xt, offset):
    """offset: rows that start on odd elements, which no wide load may read as if aligned."""
    g = np.random.default_rng(K + M)
    x = rows(g, M, K, xt, special=True)
    ld, ldq = K + 3 * offset, up16(K) + 16
    buf = torch.full((M * ld + 8,), 1e30 if xt == "f32" else 6e4, dtype=x.dtype, device=DEV)
    view = buf[offset : offset + M * ld].view(M, ld)
    view[:, :K] = x.to(DEV)
    q = torch.full((M, ldq), 99, dtype=torch.int8, device=DEV)
    s = torch.full((M,), 99.0, device=DEV)
    kq.kq_quantize_i8(TYPES[xt][0], view, M, K, ld, q, ldq, s)
    q, s = q.cpu().numpy(), s.cpu().numpy()
    want_q, want_s = quantise_reference(x.float().numpy())
    assert np.array_equal(q[:, :K], want_q)
    assert np.array_equal(s, want_s)
    assert (q[:, K : up16(K)] == 0).all() and (q[:, up16(K) :] == 99).all()


@pytest.mark.parametrize("M,N,K", [(1, 500, 2560), (1, 64, 1), (2, 100, 333), (5, 4096, 1500), (8, 33, 4096), (11, 300, 1025),
                                   (48, 640, 4096), (130, 513, 2049), (257, 1000, 777), (600, 260, 64)])
@pytest.mark.parametrize("xt,yt", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32")])
def test_dynamic(M, N, K, xt, yt):
    g = np.random.default_rng(M + N + K)
    x = rows(g, M, K, xt, special=M > 8)
    w, sw, bias = codes(g, N, K), g.random(N).astype(np.float32) / 100, g.standard_normal(N).astype(np.float32)
    ld = K + M % 2
    buf = torch.zeros((M, ld), dtype=x.dtype, device=DEV)
    buf[:, :K] = x.to(DEV)
    y = torch.full((M, N), 7.0, dtype=TYPES[yt][1], device=DEV)
    n = kq.kq_gemm_i8_workspace_bytes(M, N, K)
    ws = torch.full((n,), 0xAB, dtype=torch.uint8, device=DEV)
    dw, dsw, db = (torch.from_numpy(a).to(DEV) for a in (w, sw, bias))
    kq.kq_gemm_i8_dyn(TYPES[xt][0], buf, ld, dw, w.shape[1], dsw, db, M, N, K, TYPES[yt][0], y, N, ws, n)
    torch.cuda.synchronize()
    assert kq.kq_read_device_flag(ws) == 0
    q, sx = quantise_reference(x.float().numpy())
    same(y.cpu(), reference(q, sx, w, sw, bias, K, yt))


@pytest.mark.parametrize("M", [2, 100])
def test_offsets_past_32_bits(M):
    """Weights, outputs and their strides past 2^31 elements."""
    g = np.random.default_rng(1)
    N, K, ldw, ldy = 300, 200, 1 << 23, (1 << 31) // M + 512
    q, w = codes(g, M, K), codes(g, N, K)
    big = torch.zeros(N * ldw, dtype=torch.int8, device=DEV)
    big.view(N, ldw)[:, : w.shape[1]] = torch.from_numpy(w).to(DEV)
    y = torch.empty(M * ldy, dtype=torch.float16, device=DEV)
    one, ones = torch.ones(M, device=DEV), torch.full((N,), 1 / 4096, device=DEV)
    n = kq.kq_gemm_i8_workspace_bytes(M, N, K)
    ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
    kq.kq_gemm_i8(torch.from_numpy(q).to(DEV), q.shape[1], one, big, ldw, ones, None, M, N, K, kq.F16, y, ldy, ws, n)
    torch.cuda.synchronize()
    want = reference(q, np.ones(M), w, np.full(N, 1 / 4096), None, K, "f16")
    same(y.view(M, ldy)[:, :N].cpu(), want)


@pytest.mark.parametrize("M", [1, 5, 64, 300])
def test_on_a_stream_of_its_own_and_again(M):
    """Work queued behind other work of a side stream; the same call again gives the same bits."""
    g = np.random.default_rng(M)
    K, N = 2048, 1024
    q, w = torch.from_numpy(codes(g, M, K)).to(DEV), torch.from_numpy(codes(g, N, K)).to(DEV)
    sx, sw = torch.rand(M, device=DEV), torch.rand(N, device=DEV)
    n = kq.kq_gemm_i8_workspace_bytes(M, N, K)
    ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
    ys = [torch.empty((M, N), device=DEV) for _ in range(3)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        later = torch.zeros_like(q)
        torch.cuda._sleep(2_000_000)
        later.copy_(q)
        for y in ys:
            kq.kq_gemm_i8(later, K, sx, w, K, sw, None, M, N, K, kq.F32, y, N, ws, n)
    side.synchronize()
    want = reference(q.cpu().numpy(), sx.cpu().numpy(), w.cpu().numpy(), sw.cpu().numpy(), None, K, "f32")
    for y in ys:
        same(y.cpu(), want)


@pytest.mark.parametrize("M,N,K", [(1, 300, 1000), (3, 129, 2060), (8, 257, 513), (20, 1000, 1025), (60, 300, 4111), (100, 260, 2049),
                                   (300, 777, 1500), (1100, 4099, 1030)])
def test_all_codes_at_random(M, N, K):
    """Codes of -128 to 127, the type's lowest among the others, in random places of both sides."""
    g = np.random.default_rng(M + N + K)
    q, w = codes(g, M, K, full=True), codes(g, N, K, full=True)
    assert (q[:, :K] == -128).any() and (w[:, :K] == -128).any()
    sx, sw = g.random(M).astype(np.float32), g.random(N).astype(np.float32)
    same(product(q, sx, w, sw, None, K, "f32"), reference(q, sx, w, sw, None, K, "f32"))
