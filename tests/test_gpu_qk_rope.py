"""Per-head norms of queries and keys with the rotation, against numpy in 64 bits.

Tolerance (u = 2^-24): the sum of squares is off by D*u at most relative, its root by half that, and the norm, the products
with gamma and the rotation's two products and sum add 8u; so an element is off by (D/2 + 8)*u of the magnitudes |a| + |b| of
its pair, and an f16 or bf16 output by half a unit of its last place more."""
import numpy as np
import pytest
import torch

import gemv_quantize_q8_gb300 as kq
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"f32": (kq.F32, torch.float32), "f16": (kq.F16, torch.float16), "bf16": (kq.BF16, torch.bfloat16)}
HALF_UNIT = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}  # 11 and 8 significant bits
N_POS = 100


def tables(rot):
    a = np.arange(N_POS)[:, None] * 1e4 ** (-2 * np.arange(rot // 2) / max(rot, 1))
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def reference(x, gamma, eps, pos, cos, sin, rot, pairs):
    """x: fp64 [M][H][D]; also the magnitude of each element's pair."""
    if gamma is not None:
        x = x / np.sqrt((x ** 2).mean(2, keepdims=True) + eps) * gamma.astype(np.float64)
    y, size = x.copy(), np.abs(x)
    if rot:
        i = np.arange(rot // 2)
        ia, ib = (2 * i, 2 * i + 1) if pairs else (i, i + rot // 2)
        ok = (pos >= 0) & (pos < N_POS)
        c, s = (t.astype(np.float64)[np.where(ok, pos, 0)][:, None] for t in (cos, sin))
        a, b = x[..., ia], x[..., ib]
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        size[..., ia] = size[..., ib] = np.abs(a) + np.abs(b)
        y[~ok] = np.nan
    return y, size


def check(M, Hq, Hk, D, rot, pairs, xt, yt, gamma=True, offset=0, pad=0, in_place=False, pos=None, eps=1e-6, x=None):
    g = np.random.default_rng(M + 10 * Hq + D)
    heads = (Hq, Hk)
    ld = (Hq + Hk) * D + pad
    if x is None:
        x = torch.from_numpy((g.standard_normal((M, ld)) * 2).astype(np.float32)).to(TYPES[xt][1])
    buf = torch.zeros(M * ld + 8, dtype=x.dtype, device=DEV)
    rows = buf[offset : offset + M * ld].view(M, ld)
    rows.copy_(x)
    gq, gk = ((1 + 0.3 * g.standard_normal(D)).astype(np.float32) if gamma else None for _ in range(2))
    cos, sin = tables(rot)
    pos = g.integers(0, N_POS, M) if pos is None else pos
    d = lambda a: None if a is None else torch.from_numpy(a).to(DEV)  # noqa: E731
    outs = []
    for h, H in enumerate(heads):
        if in_place:
            outs.append(rows[:, h * Hq * D : h * Hq * D + H * D])
        else:
            outs.append(torch.full((M * (H * D + pad) + 8,), 7.0, dtype=TYPES[yt][1], device=DEV)[offset : offset + M * (H * D + pad)]
                        .view(M, H * D + pad)[:, : H * D])
    dgq, dgk, dpos, dcos, dsin = d(gq), d(gk), d(pos.astype(np.int32)), d(cos), d(sin)
    lds = [ld, ld] if in_place else [Hq * D + pad, Hk * D + pad]
    kq.kq_qk_norm_rope(TYPES[xt][0], rows if Hq else None, ld, rows[:, Hq * D :] if Hk else None, ld, M, Hq, Hk, D, dgq, dgk, eps,
                       dpos if rot else None, dcos if rot else None, dsin if rot else None, N_POS, rot, int(pairs), TYPES[yt][0],
                       outs[0] if Hq else None, lds[0], outs[1] if Hk else None, lds[1])
    torch.cuda.synchronize()
    xs = x.double().numpy()
    at = 0
    for H, gamma_h, out in zip(heads, (gq, gk), outs):
        if H:
            ref, size = reference(xs[:, at : at + H * D].reshape(M, H, D), gamma_h, np.float64(np.float32(eps)), pos, cos, sin, rot, pairs)
            got = out.double().cpu().numpy().reshape(M, H, D)
            fine = np.isfinite(ref)
            assert np.array_equal(np.isnan(got), np.isnan(ref))
            off = np.abs(got - ref)[fine]
            tol = ((D / 2 + 8) * U * size + HALF_UNIT[yt] * (np.abs(ref) + (D / 2 + 8) * U * size) + (2.0 ** -25 if yt == "f16" else 0))[fine]
            assert (off <= tol).all(), (off.max(), tol[(off - tol).argmax()])
        at += H * D
    return outs


@pytest.mark.parametrize("M,Hq,Hk,D,rot", [(1, 1, 1, 2, 2), (1, 32, 8, 128, 128), (3, 14, 2, 80, 40), (7, 5, 1, 96, 96), (33, 8, 8, 64, 64),
                                           (129, 28, 4, 128, 64), (2, 3, 3, 256, 256), (5, 2, 1, 1024, 512), (9, 3, 1, 6, 4),
                                           (4, 2, 2, 72, 36), (17, 0, 3, 128, 128), (17, 3, 0, 64, 0), (1000, 7, 1, 112, 112)])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("xt,yt", [("f32", "bf16"), ("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("bf16", "f32")])
def test_against_64_bits(M, Hq, Hk, D, rot, pairs, xt, yt):
    check(M, Hq, Hk, D, rot, pairs, xt, yt)


@pytest.mark.parametrize("D,rot", [(128, 128), (80, 40), (64, 62), (128, 6)])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("offset,pad", [(1, 0), (0, 1), (2, 3), (4, 8)])
def test_strides_and_odd_starts(D, rot, pairs, offset, pad):
    for xt, yt in (("f32", "f16"), ("bf16", "bf16")):
        check(11, 3, 2, D, rot, pairs, xt, yt, offset=offset, pad=pad)


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("D,rot", [(128, 128), (80, 40), (10, 6)])
def test_in_place(pairs, D, rot):
    check(50, 6, 2, D, rot, pairs, "bf16", "bf16", in_place=True)
    check(50, 6, 2, D, rot, pairs, "f32", "f32", in_place=True)


def test_without_norm():
    check(20, 4, 2, 128, 128, False, "f32", "f32", gamma=False)
    check(20, 4, 2, 128, 64, True, "f16", "f32", gamma=False)


@pytest.mark.parametrize("D", [128, 80])
def test_positions_outside_the_table(D):
    check(6, 4, 1, D, D, False, "f32", "bf16", pos=np.array([0, -1, N_POS - 1, N_POS, 2 ** 31 - 1, -2 ** 31]))
    check(3, 4, 1, D, 0, False, "f32", "bf16", pos=np.array([0, -1, N_POS]))


def test_rows_of_zeros_and_extremes():
    x = torch.zeros((4, 3 * 128))
    x[1] = 1e-25          # squares underflow: eps rules
    x[2] = 1e15
    x[3, 7] = float("nan")
    check(4, 2, 1, 128, 128, False, "f32", "f32", x=x)


def test_offsets_past_32_bits():
    M, ld = 5, 1 << 29
    g = np.random.default_rng(0)
    x = torch.from_numpy(g.standard_normal((M, 128)).astype(np.float32)).to(torch.bfloat16)
    buf, out = (torch.empty(M * ld, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    buf.view(M, ld)[:, :128] = x.to(DEV)
    cos, sin = tables(128)
    gamma = torch.ones(128, device=DEV)
    pos = np.arange(M)
    kq.kq_qk_norm_rope(kq.BF16, buf, ld, None, 0, M, 1, 0, 128, gamma, None, 0.0, torch.arange(M, device=DEV, dtype=torch.int32),
                       torch.from_numpy(cos).to(DEV), torch.from_numpy(sin).to(DEV), N_POS, 128, 0, kq.BF16, out, ld, None, 0)
    ref, size = reference(x.double().numpy()[:, None], np.ones(128), 0.0, pos, cos, sin, 128, False)
    got = out.view(M, ld)[:, :128].double().cpu().numpy()[:, None]
    assert (np.abs(got - ref) <= 72 * U * size + 2.0 ** -8 * 1.001 * np.abs(ref) + 1e-30).all()


@pytest.mark.parametrize("D,rot", [(128, 0), (128, 64), (80, 40), (512, 128), (72, 36)])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("gamma", [False, True])
@pytest.mark.parametrize("offset", [0, 1])
def test_infinities_and_nan_past_the_rotated_part(D, rot, pairs, gamma, offset):
    """Elements from rot on are normed only: an infinity or NaN among them stays where it is (without a norm), or is the
    only NaN of its head (with one, whose factor is then 0).  offset 1: rows that no vector form takes give the same."""
    M, Hq, Hk, n = 9, 2, 1, D - rot
    g = np.random.default_rng(D + rot)
    x = torch.from_numpy(g.standard_normal((M, 3 * D)).astype(np.float32))
    for m in range(M):  # (a NaN makes a normed head NaN as a whole)
        x[m, m % 3 * D + rot + (5 * m) % n] = [float("inf"), float("-inf"), float("inf") if gamma else float("nan")][m % 3]
    outs = check(M, Hq, Hk, D, rot, pairs, "f32", "f32", gamma=gamma, offset=offset, x=x.clone())
    if not gamma:
        got = torch.cat([o.cpu().reshape(M, -1) for o in outs], 1).view(M, 3, D)[:, :, rot:]
        assert torch.equal(got.nan_to_num(nan=12345.0), x.view(M, 3, D)[:, :, rot:].nan_to_num(nan=12345.0))


def test_pointers_of_nothing_are_not_looked_at():
    """With no key heads the keys' gamma is unused, and without a rotation the tables: whatever they are, the call is taken
    and gives the bits of one without them."""
    M, D = 5, 128
    g = torch.Generator(device=DEV)
    g.manual_seed(0)
    x, gamma = torch.randn((M, 2 * D), generator=g, device=DEV), torch.rand(D, generator=g, device=DEV)
    outs = []
    for odd in (None, torch.zeros(4, device=DEV).data_ptr() + 1):
        y = torch.empty((M, 2 * D), device=DEV)
        kq.kq_qk_norm_rope(kq.F32, x, 2 * D, odd, 0, M, 2, 0, D, gamma, odd, 1e-6, odd, odd, odd, 0, 0, 0, kq.F32, y, 2 * D, odd, 0)
        kq.kq_qk_norm_rope(kq.F32, odd, 0, y, 2 * D, M, 0, 2, D, odd, gamma, 1e-6, odd, odd, odd, 0, 0, 0, kq.F32, odd, 0, y, 2 * D)
        outs.append(y)
    assert torch.equal(outs[0], outs[1])
