"""Appending to the paged 8-bit cache and reading it back, bit for bit against the definition in numpy."""
import numpy as np
import pytest
import torch

import gemv_quantize_q8_gb300 as kq
from tests.gpu_util import DEV
from tests.kv_util import N_POS, TYPES, Cache, ints, tables

pytestmark = pytest.mark.gpu


def append(cache, new, lens, xt="f32", rot=0, pairs=False, seed=1, offset=0, pad=0, x=None, pos=None, packed=True, behind=0, scale=1.0,
           stream=None):
    """One call on the device and on the host copies; the rows' buffer starts `offset` elements behind a boundary."""
    g = np.random.default_rng(seed)
    n_kv, D, T = cache.n_kv, cache.D, sum(new)
    ld = 2 * n_kv * D + pad
    if x is None:
        x = (g.standard_normal((T + behind, ld)) * scale).astype(np.float32)
    rows = torch.from_numpy(x).to(TYPES[xt][1])
    buf = torch.zeros((T + behind) * ld + 8, dtype=rows.dtype, device=DEV)
    dev = buf[offset : offset + (T + behind) * ld].view(T + behind, ld)
    dev.copy_(rows)
    first = np.concatenate([np.arange(t - n, t) for n, t in zip(new, lens)] + [np.zeros(behind, np.int64)]).astype(np.int64)
    pos = first if pos is None else pos
    cos, sin = tables(rot)
    dcos, dsin, dpos = torch.from_numpy(cos).to(DEV), torch.from_numpy(sin).to(DEV), ints(pos)
    cu = ints(np.concatenate([[0], np.cumsum(new)])) if packed else None
    cache.lens = ints(lens)
    torch.cuda.synchronize()
    kq.kq_kv_append_i8(TYPES[xt][0], dev, ld, dev[:, n_kv * D :], ld, cu, cache.lens, cache.B, T + behind, n_kv, D, dpos if rot else None,
                       dcos if rot else None, dsin if rot else None, N_POS, rot, int(pairs), *cache.args, stream=stream)
    torch.cuda.synchronize()
    h = rows.float().numpy()[:T, : 2 * n_kv * D].reshape(T, 2, n_kv, D)
    cache.append(h[:, 0], h[:, 1], new, lens, pos[:T], cos, sin, rot, pairs)


def same(cache):
    assert np.array_equal(cache.scale.cpu().numpy(), cache.scale_host, equal_nan=True)
    assert np.array_equal(cache.codes.cpu().numpy(), cache.codes_host)


@pytest.mark.parametrize("xt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n_kv,D,page,rot,pairs", [(1, 16, 16, 0, False), (2, 128, 64, 128, False), (3, 80, 32, 40, True), (2, 64, 16, 12, False),
                                                   (1, 256, 256, 256, True), (5, 96, 128, 48, False), (2, 48, 32, 2, True)])
def test_append(xt, n_kv, D, page, rot, pairs):
    """Sequences that end inside, at and behind pages, one without new tokens, one fresh; then a few more tokens each."""
    old = [0, 5, page, 3 * page - 1, 70, 1, 2 * page + 3]
    new = [page + 1, 1, 1, 2, 0, 2 * page, 300]
    lens = [a + b for a, b in zip(old, new)]
    c = Cache([n + 3 for n in lens], n_kv, D, page)
    append(c, old, old, xt, rot, pairs, seed=2, scale=0.3)
    same(c)
    append(c, new, lens, xt, rot, pairs, seed=3)
    same(c)
    append(c, [1] * 7, [n + 1 for n in lens], xt, rot, pairs, seed=4, packed=False, scale=2.0)
    same(c)


@pytest.mark.parametrize("xt,offset,pad", [("f32", 1, 0), ("f32", 0, 3), ("f16", 3, 0), ("bf16", 1, 5), ("f16", 4, 8)])
@pytest.mark.parametrize("pairs", [False, True])
def test_append_from_any_address(xt, offset, pad, pairs):
    c = Cache([100, 40], 2, 64, 32)
    append(c, [90, 33], [90, 33], xt, 64, pairs, offset=offset, pad=pad)
    same(c)
    append(c, [10, 7], [100, 40], xt, 64, pairs, offset=offset, pad=pad, seed=9)
    same(c)


def test_scales_grow_shrink_and_begin_anew():
    c = Cache([64], 2, 32, 16)
    for i, s in enumerate([1.0, 0.1, 30.0, 1e-3, 200.0] + [1.0] * 27):  # token by token over two pages
        append(c, [1], [i + 1], seed=i, scale=s)
        same(c)
    append(c, [3], [20], seed=99, scale=0.5)  # taken back to 17 tokens: the scale keeps its size
    same(c)
    append(c, [4], [20], seed=98, scale=0.01)  # the page's first token is written: it begins anew
    same(c)


def test_special_values():
    n_kv, D = 2, 32
    x = np.random.default_rng(0).standard_normal((9, 2 * n_kv * D)).astype(np.float32)
    x[0, 3] = np.nan
    x[1, :D] = np.nan            # nothing but NaN in a row
    x[2] = 0.0
    c = Cache([40], n_kv, D, 16)
    append(c, [9], [9], x=x)
    same(c)
    for fill in (0.0, 1e-38, 3.0e-37, 1e-45, np.nan, 3e38):
        c = Cache([40], n_kv, D, 16)
        append(c, [9], [9], x=np.full_like(x, fill))
        same(c)
    x[4, 7] = np.inf             # keys of head 0: an infinite scale until the page begins anew
    c = Cache([40], n_kv, D, 16)
    append(c, [5], [5], x=x[:5])
    same(c)
    append(c, [2], [7], x=x[5:7])
    same(c)
    assert np.isinf(c.scale_host[0, c.table_host[0, 0], 0])
    append(c, [3], [3], x=x[5:8])
    same(c)
    assert np.isfinite(c.scale_host[0, c.table_host[0, 0]]).all()


def test_positions_without_an_angle():
    c = Cache([30], 1, 32, 16)
    pos = np.arange(20)
    pos[3], pos[5], pos[7] = -1, N_POS, 2**31 - 1
    append(c, [20], [20], rot=16, pos=pos)
    same(c)


def test_tokens_without_a_place():
    """Pages out of range, past the table, rows before token 0, rows behind the last sequence, empty sequences."""
    c = Cache([40, 40, 5, 0], 2, 32, 16)
    c.table_host[0, 1], c.table_host[1, 0] = c.n_pages, -1
    c.upload()
    append(c, [40, 40, 8, 0], [40, 40, 5, 0], rot=32, behind=11)
    same(c)
    c = Cache([20], 1, 16, 16, spare=9)
    append(c, [200], [200])  # three pages in the table, the third without a page
    same(c)


@pytest.mark.parametrize("yt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("offset,pad", [(0, 0), (1, 0), (0, 5)])
def test_read(yt, offset, pad):
    lens, back = [100, 16, 0, 33, 64], [37, 16, 0, 33, 1]
    c = Cache(lens, 3, 48, 16, fill=True)
    T, width = sum(back), 3 * 48
    ld = width + pad
    out = [torch.full(((T + 4) * ld + 8,), 7.0, dtype=TYPES[yt][1], device=DEV) for _ in range(2)]
    k, v = (o[offset : offset + (T + 4) * ld].view(T + 4, ld) for o in out)
    kq.kq_kv_read_i8(*c.args, ints(np.concatenate([[0], np.cumsum(back)])), c.lens, c.B, T + 4, 3, 48, TYPES[yt][0], k, ld, v, ld)
    torch.cuda.synchronize()
    for which, o in enumerate((k, v)):
        want = []
        for b, (n, t) in enumerate(zip(back, lens)):
            i = np.arange(t - n, t)
            p = c.table_host[b, i // 16]
            want.append(c.codes_host[which][p, :, i % 16].astype(np.float32) * c.scale_host[which][p][..., None])
        want = torch.from_numpy(np.concatenate(want).reshape(T, width)).to(TYPES[yt][1])
        assert torch.equal(o[:T, :width].cpu(), want)
        assert bool((o[T:] == 7.0).all()) and bool((o[:, width:] == 7.0).all())
    torch.cuda.synchronize()


def test_read_without_a_place():
    c = Cache([40, 20], 1, 16, 16, fill=True)
    c.table_host[0, 1] = -1
    c.upload()
    k, v = (torch.full((63, 16), 7.0, device=DEV) for _ in range(2))
    kq.kq_kv_read_i8(*c.args, ints([0, 40, 63]), c.lens, 2, 63, 1, 16, kq.F32, k, 16, v, 16)
    torch.cuda.synchronize()
    left = (k == 7.0).all(1).cpu().numpy()
    assert left[16:32].all() and left[40:43].all() and not left[:16].any() and not left[32:40].any() and not left[43:].any()


def test_infinite_scale_reads_as_nan():
    c = Cache([16], 1, 16, 16, fill=True)
    c.codes_host[:] = 0
    c.scale_host[0] = np.inf
    c.upload()
    k, v = (torch.zeros((16, 16), device=DEV) for _ in range(2))
    kq.kq_kv_read_i8(*c.args, None, c.lens, 1, 16, 1, 16, kq.F32, k, 16, v, 16)
    torch.cuda.synchronize()
    assert bool(k.isnan().all()) and bool((v == 0).all())


def test_streams_and_graphs():
    """On a stream of its own, and captured and replayed with other rows."""
    c = Cache([50, 50], 2, 64, 16)
    s = torch.cuda.Stream()
    append(c, [30, 10], [30, 10], rot=64, stream=s)
    same(c)
    T, ld = 2, 2 * 2 * 64
    x, lens, pos = torch.zeros((T, ld), device=DEV), ints([31, 11]), ints([30, 10])
    cos, sin = tables(64)
    dcos, dsin = torch.from_numpy(cos).to(DEV), torch.from_numpy(sin).to(DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kq.kq_kv_append_i8(kq.F32, x, ld, x[:, 128:], ld, None, lens, 2, T, 2, 64, pos, dcos, dsin, N_POS, 64, 0, *c.args)
    for i in range(3):
        h = np.random.default_rng(i).standard_normal((T, ld)).astype(np.float32)
        x.copy_(torch.from_numpy(h))
        lens.copy_(ints([31 + i, 11 + i]))
        pos.copy_(ints([30 + i, 10 + i]))
        graph.replay()
        torch.cuda.synchronize()
        h = h.reshape(T, 2, 2, 64)
        c.append(h[:, 0], h[:, 1], [1, 1], [31 + i, 11 + i], np.array([30 + i, 10 + i]), cos, sin, 64, False)
        same(c)


def test_many_sequences_and_pages():
    """More sequences than a thread block has threads; offsets of the cache past 2^31."""
    g = np.random.default_rng(5)
    new = g.integers(0, 4, 700).tolist()
    c = Cache([n + 20 for n in new], 1, 16, 16)
    append(c, new, [n + 13 if n else 0 for n in new])
    same(c)
    n_pages, n_kv, D, page = 70000, 1, 128, 256  # 2.3e9 codes a cache
    codes = torch.zeros((2, n_pages, n_kv, page, D), dtype=torch.int8, device=DEV)
    scale = torch.zeros((2, n_pages, n_kv), device=DEV)
    x = torch.randn((2, 2 * D), device=DEV)
    table, lens = ints([[n_pages - 1], [1]]), ints([200, 1])
    args = (codes[0], codes[1], scale[0], scale[1], n_pages, page, table, 1)
    kq.kq_kv_append_i8(kq.F32, x, 2 * D, x[:, D:], 2 * D, None, lens, 2, 2, 1, D, None, None, None, 0, 0, 0, *args)
    k, v = torch.empty((2, D), device=DEV), torch.empty((2, D), device=DEV)
    kq.kq_kv_read_i8(*args, None, lens, 2, 2, 1, D, kq.F32, k, D, v, D)
    torch.cuda.synchronize()
    for got, want in ((k, x[:, :D]), (v, x[:, D:])):  # a code is off by half a step of amax / 127
        assert bool(((got - want).abs() <= want.abs().amax(1, keepdim=True) / 127 * 0.5001).all())
    assert int((codes != 0).any(-1).sum()) == 4


def test_very_many_sequences():
    """More than two steps of the search for a row's sequence find; every third without tokens."""
    new = [0 if b % 3 == 2 else 1 for b in range(70000)]
    c = Cache(new, 1, 16, 16)
    append(c, new, new, "bf16")
    same(c)
