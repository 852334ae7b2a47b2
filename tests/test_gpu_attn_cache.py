"""Attention over the paged 8-bit cache against numpy in 64 bits.

Tolerance, with u = 2^-24 and S = |scale| * max_j sum_d |q_d k_d| (which bounds every score): the queries' 22 bits and the products'
fp32 sums move a score by (D + 16) u S, and a weight relative to the others by twice that; the weights' own 22 bits, the
exponential and the division take 64 u, and the sums over L tokens, 16 at a time with up to four roundings each, L/4 u.  All
weigh values of at most V = max |v|:
    |y - y64| <= (2 (D + 16) u S + (L/4 + 64) u) V + half a unit of the output's type."""
import numpy as np
import pytest
import torch

import gemv_quantize_q8_gb300 as kq
from tests.gpu_util import DEV
from tests.kv_util import HALF_UNIT, TYPES, U, Cache, attention, ints

pytestmark = pytest.mark.gpu


def call(c, q, n_new, n_q, scale, xt="f32", yt="f32", out=None, ws=None, stream=None, ldq=None, ldy=None):
    width = n_q * c.D
    n = kq.kq_attn_cache_i8_workspace_bytes(c.B, n_new, n_q, c.n_kv, c.D)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV) if ws is None else ws  # (NaN in every float)
    y = torch.full((c.B * n_new, width), 7.0, dtype=TYPES[yt][1], device=DEV) if out is None else out
    kq.kq_attn_cache_i8(TYPES[xt][0], q, ldq or width, c.B, n_new, n_q, c.n_kv, c.D, scale, *c.args, c.lens, TYPES[yt][0], y, ldy or width,
                        ws, n, stream=stream)
    return y


def check(y, c, q, lens, n_new, n_q, scale, yt, only=None):
    q = q.double().cpu().numpy().reshape(c.B, n_new, n_q, c.D)
    y = y.double().cpu().numpy().reshape(c.B, n_new, n_q, c.D)
    for b, t in enumerate(lens):
        if only is not None and b not in only:
            continue
        limits = [max(t - n_new + 1 + i, 0) for i in range(n_new)]
        ref, V, S = attention(q[b], c.rows(b, t, 0), c.rows(b, t, 1), float(np.float32(scale)), limits)
        tol = (2 * (c.D + 16) * U * S + (t / 4 + 64) * U) * V
        tol = tol + HALF_UNIT[yt] * (np.abs(ref) + tol) + (2.0 ** -25 if yt == "f16" else 0)
        assert np.array_equal(np.isnan(y[b]), np.isnan(ref))
        bad = np.abs(y[b] - ref) > tol
        assert not bad.any(), (b, t, np.abs(y[b] - ref)[bad].max(), tol.max())


def run(lens, n_new, n_q, n_kv, D, page, xt="f32", yt="f32", scale=None, seed=0, amp=1.0, room=0):
    c = Cache(lens, n_kv, D, page, seed=seed, fill=True)
    if room:  # tables of `room` pages: long sequences may come
        c.table_host = np.pad(c.table_host, ((0, 0), (0, room - c.ldt)), constant_values=-7)
        c.ldt = room
        c.upload()
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn((c.B * n_new, n_q * D), generator=g) * amp).to(TYPES[xt][1])
    scale = D ** -0.5 if scale is None else scale
    y = call(c, q.to(DEV), n_new, n_q, scale, xt, yt)
    torch.cuda.synchronize()
    check(y, c, q, lens, n_new, n_q, scale, yt)
    return c, q, y


@pytest.mark.parametrize("n_q,n_kv", [(1, 1), (4, 1), (8, 2), (7, 7), (14, 2), (32, 2), (20, 1)])
@pytest.mark.parametrize("D", [16, 64, 80, 128, 144, 256])
def test_heads(n_q, n_kv, D):
    run([37, 0, 1, 16, 200], 1, n_q, n_kv, D, 16)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("n_new", [1, 2, 3, 5, 9])
def test_pages_and_new_tokens(page, n_new):
    """Lengths around pages and units; sequences shorter than the new tokens (rows that see nothing)."""
    run([page - 1, page, page + 1, 15, 16, 17, 2 * page + 5, 1, 2, 0, 333], n_new, 6, 3, 64, page)


@pytest.mark.parametrize("xt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("yt", ["f32", "f16", "bf16"])
def test_types(xt, yt):
    run([50, 129, 7], 1, 8, 2, 128, 32, xt, yt, amp=3.0)


@pytest.mark.parametrize("lens", [[20000], [9000, 3, 4100], [1] * 300, [17] * 400, [0] * 40 + [2500] + [0] * 40])
def test_lengths(lens):
    """One long sequence over every warp, ragged ones, many short ones, one among empty ones."""
    run(lens, 1, 4, 2, 64, 64)


@pytest.mark.parametrize("n_new,n_q,n_kv", [(1, 20, 1), (3, 14, 2), (1, 32, 2), (9, 4, 2), (2, 9, 1), (4, 4, 1), (8, 8, 2)])
@pytest.mark.parametrize("D", [16, 64, 80, 128, 256])
def test_many_rows_and_tables_with_room(n_new, n_q, n_kv, D):
    """More than eight rows of a key head, in tables that have room for much longer sequences and in those that have not."""
    lens = [37, 0, 1, 16, 200, 1500, 8]
    run(lens, n_new, n_q, n_kv, D, 16, room=3000)
    run(lens, n_new, n_q, n_kv, D, 16)


@pytest.mark.parametrize("B,n_kv,D,longest", [(6000, 2, 64, 40), (1300, 1, 256, 70), (200, 2, 64, 3000), (140, 1, 256, 3000), (90, 2, 128, 5000)])
def test_more_sequences_than_threads_and_full_shares(B, n_kv, D, longest):
    """A thread sums up several sequences; many items, of one unit or of about a hundred, in every warp's share."""
    lens = np.random.default_rng(B).integers(0, longest, B).tolist()
    run(lens, 1, 2 * n_kv, n_kv, D, 32)


def test_rows_of_sixteen_in_full_shares():
    lens = np.random.default_rng(2).integers(0, 4000, 120).tolist()
    run(lens, 4, 6, 2, 64, 64, "f16", "f16")


def test_two_calls_at_once():
    """Two streams, a workspace each."""
    work = []
    for seed, lens in ((1, [4000, 900, 0, 7]), (2, [2500, 2500, 31])):
        c = Cache(lens, 2, 128, 64, seed=seed, fill=True)
        q = torch.randn((c.B, 8 * 128), generator=torch.Generator().manual_seed(seed))
        n = kq.kq_attn_cache_i8_workspace_bytes(c.B, 1, 8, 2, 128)
        work.append((c, lens, q, q.to(DEV), torch.zeros_like(q, device=DEV), torch.zeros(n, dtype=torch.uint8, device=DEV), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for c, _, _, dq, y, ws, stream in work:
            call(c, dq, 1, 8, 128 ** -0.5, out=y, ws=ws, stream=stream)
    torch.cuda.synchronize()
    for c, lens, q, _, y, _, _ in work:
        check(y, c, q, lens, 1, 8, 128 ** -0.5, "f32")


def test_long_rows_of_sixteen():
    run([6000, 1000], 4, 8, 2, 128, 64, "bf16", "f32")


@pytest.mark.parametrize("amp,scale", [(30.0, 1.0), (1e-20, 1.0), (1e20, 1e-20), (1.0, 0.0), (5.0, -0.2), (1e4, 1e-3)])
def test_sizes_of_scores(amp, scale):
    """Weights of one token alone, flat weights, queries far outside f16's range, a negative scale."""
    run([300, 5], 1, 4, 1, 64, 16, amp=amp, scale=scale)


def test_value_scales_of_different_size():
    """Blocks whose scales rise and fall by many orders: each token keeps its own weight."""
    c = Cache([256], 1, 64, 16, fill=True)
    for i, e in enumerate([-30, 0, -6, 12, 3, 20, -38, 20, 0, 5, 25, -10, 1, 2, 30, 0]):
        c.scale_host[1, c.table_host[0, i]] = 10.0 ** e if e > -38 else 0.0
    c.upload()
    q = torch.randn((1, 256), generator=torch.Generator().manual_seed(1)) * 4
    y = call(c, q.to(DEV), 1, 4, 0.125)
    torch.cuda.synchronize()
    check(y, c, q, [256], 1, 4, 0.125, "f32")


def test_strides_in_place_and_rows_behind():
    c = Cache([70, 33], 2, 32, 16, fill=True)
    for xt, offset, pad in (("f32", 0, 12), ("f32", 1, 3), ("bf16", 3, 0), ("f16", 4, 8)):
        ld = 4 * 32 + pad
        buf = torch.full((4 * ld + 8,), 5.0, dtype=TYPES[xt][1], device=DEV)
        rows = buf[offset : offset + 4 * ld].view(4, ld)
        q = torch.randn((2, 128), generator=torch.Generator().manual_seed(pad)).to(TYPES[xt][1])
        rows[:2, :128] = q.to(DEV)
        call(c, rows, 1, 4, 0.2, xt, xt, out=rows, ldq=ld, ldy=ld)
        torch.cuda.synchronize()
        check(rows[:2, :128].contiguous(), c, q, [70, 33], 1, 4, 0.2, xt)
        assert bool((rows[2:] == 5.0).all()) and bool((rows[:, 128:] == 5.0).all())


def test_junk_behind_the_last_token():
    """Codes behind a sequence's end, and pages behind its last, have no influence (infinite scales among them)."""
    lens = [40, 5]
    c, q, y = run(lens, 1, 4, 1, 64, 16)
    for b, t in enumerate(lens):
        p = c.table_host[b, (t - 1) // 16]
        c.codes_host[:, p, :, t % 16 :] = -128 if t % 16 else c.codes_host[:, p, :, t % 16 :]
    used = {int(p) for b, t in enumerate(lens) for p in c.table_host[b, : -(-t // 16)]}
    for p in set(range(c.n_pages)) - used:
        c.scale_host[:, p] = np.inf
    c.upload()
    again = call(c, q.to(DEV), 1, 4, 64 ** -0.5)
    torch.cuda.synchronize()
    assert torch.equal(y, again)


def test_infinite_blocks_reach_those_that_see_them():
    """Keys or values of an infinite scale: NaN for the tokens that see the block, the others as before."""
    for which in (0, 1):
        c, q, y = run([33, 40], 2, 4, 2, 64, 16)  # sequence 0: its last token alone is in its third page
        c.scale_host[which, c.table_host[0, 2], 0] = np.inf
        c.codes_host[which, c.table_host[0, 2], 0] = 0
        c.upload()
        again = call(c, q.to(DEV), 2, 4, 64 ** -0.5)
        torch.cuda.synchronize()
        nan = again.isnan().view(2, 2, 4, 64)
        assert bool(nan[0, 1, :2].all()) and int(nan.sum()) == 2 * 64
        assert torch.equal(again[~again.isnan()], y[~again.isnan()])


def test_queries_that_are_not_finite():
    c, q, y = run([100, 20], 1, 4, 2, 64, 32)
    bad = q.clone().view(2, 4, 64)
    bad[0, 1, 5], bad[1, 2, 9], bad[1, 3, 0] = float("nan"), float("inf"), -float("inf")
    again = call(c, bad.to(DEV), 1, 4, 64 ** -0.5).view(2, 4, 64)
    torch.cuda.synchronize()
    hit = torch.zeros((2, 4), dtype=torch.bool)
    hit[0, 1] = hit[1, 2] = hit[1, 3] = True
    assert bool(again[hit].isnan().all()) and torch.equal(again[~hit], y.view(2, 4, 64)[~hit])


def test_bad_pages_and_lengths():
    """A page out of range or a length past the table: NaN for that sequence, nothing else is touched."""
    lens = [50, 20, 64, 33]
    c, q, y = run(lens, 1, 2, 1, 32, 16)
    c.table_host[0, 2], c.table_host[3, 0] = c.n_pages, -1
    c.upload()
    c.lens = ints([50, 20, 16 * c.ldt + 1, 33])
    again = call(c, q.to(DEV), 1, 2, 32 ** -0.5)
    torch.cuda.synchronize()
    assert bool(again[[0, 2, 3]].isnan().all())
    check(again, c, q, lens, 1, 2, 32 ** -0.5, "f32", only=[1])  # (its sums may be cut elsewhere: another length is another line)


def test_shared_pages():
    """Two sequences that begin with the same pages."""
    c = Cache([48, 40], 2, 64, 16, fill=True)
    c.table_host[1, :2] = c.table_host[0, :2]
    c.upload()
    q = torch.randn((2, 256), generator=torch.Generator().manual_seed(3))
    y = call(c, q.to(DEV), 1, 4, 0.125)
    torch.cuda.synchronize()
    check(y, c, q, [48, 40], 1, 4, 0.125, "f32")


def test_repeatable_streams_and_graphs():
    c, q, y = run([3000, 77, 500], 1, 8, 2, 128, 64)
    n = kq.kq_attn_cache_i8_workspace_bytes(3, 1, 8, 2, 128)
    ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
    dq = q.to(DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = torch.zeros_like(y)
    torch.cuda.synchronize()
    call(c, dq, 1, 8, 128 ** -0.5, out=again, ws=ws, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(again, y)
    out = torch.zeros_like(y)
    graphs = []
    for _ in range(2):  # two graphs that share the workspace, one after the other
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(c, dq, 1, 8, 128 ** -0.5, out=out, ws=ws)
        graphs.append(graph)
    for lens in ([3000, 77, 500], [1, 128, 0], [2999, 0, 500]):
        c.lens.copy_(ints(lens))
        for graph in graphs:
            out.fill_(3.0)
            graph.replay()
            torch.cuda.synchronize()
            check(out, c, q, lens, 1, 8, 128 ** -0.5, "f32")


def test_offsets_past_32_bits():
    """Pages past 2^31 bytes of the cache."""
    n_pages, D, page = 70000, 128, 256
    codes = torch.zeros((2, n_pages, 1, page, D), dtype=torch.int8, device=DEV)
    scale = torch.ones((2, n_pages, 1), device=DEV)
    codes[1, n_pages - 1] = 3
    codes[1, 2] = 5
    table, lens = ints([[n_pages - 1, 2], [2, n_pages - 1]]), ints([256, 512])
    q, y = torch.randn((2, 2 * D), device=DEV), torch.zeros((2, 2 * D), device=DEV)
    n = kq.kq_attn_cache_i8_workspace_bytes(2, 1, 2, 1, D)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    kq.kq_attn_cache_i8(kq.F32, q, 2 * D, 2, 1, 2, 1, D, 0.1, codes[0], codes[1], scale[0], scale[1], n_pages, page, table, 2, lens, kq.F32, y,
                        2 * D, ws, n)
    torch.cuda.synchronize()
    # all scores are 0; the weights 1/L are powers of two
    assert bool((y[0] == 3.0).all()) and bool((y[1] == 4.0).all())
