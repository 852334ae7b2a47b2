"""The attention calls together, as a serving program uses them: a prompt in two parts, then token by token.

The plain side knows the same bf16 queries, keys and values.  Its cache holds the values that the codes stand for (read from the
device and checked apart, bit by bit), so what is left is each attention's own tolerance: weights and outputs rounded
to bf16 (2^-8 each of the largest value, and of the result), and fp32 sums."""
import numpy as np
import pytest
import torch

import gemv_quantize_q8_gb300 as kq
from tests.gpu_util import DEV
from tests.kv_util import ints

pytestmark = pytest.mark.gpu

HQ, HK, D, PAGE, MAX = 8, 2, 128, 32, 1024
WQ, WK = HQ * D, HK * D


def tables():
    a = torch.arange(MAX, device=DEV, dtype=torch.float64)[:, None] * 1e4 ** (-torch.arange(0, D, 2, device=DEV, dtype=torch.float64) / D)
    return a.cos().float(), a.sin().float()


def plain(q, k, v, past):
    """q [n][HQ][D] (tokens past, past + 1, ..), k and v [past + n][HK][D], in 64 bits."""
    n, L = q.shape[0], k.shape[0]
    k, v = (x.repeat_interleave(HQ // HK, 1) for x in (k, v))
    s = torch.einsum("qhd,khd->hqk", q, k) * D ** -0.5
    hidden = torch.arange(L, device=DEV) > past + torch.arange(n, device=DEV)[:, None]
    return torch.einsum("hqk,khd->qhd", s.masked_fill(hidden, -float("inf")).softmax(2), v)


def close(got, want, values):
    tol = 2.5 * 2.0 ** -8 * values.abs().max() + 2.0 ** -8 * want.abs()
    assert bool(((got.double().view_as(want) - want).abs() <= tol).all())


def test_prompt_in_two_parts_then_token_by_token():
    lens, more, steps = [300, 45, 130], [100, 7, 64], 40
    B = len(lens)
    g = torch.Generator(device=DEV).manual_seed(0)
    cos, sin = tables()
    ldt = MAX // PAGE
    n_pages = B * ldt
    table = torch.randperm(n_pages, generator=torch.Generator().manual_seed(1)).int().to(DEV).view(B, ldt)
    codes = torch.randint(-128, 128, (2, n_pages, HK, PAGE, D), generator=g, device=DEV, dtype=torch.int8)
    scales = torch.full((2, n_pages, HK), float("nan"), device=DEV)
    pages = (codes[0], codes[1], scales[0], scales[1], n_pages, PAGE, table, ldt)
    have = torch.zeros(B, dtype=torch.int32, device=DEV)

    def product(T):
        return torch.randn((T, WQ + 2 * WK), generator=g, device=DEV)

    def heads(qkv, pos):
        """Queries rotated in bf16, keys for the prompt's attention likewise, values in bf16."""
        T, ld = qkv.shape
        q = torch.empty((T, WQ), dtype=torch.bfloat16, device=DEV)
        k, v = (torch.empty((T, WK), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        kq.kq_qk_norm_rope(kq.F32, qkv, ld, qkv[:, WQ:], ld, T, HQ, HK, D, None, None, 0.0, pos, cos, sin, MAX, D, 0, kq.BF16, q, WQ, k, WK)
        kq.kq_qk_norm_rope(kq.F32, None, 0, qkv[:, WQ + WK :], ld, T, 0, HK, D, None, None, 0.0, None, None, None, 0, 0, 0, kq.BF16, None, 0,
                           v, WK)
        return q, k, v

    def append(qkv, pos, cu, T):
        kq.kq_kv_append_i8(kq.F32, qkv[:, WQ:], qkv.shape[1], qkv[:, WQ + WK :], qkv.shape[1], cu, have, B, T, HK, D, pos, cos, sin, MAX, D, 0,
                           *pages)

    def positions(new):
        return ints(np.concatenate([np.arange(h - n, h) for n, h in zip(new, have.tolist())]))

    def cu_of(n):
        return ints(np.concatenate([[0], np.cumsum(n)]))

    def read(n, dtype=torch.bfloat16):
        """The last n tokens of every sequence."""
        T = sum(n)
        k, v = (torch.empty((T, WK), dtype=dtype, device=DEV) for _ in range(2))
        kq.kq_kv_read_i8(*pages, cu_of(n), have, B, T, HK, D, kq.BF16 if dtype == torch.bfloat16 else kq.F32, k, WK, v, WK)
        return k, v

    def attend(q, k, v, nq, nk):
        y = torch.empty_like(q)
        n = kq.kq_attn_prompt_workspace_bytes(B, q.shape[0], HQ, HK, D)
        ws = torch.empty(n, dtype=torch.uint8, device=DEV)
        kq.kq_attn_prompt(kq.BF16, q, WQ, k, WK, v, WK, cu_of(nq), cu_of(nk), B, q.shape[0], k.shape[0], HQ, HK, D, D ** -0.5, 1, y, WQ, ws, n)
        assert kq.kq_read_device_flag(ws) == 0
        return y

    def compare(y, q, k, v, nq, nk):
        aq = ak = 0
        for n, L in zip(nq, nk):
            kk, vv = (x[ak : ak + L].double().view(L, HK, D) for x in (k, v))
            close(y[aq : aq + n], plain(q[aq : aq + n].double().view(n, HQ, D), kk, vv, L - n), vv)
            aq, ak = aq + n, ak + L

    # the prompts' first parts: attention over their own rows, which go to the cache as well
    have += ints(lens)
    qkv, pos = product(sum(lens)), positions(lens)
    q, k, v = heads(qkv, pos)
    compare(attend(q, k, v, lens, lens), q, k, v, lens, lens)
    append(qkv, pos, cu_of(lens), sum(lens))
    kc, vc = read(lens, torch.float32)
    for cached, rows in ((kc, k), (vc, v)):  # a code is off by half a step of its block's largest, about 4.5 / 127
        assert float((cached - rows.float()).abs().max()) < 6.0 / 127 / 2 + 0.02
    # their second parts: appended, and attended with the cached rows read back
    have += ints(more)
    qkv, pos = product(sum(more)), positions(more)
    q, _, _ = heads(qkv, pos)
    append(qkv, pos, cu_of(more), sum(more))
    total = have.tolist()
    kc, vc = read(total)
    compare(attend(q, kc, vc, more, total), q, kc, vc, more, total)
    # token by token, the step captured once
    qkv, pos = product(B), torch.zeros(B, dtype=torch.int32, device=DEV)
    q = torch.empty((B, WQ), dtype=torch.bfloat16, device=DEV)
    y = torch.empty_like(q)
    n = kq.kq_attn_cache_i8_workspace_bytes(B, 1, HQ, HK, D)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    ld = qkv.shape[1]

    def step():
        kq.kq_qk_norm_rope(kq.F32, qkv, ld, None, 0, B, HQ, 0, D, None, None, 0.0, pos, cos, sin, MAX, D, 0, kq.BF16, q, WQ, None, 0)
        append(qkv, pos, None, B)
        kq.kq_attn_cache_i8(kq.BF16, q, WQ, B, 1, HQ, HK, D, D ** -0.5, *pages, have, kq.BF16, y, WQ, ws, n)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(steps):
        qkv.copy_(product(B) * (1 + 0.2 * i))  # (rows that grow: blocks' scales grow with them)
        pos.copy_(have)
        have += 1
        graph.replay()
        torch.cuda.synchronize()
        total = have.tolist()
        kc, vc = read(total, torch.float32)
        compare(y, q, kc, vc, [1] * B, total)
    assert kq.kq_read_device_flag(ws) == 0


def test_cache_and_prompt_agree():
    """The newest tokens' attention over the cache, and the prompt's over the rows read back: both round only what they are
    documented to (the read rows to f16, 2^-11; weights and outputs likewise)."""
    g = torch.Generator(device=DEV).manual_seed(3)
    L, n = 777, 5
    pages = -(-L // PAGE)
    codes = torch.randint(-127, 128, (2, pages, HK, PAGE, D), generator=g, device=DEV, dtype=torch.int8)
    scales = torch.rand((2, pages, HK), generator=g, device=DEV) * 0.02 + 0.01
    table, lens = torch.arange(pages, device=DEV, dtype=torch.int32), ints([L])
    cache = (codes[0], codes[1], scales[0], scales[1], pages, PAGE, table, pages)
    q = torch.randn((n, WQ), generator=g, device=DEV).to(torch.float16)
    a, b = torch.empty_like(q), torch.empty_like(q)
    size = kq.kq_attn_cache_i8_workspace_bytes(1, n, HQ, HK, D)
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    kq.kq_attn_cache_i8(kq.F16, q, WQ, 1, n, HQ, HK, D, D ** -0.5, *cache, lens, kq.F16, a, WQ, ws, size)
    k, v = (torch.empty((L, WK), dtype=torch.float16, device=DEV) for _ in range(2))
    kq.kq_kv_read_i8(*cache, None, lens, 1, L, HK, D, kq.F16, k, WK, v, WK)
    size = kq.kq_attn_prompt_workspace_bytes(1, n, HQ, HK, D)
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    kq.kq_attn_prompt(kq.F16, q, WQ, k, WK, v, WK, ints([0, n]), ints([0, L]), 1, n, L, HQ, HK, D, D ** -0.5, 1, b, WQ, ws, size)
    # keys off by 2^-11 move a score by S * 2^-11, S = sum |q_d k_d| / sqrt(D) at most; a weight by twice that
    S = float(torch.einsum("nhd,lhd->nhl", q.float().view(n, HQ, D).abs(), k.float().abs().view(L, HK, D).repeat_interleave(HQ // HK, 1)).max()) * D ** -0.5
    V = float(v.float().abs().max())
    assert float((a.float() - b.float()).abs().max()) <= (2 * S + 4) * 2.0 ** -11 * V
