"""Bounded waits of the prompt attention that no stalled role explains: a pair of row tiles that takes longer than the limit, and
a row tile that is left waiting when the other has finished."""
import pytest
import torch

import gemv_quantize_q8_gb300 as kq
from tests.gpu_util import DEV
from tests.kv_util import ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads", [1, 3])
def test_pairs_longer_than_the_limit(heads):
    """One token over 2^20 keys: 8192 key tiles, 16 KB each of keys and of values, are more than 2 ms of a block's work, and the
    second row tile of the last pair of heads is not there.  No single wait for a tile comes near 2 ms."""
    T, D = 1 << 20, 64
    g = torch.Generator(device=DEV).manual_seed(0)
    q = torch.randn((1, heads * D), generator=g, device=DEV).to(torch.bfloat16)
    k, v = (torch.randn((T, D), generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    n = kq.kq_attn_prompt_workspace_bytes(1, 1, heads, 1, D)
    ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
    y, again = torch.zeros_like(q), torch.zeros_like(q)
    args = (kq.BF16, q, heads * D, k, D, v, D, ints([0, 1]), ints([0, T]), 1, 1, T, heads, 1, D, D ** -0.5, 1)
    kq.kq_attn_prompt(*args, y, heads * D, ws, n)
    assert kq.kq_read_device_flag(ws) == 0
    kq.kq_debug_attn_prompt_wait_timeout(*args, again, heads * D, 0, 2_000_000, ws, n)
    assert kq.kq_read_device_flag(ws) == 0 and torch.equal(again, y)


@pytest.mark.parametrize("tokens", [100, 700])
def test_a_row_tile_that_waits_alone(tokens):
    """The first row tile of a pair finishes, the second one's products never come: the flag tells it all the same."""
    H, D = 2, 128
    g = torch.Generator(device=DEV).manual_seed(0)
    q = torch.randn((tokens, H * D), generator=g, device=DEV).to(torch.bfloat16)
    k, v = (torch.randn((tokens, D), generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    cu = ints([0, tokens])
    n = kq.kq_attn_prompt_workspace_bytes(1, tokens, H, 1, D)
    ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
    y, again = torch.zeros_like(q), torch.zeros_like(q)
    args = (kq.BF16, q, H * D, k, D, v, D, cu, cu, 1, tokens, tokens, H, 1, D, D ** -0.5, 1)
    kq.kq_attn_prompt(*args, y, H * D, ws, n)
    assert kq.kq_read_device_flag(ws) == 0
    kq.kq_debug_attn_prompt_wait_timeout(*args, again, H * D, 4, 2_000_000, ws, n)
    assert kq.kq_read_device_flag(ws) > 0
    kq.kq_attn_prompt(*args, again, H * D, ws, n)
    assert kq.kq_read_device_flag(ws) == 0 and torch.equal(again, y)
