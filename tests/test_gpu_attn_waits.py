"""The attention kernels' bounded waits: with a role idle they run out, the device flag tells it, and the stream goes on."""
import pytest
import torch

import gemv_quantize_q8_gb300 as kq
from tests.gpu_util import DEV
from tests.kv_util import Cache, ints
from tests.test_gpu_attn_cache import call as cache_call
from tests.test_gpu_attn_cache import check as cache_check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("idle", [1, 2])
@pytest.mark.parametrize("lens", [[300], [700, 900, 33, 1500]])  # one turn of the blocks, and many
def test_prompt(idle, lens):
    T, D, H = sum(lens), 128, 8
    g = torch.Generator(device=DEV).manual_seed(0)
    q, k, v = (torch.randn((T, H * D), generator=g, device=DEV).to(torch.bfloat16) for _ in range(3))
    y = torch.zeros_like(q)
    cu = ints([0] + list(torch.tensor(lens).cumsum(0)))
    n = kq.kq_attn_prompt_workspace_bytes(len(lens), T, H, H, D)
    ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
    args = (kq.BF16, q, H * D, k, H * D, v, H * D, cu, cu, len(lens), T, T, H, H, D, D ** -0.5, 1)
    kq.kq_attn_prompt(*args, y, H * D, ws, n)
    assert kq.kq_read_device_flag(ws) == 0
    again = torch.zeros_like(q)
    kq.kq_debug_attn_prompt_wait_timeout(*args, again, H * D, idle, 2_000_000, ws, n)
    assert kq.kq_read_device_flag(ws) > 0
    kq.kq_attn_prompt(*args, again, H * D, ws, n)
    assert kq.kq_read_device_flag(ws) == 0 and torch.equal(again, y)


@pytest.mark.parametrize("lens", [[40], [900, 5000, 0, 77]])
def test_cache(lens):
    c = Cache(lens, 2, 128, 16, fill=True)
    q = torch.randn((len(lens), 8 * 128), generator=torch.Generator().manual_seed(0))
    dq = q.to(DEV)
    n = kq.kq_attn_cache_i8_workspace_bytes(c.B, 1, 8, 2, 128)
    ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
    y = torch.zeros((c.B, 1024), device=DEV)
    kq.kq_debug_attn_cache_wait_timeout(kq.F32, dq, 1024, c.B, 1, 8, 2, 128, 0.1, *c.args, c.lens, kq.F32, y, 1024, 2_000_000, ws, n)
    assert kq.kq_read_device_flag(ws) > 0
    y = cache_call(c, dq, 1, 8, 0.1, ws=ws)
    assert kq.kq_read_device_flag(ws) == 0
    cache_check(y, c, q, lens, 1, 8, 0.1, "f32")


def test_refusals():
    x = torch.zeros(4096, device=DEV)
    for changes in ((3, 10000), (1, 10), (1, 10**10)):
        with pytest.raises(kq.KqError):
            kq.kq_debug_attn_prompt_wait_timeout(kq.BF16, x, 128, x, 128, x, 128, x, x, 1, 1, 1, 1, 1, 128, 1.0, 1, x, 128, *changes, x, 4096)
    with pytest.raises(kq.KqError, match="tensor-core"):  # heads of 256 take another form
        kq.kq_debug_attn_prompt_wait_timeout(kq.BF16, x, 256, x, 256, x, 256, x, x, 1, 1, 1, 1, 1, 256, 1.0, 1, x, 256, 1, 10000, x, 4096)
