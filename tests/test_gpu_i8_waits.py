"""The int8 product's bounded waits: each form of the tensor-core kernel with a role kept idle returns, reports it, and
leaves the stream usable.  Nothing faults or hangs: every CTA lets its copies and MMAs in flight end and frees its tensor
memory before it leaves."""
import ctypes

import pytest
import torch

import gemv_quantize_q8_gb300 as kq
from tests.gpu_util import DEV

#: CTAs that share a tile's rows, its tokens, whether its K is split; and sizes among which one takes that form.
FORMS = [
    (1, 32, False, [(16, 19456, 2048), (20, 300, 256)]),
    (1, 32, True, [(16, 300, 4096), (32, 300, 8192)]),
    (1, 64, False, [(64, 14336, 4096), (50, 19456, 2048)]),
    (1, 64, True, [(48, 600, 4096), (64, 300, 8192)]),
    (1, 128, False, [(128, 19456, 2048), (100, 14336, 2048)]),
    (1, 128, True, [(100, 600, 4096), (300, 512, 4096)]),
    (2, 256, False, [(2048, 4096, 2048), (2048, 14336, 2048)]),
    (2, 256, True, [(512, 4096, 14336), (2048, 512, 16384), (1024, 1024, 32768)]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("idle", [1, 2])
@pytest.mark.parametrize("ctas,tokens,split,sizes", FORMS)
def test_waits_run_out_and_the_next_call_is_right(ctas, tokens, split, sizes, idle):
    forms = {s: kq.kq_debug_i8_form(*s) for s in sizes}
    fits = [s for s, f in forms.items() if f[:2] == (ctas, tokens) and (f[2] > 1) == split]
    assert fits, forms
    M, N, K = fits[0]
    g = torch.Generator(device=DEV)
    g.manual_seed(M + N)
    q, w = (torch.randint(-128, 128, (r, K), generator=g, device=DEV, dtype=torch.int8) for r in (M, N))
    one, ones = torch.ones(M, device=DEV), torch.ones(N, device=DEV)
    n = kq.kq_gemm_i8_workspace_bytes(M, N, K)
    ws, y = torch.full((n,), 0xAB, dtype=torch.uint8, device=DEV), torch.zeros((M, N), device=DEV)
    for _ in range(2):
        kq.kq_debug_i8_wait_timeout(q, K, one, w, K, ones, M, N, K, y, N, idle, 200_000, ws, n)
        torch.cuda.synchronize()
        bad = ctypes.c_int64(0)
        status = kq.lib().kq_read_device_flag(ws.data_ptr(), ctypes.byref(bad), torch.cuda.current_stream().cuda_stream)
        assert status == 6, kq.lib().kq_status_string(status)    # KQ_ERR_DEVICE_FLAG
        tiles = -(-N // (128 * ctas)) * -(-M // tokens)
        assert 1 <= bad.value <= tiles * ctas * forms[M, N, K][2]  # one a CTA that gave up
        if split:
            assert bad.value == tiles * ctas * forms[M, N, K][2]
        assert kq.kq_read_device_flag(ws) == 0                   # reading clears it
    kq.kq_gemm_i8(q, K, one, w, K, ones, None, M, N, K, kq.F32, y, N, ws, n)
    torch.cuda.synchronize()
    assert kq.kq_read_device_flag(ws) == 0
    rows = torch.arange(0, M, max(1, M // 40), device=DEV)
    want = (q[rows].double() @ w.double().T).float()
    assert torch.equal(y[rows], want)


@pytest.mark.parametrize("changes,text", [(dict(idle=0), "idle=0"), (dict(idle=3), "idle=3"), (dict(limit=999), "wait_limit_ns"),
                                          (dict(limit=10 ** 9 + 1), "wait_limit_ns"), (dict(M=8), "tensor-core path"), (dict(K=0), "K=0")])
def test_refusals(changes, text):
    from gemv_quantize_q8_gb300 import build as kqbuild
    kqbuild.build()
    P = 4096  # stands for a device pointer: nothing is read before the checks
    args = {**dict(q=P, ldq=112, sx=P, w=P, ldw=112, sw=P, M=20, N=5, K=100, y=P, ldy=5, idle=1, limit=10 ** 5, ws=P, n=1 << 20), **changes}
    assert kq.lib().kq_debug_i8_wait_timeout(*args.values(), None) == 1
    assert text in kq.lib().kq_last_error().decode()


def test_forms():
    """What the header says of kq_debug_i8_form: a host estimate, right without a GPU too."""
    assert kq.kq_debug_i8_form(8, 4096, 4096) == (0, 0, 0)
    for M, tokens in ((9, 32), (32, 32), (33, 64), (64, 64), (65, 128), (128, 128)):
        assert kq.kq_debug_i8_form(M, 4096, 4096)[:2] == (1, tokens)
    assert kq.kq_debug_i8_form(2048, 14336, 4096) == (2, 256, 1)
    for K in (1, 128, 256):  # a split leaves each CTA two units of 128 at least
        assert kq.kq_debug_i8_form(20, 300, K)[2] == 1
    with pytest.raises(kq.KqError):
        kq.kq_debug_i8_form(0, 1, 1)
