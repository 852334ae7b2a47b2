"""How many row tiles a prompt attention may have (host checks, no GPU)."""
import pytest

import gemv_quantize_q8_gb300 as kq
from gemv_quantize_q8_gb300 import build as kqbuild
from tests.test_attention_refusals import BAD, PROMPT, SPACE


@pytest.fixture(scope="module")
def lib():
    kqbuild.build()
    return kq.lib()


def documented(B, Tq, n_q, n_kv):
    return (Tq // 64 + B) * n_q + B * n_kv < 2**31


# B, Tq, n_q, n_kv, D
SHAPES = [(1 << 24, 7, 64, 63, 128), (1 << 24, 7, 64, 64, 128), (1 << 24, 7, 120, 120, 128), (1 << 24, 7, 120, 8, 256), (1 << 24, 7, 256, 2, 256),
          (1 << 24, 7, 65535, 65535, 64), (1, 0x7FFFFF00, 32, 8, 128), (1, 0x7FFFFF00, 65535, 1, 128), (1 << 24, 7, 128, 1, 64)]


@pytest.mark.parametrize("B,Tq,n_q,n_kv,D", [s for s in SHAPES if s[2] % s[3] == 0])
@pytest.mark.parametrize("offset", [0, 2])
def test_what_the_header_allows_is_not_refused(lib, B, Tq, n_q, n_kv, D, offset):
    """A workspace that is too small is what is looked at last, and it never helps where there are too many tiles."""
    size = kq.kq_attn_prompt_workspace_bytes(B, Tq, n_q, n_kv, D)
    p, wide = PROMPT["q"] + offset, n_q * D
    changes = dict(q=p, k=p, v=p, y=p, B=B, Tq=Tq, n_q=n_q, n_kv=n_kv, D=D, ldq=wide, ldy=wide, ldk=n_kv * D, ldv=n_kv * D, n=max(size, 1) - 1)
    status = lib.kq_attn_prompt(*{**PROMPT, **changes}.values(), None)
    assert status == SPACE or (status == BAD and "row tiles" in lib.kq_last_error().decode())
    if documented(B, Tq, n_q, n_kv):
        assert size > 0 and status == SPACE
    if size == 0:
        assert status == BAD


@pytest.mark.parametrize("shape", [(1 << 24, 7, 256, 2, 256), (1 << 24, 7, 128, 1, 136), (1 << 24, 7, 65535, 65535, 64), (1, 0x7FFFFF00, 65535, 1, 128)])
def test_no_workspace_for_what_is_refused(shape):
    assert kq.kq_attn_prompt_workspace_bytes(*shape) == 0
    assert kq.kq_attn_prompt_workspace_bytes(shape[0] >> 12 or 1, min(shape[1], 1 << 20), *shape[2:]) > 0
