"""Every limit of the int8 products, the rotation and the log probabilities is refused one step past it and stated in the
header (host checks, no GPU)."""
import os
import re

import pytest

import gemv_quantize_q8_gb300 as kq
from gemv_quantize_q8_gb300 import build as kqbuild
from tests.test_i8_refusals import BAD, DYN, LP, PRODUCT, QK, QUANT, _call

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "kq.h")
SECTION = "int8 products with one scale per token"


def _comment(name):
    """What the header says of a function: its own comment and, for the products, their section's."""
    text = open(HEADER).read()
    upto = text[: text.index(f" {name}(")]
    own = upto[upto.rindex("/*") :]
    if "i8" in name:
        own += text[text.index(SECTION) : text.index("*/", text.index(SECTION))]
    return re.sub(r"\s+\*?\s*", " ", own)


PAST = [
    ("kq_quantize_i8", QUANT, dict(M=2 ** 31 - 255), "M and N are 1 .. 2^31 - 256"),
    ("kq_quantize_i8", QUANT, dict(K=131072, ldx=131072, ldq=131072), "1 to 131071"),
    ("kq_gemm_i8", PRODUCT, dict(N=2 ** 31 - 255, ldy=2 ** 31), "M and N are 1 .. 2^31 - 256"),
    ("kq_gemm_i8_dyn", DYN, dict(M=2 ** 31 - 255), "M and N are 1 .. 2^31 - 256"),
    ("kq_qk_norm_rope", QK, dict(n_q=65537, ldq=1 << 40, ldqo=1 << 40), "n_q and n_k are at most 65536 each"),
    ("kq_qk_norm_rope", QK, dict(n_k=65537, ldk=1 << 40, ldko=1 << 40), "n_q and n_k are at most 65536 each"),
    ("kq_qk_norm_rope", QK, dict(M=(1 << 31) // 5 + 1), "M*(n_q + n_k) is below 2^31"),
    ("kq_qk_norm_rope", QK, dict(eps=float("inf")), "eps is finite and not negative"),
    ("kq_qk_norm_rope", QK, dict(D=1026, ldq=1 << 20, ldk=1 << 20, ldqo=1 << 20, ldko=1 << 20), "D is even, 2 .. 1024"),
    ("kq_logprobs", LP, dict(T=51), "n_targets is 0 .. V"),
    ("kq_logprobs", LP, dict(k=33), "top_k is 0 .. 32"),
    ("kq_logprobs", LP, dict(V=(1 << 30) + 1, ldx=1 << 31), "V is 1 .. 2^30"),
    ("kq_logprobs", LP, dict(M=1 << 31), "M 1 .. 2^31 - 1"),
]


@pytest.fixture(scope="module")
def lib():
    kqbuild.build()
    return kq.lib()


@pytest.mark.parametrize("name,args,changes,stated", PAST)
def test_limit_is_refused_and_stated(lib, name, args, changes, stated):
    assert _call(lib, name, args, changes) == BAD, lib.kq_last_error()
    assert stated in _comment(name)


def test_workspaces_grow_with_the_shape(lib):
    """What the header promises of the workspace: 0 for a refused shape, never less for more."""
    assert "0 for one that they refuse" in _comment("kq_gemm_i8_workspace_bytes")
    sizes = [1, 2, 8, 9, 16, 63, 64, 65, 128, 129, 1000]
    for K in (1, 15, 16, 17, 64, 65, 131071):
        n = [kq.kq_gemm_i8_workspace_bytes(M, 5, K) for M in sizes]
        assert n == sorted(n) and n[0] > 0
    for M in sizes:
        n = [kq.kq_gemm_i8_workspace_bytes(M, 5, K) for K in range(1, 300)]
        assert n == sorted(n)
    assert kq.kq_gemm_i8_workspace_bytes(1, 1, 131072) == 0
