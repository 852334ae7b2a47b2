"""Arguments that the int8 products, the rotation and the log probabilities refuse (host checks, no GPU)."""
import pytest

import gemv_quantize_q8_gb300 as kq
from gemv_quantize_q8_gb300 import build as kqbuild

BAD, TYPE, ALIGN, SPACE = 1, 2, 3, 4
P = 4096  # stands for a device pointer: nothing is read before the checks


@pytest.fixture(scope="module")
def lib():
    kqbuild.build()
    return kq.lib()


def _call(lib, name, args, changes):
    return getattr(lib, name)(*{**args, **changes}.values(), None)


QUANT = dict(xt=kq.F32, x=P, M=3, K=100, ldx=100, q=P, ldq=112, scale=P)
PRODUCT = dict(q=P, ldq=112, sx=P, w=P, ldw=112, sw=P, bias=None, M=3, N=5, K=100, yt=kq.F32, y=P, ldy=5, ws=P, n=1 << 20)
DYN = dict(xt=kq.BF16, x=P, ldx=100, w=P, ldw=112, sw=P, bias=None, M=3, N=5, K=100, yt=kq.F16, y=P, ldy=5, ws=P, n=1 << 20)
QK = dict(xt=kq.F32, q=P, ldq=512, k=P, ldk=128, M=3, n_q=4, n_k=1, D=128, gq=P, gk=P, eps=1e-6, pos=P, cos=P, sin=P,
          n_pos=9, rot=128, pairs=0, yt=kq.F32, qo=P, ldqo=512, ko=P, ldko=128)
LP = dict(xt=kq.F32, x=P, ldx=50, M=3, V=50, t=P, T=1, lp=P, ent=P, k=5, ids=P, top=P)

CASES = [
    ("kq_quantize_i8", QUANT, [
        (dict(xt=kq.Q8_0), TYPE, "x type Q8_0"), (dict(x=None), BAD, "null x"), (dict(q=None), BAD, "null q"),
        (dict(scale=None), BAD, "null scale"), (dict(M=0), BAD, "M=0"), (dict(K=0), BAD, "K=0"),
        (dict(K=131072, ldx=131072, ldq=131072), BAD, "131071"), (dict(ldx=99), BAD, "ldx=99"),
        (dict(ldq=96), BAD, "ldq=96"), (dict(ldq=104), ALIGN, "multiple of 16"), (dict(q=P + 8), ALIGN, "16-byte"),
        (dict(x=P + 2), ALIGN, "x must be"), (dict(scale=P + 2), ALIGN, "scale")]),
    ("kq_gemm_i8", PRODUCT, [
        (dict(yt=kq.Q8_K), TYPE, "y type Q8_K"), (dict(yt=0), TYPE, "y type"), (dict(q=None), BAD, "null q"),
        (dict(sx=None), BAD, "null sx"), (dict(w=None), BAD, "null w"), (dict(sw=None), BAD, "null sw"),
        (dict(y=None), BAD, "null y"), (dict(M=-1), BAD, "M=-1"), (dict(N=0), BAD, "N=0"), (dict(ldy=4), BAD, "ldy=4"),
        (dict(K=131072), BAD, "131071"), (dict(ldw=96), BAD, "ldw=96"), (dict(ldw=100), ALIGN, "ldw"),
        (dict(w=P + 4), ALIGN, "w must be"), (dict(ldq=100), ALIGN, "ldq"), (dict(y=P + 2), ALIGN, "y must be"),
        (dict(bias=P + 1), ALIGN, "bias"), (dict(sx=P + 1), ALIGN, "sx"), (dict(ws=None), SPACE, "workspace"),
        (dict(n=16), SPACE, "16 bytes"), (dict(ws=P + 16), ALIGN, "256-byte")]),
    ("kq_gemm_i8_dyn", DYN, [
        (dict(xt=kq.Q4_K), TYPE, "x type Q4_K"), (dict(x=None), BAD, "null x"), (dict(ldx=64), BAD, "ldx=64"),
        (dict(x=P + 1), ALIGN, "x must be"), (dict(w=None), BAD, "null w"), (dict(N=0), BAD, "N=0"),
        (dict(n=255), SPACE, "255 bytes")]),
    ("kq_qk_norm_rope", QK, [
        (dict(xt=kq.Q8_1), TYPE, "input type Q8_1"), (dict(yt=3), TYPE, "output type Q8_0"), (dict(M=0), BAD, "M=0"),
        (dict(n_q=0, n_k=0), BAD, "heads"), (dict(n_k=-1), BAD, "n_k=-1"), (dict(D=127), BAD, "D=127"),
        (dict(D=1026), BAD, "D=1026"), (dict(rot=130), BAD, "rot=130"), (dict(rot=63), BAD, "rot=63"),
        (dict(pairs=2), BAD, "pairs=2"), (dict(eps=-1.0), BAD, "eps"), (dict(eps=float("nan")), BAD, "eps"),
        (dict(q=None), BAD, "null rows"), (dict(ko=None), BAD, "null rows"), (dict(ldq=511), BAD, "ldq=511"),
        (dict(ldko=127), BAD, "ldko=127"), (dict(pos=None), BAD, "positions"), (dict(n_pos=0), BAD, "n_pos"),
        (dict(q=P + 2), ALIGN, "aligned"), (dict(cos=P + 2), ALIGN, "aligned")]),
    ("kq_logprobs", LP, [
        (dict(xt=kq.Q6_K), TYPE, "logits type Q6_K"), (dict(x=None), BAD, "null logits"), (dict(M=0), BAD, "M=0"),
        (dict(V=0), BAD, "V=0"), (dict(ldx=49), BAD, "ldx=49"), (dict(T=-1), BAD, "n_targets=-1"),
        (dict(T=51), BAD, "n_targets=51"), (dict(t=None), BAD, "targets"), (dict(lp=None), BAD, "targets"),
        (dict(k=33), BAD, "top_k=33"), (dict(V=4, k=5), BAD, "top_k=5"), (dict(ids=None), BAD, "top_ids"),
        (dict(x=P + 2), ALIGN, "aligned"), (dict(ids=P + 2), ALIGN, "aligned")]),
]


@pytest.mark.parametrize("name,args,changes,status,text",
                         [(n, a, ch, st, tx) for n, a, rows in CASES for ch, st, tx in rows])
def test_refused(lib, name, args, changes, status, text):
    before = kq.launch_count()
    assert _call(lib, name, args, changes) == status
    message = lib.kq_last_error().decode()
    assert message.startswith(name) and text in message, message
    assert kq.launch_count() == before


def test_workspace_bytes(lib):
    assert kq.kq_gemm_i8_workspace_bytes(0, 5, 5) == 0 and kq.kq_gemm_i8_workspace_bytes(5, 5, 131072) == 0
    assert 0 < kq.kq_gemm_i8_workspace_bytes(1, 1, 1) <= kq.kq_gemm_i8_workspace_bytes(100, 1, 1000)
