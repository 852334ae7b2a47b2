"""Arguments that the cache's and the attention's calls refuse (host checks, no GPU)."""
import pytest

import gemv_quantize_q8_gb300 as kq
from gemv_quantize_q8_gb300 import build as kqbuild

BAD, TYPE, ALIGN, SPACE = 1, 2, 3, 4
P = 4096  # stands for a device pointer: nothing is read before the checks


@pytest.fixture(scope="module")
def lib():
    kqbuild.build()
    return kq.lib()


APPEND = dict(xt=kq.F32, k=P, ldk=256, v=P, ldv=256, cu=P, lens=P, B=3, T=7, n_kv=2, D=128, pos=P, cos=P, sin=P, n_pos=9, rot=128,
              pairs=0, kc=P, vc=P, ks=P, vs=P, n_pages=5, page=64, table=P, ldt=4)
READ = dict(kc=P, vc=P, ks=P, vs=P, n_pages=5, page=64, table=P, ldt=4, cu=P, lens=P, B=3, T=7, n_kv=2, D=128, yt=kq.BF16, ko=P,
            ldk=256, vo=P, ldv=256)
CACHE = dict(xt=kq.F32, q=P, ldq=512, B=3, n_new=1, n_q=4, n_kv=2, D=128, scale=0.1, kc=P, vc=P, ks=P, vs=P, n_pages=5, page=64,
             table=P, ldt=4, lens=P, yt=kq.F32, y=P, ldy=512, ws=P, n=1 << 30)
PROMPT = dict(xt=kq.BF16, q=P, ldq=512, k=P, ldk=256, v=P, ldv=256, cu_q=P, cu_k=P, B=3, Tq=7, Tk=9, n_q=4, n_kv=2, D=128, scale=0.1,
              causal=1, y=P, ldy=512, ws=P, n=1 << 20)

PAGED = [(dict(kc=None), BAD, "null cache"), (dict(vs=None), BAD, "null cache"), (dict(table=None), BAD, "null table"),
         (dict(lens=None), BAD, "null lens"), (dict(B=0), BAD, "B=0"), (dict(n_kv=0), BAD, "n_kv=0"), (dict(D=0), BAD, "D=0"),
         (dict(D=24), BAD, "D=24"), (dict(D=272), BAD, "D=272"), (dict(page=8), BAD, "page=8"), (dict(page=48), BAD, "page=48"),
         (dict(page=512), BAD, "page=512"), (dict(n_pages=0), BAD, "n_pages=0"), (dict(n_pages=1 << 31), BAD, "n_pages"),
         (dict(ldt=0), BAD, "ldt=0"), (dict(kc=P + 8), ALIGN, "16-byte"), (dict(ks=P + 2), ALIGN, "aligned"),
         (dict(lens=P + 1), ALIGN, "aligned")]
ROWS = [(dict(T=0), BAD, "T=0"), (dict(cu=None), BAD, "multiple of B"), (dict(ldk=255), BAD, "ldk=255"), (dict(ldv=64), BAD, "ldv=64"),
        (dict(cu=P + 2), ALIGN, "aligned")]
CASES = [
    ("kq_kv_append_i8", APPEND, PAGED + ROWS + [
        (dict(xt=kq.Q8_0), TYPE, "row type Q8_0"), (dict(k=None), BAD, "null rows"), (dict(v=None), BAD, "null rows"),
        (dict(rot=130), BAD, "rot=130"), (dict(rot=3), BAD, "rot=3"), (dict(rot=-2), BAD, "rot=-2"), (dict(pairs=2), BAD, "pairs=2"),
        (dict(pos=None), BAD, "positions"), (dict(n_pos=0), BAD, "n_pos"), (dict(k=P + 2), ALIGN, "aligned"),
        (dict(sin=P + 2), ALIGN, "aligned")]),
    ("kq_kv_read_i8", READ, PAGED + ROWS + [
        (dict(yt=kq.Q4_K), TYPE, "row type Q4_K"), (dict(ko=None), BAD, "null rows"), (dict(vo=P + 1), ALIGN, "aligned")]),
    ("kq_attn_cache_i8", CACHE, PAGED + [
        (dict(xt=kq.Q8_1), TYPE, "query type Q8_1"), (dict(yt=3), TYPE, "output type Q8_0"), (dict(q=None), BAD, "null q"),
        (dict(y=None), BAD, "null y"), (dict(n_new=0), BAD, "n_new=0"), (dict(n_q=3), BAD, "n_q=3"), (dict(n_q=0), BAD, "n_q=0"),
        (dict(n_new=20000), BAD, "65536"), (dict(ldq=511), BAD, "ldq=511"), (dict(ldy=511), BAD, "ldy=511"),
        (dict(scale=float("inf")), BAD, "scale"), (dict(scale=float("nan")), BAD, "scale"), (dict(q=P + 2), ALIGN, "aligned"),
        (dict(ws=None), SPACE, "workspace"), (dict(n=16), SPACE, "16 bytes"), (dict(ws=P + 16), ALIGN, "256-byte")]),
    ("kq_attn_prompt", PROMPT, [
        (dict(xt=kq.F32), TYPE, "row type F32"), (dict(xt=kq.Q8_K), TYPE, "row type Q8_K"), (dict(q=None), BAD, "null rows"),
        (dict(v=None), BAD, "null rows"), (dict(cu_q=None), BAD, "null cu_q"), (dict(cu_k=None), BAD, "null cu_k"), (dict(B=0), BAD, "B=0"),
        (dict(Tq=0), BAD, "Tq=0"), (dict(Tk=0), BAD, "Tk=0"), (dict(n_q=3), BAD, "n_q=3"), (dict(n_kv=0), BAD, "n_kv=0"),
        (dict(D=12), BAD, "D=12"), (dict(D=264), BAD, "D=264"), (dict(ldq=511), BAD, "ldq=511"), (dict(ldk=255), BAD, "ldk=255"),
        (dict(ldv=255), BAD, "ldv=255"), (dict(ldy=8), BAD, "ldy=8"), (dict(causal=2), BAD, "causal=2"),
        (dict(scale=float("nan")), BAD, "scale"), (dict(k=P + 1), ALIGN, "aligned"), (dict(cu_k=P + 2), ALIGN, "aligned"),
        (dict(ws=None), SPACE, "workspace"), (dict(n=511), SPACE, "511 bytes"), (dict(ws=P + 64), ALIGN, "256-byte")]),
]


@pytest.mark.parametrize("name,args,changes,status,text", [(n, a, ch, st, tx) for n, a, rows in CASES for ch, st, tx in rows])
def test_refused(lib, name, args, changes, status, text):
    before = kq.launch_count()
    assert set(changes) <= set(args)
    assert getattr(lib, name)(*{**args, **changes}.values(), None) == status
    message = lib.kq_last_error().decode()
    assert message.startswith(name) and text in message, message
    assert kq.launch_count() == before


def test_too_many_row_tiles(lib):
    changes = dict(B=1 << 24, n_q=256, D=256, ldq=1 << 16, ldk=512, ldv=512, ldy=1 << 16, n=1 << 40)
    assert getattr(lib, "kq_attn_prompt")(*{**PROMPT, **changes}.values(), None) == BAD
    assert "row tiles" in lib.kq_last_error().decode()


def test_workspace_bytes(lib):
    assert kq.kq_attn_cache_i8_workspace_bytes(1, 1, 32, 8, 128) > 256
    for shape in ((0, 1, 32, 8, 128), (1, 0, 32, 8, 128), (1, 1, 30, 8, 128), (1, 1, 32, 8, 120), (1, 1, 32, 8, 512)):
        assert kq.kq_attn_cache_i8_workspace_bytes(*shape) == 0
    assert kq.kq_attn_prompt_workspace_bytes(1, 1, 1, 1, 8) >= 8
    for shape in ((0, 1, 4, 2, 128), (1, 0, 4, 2, 128), (1, 1, 3, 2, 128), (1, 1, 4, 2, 4), (1, 1, 4, 2, 320)):
        assert kq.kq_attn_prompt_workspace_bytes(*shape) == 0


@pytest.mark.parametrize("name,args", [("kq_attn_cache_i8", CACHE), ("kq_attn_prompt", PROMPT)])
@pytest.mark.parametrize("scale", [3e38, -2.1e38, float("-inf")])
def test_scales_that_leave_fp32(lib, name, args, scale):
    """The exponent's base is 2: the scale times log2 e has to be finite, too."""
    assert getattr(lib, name)(*{**args, "scale": scale}.values(), None) == BAD
    assert "scale" in lib.kq_last_error().decode()
