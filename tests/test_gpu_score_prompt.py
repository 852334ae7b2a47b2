"""The scoring example against the same decoder in plain torch: dequantised int8 products, norms, rotation, log softmax."""
import importlib.util
import os

import pytest
import torch

from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "score_prompt.py")


def _load():
    spec = importlib.util.spec_from_file_location("score_prompt", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _linear(layer, x):
    full = torch.full((1, 1), 127.0, device=DEV)
    amax = x.abs().amax(1, keepdim=True)
    q = torch.round(x * (full / amax))
    y = q.double() @ layer.codes[:, : layer.K].double().T
    return (y * (amax / full).double() * layer.scales.double()).float()


def _heads(m, x, n, gamma):
    x = x.double().reshape(x.shape[0], n, m.D)
    x = x / (x.square().mean(2, keepdim=True) + 1e-6).sqrt() * gamma.double()
    c, s = (t[: x.shape[0]].double()[:, None] for t in (m.cos, m.sin))
    a, b = x.chunk(2, 2)
    return torch.cat([a * c - b * s, b * c + a * s], 2).to(torch.bfloat16).double().repeat_interleave(m.heads // n, 1)


def _plain_logits(m, tokens):
    T, nq, nk = tokens.numel(), m.heads * m.D, m.kv_heads * m.D
    x = m.embed[tokens]
    qkv = _linear(m.qkv, x)
    q, k = _heads(m, qkv[:, :nq], m.heads, m.q_gamma), _heads(m, qkv[:, nq : nq + nk], m.kv_heads, m.k_gamma)
    v = qkv[:, nq + nk :].double().reshape(T, m.kv_heads, m.D).repeat_interleave(m.heads // m.kv_heads, 1)
    s = torch.einsum("qhd,khd->hqk", q, k) * m.D ** -0.5
    s = s.masked_fill(torch.ones((T, T), dtype=torch.bool, device=DEV).triu(1), float("-inf"))
    o = torch.einsum("hqk,khd->qhd", s.softmax(2), v).reshape(T, nq).float()
    return _linear(m.head, x + _linear(m.out, o)).double()


@pytest.mark.parametrize("T", [2, 7, 150])
def test_scores(T):
    """Tolerance: a code of the attention's or the head's input may round the other way (the two sides' sums differ in the
    last bits, and queries and keys by a unit of bf16, 2^-8 relative, in a few elements): each such step moves a logit by
    about scale_x * |w| = (4/127) * 0.07 = 0.002; ten of them in one row bound what is allowed."""
    example = _load()
    m = example.Decoder(vocab=1999, hidden=512, heads=8, kv_heads=2, D=64, max_len=256, seed=T)
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    tokens = torch.randint(0, m.vocab, (T,), generator=g, device=DEV)
    logprob, entropy, ids, best = m.score(tokens, top=4)
    want = _plain_logits(m, tokens)[:-1].log_softmax(1)
    tol = 0.02
    assert (logprob.double() - want.gather(1, tokens[1:, None])[:, 0]).abs().max() < tol
    assert (entropy.double() + (want.exp() * want).sum(1)).abs().max() < tol
    assert (best.double() - want.topk(4, 1).values).abs().max() < tol
    assert (want.gather(1, ids.long()) - want.topk(4, 1).values).abs().max() < 2 * tol
    assert bool((best[:, 0] >= logprob).all()) and bool((best[:, :-1] >= best[:, 1:]).all())


def test_example_runs(capsys):
    _load().main()
    out = capsys.readouterr().out
    assert "perplexity" in out and out.count("position") == 3


def test_prompt_of_one_token():
    """Nothing precedes the only token, so nothing is scored: empty results, not an error."""
    m = _load().Decoder(vocab=199, hidden=128, heads=2, kv_heads=1, D=64, max_len=16)
    logprob, entropy, ids, best = m.score(torch.tensor([7], device=DEV), top=4)
    assert logprob.shape == entropy.shape == (0,) and ids.shape == best.shape == (0, 4)
