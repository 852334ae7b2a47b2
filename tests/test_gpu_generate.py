"""The generating example runs; its first tokens are those that the scoring example finds likeliest behind the same prompts."""
import importlib.util
import os
import sys

import pytest
import torch

from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu

FOLDER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples")


def _load(name):
    sys.path.insert(0, FOLDER)
    try:
        spec = importlib.util.spec_from_file_location(name, os.path.join(FOLDER, name + ".py"))
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        return module
    finally:
        sys.path.remove(FOLDER)


def test_example_runs(capsys):
    _load("generate").main()
    assert capsys.readouterr().out.count("prompt of") == 3


def test_next_tokens_are_likely_ones():
    """The cache's keys and values are off by up to half a step, 1/254 of their block's largest (some 1% of a typical element),
    so logits move by a few hundredths: the chosen token is the scoring path's likeliest, or within 0.5 of it."""
    generate = _load("generate")
    m = generate.Decoder(vocab=499, hidden=256, heads=4, kv_heads=2, D=64, max_len=64)
    g = torch.Generator(device=DEV).manual_seed(0)
    prompts = [torch.randint(0, m.vocab, (n,), generator=g, device=DEV) for n in (9, 1, 30)]
    gen = generate.Generator(m, 3, 64, page=16)
    tokens, logprob = gen.prompt(prompts)
    for _ in range(5):
        for b in range(3):
            want = m.logits(prompts[b])[-1].log_softmax(0)
            assert want.max() - want[tokens[b]] < 0.5 and abs(float(want[tokens[b]] - logprob[b])) < 0.5
        prompts = [torch.cat([p, tokens[b : b + 1]]) for b, p in enumerate(prompts)]
        tokens, logprob = gen.step(tokens)
