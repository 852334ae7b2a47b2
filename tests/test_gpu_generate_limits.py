"""The generating example refuses prompts and steps that it has no room for."""
import pytest
import torch

from tests.gpu_util import DEV
from tests.test_gpu_generate import _load

pytestmark = pytest.mark.gpu


def test_prompts_and_steps_without_room():
    generate = _load("generate")
    m = generate.Decoder(vocab=64, hidden=128, heads=2, kv_heads=1, D=64, max_len=40)
    tokens = lambda n: torch.zeros(n, dtype=torch.int64, device=DEV)  # noqa: E731
    gen = generate.Generator(m, 2, 30, page=16)
    for prompts in ([tokens(3)], [tokens(3), tokens(0)], [tokens(3), tokens(33)]):
        with pytest.raises(ValueError):
            gen.prompt(prompts)
    ids, logprob = gen.prompt([tokens(3), tokens(31)])
    ids, logprob = gen.step(ids)
    assert bool(logprob.isfinite().all())
    with pytest.raises(ValueError, match="33 tokens"):
        gen.step(ids)
    with pytest.raises(ValueError):  # the tables are shorter than the pages
        generate.Generator(m, 1, 48, page=16).prompt([tokens(41)])
