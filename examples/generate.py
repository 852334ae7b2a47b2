"""Generates tokens with the one-layer decoder of score_prompt.py for several prompts at once: packed prompts first, then
a token each a step, keys and values in a paged cache of 8-bit codes.

    python examples/generate.py

What the example shows is how the calls fit together:
    queries, keys        kq_qk_norm_rope (norms; the queries' rotation)
    prompts              kq_kv_append_i8 (the keys' rotation on the way), kq_kv_read_i8 and kq_attn_prompt: the prompt attends what
                         the cache holds, as its continuation will
    steps                kq_kv_append_i8, kq_attn_cache_i8
    next tokens          kq_logprobs (the likeliest one)
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from score_prompt import DEV, Decoder, kq  # noqa: E402


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


class Generator:
    def __init__(self, model: Decoder, batch: int, max_len: int, page: int = 64):
        self.m, self.B, self.page = model, batch, page
        self.width = -(-max_len // page)  # pages of a sequence
        n = batch * self.width
        self.table = torch.arange(n, dtype=torch.int32, device=DEV).view(batch, self.width)
        self.codes = torch.zeros((2, n, model.kv_heads, page, model.D), dtype=torch.int8, device=DEV)
        self.scales = torch.zeros((2, n, model.kv_heads), device=DEV)
        self.cache = (self.codes[0], self.codes[1], self.scales[0], self.scales[1], n, page, self.table, self.width)
        self.lens = torch.zeros(batch, dtype=torch.int32, device=DEV)
        self.room, self.longest = min(self.width * page, model.max_len), 0

    def _grow(self, longest):
        """A token past the last page would have no place, and one past the tables no angle."""
        if longest > self.room:
            raise ValueError(f"{longest} tokens; the cache and the rotation's tables have room for {self.room}")
        self.longest = longest

    def _heads(self, tokens, pos, cu):
        """The residual, rotated queries in bf16; keys and values go to the cache."""
        m, T = self.m, tokens.numel()
        nq, nk = m.heads * m.D, m.kv_heads * m.D
        x = m.embed[tokens]
        qkv = m.qkv(x)
        ld = qkv.stride(0)
        q, k = (torch.empty((T, n), dtype=t, device=DEV) for n, t in ((nq, torch.bfloat16), (nk, torch.float32)))
        kq.kq_qk_norm_rope(kq.F32, qkv, ld, None, 0, T, m.heads, 0, m.D, m.q_gamma, None, 1e-6, pos, m.cos, m.sin, m.max_len, m.D, 0,
                           kq.BF16, q, nq, None, 0)
        kq.kq_qk_norm_rope(kq.F32, None, 0, qkv[:, nq:], ld, T, 0, m.kv_heads, m.D, None, m.k_gamma, 1e-6, None, None, None, 0, 0, 0,
                           kq.F32, None, 0, k, nk)
        kq.kq_kv_append_i8(kq.F32, k, nk, qkv[:, nq + nk :], ld, cu, self.lens, self.B, T, m.kv_heads, m.D, pos, m.cos, m.sin, m.max_len,
                           m.D, 0, *self.cache)
        return x, q

    def _next(self, x, o):
        """The likeliest token behind every row, and its log probability."""
        m, T = self.m, x.shape[0]
        logits = m.head(x + m.out(o.float()))
        ids, best = torch.empty((T, 1), dtype=torch.int32, device=DEV), torch.empty((T, 1), device=DEV)
        kq.kq_logprobs(kq.F32, logits, m.vocab, T, m.vocab, None, 0, None, None, 1, ids, best)
        return ids[:, 0].long(), best[:, 0]

    def prompt(self, prompts):
        m, new = self.m, [len(p) for p in prompts]
        if len(new) != self.B or min(new) < 1:
            raise ValueError(f"need {self.B} prompts of a token at least")
        self._grow(max(new))
        T, nq, nk = sum(new), m.heads * m.D, m.kv_heads * m.D
        cu = _ints([0] + torch.tensor(new).cumsum(0).tolist())
        self.lens.copy_(_ints(new))
        pos = _ints([i for n in new for i in range(n)])
        x, q = self._heads(torch.cat(prompts), pos, cu)
        k, v = (torch.empty((T, nk), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        kq.kq_kv_read_i8(*self.cache, cu, self.lens, self.B, T, m.kv_heads, m.D, kq.BF16, k, nk, v, nk)
        n = kq.kq_attn_prompt_workspace_bytes(self.B, T, m.heads, m.kv_heads, m.D)
        o = torch.empty_like(q)
        kq.kq_attn_prompt(kq.BF16, q, nq, k, nk, v, nk, cu, cu, self.B, T, T, m.heads, m.kv_heads, m.D, m.D ** -0.5, 1, o, nq,
                          torch.empty(n, dtype=torch.uint8, device=DEV), n)
        last = cu[1:].long() - 1
        return self._next(x[last], o[last])

    def step(self, tokens):
        m, nq = self.m, self.m.heads * self.m.D
        self._grow(self.longest + 1)
        pos = self.lens.clone()
        self.lens += 1
        x, q = self._heads(tokens, pos, None)
        n = kq.kq_attn_cache_i8_workspace_bytes(self.B, 1, m.heads, m.kv_heads, m.D)
        o = torch.empty_like(q)
        kq.kq_attn_cache_i8(kq.BF16, q, nq, self.B, 1, m.heads, m.kv_heads, m.D, m.D ** -0.5, *self.cache, self.lens, kq.BF16, o, nq,
                            torch.empty(n, dtype=torch.uint8, device=DEV), n)
        return self._next(x, o)


def main():
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    model = Decoder()
    prompts = [torch.randint(0, model.vocab, (n,), generator=g, device=DEV) for n in (70, 5, 233)]
    gen = Generator(model, len(prompts), 400)
    tokens, logprob = gen.prompt(prompts)
    out, total = [tokens], logprob
    for _ in range(24):
        tokens, logprob = gen.step(tokens)
        out.append(tokens)
        total = total + logprob
    for b, p in enumerate(prompts):
        print(f"prompt of {len(p)}: {' '.join(str(t[b].item()) for t in out[:12])} .. ({total[b].item():.2f} in all)")


if __name__ == "__main__":
    main()
