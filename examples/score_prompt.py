"""Scores a prompt with a one-layer decoder whose products are int8 with scales per token and per channel:
log probabilities of the prompt's own tokens (its perplexity), the entropy at every position and the likeliest
alternatives.

    python examples/score_prompt.py

Random weights stand for a model; what the example shows is how the calls fit together:
    weights            kq_quantize_i8 (a row of weights has one scale, as a token has)
    q/k/v, output,
    head products      kq_gemm_i8_dyn (rows quantised on the way)
    norms, rotation    kq_qk_norm_rope (from the product's fp32 rows into bf16 queries and keys)
    scores             kq_logprobs (on the head product's fp32 rows)
Attention itself is left to PyTorch.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gemv_quantize_q8_gb300 as kq  # noqa: E402

DEV = "cuda"


class Int8Linear:
    """y = x @ w.T with int8 weights (one scale a row of w) and rows of x quantised in the call."""

    def __init__(self, w: torch.Tensor):
        self.N, self.K = w.shape
        self.ld = (self.K + 15) // 16 * 16
        self.codes = torch.empty((self.N, self.ld), dtype=torch.int8, device=DEV)
        self.scales = torch.empty(self.N, device=DEV)
        kq.kq_quantize_i8(kq.F32, w.float().contiguous(), self.N, self.K, self.K, self.codes, self.ld, self.scales)

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        M = x.shape[0]
        y = torch.empty((M, self.N), device=DEV)
        n = kq.kq_gemm_i8_workspace_bytes(M, self.N, self.K)
        kq.kq_gemm_i8_dyn(kq.F32, x, x.stride(0), self.codes, self.ld, self.scales, None, M, self.N, self.K, kq.F32, y,
                          self.N, torch.empty(n, dtype=torch.uint8, device=DEV), n)
        return y


class Decoder:
    def __init__(self, vocab=32000, hidden=2048, heads=16, kv_heads=4, D=128, max_len=4096, seed=0):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
        self.heads, self.kv_heads, self.D, self.vocab, self.max_len = heads, kv_heads, D, vocab, max_len
        self.embed = rand(vocab, hidden)
        self.qkv = Int8Linear(rand((heads + 2 * kv_heads) * D, hidden) * hidden ** -0.5)
        self.out = Int8Linear(rand(hidden, heads * D) * (heads * D) ** -0.5)
        self.head = Int8Linear(rand(vocab, hidden) * 3 * hidden ** -0.5)
        self.q_gamma, self.k_gamma = 1 + 0.1 * rand(D), 1 + 0.1 * rand(D)
        angle = torch.arange(max_len, device=DEV, dtype=torch.float64)[:, None] * 1e4 ** (
            -torch.arange(0, D, 2, device=DEV, dtype=torch.float64) / D)
        self.cos, self.sin = angle.cos().float(), angle.sin().float()

    def logits(self, tokens: torch.Tensor) -> torch.Tensor:
        T, D, nq, nk = tokens.numel(), self.D, self.heads * self.D, self.kv_heads * self.D
        x = self.embed[tokens]
        qkv = self.qkv(x)
        q = torch.empty((T, nq), dtype=torch.bfloat16, device=DEV)
        k = torch.empty((T, nk), dtype=torch.bfloat16, device=DEV)
        ld = qkv.stride(0)
        kq.kq_qk_norm_rope(kq.F32, qkv, ld, qkv[:, nq:], ld, T, self.heads, self.kv_heads, D, self.q_gamma, self.k_gamma, 1e-6,
                           torch.arange(T, device=DEV, dtype=torch.int32), self.cos, self.sin, self.max_len, D, 0, kq.BF16,
                           q, nq, k, nk)
        v = qkv[:, nq + nk :].reshape(T, self.kv_heads, D).repeat_interleave(self.heads // self.kv_heads, 1)
        q, k = q.float().reshape(T, self.heads, D), k.float().reshape(T, self.kv_heads, D)
        k = k.repeat_interleave(self.heads // self.kv_heads, 1)
        s = torch.einsum("qhd,khd->hqk", q, k) * D ** -0.5
        s = s.masked_fill(torch.ones((T, T), dtype=torch.bool, device=DEV).triu(1), float("-inf"))
        o = torch.einsum("hqk,khd->qhd", s.softmax(2), v).reshape(T, nq)
        return self.head(x + self.out(o))

    def score(self, tokens: torch.Tensor, top: int = 5):
        """Log probabilities of tokens[1:], entropies, and the `top` likeliest ids with theirs."""
        logits, M = self.logits(tokens), tokens.numel() - 1
        given = tokens[1:].int().contiguous()
        logprob, entropy = torch.empty(M, device=DEV), torch.empty(M, device=DEV)
        ids, best = torch.empty((M, top), dtype=torch.int32, device=DEV), torch.empty((M, top), device=DEV)
        if M:  # (the only token of a prompt follows nothing)
            kq.kq_logprobs(kq.F32, logits, self.vocab, M, self.vocab, given, 1, logprob, entropy, top, ids, best)
        return logprob, entropy, ids, best


def main():
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    model = Decoder()
    tokens = torch.randint(0, model.vocab, (200,), generator=g, device=DEV)
    logprob, entropy, ids, best = model.score(tokens)
    print(f"{tokens.numel()} tokens: perplexity {logprob.mean().neg().exp().item():.1f}, mean entropy {entropy.mean().item():.3f}")
    for t in (0, 100, 198):
        tops = ", ".join(f"{i} ({p:.2f})" for i, p in zip(ids[t].tolist(), best[t].tolist()))
        print(f"position {t}: given {tokens[t + 1].item()} ({logprob[t].item():.2f}); likeliest {tops}")


if __name__ == "__main__":
    main()
