"""The operators' cases: the int8 product with scales per token and channel, the log probabilities of given
tokens, and the per-head norms of queries and keys with the position rotation.

``run`` computes a case in its plain form (elementary torch operations in 32 bits) or, with ``own`` set,
through this library's entry points.  Sizes are those of the library's own workloads ([9728 x 2560],
[4096 x 14336], [14336 x 4096]) and generic ones.
"""
import math

import torch

own = False

DEV = "cuda"
FLOATS = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"i8": 1, "f16": 2, "bf16": 2, "f32": 4}

#: The largest listed product (M*N*K), set of logits (M*V) and set of heads (tokens * elements).
MOST_MNK = 2048 * 14336 * 4096
MOST_LOGITS = 2048 * 131072
MOST_SORTED = 64 * 131072
MOST_HEADS = 8192 * 40 * 128


# --------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # One token through a feed-forward product, quantised inside the call: decoding for one user.
        dict(name="i8 1 token", op="i8", M=1, N=9728, K=2560, x="f32", y="f32", bias=False),
        # A handful of users decoding together, rows already quantised, the long reduction of a down product.
        dict(name="i8 5 tokens", op="i8", M=5, N=4096, K=14336, x="i8", y="f32", bias=False),
        # A busy decoding batch with a bias, as query/key/value products have.
        dict(name="i8 48 tokens", op="i8", M=48, N=14336, K=4096, x="bf16", y="bf16", bias=True),
        # A prompt of odd length against odd widths: tiles are cut on every side, rows end inside a vector.
        dict(name="i8 ragged", op="i8", M=777, N=4099, K=4111, x="i8", y="f32", bias=True),
        # A long prompt through the widest product of the prefill workload.
        dict(name="i8 2048 tokens", op="i8", M=2048, N=14336, K=4096, x="bf16", y="bf16", bias=False),
        # One decoded token's alternatives, as a sampling interface returns them.
        dict(name="lp 1 row", op="lp", M=1, V=65536, x="f32", T=1, top=5, masked=False),
        # A batch of decoded tokens with grammar masks (most of the vocabulary at -inf) and 20 alternatives.
        dict(name="lp 64 rows", op="lp", M=64, V=131072, x="bf16", T=1, top=20, masked=True),
        # Multiple choice over an odd vocabulary: three given tokens a row.
        dict(name="lp ragged", op="lp", M=167, V=49999, x="f16", T=3, top=8, masked=False),
        # Scoring a whole prompt (perplexity): no alternatives, the logits as the head product writes them.
        dict(name="lp 2048 rows", op="lp", M=2048, V=131072, x="f32", T=1, top=0, masked=False),
        # One token's heads at decode, from the fp32 product into a bf16 cache row.
        dict(name="qk 1 token", op="qk", M=1, Hq=32, Hk=8, D=128, rot=128, pairs=False, x="f32", y="bf16"),
        # Odd numbers of heads, a head width that is no power of two, half of it rotated, neighbours paired.
        dict(name="qk ragged", op="qk", M=1001, Hq=14, Hk=2, D=80, rot=40, pairs=True, x="f16", y="f16"),
        # A long prompt.
        dict(name="qk 8192 tokens", op="qk", M=8192, Hq=32, Hk=8, D=128, rot=128, pairs=False, x="f32", y="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number in lo..hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["i8", "i8", "lp", "qk"])
    if op == "i8":
        while True:
            M, N, K = _log(rng, 1, 2048), _log(rng, 64, 14336), _log(rng, 64, 14336)
            if M * N * K <= MOST_MNK:
                return dict(op=op, M=M, N=N, K=K, x=rng.choice(["i8", "f32", "f16", "bf16"]),
                            y=rng.choice(["f32", "f16", "bf16"]), bias=rng.random() < 0.5)
    if op == "lp":
        while True:
            M, V = _log(rng, 1, 2048), _log(rng, 1000, 131072)
            top = rng.choice([0, 1, 5, 20, 32])
            if M * V <= (MOST_SORTED if top else MOST_LOGITS):
                return dict(op=op, M=M, V=V, x=rng.choice(["f32", "f16", "bf16"]), T=rng.choice([1, 1, 4]), top=top,
                            masked=rng.random() < 0.3)
    while True:
        M, Hk, D = _log(rng, 1, 8192), rng.choice([1, 2, 4, 8]), rng.choice([64, 80, 96, 128, 256])
        Hq = Hk * rng.choice([1, 3, 4, 7])
        if M * (Hq + Hk) * D <= MOST_HEADS:
            return dict(op=op, M=M, Hq=Hq, Hk=Hk, D=D, rot=rng.choice([D, D, D // 2]), pairs=rng.random() < 0.4,
                        x=rng.choice(["f32", "f16", "bf16"]), y=rng.choice(["f32", "f16", "bf16"]))


# --------------------------------------------------------------------------------------------- the inputs
def _up16(k):
    return (k + 15) // 16 * 16


def _codes(v):
    """Whole numbers of -127..127 and their scale for each row of v, and the rows' ends padded to 16 bytes."""
    s = v.abs().amax(1, keepdim=True) / 127
    q = torch.zeros((v.shape[0], _up16(v.shape[1])), dtype=torch.int8, device=v.device)
    q[:, : v.shape[1]] = torch.round(v / s).to(torch.int8)
    return q, s[:, 0].contiguous()


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    c = case
    s = {"case": c}
    if c["op"] == "i8":
        x = normal(c["M"], c["K"])
        x = torch.where(torch.rand(x.shape, generator=g, device=DEV) < 0.01, x * 10, x)  # outliers
        if c["x"] == "i8":
            s["q"], s["sx"] = _codes(x)
        else:
            s["x"] = x.to(FLOATS[c["x"]])
        s["w"], s["sw"] = _codes(normal(c["N"], c["K"]) * 0.02)
        s["bias"] = normal(c["N"]) if c["bias"] else None
    elif c["op"] == "lp":
        x = normal(c["M"], c["V"]) * 2.5
        if c["masked"]:  # a grammar leaves about 300 tokens of a row
            x = x.masked_fill(torch.rand(x.shape, generator=g, device=DEV) * c["V"] > 300, -math.inf)
        s["x"] = x.to(FLOATS[c["x"]])
        s["t"] = torch.randint(0, c["V"], (c["M"], c["T"]), generator=g, device=DEV, dtype=torch.int32)
        if c["masked"]:  # the given tokens are among those that the grammar leaves
            at = torch.arange(c["M"], device=DEV)[:, None]
            s["x"][at, s["t"].long()] = normal(c["M"], c["T"]).to(s["x"].dtype)
    else:
        # one row of the q/k/v product for each token: the query heads, the key heads, the value heads
        s["qkv"] = normal(c["M"], (c["Hq"] + 2 * c["Hk"]) * c["D"]).to(FLOATS[c["x"]])
        s["gq"], s["gk"] = 1 + 0.2 * normal(c["D"]), 1 + 0.2 * normal(c["D"])
        start = int(torch.randint(0, 16384, (1,), generator=g, device=DEV))
        s["pos"] = torch.arange(start, start + c["M"], device=DEV, dtype=torch.int32)
        i = torch.arange(c["rot"] // 2, device=DEV, dtype=torch.float64)
        a = torch.arange(32768, device=DEV, dtype=torch.float64)[:, None] * 1e6 ** (-2 * i / c["rot"])
        s["cos"], s["sin"] = a.cos().float(), a.sin().float()
        s["eps"] = 1e-6
    return s


# --------------------------------------------------------------------------------------------- plain forms
def _plain_i8(s, c):
    if c["x"] == "i8":
        q, sx = s["q"][:, : c["K"]].float(), s["sx"][:, None]
    else:
        x = s["x"].float()
        amax, full = x.abs().amax(1, keepdim=True), torch.full((1, 1), 127.0, device=x.device)
        q, sx = torch.round(x * (full / amax)), amax / full
    y = (q @ s["w"][:, : c["K"]].float().T) * sx * s["sw"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(FLOATS[c["y"]])


def _plain_lp(s, c):
    x, t = s["x"].float(), s["t"].long()
    d = x - x.amax(1, keepdim=True)
    e = d.exp()
    total = e.sum(1, keepdim=True)
    log_total = total.log()
    lp = d.gather(1, t) - log_total
    entropy = log_total[:, 0] - torch.where(e > 0, e * d, 0).sum(1) / total[:, 0]
    if not c["top"]:
        return {"logprob": lp, "entropy": entropy}
    ids = x.sort(dim=1, descending=True, stable=True).indices[:, : c["top"]]  # the lowest id first among equals
    return {"logprob": lp, "entropy": entropy, "ids": ids.int(), "top": d.gather(1, ids) - log_total}


def _plain_heads(x, gamma, s, c):
    x = x.float().reshape(c["M"], -1, c["D"])
    x = x * (x.square().mean(2, keepdim=True) + s["eps"]).rsqrt() * gamma
    cos, sin = s["cos"][s["pos"].long()][:, None], s["sin"][s["pos"].long()][:, None]
    r, rest = x[..., : c["rot"]], x[..., c["rot"] :]
    if c["pairs"]:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], 3).flatten(2)
    else:
        a, b = r.chunk(2, 2)
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], 2)
    return torch.cat([r, rest], 2).flatten(1).to(FLOATS[c["y"]])


def _plain_qk(s, c):
    nq, nk = c["Hq"] * c["D"], c["Hk"] * c["D"]
    return {"q": _plain_heads(s["qkv"][:, :nq], s["gq"], s, c), "k": _plain_heads(s["qkv"][:, nq : nq + nk], s["gk"], s, c)}


# --------------------------------------------------------------------------------------------- the kernels
def _types(kq):
    return {"f32": kq.F32, "f16": kq.F16, "bf16": kq.BF16}


def _buffers(s, c, kq):
    """The outputs and the workspace that a program keeps from call to call."""
    if c["op"] == "i8":
        n = kq.kq_gemm_i8_workspace_bytes(c["M"], c["N"], c["K"])
        return {"y": torch.empty((c["M"], c["N"]), dtype=FLOATS[c["y"]], device=DEV),
                "ws": torch.zeros(n, dtype=torch.uint8, device=DEV), "n": n}
    if c["op"] == "lp":
        k = min(c["top"], c["V"])
        out = {"logprob": torch.empty((c["M"], c["T"]), device=DEV), "entropy": torch.empty(c["M"], device=DEV)}
        if k:
            out["ids"] = torch.empty((c["M"], k), dtype=torch.int32, device=DEV)
            out["top"] = torch.empty((c["M"], k), device=DEV)
        return out
    return {h: torch.empty((c["M"], c[n] * c["D"]), dtype=FLOATS[c["y"]], device=DEV) for h, n in (("q", "Hq"), ("k", "Hk"))}


def _run_own(s, c):
    import gemv_quantize_q8_gb300 as kq

    types = _types(kq)
    if "buffers" not in s:
        s["buffers"] = _buffers(s, c, kq)
    b = s["buffers"]
    M = c["M"]
    if c["op"] == "i8":
        N, K, w = c["N"], c["K"], s["w"]
        if c["x"] == "i8":
            kq.kq_gemm_i8(s["q"], s["q"].shape[1], s["sx"], w, w.shape[1], s["sw"], s["bias"], M, N, K, types[c["y"]],
                          b["y"], N, b["ws"], b["n"])
        else:
            kq.kq_gemm_i8_dyn(types[c["x"]], s["x"], K, w, w.shape[1], s["sw"], s["bias"], M, N, K, types[c["y"]],
                              b["y"], N, b["ws"], b["n"])
        return b["y"]
    if c["op"] == "lp":
        k = min(c["top"], c["V"])
        kq.kq_logprobs(types[c["x"]], s["x"], c["V"], M, c["V"], s["t"], c["T"], b["logprob"], b["entropy"], k,
                       b.get("ids"), b.get("top"))
        return b
    nq, row = c["Hq"] * c["D"], s["qkv"].shape[1]
    kq.kq_qk_norm_rope(types[c["x"]], s["qkv"], row, s["qkv"][:, nq:], row, M, c["Hq"], c["Hk"], c["D"], s["gq"], s["gk"],
                       s["eps"], s["pos"], s["cos"], s["sin"], 32768, c["rot"], int(c["pairs"]), types[c["y"]],
                       b["q"], nq, b["k"], c["Hk"] * c["D"])
    return b


def run(state):
    c = state["case"]
    if own:
        return _run_own(state, c)
    return {"i8": _plain_i8, "lp": _plain_lp, "qk": _plain_qk}[c["op"]](state, c)


# --------------------------------------------------------------------------------------------- the measure
def work(case):
    c = case
    M = c["M"]
    if c["op"] == "i8":
        N, K = c["N"], c["K"]
        read = M * K * SIZE[c["x"]] + N * K + 4 * N + (4 * M if c["x"] == "i8" else 0) + (4 * N if c["bias"] else 0)
        return {"bytes": read + M * N * SIZE[c["y"]], "flops": 2 * M * N * K}
    if c["op"] == "lp":
        n = M * c["V"]
        return {"bytes": n * SIZE[c["x"]] + M * (8 * c["T"] + 4 + 8 * min(c["top"], c["V"])), "flops": 6 * n}
    n = M * (c["Hq"] + c["Hk"]) * c["D"]
    return {"bytes": n * (SIZE[c["x"]] + SIZE[c["y"]]) + M * 4 * (1 + c["rot"]) + 8 * c["D"], "flops": 7 * n}


# --------------------------------------------------------------------------------------------- in 64 bits
def _exact_i8(s, c):
    if c["x"] == "i8":
        q, sx = s["q"][:, : c["K"]].double(), s["sx"].double()
    else:
        # the codes are whole numbers that the definition fixes in 32 bits; all that follows is in 64
        x = s["x"].to(torch.float32)
        largest = torch.maximum(x.amax(1), -x.amin(1))
        inverse = torch.div(torch.full_like(largest, 127), largest)
        q, sx = torch.round(torch.einsum("mk,m->mk", x, inverse)).double(), largest.double() / 127
    y = torch.einsum("mk,nk->mn", q, s["w"][:, : c["K"]].double()) * torch.outer(sx, s["sw"].double())
    return y if s["bias"] is None else y + s["bias"].double()


def _exact_lp(s, c):
    x, t = s["x"].double(), s["t"].long()
    log_z = torch.logsumexp(x, 1)
    p = torch.exp(x - log_z[:, None])
    entropy = -torch.xlogy(p, p).sum(1)
    out = {"logprob": torch.gather(x, 1, t) - log_z[:, None], "entropy": entropy}
    if c["top"]:
        out["ids"] = None
        out["top"] = torch.topk(x, min(c["top"], c["V"]), 1).values - log_z[:, None]
    return out


def _exact_heads(x, gamma, s, c):
    M, D, half = c["M"], c["D"], c["rot"] // 2
    x = x.double().view(M, -1, D)
    x = x / torch.sqrt(torch.linalg.vecdot(x, x)[..., None] / D + s["eps"]) * gamma.double()
    turn = torch.complex(s["cos"].double(), s["sin"].double())[s["pos"].long()][:, None]
    first = torch.arange(half, device=x.device) * (2 if c["pairs"] else 1)
    second = first + (1 if c["pairs"] else half)
    z = torch.complex(x[..., first], x[..., second]) * turn
    x[..., first], x[..., second] = z.real, z.imag
    return x.reshape(M, -1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "i8":
        return _exact_i8(s, c)
    if c["op"] == "lp":
        return _exact_lp(s, c)
    nq, nk = c["Hq"] * c["D"], c["Hk"] * c["D"]
    return {"q": _exact_heads(s["qkv"][:, :nq], s["gq"], s, c), "k": _exact_heads(s["qkv"][:, nq : nq + nk], s["gk"], s, c)}
