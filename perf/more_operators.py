"""The cases of attention and its cache: appending to a paged cache of 8-bit codes (with the position rotation)
and reading it back, attention of a few tokens over that cache, and attention over whole prompts.

``run`` computes a case in its plain form (elementary torch operations in 32 bits) or, with ``own`` set,
through this library's entry points.  Head layouts (32 over 8 of 128 elements, 14 over 2 of 80) are those of the
library's other workloads, the rest is generic.

The cache: a page holds `page` consecutive tokens of a sequence, keys and values each [n_pages][heads][page][D]
int8 with one fp32 scale for a page and head; table[b][i] is sequence b's i-th page.
"""
import math
import random

import torch

own = False

DEV = "cuda"
FLOATS = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}
N_POS = 32768  # positions that the angle tables cover

#: The largest listed append (elements of the new rows), cache (elements) and prompt (query/key pairs * heads * D).
MOST_APPENDED = 8192 * 2 * 8 * 128
MOST_TOUCHED = 64 * 64 * 2 * 8 * 128
MOST_CACHED = 2 * 131072 * 2 * 8 * 128
MOST_PAIRS = 16384 * 16385 // 2 * 32 * 128


# --------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # One decoded token of one user into a part-filled page, from the fp32 product's rows.
        dict(name="append 1 token", op="append", B=1, new=1, past=1000, even=True, Hk=8, D=128, rot=128, pairs=False, x="f32",
             page=64, y="bf16"),
        # A decoding batch: one token each, short pages.
        dict(name="append 64 users", op="append", B=64, new=1, past=2000, even=False, Hk=8, D=128, rot=128, pairs=False, x="bf16",
             page=16, y="bf16"),
        # Packed prompts of different lengths behind pasts that end inside pages; half of 80 elements rotated, neighbours paired.
        dict(name="append ragged", op="append", B=7, new=301, past=77, even=False, Hk=2, D=80, rot=40, pairs=True, x="f16", page=32,
             y="f16"),
        # A long prompt's keys and values, and the rows back as a later part of the prompt would attend them.
        dict(name="append 8192 tokens", op="append", B=1, new=8192, past=0, even=True, Hk=8, D=128, rot=128, pairs=False, x="f32",
             page=64, y="bf16"),
        # One user's next token: the smallest call.
        dict(name="cache 1 user", op="cache", B=1, new=1, len=900, even=True, Hq=32, Hk=8, D=128, page=64, x="bf16", y="bf16"),
        # Three draft tokens each for five users, odd numbers of heads, fp32 queries and outputs.
        dict(name="cache drafts", op="cache", B=5, new=3, len=5001, even=False, Hq=14, Hk=2, D=80, page=32, x="f32", y="f32"),
        # A decoding batch of users at different lengths.
        dict(name="cache 64 users", op="cache", B=64, new=1, len=8192, even=False, Hq=32, Hk=8, D=128, page=16, x="bf16", y="bf16"),
        # Two long documents in the cache.
        dict(name="cache long", op="cache", B=2, new=1, len=131072, even=True, Hq=32, Hk=8, D=128, page=64, x="f16", y="f16"),
        # A short question.
        dict(name="prompt short", op="prompt", B=1, len=37, past=0, even=True, Hq=32, Hk=8, D=128, causal=True, x="bf16"),
        # Packed prompts of different lengths, heads of 80.
        dict(name="prompt packed", op="prompt", B=9, len=1501, past=0, even=False, Hq=14, Hk=2, D=80, causal=True, x="f16"),
        # The next 1024 tokens of prompts that are partly in the cache already.
        dict(name="prompt chunk", op="prompt", B=4, len=1024, past=4096, even=False, Hq=32, Hk=8, D=128, causal=True, x="bf16"),
        # A long prompt.
        dict(name="prompt 16384", op="prompt", B=1, len=16384, past=0, even=True, Hq=32, Hk=8, D=128, causal=True, x="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number in lo..hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "cache", "cache", "prompt", "prompt"])
    while True:
        c = dict(op=op, B=_log(rng, 1, 64), even=rng.random() < 0.3, Hk=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 80, 96, 128, 128, 256]))
        if op == "append":
            c.update(new=rng.choice([1, _log(rng, 1, 8192)]), past=_log(rng, 1, 4096) - 1, rot=rng.choice([c["D"], c["D"], c["D"] // 2]),
                     pairs=rng.random() < 0.4, x=rng.choice(["f32", "f16", "bf16"]), page=rng.choice([16, 32, 64, 128]),
                     y=rng.choice(["f32", "f16", "bf16"]))
            touched = (c["new"] + c["page"]) * c["B"] * 2 * c["Hk"] * c["D"]
            if touched <= MOST_APPENDED + MOST_TOUCHED:
                return c
            continue
        c["Hq"] = c["Hk"] * rng.choice([1, 2, 4, 7, 8])
        if op == "cache":
            c.update(new=rng.choice([1, 1, 1, 2, 3, 5, 8]), len=_log(rng, 9, 131072), page=rng.choice([16, 32, 64, 128]),
                     x=rng.choice(["f32", "f16", "bf16"]), y=rng.choice(["f32", "f16", "bf16"]))
            if c["B"] * c["len"] * 2 * c["Hk"] * c["D"] <= MOST_CACHED and c["Hq"] * c["new"] <= 128:
                return c
            continue
        c.update(len=_log(rng, 1, 16384), past=rng.choice([0, 0, _log(rng, 1, 16384)]), causal=rng.random() < 0.8,
                 x=rng.choice(["f16", "bf16"]), D=rng.choice([64, 80, 96, 128, 128]))
        if c["B"] * c["len"] * (c["len"] + c["past"]) * c["Hq"] * c["D"] <= MOST_PAIRS:
            return c


def _lengths(c, most, least=1):
    """Every sequence's length: all `most`, or spread over least..most (one of them `most`)."""
    rng = random.Random(f"{c['B']} {most} {c['Hk']} {c['D']}")
    return [most if c["even"] or b == c["B"] // 2 else rng.randint(least, most) for b in range(c["B"])]


def _plan(c):
    """(new tokens, all tokens) of every sequence."""
    if c["op"] == "cache":
        lens = _lengths(c, c["len"], min(c["new"], c["len"]))
        return [c["new"]] * c["B"], [max(n, c["new"]) for n in lens]
    new = _lengths(c, c["new"] if c["op"] == "append" else c["len"])
    past = [0] * c["B"] if not c["past"] else _lengths(c, c["past"], 0)
    return new, [n + p for n, p in zip(new, past)]


# --------------------------------------------------------------------------------------------- the inputs
def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _sums(values):
    out = [0]
    for v in values:
        out.append(out[-1] + v)
    return out


def _pages(c, total, g):
    """The table of a pool whose pages are handed out in random order, and the pool's size."""
    ps = c["page"]
    counts = [(n + ps - 1) // ps for n in total]
    n = sum(counts) + 3
    order = torch.randperm(n, generator=g, device=DEV).int()
    table = torch.full((c["B"], max(counts)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, k in enumerate(counts):
        table[b, :k] = order[at : at + k]
        at += k
    return table, n


def _filled(n, Hk, ps, D, g):
    """A pool of normally distributed rows as codes, and its scales."""
    codes = torch.empty((n, Hk, ps, D), dtype=torch.int8, device=DEV)
    scale = torch.empty((n, Hk), device=DEV)
    step = max(1, (1 << 26) // (Hk * ps * D))
    for i in range(0, n, step):
        x = torch.randn(codes[i : i + step].shape, generator=g, device=DEV)
        scale[i : i + step] = x.abs().amax((2, 3)) / 127
        codes[i : i + step] = torch.round(x / scale[i : i + step, :, None, None]).to(torch.int8)
    return codes, scale


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    c = case
    new, total = _plan(c)
    D, Hk = c["D"], c["Hk"]
    s = {"case": c, "new": new, "total": total, "lens": _ints(total)}
    if c["op"] == "prompt":
        s["q"] = (normal(sum(new), c["Hq"] * D) * 1.5).to(FLOATS[c["x"]])
        # one row of keys and values for each token
        s["kv"] = normal(sum(total), 2 * Hk * D).to(FLOATS[c["x"]])
        s["cu_q"], s["cu_k"] = _ints(_sums(new)), _ints(_sums(total))
        return s
    s["table"], n = _pages(c, total, g)
    s["kc"], s["ks"] = _filled(n, Hk, c["page"], D, g)
    s["vc"], s["vs"] = _filled(n, Hk, c["page"], D, g)
    if c["op"] == "cache":
        s["q"] = (normal(c["B"] * c["new"], c["Hq"] * D) * 1.5).to(FLOATS[c["x"]])
        return s
    T = sum(new)
    s["kv"] = normal(T, 2 * Hk * D).to(FLOATS[c["x"]])
    s["pos"] = _ints([p for n_b, t in zip(new, total) for p in range(t - n_b, t)])
    i = torch.arange(c["rot"] // 2, device=DEV, dtype=torch.float64)
    a = torch.arange(N_POS, device=DEV, dtype=torch.float64)[:, None] * 1e6 ** (-2 * i / c["rot"])
    s["cos"], s["sin"] = a.cos().float(), a.sin().float()
    s["cu"] = _ints(_sums(new))
    # what is read back: the tokens of every page that the call touches
    ps = c["page"]
    back = [t - (t - n_b) // ps * ps for n_b, t in zip(new, total)]
    s["back"], s["cu_back"] = back, _ints(_sums(back))
    # for the plain form: every new token's page and offset, and every sequence's first touched page
    seq = torch.repeat_interleave(torch.arange(c["B"], device=DEV), _ints(new).long())
    s["slot"] = (s["table"][seq, s["pos"].long() // ps].long(), s["pos"].long() % ps)
    first = _ints([t - n_b for n_b, t in zip(new, total)]).long()
    s["first"] = (s["table"][torch.arange(c["B"], device=DEV), first // ps].long(), first % ps)
    seq = torch.repeat_interleave(torch.arange(c["B"], device=DEV), _ints(back).long())
    at = _ints([p for n_b, t in zip(back, total) for p in range(t - n_b, t)]).long()
    s["slot_back"] = (s["table"][seq, at // ps].long(), at % ps)
    return s


# --------------------------------------------------------------------------------------------- plain forms
def _rotated(x, s, c):
    """x: [T][Hk][D] in 32 bits, every product and sum rounded."""
    cos, sin = s["cos"][s["pos"].long()][:, None], s["sin"][s["pos"].long()][:, None]
    r, rest = x[..., : c["rot"]], x[..., c["rot"] :]
    if c["pairs"]:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], 3).flatten(2)
    else:
        a, b = r.chunk(2, 2)
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], 2)
    return torch.cat([r, rest], 2)


def _plain_store(x, codes, scale, s, c):
    """The rows x [T][Hk][D] into the pages: scales grow to what the new rows need, old codes follow."""
    page, offset = s["slot"]
    fp, fo = s["first"]
    full = torch.full((1, 1), 127.0, device=x.device)
    # a page's first token starts it anew
    scale.index_reduce_(0, page, torch.where(offset[:, None] == 0, 0.0, scale[page]), "amin")
    old = scale[fp]
    need = x.abs().amax(2) / full
    scale.index_reduce_(0, page, need, "amax")
    grown = scale[fp]
    r = torch.where((grown > old) & (old > 0), old / grown, 1.0)
    kept = torch.arange(c["page"], device=x.device)[None, None, :, None] < fo[:, None, None, None]
    block = codes[fp]
    codes[fp] = torch.where(kept, torch.round(block.float() * r[:, :, None, None]).to(torch.int8), block)
    inverse = torch.ones((1, 1), device=x.device) / scale[page]
    codes[page, :, offset] = torch.round(x * inverse[..., None]).clamp(-127, 127).to(torch.int8)


def _plain_append(s, c):
    T, Hk, D = s["kv"].shape[0], c["Hk"], c["D"]
    kv = s["kv"].float().view(T, 2, Hk, D)
    _plain_store(_rotated(kv[:, 0], s, c), s["kc"], s["ks"], s, c)
    _plain_store(kv[:, 1], s["vc"], s["vs"], s, c)
    page, offset = s["slot_back"]
    out = {"k_scale": s["ks"], "v_scale": s["vs"]}
    for name, codes, scale in (("k", s["kc"], s["ks"]), ("v", s["vc"], s["vs"])):
        rows = codes[page, :, offset].float() * scale[page][..., None]
        out[name] = rows.flatten(1).to(FLOATS[c["y"]])
    return out


def _plain_rows(q, k, v, past, causal, D):
    """Softmax attention of q [n][Hq][D] (tokens past, past + 1, ..) over k, v [len][Hk][D], all in 32 bits."""
    n, Hq = q.shape[:2]
    Hk, L = k.shape[1], k.shape[0]
    out = torch.empty((n, Hq, D), device=q.device)
    G = Hq // Hk
    step = max(1, (1 << 29) // (G * n * L))  # heads at once: 2 GB of scores
    for h in range(0, Hk, step):
        m = min(step, Hk - h)
        x = q[:, h * G : (h + m) * G].unflatten(1, (m, G)).permute(1, 2, 0, 3).reshape(m, G * n, D)
        p = (x @ k[:, h : h + m].permute(1, 2, 0)) * (1.0 / math.sqrt(D))
        if causal:
            hidden = torch.arange(L, device=q.device) > past + torch.arange(n, device=q.device)[:, None]
            p.view(m, G, n, L).masked_fill_(hidden, -math.inf)
        p.sub_(p.amax(2, keepdim=True)).exp_()
        o = (p @ v[:, h : h + m].transpose(0, 1)) / p.sum(2, keepdim=True)
        out[:, h * G : (h + m) * G] = o.view(m, G, n, D).permute(2, 0, 1, 3).flatten(1, 2)
    return out.flatten(1)


def _plain_cache(s, c):
    D, n = c["D"], c["new"]
    out = []
    for b, t in enumerate(s["total"]):
        pages = s["table"][b, : (t + c["page"] - 1) // c["page"]].long()
        k, v = ((codes[pages].float() * scale[pages][..., None, None]).transpose(1, 2).flatten(0, 1)[:t]
                for codes, scale in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
        q = s["q"][b * n : (b + 1) * n].float().view(n, c["Hq"], D)
        out.append(_plain_rows(q, k, v, t - n, True, D))
    return torch.cat(out).to(FLOATS[c["y"]])


def _plain_prompt(s, c):
    D, Hk = c["D"], c["Hk"]
    out, at_q, at_k = [], 0, 0
    for n, t in zip(s["new"], s["total"]):
        kv = s["kv"][at_k : at_k + t].float().view(t, 2, Hk, D)
        q = s["q"][at_q : at_q + n].float().view(n, c["Hq"], D)
        out.append(_plain_rows(q, kv[:, 0], kv[:, 1], t - n, c["causal"], D))
        at_q, at_k = at_q + n, at_k + t
    return torch.cat(out).to(FLOATS[c["x"]])


# --------------------------------------------------------------------------------------------- the kernels
def _buffers(s, c, kq):
    """The outputs and the workspace that a program keeps from call to call."""
    D = c["D"]
    if c["op"] == "append":
        T = sum(s["back"])
        return {n: torch.empty((T, c["Hk"] * D), dtype=FLOATS[c["y"]], device=DEV) for n in "kv"}
    T = s["q"].shape[0]
    if c["op"] == "cache":
        n = kq.kq_attn_cache_i8_workspace_bytes(c["B"], c["new"], c["Hq"], c["Hk"], D)
    else:
        n = kq.kq_attn_prompt_workspace_bytes(c["B"], T, c["Hq"], c["Hk"], D)
    return {"y": torch.empty((T, c["Hq"] * D), dtype=FLOATS[c["y"] if c["op"] == "cache" else c["x"]], device=DEV),
            "ws": torch.zeros(n, dtype=torch.uint8, device=DEV), "n": n}


def _run_own(s, c):
    import gemv_quantize_q8_gb300 as kq

    types = {"f32": kq.F32, "f16": kq.F16, "bf16": kq.BF16}
    if "buffers" not in s:
        s["buffers"] = _buffers(s, c, kq)
    b = s["buffers"]
    B, Hk, D = c["B"], c["Hk"], c["D"]
    nk = Hk * D
    if c["op"] == "prompt":
        k, v = s["kv"], s["kv"][:, nk:]
        kq.kq_attn_prompt(types[c["x"]], s["q"], c["Hq"] * D, k, 2 * nk, v, 2 * nk, s["cu_q"], s["cu_k"], B, s["q"].shape[0],
                          k.shape[0], c["Hq"], Hk, D, 1.0 / math.sqrt(D), int(c["causal"]), b["y"], c["Hq"] * D, b["ws"], b["n"])
        return b["y"]
    n_pages, page, width = s["kc"].shape[0], c["page"], s["table"].shape[1]
    if c["op"] == "cache":
        kq.kq_attn_cache_i8(types[c["x"]], s["q"], c["Hq"] * D, B, c["new"], c["Hq"], Hk, D, 1.0 / math.sqrt(D), s["kc"], s["vc"],
                            s["ks"], s["vs"], n_pages, page, s["table"], width, s["lens"], types[c["y"]], b["y"], c["Hq"] * D,
                            b["ws"], b["n"])
        return b["y"]
    kq.kq_kv_append_i8(types[c["x"]], s["kv"], 2 * nk, s["kv"][:, nk:], 2 * nk, s["cu"], s["lens"], B, s["kv"].shape[0], Hk, D,
                       s["pos"], s["cos"], s["sin"], N_POS, c["rot"], int(c["pairs"]), s["kc"], s["vc"], s["ks"], s["vs"],
                       n_pages, page, s["table"], width)
    kq.kq_kv_read_i8(s["kc"], s["vc"], s["ks"], s["vs"], n_pages, page, s["table"], width, s["cu_back"], s["lens"], B,
                     b["k"].shape[0], Hk, D, types[c["y"]], b["k"], nk, b["v"], nk)
    return {"k_scale": s["ks"], "v_scale": s["vs"], "k": b["k"], "v": b["v"]}


def run(state):
    c = state["case"]
    if own:
        return _run_own(state, c)
    return {"append": _plain_append, "cache": _plain_cache, "prompt": _plain_prompt}[c["op"]](state, c)


# --------------------------------------------------------------------------------------------- the measure
def work(case):
    c = case
    new, total = _plan(c)
    D, Hk, ps = c["D"], c["Hk"], c.get("page", 1)
    if c["op"] == "append":
        n, rows = sum(new) * 2 * Hk * D, 2 * Hk * D
        back = [t - (t - n_b) // ps * ps for n_b, t in zip(new, total)]
        touched = sum((b + ps - 1) // ps for b in back) * 2 * Hk
        # the new rows in and their codes out; the touched pages' codes in and their rows out; scales and angles
        return {"bytes": n * (SIZE[c["x"]] + 1) + sum(back) * rows * (1 + SIZE[c["y"]]) + 12 * touched
                + sum(new) * 4 * (1 + c["rot"]), "flops": 8 * n + sum(back) * rows}
    if c["op"] == "cache":
        n = c["new"]
        pairs = sum(t - n + 1 + i for t in total for i in range(n))
        pages = sum((t + ps - 1) // ps for t in total)
        return {"bytes": sum(total) * 2 * Hk * D + pages * (8 * Hk + 4) + c["B"] * n * c["Hq"] * D * (SIZE[c["x"]] + SIZE[c["y"]]),
                "flops": 4 * D * c["Hq"] * pairs}
    pairs = sum(n * (t - n) + n * (n + 1) // 2 if c["causal"] else n * t for n, t in zip(new, total))
    return {"bytes": SIZE[c["x"]] * D * (2 * sum(new) * c["Hq"] + 2 * sum(total) * Hk), "flops": 4 * D * c["Hq"] * pairs}


# --------------------------------------------------------------------------------------------- in 64 bits
def _exact_attention(q, k, v, past, causal):
    """q [n][Hq][D], k and v [len][Hk][D] in 64 bits; queries in slices of about a GB of scores."""
    n, Hq, D = q.shape
    L, Hk = k.shape[:2]
    q = q.view(n, Hk, Hq // Hk, D)
    parts = []
    step = max(1, (1 << 27) // (L * Hq))
    for i in range(0, n, step):
        x = torch.einsum("nhgd,lhd->hgnl", q[i : i + step], k) / D**0.5
        if causal:
            m = x.shape[2]
            hidden = torch.ones((m, L), dtype=torch.bool, device=x.device).triu(past + i + 1)
            x[:, :, hidden] = -math.inf
        w = torch.softmax(x, -1)
        parts.append(torch.einsum("hgnl,lhd->nhgd", w, v).reshape(-1, Hq * D))
    return torch.cat(parts)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    D, Hk, B = c["D"], c["Hk"], c["B"]
    new, total = _plan(c)
    if c["op"] == "append":
        return _exact_append(c, s)
    out = []
    at_k = 0
    for b in range(B):
        first = sum(new[:b])
        q = s["q"][first : first + new[b]].double().unflatten(1, (c["Hq"], D))
        if c["op"] == "prompt":
            kv = s["kv"][at_k : at_k + total[b]].double()
            k, v = kv[:, : Hk * D].unflatten(1, (Hk, D)), kv[:, Hk * D :].unflatten(1, (Hk, D))
            at_k += total[b]
        else:
            token = torch.arange(total[b], device=DEV)
            page, offset = s["table"][b].long()[token // c["page"]], token % c["page"]
            k = torch.einsum("thd,th->thd", s["kc"][page, :, offset].double(), s["ks"][page].double())
            v = torch.einsum("thd,th->thd", s["vc"][page, :, offset].double(), s["vs"][page].double())
        out.append(_exact_attention(q, k, v, total[b] - new[b], c["op"] == "cache" or c["causal"]))
    return torch.cat(out)


def _exact_append(c, s):
    """Scales and codes are fixed by the definition in 32 bits (a code is a whole number next to a border); the values
    that they stand for are in 64."""
    D, Hk, ps = c["D"], c["Hk"], c["page"]
    f32 = torch.float32
    half = c["rot"] // 2
    x = s["kv"].to(f32).reshape(-1, 2 * Hk, D)
    cos, sin = s["cos"].index_select(0, s["pos"].long()), s["sin"].index_select(0, s["pos"].long())
    i = torch.arange(half, device=DEV)
    ia, ib = (2 * i, 2 * i + 1) if c["pairs"] else (i, i + half)
    y = x.clone()
    for h in range(Hk):
        a, b = x[:, h][:, ia], x[:, h][:, ib]
        y[:, h, ia] = torch.mul(a, cos).sub_(torch.mul(b, sin))
        y[:, h, ib] = torch.mul(b, cos).add_(torch.mul(a, sin))
    codes, scale = torch.cat([s["kc"], s["vc"]], 1), torch.cat([s["ks"], s["vs"]], 1)
    out, at = [], 0
    one, full = torch.ones(1, device=DEV), torch.full((1,), 127.0, device=DEV)
    for b, (n, t) in enumerate(zip(s["new"], s["total"])):
        pages = s["table"][b].tolist()
        for i in range((t - n) // ps, (t + ps - 1) // ps):
            lo, hi = max(t - n, i * ps), min(t, (i + 1) * ps)
            rows = y[at + lo - (t - n) : at + hi - (t - n)].transpose(0, 1)  # [2*Hk][tokens][D]
            kept = lo - i * ps
            was = scale[pages[i]] if kept else torch.zeros(2 * Hk, device=DEV)
            now = torch.maximum(was, torch.maximum(rows.amax((1, 2)), -rows.amin((1, 2))) / full)
            grows = (now > was) & (was > 0)
            r = torch.where(grows, was / now, one)
            block = codes[pages[i]]
            if kept:
                block[:, :kept] = torch.round(block[:, :kept].to(f32) * r[:, None, None]).to(torch.int8)
            q = torch.round(rows * (one / now)[:, None, None])
            block[:, kept : kept + hi - lo] = q.clamp(-127, 127).to(torch.int8)
            scale[pages[i]] = now
            out.append((block[:, : hi - i * ps].double() * now.double()[:, None, None]).transpose(0, 1))
        at += n
    rows = torch.cat(out)
    return {"k_scale": scale[:, :Hk].double(), "v_scale": scale[:, Hk:].double(), "k": rows[:, :Hk].flatten(1),
            "v": rows[:, Hk:].flatten(1)}
