"""A paged 8-bit cache for the GPU tests: its buffers, its definition in numpy, and plain attention in 64 bits."""
import numpy as np
import torch

import gemv_quantize_q8_gb300 as kq
from tests.gpu_util import DEV

U = 2.0 ** -24
TYPES = {"f32": (kq.F32, torch.float32), "f16": (kq.F16, torch.float16), "bf16": (kq.BF16, torch.bfloat16)}
HALF_UNIT = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
N_POS = 6000


def ints(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def tables(rot):
    a = np.arange(N_POS)[:, None] * 1e4 ** (-2 * np.arange(rot // 2) / max(rot, 1))
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


class Cache:
    """Pages handed out in random order; spare pages and codes beyond the tokens hold junk."""

    def __init__(self, lens, n_kv, D, page, seed=0, spare=2, fill=False):
        g = np.random.default_rng(seed)
        self.n_kv, self.D, self.page, self.B = n_kv, D, page, len(lens)
        counts = [-(-max(n, 0) // page) for n in lens]
        self.n_pages = sum(counts) + spare
        order = g.permutation(self.n_pages)
        self.ldt = max(counts + [1]) + 1
        self.table_host = np.full((self.B, self.ldt), -7, np.int64)
        at = 0
        for b, n in enumerate(counts):
            self.table_host[b, :n] = order[at : at + n]
            at += n
        shape = (2, self.n_pages, n_kv, page, D)
        self.codes_host = g.integers(-127, 128, shape).astype(np.int8)
        self.scale_host = (g.random(shape[:3]) * 0.02 + 0.001 if fill else np.full(shape[:3], 3.0)).astype(np.float32)
        self.upload()
        self.lens = ints(lens)

    def upload(self):
        self.codes, self.scale = (torch.from_numpy(a).to(DEV) for a in (self.codes_host, self.scale_host))
        self.table = ints(self.table_host)

    @property
    def args(self):
        return (self.codes[0], self.codes[1], self.scale[0], self.scale[1], self.n_pages, self.page, self.table, self.ldt)

    def rows(self, b, n, which):
        """The first n tokens of sequence b in 64 bits, [n][n_kv][D]."""
        i = np.arange(n)
        p = self.table_host[b, i // self.page]
        return self.codes_host[which][p, :, i % self.page].astype(np.float64) * self.scale_host[which][p].astype(np.float64)[..., None]

    def append(self, k, v, new, lens, pos, cos, sin, rot, pairs):
        """The definition, on the host copies; k, v: fp32 [T][n_kv][D]."""
        f = np.float32
        k = k.copy()
        if rot:
            i = np.arange(rot // 2)
            ia, ib = (2 * i, 2 * i + 1) if pairs else (i, i + rot // 2)
            known = (pos >= 0) & (pos < N_POS)
            c, s = (t[np.where(known, pos, 0)][:, None] for t in (cos, sin))
            a, b = k[..., ia], k[..., ib]
            k[..., ia], k[..., ib] = a * c - b * s, b * c + a * s
            k[~known, :, :rot] = np.nan
        at = 0
        for b, (n, t) in enumerate(zip(new, lens)):
            for which, x in ((0, k), (1, v)):
                first, begin = t - n, max(t - n, 0)
                for i in range(begin // self.page, -(-t // self.page)) if n else ():
                    lo, hi = max(begin, i * self.page), min(t, (i + 1) * self.page)
                    p = self.table_host[b, i] if i < self.ldt else -1
                    if not 0 <= p < self.n_pages:
                        continue
                    r = x[at + lo - first : at + hi - first]
                    kept = lo - i * self.page
                    with np.errstate(all="ignore"):
                        amax = np.fmax(np.abs(np.where(np.isnan(r), f(0), r)).max((0, 2)), f(0))
                        was = self.scale_host[which][p] if kept else np.zeros(self.n_kv, f)
                        now = np.fmax(was, amax / f(127))
                        inv = f(1) / now
                        inv = np.where(np.isinf(inv), f(0), inv)
                        code = r * inv[:, None]
                        code = np.where(np.isnan(code), f(0), np.clip(code, f(-127), f(127)))
                        for h in np.flatnonzero((now > was) & (was > 0)):
                            old = self.codes_host[which][p, h, :kept].astype(f) * f(was[h] / now[h])
                            self.codes_host[which][p, h, :kept] = np.rint(old).astype(np.int8)
                    self.codes_host[which][p, :, kept : kept + hi - lo] = np.rint(code).astype(np.int8).transpose(1, 0, 2)
                    self.scale_host[which][p] = now
            at += n


def attention(q, k, v, scale, limits):
    """q [n][Hq][D], k and v [L][Hk][D] in 64 bits; token i sees the first limits[i] keys.  Also the largest visible |v| of each
    element and the largest sum |q_d k_d| * |scale|."""
    n, Hq, D = q.shape
    L, Hk = k.shape[:2]
    out, vmax, smax = (np.zeros((n, Hq, D)), np.zeros((n, Hq, D)), np.zeros((n, Hq, 1)))
    for i in range(n):
        m = min(max(limits[i], 0), L)
        if m == 0:
            continue
        for h in range(Hq):
            kk, vv = k[:m, h // (Hq // Hk)], v[:m, h // (Hq // Hk)]
            with np.errstate(all="ignore"):
                s = kk @ q[i, h] * scale
                p = np.exp(s - s.max())
                out[i, h] = p @ vv / p.sum()
                vmax[i, h], smax[i, h] = np.abs(vv).max(0), (np.abs(kk) @ np.abs(q[i, h])).max() * abs(scale)
    return out, vmax, smax
