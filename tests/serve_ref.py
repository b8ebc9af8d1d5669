"""Plain 64-bit definitions of the calls around the recall (per-head norm +
rotation, paged append, paged attention), and the inputs their tests share."""
from __future__ import annotations

import math

import torch

from paged_kv_cache_meank_gb300 import configs

TDT = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.uint8}
EPS2 = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -4}    # half a step, relative
U = 2.0 ** -24                                                      # float32's half step


def workload(*, L=1, G=2, H=4, d=64, kv="f32", act="f32", theta=1e4, n_blocks=8, index="f32"):
    return configs.Workload(
        name="serve", n_layers=L, n_kv_heads=G, n_q_heads=H, head_dim=d, rope_theta=theta,
        kv_dtype=kv, index_dtype=index, q_dtype=act, n_blocks=n_blocks, n_queries=1,
        sink_blocks=0, recent_blocks=0, view_blocks=1, planted_frac=0.0)


def decode(codes):
    return codes.cpu().view(torch.float8_e4m3fn).double()


def encode(x):
    """float64 -> the nearest e4m3 (ties to even, saturating), as codes."""
    a = x.abs().clamp(max=448.0)
    step = torch.exp2((torch.frexp(a)[1].double() - 4).clamp(min=-9))
    v = torch.copysign(torch.round(a / step) * step, x)
    return torch.where(torch.isnan(x), x, v).float().to(torch.float8_e4m3fn).view(torch.uint8)


def values(t, dtype):
    return decode(t) if dtype == "e4m3" else t.cpu().double()


def rotate(x, pos, theta, sign=1.0):
    """[..., n, d] turned at positions [n]."""
    d = x.shape[-1]
    w = theta ** (-2.0 * torch.arange(d // 2, dtype=torch.float64) / d)
    a = sign * pos.double()[:, None] * w
    p, q = x[..., :d // 2], x[..., d // 2:]
    return torch.cat((p * a.cos() - q * a.sin(), p * a.sin() + q * a.cos()), -1)


def pair_mag(x):
    h = x.shape[-1] // 2
    m = torch.hypot(x[..., :h], x[..., h:])
    return torch.cat((m, m), -1)


def scale_for(amax, most):
    """The least 2^e with amax <= most 2^e, -100 <= e <= 119."""
    e = -100
    if amax > 0:
        e = math.frexp(amax / most)[1] - 1
        while amax > math.ldexp(most, e):
            e += 1
        while e > -100 and amax <= math.ldexp(most, e - 1):
            e -= 1
    return math.ldexp(1.0, min(119, max(-100, e)))


def attention(q, keys, vals, scale, first, causal):
    """One head: q [n, d], keys / vals [kv, d] -> out [n, d], lse [n], and the
    weighted mean of |v| (what a relative error of the weights multiplies)."""
    n, kv = q.shape[0], keys.shape[0]
    if kv == 0:
        z = torch.zeros(n, q.shape[1], dtype=torch.float64)
        return z, torch.full((n,), -math.inf, dtype=torch.float64), z
    s = q @ keys.T * scale
    if causal:
        s = s.masked_fill(torch.arange(kv)[None, :] > first + torch.arange(n)[:, None], -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.where(lse[:, None] == -math.inf, 0.0, torch.exp(s - lse[:, None].clamp(min=-1e300)))
    return p @ vals, lse, p @ vals.abs()


class Paged:
    """A paged cache and a batch over it: random values in the rows below each
    kv_len, NaN (or a NaN code) everywhere else, permuted pages."""

    def __init__(self, lens, *, L=1, G=2, H=4, d=64, kv="f32", act="f32", layer=0, scaled=False,
                 seed=0, spare=3, own_rows=False, table_pad=0, lead=0, tail=0, vstd=1.0, qstd=1.5):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.L, self.G, self.H, self.d = lens, L, G, H, d
        self.kv, self.act, self.layer, self.scaled = kv, act, layer, scaled
        need = [-(-k // 32) for _, k in lens]
        n_pages = sum(need) + spare
        order = torch.randperm(n_pages, generator=g)
        width = max(max(need), 1) + table_pad
        self.table = torch.full((len(lens), width), -7, dtype=torch.int32)   # unused: no page
        shape = (n_pages, L, G, 32, d)
        nan = 0x7F if kv == "e4m3" else math.nan
        self.k = torch.full(shape, nan, dtype=TDT[kv])
        self.v = torch.full(shape, nan, dtype=TDT[kv])
        rows = n_pages + 5 if own_rows else n_pages
        self.ks = self.vs = self.rows = None
        if scaled:
            self.ks = torch.exp2(torch.randint(-9, -4, (rows, L, G), generator=g).float())
            self.vs = torch.exp2(torch.randint(-12, 3, (rows, L, G), generator=g).float())
            if own_rows:
                self.rows = torch.full_like(self.table, -3)
                rorder = torch.randperm(rows, generator=g)
        at = 0
        for s, (_, kvl) in enumerate(lens):
            for b in range(need[s]):
                p = int(order[at])
                self.table[s, b] = p
                if self.rows is not None:
                    self.rows[s, b] = int(rorder[at])
                at += 1
                n = min(32, kvl - b * 32)
                for pages, std in ((self.k, 1.0), (self.v, vstd)):
                    x = torch.randn(L, G, n, d, generator=g) * std
                    if kv == "e4m3":
                        x = (x * (60.0 if scaled else 1.0)).to(torch.float8_e4m3fn).view(torch.uint8)
                    pages[p, :, :, :n] = x.to(TDT[kv])
        self.q_start = [lead]
        for qn, _ in lens:
            self.q_start.append(self.q_start[-1] + qn)
        self.n = self.q_start[-1] + tail
        self.q = (torch.randn(self.n, H, d, generator=g) * qstd).to(TDT[act])
        self.max_q = max(qn for qn, _ in lens)
        self.max_kv = max(kvl for _, kvl in lens)

    def heads(self, s, g):
        """Sequence s's keys and values of kv head g in 64 bits."""
        kvl = self.lens[s][1]
        nb = -(-kvl // 32)
        pages = self.table[s, :nb].long()
        rows = (self.rows if self.rows is not None else self.table)[s, :nb].long()
        got = []
        for t, sc in ((self.k, self.ks), (self.v, self.vs)):
            x = values(t[pages, self.layer, g], self.kv)
            if sc is not None:
                x = x * sc[rows, self.layer, g].double()[:, None, None]
            got.append(x.reshape(-1, self.d)[:kvl])
        return got

    def reference(self, scale, causal):
        """out, lse, mean |v| per row, and the absolute error that float32 dot
        products can leave in a score (d + 2 roundings of |q||k|)."""
        out = torch.zeros(self.n, self.H, self.d, dtype=torch.float64)
        absv = torch.zeros_like(out)
        lse = torch.full((self.n, self.H), -math.inf, dtype=torch.float64)
        ds = torch.zeros(self.n, self.H, dtype=torch.float64)
        r = self.H // self.G
        for s, (qn, kvl) in enumerate(self.lens):
            a = self.q_start[s]
            for g in range(self.G):
                k, v = self.heads(s, g)
                for h in range(g * r, (g + 1) * r):
                    q = self.q[a:a + qn, h].double()
                    o, e, m = attention(q, k, v, scale, kvl - qn, causal)
                    out[a:a + qn, h], lse[a:a + qn, h], absv[a:a + qn, h] = o, e, m
                    if kvl and qn:
                        dot = (q.abs() @ k.abs().T).amax(-1) * abs(scale)
                        ds[a:a + qn, h] = (self.d + 2) * U * dot
        return out, lse, absv, ds

    def on(self, ctx, device="cuda"):
        """(batch, cache) on the device."""
        cuda = lambda t: None if t is None else t.to(device)   # noqa: E731
        self.dk, self.dv, self.dks, self.dvs = map(cuda, (self.k, self.v, self.ks, self.vs))
        cache = ctx.cache(self.dk, self.dv, self.dks, self.dvs)
        batch = ctx.batch(torch.tensor(self.q_start, dtype=torch.int32, device=device),
                          torch.tensor([k for _, k in self.lens], dtype=torch.int32, device=device),
                          cuda(self.table), n_tokens=self.n, max_q_len=self.max_q,
                          max_kv_len=self.max_kv, scale_rows=cuda(self.rows))
        return batch, cache


def attend_tolerance(out, absv, ds, act, kv, n_keys):
    """What the arithmetic can leave: the output's rounding; the weights' relative
    error (twice the score's, the exponential's few float32 roundings and one
    for each key summed) on the weighted |v|; on the tensor cores also the weights'
    rounding to bf16, half a step of 2^-7."""
    w = 2 * ds[..., None] + (2 * n_keys + 16) * U
    if act == "bf16" and kv != "f32":
        w = w + EPS2["bf16"]
    return EPS2[act] * out.abs() + w * (1 + EPS2[act]) * absv + 1e-30
