"""The operators around the recall step, measured: queries and keys normalised per head and rotated, keys and values
appended to the paged cache, attention over the paged cache, and the Mean-K index of 8-bit pages with scales.

Each case is one call as a serving loop makes it for one layer (the index build: for all layers of a chunk).  Pages are
[page][layer][kv head][32][d]; 8-bit pages hold e4m3 codes with one power-of-two scale for each (page, layer, kv head).
``run`` computes a case in plain torch operations, or with ``own`` through the framework's calls.
"""
import math

import torch

own = False

B = 32                      # tokens of a page
K_MOST = 316.75             # a little below 448 / sqrt(2): a rotated pair of such entries stays within 448
V_MOST = 448.0
E_LEAST, E_MOST = -100, 119  # exponents a block's scale may have
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.uint8}

# Attention shapes of this repository: the 27B-class model, the tiny workspace, the small d = 64 test shape.
Q27 = dict(G=8, H=48, d=128, theta=1e6, act="bf16")
TINY = dict(G=2, H=4, d=64, theta=1e4, act="f32")
MID64 = dict(G=4, H=8, d=64, theta=1e4, act="bf16")


def listed():
    return [
        # one decoded token of the tiny float32 workspace: nothing but latency
        dict(name="attend-decode-tiny-f32", op="attend", L=2, kv="f32", seqs=1, q=1, kv_len=77, ragged=False, causal=True, **TINY),
        # one decoded token over a 32K-token view and its tail, the recall step's ordinary successor
        dict(name="attend-decode-32k-bf16", op="attend", L=4, kv="bf16", seqs=1, q=1, kv_len=32785, ragged=False, causal=True, **Q27),
        # a batch of agents of different lengths decoding together from 8-bit pages, one slot of the batch unused
        dict(name="attend-decode-batch-e4m3", op="attend", L=2, kv="e4m3", seqs=24, q=1, kv_len=20011, ragged=True, causal=True, **Q27),
        # the 32 current-step queries that the recall scored with, over the 64K-token 8-bit view that it assembled
        dict(name="attend-step-64k-e4m3", op="attend", L=2, kv="e4m3", seqs=1, q=32, kv_len=65568, ragged=False, causal=True, **Q27),
        # a chunk of prefill (a long tool answer) over a 32K-token view
        dict(name="attend-prefill-bf16", op="attend", L=2, kv="bf16", seqs=1, q=2048, kv_len=34816, ragged=False, causal=True, **Q27),
        # several short prompts prefilled together, d = 64, odd sizes
        dict(name="attend-prefill-ragged-d64", op="attend", L=2, kv="bf16", seqs=9, q=709, kv_len=1501, ragged=True, causal=True, **MID64),
        # one decoded token's queries and keys
        dict(name="norm-decode", op="norm", tokens=1, free=True, **Q27),
        # a prefill chunk's queries and keys, the RoPE-free queries kept for scoring
        dict(name="norm-prefill", op="norm", tokens=8192, free=True, **Q27),
        # one decoded token of each of 24 agents into 8-bit pages
        dict(name="append-decode-e4m3", op="append", L=2, kv="e4m3", seqs=24, q=1, kv_len=20011, ragged=True, raw=False, **Q27),
        # a prefill chunk into 8-bit pages, its raw K kept for the repository
        dict(name="append-prefill-e4m3", op="append", L=2, kv="e4m3", seqs=1, q=8192, kv_len=32785, ragged=False, raw=True, **Q27),
        # one completed block of 8-bit pages indexed
        dict(name="index-block-e4m3", op="index", L=64, blocks=1, first=1023, capacity=1088, raw=True, kv="e4m3", **Q27),
        # a prefill chunk of 8192 tokens indexed, its raw K kept
        dict(name="index-chunk-e4m3", op="index", L=64, blocks=256, first=768, capacity=1088, raw=True, kv="e4m3", **Q27),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("attend", "attend", "attend", "norm", "append", "append", "index"))
    shape = dict(rng.choice((Q27, Q27, MID64, TINY)))
    if shape["act"] == "bf16" and rng.random() < 0.5:       # other numbers of query heads to a kv head
        shape["G"] = rng.choice((1, 2, 4, 8))
        shape["H"] = shape["G"] * rng.choice((1, 2, 3, 4, 6, 7, 8))
    small = shape["act"] == "f32"
    kv = "f32" if small else rng.choice(("bf16", "e4m3"))
    if op == "norm":
        return dict(op=op, tokens=_log(rng, 1, 512 if small else 8192), free=rng.random() < 0.5, **shape)
    if op == "index":
        first = rng.randrange(0, 800)
        return dict(op=op, L=rng.choice((1, 3, 16, 64)), blocks=_log(rng, 1, 256), first=first, capacity=1088,
                    raw=rng.random() < 0.5, kv="e4m3", **shape)
    kind = rng.choice(("decode", "step", "prefill"))
    if kind == "decode":
        seqs, q = _log(rng, 1, 8 if small else 64), rng.choice((1, 1, 2, 4))
        kv_len = _log(rng, q + 1, 4096 if small else 32768 if seqs < 16 else 8192)
    elif kind == "step":
        seqs, q = _log(rng, 1, 2 if small else 4), _log(rng, 5, 40)
        kv_len = _log(rng, q + 1, 2048 if small else 32768)
    else:
        seqs, q = _log(rng, 1, 2 if small else 6), _log(rng, 41, 256 if small else 1024)
        kv_len = _log(rng, q + 1, 2048 if small else 16384)
    more = dict(L=rng.choice((1, 2, 3)), kv=kv, seqs=seqs, q=q, kv_len=kv_len, ragged=seqs > 1, **shape)
    if op == "append":
        return dict(op=op, raw=rng.random() < 0.5, **more)
    return dict(op=op, causal=rng.random() < 0.75, **more)


def _lengths(c):
    """The batch's (query tokens, kv tokens) of each sequence: all alike, or spread over the range with the first one
    the longest and, from four sequences on, the last one an unused slot (one query row, nothing to see)."""
    if not c["ragged"]:
        return [(c["q"], c["kv_len"])] * c["seqs"]
    got = []
    for i in range(c["seqs"]):
        part = 1.0 if i == 0 else (i * 0.6180339887) % 1.0
        kv = max(1, round(c["kv_len"] * part))
        q = min(kv, c["q"] if c["q"] <= 4 else max(1, round(c["q"] * ((i * 0.7548776662 + 1.0) % 1.0 if i else 1.0))))
        got.append((q, kv))
    if c["op"] == "attend" and c["seqs"] >= 4:
        got[-1] = (1, 0)
    return got


def _normal(g, *shape, std=1.0, dtype=torch.float32):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    for at in range(0, flat.numel(), 1 << 27):
        n = min(1 << 27, flat.numel() - at)
        x = torch.randn(n, generator=g, device="cuda") * std
        flat[at:at + n] = x.to(torch.float8_e4m3fn).view(torch.uint8) if dtype == torch.uint8 else x.to(dtype)
    return out


def _pages(g, c, n):
    """A cache of n pages as earlier tokens left it: codes and scales, or values."""
    shape = (n, c["L"], c["G"], B, c["d"])
    if c["kv"] != "e4m3":
        return dict(k=_normal(g, *shape, dtype=DT[c["kv"]]), v=_normal(g, *shape, dtype=DT[c["kv"]]), ks=None, vs=None)
    # blocks whose largest entry is near 4, stored as appending stores them: scales 2^-6 or 2^-5 for K
    scale = lambda least: torch.exp2(least + torch.randint(0, 2, shape[:3], generator=g, device="cuda").float())  # noqa: E731
    ks, vs = scale(-6), scale(-7)
    return dict(k=_normal(g, *shape, std=48.0, dtype=torch.uint8), v=_normal(g, *shape, std=64.0, dtype=torch.uint8), ks=ks, vs=vs)


def _context(c, max_blocks, positions):
    """The framework's handle for this shape."""
    import paged_kv_cache_meank_gb300 as kvm
    from paged_kv_cache_meank_gb300 import configs
    wl = configs.Workload(
        name="operators", n_layers=c.get("L", 1), n_kv_heads=c["G"], n_q_heads=c["H"], head_dim=c["d"], rope_theta=c["theta"],
        kv_dtype=c.get("kv", c["act"]), index_dtype="bf16", q_dtype=c["act"], n_blocks=max_blocks, n_queries=1, sink_blocks=0,
        recent_blocks=0, view_blocks=1, planted_frac=0.0)
    return kvm.Context(kvm.config_for(wl, max_positions=max(positions, B)))


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = dict(c=c)
    G, H, d, act = c["G"], c["H"], c["d"], DT[c["act"]]
    ctx_pos = 65600
    if c["op"] == "norm":
        n = c["tokens"]
        first = int(torch.randint(0, 32768, (1,), generator=g, device="cuda"))
        s.update(qkv=_normal(g, n, (H + 2 * G) * d, std=2.0, dtype=act), qw=1 + _normal(g, d, std=0.2), kw=1 + _normal(g, d, std=0.2),
                 pos=torch.arange(first, first + n, dtype=torch.int32, device="cuda"), eps=1e-6)
        s["qw"], s["kw"] = s["qw"].to(act), s["kw"].to(act)
        s["q_rot"], s["q_free"] = (torch.empty(n, H, d, dtype=act, device="cuda") for _ in range(2))
        s["k_rot"], s["k_free"] = (torch.empty(n, G, d, dtype=act, device="cuda") for _ in range(2))
        if own:
            s["ctx"] = _context(c, 1, ctx_pos)
        return s
    if c["op"] == "index":
        L, n = c["L"], c["blocks"]
        s.update(_pages(g, c, n))
        del s["v"], s["vs"]
        s["index"] = torch.zeros(L, G, c["capacity"], d, dtype=torch.bfloat16, device="cuda")
        s["raw"] = torch.zeros(n, L, G, B, d, dtype=torch.uint8, device="cuda") if c["raw"] else None
        if own:
            s["ctx"] = _context(c, c["capacity"], c["capacity"] * B)
        return s
    lens = _lengths(c)
    most = max(1, -(-max(kv for _, kv in lens) // B))
    need = [-(-kv // B) for _, kv in lens]
    n_pages = sum(need) + 3
    s.update(_pages(g, c, n_pages))
    order = torch.randperm(n_pages, generator=g, device="cuda")
    table = torch.zeros(c["seqs"], most, dtype=torch.int32, device="cuda")
    at = 0
    for i, m in enumerate(need):
        table[i, :m] = order[at:at + m]
        at += m
    starts = [0]
    for q, _ in lens:
        starts.append(starts[-1] + q)
    n = starts[-1]
    s.update(table=table, n=n, max_q=max(q for q, _ in lens), max_kv=max(kv for _, kv in lens), layer=c["L"] - 1,
             q_start=torch.tensor(starts, dtype=torch.int32, device="cuda"),
             kv_len=torch.tensor([kv for _, kv in lens], dtype=torch.int32, device="cuda"))
    if c["op"] == "append":
        s["k_new"], s["qkv"] = _normal(g, n, G, d, dtype=act), _normal(g, n, (H + 2 * G) * d, dtype=act)
        s["raw"] = torch.zeros_like(s["k"]) if c["raw"] else None
    else:
        s["q"] = _normal(g, n, H, d, std=2.0, dtype=act)
        s["out"] = torch.empty(n, H, d, dtype=act, device="cuda")
        s["lse"] = torch.empty(n, H, device="cuda")
    if own:
        s["ctx"] = ctx = _context(c, n_pages, ctx_pos)
        s["cache"] = ctx.cache(s["k"], s["v"], s["ks"], s["vs"])
        s["batch"] = ctx.batch(s["q_start"], s["kv_len"], s["table"], n_tokens=n, max_q_len=s["max_q"], max_kv_len=s["max_kv"])
    return s


def _v_of(s):
    """The values of the packed projection rows [tokens][q heads, k heads, v heads]."""
    c = s["c"]
    at = (c["H"] + c["G"]) * c["d"]
    return s["qkv"][:, at:].view(s["n"], c["G"], c["d"])


def run(s):
    c = s["c"]
    return {"norm": _norm, "append": _append, "attend": _attend, "index": _index}[c["op"]](s, c)


def _angles(pos, c):
    """cos and sin of each position's angles, from 64 bits, rounded once."""
    w = c["theta"] ** (-torch.arange(0, c["d"], 2, dtype=torch.float64, device="cuda") / c["d"])
    a = pos.double()[:, None] * w
    return a.cos().float(), a.sin().float()


def _rotate(x, cos, sin):
    x, y = x.chunk(2, -1)
    return torch.cat((x * cos - y * sin, x * sin + y * cos), -1)


def _values(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _codes(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


# ---- queries and keys normalised per head and rotated

def _norm(s, c):
    n, G, H, d = c["tokens"], c["G"], c["H"], c["d"]
    q, k = s["qkv"][:, :H * d].view(n, H, d), s["qkv"][:, H * d:(H + G) * d].view(n, G, d)
    if own:
        s["ctx"].qk_norm_rope(s["pos"], q=q, k=k, q_weight=s["qw"], k_weight=s["kw"], eps=s["eps"], q_rot=s["q_rot"], k_rot=s["k_rot"],
                              q_free=s["q_free"] if c["free"] else None, k_free=s["k_free"] if c["free"] else None)
        got = (s["q_rot"], s["k_rot"]) + ((s["q_free"], s["k_free"]) if c["free"] else ())
        return list(got)
    cos, sin = (t[:, None] for t in _angles(s["pos"], c))
    rot, free = [], []
    for x, w in ((q.float(), s["qw"].float()), (k.float(), s["kw"].float())):
        y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * w
        rot.append(_rotate(y, cos, sin).to(s["qkv"].dtype))
        free.append(y.to(s["qkv"].dtype))
    return rot + (free if c["free"] else [])


# ---- keys and values appended to the paged cache

def _where(s):
    """For each token: its place in its sequence, its page and its row in the page."""
    q_len = s["q_start"][1:] - s["q_start"][:-1]
    tok = torch.arange(s["n"], device="cuda")
    seq = torch.searchsorted(s["q_start"][1:].long(), tok, right=True)
    at = s["kv_len"].long()[seq] - q_len.long()[seq] + tok - s["q_start"].long()[seq]
    return at, s["table"][seq, at // B].long(), at % B


def _rescaled(pages, scale, layer, page, row, x, largest, most):
    """The rows x (float32) written into 8-bit pages: the pages' scales grow to hold `largest` of each row and head (or
    start anew where row 0 is written), and the codes of the rows before follow."""
    n_pages, G = scale.shape[0], x.shape[1]
    two = lambda e: ((e.int() + 127) << 23).view(torch.float32)  # noqa: E731  (2^e)
    need = torch.zeros(n_pages, G, device="cuda").index_reduce_(0, page, largest, "amax")
    m, e = torch.frexp(need / most)                       # need = m 2^e most, m in [1/2, 1)
    e = torch.where(need > 0, e - (m == 0.5).int(), E_LEAST)
    e = e.clamp(E_LEAST, E_MOST)
    e = torch.where(two(e) * most < need, e + 1, e).clamp(E_LEAST, E_MOST)   # the division rounded down
    first = torch.full((n_pages,), B, device="cuda").index_reduce_(0, page, row, "amin")       # B: no row written
    old = scale[:, layer]
    new = torch.where((first == 0)[:, None], two(e), torch.maximum(old, two(e)))
    new = torch.where((first < B)[:, None], new, old)
    before, at = (torch.arange(B, device="cuda") < first[:, None]).logical_and((first < B)[:, None]).nonzero(as_tuple=True)
    pages[before, layer, :, at] = _codes(_values(pages[before, layer, :, at]) * (old / new)[before][:, :, None])
    scale[:, layer] = new
    pages[page, layer, :, row] = _codes(x / new[page][:, :, None])


def _append(s, c):
    k, v, layer = s["k_new"], _v_of(s), s["layer"]
    if own:
        s["ctx"].append_kv(s["batch"], s["cache"], layer, k, v, raw_k_pages=s["raw"])
    else:
        at, page, row = _where(s)
        cos, sin = (t[:, None] for t in _angles(at, c))
        raw, v = k.float(), v.float()
        rot = _rotate(raw, cos, sin)
        if c["kv"] == "e4m3":
            _rescaled(s["k"], s["ks"], layer, page, row, rot, raw.abs().amax(-1), K_MOST)
            _rescaled(s["v"], s["vs"], layer, page, row, v, v.abs().amax(-1), V_MOST)
            if s["raw"] is not None:
                s["raw"][page, layer, :, row] = _codes(raw / s["ks"][page, layer][:, :, None])
        else:
            s["k"][page, layer, :, row] = rot.to(s["k"].dtype)
            s["v"][page, layer, :, row] = v.to(s["v"].dtype)
            if s["raw"] is not None:
                s["raw"][page, layer, :, row] = raw.to(s["k"].dtype)
    pages = [s["k"], s["v"]] + ([s["raw"]] if s["raw"] is not None else [])
    if c["kv"] != "e4m3":
        return pages
    return [p.view(torch.float8_e4m3fn) for p in pages] + [s["ks"], s["vs"]]


# ---- attention over the paged cache

def _attend(s, c):
    scale = 1.0 / math.sqrt(c["d"])
    if own:
        s["ctx"].attend(s["batch"], s["cache"], s["layer"], s["q"], s["out"], lse=s["lse"], scale=scale, causal=c["causal"])
        return {"out": s["out"], "lse": s["lse"]}
    S, G, H, d, Q = c["seqs"], c["G"], c["H"], c["d"], s["max_q"]
    table = s["table"].long()

    def gathered(pages, scales):
        x = pages[table, s["layer"]]                                              # [S][pages][G][32][d]
        x = x.float() if scales is None else _values(x) * scales[table, s["layer"]][..., None, None]
        return x.transpose(1, 2).reshape(S, G, table.shape[1] * B, d)

    q_len = (s["q_start"][1:] - s["q_start"][:-1]).long()
    i = torch.arange(Q, device="cuda")
    mine = i < q_len[:, None]                                                     # [S][Q]
    tok = (s["q_start"][:-1].long()[:, None] + i).clamp(max=s["n"] - 1)
    q = s["q"].float()[tok].view(S, Q, G, H // G, d).permute(0, 2, 3, 1, 4).reshape(S, G, H // G * Q, d)
    p = torch.matmul(q, gathered(s["k"], s["ks"]).transpose(2, 3)).mul_(scale).view(S, G, H // G, Q, -1)
    j = torch.arange(p.shape[-1], device="cuda")
    last = s["kv_len"].long()[:, None] - 1 + ((i - q_len[:, None] + 1) if c["causal"] else 0 * i)   # [S][Q]
    p.masked_fill_((j > last[..., None])[:, None, None], float("-inf"))
    most = p.amax(-1, keepdim=True)
    p.sub_(most.clamp(min=-3e38)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(S, G, H // G * Q, -1), gathered(s["v"], s["vs"])).view(S, G, H // G, Q, d)
    o = (o / total.clamp(min=1e-38)).permute(0, 3, 1, 2, 4).reshape(S, Q, H, d)
    lse = (most + total.log()).permute(0, 3, 1, 2, 4).reshape(S, Q, H)
    return {"out": o[mine].to(s["q"].dtype), "lse": lse[mine]}


# ---- the Mean-K index of 8-bit pages with scales

def _index(s, c):
    n, first = c["blocks"], c["first"]
    if own:
        s["ctx"].build_index(s["k"], first, n, s["index"], s["raw"], k_scale=s["ks"])
    else:
        cos, sin = _angles(torch.arange(first * B, (first + n) * B, device="cuda"), c)
        cos, sin = (t.view(n, 1, 1, B, -1) for t in (cos, -sin))
        raw = _rotate(_values(s["k"]), cos, sin)
        s["index"][:, :, first:first + n] = (raw.mean(3) * s["ks"][..., None]).permute(1, 2, 0, 3).to(s["index"].dtype)
        if s["raw"] is not None:
            s["raw"].copy_(_codes(raw))
    return [s["index"]] + ([s["raw"].view(torch.float8_e4m3fn)] if s["raw"] is not None else [])


def work(case):
    c = case
    act = DT[c["act"]].itemsize
    if c["op"] == "norm":
        e = c["tokens"] * (c["H"] + c["G"]) * c["d"]
        return {"bytes": e * act * (3 if c["free"] else 2) + c["tokens"] * c["d"] * 4, "flops": 10 * e}
    b = DT[c["kv"]].itemsize
    if c["op"] == "index":
        e = c["blocks"] * c["L"] * c["G"] * B * c["d"]
        return {"bytes": e * b * (2 if c["raw"] else 1) + e // B * 2 + e // B // c["d"] * 4, "flops": 4 * e}
    lens, row = _lengths(c), c["G"] * c["d"]
    if c["op"] == "append":
        n = sum(q for q, _ in lens)
        return {"bytes": n * row * (2 * act + (3 if c["raw"] else 2) * b), "flops": 4 * n * row}
    seen = sum(q * kv - (q * (q - 1) // 2 if c["causal"] else 0) for q, kv in lens if kv)
    n = sum(q for q, _ in lens)
    cache = sum(-(-kv // B) * 4 + kv * row * 2 * b + (-(-kv // B) * c["G"] * 8 if b == 1 else 0) for _, kv in lens)
    return {"bytes": cache + n * c["H"] * (c["d"] * 2 * act + 4), "flops": 4 * seen * c["H"] * c["d"]}


# ---- the same from the definitions, in 64 bits

def _turn(x, pos, c, sign=1.0):
    """Each token's pairs (i, i + d/2) turned by pos theta^(-2i/d): as complex numbers."""
    h = c["d"] // 2
    a = pos.double()[:, None] * torch.pow(torch.tensor(float(c["theta"]), dtype=torch.float64, device="cuda"),
                                          -2.0 * torch.arange(h, dtype=torch.float64, device="cuda") / c["d"])
    z = torch.complex(x[..., :h], x[..., h:]) * torch.polar(torch.ones_like(a), sign * a)
    return torch.cat((z.real, z.imag), -1)


def _decoded(codes):
    return codes.view(torch.float8_e4m3fn).double()


def _to_8(x):
    """The nearest e4m3 value (ties to the even mantissa), of 64-bit values."""
    m, e = torch.frexp(x.abs().clamp(max=448.0))
    step = torch.exp2((e.double() - 4).clamp(min=-9))
    return torch.copysign(torch.round(x.abs().clamp(max=448.0) / step) * step, x)


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    G, H, d = c["G"], c["H"], c["d"]
    if c["op"] == "norm":
        n, got = c["tokens"], []
        x = s["qkv"].double()[:, :(H + G) * d].view(n, H + G, d)
        y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / d + s["eps"])
        parts = (y[:, :H] * s["qw"].double(), y[:, H:] * s["kw"].double())
        for p in parts:
            got.append(_turn(p.transpose(0, 1), s["pos"], c).transpose(0, 1))
        return got + (list(parts) if c["free"] else [])
    if c["op"] == "index":
        first, n = c["first"], c["blocks"]
        index, raws = s["index"].double(), []
        for b in range(n):
            raw = _turn(_decoded(s["k"][b]), torch.arange((first + b) * B, (first + b + 1) * B, device="cuda"), c, -1.0)
            index[:, :, first + b] = raw.sum(2) / B * s["ks"][b].double()[..., None]
            raws.append(_to_8(raw).to(torch.float32))
        return [index] + ([torch.stack(raws)] if c["raw"] else [])
    lens, lay = _lengths(c), s["layer"]
    if c["op"] == "append":
        eight = c["kv"] == "e4m3"
        table, whole = s["table"].tolist(), (lambda t: _decoded(t).float()) if eight else (lambda t: t.float())
        k, v = whole(s["k"]), whole(s["v"])
        raw = torch.zeros_like(k) if c["raw"] else None
        values, at = _v_of(s).double(), 0
        for i, (q, kv) in enumerate(lens):
            for b in range((kv - q) // B, -(-kv // B)):
                lo, hi = max(b * B, kv - q), min((b + 1) * B, kv)
                p, rows = table[i][b], slice(lo - b * B, hi - b * B)
                xk = s["k_new"][at + lo - (kv - q):at + hi - (kv - q)].double()
                xv = values[at + lo - (kv - q):at + hi - (kv - q)]
                rk = _turn(xk.transpose(0, 1), torch.arange(lo, hi, device="cuda"), c)
                xk, xv = xk.transpose(0, 1), xv.transpose(0, 1)
                if not eight:
                    k[p, lay, :, rows], v[p, lay, :, rows] = rk, xv
                    if raw is not None:
                        raw[p, lay, :, rows] = xk
                    continue
                for x, largest, most, pages, scales in ((rk, xk, K_MOST, k, s["ks"]), (xv, xv, V_MOST, v, s["vs"])):
                    t = torch.ceil(torch.log2(largest.abs().amax((1, 2)) / most)).clamp(E_LEAST, E_MOST).cpu().exp2().cuda()
                    if lo % B:
                        old = scales[p, lay].double()
                        t = torch.maximum(t, old)
                        pages[p, lay, :, :lo % B] = _to_8(pages[p, lay, :, :lo % B].double() * (old / t)[:, None, None]).float()
                    scales[p, lay] = t
                    pages[p, lay, :, rows] = _to_8(x / t[:, None, None]).float()
                    if x is rk and raw is not None:
                        raw[p, lay, :, rows] = _to_8(xk / t[:, None, None]).float()
            at += q
        return [k, v] + ([raw] if raw is not None else []) + ([s["ks"].double(), s["vs"].double()] if eight else [])
    out = torch.zeros(s["n"], H, d, dtype=torch.float64, device="cuda")
    lse = torch.full((s["n"], H), float("-inf"), dtype=torch.float64, device="cuda")
    at = 0
    for i, (q, kv) in enumerate(lens):
        if kv:
            page = s["table"][i, :-(-kv // B)].long()
            hidden = torch.arange(kv, device="cuda") > torch.arange(kv - q, kv, device="cuda")[:, None]
            for h in range(H):
                g = h // (H // G)
                keys, vals = (t[page, lay, g] for t in (s["k"], s["v"]))
                if c["kv"] == "e4m3":
                    keys, vals = (_decoded(t) * sc[page, lay, g].double()[:, None, None] for t, sc in ((keys, s["ks"]), (vals, s["vs"])))
                keys, vals = (t.double().reshape(-1, d)[:kv] for t in (keys, vals))
                x = s["q"][at:at + q, h].double() @ keys.T / math.sqrt(d)
                if c["causal"]:
                    x[hidden] = float("-inf")
                lse[at:at + q, h] = torch.logsumexp(x, -1)
                out[at:at + q, h] = torch.softmax(x, -1) @ vals
        at += q
    return {"out": out, "lse": lse}
