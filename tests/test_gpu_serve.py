"""The calls around the recall on the GPU, against their 64-bit definitions:
kvm_qk_norm_rope, kvm_append_kv, kvm_attend and kvm_build_index_scaled, their
refusals, and a run of them together with the recall of KVMem ("Virtualizing
Million-Token Agent Workspaces on a Consumer GPU", §4.3 and §4.4).

Tolerances come from the arithmetic and are stated where they are used: one
rounding to the output type (half a step), plus what float32 sums can leave."""
import math

import pytest
import torch

import serve_ref as ref
from serve_ref import EPS2, TDT, U, Paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvm():
    import paged_kv_cache_meank_gb300 as kvm
    from paged_kv_cache_meank_gb300 import build
    build.build()
    assert torch.cuda.is_available()
    return kvm


_CTX = {}


def context(kvm, **kw):
    positions = kw.pop("positions", 4096)
    key = (positions,) + tuple(sorted(kw.items()))
    if key not in _CTX:
        _CTX[key] = kvm.Context(kvm.config_for(ref.workload(**kw), max_positions=positions))
    return _CTX[key]


# ---------------------------------------------------------------- attention

def run_attend(kvm, p, causal, *, packed=False, lse=True, scale=None, ctx=None):
    ctx = ctx or context(kvm, L=p.L, G=p.G, H=p.H, d=p.d, kv=p.kv, act=p.act)
    batch, cache = p.on(ctx)
    scale = p.d ** -0.5 if scale is None else scale
    q = p.q.cuda()
    if packed:                       # rows of a wider buffer
        wide = torch.randn(p.n, p.H + 3, p.d, device="cuda").to(TDT[p.act])
        wide[:, 1:1 + p.H] = q
        q = wide[:, 1:1 + p.H]
        out = torch.full((p.n, p.H + 2, p.d), 7.0, device="cuda").to(TDT[p.act])[:, :p.H]
    else:
        out = torch.full((p.n, p.H, p.d), 7.0, device="cuda").to(TDT[p.act])
    le = torch.full((p.n, p.H), 7.0, device="cuda") if lse else None
    ctx.attend(batch, cache, p.layer, q, out, lse=le, scale=scale, causal=causal)
    ctx.sync()
    check_attend(p, causal, scale, out, le)
    return out, le


def check_attend(p, causal, scale, out, lse):
    want, wl, absv, ds = p.reference(scale, causal)
    got = out.cpu().double()
    first, last = p.q_start[0], p.q_start[-1]
    assert (got[:first] == 7).all() and (got[last:] == 7).all(), "rows outside the sequences"
    got, want, absv, ds = (t[first:last] for t in (got, want, absv, ds))
    assert bool(torch.isfinite(got).all())
    n_keys = max(p.max_kv, 1)
    err = (got - want).abs()
    tol = ref.attend_tolerance(want, absv, ds, p.act, p.kv, n_keys)
    assert (err <= tol).all(), f"worst error / tolerance {(err / tol).max():.3g}"
    if lse is not None:
        gl = lse.cpu().double()
        assert (gl[:first] == 7).all() and (gl[last:] == 7).all()
        gl, wl = gl[first:last], wl[first:last]
        empty = wl == -math.inf
        assert torch.equal(gl == -math.inf, empty)
        el = (gl - wl)[~empty].abs()
        tl = (ds[~empty] * 2 + (n_keys + 16) * U + 4 * U * wl[~empty].abs())
        assert (el <= tl).all(), f"lse: worst {(el / tl).max():.3g}"


TYPES = [("f32", "f32", False), ("f32", "bf16", False), ("f32", "e4m3", True), ("bf16", "f32", False),
         ("bf16", "bf16", False), ("bf16", "e4m3", False), ("bf16", "e4m3", True)]
IDS = [f"{a}-{k}{'-scaled' if s else ''}" for a, k, s in TYPES]


@pytest.mark.parametrize("act,kv,scaled", TYPES, ids=IDS)
@pytest.mark.parametrize("d", [64, 128])
def test_attend_decode_ragged(kvm, act, kv, scaled, d):
    """One token each: every edge of a page, a sequence without keys, one
    without tokens, unused batch rows before and behind, padded tables."""
    lens = [(1, 1), (1, 31), (1, 32), (1, 33), (0, 64), (1, 0), (1, 300), (1, 95), (1, 1025)]
    p = Paged(lens, L=2, layer=1, G=2, H=12, d=d, kv=kv, act=act, scaled=scaled, lead=2, tail=3,
              table_pad=2, seed=3)
    run_attend(kvm, p, True, packed=True)
    run_attend(kvm, p, False, lse=False)


@pytest.mark.parametrize("act,kv,scaled", TYPES, ids=IDS)
@pytest.mark.parametrize("G,H", [(1, 1), (2, 2), (2, 14), (1, 8), (4, 12), (1, 48)])
def test_attend_head_layouts(kvm, act, kv, scaled, G, H):
    p = Paged([(2, 70), (5, 163), (3, 3)], G=G, H=H, d=64, kv=kv, act=act, scaled=scaled, seed=G + H)
    run_attend(kvm, p, True)


@pytest.mark.parametrize("act,kv,scaled", TYPES, ids=IDS)
@pytest.mark.parametrize("q,kv_len", [(1, 2000), (4, 77), (7, 640), (32, 1000), (65, 65), (130, 517),
                                      (257, 900)])
def test_attend_lengths(kvm, act, kv, scaled, q, kv_len):
    """One sequence from a decoded token to a chunk of prefill, both masks."""
    p = Paged([(q, kv_len)], G=2, H=6, d=128, kv=kv, act=act, scaled=scaled, seed=q)
    run_attend(kvm, p, True)
    run_attend(kvm, p, False, packed=True)


@pytest.mark.parametrize("act,kv,scaled", TYPES, ids=IDS)
def test_attend_rows_that_see_nothing(kvm, act, kv, scaled):
    """More new tokens than keys: the first rows see none (out 0, lse -inf)."""
    p = Paged([(40, 7), (9, 0), (33, 33), (3, 2)], G=1, H=3, d=64, kv=kv, act=act, scaled=scaled, seed=5)
    run_attend(kvm, p, True)


@pytest.mark.parametrize("act,kv,scaled", [TYPES[0], TYPES[4], TYPES[6]], ids=[IDS[0], IDS[4], IDS[6]])
@pytest.mark.parametrize("q", [1, 6, 70])
def test_attend_ragged_chunks(kvm, act, kv, scaled, q):
    """Many sequences of mixed lengths, more than one CTA's run each."""
    lens = [(1 + (i * 7) % q if q > 1 else 1, 1 + (i * 389) % 1500 + q) for i in range(21)]
    p = Paged(lens, G=2, H=8, d=128, kv=kv, act=act, scaled=scaled, seed=q, own_rows=scaled)
    run_attend(kvm, p, True)


@pytest.mark.parametrize("act,kv", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "e4m3")])
@pytest.mark.parametrize("q", [1, 40])
def test_attend_sharp_and_flat_weights(kvm, act, kv, q):
    """Scores far apart (one key takes all the weight, others underflow), a
    softmax scale of zero, a negative one, and a growing maximum."""
    for scale, qstd in ((4.0, 3.0), (0.0, 1.0), (-0.3, 1.0)):
        p = Paged([(q, 700), (q, 90)], G=2, H=4, d=64, kv=kv, act=act, scaled=kv == "e4m3", seed=9,
                  qstd=qstd)
        run_attend(kvm, p, True, scale=scale)
    # keys that grow along the sequence, so that the running maximum rises in every tile
    p = Paged([(q, 1200)], G=1, H=2, d=64, kv=kv, act=act, seed=10)
    if kv != "e4m3":
        one = torch.ones(64).to(TDT[kv])
        for b in range(-(-1200 // 32)):
            rows = min(32, 1200 - 32 * b)
            page = int(p.table[0, b])
            p.k[page, 0, 0, :rows] = (one * (0.02 * b)).to(TDT[kv])
        p.q[:] = 1.0
        run_attend(kvm, p, True, scale=1.0)


@pytest.mark.parametrize("act,kv,scaled", [TYPES[0], TYPES[4], TYPES[6]], ids=[IDS[0], IDS[4], IDS[6]])
def test_attend_is_deterministic(kvm, act, kv, scaled):
    """Split rows are joined in a fixed order: the same bits on every run."""
    for q in (1, 24, 200):
        p = Paged([(q, 1900), (q, 333)], G=2, H=12, d=128, kv=kv, act=act, scaled=scaled, seed=11)
        a, la = run_attend(kvm, p, True)
        b, lb = run_attend(kvm, p, True)
        assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("act,kv,scaled", [TYPES[0], TYPES[4], TYPES[6]], ids=[IDS[0], IDS[4], IDS[6]])
@pytest.mark.parametrize("q", [1, 50])
def test_attend_in_a_graph_follows_the_lengths(kvm, act, kv, scaled, q):
    """A captured call reads lengths and tables when it is launched."""
    p = Paged([(q, 900), (q, 450)], G=2, H=4, d=64, kv=kv, act=act, scaled=scaled, seed=12)
    ctx = context(kvm, L=1, G=2, H=4, d=64, kv=kv, act=act)
    batch, cache = p.on(ctx)
    q_d = p.q.cuda()
    out = torch.zeros(p.n, p.H, p.d, device="cuda", dtype=TDT[act])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        ctx.attend(batch, cache, 0, q_d, out)
    for kv_a, kv_b in ((900, 450), (q, 33 + q), (640, 450)):
        batch.tensors[1].copy_(torch.tensor([kv_a, kv_b], dtype=torch.int32))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        p.lens = [(q, kv_a), (q, kv_b)]
        check_attend(p, True, p.d ** -0.5, out, None)
    ctx.sync()


def test_attend_bad_tables_are_flagged_and_skipped(kvm):
    """Pages, lengths and scale rows out of range raise the device flag; the
    other sequences' rows are right and nothing else is written."""
    for act, kv, scaled in (("f32", "f32", False), ("bf16", "bf16", False), ("bf16", "e4m3", True)):
        for q in (1, 40):
            ctx = context(kvm, L=1, G=2, H=4, d=64, kv=kv, act=act)
            for what in ("page", "negative page", "kv_len", "q_start", "row"):
                if what == "row" and not scaled:
                    continue
                p = Paged([(q, 200), (q, 100)], G=2, H=4, d=64, kv=kv, act=act, scaled=scaled,
                          seed=13, own_rows=scaled)
                batch, cache = p.on(ctx)
                q_start, kv_len, table, rows = batch.tensors
                if what == "page":
                    table[0, 2] = cache.c.n_pages
                elif what == "negative page":
                    table[0, 0] = -1
                elif what == "kv_len":
                    kv_len[0] = p.max_kv + 1
                elif what == "q_start":
                    q_start[0] = -1
                else:
                    rows[0, 1] = cache.c.n_scale_rows
                out = torch.full((p.n, 4, 64), 7.0, device="cuda").to(TDT[act])
                ctx.attend(batch, cache, 0, p.q.cuda(), out)
                with pytest.raises(kvm.KvmError) as e:
                    ctx.sync()
                assert e.value.name == "KVM_ERR_DEVICE", what
                ctx.sync()                       # reported once
                want, _, absv, ds = p.reference(64 ** -0.5, True)
                err = (out.cpu().double() - want)[q:].abs()
                tol = ref.attend_tolerance(want, absv, ds, act, kv, 200)[q:]
                assert (err <= tol).all(), what
                if what in ("kv_len", "q_start"):
                    assert (out[:q] == 7).all(), what


def test_attend_scale_that_is_no_power_of_two_is_flagged(kvm):
    for q in (1, 40):
        ctx = context(kvm, L=1, G=2, H=4, d=64, kv="e4m3", act="bf16")
        for bad in (0.3, 0.0, -0.5, math.inf, math.nan, 2.0 ** -110):
            p = Paged([(q, 100)], G=2, H=4, d=64, kv="e4m3", act="bf16", scaled=True, seed=14)
            p.vs[int(p.table[0, 1]), 0, 1] = bad
            batch, cache = p.on(ctx)
            out = torch.zeros(p.n, 4, 64, device="cuda", dtype=torch.bfloat16)
            ctx.attend(batch, cache, 0, p.q.cuda(), out)
            with pytest.raises(kvm.KvmError) as e:
                ctx.sync()
            assert e.value.name == "KVM_ERR_DEVICE", bad


# ---------------------------------------------------------------- norm + rotation

@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,H,n", [(1, 1, 1), (2, 4, 1), (8, 48, 1), (2, 14, 37), (3, 9, 300), (8, 48, 3000)])
def test_norm_rope(kvm, act, d, G, H, n):
    ctx = context(kvm, G=G, H=H, d=d, kv=act, act=act, theta=1e6, positions=70000)
    g = torch.Generator().manual_seed(n + d)
    dt = TDT[act]
    qkv = (torch.randn(n, (H + 2 * G) * d, generator=g) * 3).to(dt)
    qkv[0, :d] = 0                                       # a head of zeros
    qw, kw = ((1 + 0.3 * torch.randn(d, generator=g)).to(dt) for _ in range(2))
    pos = torch.randint(0, 70000, (n,), generator=g, dtype=torch.int32)
    pos[0] = 69999
    dev = qkv.cuda()
    q, k = dev[:, :H * d].view(n, H, d), dev[:, H * d:(H + G) * d].view(n, G, d)
    new = lambda h: torch.full((n, h, d), 7.0, device="cuda").to(dt)     # noqa: E731
    for weights in (True, False):
        qf, qr, kf, kr = new(H), new(H), new(G), new(G)
        ctx.qk_norm_rope(pos.cuda(), q=q, k=k, q_weight=qw.cuda() if weights else None,
                         k_weight=kw.cuda() if weights else None, eps=1e-6, q_free=qf, q_rot=qr,
                         k_free=kf, k_rot=kr)
        ctx.sync()
        for x, w, free, rot in ((q, qw, qf, qr), (k, kw, kf, kr)):
            y = x.cpu().double()
            if weights:
                y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w.double()
            r = ref.rotate(y.transpose(0, 1), pos, 1e6).transpose(0, 1)
            # the mean's d roundings (halved by the root), rsqrtf's two steps, two
            # products; the rotation's products, sum and rounded cos / sin
            f32 = (d / 2 + 4 + 2) * U if weights else 0.0
            for got, want, more in ((free, y, 0.0), (rot, r, 6 * U)):
                err = (got.cpu().double() - want).abs()
                tol = EPS2[act] * want.abs() + (f32 + more) * (1 + EPS2[act]) * 1.5 * ref.pair_mag(y) + 1e-30
                assert (err <= tol).all(), float((err / tol).max())
    # one side, one output, in place
    packed = k.contiguous()
    both = packed.clone()
    ctx.qk_norm_rope(pos.cuda(), k=both, k_weight=kw.cuda(), k_rot=both)
    alone = new(G)
    ctx.qk_norm_rope(pos.cuda(), k=packed, k_weight=kw.cuda(), k_rot=alone)
    ctx.sync()
    assert torch.equal(both, alone)


def test_norm_rope_positions_out_of_range_are_flagged_and_skipped(kvm):
    ctx = context(kvm, G=2, H=4, d=64, kv="bf16", act="bf16", positions=128)
    x = torch.randn(3, 4, 64, device="cuda").bfloat16()
    for bad in (128, -1, 2 ** 31 - 1):
        out = torch.full_like(x, 7.0)
        ctx.qk_norm_rope(torch.tensor([5, bad, 127], dtype=torch.int32, device="cuda"), q=x, q_rot=out)
        with pytest.raises(kvm.KvmError) as e:
            ctx.sync()
        assert e.value.name == "KVM_ERR_DEVICE"
        assert (out[1] == 7).all() and not (out[0] == 7).all() and not (out[2] == 7).all()


# ---------------------------------------------------------------- append

def append_reference(p, k, v, pos, theta, raw):
    """The pages, scales and raw pages after the append, in 64 bits: (values
    unrounded where written, else as stored; the scales; which rows were written)."""
    eight = p.kv == "e4m3"
    kp, vp = ref.values(p.k, p.kv), ref.values(p.v, p.kv)
    rp = ref.values(raw, p.kv)
    ks, vs = (t.clone() if t is not None else None for t in (p.ks, p.vs))
    wrote = torch.zeros(p.k.shape[0], 32, dtype=torch.bool)
    for s, (qn, kvl) in enumerate(p.lens):
        a = p.q_start[s]
        for b in range((kvl - qn) // 32, -(-kvl // 32)):
            lo, hi = max(32 * b, kvl - qn), min(32 * b + 32, kvl)
            if lo >= hi:
                continue
            page = int(p.table[s, b])
            row = int((p.rows if p.rows is not None else p.table)[s, b])
            at = slice(lo - 32 * b, hi - 32 * b)
            tok = slice(a + lo - (kvl - qn), a + hi - (kvl - qn))
            wrote[page, at] = True
            xk, xv = k[tok].double().transpose(0, 1), v[tok].double().transpose(0, 1)
            rk = ref.rotate(xk, pos[tok], theta)
            for g in range(p.G):
                sk = sv = 1.0
                if p.scaled:
                    fin = lambda t: float(t[torch.isfinite(t)].abs().max())     # noqa: E731
                    sk, sv = ref.scale_for(fin(xk[g]), 316.75), ref.scale_for(fin(xv[g]), 448.0)
                    if lo % 32:
                        ok, ov = float(ks[row, p.layer, g]), float(vs[row, p.layer, g])
                        sk, sv = max(sk, ok), max(sv, ov)
                        n = lo % 32
                        for pages, f in ((kp, ok / sk), (vp, ov / sv), (rp, ok / sk)):
                            old = pages[page, p.layer, g, :n]
                            pages[page, p.layer, g, :n] = ref.decode(ref.encode(old * f))
                    ks[row, p.layer, g], vs[row, p.layer, g] = sk, sv
                kp[page, p.layer, g, at] = rk[g] / sk
                vp[page, p.layer, g, at] = xv[g] / sv
                rp[page, p.layer, g, at] = xk[g] / sk
    return kp, vp, rp, ks, vs, wrote


def check_append(kvm, p, *, act, theta=1e4, given=False, raw=True, wild=False, seed=0):
    ctx = context(kvm, L=p.L, G=p.G, H=p.H, d=p.d, kv=p.kv, act=act, theta=theta, positions=4096)
    g = torch.Generator().manual_seed(seed)
    n = p.n
    # entries of many sizes, so that scales differ and grow
    size = torch.exp2(torch.randint(-6, 7, (n, p.G, 1), generator=g).float())
    k, v = ((torch.randn(n, p.G, p.d, generator=g) * size).to(TDT[act]) for _ in range(2))
    k[0] = 0
    if wild:
        k[1, 0, 3], v[1, 0, 5], v[2, 0, 1] = 1e30, -1e30, 1e-30
    pos = torch.randint(0, 4096, (n,), generator=g, dtype=torch.int32)
    if not given:
        for s, (qn, kvl) in enumerate(p.lens):
            a = p.q_start[s]
            pos[a:a + qn] = torch.arange(kvl - qn, kvl, dtype=torch.int32)
    for t in (p.k, p.v):                                  # finite stale rows where codes may be rescaled
        if p.kv == "e4m3":
            t[t == 0x7F] = 0x35
    raw_pages = torch.randint(0, 100, p.k.shape, generator=g).to(TDT[p.kv])
    batch, cache = p.on(ctx)
    wide = torch.randn(n, p.G + 1, p.d).to(TDT[act])
    wide[:, 1:] = v
    dv = wide.cuda()[:, 1:]
    draw = raw_pages.cuda() if raw else None
    ctx.append_kv(batch, cache, p.layer, k.cuda(), dv, positions=pos.cuda() if given else None,
                  raw_k_pages=draw)
    ctx.sync()
    kp, vp, rp, ks, vs, wrote = append_reference(p, k, v, pos, theta, raw_pages)
    if p.scaled:
        assert torch.equal(p.dks.cpu(), ks) and torch.equal(p.dvs.cpu(), vs)
    pairs = [(p.dk, kp, True), (p.dv, vp, False)] + ([(draw, rp, False)] if raw else [])
    for got, want, rotated in pairs:
        got = ref.values(got, p.kv)
        mask = torch.zeros_like(got, dtype=torch.bool)
        mask[:, p.layer] = wrote[:, None, :, None]
        same = (got == want) | (torch.isnan(got) & torch.isnan(want))
        assert same[~mask].all(), "rows that were not written"
        sat = want.clamp(-448, 448) if p.kv == "e4m3" else want
        tol = EPS2[p.kv] * sat.abs()
        if rotated:                       # the products, the sum, cos and sin, each rounded once
            tol = tol + 4 * U * ref.pair_mag(want)
        if p.kv == "e4m3":
            tol = tol.clamp(min=2.0 ** -10)              # half the subnormal step
            if rotated:
                tol = tol + 4 * U * ref.pair_mag(want)
        err = (got - sat).abs()
        assert (err[mask] <= tol[mask] + 1e-38).all(), float((err / tol)[mask].max())


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("kv,scaled", [("f32", False), ("bf16", False), ("e4m3", False), ("e4m3", True)])
@pytest.mark.parametrize("d", [64, 128])
def test_append(kvm, act, kv, scaled, d):
    """Every place in a page a run can begin and end, one token to several
    pages, a sequence that adds nothing, pages and rows permuted."""
    lens = [(1, 1), (1, 32), (1, 33), (5, 34), (32, 32), (33, 64), (70, 133), (0, 40), (31, 63), (2, 95)]
    p = Paged(lens, L=2, layer=1, G=3, H=3, d=d, kv=kv, scaled=scaled, lead=1, tail=2, seed=21,
              own_rows=scaled, table_pad=1)
    check_append(kvm, p, act=act, given=False)
    p = Paged(lens[::-1], L=1, G=2, H=2, d=d, kv=kv, scaled=scaled, seed=22)
    check_append(kvm, p, act=act, given=True, raw=False, wild=kv == "e4m3", seed=4)


def test_append_token_by_token_keeps_every_token(kvm):
    """40 tokens of growing size one by one into scaled pages: every code stays
    within its block's final rounding of the value (each growth halves at most
    what was a half step, and rounds again only entries that became subnormal)."""
    d, G = 64, 2
    ctx = context(kvm, L=1, G=G, H=2, d=d, kv="e4m3", act="bf16", positions=4096)
    g = torch.Generator().manual_seed(31)
    n = 40
    k, v = ((torch.randn(n, G, d, generator=g) * torch.exp2(torch.arange(n).float() / 4 - 6)[:, None, None])
            .bfloat16() for _ in range(2))
    kp, vp = (torch.zeros(3, 1, G, 32, d, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.ones(3, 1, G, device="cuda") for _ in range(2))
    cache = ctx.cache(kp, vp, ks, vs)
    table = torch.tensor([[2, 0]], dtype=torch.int32, device="cuda")
    q_start = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    kv_len = torch.zeros(1, dtype=torch.int32, device="cuda")
    batch = ctx.batch(q_start, kv_len, table, n_tokens=1, max_q_len=1, max_kv_len=64)
    for t in range(n):
        kv_len.fill_(t + 1)
        ctx.append_kv(batch, cache, 0, k[t:t + 1].cuda(), v[t:t + 1].cuda())
    ctx.sync()
    for b, page in ((0, 2), (1, 0)):
        rows = slice(32 * b, min(n, 32 * b + 32))
        for x, pages, sc in ((ref.rotate(k[rows].double().transpose(0, 1), torch.arange(n)[rows], 1e4), kp, ks),
                             (v[rows].double().transpose(0, 1), vp, vs)):
            s = sc[page, 0].cpu().double()[:, None, None]
            got = ref.decode(pages[page, 0])[:, :x.shape[1]] * s
            # half a step, and half the final subnormal step for each of the growths
            # (each adds at most that: ten of them)
            tol = 2.0 ** -4 * x.abs() + 11 * 2.0 ** -10 * s
            assert ((got - x).abs() <= tol).all()
        want = ref.scale_for(float(k[rows].double().abs().amax((0, 2))[0]), 316.75)
        assert float(ks[page, 0, 0]) == want


def test_append_refuses_and_flags(kvm):
    ctx = context(kvm, L=1, G=2, H=4, d=64, kv="e4m3", act="bf16")
    for what in ("page", "short", "long", "row", "position"):
        p = Paged([(3, 40), (2, 70)], G=2, H=4, d=64, kv="e4m3", act="bf16", scaled=True, seed=41,
                  own_rows=True)
        batch, cache = p.on(ctx)
        q_start, kv_len, table, rows = batch.tensors
        pos = torch.arange(5, dtype=torch.int32, device="cuda")
        if what == "page":
            table[0, 1] = cache.c.n_pages + 3
        elif what == "short":
            kv_len[0] = 2
        elif what == "long":
            kv_len[0] = 71
        elif what == "row":
            rows[0, 1] = -1
        else:
            pos[:3] = 4096
        before = p.dk.clone()
        x = torch.randn(5, 2, 64, device="cuda").bfloat16()
        ctx.append_kv(batch, cache, 0, x, x, positions=pos)
        with pytest.raises(kvm.KvmError) as e:
            ctx.sync()
        assert e.value.name == "KVM_ERR_DEVICE", what
        changed = (p.dk != before).flatten(1).any(1).nonzero().flatten().tolist()
        assert changed == [int(p.table[1, 2])], what          # the other sequence's page alone


# ---------------------------------------------------------------- scaled Mean-K

@pytest.mark.parametrize("index", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("L,G,n,first", [(1, 1, 1, 0), (2, 3, 7, 4), (5, 8, 40, 9)])
def test_index_of_scaled_pages(kvm, index, d, L, G, n, first):
    wl = ref.workload(L=L, G=G, H=G, d=d, kv="e4m3", act="bf16", index=index, n_blocks=64, theta=1e6)
    ctx = kvm.Context(kvm.config_for(wl))
    g = torch.Generator().manual_seed(n + d)
    codes = (torch.randn(n, L, G, 32, d, generator=g) * 60).to(torch.float8_e4m3fn).view(torch.uint8)
    ks = torch.exp2(torch.randint(-9, 4, (n, L, G), generator=g).float())
    idx = torch.full(ctx.index_shape(), 7.0, device="cuda").to(TDT[index])
    raw = torch.zeros_like(codes).cuda()
    ctx.build_index(codes.cuda(), first, n, idx, raw, k_scale=ks.cuda())
    ctx.sync()
    got = idx.cpu().double()
    assert (got[:, :, :first] == 7).all() and (got[:, :, first + n:] == 7).all()
    for b in range(n):
        pos = torch.arange(32) + 32 * (first + b)
        un = ref.rotate(ref.decode(codes[b]), pos, 1e6, -1.0)
        s = ks[b].double()[..., None]
        want = un.mean(2) * s
        # 32 float32 sums of rotated entries (4 roundings each), one rounding of the entry
        tol = EPS2[index] * want.abs() + 36 * U * s * ref.pair_mag(un).amax(2)
        assert ((got[:, :, first + b] - want).abs() <= tol).all()
        err = (ref.decode(raw[b]) - un.clamp(-448, 448)).abs()
        assert (err <= (2.0 ** -4 * un.abs()).clamp(min=2.0 ** -10) + 4 * U * ref.pair_mag(un)).all()
    # unit scales: the same as the plain call, bit for bit
    one = torch.zeros_like(idx)
    two = torch.zeros_like(idx)
    ctx.build_index(codes.cuda(), first, n, one, k_scale=torch.ones_like(ks).cuda())
    ctx.build_index(codes.cuda(), first, n, two)
    ctx.sync()
    assert torch.equal(one, two)
    ks[0, 0, 0] = 0.7
    ctx.build_index(codes.cuda(), first, n, one, k_scale=ks.cuda())
    with pytest.raises(kvm.KvmError):
        ctx.sync()
    ctx.close()


# ---------------------------------------------------------------- refusals

def test_refusals_on_the_host(kvm):
    """Every argument error is found before anything is enqueued."""
    from paged_kv_cache_meank_gb300._abi import KvmBatch, KvmCache
    import ctypes
    ctx = context(kvm, L=2, G=2, H=4, d=64, kv="bf16", act="bf16")
    lib, h = ctx.lib, ctx.handle
    p = Paged([(1, 40)], L=2, G=2, H=4, d=64, kv="bf16", act="bf16")
    batch, cache = p.on(ctx)
    q = p.q.cuda()
    out = torch.empty_like(q)
    lse = torch.empty(1, 4, device="cuda")
    pinned = torch.zeros(1 << 16, dtype=torch.bfloat16).pin_memory()
    pageable = torch.zeros(1 << 16, dtype=torch.bfloat16)
    stream = torch.cuda.current_stream().cuda_stream
    n0 = kvm.launch_count()

    def attend(b=None, c=None, layer=0, q_=q.data_ptr(), qs=256, scale=0.1, causal=1,
               o=out.data_ptr(), os_=256, ls=lse.data_ptr()):
        return lib.kvm_attend(h, ctypes.addressof(b or batch.c), ctypes.addressof(c or cache.c),
                              layer, q_, qs, scale, causal, o, os_, ls, stream)

    def but(struct, **kw):
        x = type(struct).from_buffer_copy(struct)
        for k, v in kw.items():
            setattr(x, k, v)
        return x

    bad = -1
    for kw in (dict(layer=-1), dict(layer=2), dict(q_=None), dict(o=None), dict(qs=255), dict(qs=252),
               dict(os_=100), dict(scale=math.inf), dict(scale=math.nan), dict(causal=2),
               dict(q_=q.data_ptr() + 2), dict(o=q.data_ptr()), dict(ls=lse.data_ptr() + 1),
               dict(q_=pageable.data_ptr()), dict(q_=pinned.data_ptr()), dict(o=pinned.data_ptr()),
               dict(b=but(batch.c, n_seqs=-1)), dict(b=but(batch.c, q_start=None)),
               dict(b=but(batch.c, kv_len=None)), dict(b=but(batch.c, page_table=None)),
               dict(b=but(batch.c, max_kv_len=65)), dict(b=but(batch.c, table_stride=0)),
               dict(b=but(batch.c, scale_rows=lse.data_ptr())), dict(b=but(batch.c, n_tokens=-1)),
               dict(c=but(cache.c, k_pages=None)), dict(c=but(cache.c, n_pages=-1)),
               dict(c=but(cache.c, k_pages=pinned.data_ptr())),
               dict(c=but(cache.c, k_scale=lse.data_ptr())),
               dict(c=but(cache.c, k_scale=lse.data_ptr(), v_scale=lse.data_ptr(), n_scale_rows=1))):
        assert attend(**kw) == bad, kw
    assert attend(b=but(batch.c, n_seqs=1025)) == -3
    assert lib.kvm_attend(h, None, ctypes.addressof(cache.c), 0, q.data_ptr(), 256, 0.1, 1,
                          out.data_ptr(), 256, None, stream) == bad
    for kw in (dict(n_seqs=0), dict(n_tokens=0), dict(max_q_len=0)):
        assert attend(b=but(batch.c, **kw)) == 0           # nothing to do

    kx = torch.zeros(1, 2, 64, device="cuda", dtype=torch.bfloat16)

    def append(k=kx.data_ptr(), ks=128, v=kx.data_ptr(), vs=128, pos=None, raw=None, c=None, b=None):
        return lib.kvm_append_kv(h, ctypes.addressof(b or batch.c), ctypes.addressof(c or cache.c), 0,
                                 k, ks, v, vs, pos, raw, stream)

    for kw in (dict(k=None), dict(v=None), dict(ks=64), dict(vs=132), dict(k=kx.data_ptr() + 8),
               dict(raw=cache.c.k_pages), dict(raw=cache.c.v_pages), dict(pos=lse.data_ptr() + 2),
               dict(c=but(cache.c, v_pages=cache.c.k_pages)), dict(k=pinned.data_ptr())):
        assert append(**kw) == bad, kw

    pos = torch.zeros(1, dtype=torch.int32, device="cuda")

    def norm(n=1, pos=pos.data_ptr(), q=q.data_ptr(), qs=256, k=None, ks=0, qw=None, kw=None, eps=1e-6,
             qf=None, qr=out.data_ptr(), kf=None, kr=None):
        return lib.kvm_qk_norm_rope(h, n, pos, q, qs, k, ks, qw, kw, eps, qf, qr, kf, kr, stream)

    wide = torch.zeros(2, 300, device="cuda", dtype=torch.bfloat16)
    for kw in (dict(n=-1), dict(pos=None), dict(q=None), dict(qr=None), dict(kr=out.data_ptr()),
               dict(kw=out.data_ptr()), dict(qf=out.data_ptr()), dict(eps=-1.0), dict(eps=math.nan),
               dict(qs=128), dict(qs=260), dict(q=wide.data_ptr(), qs=264, qr=wide.data_ptr()),
               dict(k=kx.data_ptr(), ks=64, kr=out.data_ptr()), dict(q=pageable.data_ptr())):
        assert norm(**kw) == bad, kw
    assert norm(n=0) == 0
    assert lib.kvm_build_index_scaled(h, kx.data_ptr(), lse.data_ptr(), 0, 1, out.data_ptr(), None,
                                      stream) == bad       # bf16 pages have no scales
    assert kvm.launch_count() == n0
    assert attend() == 0 and append() == 0 and norm() == 0
    assert kvm.launch_count() >= n0 + 3
    ctx.sync()
    with pytest.raises(ValueError):
        ctx.attend(batch, cache, 0, q.float(), out)
    with pytest.raises(ValueError):
        ctx.attend(batch, cache, 0, q[:0], out)
    with pytest.raises(ValueError):
        ctx.cache(p.dk, p.dv.float())
    with pytest.raises(ValueError):
        ctx.batch(batch.tensors[0], batch.tensors[1].long(), batch.tensors[2], n_tokens=1, max_q_len=1,
                  max_kv_len=40)
    with pytest.raises(ValueError):
        ctx.qk_norm_rope(pos.long(), q=q, q_rot=out)
    with pytest.raises(ValueError):
        ctx.append_kv(batch, cache, 0, kx[:, :1], kx)


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
def test_prefill_recall_decode(kvm, kv, graph):
    """Two layers of an agent step from end to end: a history prefilled through
    the norm, the append and the index build, the recall, then three decoded
    tokens attending over the assembled view and their own tail page, against the
    same attention in 64 bits over the pages' values; eager, and with the step and
    the decode calls captured into one graph."""
    L, G, H, d, N, V, theta = 2, 2, 12, 128, 40, 16, 1e6
    wl = ref.workload(L=L, G=G, H=H, d=d, kv=kv, act="bf16", theta=theta, n_blocks=N, index="bf16")
    wl = wl.with_(sink_blocks=1, recent_blocks=2, view_blocks=V, n_queries=3)
    scaled = kv == "e4m3"
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        ctx = kvm.Context(kvm.config_for(wl, max_blocks=N + 1, max_positions=32 * (N + 1), pool_pages=V))
        g = torch.Generator(device="cuda").manual_seed(7)
        rnd = lambda *sh: torch.randn(*sh, generator=g, device="cuda").bfloat16()     # noqa: E731
        qw, kw = 1 + 0.1 * rnd(d), 1 + 0.1 * rnd(d)
        dt = TDT[kv]
        n = 32 * N
        pages = [torch.zeros(N + 1, L, G, 32, d, dtype=dt, device="cuda") for _ in range(3)]   # K, V, raw K
        ks, vs = ((torch.ones(N + 1, L, G, device="cuda") for _ in range(2)) if scaled else (None, None))
        index = torch.zeros(ctx.index_shape(), dtype=torch.bfloat16, device="cuda")
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")             # noqa: E731
        hist = ctx.cache(pages[0], pages[1], ks, vs)
        # prefill in two chunks, the first ending inside a block
        for a, b in ((0, 650), (650, n)):
            chunk = ctx.batch(i32([0, b - a]), i32([b]), torch.arange(N + 1, dtype=torch.int32, device="cuda")[None].contiguous(),
                              n_tokens=b - a, max_q_len=b - a, max_kv_len=b)
            for layer in range(L):
                qkv = rnd(b - a, (H + 2 * G) * d)
                k_free = torch.empty(b - a, G, d, dtype=torch.bfloat16, device="cuda")
                ctx.qk_norm_rope(torch.arange(a, b, dtype=torch.int32, device="cuda"),
                                 k=qkv[:, H * d:(H + G) * d].view(-1, G, d), k_weight=kw, k_free=k_free)
                ctx.append_kv(chunk, hist, layer, k_free, qkv[:, (H + G) * d:].view(-1, G, d),
                              raw_k_pages=pages[2])
        ctx.build_index(pages[0][:N], 0, N, index, k_scale=ks[:N] if scaled else None)
        # the recall's buffers: the view's pages, and one page behind them for the tail
        pool_k, pool_v = (torch.zeros(V + 1, L, G, 32, d, dtype=dt, device="cuda") for _ in range(2))
        table = torch.full((1, V + 1), V, dtype=torch.int32, device="cuda")
        rows = torch.full((1, V + 1), N, dtype=torch.int32, device="cuda")            # sel_ids, then the tail's row
        scores = torch.empty(N + 1, device="cuda")
        ctx.bind(index=index, raw_k=pages[2], v=pages[1], pool_k=pool_k, pool_v=pool_v,
                 page_table=table[0, :V], scores=scores, sel_ids=rows[0, :V])
        view = ctx.cache(pool_k, pool_v, ks, vs)
        T = 3
        kv_len = i32([32 * V + T])
        tail = ctx.batch(i32([0, T]), kv_len, table, n_tokens=T, max_q_len=T, max_kv_len=32 * (V + 1),
                         scale_rows=rows if scaled else None)
        pos = torch.arange(32 * V, 32 * V + T, dtype=torch.int32, device="cuda")
        x = [rnd(T, (H + 2 * G) * d) for _ in range(L)]
        q_free = torch.empty(L, T, H, d, dtype=torch.bfloat16, device="cuda")
        q_rot = torch.empty_like(q_free)
        k_free = torch.empty(L, T, G, d, dtype=torch.bfloat16, device="cuda")
        out = torch.zeros(L, T, H, d, dtype=torch.bfloat16, device="cuda")

        def decode():
            for layer in range(L):
                ctx.qk_norm_rope(pos, q=x[layer][:, :H * d].view(T, H, d),
                                 k=x[layer][:, H * d:(H + G) * d].view(T, G, d), q_weight=qw, k_weight=kw,
                                 q_free=q_free[layer], q_rot=q_rot[layer], k_free=k_free[layer])
            ctx.step(q_free, T, N, stats=False)
            for layer in range(L):
                ctx.append_kv(tail, view, layer, k_free[layer], x[layer][:, (H + G) * d:].view(T, G, d))
                ctx.attend(tail, view, layer, q_rot[layer], out[layer])

        if graph:
            cg = torch.cuda.CUDAGraph()
            s.synchronize()
            with torch.cuda.graph(cg, stream=s):
                decode()
            assert not out.any()
            cg.replay()
        else:
            decode()
        ctx.sync(s)
    s.synchronize()
    sel = rows[0, :V].tolist()
    assert sel == sorted(set(sel)) and sel[0] == 0 and sel[-2:] == [N - 2, N - 1]
    # the view's K is the raw K re-rotated at compact positions, within one rounding
    # of pages and one of raw K (both relative to the pair)
    raw = ref.values(pages[2].cpu()[sel], kv)
    for j in range(V):
        want = ref.rotate(raw[j], torch.arange(32 * j, 32 * j + 32), theta)
        got = ref.values(pool_k[int(table[0, j])].cpu(), kv)
        step = (EPS2[kv] * want.abs()).clamp(min=2.0 ** -10 if scaled else 0)
        assert ((got - want).abs() <= step + 4 * U * ref.pair_mag(raw[j])).all()
    # attention over what the pages hold
    p = Paged.__new__(Paged)
    p.lens, p.L, p.G, p.H, p.d, p.kv, p.act, p.scaled = [(T, 32 * V + T)], L, G, H, d, kv, "bf16", scaled
    p.k, p.v, p.ks, p.vs = (None if t is None else t.cpu() for t in (pool_k, pool_v, ks, vs))
    p.table, p.rows = table.cpu(), rows.cpu() if scaled else None
    p.q_start, p.n, p.max_kv = [0, T], T, 32 * V + T
    for layer in range(L):
        p.layer, p.q = layer, q_rot[layer].cpu()
        check_attend(p, True, d ** -0.5, out[layer], None)
        # the tail's K: the normalised key rotated at its logical index
        y = x[layer][:, H * d:(H + G) * d].view(T, G, d).cpu().double()
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-6) * kw.cpu().double()
        want = ref.rotate(y.transpose(0, 1), torch.arange(32 * V, 32 * V + T), theta)
        got = ref.values(p.k[V, layer, :, :T], kv)
        sc = p.ks[N, layer].double()[:, None, None] if scaled else torch.ones(G, 1, 1)
        # a rounding of the key to bf16, then one to the page's type
        tol = (EPS2["bf16"] + EPS2[kv]) * 1.01 * ref.pair_mag(want) + (2.0 ** -10 * sc if scaled else 0) + 1e-4 * U
        assert ((got * sc - want).abs() <= tol + 80 * U * ref.pair_mag(want)).all()
    ctx.close()


def test_two_contexts_on_two_streams(kvm):
    """Calls of different contexts at the same time keep apart."""
    ps = [Paged([(q, 1500)], G=2, H=12, d=128, kv="bf16", act="bf16", seed=q) for q in (1, 150)]
    ctxs, outs, work = [], [], []
    for p in ps:
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            ctx = kvm.Context(kvm.config_for(ref.workload(G=2, H=12, d=128, kv="bf16", act="bf16")))
            batch, cache = p.on(ctx)
            out = torch.full((p.n, 12, 128), 7.0, device="cuda").bfloat16()
            work.append((ctx, s, batch, cache, p.q.cuda(), out))
    torch.cuda.synchronize()
    for _ in range(20):
        for ctx, s, batch, cache, q, out in work:
            ctx.attend(batch, cache, 0, q, out, stream=s)
    for p, (ctx, s, _, _, _, out) in zip(ps, work):
        ctx.sync(s)
        check_attend(p, True, 128 ** -0.5, out, None)
        ctx.close()
