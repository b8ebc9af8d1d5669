"""kvm_attend, kvm_append_kv and kvm_build_index_scaled at the limits of what their
documentation allows: scales far apart, weights far apart, entries that are not
finite, stored scales that are no scales, buffers in host memory, waits that give
up.  Against the 64-bit definitions of serve_ref; what a test adds to its
tolerances is derived in place."""
import math

import pytest
import torch

import serve_ref as ref
from serve_ref import EPS2, TDT, U, Paged
from test_gpu_serve import context, kvm, run_attend   # noqa: F401

pytestmark = pytest.mark.gpu


def attend(kvm, p, scale, causal=True):
    """One call: (out, lse) in 64 bits on the host."""
    ctx = context(kvm, L=p.L, G=p.G, H=p.H, d=p.d, kv=p.kv, act=p.act)
    batch, cache = p.on(ctx)
    out = torch.full((p.n, p.H, p.d), 7.0, device="cuda").to(TDT[p.act])
    lse = torch.full((p.n, p.H), 7.0, device="cuda")
    ctx.attend(batch, cache, p.layer, p.q.cuda(), out, lse=lse, scale=scale, causal=causal)
    ctx.sync()
    return out.cpu().double(), lse.cpu().double()


def products(p, scale, lse):
    """For every query row: the largest of its weights times v_scale, the sum of the
    |codes| it sees, and what weights below 2^-110 of its largest give, which may
    count for less: [n, H], [n, H, d] twice."""
    top = torch.zeros(p.n, p.H, dtype=torch.float64)
    codes = torch.zeros(p.n, p.H, p.d, dtype=torch.float64)
    faint = torch.zeros_like(codes)
    r = p.H // p.G
    for s, (qn, kvl) in enumerate(p.lens):
        at = slice(p.q_start[s], p.q_start[s] + qn)
        rows = (p.rows if p.rows is not None else p.table)[s, :-(-kvl // 32)].long()
        seen = torch.arange(kvl)[None, :] <= kvl - qn + torch.arange(qn)[:, None]
        for g in range(p.G):
            k, v = p.heads(s, g)
            vs = p.vs[rows, p.layer, g].double().repeat_interleave(32)[:kvl]
            h = slice(g * r, (g + 1) * r)
            x = torch.einsum("nhd,kd->nhk", p.q[at, h].double(), k) * scale - lse[at, h][..., None]
            w = torch.where(seen[:, None], torch.exp(torch.where(seen[:, None], x, 0.0)), 0.0)
            small = torch.where(w < 2.0 ** -110 * w.amax(-1, keepdim=True), w, 0.0)
            faint[at, h] = torch.einsum("nhk,kd->nhd", small, v.abs())
            top[at, h] = (w * vs).amax(-1)
            codes[at, h] = torch.einsum("nk,kd->nd", seen.double(), (v / vs[:, None]).abs())[:, None]
    return top, codes, faint


def check_scaled(p, scale, out, lse, bits):
    """Against the 64-bit attention.  The e4m3 form holds a weight times its v_scale
    as a 16-bit float whose rounding is at most 2^-(bits + 1) of the row's largest such
    product, 2^-bits with that maximum itself up to one float32 rounding off;
    a key adds that times its code to the sum."""
    want, wl, absv, ds = p.reference(scale, True)
    top, codes, faint = products(p, scale, wl)
    lost = 2.0 ** -bits * top[..., None] * codes
    assert bool(torch.isfinite(out).all())
    err = (out - want).abs()
    tol = ref.attend_tolerance(want, absv, ds, p.act, p.kv, p.max_kv) + lost + faint
    assert (err <= tol).all(), f"worst error / tolerance {(err / tol).max():.3g}"
    assert torch.equal(lse == -math.inf, wl == -math.inf)
    tl = ds * 2 + (p.max_kv + 16) * U + 4 * U * wl.abs()
    assert ((lse - wl).abs() <= tl).all()


# One sequence, several, more row tiles than SMs: the forms for a decoded token (with
# eight warps and with four), for one row tile and for pairs of them.
FORMS = {"decode": ([2], 1), "decode, many": ([2] * 90, 2), "tile": ([40], 1), "pairs": ([100] * 30, 2)}


# ---------------------------------------------------------------- scales far apart

def far_apart(form, n_keys, seed):
    lens, G = FORMS[form]
    return Paged([(q, n_keys) for q in lens], G=G, H=6 * G, d=64, kv="e4m3", act="bf16", scaled=True,
                 seed=seed)


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("exponent", [20, 28, 30, 64, 105])
def test_attend_masked_page_of_a_far_larger_scale(kvm, form, exponent):
    """Rows that see only pages whose v_scale is the least there is, beside a page
    that they do not see, whose scale is 2^128 and more times that."""
    p = far_apart(form, 289, 1)                          # the last page: one key, seen by the last token
    for s in range(len(p.lens)):
        pages = p.table[s, :10].long()
        p.vs[pages] = 2.0 ** -100
        p.vs[pages[9]] = 2.0 ** exponent
    scale = p.d ** -0.5
    check_scaled(p, scale, *attend(kvm, p, scale), 24)


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("gap,low,high", [(60, -40, 100), (100, -100, 40), (109, -100, 100), (126.5, -100, 27),
                                          (127, -100, 27), (127.5, -100, 28), (130, -100, 40), (140, -100, 100),
                                          (180, -100, 105)])
@pytest.mark.parametrize("first", [True, False], ids=["early", "late"])
def test_attend_small_weights_of_a_far_larger_scale(kvm, form, gap, low, high, first):
    """Half the pages score `gap` (log2) above the other half and have v_scale
    2^low, the other half 2^high: a weight of 2^-gap, which float32 may not hold, times
    a scale that brings it back into the result."""
    p = far_apart(form, 512, 2)
    scale = gap * math.log(2) / 128                      # q.k = +-64
    p.q[:] = 1.0
    p.ks[:] = 1.0
    one = torch.tensor(1.0).to(torch.float8_e4m3fn).view(torch.uint8)
    for s in range(len(p.lens)):
        pages = p.table[s, :16].long()
        top = pages[:8] if first else pages[8:]
        p.k[pages] = one | 0x80
        p.k[top] = one
        p.vs[pages] = 2.0 ** high
        p.vs[top] = 2.0 ** low
    check_scaled(p, scale, *attend(kvm, p, scale), 24)


@pytest.mark.parametrize("q,kv_len", [(2, 33), (64, 64)], ids=["decode", "tile"])
def test_attend_after_a_block_of_zeros(kvm, q, kv_len):
    """V of the first block all zeros (kvm_append_kv gives it the least scale), of the
    next 1e12: a token of the first block gets zeros."""
    G, H, d = 2, 12, 128
    ctx = context(kvm, L=1, G=G, H=H, d=d, kv="e4m3", act="bf16")
    g = torch.Generator().manual_seed(5)
    k = torch.randn(kv_len, G, d, generator=g).bfloat16()
    v = torch.zeros(kv_len, G, d).bfloat16()
    v[32:] = 1e12
    kp, vp = (torch.zeros(2, 1, G, 32, d, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.ones(2, 1, G, device="cuda") for _ in range(2))
    cache = ctx.cache(kp, vp, ks, vs)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")     # noqa: E731
    table = i32([[1, 0]])
    ctx.append_kv(ctx.batch(i32([0, kv_len]), i32([kv_len]), table, n_tokens=kv_len, max_q_len=kv_len,
                            max_kv_len=64), cache, 0, k.cuda(), v.cuda())
    batch = ctx.batch(i32([0, q]), i32([kv_len]), table, n_tokens=q, max_q_len=q, max_kv_len=64)
    out = torch.full((q, H, d), 7.0, device="cuda").bfloat16()
    ctx.attend(batch, cache, 0, torch.randn(q, H, d, generator=g).bfloat16().cuda(), out)
    ctx.sync()
    assert float(vs[1, 0, 0]) == 2.0 ** -100
    first = 32 - (kv_len - q)                            # tokens of the first block
    assert (out[:first] == 0).all()
    assert torch.isfinite(out).all() and (out[first:] > 0).all()


# ---------------------------------------------------------------- weights far apart

@pytest.mark.parametrize("q", [1, 20, 40])
@pytest.mark.parametrize("below", [22.3, 25.4, 26.5])
def test_attend_flat_tail_far_below_the_largest_weight(kvm, q, below):
    """One key takes all but 2^-below n of the weight and has V = 0: what is left is
    the sum of many products far below the row's largest."""
    kv_len = 6000
    p = Paged([(q, kv_len)], G=1, H=6, d=64, kv="e4m3", act="bf16", scaled=True, seed=3)
    scale = below * math.log(2) / 128                    # q.k = +-64
    one = torch.tensor(1.0).to(torch.float8_e4m3fn).view(torch.uint8)
    p.q[:] = 1.0
    p.ks[:] = 1.0
    p.vs[:] = 0.25
    p.k[:] = one | 0x80
    p.v[p.v == 0x7F] = 0x30
    p.v &= 0x7F                                          # all of one sign: nothing cancels
    page = int(p.table[0, 40])
    p.k[page, 0, 0, 7] = one
    p.v[page, 0, 0, 7] = 0
    check_scaled(p, scale, *attend(kvm, p, scale), 31)


@pytest.mark.parametrize("q", [2, 40])
@pytest.mark.parametrize("size", [-16, -20, -27])
def test_attend_query_rows_of_one_large_entry(kvm, q, size):
    """Query entries 2^size of their row's largest, which meets zeros in K: the
    scores are made of the small ones alone."""
    p = Paged([(q, 200), (q, 77)], G=1, H=6, d=64, kv="e4m3", act="bf16", scaled=True, seed=4)
    p.q = (p.q.double() * 2.0 ** size).bfloat16()
    p.q[:, :, 5] = 1.5
    p.k[..., 5] = 0
    p.ks[:] = 2.0 ** (-6 - size)
    check_scaled(p, 64 ** -0.5, *attend(kvm, p, 64 ** -0.5), 24)


@pytest.mark.parametrize("q", [2, 40])
@pytest.mark.parametrize("size", [-100, -112, -120, -130, 60, 100, 119, 125])
def test_attend_query_rows_of_any_size(kvm, q, size):
    """Rows as small as bf16 has them, subnormal entries among them, and as large,
    against K whose scale makes up for it where the range of scales allows."""
    p = Paged([(q, 200), (q, 77)], G=1, H=6, d=64, kv="e4m3", act="bf16", scaled=True, seed=5)
    p.q = (p.q.double() * 2.0 ** size).bfloat16()
    p.ks[:] = 2.0 ** max(-100, min(119, -6 - size))
    scale = 64 ** -0.5 * 2.0 ** (-6 - size - max(-100, min(119, -6 - size)))
    check_scaled(p, scale, *attend(kvm, p, scale), 24)


# ---------------------------------------------------------------- the index of scaled pages

def test_index_of_scaled_pages_in_host_memory(kvm):
    """Buffers where kvm_build_index takes them: pinned host memory too (an index with
    index_location KVM_HOST_PINNED lives there)."""
    wl = ref.workload(L=2, G=3, H=3, d=64, kv="e4m3", act="bf16", index="bf16", n_blocks=64, theta=1e6)
    ctx = kvm.Context(kvm.config_for(wl))
    g = torch.Generator().manual_seed(6)
    n, first = 7, 9
    codes = (torch.randn(n, 2, 3, 32, 64, generator=g) * 60).to(torch.float8_e4m3fn).view(torch.uint8)
    ks = torch.exp2(torch.randint(-9, 4, (n, 2, 3), generator=g).float())
    index, raw = torch.zeros(ctx.index_shape(), dtype=torch.bfloat16), torch.zeros_like(codes)
    got = [t.cuda() for t in (index, raw)]
    ctx.build_index(codes.cuda(), first, n, got[0], got[1], k_scale=ks.cuda())
    host = [t.pin_memory() for t in (codes, index, raw, ks)]
    ctx.build_index(host[0], first, n, host[1], host[2], k_scale=host[3])
    ctx.sync()
    assert host[1].any() and torch.equal(host[1], got[0].cpu()) and torch.equal(host[2], got[1].cpu())
    plain = [t.pin_memory() for t in (index, raw)]
    ctx.build_index(host[0], first, n, plain[0], plain[1])          # the call it follows
    ctx.sync()
    assert torch.equal(plain[1], host[2])
    for bad in ((codes, host[1]), (host[0], index)):                # pageable memory
        with pytest.raises(kvm.KvmError) as e:
            ctx.build_index(bad[0], first, n, bad[1], k_scale=host[3])
        assert e.value.name == "KVM_ERR_INVALID_ARG"
    ctx.close()


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("side", ["k", "v"])
@pytest.mark.parametrize("bad", [0.0, math.nan, 0.3, -0.5, math.inf, 2.0 ** -110, 2.0 ** 120])
def test_append_behind_a_stored_scale_that_is_none(kvm, side, bad):
    """A block whose stored scale is no allowed power of two: the flag is raised, its
    codes and scales stay (of K, V and raw K), the other heads and blocks are
    appended to."""
    G, d = 3, 64
    ctx = context(kvm, L=1, G=G, H=6, d=d, kv="e4m3", act="bf16")
    p = Paged([(40, 50), (2, 70)], G=G, H=6, d=d, kv="e4m3", act="bf16", scaled=True, seed=7, own_rows=True)
    x = torch.randn(42, G, d, generator=torch.Generator().manual_seed(8)).bfloat16().cuda() * 1000
    after = []
    for spoil in (False, True):
        batch, cache = p.on(ctx)                          # fresh copies
        raw = torch.full_like(p.dk, 0x21)
        if spoil:
            row = int(p.rows[0, 0])
            (p.dks if side == "k" else p.dvs)[row, 0, 1] = bad
        before = [t.clone() for t in (p.dk, p.dv, raw, p.dks, p.dvs)]
        ctx.append_kv(batch, cache, 0, x, x, raw_k_pages=raw)
        if spoil:
            with pytest.raises(kvm.KvmError) as e:
                ctx.sync()
            assert e.value.name == "KVM_ERR_DEVICE"
        ctx.sync()
        after.append([t.clone() for t in (p.dk, p.dv, raw, p.dks, p.dvs)])
    page = int(p.table[0, 0])
    for i, (good, got, was) in enumerate(zip(*after, before)):
        at = (page, 0, 1) if i < 3 else (row, 0, 1)
        bits = (lambda t: t) if i < 3 else (lambda t: t.view(torch.int32))     # noqa: E731
        assert torch.equal(bits(got)[at], bits(was)[at]), "the block and head of the bad scale"
        good[at] = got[at]
        assert torch.equal(bits(got), bits(good)), "everything else"


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_append_entries_that_are_not_finite(kvm, act, d):
    """Scaled pages: an infinity counts as 448 times the scale, which the finite entries
    set, before K is rotated; a NaN stays one, and in K's rotated row its partner."""
    G, n = 2, 40
    ctx = context(kvm, L=1, G=G, H=4, d=d, kv="e4m3", act=act)
    g = torch.Generator().manual_seed(9)
    k, v = ((torch.randn(n, G, d, generator=g) * 3).to(TDT[act]) for _ in range(2))
    h = d // 2
    inf, nan = math.inf, math.nan
    k[0, 0, 3], k[0, 0, 5 + h] = inf, -inf               # position 0: the sine is 0
    k[1, 0, 3], k[1, 0, 3 + h] = inf, inf                # both of a pair
    k[7, 1, 9], k[7, 1, 9 + h] = -inf, inf
    k[33, 0, 1], k[34, 1, 2] = nan, inf
    k[35, 0, 4], k[35, 0, 4 + h] = nan, inf
    k[36] = inf                                          # a whole row
    v[0, 0, 3], v[2, 1, 5], v[33, 0, 1] = inf, -inf, nan
    kp, vp, raw = (torch.zeros(2, 1, G, 32, d, dtype=torch.uint8, device="cuda") for _ in range(3))
    ks, vs = (torch.ones(2, 1, G, device="cuda") for _ in range(2))
    cache = ctx.cache(kp, vp, ks, vs)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")     # noqa: E731
    batch = ctx.batch(i32([0, n]), i32([n]), i32([[1, 0]]), n_tokens=n, max_q_len=n, max_kv_len=64)
    ctx.append_kv(batch, cache, 0, k.cuda(), v.cuda(), raw_k_pages=raw)
    ctx.sync()
    for b, page in ((0, 1), (1, 0)):
        rows = slice(32 * b, min(n, 32 * b + 32))
        for gg in range(G):
            for x, sc, pages, most, rot in ((k, ks, kp, 316.75, True), (k, ks, raw, 316.75, False),
                                            (v, vs, vp, 448.0, False)):
                x = x[rows, gg].double()
                s = ref.scale_for(float(x[torch.isfinite(x)].abs().max()), most)
                assert float(sc[page, 0, gg]) == s
                x = torch.where(x.isinf(), torch.sign(x) * 448 * s, x) / s
                mag = ref.pair_mag(x)
                want = ref.rotate(x, torch.arange(n)[rows], 1e4) if rot else x
                got = ref.decode(pages[page, 0, gg])[:want.shape[0]]
                assert torch.equal(got.isnan(), want.isnan())
                at = ~want.isnan()
                sat = want.clamp(-448, 448)
                # half an e4m3 step; the rotation's two products, sum, cos and sin, each rounded once
                tol = (2.0 ** -4 * sat.abs()).clamp(min=2.0 ** -10) + (8 * U * mag if rot else 0)
                assert ((got - sat).abs() <= tol)[at].all()


# ---------------------------------------------------------------- waits that give up

@pytest.mark.parametrize("kv,scaled", [("bf16", False), ("e4m3", True)])
@pytest.mark.parametrize("G,lens", [(1, [(40, 9000)]), (2, [(300, 4000), (9, 700)]), (4, [(600, 3000)])],
                         ids=["single row tiles", "cut and ragged", "pairs"])
def test_attend_bounded_waits_and_recovery(kvm, kv, scaled, G, lens):
    """One CTA's producer stops after its first key tile: waits run out, the parts of
    shared tiles stay uncounted, kvm_sync reports KVM_ERR_TIMEOUT, and the next
    calls of every form on the same context are right."""
    import time
    ctx = kvm.Context(kvm.config_for(ref.workload(G=G, H=6 * G, d=64, kv=kv, act="bf16")))
    p = Paged(lens, G=G, H=6 * G, d=64, kv=kv, act="bf16", scaled=scaled, seed=10)
    batch, cache = p.on(ctx)
    out = torch.zeros(p.n, p.H, 64, device="cuda", dtype=torch.bfloat16)
    q = p.q.cuda()
    ctx.attend(batch, cache, 0, q, out)
    ctx.sync()
    want = out.clone()
    ctx.debug_inject(4, 2)
    ctx.attend(batch, cache, 0, q, out)                  # the first is as ever
    ctx.sync()
    assert torch.equal(out, want)
    t0 = time.monotonic()
    ctx.attend(batch, cache, 0, q, out)
    with pytest.raises(kvm.KvmError) as e:
        ctx.sync()
    assert e.value.name == "KVM_ERR_TIMEOUT"
    assert time.monotonic() - t0 < 30.0
    for again in (p, Paged([(1, 3000), (1, 1000)], G=G, H=6 * G, d=64, kv=kv, act="bf16", scaled=scaled, seed=11), p):
        run_attend(kvm, again, True, ctx=ctx)
    ctx.attend(batch, cache, 0, q, out)
    ctx.sync()
    assert torch.equal(out, want)
    ctx.close()


def test_attend_recovers_on_a_stream_of_its_own(kvm):
    """The counters are cleared when kvm_sync returns, for a stream that does not wait for
    the default one."""
    p = Paged([(600, 3000)], G=4, H=24, d=64, kv="bf16", act="bf16", seed=13)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        ctx = kvm.Context(kvm.config_for(ref.workload(G=4, H=24, d=64, kv="bf16", act="bf16")))
        batch, cache = p.on(ctx)
        q, out = p.q.cuda(), torch.zeros(p.n, 24, 64, device="cuda", dtype=torch.bfloat16)
        ctx.attend(batch, cache, 0, q, out)
        ctx.sync(s)
        want = out.clone()
        ctx.debug_inject(4, 1)
        ctx.attend(batch, cache, 0, q, out)
        with pytest.raises(kvm.KvmError) as e:
            ctx.sync(s)
        assert e.value.name == "KVM_ERR_TIMEOUT"
        for _ in range(5):
            ctx.attend(batch, cache, 0, q, out)
        ctx.sync(s)
        assert torch.equal(out, want)
        ctx.close()


# ---------------------------------------------------------------- the binding

def test_calls_of_no_tokens(kvm):
    """Empty tensors (whose address is none) do nothing."""
    ctx = context(kvm, L=1, G=2, H=4, d=64, kv="bf16", act="bf16")
    z = lambda h: torch.empty(0, h, 64, device="cuda", dtype=torch.bfloat16)     # noqa: E731
    n0 = kvm.launch_count()
    ctx.qk_norm_rope(torch.empty(0, dtype=torch.int32, device="cuda"), q=z(4), k=z(2), q_rot=z(4), q_free=z(4),
                     k_free=z(2), q_weight=torch.ones(64, device="cuda").bfloat16())
    assert kvm.launch_count() == n0


def test_one_token_of_any_row_stride(kvm):
    """The stride of a dimension of one element means nothing."""
    ctx = context(kvm, L=1, G=1, H=4, d=64, kv="bf16", act="bf16")
    p = Paged([(1, 40)], G=1, H=4, d=64, kv="bf16", act="bf16", seed=12)
    batch, cache = p.on(ctx)
    pos = torch.tensor([39], dtype=torch.int32, device="cuda")
    base = torch.randn(4, 64, device="cuda").bfloat16()
    got = []
    for stride in (256, 259):
        q = torch.as_strided(base, (1, 4, 64), (stride, 64, 1))
        k = torch.as_strided(base, (1, 1, 64), (stride - 192, stride - 192, 1))
        out, rot = (torch.zeros(1, 4, 64, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        ctx.append_kv(batch, cache, 0, k, k)
        ctx.qk_norm_rope(pos, q=q, q_rot=rot)
        ctx.attend(batch, cache, 0, q, out)
        ctx.sync()
        got.append((p.dk.clone(), rot, out))
    for a, b in zip(*got):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


# ---------------------------------------------------------------- weights of decoded tokens

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q,kv_len", [(1, 3), (1, 40), (2, 5), (2, 300), (1, 3000)])
def test_attend_decode_keeps_its_weights(kvm, q, kv_len, d):
    """bf16 pages, up to 16 query rows: weights are held as the sum of two bf16, so
    that what is left of values that cancel is not their rounding."""
    p = Paged([(q, kv_len), (q, kv_len)], G=2, H=12, d=d, kv="bf16", act="bf16", seed=14, qstd=0.3)
    p.v = (p.v.double().sign() * (100 + p.v.double().abs())).bfloat16()
    out, _ = attend(kvm, p, d ** -0.5)
    want, _, absv, ds = p.reference(d ** -0.5, True)
    # the output's rounding; of the weights, the second bf16's rounding (2^-8 of 2^-8),
    # and what float32 leaves, as in ref.attend_tolerance
    w = 2 * ds[..., None] + (2 * kv_len + 16) * U + 2.0 ** -16
    err = (out - want).abs()
    tol = EPS2["bf16"] * want.abs() + w * (1 + EPS2["bf16"]) * absv
    assert (err <= tol).all(), f"worst error / tolerance {(err / tol).max():.3g}"
