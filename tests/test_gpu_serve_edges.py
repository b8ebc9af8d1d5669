"""kvm_attend and kvm_append_kv where they can go wrong: long runs whose parts
are joined, many tiles alike, extreme scales, shared pages, offsets past 32
bits, graphs that share a context.  Against the 64-bit definitions of
serve_ref, with its tolerances; what a test adds to them is derived in place."""
import math

import pytest
import torch

import serve_ref as ref
from serve_ref import EPS2, TDT, Paged
from test_gpu_serve import check_attend, context, kvm, run_attend   # noqa: F401

pytestmark = pytest.mark.gpu

TYPES = [("bf16", "bf16", False), ("bf16", "e4m3", True), ("f32", "f32", False)]
IDS = ["bf16", "e4m3-scaled", "f32"]


# One kv head, so that every CTA of the grid has a part of the same tile: decoded
# tokens (8 and 16 row tiles), one 128-row tile, two row tiles, five; with the
# last key tile whole, one key long, and cut inside a page.
@pytest.mark.parametrize("act,kv,scaled", TYPES, ids=IDS)
@pytest.mark.parametrize("q,kv_len", [(1, 33000), (2, 20017), (20, 16385), (40, 9984), (100, 7000)])
def test_attend_long_runs_are_joined(kvm, act, kv, scaled, q, kv_len):
    p = Paged([(q, kv_len)], G=1, H=6, d=128, kv=kv, act=act, scaled=scaled, seed=q, own_rows=scaled)
    run_attend(kvm, p, True)


@pytest.mark.parametrize("act,kv,scaled", TYPES, ids=IDS)
@pytest.mark.parametrize("q,kv_len", [(1, 20000), (33, 8000), (150, 4100)])
def test_attend_long_runs_of_several_heads(kvm, act, kv, scaled, q, kv_len):
    """Several heads and sequences on the line, not a power of two of anything."""
    p = Paged([(q, kv_len), (max(1, q // 3), kv_len // 7), (q, q)], G=3, H=6, d=64, kv=kv, act=act,
              scaled=scaled, seed=q + 1)
    run_attend(kvm, p, True, packed=True)


# More tiles than SMs, equally long (counted alike, up to 24 units and more) and
# not, for the forms that a decoded token, a few rows and a tile take.
@pytest.mark.parametrize("act,kv,scaled", TYPES, ids=IDS)
@pytest.mark.parametrize("d,H,q", [(64, 4, 1), (128, 4, 1), (64, 4, 5), (128, 4, 5), (64, 2, 40)])
@pytest.mark.parametrize("alike", [True, False], ids=["alike", "ragged"])
def test_attend_many_tiles(kvm, act, kv, scaled, d, H, q, alike):
    n = 80 if q < 40 else 160
    lens = [(q, 800) if alike else (1 + i % q, 1 + (i * 97) % 800 + q) for i in range(n)]
    p = Paged(lens, G=2 if q < 40 else 1, H=H, d=d, kv=kv, act=act, scaled=scaled, seed=d + q)
    run_attend(kvm, p, True)


# Row tiles taken in pairs: more of them than SMs, alike and ragged, the last one of
# a pair empty or short; and few with so many keys that they are cut and joined.
@pytest.mark.parametrize("act,kv,scaled", TYPES[:2], ids=IDS[:2])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,G,H", [
    ([(100, 600)] * 30, 2, 6),
    ([(1 + (i * 37) % 170, 1 + (i * 211) % 900 + (i * 37) % 170) for i in range(40)], 2, 6),
    ([(44, 44 + 13 * i) for i in range(60)], 1, 6),
    ([(700, 5001)], 3, 18),
    ([(300, 9990), (129, 700), (1, 0)], 4, 8),
], ids=["alike", "ragged", "short second tile", "cut", "cut and ragged"])
def test_attend_pairs_of_row_tiles(kvm, act, kv, scaled, d, lens, G, H):
    p = Paged(lens, G=G, H=H, d=d, kv=kv, act=act, scaled=scaled, seed=d, own_rows=scaled)
    run_attend(kvm, p, True)


@pytest.mark.parametrize("act,kv,scaled", TYPES[:2], ids=IDS[:2])
def test_attend_many_long_tiles_alike(kvm, act, kv, scaled):
    """More row tiles than CTAs, each of 27 key tiles: runs of parts of a tile."""
    p = Paged([(9, 3400)] * 40, G=4, H=8, d=64, kv=kv, act=act, scaled=scaled, seed=3)
    run_attend(kvm, p, True, lse=False)


def test_attend_1024_sequences(kvm):
    """The most a call takes; one more is refused."""
    for q in (1, 12):
        lens = [(1 + i % q, 1 + i % 70 + q) for i in range(1024)]
        p = Paged(lens, G=1, H=2, d=64, kv="bf16", act="bf16", seed=4)
        run_attend(kvm, p, True)
    p = Paged([(1, 1)] * 1025, G=1, H=2, d=64, kv="bf16", act="bf16")
    ctx = context(kvm, L=1, G=1, H=2, d=64, kv="bf16", act="bf16")
    batch, cache = p.on(ctx)
    out = torch.zeros(p.n, 2, 64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(kvm.KvmError) as e:
        ctx.attend(batch, cache, 0, p.q.cuda(), out)
    assert e.value.name == "KVM_ERR_CAPACITY"


# Scales over most of their range.  In the e4m3 form of the tensor cores a
# weight times its v_scale is a 16-bit float against the row's largest product:
# half a step is at least 2^-25 of it, 2^-24 with the row's maximum up to one
# float32 rounding off.  A key adds that times its code to a sum.
@pytest.mark.parametrize("q", [1, 2, 40, 90])
@pytest.mark.parametrize("span", [6, 40, 90])
def test_attend_extreme_scales(kvm, q, span):
    p = Paged([(q, 500), (q, 130)], G=1, H=6, d=64, kv="e4m3", act="bf16", scaled=True, seed=span)
    g = torch.Generator().manual_seed(span)
    p.ks = torch.exp2(torch.randint(-100, 1, p.ks.shape, generator=g).float()) if span > 6 else p.ks
    p.vs = torch.exp2(torch.randint(-span, span + 1, p.vs.shape, generator=g).float())
    ctx = context(kvm, L=1, G=1, H=6, d=64, kv="e4m3", act="bf16")
    batch, cache = p.on(ctx)
    out = torch.zeros(p.n, 6, 64, device="cuda", dtype=torch.bfloat16)
    ctx.attend(batch, cache, 0, p.q.cuda(), out)
    ctx.sync()
    want, lse, absv, ds = p.reference(64 ** -0.5, True)
    lost = torch.zeros_like(want)
    for s, (qn, kvl) in enumerate(p.lens):
        k, v = p.heads(s, 0)
        at = slice(p.q_start[s], p.q_start[s] + qn)
        vs = p.vs[p.table[s, :-(-kvl // 32)].long(), 0, 0].double().repeat_interleave(32)[:kvl]
        x = torch.einsum("nhd,kd->nhk", p.q[at].double(), k) * 64 ** -0.5
        seen = torch.arange(kvl)[None, :] <= kvl - qn + torch.arange(qn)[:, None]
        w = torch.where(seen[:, None], torch.exp(x - lse[at][..., None]), 0.0) * vs
        codes = (v / vs[:, None]).abs()
        lost[at] = 2.0 ** -24 * w.amax(-1)[..., None] * torch.einsum("nk,kd->nd", seen.double(), codes)[:, None]
    err = (out.cpu().double() - want).abs()
    tol = ref.attend_tolerance(want, absv, ds, "bf16", "e4m3", 500) + lost
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("act,kv,scaled", TYPES, ids=IDS)
@pytest.mark.parametrize("q", [1, 3, 50, 200])
def test_attend_rows_of_zeros_and_of_many_sizes(kvm, act, kv, scaled, q):
    """Query rows of zeros, of the smallest normal sizes and of large ones."""
    p = Paged([(q, 300), (q, 77)], G=2, H=6, d=64, kv=kv, act=act, scaled=scaled, seed=6)
    size = torch.tensor([0.0, 2.0 ** -120, 2.0 ** -20, 1.0, 4.0])
    p.q = (p.q.double() * size[torch.arange(p.n * p.H) % 5].view(p.n, p.H, 1)).to(TDT[act])
    run_attend(kvm, p, True)


@pytest.mark.parametrize("q", [1, 2, 40, 90])
def test_attend_negative_and_zero_softmax_scales(kvm, q):
    for act, kv, scaled in TYPES:
        p = Paged([(q, 420)], G=2, H=6, d=128, kv=kv, act=act, scaled=scaled, seed=7)
        for scale in (-0.05, 0.0, -0.0, 1e-30):
            run_attend(kvm, p, True, scale=scale)


@pytest.mark.parametrize("act,kv,scaled", TYPES, ids=IDS)
@pytest.mark.parametrize("q", [1, 30])
def test_attend_shared_pages(kvm, act, kv, scaled, q):
    """Two sequences with the same first pages, and one page twice in a sequence."""
    p = Paged([(q, 400), (q, 333)], G=2, H=4, d=64, kv=kv, act=act, scaled=scaled, seed=8)
    p.table[1, :5] = p.table[0, :5]
    p.table[0, 7] = p.table[0, 2]
    p.table[0, 8] = p.table[0, 2]
    run_attend(kvm, p, True)


def test_attend_nan_codes_stay_in_their_rows(kvm):
    """A NaN below kv_len makes the rows that see it NaN, of its kv head and its
    sequence only; behind kv_len it is not seen (Paged fills those rows with it)."""
    for act, kv in (("bf16", "bf16"), ("bf16", "e4m3"), ("f32", "f32")):
        for q in (1, 30):
            p = Paged([(q, 200), (q, 100)], G=2, H=4, d=64, kv=kv, act=act, seed=9)
            bad = 0x7F if kv == "e4m3" else math.nan
            p.k[int(p.table[0, 1]), 0, 1, 3, 5] = bad
            ctx = context(kvm, L=1, G=2, H=4, d=64, kv=kv, act=act)
            batch, cache = p.on(ctx)
            out = torch.zeros(p.n, 4, 64, device="cuda", dtype=TDT[act])
            ctx.attend(batch, cache, 0, p.q.cuda(), out)
            ctx.sync()
            got = out.cpu().double()
            assert torch.isnan(got[:q, 2:]).all()
            assert torch.isfinite(got[:q, :2]).all() and torch.isfinite(got[q:]).all()


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("act,kv,scaled", TYPES, ids=IDS)
def test_two_graphs_and_eager_calls_share_a_context(kvm, act, kv, scaled):
    """Two captured calls whose parts use the same workspace, replayed in turn
    with eager calls between them: the results of each alone, bit by bit."""
    ctx = context(kvm, L=1, G=2, H=12, d=128, kv=kv, act=act)
    jobs = []
    for q, kv_len in ((1, 9000), (32, 7000), (2, 4000)):
        p = Paged([(q, kv_len)], G=2, H=12, d=128, kv=kv, act=act, scaled=scaled, seed=q)
        batch, cache = p.on(ctx)
        qd, out = p.q.cuda(), torch.zeros(p.n, 12, 128, device="cuda", dtype=TDT[act])
        ctx.attend(batch, cache, 0, qd, out)
        ctx.sync()
        jobs.append((p, batch, cache, qd, out, out.clone()))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs = []
    for p, batch, cache, qd, out, _ in jobs[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            ctx.attend(batch, cache, 0, qd, out)
        graphs.append(g)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(20):
            for job in jobs:
                job[4].zero_()
            graphs[0].replay()
            graphs[1].replay()
            _, batch, cache, qd, out, _ = jobs[2]
            ctx.attend(batch, cache, 0, qd, out)
            graphs[0].replay()
            s.synchronize()
            for job in jobs:
                assert torch.equal(job[4], job[5])
    ctx.sync(s)


# Pages far up in a cache of more than 2^31 elements (every offset a product of
# page, layer, head and row); only the pages in use are ever written.
@pytest.mark.parametrize("act,kv,scaled", TYPES, ids=IDS)
def test_offsets_past_32_bits(kvm, act, kv, scaled):
    L, G, H, d = 32, 8, 16, 128
    n_pages = 2 ** 31 // (L * G * 32 * d) + 300
    ctx = context(kvm, L=L, G=G, H=H, d=d, kv=kv, act=act)
    k, v = (torch.empty(n_pages, L, G, 32, d, device="cuda", dtype=TDT[kv]) for _ in range(2))
    ks = vs = None
    rows = n_pages
    if scaled:
        ks, vs = (torch.ones(rows, L, G, device="cuda") for _ in range(2))
    cache = ctx.cache(k, v, ks, vs)
    layer = L - 1
    for q, kv_len in ((1, 200), (40, 200), (100, 300)):
        nb = -(-kv_len // 32)
        pages = torch.randperm(250, generator=torch.Generator().manual_seed(q))[:nb] + n_pages - 260
        small = Paged([(q, kv_len)], L=1, G=G, H=H, d=d, kv=kv, act=act, scaled=scaled, seed=q)
        mine = small.table[0, :nb].long()
        for big, own in ((k, small.k), (v, small.v)):
            big[pages.cuda(), layer] = own[mine, 0].cuda()
        if scaled:
            ks[pages.cuda(), layer], vs[pages.cuda(), layer] = small.ks[mine, 0].cuda(), small.vs[mine, 0].cuda()
        batch = ctx.batch(torch.tensor([0, q], dtype=torch.int32, device="cuda"),
                          torch.tensor([kv_len], dtype=torch.int32, device="cuda"),
                          pages.int()[None].cuda(), n_tokens=q, max_q_len=q, max_kv_len=kv_len)
        out = torch.zeros(q, H, d, device="cuda", dtype=TDT[act])
        ctx.attend(batch, cache, layer, small.q.cuda(), out)
        ctx.sync()
        check_attend(small, True, d ** -0.5, out, None)
    # V rows are appended as they are: the same values have to come back
    n = 70
    g = torch.Generator().manual_seed(1)
    x = torch.randint(-15, 16, (n, G, d), generator=g).float()
    x[:, :, 0] = 15.0                                    # a scale that keeps integers below 16 exact
    kd, vd = x.to(TDT[act]).cuda(), x.to(TDT[act]).cuda()
    pages = torch.tensor([[n_pages - 1, n_pages - 7, n_pages - 3]], dtype=torch.int32, device="cuda")
    batch = ctx.batch(torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                      torch.tensor([n], dtype=torch.int32, device="cuda"), pages, n_tokens=n,
                      max_q_len=n, max_kv_len=n)
    ctx.append_kv(batch, cache, layer, kd, vd)
    ctx.sync()
    got = v[pages[0].long(), layer].cpu()                # [3][G][32][d]
    got = ref.values(got, kv)
    if scaled:
        got = got * vs[pages[0].long(), layer].cpu().double()[:, :, None, None]
    got = got.transpose(1, 2).reshape(-1, G, d)[:n]
    assert torch.equal(got, x.double())


# ---------------------------------------------------------------- refusals

def test_attend_refuses_batches_beyond_its_counts(kvm):
    """Bounds whose work does not fit 32-bit counts are refused before a launch.
    2^30 - 300 tokens of two rows are 2^31 - 600 rows: over 32 keys, 128-row tiles
    make 2 * 2^24 tiles of at most 14 units, which 32 bits count; the float32 form is
    held to tiles of 4 rows, 2 * 2^29 of them, which they do not."""
    for act, kv in (("bf16", "bf16"), ("f32", "f32")):
        ctx = context(kvm, L=1, G=2, H=4, d=64, kv=kv, act=act)
        p = Paged([(1, 32)], G=2, H=4, d=64, kv=kv, act=act)
        batch, cache = p.on(ctx)
        out = torch.zeros(1, 4, 64, device="cuda", dtype=TDT[act])
        table = torch.zeros(1, 2 ** 25, dtype=torch.int32, device="cuda")
        q_start, kv_len, _, _ = batch.tensors
        for max_q, max_kv in ((2 ** 20, 2 ** 30), (2 ** 30 - 300, 32), (2 ** 31 - 1, 32)):
            big = ctx.batch(q_start, kv_len, table, n_tokens=1, max_q_len=max_q, max_kv_len=max_kv)
            if act == "bf16" and max_q == 2 ** 30 - 300:
                ctx.attend(big, cache, 0, p.q.cuda(), out)
                ctx.sync()
                check_attend(p, True, 64 ** -0.5, out, None)
                continue
            with pytest.raises(kvm.KvmError) as e:
                ctx.attend(big, cache, 0, p.q.cuda(), out)
            assert e.value.name == "KVM_ERR_CAPACITY", (max_q, max_kv)
        ctx.attend(batch, cache, 0, p.q.cuda(), out)
        ctx.sync()
        check_attend(p, True, 64 ** -0.5, out, None)


def test_append_refuses_batches_beyond_its_grid(kvm):
    ctx = context(kvm, L=1, G=2, H=4, d=64, kv="bf16", act="bf16")
    p = Paged([(1, 32)] * 1024, G=2, H=4, d=64, kv="bf16", act="bf16")
    batch, cache = p.on(ctx)
    q_start, kv_len, table, _ = batch.tensors
    x = torch.zeros(p.n, 2, 64, device="cuda", dtype=torch.bfloat16)
    big = ctx.batch(q_start, kv_len, table, n_tokens=p.n, max_q_len=2 ** 30 - 300, max_kv_len=32)
    with pytest.raises(kvm.KvmError) as e:
        ctx.append_kv(big, cache, 0, x, x)
    assert e.value.name == "KVM_ERR_CAPACITY"


def test_attend_refuses_scales_that_overflow(kvm):
    ctx = context(kvm, L=1, G=2, H=4, d=64, kv="bf16", act="bf16")
    p = Paged([(1, 32)], G=2, H=4, d=64, kv="bf16", act="bf16")
    batch, cache = p.on(ctx)
    out = torch.zeros(1, 4, 64, device="cuda", dtype=torch.bfloat16)
    for scale in (2e30, -3e38, math.inf, math.nan):
        with pytest.raises(kvm.KvmError) as e:
            ctx.attend(batch, cache, 0, p.q.cuda(), out, scale=scale)
        assert e.value.name == "KVM_ERR_INVALID_ARG"


def test_a_call_with_nothing_to_do(kvm):
    """No sequences, no tokens, or sequences without tokens: nothing is written."""
    ctx = context(kvm, L=1, G=2, H=4, d=64, kv="bf16", act="bf16")
    p = Paged([(1, 40), (2, 50)], G=2, H=4, d=64, kv="bf16", act="bf16")
    batch, cache = p.on(ctx)
    q_start, kv_len, table, _ = batch.tensors
    k0, v0 = p.dk.clone(), p.dv.clone()
    x = torch.randn(3, 2, 64, device="cuda").bfloat16()
    out = torch.full((3, 4, 64), 7.0, device="cuda").bfloat16()
    zero = torch.zeros_like(q_start)
    for b in (ctx.batch(zero[:1], kv_len[:0], table[:0], n_tokens=3, max_q_len=1, max_kv_len=50),
              ctx.batch(zero, kv_len, table, n_tokens=3, max_q_len=2, max_kv_len=50),
              ctx.batch(zero, kv_len, table, n_tokens=0, max_q_len=2, max_kv_len=50)):
        ctx.attend(b, cache, 0, p.q.cuda(), out)
        ctx.append_kv(b, cache, 0, x, x)
        ctx.sync()
    same = lambda a, b: torch.equal(a.view(torch.int16), b.view(torch.int16))     # noqa: E731
    assert (out == 7).all() and same(p.dk, k0) and same(p.dv, v0)
