"""GPU parity of appending rotated rows to a paged cache, against the float64 oracle and
bd_cache_write of the turned rows."""
import numpy as np
import pytest
import torch

from oracle import paged as op
from oracle import rope as orope

pytestmark = pytest.mark.gpu

bd = pytest.importorskip("block_causal_varlen_gb300")
pm = pytest.importorskip("paged_more_util")

FORMATS = ["bf16", "e4m3", "e2m1"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bd.load()


def freqs(r, base=10000.0):
    return (1.0 / base ** (torch.arange(0, r, 2, dtype=torch.float64) / r)).float()


def positions(new, kv):
    return [n - q + i for q, n in zip(new, kv) for i in range(q)]


def check_turned(got, x, pos, f, interleaved=False, scale=1.0):
    """Half a step of bf16 (2^-8 relative) and 2^-21 of the pair's length: the angle's float 2^-25
    of a half turn (times pi), sine and cosine 2^-24 each, the factor, two products and a sum 2^-24
    each of at most the pair's 1-norm."""
    want = orope.turn(x, pos, f, interleaved, scale)
    tol = want.abs() * 2.0 ** -8 + orope.lengths(x, f, interleaved) * scale * 2.0 ** -21 + 1e-38
    bad = (got.double() - want).abs() > tol
    assert not bad.any(), (bad.sum().item(), bad.nonzero()[:4].tolist())
    stays = torch.ones(x.shape[-1], dtype=torch.bool)
    stays[:2 * len(f)] = False
    assert torch.equal(got[..., stays], x[..., stays])


def pools(c):
    return [t for t in (c.k, c.v, c.ke, c.ve) if t is not None]


def clone_cache(c):
    """The pools' bytes in memory of their own, with the same strides."""
    out = []
    for t in (c.k, c.v, c.ke, c.ve):
        if t is None:
            out.append(None)
            continue
        x = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device=t.device)
        x.view(torch.uint8).copy_(t.view(torch.uint8))
        out.append(x)
    return bd.PagedCache(*out)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("H,Hkv,d,r", [(4, 4, 64, 64), (4, 4, 64, 16), (8, 2, 128, 128), (8, 2, 128, 64), (8, 2, 128, 48),
                                       (4, 1, 256, 256), (4, 1, 256, 80), (10, 5, 128, 128)])
@pytest.mark.parametrize("new,kv", [([1], [1]), ([1, 0, 40, 200], [55, 20, 40, 700]), ([5, 3], [2, 0])])
def test_append(new, kv, H, Hkv, d, r, interleaved, fmt):
    """q against the oracle; the cache against a write of the turned K; everything else in the
    pool, and rows past the new ones, as they were."""
    c = pm.Case(new, kv, H, Hkv, d, fmt=fmt, heads_first=r % 3 == 1, junk=0.5, seed=d + r, pad_rows=2)
    f, pos = freqs(r), positions(new, kv)
    rope = bd.Rope(f, interleaved=interleaved, device="cuda")
    big = torch.randn(c.T + 2, (H + 2 * Hkv) * d, generator=torch.Generator().manual_seed(r)).bfloat16().cuda()
    q, k, v = (big[:, a * d:b * d].view(c.T + 2, b - a, d) for a, b in ((0, H), (H, H + Hkv), (H + Hkv, H + 2 * Hkv)))
    ref = clone_cache(c)
    out = torch.full((c.T + 2, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    bd.bd_cache_append(c.plan, q, k, v, rope, c.cache, out)
    # K's turned rows, as q of a call with as many heads as K has
    kt = torch.empty(c.T + 2, Hkv, d, dtype=torch.bfloat16, device="cuda")
    same = bd.PagedPlan(new, kv, c.pages, Hkv, Hkv, d, page_size=c.page, num_pages=c.num_pages, fmt=c.cache.fmt).upload("cuda")
    bd.bd_cache_append(same, k, k, v, rope, clone_cache(c), kt)
    bd.bd_cache_write(c.plan, kt, v, ref)
    torch.cuda.synchronize()
    assert (out[c.T:] == 7).all()
    check_turned(out[:c.T].cpu(), q[:c.T].cpu(), pos, f, interleaved)
    check_turned(kt[:c.T].cpu(), k[:c.T].cpu(), pos, f, interleaved)
    for a, b in ((c.k, ref.k), (c.v, ref.v), (c.ke, ref.k_exp), (c.ve, ref.v_exp)):
        assert a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    if fmt == "bf16":
        for t, s in enumerate(op.slots(new, kv, c.pages, c.page)):
            if s >= 0:
                assert torch.equal(c.k[s // c.page, s % c.page], kt[t]) and torch.equal(c.v[s // c.page, s % c.page], v[t])


def test_many_rows_take_several_heads_a_group():
    """Rows enough for groups of several heads of a row, whose last group is short."""
    H, Hkv, d = 7, 1, 128
    T = 40000
    c = pm.Case([T], [T], H, Hkv, d, page=1024, junk=0.0)
    f = freqs(d)
    g = torch.Generator(device="cuda").manual_seed(0)
    q, k, v = (torch.randn(T, h, d, generator=g, device="cuda").bfloat16() for h in (H, Hkv, Hkv))
    out = torch.empty_like(q)
    bd.bd_cache_append(c.plan, q, k, v, bd.Rope(f, device="cuda"), c.cache, out)
    torch.cuda.synchronize()
    at = [0, 1, 2, 777, 20001, T - 2, T - 1]
    check_turned(out[at].cpu(), q[at].cpu(), at, f)
    rows = torch.stack([c.k[c.pages[0][p // 1024], p % 1024] for p in at])
    check_turned(rows.cpu(), k[at].cpu(), at, f)
    a = torch.arange(T, device="cuda").double()[:, None] * f.cuda().double()
    u, w = q.double()[..., :64], q.double()[..., 64:]
    want = torch.cat([u * a.cos()[:, None] - w * a.sin()[:, None], w * a.cos()[:, None] + u * a.sin()[:, None]], -1)
    size = (u.abs() + w.abs()).repeat(1, 1, 2)
    assert ((out.double() - want).abs() <= want.abs() * 2.0 ** -8 + size * (2.0 ** -21 + 1e-9)).all()
    vr = torch.stack([c.v[c.pages[0][p // 1024], p % 1024] for p in at])
    assert torch.equal(vr, v[at])


@pytest.mark.parametrize("kv", [1 << 20, 123_456_789, 2_000_000_000])
def test_far_positions(kv):
    """Angles of positions up to 2^31 lose nothing (one page stands for all earlier ones)."""
    P, new = 1024, 5
    npg = -(-kv // P)
    pages = np.zeros(npg, dtype=np.int32)
    pages[-1], pages[-2] = 1, 2
    plan = bd.PagedPlan([new], [kv], [pages], 2, 2, 64, page_size=P, num_pages=3).upload("cuda")
    cache = bd.PagedCache(*(torch.zeros(3, P, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    x = torch.randn(new, 2, 64, generator=torch.Generator().manual_seed(1)).bfloat16()
    f = torch.cat([freqs(32), torch.tensor([3.0, 100.5, 0.0, -0.25] + [1e-9] * 12)])
    out = torch.empty(new, 2, 64, dtype=torch.bfloat16, device="cuda")
    bd.bd_cache_append(plan, x.cuda(), x.cuda(), x.cuda(), bd.Rope(f, device="cuda"), cache, out)
    torch.cuda.synchronize()
    check_turned(out.cpu(), x, range(kv - new, kv), f)


@pytest.mark.parametrize("fmt", FORMATS)
def test_q_in_place_and_no_q(fmt):
    c = pm.Case([1, 30], [90, 300], 8, 2, 128, fmt=fmt, junk=0.5)
    d = pm.Case([1, 30], [90, 300], 8, 2, 128, fmt=fmt, junk=0.5)
    rope = bd.Rope(freqs(128), device="cuda")
    q, k, v = c.q.cuda(), c.k_new.cuda(), c.v_new.cuda()
    out = torch.empty_like(q)
    bd.bd_cache_append(c.plan, q, k, v, rope, c.cache, out)
    bd.bd_cache_append(d.plan, None, k, v, rope, d.cache)
    bd.bd_cache_append(d.plan, q, k, v, rope, d.cache, q)
    torch.cuda.synchronize()
    assert torch.equal(q, out)
    for a, b in zip(pools(c), pools(d)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_scale():
    c = pm.Case([30], [300], 8, 2, 128, junk=0.5)
    f, q = freqs(64), c.q.cuda()
    out = torch.empty_like(q)
    bd.bd_cache_append(c.plan, q, c.k_new.cuda(), c.v_new.cuda(), bd.Rope(f, scale=1.25, device="cuda"), c.cache, out)
    check_turned(out.cpu(), c.q, positions([30], [300]), f, scale=1.25)


@pytest.mark.parametrize("fmt", FORMATS)
def test_infinities_stay_where_they_are(fmt):
    """An infinity in V, or in elements that do not turn, meets no other element."""
    c = pm.Case([3], [40], 4, 1, 128, fmt=fmt, junk=0.5)
    f, q, v = freqs(64), c.q.clone(), c.v_new.clone()
    q[:, :, 100], v[:, :, 100] = float("inf"), float("-inf")
    out = torch.empty_like(q, device="cuda")
    bd.bd_cache_append(c.plan, q.cuda(), c.k_new.cuda(), v.cuda(), bd.Rope(f, device="cuda"), c.cache, out)
    back = [torch.empty(40, 1, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    bd.bd_cache_read(c.plan, c.cache, *back)
    got = out.cpu()
    assert torch.equal(torch.isinf(got), torch.isinf(q)) and not torch.isnan(got).any()
    odd = ~torch.isfinite(back[1][37:].cpu())
    wide = {"bf16": slice(100, 101), "e4m3": slice(0, 128), "e2m1": slice(96, 112)}[fmt]
    assert odd[:, :, wide].all() and odd.sum() == 3 * (wide.stop - wide.start)
    assert torch.isfinite(back[0]).all() and torch.isfinite(back[1][:37]).all()


def test_captured_append_replays_over_the_next_positions():
    H, Hkv, d, P, f = 8, 2, 128, 16, freqs(128)
    pages = [list(range(20)), list(range(20, 60))]
    cache = bd.PagedCache(*(torch.zeros(60, P, Hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    rope = bd.Rope(f, device="cuda")

    def plan_of(i):
        return bd.PagedPlan([1, 2], [100 + i, 555 + 2 * i], pages, H, Hkv, d, page_size=P, num_pages=60)

    plan = plan_of(0)
    buf = torch.zeros(plan.nbytes // 4 + 64, dtype=torch.int32, device="cuda")
    plan.upload(buffer=buf)
    g = torch.Generator().manual_seed(2)
    q, k, v = (torch.zeros(3, h, d, dtype=torch.bfloat16, device="cuda") for h in (H, Hkv, Hkv))
    out = torch.zeros_like(q)
    bd.bd_cache_append(plan, q, k, v, rope, cache, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bd.bd_cache_append(plan, q, k, v, rope, cache, out)
    for i in range(3):
        nxt = plan_of(i)
        assert nxt.key() == plan.key()
        nxt.upload(buffer=buf)
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=g).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        pos = positions([1, 2], [100 + i, 555 + 2 * i])
        check_turned(out.cpu(), q.cpu(), pos, f)
        rows = torch.stack([cache.k[s // P, s % P] for s in op.slots([1, 2], [100 + i, 555 + 2 * i], pages, P)])
        check_turned(rows.cpu(), k.cpu(), pos, f)


@pytest.mark.parametrize("fmt", FORMATS)
def test_prompt_and_decode_as_they_are_used(fmt):
    """A prompt and then single rows appended turned and attended: the attention of turned rows
    over what the cache holds of turned rows."""
    H, Hkv, d, P, n0, steps = 8, 2, 128, 16, 150, 3
    f, total = freqs(128), 150 + 3
    g = torch.Generator().manual_seed(9)
    q, k, v = (torch.randn(total, h, d, generator=g).bfloat16().cuda() for h in (H, Hkv, Hkv))
    c = pm.Case([0], [total], H, Hkv, d, fmt=fmt, junk=0.0)
    rope = bd.Rope(f, device="cuda")
    at = 0
    for n in [n0] + [1] * steps:
        plan = bd.PagedPlan([n], [at + n], c.pages, H, Hkv, d, page_size=P, num_pages=c.num_pages, fmt=c.cache.fmt).upload("cuda")
        x = q[at:at + n].clone()
        bd.bd_cache_append(plan, x, k[at:at + n], v[at:at + n], rope, c.cache, x)
        out, lse = bd.paged_attn(plan, x, c.cache)
        back = [torch.empty(at + n, Hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        bd.bd_cache_read(plan, c.cache, *back)
        torch.cuda.synchronize()
        bd.bd_check_status(plan)
        check_turned(x.cpu(), q[at:at + n].cpu(), range(at, at + n), f)
        K, V = (b.cpu().double() for b in back)
        if fmt == "bf16":
            check_turned(back[0].cpu(), k[:at + n].cpu(), range(at + n), f)
        o, l, A, big = op.attention(x.cpu(), K, V, at + n)
        to, tl = pm.tolerances(d, at + n, A, big, fmt, n * H // Hkv, V.abs().max().item())
        pm.compare(out.cpu(), lse.cpu(), o, l, to, tl, at)
        at += n
