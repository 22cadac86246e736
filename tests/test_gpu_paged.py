"""GPU parity of the paged K/V cache: writing, reading back and attention of new rows,
through the C ABI, against the float64 oracle."""
import pytest
import torch

import oracle
from oracle import paged as op

pytestmark = pytest.mark.gpu

bd = pytest.importorskip("block_causal_varlen_gb300")
pu = pytest.importorskip("paged_util")

HEADS = [(4, 4, 64), (8, 2, 128), (4, 1, 256)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bd.load()


def bits(t):
    return t.contiguous().view(torch.uint8).cpu()


# ------------------------------------------------------------------ attention: shapes

SMALL = [([1], [1]), ([1], [16]), ([1, 1, 1], [17, 15, 130]), ([2, 0, 1], [33, 40, 257])]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,Hkv,d", HEADS)
@pytest.mark.parametrize("new,kv", SMALL)
def test_few_rows(new, kv, H, Hkv, d, fmt):
    c = pu.Case(new, kv, H, Hkv, d, fmt=fmt, seed=len(kv) + d)
    pu.check_attention(c, *pu.run_attention(c))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new,kv", [([8, 9], [300, 1000]), ([12, 5, 13], [700, 33, 2000]), ([12], [9001])])
def test_around_the_few_rows_limit(new, kv, d, fmt):
    """32 (bf16) and 48 (e4m3) pairs of a K/V head, in several blocks, and one row more."""
    c = pu.Case(new, kv, 8, 2, d, page=32, fmt=fmt, seed=d + len(new))
    pu.check_attention(c, *pu.run_attention(c))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,Hkv,d", HEADS)
def test_long_context_is_split_and_joined(H, Hkv, d, fmt):
    c = pu.Case([1], [6001], H, Hkv, d, page=64, fmt=fmt, seed=d)
    pu.check_attention(c, *pu.run_attention(c))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,Hkv", [(10, 2), (7, 1), (32, 1), (20, 1), (6, 6), (24, 8), (128, 1)])
def test_head_groups(H, Hkv, fmt):
    c = pu.Case([1, 3, 9], [40, 700, 9], H, Hkv, 128, page=32, fmt=fmt, seed=H)
    pu.check_attention(c, *pu.run_attention(c))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,Hkv,d", HEADS)
@pytest.mark.parametrize("new,kv", [([130], [130]), ([40, 1, 300, 17], [40, 500, 333, 150]), ([257], [1031])])
def test_chunks(new, kv, H, Hkv, d, fmt):
    c = pu.Case(new, kv, H, Hkv, d, page=64, fmt=fmt, seed=sum(kv))
    pu.check_attention(c, *pu.run_attention(c))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 128, 1024])
@pytest.mark.parametrize("heads_first", [False, True])
def test_page_sizes_and_orders(page, heads_first, fmt):
    c = pu.Case([1, 70, 200], [1500, 70, 1100], 8, 2, 128, page=page, fmt=fmt, heads_first=heads_first, seed=page)
    pu.check_attention(c, *pu.run_attention(c))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kv", [1, 15, 17, 33, 40, 47, 49, 64, 131])
def test_last_chunk_in_the_pools_first_page(kv, d, fmt):
    """Pages of 16 and chunks of 32 keys: a last chunk of one page, which is the first of the
    pool (exponents past the keys' end are the last key's, never before the page)."""
    c = pu.Case([1, 2], [kv, 5], 4, 2, d, page=16, fmt=fmt, seed=kv)
    a, b = c.pages[0][-1], 0
    for pool in (c.k, c.v, c.ke, c.ve):
        if pool is not None:
            raw = pool.view(torch.uint8)
            raw[[a, b]] = raw[[b, a]]
    for t in (c.kd, c.vd):
        t[[a, b]] = t[[b, a]]
    swap = {a: b, b: a}
    c.pages = [[swap.get(x, x) for x in pg] for pg in c.pages]
    assert c.pages[0][-1] == 0
    c.plan = c.make_plan().upload("cuda")
    pu.check_attention(c, *pu.run_attention(c))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_rows_that_see_nothing(fmt):
    """Sequences with nothing cached, and more new rows than cached ones."""
    c = pu.Case([1, 3, 5, 90, 40], [0, 2, 0, 60, 500], 8, 2, 128, fmt=fmt)
    pu.check_attention(c, *pu.run_attention(c))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_every_row_sees_the_whole_slice(fmt):
    """causal = False: a slice of a context held elsewhere as well; an empty slice gives
    O = 0, LSE = -inf."""
    c = pu.Case([1, 3, 70, 2], [100, 1, 300, 0], 8, 2, 128, fmt=fmt, causal=False)
    pu.check_attention(c, *pu.run_attention(c))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("qscale", [2.0 ** -40, 30.0])
def test_flat_and_peaked_scores(fmt, qscale):
    """Scores near zero (every key the same weight) and scores of some hundreds (one key
    takes all; the running maximum moves by large steps)."""
    c = pu.Case([1, 5, 150], [2000, 300, 150], 8, 2, 128, fmt=fmt, qscale=qscale)
    pu.check_attention(c, *pu.run_attention(c))


def test_rows_past_the_last_sequence_are_left_alone():
    c = pu.Case([1, 20], [40, 333], 8, 2, 128, pad_rows=5)
    out = torch.full((26, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((8, 26), 7.0, device="cuda")
    bd.bd_paged_attn(c.plan, c.q.cuda(), c.cache, out, lse)
    torch.cuda.synchronize()
    assert (out[21:] == 7).all() and (lse[:, 21:] == 7).all()
    pu.check_attention(c, out.cpu(), lse.cpu())


def test_strided_rows_and_no_lse():
    """q and out as slices of a fused projection's rows; LSE not asked for."""
    c = pu.Case([1, 40, 130], [900, 40, 600], 8, 2, 128, page=64)
    big = torch.full((c.T, 14 * 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    q = big[:, 128:9 * 128].view(c.T, 8, 128)
    q.copy_(c.q)
    wide = torch.zeros(c.T, 8, 256, dtype=torch.bfloat16, device="cuda")
    out = wide[:, :, 128:]
    bd.bd_paged_attn(c.plan, q, c.cache, out)
    torch.cuda.synchronize()
    _, lse = pu.run_attention(c)
    pu.check_attention(c, out.cpu(), lse)
    assert (wide[:, :, :128] == 0).all()


def test_shared_pages():
    """Two sequences over the same pages, at different lengths."""
    c = pu.Case([1, 2], [200, 100], 8, 2, 128, page=16)
    c.pages[1] = c.pages[0][:7]
    c.kd = c.kd.clone()
    c.plan = c.make_plan().upload("cuda")
    pu.check_attention(c, *pu.run_attention(c))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_nan_in_the_cache_reaches_those_who_see_it_only(fmt):
    """A NaN row in the middle of a sequence makes that sequence's rows NaN, nobody else's."""
    c = pu.Case([1, 1], [100, 300], 8, 2, 128, fmt=fmt, junk=0.0)
    page, row = c.pages[1][3], 5
    if fmt == "bf16":
        c.v[page, row, 0] = float("nan")
    else:
        c.ve[page, row, 0] = 255
    out, lse = pu.run_attention(c)
    assert torch.isnan(out[1, :4]).all() and torch.isfinite(out[1, 4:]).all() and torch.isfinite(out[0]).all()
    assert torch.isfinite(lse).all()
    if fmt == "bf16":
        c.k[page, row, 0] = float("nan")
    else:
        c.ke[page, row, 0] = 255
    out, lse = pu.run_attention(c)
    assert torch.isnan(lse[:4, 1]).all() and torch.isfinite(lse[4:, 1]).all() and torch.isfinite(lse[:, 0]).all()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,Hkv,d,new,kv", [(8, 2, 64, 4, 100), (8, 2, 128, 4, 100), (8, 2, 256, 4, 100), (8, 2, 128, 8, 70),
                                            (8, 2, 256, 8, 70), (8, 2, 128, 3, 3000), (8, 2, 64, 150, 400),
                                            (8, 2, 128, 150, 400), (8, 2, 256, 150, 400), (2, 2, 128, 300, 300),
                                            (2, 2, 64, 300, 290), (8, 2, 128, 70, 9001), (8, 2, 256, 40, 5000)])
def test_rows_take_nothing_from_keys_they_do_not_see(H, Hkv, d, new, kv, fmt):
    """Infinities and NaN in cached rows of the step itself reach the new rows that see
    them, in the columns they are in, and no others."""
    c = pu.Case([new], [kv], H, Hkv, d, fmt=fmt, page=32, seed=new)
    first = kv - new  # position of new row 0
    spots = sorted({max(0, first + new // 2), max(0, first + 1), kv - 1})
    bad = torch.zeros(new, d, dtype=torch.bool)  # of K/V head 0
    for n, pos in enumerate(spots):
        page, row = c.pages[0][pos // 32], pos % 32
        if fmt == "bf16":
            for col, x in ((7 + n, float("nan")), (d // 2 + n, float("inf")), (d - 9 + n, float("-inf"))):
                c.v[page, row, 0, col] = x
                c.vd[page, row, 0, col] = 0
                bad[pos - first:, col] = True
        else:
            c.v.view(torch.uint8)[page, row, 0] = 0x7f
            c.ve[page, row, 0] = 255
            c.vd[page, row, 0] = 0
            bad[pos - first:] = True
    out, lse = pu.run_attention(c)
    G = H // Hkv
    o, l, A, big = op.attention(c.q[:new], *c.rows(0), kv)
    to, tl = pu.tolerances(d, kv, A, big, fmt, new * G)
    hit = torch.zeros(new, H, d, dtype=torch.bool)
    hit[:, :G] = bad[:, None]
    assert not torch.isfinite(out[hit]).any()
    assert torch.isfinite(out[~hit]).all()
    assert ((out.double() - o).abs() <= to)[~hit].all()
    seen = ~torch.isneginf(l)
    assert torch.equal(~torch.isneginf(lse), seen) and ((lse.double() - l).abs() <= tl)[seen].all()
    # a K row of NaN
    page, row = c.pages[0][spots[1] // 32], spots[1] % 32
    if fmt == "bf16":
        c.k[page, row, 0, 3] = float("nan")
    else:
        c.ke[page, row, 0] = 255
    out2, lse2 = pu.run_attention(c)
    rows = torch.zeros(new, dtype=torch.bool)
    rows[spots[1] - first:] = True
    assert torch.isnan(lse2[:G, rows]).all() and torch.isnan(out2[rows, :G]).all()
    assert torch.equal(lse2[:G, ~rows], lse[:G, ~rows]) and torch.equal(lse2[G:], lse[G:])
    assert torch.equal(out2[:, G:], out[:, G:])
    a, b = out2[~rows, :G], out[~rows, :G]
    assert torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(1.0), b.nan_to_num(1.0))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,Hkv,d", HEADS)
def test_chunk_over_a_long_context_is_split_and_joined(H, Hkv, d, fmt):
    """Few blocks of tiles: their keys are cut over the SMs; at G = 3 a tile has idle rows."""
    c = pu.Case([70], [9001], H, Hkv, d, page=64, fmt=fmt, seed=d)
    pu.check_attention(c, *pu.run_attention(c))
    c = pu.Case([50, 3], [5000, 700], 3, 1, d, page=16, fmt=fmt, seed=d + 1)
    pu.check_attention(c, *pu.run_attention(c))


@pytest.mark.parametrize("new,kv", [([1, 2], [300, 90]), ([60], [200])])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("vmag", [(20, 40), (-40, 40), (-58, -50)])
def test_exponents_of_any_size(vmag, d, new, kv):
    """V rows whose exponents take two factors in a bf16 tile, span 2^80, or sit at the
    format's lower end; K's exponents away from q's."""
    c = pu.Case(new, kv, 4, 1, d, fmt="e4m3", seed=d, vmag=vmag, kmag=(18, 20), qscale=2.0 ** -20)
    pu.check_attention(c, *pu.run_attention(c))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_one_pool_for_k_and_v(fmt):
    """K and V as slices of one pool [pages, 2, page, heads, d], exponents likewise."""
    c = pu.Case([1, 40], [300, 90], 8, 2, 128, page=32, fmt=fmt)
    want = pu.run_attention(c)
    both = torch.stack([c.k.view(torch.uint8), c.v.view(torch.uint8)], 1).view(c.k.dtype)
    ex = (None, None) if fmt == "bf16" else torch.stack([c.ke, c.ve], 1).unbind(1)
    c.cache = bd.PagedCache(both[:, 0], both[:, 1], *ex)
    got = pu.run_attention(c)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    k = torch.empty(390, 2, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    bd.bd_cache_read(c.plan, c.cache, k, v)
    assert torch.equal(k.cpu().double(), torch.cat([c.rows(b)[0] for b in range(2)]))
    assert torch.equal(v.cpu().double(), torch.cat([c.rows(b)[1] for b in range(2)]))


def test_pools_past_2_31_elements():
    """The last pages of pools of more than 2^31 elements each."""
    H, Hkv, d, P = 8, 8, 128, 1024
    n = 2 ** 31 // (P * Hkv * d) + 3
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    k = torch.empty(n, P, Hkv, d, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    cache = bd.PagedCache(k, v)
    g = torch.Generator().manual_seed(0)
    new = [40, 1]
    kn, vn, q = (torch.randn(41, h, d, generator=g).bfloat16() for h in (Hkv, Hkv, H))
    plan = bd.PagedPlan(new, new, [[n - 1], [n - 2]], H, Hkv, d, page_size=P, num_pages=n).upload("cuda")
    bd.bd_cache_write(plan, kn.cuda(), vn.cuda(), cache)
    out, lse = bd.paged_attn(plan, q.cuda(), cache)
    kr, vr = torch.empty(41, Hkv, d, dtype=torch.bfloat16, device="cuda"), torch.empty(41, Hkv, d, dtype=torch.bfloat16, device="cuda")
    bd.bd_cache_read(plan, cache, kr, vr)
    torch.cuda.synchronize()
    bd.bd_check_status(plan)
    assert torch.equal(kr.cpu(), kn) and torch.equal(vr.cpu(), vn)
    assert torch.equal(k[n - 1, :40].cpu(), kn[:40]) and torch.equal(v[n - 2, :1].cpu(), vn[40:])
    at = 0
    for m in new:
        o, l, A, big = op.attention(q[at:at + m], kn[at:at + m], vn[at:at + m], m)
        to, tl = pu.tolerances(d, m, A, big, "bf16")
        assert ((out[at:at + m].cpu().double() - o).abs() <= to).all() and ((lse[:, at:at + m].cpu().double() - l).abs() <= tl).all()
        at += m


# ------------------------------------------------------------------ attention: calls

def _mixed(fmt="bf16", seed=0):
    return pu.Case([1, 1, 60, 200], [5000, 40, 700, 900], 8, 2, 128, page=32, fmt=fmt, seed=seed)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_same_bits_every_time(fmt):
    c = _mixed(fmt)
    a, b = pu.run_attention(c), pu.run_attention(c)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_two_calls_at_once_on_one_plan():
    """Calls on two streams share the device plan and have workspaces of their own."""
    c = _mixed()
    want = pu.run_attention(c)
    q = c.q.cuda()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    torch.cuda.synchronize()
    for i in range(6):
        s = streams[i % 2]
        with torch.cuda.stream(s):
            out = torch.empty(c.T, 8, 128, dtype=torch.bfloat16, device="cuda")
            lse = torch.empty(8, c.T, device="cuda")
            bd.bd_paged_attn(c.plan, q, c.cache, out, lse)
            outs.append((out, lse))
    torch.cuda.synchronize()
    for out, lse in outs:
        assert torch.equal(out.cpu(), want[0]) and torch.equal(lse.cpu(), want[1])


def test_stream_argument():
    c = _mixed()
    want = pu.run_attention(c)
    s = torch.cuda.Stream()
    got = pu.run_attention(c, stream=s)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_captured_step_replays_with_the_next_steps_plan():
    """write + attention of a decode step captured once and replayed over three steps,
    the device plan overwritten between them."""
    H, Hkv, d, P = 8, 2, 128, 16
    pages = [list(range(0, 320)), list(range(320, 340))]
    kv0 = [5000, 250]
    g = torch.Generator().manual_seed(2)
    k = torch.randn(340, P, Hkv, d, generator=g).bfloat16().cuda()
    v = torch.randn(340, P, Hkv, d, generator=g).bfloat16().cuda()
    cache = bd.PagedCache(k, v)

    def plan_of(step):
        return bd.PagedPlan([1, 1], [n + step for n in kv0], pages, H, Hkv, d, page_size=P, num_pages=340)

    plan = plan_of(1)
    buf = torch.zeros(plan.nbytes // 4 + 64, dtype=torch.int32, device="cuda")
    plan.upload(buffer=buf)
    q, kn, vn = (torch.zeros(2, h, d, dtype=torch.bfloat16, device="cuda") for h in (H, Hkv, Hkv))
    out, lse = torch.zeros(2, H, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(H, 2, device="cuda")
    ws = torch.empty(bd.bd_paged_attn_workspace(plan), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):      # the first calls set kernel attributes
        bd.bd_cache_write(plan, kn, vn, cache)
        bd.bd_paged_attn(plan, q, cache, out, lse, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bd.bd_cache_write(plan, kn, vn, cache)
        bd.bd_paged_attn(plan, q, cache, out, lse, ws)
    for step in range(1, 4):
        nxt = plan_of(step)
        assert nxt.key() == plan.key()
        nxt.upload(buffer=buf)
        for t in (q, kn, vn):
            t.copy_(torch.randn(t.shape, generator=g).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        for b in range(2):
            n = kv0[b] + step
            K, V = op.rows_of(k.cpu(), n, pages[b], P), op.rows_of(v.cpu(), n, pages[b], P)
            assert torch.equal(K[-1], kn[b].cpu()) and torch.equal(V[-1], vn[b].cpu())
            o, l, A, big = op.attention(q[b:b + 1].cpu(), K, V, n)
            to, tl = pu.tolerances(d, n, A, big, "bf16")
            assert ((out[b:b + 1].cpu().double() - o).abs() <= to).all() and ((lse[:, b:b + 1].cpu().double() - l).abs() <= tl).all()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_captured_layers_replay_with_tiles_and_few_rows(fmt):
    """Two layers' writes and attention (few-rows blocks, tiles and both joins) in one graph,
    on one workspace, replayed over other lengths of the same key: the bits of eager calls."""
    H, Hkv, d, P, pages = 8, 2, 128, 32, [list(range(0, 300)), list(range(300, 600)), list(range(600, 700))]
    g = torch.Generator().manual_seed(5)

    def pool():
        x = [torch.randn(700, P, Hkv, d, generator=g).bfloat16() for _ in range(2)]
        if fmt == "bf16":
            return bd.PagedCache(*[t.cuda() for t in x])
        (kc, ke), (vc, ve) = op.quantise(x[0]), op.quantise(x[1])
        return bd.PagedCache(*[t.cuda().view(torch.float8_e4m3fn) for t in (kc, vc)], ke.cuda(), ve.cuda())

    layers = [pool() for _ in range(2)]

    def plan_of(new, kv):
        return bd.PagedPlan(new, kv, pages, H, Hkv, d, page_size=P, num_pages=700, fmt=layers[0].fmt)

    steps = [([70, 1, 3], [9001, 8000, 900]), ([50, 3, 1], [7000, 9500, 3]), ([90, 1, 4], [9600, 6000, 1000])]
    plans = [plan_of(*s) for s in steps]
    assert len({p.key() for p in plans}) == 1
    buf = torch.zeros(max(p.nbytes for p in plans) // 4, dtype=torch.int32, device="cuda")
    ws = torch.empty(bd.bd_paged_attn_workspace(plans[0]), dtype=torch.uint8, device="cuda")
    q, kn, vn = (torch.randn(2, 100, h, d, generator=g).bfloat16().cuda() for h in (H, Hkv, Hkv))
    out = torch.zeros(2, 100, H, d, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(2, H, 100, device="cuda")

    def step(plan):
        for i, c in enumerate(layers):
            bd.bd_cache_write(plan, kn[i], vn[i], c)
            bd.bd_paged_attn(plan, q[i], c, out[i], lse[i], ws)

    want = []
    for p in plans + plans:  # (rows one step writes are others' context: they are there the second time)
        out.fill_(7)
        lse.fill_(7)
        step(p.upload("cuda"))
        want.append((out.clone(), lse.clone()))
    want = want[3:]
    torch.cuda.synchronize()
    plans[0].upload(buffer=buf)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(plans[0])
    for i in (1, 2, 0):
        plans[i].upload(buffer=buf)
        out.fill_(7)
        lse.fill_(7)
        graph.replay()
        assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])
        bd.bd_check_status(plans[i])


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,kv", [([1], [90]), ([1, 2], [3000, 40]), ([60, 1, 200], [5000, 700, 260])])
def test_calls_in_a_row_wait_for_each_other(new, kv, fmt):
    """Grids may start before the one in front of them has ended: q, K and V written by other
    kernels right before a call, the cache rows that a write leaves for the attention behind it, results
    read right after, a plan copied in between; eager and in a graph, the bits of calls with a
    synchronisation after each operation."""
    c = pu.Case(new, kv, 8, 2, 128, page=32, fmt=fmt, junk=0.0)
    other = pu.Case(new, kv, 8, 2, 128, page=32, fmt=fmt, junk=0.0, seed=1)  # same key, other pages
    assert c.plan.key() == other.plan.key() and c.num_pages == other.num_pages
    buf = torch.zeros(max(c.plan.nbytes, other.plan.nbytes) // 4, dtype=torch.int32, device="cuda")
    blobs = [torch.zeros_like(buf) for _ in range(2)]
    for b, x in zip(blobs, (c, other)):
        b[:len(x.plan.host)] = torch.from_numpy(x.plan.host).cuda()
    c.plan.upload(buffer=buf)
    T, N = c.T, 12
    g = torch.Generator().manual_seed(3)
    qs, ks, vs = (torch.randn(N, T, h, 128, generator=g).bfloat16().cuda() for h in (8, 2, 2))
    q, k, v = (torch.empty_like(t[0]) for t in (qs, ks, vs))
    out, lse = torch.empty_like(q), torch.empty(8, T, device="cuda")
    ws = torch.empty(max(256, bd.bd_paged_attn_workspace(c.plan)), dtype=torch.uint8, device="cuda")
    back = [torch.empty(sum(kv), 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    start = [t.clone() if t is not None else None for t in (c.k, c.v, c.ke, c.ve)]

    def rows(sync):
        ops = []
        for t, t0 in zip((c.k, c.v, c.ke, c.ve), start):
            if t is not None:
                t.view(torch.uint8).copy_(t0.view(torch.uint8))
        got = []
        for i in range(N):
            ops = [lambda: buf.copy_(blobs[i % 2]), lambda: q.copy_(qs[i]), lambda: k.copy_(ks[i]), lambda: v.copy_(vs[i]),
                   lambda: bd.bd_cache_write(c.plan, k, v, c.cache), lambda: bd.bd_paged_attn(c.plan, q, c.cache, out, lse, ws),
                   lambda: got.extend([out.clone(), lse.clone()]), lambda: bd.bd_cache_read(c.plan, c.cache, *back),
                   lambda: got.extend([b.clone() for b in back])]
            for op_ in ops:
                op_()
                if sync:
                    torch.cuda.synchronize()
        return got

    want = rows(True)
    for _ in range(3):
        got = rows(False)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = rows(False)
    for _ in range(3):
        for t in got:
            t.fill_(1)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_captured_fork_and_join():
    """A call behind two branches of a graph, one of kernels and one of a copy, and two calls
    in branches of their own: each waits for what is in front of it."""
    c = _mixed()
    q0 = c.q.cuda()
    want = pu.run_attention(c)
    q, half, big = torch.zeros_like(q0), torch.zeros_like(q0), torch.ones(1 << 24, device="cuda")
    outs = [torch.zeros(c.T, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    lses = [torch.zeros(8, c.T, device="cuda") for _ in range(3)]
    ws = [torch.empty(bd.bd_paged_attn_workspace(c.plan), dtype=torch.uint8, device="cuda") for _ in range(3)]
    side = torch.cuda.Stream()
    bd.bd_paged_attn(c.plan, q0, c.cache, outs[0], lses[0], ws[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            for _ in range(8):
                big.mul_(1.0)
            torch.mul(q0, 0.5, out=half)
        big2 = big.clone()
        main.wait_stream(side)
        torch.add(half, half, out=q)
        bd.bd_paged_attn(c.plan, q, c.cache, outs[0], lses[0], ws[0])
        side.wait_stream(main)
        with torch.cuda.stream(side):
            bd.bd_paged_attn(c.plan, q, c.cache, outs[1], lses[1], ws[1])
        bd.bd_paged_attn(c.plan, q, c.cache, outs[2], lses[2], ws[2])
        main.wait_stream(side)
        sums = [o.float().sum() for o in outs]
    for _ in range(5):
        for t in outs + lses + [q, half]:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for o, l, s in zip(outs, lses, sums):
            assert torch.equal(o.cpu(), want[0]) and torch.equal(l.cpu(), want[1])
            assert torch.equal(s, o.float().sum())
    assert big2.numel() == big.numel()


def test_upload_leaves_another_plans_buffer_alone():
    """A plan once uploaded into a shared buffer takes memory of its own the next time."""
    a, b = (bd.PagedPlan([1], [n], [[0, 1, 2]], 4, 2, 64, page_size=16, num_pages=3) for n in (20, 40))
    buf = torch.zeros(max(a.nbytes, b.nbytes) // 4, dtype=torch.int32, device="cuda")
    a.upload(buffer=buf)
    b.upload(buffer=buf)
    a.upload("cuda:0")
    assert torch.equal(buf[:len(b.host)].cpu(), torch.from_numpy(b.host))
    assert torch.equal(a.dev.cpu(), torch.from_numpy(a.host))
    own = a.dev.data_ptr()
    assert a.upload("cuda:0").dev.data_ptr() == own  # and keeps that


def test_memory_allocated_for_a_call_is_its_streams():
    """Results and workspace allocated by a call on a stream argument are not memory the
    caller's stream still works on."""
    c = _mixed()
    want = pu.run_attention(c)
    q, s = c.q.cuda(), torch.cuda.Stream()
    n = 1 << 28
    bd.paged_attn(c.plan, q, c.cache, stream=s)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    x = torch.ones(n, device="cuda")
    for _ in range(20):  # work in flight on the caller's stream, its memory given back
        x = x * 1.5
    x = None
    got = bd.paged_attn(c.plan, q, c.cache, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got[0].cpu(), want[0]) and torch.equal(got[1].cpu(), want[1])


def test_nothing_new_and_nothing_cached():
    c = pu.Case([0, 0], [20, 0], 8, 2, 128)
    out = torch.full((1, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    k = torch.full((1, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    bd.bd_paged_attn(c.plan, out, c.cache, out)
    before = bits(c.k)
    bd.bd_cache_write(c.plan, k, k, c.cache)
    torch.cuda.synchronize()
    assert (out == 7).all() and torch.equal(bits(c.k), before)
    z = pu.Case([1], [0], 8, 2, 128)
    bd.bd_cache_read(z.plan, z.cache, k, k)
    torch.cuda.synchronize()
    assert (k == 7).all()


# ------------------------------------------------------------------ write and read

@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,Hkv,d", HEADS + [(10, 5, 128)])
@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("new,kv", [([1], [1]), ([1, 0, 40, 300], [55, 20, 40, 700]), ([5, 3], [2, 0])])
def test_write(new, kv, heads_first, H, Hkv, d, fmt):
    c = pu.Case(new, kv, H, Hkv, d, fmt=fmt, heads_first=heads_first, seed=d, junk=0.5, pad_rows=2)
    want = {n: getattr(c, n).cpu().clone().contiguous() for n in ("k", "v")}
    exps = {n: getattr(c, n + "e").cpu().clone().contiguous() if fmt == "e4m3" else None for n in ("k", "v")}
    # the rows come as slices of a fused projection
    big = torch.randn(c.T + 2, 2 * Hkv * d + 64, generator=torch.Generator().manual_seed(d)).bfloat16()
    if c.T > 4:   # values the format has to deal with: all zeros, subnormals, a row at a power's edge
        big[0] = 0
        big[1] = 2.0 ** -130
        big[2, 64] = 448.0
        big[3] *= 2.0 ** 40
    dev = big.cuda()
    kn, vn = (dev[:, 64 + i * Hkv * d:64 + (i + 1) * Hkv * d].view(c.T + 2, Hkv, d) for i in range(2))
    bd.bd_cache_write(c.plan, kn, vn, c.cache)
    torch.cuda.synchronize()
    for t, s in enumerate(op.slots(new, kv, c.pages, c.page)):
        if s < 0:
            continue
        for n, x in (("k", kn), ("v", vn)):
            row = x[t].cpu()
            if fmt == "bf16":
                want[n][s // c.page, s % c.page] = row
            else:
                codes, e = op.quantise(row)
                want[n].view(torch.uint8)[s // c.page, s % c.page] = codes
                exps[n][s // c.page, s % c.page] = e
    for n in ("k", "v"):
        assert torch.equal(bits(getattr(c, n)), bits(want[n])), n
        if fmt == "e4m3":
            assert torch.equal(getattr(c, n + "e").cpu(), exps[n]), n


def test_write_infinities_and_extremes():
    c = pu.Case([6], [6], 4, 1, 64, fmt="e4m3", junk=0.0)
    x = torch.randn(6, 1, 64, generator=torch.Generator().manual_seed(4)).bfloat16()
    x[0, 0, 3], x[1, 0, 9], x[2, 0, 60] = float("inf"), float("nan"), float("-inf")
    x[3] = 3e38          # past the largest exponent: saturates
    x[4] = 1e-30         # below the smallest one: rounds to codes of 2^-60
    bd.bd_cache_write(c.plan, x.cuda(), x.cuda(), c.cache)
    out = torch.empty(6, 1, 64, dtype=torch.bfloat16, device="cuda")
    bd.bd_cache_read(c.plan, c.cache, out, torch.empty_like(out))
    torch.cuda.synchronize()
    want = op.dequantise(*op.quantise(x))
    got = out.cpu().double()
    assert torch.isnan(got[:3]).all() and torch.equal(got[3:], want[3:])
    assert (got[3] == 448.0 * 2.0 ** 60).all()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,Hkv,d", HEADS + [(10, 5, 128)])
@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("kv", [[1], [16], [33, 0, 500, 7]])
def test_read(kv, heads_first, H, Hkv, d, fmt):
    c = pu.Case([0] * len(kv), kv, H, Hkv, d, page=32, fmt=fmt, heads_first=heads_first, seed=d)
    n = sum(kv)
    k = torch.full((n + 3, Hkv, 2 * d), 7.0, dtype=torch.bfloat16, device="cuda")[:, :, :d]
    v = torch.full((n + 3, Hkv, d), 7.0, dtype=torch.bfloat16, device="cuda")
    bd.bd_cache_read(c.plan, c.cache, k, v)
    torch.cuda.synchronize()
    assert (k[n:] == 7).all() and (v[n:] == 7).all()
    K = torch.cat([c.rows(b)[0] for b in range(len(kv))])
    V = torch.cat([c.rows(b)[1] for b in range(len(kv))])
    assert torch.equal(k[:n].cpu().double(), K) and torch.equal(v[:n].cpu().double(), V)


# ------------------------------------------------------------------ as they are used

@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_prompt_then_chunk_then_decode(fmt):
    """Packed prompts through the block-causal forward, their K/V written to the cache, a
    chunk and then single rows attended over it: the same O as whole documents give, and
    the rows read back feed the forward again."""
    H, Hkv, d, P = 8, 2, 128, 16
    lens, chunk, steps = [200, 37, 150], 70, 3
    total = [n + chunk + steps for n in lens]
    g = torch.Generator().manual_seed(9)
    full = [[torch.randn(n, h, d, generator=g).bfloat16() for h in (H, Hkv, Hkv)] for n in total]
    if fmt == "e4m3":   # whole documents of the values that the cache holds
        for f in full:
            for i in (1, 2):
                f[i] = op.dequantise(*op.quantise(f[i])).bfloat16()
    npg = [-(-n // P) for n in total]
    num_pages = sum(npg)
    perm = torch.randperm(num_pages, generator=g).tolist()
    pages, at = [], 0
    for n in npg:
        pages.append(perm[at:at + n])
        at += n
    dt = torch.bfloat16 if fmt == "bf16" else torch.float8_e4m3fn
    k = torch.full((num_pages, P, Hkv, d), 0xFF, dtype=torch.uint8, device="cuda").to(torch.float32)
    k = k.fill_(float("nan")).to(dt)
    v = k.clone()
    ex = [torch.full((num_pages, P, Hkv), 255, dtype=torch.uint8, device="cuda") for _ in range(2)] if fmt == "e4m3" else [None] * 2
    cache = bd.PagedCache(k, v, *ex)
    done = [0] * 3

    def step(new):
        nonlocal done
        kv = [a + b for a, b in zip(done, new)]
        plan = bd.PagedPlan(new, kv, pages, H, Hkv, d, page_size=P, num_pages=num_pages, fmt=cache.fmt).upload("cuda")
        q, kn, vn = (torch.cat([f[i][a:b] for f, a, b in zip(full, done, kv)]).cuda() for i in range(3))
        bd.bd_cache_write(plan, kn, vn, cache)
        out, lse = bd.paged_attn(plan, q, cache)
        torch.cuda.synchronize()
        bd.bd_check_status(plan)
        at = 0
        for b in range(3):
            o, l, A, big = op.attention(full[b][0][done[b]:kv[b]], full[b][1][:kv[b]], full[b][2][:kv[b]], kv[b])
            to, tl = pu.tolerances(d, kv[b], A, big, fmt, new[b] * H // Hkv)
            assert ((out[at:at + new[b]].cpu().double() - o).abs() <= to).all(), (new, b)
            assert ((lse[:, at:at + new[b]].cpu().double() - l).abs() <= tl).all(), (new, b)
            at += new[b]
        done = kv
        return plan, q, out

    # the prompts: the block-causal forward and the paged one agree
    _, q, out = step(lens)
    S = sum(lens)
    cu = [0, lens[0], lens[0] + lens[1], S]
    fp = bd.Plan([cu], S, 1, H, Hkv, d).upload("cuda")
    kk, vv = (torch.cat([f[i][:n] for f, n in zip(full, lens)]).cuda() for i in (1, 2))
    ref, _ = bd.attn_fwd(fp, q.view(1, 1, S, H, d), kk.view(1, 1, S, Hkv, d), vv.view(1, 1, S, Hkv, d))
    torch.cuda.synchronize()
    _, _, A, _ = op.attention(q.cpu(), kk.cpu(), vv.cpu(), S, causal=False)
    assert ((ref.view(S, H, d) - out).abs().cpu().double() <= 4 * 2.0 ** -8 * 3).all()
    step([chunk] * 3)
    for _ in range(steps):
        plan, _, _ = step([1] * 3)
    n = sum(done)
    kr, vr = (torch.empty(n, Hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    bd.bd_cache_read(plan, cache, kr, vr)
    torch.cuda.synchronize()
    assert torch.equal(kr.cpu(), torch.cat([f[1] for f in full])) and torch.equal(vr.cpu(), torch.cat([f[2] for f in full]))


def test_slices_join_by_lse():
    """A context cut in two slices (as context-parallel ranks hold it), attended without a
    causal mask and joined by the LSEs, is the whole."""
    c = pu.Case([1], [900], 8, 2, 128, page=16)
    K, V = c.rows(0)
    parts = []
    for lo, hi in ((0, 512), (512, 900)):
        plan = bd.PagedPlan([1], [hi - lo], [c.pages[0][lo // 16:]], 8, 2, 128, page_size=16, num_pages=c.num_pages,
                            causal=False).upload("cuda")
        parts.append([t.cpu().double() for t in bd.paged_attn(plan, c.q.cuda(), c.cache)])
    lse = torch.logaddexp(parts[0][1], parts[1][1])
    out = sum(o * torch.exp(l - lse).t()[..., None] for o, l in parts)
    want, wl, A, big = op.attention(c.q, K, V, 900)
    to, tl = pu.tolerances(128, 900, A, big, "bf16")
    assert ((out - want).abs() <= 2 * to).all() and ((lse - wl).abs() <= 2 * tl).all()
