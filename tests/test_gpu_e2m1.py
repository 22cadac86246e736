"""GPU parity of a paged K/V cache held in 4 bits: writing, reading back and attention of new
rows, through the C ABI, against the float64 oracle."""
import pytest
import torch

from oracle import paged as op
from oracle import paged_e2m1 as o4

pytestmark = pytest.mark.gpu

bd = pytest.importorskip("block_causal_varlen_gb300")
pu = pytest.importorskip("paged_util")
pm = pytest.importorskip("paged_more_util")

HEADS = [(4, 4, 64), (8, 2, 128), (4, 1, 256)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bd.load()


def Case(*a, **k):
    return pm.Case(*a, fmt="e2m1", **k)


# ------------------------------------------------------------------ write and read

@pytest.mark.parametrize("H,Hkv,d", HEADS + [(10, 5, 128)])
@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("new,kv", [([1], [1]), ([1, 0, 40, 300], [55, 20, 40, 700]), ([5, 3], [2, 0])])
def test_write(new, kv, heads_first, H, Hkv, d):
    c = Case(new, kv, H, Hkv, d, heads_first=heads_first, seed=d, junk=0.5, pad_rows=2)
    want = {n: getattr(c, n).cpu().clone().contiguous() for n in ("k", "v", "ke", "ve")}
    big = torch.randn(c.T + 2, 2 * Hkv * d + 64, generator=torch.Generator().manual_seed(d)).bfloat16()
    if c.T > 4:   # zeros, values below the least scale, past the largest, spread over a scale's range
        big[0] = 0
        big[1] *= 2.0 ** -18
        big[2] *= 2.0 ** 15
        big[3] = torch.randn(big.shape[1]).mul(3).exp2().bfloat16()
    dev = big.cuda()
    kn, vn = (dev[:, 64 + i * Hkv * d:64 + (i + 1) * Hkv * d].view(c.T + 2, Hkv, d) for i in range(2))
    bd.bd_cache_write(c.plan, kn, vn, c.cache)
    torch.cuda.synchronize()
    for t, s in enumerate(op.slots(new, kv, c.pages, c.page)):
        if s < 0:
            continue
        for n, x in (("k", kn), ("v", vn)):
            codes, e = o4.quantise(x[t].cpu())
            want[n][s // c.page, s % c.page], want[n + "e"][s // c.page, s % c.page] = codes, e
    for n in want:
        assert torch.equal(getattr(c, n).cpu(), want[n]), n


def test_write_every_tie():
    """Quotients midway between two codes, and their neighbours in bf16, for every scale byte;
    every maximum that is 6 times a scale or next to it."""
    rows = []
    for b in range(8, 227):
        s = o4.SCALES[b].item()
        x = torch.tensor([6 * s] + [m * s for m in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)]).bfloat16()
        assert torch.equal(x.double(), torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64) * s)
        bits = x.view(torch.int16)
        up, down = (bits + 1).view(torch.bfloat16), (bits - 1).view(torch.bfloat16)
        lo = torch.cat([x, -up[1:], down[:1]])           # the maximum is 6 s
        hi = torch.cat([x[1:], -down, up[:1]])           # the maximum is one step above
        mid = torch.cat([down, -x[1:], down[:1]])        # the maximum is one step below
        rows += [lo, hi, mid, -lo]
    x = torch.stack(rows)
    x = torch.cat([x, torch.zeros(-len(x) % 8, 16, dtype=x.dtype)]).view(-1, 1, 128)
    T = len(x)
    c = Case([T], [T], 1, 1, 128, page=64, junk=0.0)
    bd.bd_cache_write(c.plan, x.cuda(), x.flip(0).contiguous().cuda(), c.cache)
    back = [torch.empty(T, 1, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    bd.bd_cache_read(c.plan, c.cache, *back)
    torch.cuda.synchronize()
    want = o4.dequantise(*o4.quantise(x))
    assert torch.equal(back[0].cpu().double(), want)
    assert torch.equal(back[1].cpu().double().flip(0), want)


def test_write_infinities_and_extremes():
    c = Case([6], [6], 4, 1, 64, junk=0.0)
    x = torch.randn(6, 1, 64, generator=torch.Generator().manual_seed(4)).bfloat16()
    x[0, 0, 3], x[1, 0, 19], x[2, 0, 60] = float("inf"), float("nan"), float("-inf")
    x[3] = 3e38          # past the largest scale: saturates
    x[4] = 1e-30         # below the least one: rounds to zeros
    bd.bd_cache_write(c.plan, x.cuda(), x.cuda(), c.cache)
    out = torch.empty(6, 1, 64, dtype=torch.bfloat16, device="cuda")
    bd.bd_cache_read(c.plan, c.cache, out, torch.empty_like(out))
    torch.cuda.synchronize()
    want, got = o4.dequantise(*o4.quantise(x)), out.cpu().double()
    nan = torch.isnan(want)
    assert nan.sum() == 48 and torch.equal(torch.isnan(got), nan) and torch.equal(got[~nan], want[~nan])
    assert (got[3] == 61440).all() and (got[4] == 0).all()


@pytest.mark.parametrize("H,Hkv,d", HEADS + [(10, 5, 128)])
@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("kv", [[1], [16], [33, 0, 500, 7]])
def test_read(kv, heads_first, H, Hkv, d):
    c = Case([0] * len(kv), kv, H, Hkv, d, page=32, heads_first=heads_first, seed=d)
    n = sum(kv)
    k = torch.full((n + 3, Hkv, 2 * d), 7.0, dtype=torch.bfloat16, device="cuda")[:, :, :d]
    v = torch.full((n + 3, Hkv, d), 7.0, dtype=torch.bfloat16, device="cuda")
    bd.bd_cache_read(c.plan, c.cache, k, v)
    torch.cuda.synchronize()
    assert (k[n:] == 7).all() and (v[n:] == 7).all()
    K = torch.cat([c.rows(b)[0] for b in range(len(kv))])
    V = torch.cat([c.rows(b)[1] for b in range(len(kv))])
    assert torch.equal(k[:n].cpu().double(), K) and torch.equal(v[:n].cpu().double(), V)


def test_every_code_and_scale_reads_back():
    """All bytes of codes with all scale bytes that a cache may hold."""
    scales = torch.tensor(list(range(227)) + [255], dtype=torch.uint8)
    codes = torch.arange(256).to(torch.uint8).view(4, 64)                 # [4 rows, 64 bytes]
    page = codes.repeat(len(scales), 1).view(-1, 1, 64)                     # rows of 128 values
    n = len(page)
    num = -(-n // 16)
    k = torch.zeros(num * 16, 1, 64, dtype=torch.uint8)
    e = torch.zeros(num * 16, 1, 8, dtype=torch.uint8)
    k[:n], e[:n] = page, scales.repeat_interleave(4)[:, None, None]
    kd, ed = k.view(num, 16, 1, 64).cuda(), e.view(num, 16, 1, 8).cuda()
    cache = bd.PagedCache(kd, kd.clone(), ed, ed.clone())
    plan = bd.PagedPlan([0], [n], [list(range(num))], 1, 1, 128, page_size=16, num_pages=num, fmt=cache.fmt).upload("cuda")
    out = [torch.empty(n, 1, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    bd.bd_cache_read(plan, cache, *out)
    want = o4.dequantise(k[:n], e[:n])
    for t in out:
        got = t.cpu().double()
        nan = torch.isnan(want)
        assert torch.equal(torch.isnan(got), nan) and torch.equal(got[~nan], want[~nan])


# ------------------------------------------------------------------ attention

SMALL = [([1], [1]), ([1], [16]), ([1, 1, 1], [17, 15, 130]), ([2, 0, 1], [33, 40, 257])]


@pytest.mark.parametrize("H,Hkv,d", HEADS)
@pytest.mark.parametrize("new,kv", SMALL)
def test_few_rows(new, kv, H, Hkv, d):
    c = Case(new, kv, H, Hkv, d, seed=len(kv) + d)
    pm.check_attention(c, *pu.run_attention(c))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new,kv", [([8, 9], [300, 1000]), ([12, 5, 13], [700, 33, 2000]), ([12], [9001]), ([5, 6, 2], [700, 50, 3000]),
                                    ([6, 90], [5000, 300])])
def test_around_the_few_rows_limit(new, kv, d):
    c = Case(new, kv, 8, 2, d, page=32, seed=d + len(new))
    pm.check_attention(c, *pu.run_attention(c))


@pytest.mark.parametrize("H,Hkv,d", HEADS)
def test_long_context_is_split_and_joined(H, Hkv, d):
    c = Case([1], [6001], H, Hkv, d, page=64, seed=d)
    pm.check_attention(c, *pu.run_attention(c))


@pytest.mark.parametrize("H,Hkv", [(10, 2), (7, 1), (32, 1), (20, 1), (6, 6), (24, 8), (128, 1)])
def test_head_groups(H, Hkv):
    c = Case([1, 3, 9], [40, 700, 9], H, Hkv, 128, page=32, seed=H)
    pm.check_attention(c, *pu.run_attention(c))


@pytest.mark.parametrize("H,Hkv,d", HEADS)
@pytest.mark.parametrize("new,kv", [([130], [130]), ([40, 1, 300, 17], [40, 500, 333, 150]), ([257], [1031]), ([70], [9001])])
def test_chunks(new, kv, H, Hkv, d):
    c = Case(new, kv, H, Hkv, d, page=64, seed=sum(kv))
    pm.check_attention(c, *pu.run_attention(c))


@pytest.mark.parametrize("page", [16, 128, 1024])
@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_page_sizes_and_orders(page, heads_first, d):
    c = Case([1, 70, 200], [1500, 70, 1100], 8, 2, d, page=page, heads_first=heads_first, seed=page)
    pm.check_attention(c, *pu.run_attention(c))


@pytest.mark.parametrize("kv", [1, 15, 17, 31, 33, 47, 64, 131])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_chunks_of_one_and_two_pages(kv, d):
    c = Case([1, 2], [kv, 5], 4, 2, d, page=16, seed=kv)
    pm.check_attention(c, *pu.run_attention(c))


def test_rows_that_see_nothing():
    c = Case([1, 3, 5, 90, 40], [0, 2, 0, 60, 500], 8, 2, 128)
    pm.check_attention(c, *pu.run_attention(c))


def test_every_row_sees_the_whole_slice():
    c = Case([1, 3, 70, 2], [100, 1, 300, 0], 8, 2, 128, causal=False)
    pm.check_attention(c, *pu.run_attention(c))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("qscale", [2.0 ** -40, 30.0])
def test_flat_and_peaked_scores(qscale, d):
    c = Case([1, 5, 150], [2000, 300, 150], 8, 2, d, qscale=qscale)
    pm.check_attention(c, *pu.run_attention(c))


@pytest.mark.parametrize("new,kv", [([1, 2], [300, 90]), ([60], [200])])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("vmag", [(10, 13), (-13, 12), (-14, -12)])
def test_scales_of_any_size(vmag, d, new, kv):
    """V at both ends of the scales' range and over all of it; K's scales away from q's."""
    c = Case(new, kv, 4, 1, d, seed=d, vmag=vmag, kmag=(10, 12), qscale=2.0 ** -12)
    pm.check_attention(c, *pu.run_attention(c))


@pytest.mark.parametrize("new,kv", [([1, 2], [300, 90]), ([60], [200])])
def test_rows_of_q_of_any_size(new, kv):
    """Rows of q from 2^-100 to 2^60, each with its own power of two; keys to match."""
    c = Case(new, kv, 4, 1, 128, kmag=(0, 0))
    mag = torch.randint(-100, 3, c.q.shape[:2], generator=torch.Generator().manual_seed(1))
    c.q = (c.q.double() * 2.0 ** mag[..., None].double()).bfloat16()
    pm.check_attention(c, *pu.run_attention(c))
    c = Case(new, kv, 4, 1, 128, kmag=(-13, -13))
    c.q = (c.q.double() * 2.0 ** 14).bfloat16()
    pm.check_attention(c, *pu.run_attention(c))


def test_rows_past_the_last_sequence_are_left_alone():
    c = Case([1, 60], [40, 333], 8, 2, 128, pad_rows=5)
    out = torch.full((66, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((8, 66), 7.0, device="cuda")
    bd.bd_paged_attn(c.plan, c.q.cuda(), c.cache, out, lse)
    torch.cuda.synchronize()
    assert (out[61:] == 7).all() and (lse[:, 61:] == 7).all()
    pm.check_attention(c, out.cpu(), lse.cpu())


def test_one_pool_for_k_and_v():
    """K and V as slices of one pool [pages, 2, page, heads, d / 2], scales likewise, with room
    between the heads' scales."""
    c = Case([1, 60], [300, 90], 8, 2, 128, page=32)
    want = pu.run_attention(c)
    both = torch.stack([c.k, c.v], 1)
    wide = torch.full((c.num_pages, 2, 32, 2, 24), 255, dtype=torch.uint8, device="cuda")
    wide[..., 8:16] = torch.stack([c.ke, c.ve], 1)
    c.cache = bd.PagedCache(both[:, 0], both[:, 1], wide[:, 0, ..., 8:16], wide[:, 1, ..., 8:16])
    got = pu.run_attention(c)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("H,Hkv,d,new,kv", [(8, 2, 64, 4, 100), (8, 2, 128, 4, 100), (8, 2, 256, 4, 100), (8, 2, 128, 8, 70),
                                            (8, 2, 128, 3, 3000), (8, 2, 64, 150, 400), (8, 2, 128, 150, 400),
                                            (8, 2, 256, 150, 400), (2, 2, 128, 300, 300), (8, 2, 128, 70, 9001)])
def test_rows_take_nothing_from_keys_they_do_not_see(H, Hkv, d, new, kv):
    """Scales of NaN in cached rows of the step itself reach the new rows that see them, in
    their 16 columns, and no others; a K of NaN reaches those who see its key."""
    c = Case([new], [kv], H, Hkv, d, page=32, seed=new)
    first, G = kv - new, H // Hkv
    spots = sorted({max(0, first + new // 2), max(0, first + 1), kv - 1})
    bad = torch.zeros(new, d, dtype=torch.bool)  # of K/V head 0
    for n, pos in enumerate(spots):
        page, row, grp = c.pages[0][pos // 32], pos % 32, (n * 3) % (d // 16)
        c.ve[page, row, 0, grp] = 255
        c.vd[page, row, 0, 16 * grp:16 * grp + 16] = 0
        bad[max(0, pos - first):, 16 * grp:16 * grp + 16] = True
    out, lse = pu.run_attention(c)
    o, l, A, big = op.attention(c.q[:new], *c.rows(0), kv)
    to, tl = pm.tolerances(d, kv, A, big, "e2m1", new * G, c.vd[c.used].abs().max().item())
    hit = torch.zeros(new, H, d, dtype=torch.bool)
    hit[:, :G] = bad[:, None]
    assert torch.isnan(out[hit]).all() and torch.isfinite(out[~hit]).all()
    assert ((out.double() - o).abs() <= to)[~hit].all()
    assert ((lse.double() - l).abs() <= tl).all()
    page, row = c.pages[0][spots[1] // 32], spots[1] % 32
    c.ke[page, row, 0, 1] = 255
    out2, lse2 = pu.run_attention(c)
    rows = torch.zeros(new, dtype=torch.bool)
    rows[max(0, spots[1] - first):] = True
    assert torch.isnan(lse2[:G, rows]).all() and torch.isnan(out2[rows, :G]).all()
    assert torch.equal(lse2[:G, ~rows], lse[:G, ~rows]) and torch.equal(lse2[G:], lse[G:])
    assert torch.equal(out2[:, G:], out[:, G:])


def _mixed(seed=0):
    return Case([1, 1, 60, 200], [5000, 40, 700, 900], 8, 2, 128, page=32, seed=seed)


def test_same_bits_every_time_and_on_a_stream():
    c = _mixed()
    a, b = pu.run_attention(c), pu.run_attention(c, stream=torch.cuda.Stream())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    pm.check_attention(c, *a)


def test_captured_layers_replay():
    """Writes and attention of both kinds in one graph, replayed over other lengths."""
    H, Hkv, d, P, pages = 8, 2, 128, 32, [list(range(0, 300)), list(range(300, 600)), list(range(600, 700))]
    g = torch.Generator().manual_seed(5)
    codes = [torch.randint(0, 256, (700, P, Hkv, d // 2), generator=g).to(torch.uint8).cuda() for _ in range(2)]
    scales = [torch.randint(100, 130, (700, P, Hkv, d // 16), generator=g).to(torch.uint8).cuda() for _ in range(2)]
    cache = bd.PagedCache(*codes, *scales)
    steps = [([70, 1, 3], [9001, 8000, 900]), ([50, 3, 1], [7000, 9500, 3]), ([90, 1, 4], [9600, 6000, 1000])]
    plans = [bd.PagedPlan(n, kv, pages, H, Hkv, d, page_size=P, num_pages=700, fmt=cache.fmt) for n, kv in steps]
    assert len({p.key() for p in plans}) == 1
    buf = torch.zeros(max(p.nbytes for p in plans) // 4, dtype=torch.int32, device="cuda")
    ws = torch.empty(bd.bd_paged_attn_workspace(plans[0]), dtype=torch.uint8, device="cuda")
    q, kn, vn = (torch.randn(100, h, d, generator=g).bfloat16().cuda() for h in (H, Hkv, Hkv))
    out, lse = torch.zeros(100, H, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(H, 100, device="cuda")

    def step(plan):
        bd.bd_cache_write(plan, kn, vn, cache)
        bd.bd_paged_attn(plan, q, cache, out, lse, ws)

    want = []
    for p in plans + plans:
        out.fill_(7)
        lse.fill_(7)
        step(p.upload("cuda"))
        want.append((out.clone(), lse.clone()))
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
        assert torch.equal(out, want[3 + i][0]) and torch.equal(lse, want[3 + i][1])
        bd.bd_check_status(plans[i])
