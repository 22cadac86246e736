"""GPU parity of attention over selected blocks of a paged cache: bounds, lists and outputs,
through the C ABI, against the plain oracle."""
import pytest
import torch

from oracle import blocks as ob
from oracle import paged as op

pytestmark = pytest.mark.gpu

bd = pytest.importorskip("block_causal_varlen_gb300")
pm = pytest.importorskip("paged_more_util")

FORMATS = ["bf16", "e4m3", "e2m1"]
HEADS = [(4, 4, 64), (8, 2, 128), (4, 1, 256)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bd.load()


class Sparse:
    """A case with a sparse plan, and bounds of all its blocks."""

    def __init__(self, new, kv, H, Hkv, d, blocks, first=0, recent=1, **kw):
        self.c = c = pm.Case(new, kv, H, Hkv, d, **kw)
        self.blocks, self.first, self.recent = blocks, first, recent
        self.plan = c.make_plan(blocks=blocks, first=first, recent=recent).upload("cuda")
        self.bounds = bd.BlockBounds.empty(c.cache)
        whole = c.make_plan(q_len=c.kv).upload("cuda")     # every cached row counts as new
        bd.bd_block_bounds(whole, c.cache, self.bounds)
        torch.cuda.synchronize()

    def lists(self, q=None):
        out = torch.full((self.c.q.shape[0], self.c.Hkv, self.blocks), -7, dtype=torch.int32, device="cuda")
        bd.bd_block_select(self.plan, self.c.q.cuda() if q is None else q, self.bounds, out)
        torch.cuda.synchronize()
        return out

    def attend(self, lists):
        c = self.c
        out = torch.full(c.q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        lse = torch.full((c.H, c.q.shape[0]), float("nan"), device="cuda")
        ws = torch.full((max(1, bd.bd_paged_attn_workspace(self.plan)),), 255, dtype=torch.uint8, device="cuda")
        bd.bd_sparse_attn(self.plan, c.q.cuda(), c.cache, lists, out, lse, ws)
        torch.cuda.synchronize()
        bd.bd_check_status(self.plan)
        return out.cpu(), lse.cpu()

    def rows(self):
        """(packed row, sequence, position) of every new row."""
        t = 0
        for b, (n, kv) in enumerate(zip(self.c.new, self.c.kv)):
            for i in range(n):
                yield t, b, kv - n + i
                t += 1

    def want_lists(self):
        c = self.c
        out = torch.full((c.T, c.Hkv, self.blocks), -1, dtype=torch.int32)
        code, exp = self.bounds.code.cpu(), self.bounds.exp.cpu()
        G = c.H // c.Hkv
        for t, b, pos in self.rows():
            pages = c.pages[b][:max(0, pos // c.page + 1)] if pos >= 0 else []
            for g in range(c.Hkv):
                out[t, g] = torch.tensor(ob.select(c.q[t, g * G:(g + 1) * G], [code[p, g, 0] for p in pages],
                                                   [code[p, g, 1] for p in pages], [exp[p, g] for p in pages],
                                                   self.blocks, self.first, self.recent))
        return out

    def check_attention(self, lists, out, lse):
        c, G = self.c, self.c.H // self.c.Hkv
        cached = [c.rows(b) for b in range(len(c.kv))]
        for t, b, pos in self.rows():
            for g in range(c.Hkv):
                keys = [j * c.page + r for j in lists[t, g].tolist() if j >= 0 for r in range(c.page) if j * c.page + r <= pos]
                heads = slice(g * G, (g + 1) * G)
                k, v = (x[keys][:, g:g + 1] for x in cached[b])
                o, l, A, big = op.attention(c.q[t:t + 1, heads], k, v, len(keys))
                to, tl = pm.tolerances(c.d, max(1, len(keys)), A, big, c.fmt, min(G, 16), v.abs().max().item() if keys else 0.0)
                if c.fmt == "e4m3" and G > 16:   # paged_util counts by rows of the whole call: blocks are of 16
                    to = to + A * 2.0 ** -8
                pm.compare(out[t:t + 1, heads], lse[heads, t:t + 1], o, l, to, tl, (t, g, len(keys)))


# ------------------------------------------------------------------ bounds

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("H,Hkv,d", HEADS)
@pytest.mark.parametrize("page", [16, 64, 256])
def test_bounds(page, H, Hkv, d, fmt):
    """Blocks that new rows entered, and no others, from the rows below kv_len."""
    new, kv = [1, 40, 0, 3, 5], [page + 1, 40, 70, 2, 3 * page + 2]
    c = pm.Case(new, kv, H, Hkv, d, page=page, fmt=fmt, heads_first=page == 64, seed=d)
    b = bd.BlockBounds(torch.full((c.num_pages, Hkv, 2, d), 99, dtype=torch.int8, device="cuda"),
                       torch.full((c.num_pages, Hkv), 9, dtype=torch.uint8, device="cuda"))
    bd.bd_block_bounds(c.plan, c.cache, b)
    torch.cuda.synchronize()
    code, exp = b.code.cpu(), b.exp.cpu()
    left = set(range(c.num_pages))
    for s in range(len(kv)):
        K = c.rows(s)[0]
        for j in range(max(0, kv[s] - new[s]) // page, (kv[s] - 1) // page + 1 if new[s] else 0):
            p = c.pages[s][j]
            left.discard(p)
            for g in range(Hkv):
                lo, hi, e = ob.bounds(K[j * page:(j + 1) * page, g])
                assert exp[p, g] == e and torch.equal(code[p, g, 0], lo) and torch.equal(code[p, g, 1], hi), (s, j, g)
    for p in left:
        assert (code[p] == 99).all() and (exp[p] == 9).all()


def test_bounds_of_any_size():
    """Zeros, infinities and NaN, values past both ends of the exponents, maxima at a power's edge."""
    c = pm.Case([128], [128], 4, 1, 64, page=16, junk=0.0)
    k = c.k_new.clone()
    k[0:16] = 0
    k[17, 0, 5] = float("inf")
    k[33, 0, 60] = float("nan")
    k[48:64] *= 2.0 ** 60
    k[64:80] *= 2.0 ** -70
    k[80:96] = 127 * 2.0 ** 3
    k[96:112] = 128.0
    k[112:128] = -127.5
    bd.bd_cache_write(c.plan, k.cuda(), k.cuda(), c.cache)
    b = bd.BlockBounds.empty(c.cache)
    bd.bd_block_bounds(c.plan, c.cache, b)
    torch.cuda.synchronize()
    for j in range(8):
        p = c.pages[0][j]
        lo, hi, e = ob.bounds(k[16 * j:16 * j + 16, 0])
        assert b.exp[p, 0].item() == e and torch.equal(b.code[p, 0].cpu(), torch.stack([lo, hi])), j


# ------------------------------------------------------------------ lists

@pytest.mark.parametrize("H,Hkv,d", HEADS + [(10, 2, 128), (7, 1, 64), (128, 1, 64)])
@pytest.mark.parametrize("blocks,first,recent", [(4, 0, 1), (7, 1, 2), (3, 1, 2), (1, 0, 1), (33, 0, 1)])
def test_lists(blocks, first, recent, H, Hkv, d):
    s = Sparse([1, 3, 0, 20, 2], [300, 33, 40, 530, 1], H, Hkv, d, blocks, first, recent, seed=d + blocks)
    got = s.lists()
    assert torch.equal(got.cpu(), s.want_lists())


@pytest.mark.parametrize("fmt", FORMATS)
def test_lists_over_many_blocks(fmt):
    s = Sparse([2, 1], [9001, 40000], 8, 2, 128, 40, 1, 1, fmt=fmt, junk=0.0)
    assert torch.equal(s.lists().cpu(), s.want_lists())


def test_ties_go_to_the_lowest_block():
    """Blocks of equal bounds, all of them or by pairs; q of zeros scores all the same."""
    s = Sparse([2], [640], 4, 2, 64, 9, 0, 1)
    s.bounds.code[:] = s.bounds.code[s.c.pages[0][0]].clone()
    s.bounds.exp[:] = s.bounds.exp[s.c.pages[0][0]].clone()
    got = s.lists().cpu()
    assert torch.equal(got, s.want_lists()) and (got[1, 0] == torch.tensor(list(range(8)) + [39])).all()
    s = Sparse([2], [640], 4, 2, 64, 9, 0, 1)
    for j in range(0, 40, 2):
        s.bounds.code[s.c.pages[0][j + 1]] = s.bounds.code[s.c.pages[0][j]]
        s.bounds.exp[s.c.pages[0][j + 1]] = s.bounds.exp[s.c.pages[0][j]]
    assert torch.equal(s.lists().cpu(), s.want_lists())
    s.c.q[:] = 0
    assert torch.equal(s.lists().cpu(), s.want_lists())


def test_odd_blocks_and_rows():
    """A block with a NaN outscores the others; more of them than there is room for: the first ones, but
    never in place of those that are always listed; heads of q with an infinity or a NaN count as zeros;
    rows of q of any size."""
    s = Sparse([3], [640], 4, 2, 64, 6, 1, 2, junk=0.0)
    for j in (3, 17):
        s.bounds.exp[s.c.pages[0][j], 0] = 255
    got = s.lists().cpu()
    assert torch.equal(got, s.want_lists()) and all({0, 3, 17, 38, 39} <= set(r.tolist()) for r in got[:, 0])
    s.bounds.exp[:] = 255
    got = s.lists().cpu()
    assert (got == torch.tensor([0, 1, 2, 3, 38, 39])).all()
    s = Sparse([3], [640], 4, 2, 64, 6, 1, 2, junk=0.0)
    s.c.q[0, 0, 3], s.c.q[0, 2, 5], s.c.q[1, 1, 7] = float("inf"), float("nan"), float("-inf")
    s.c.q[2, 0] *= 2.0 ** 80
    s.c.q[2, 1] *= 2.0 ** -80
    s.c.q[2, 2] *= 2.0 ** -120
    assert torch.equal(s.lists().cpu(), s.want_lists())


def test_most_blocks():
    """A sequence of 16384 blocks, the most there may be."""
    P, n = 16, 16384 * 16
    c = bd.PagedCache(*(torch.randn(16384, P, 1, 64, generator=torch.Generator("cuda").manual_seed(i), device="cuda").bfloat16()
                        for i in range(2)))
    pages = [torch.randperm(16384, generator=torch.Generator().manual_seed(2)).numpy()]
    plan = bd.PagedPlan([1], [n], pages, 2, 1, 64, page_size=P, num_pages=16384, blocks=4096).upload("cuda")
    whole = bd.PagedPlan([n], [n], pages, 2, 1, 64, page_size=P, num_pages=16384).upload("cuda")
    b = bd.BlockBounds.empty(c)
    bd.bd_block_bounds(whole, c, b)
    q = torch.randn(1, 2, 64, generator=torch.Generator().manual_seed(3)).bfloat16()
    out, lse, lists = bd.sparse_attn(plan, q.cuda(), c, b)
    torch.cuda.synchronize()
    bd.bd_check_status(plan)
    lo, hi = (b.code[torch.from_numpy(pages[0]).cuda(), 0, i].cpu().double() for i in range(2))
    eb = b.exp[torch.from_numpy(pages[0]).cuda(), 0].cpu().double() - 127
    best = None
    for row in q[0].double():
        e = ob._power(row.abs().max().item())
        x = torch.round(row * 2.0 ** -e)
        s = torch.maximum(x * lo, x * hi).sum(1) * 2.0 ** (e + eb)
        best = s if best is None else torch.maximum(best, s)
    order = sorted(range(16383), key=lambda j: (-best[j].item(), j))[:4095]
    assert lists[0, 0].tolist() == sorted(order) + [16383]
    at = torch.from_numpy(pages[0])[lists[0, 0].long().cpu()].cuda()
    K, V = (t[at].flatten(0, 1).cpu() for t in (c.k, c.v))
    o, l, A, big = op.attention(q, K, V, len(K))
    to, tl = pm.tolerances(64, len(K), A, big, "bf16", 2, 0)
    pm.compare(out.cpu(), lse.cpu(), o, l, to, tl, "4096 blocks")


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("H,Hkv,d", HEADS + [(10, 2, 128), (40, 1, 128), (24, 1, 128)])
@pytest.mark.parametrize("page,blocks", [(16, 5), (64, 3)])
def test_attention(page, blocks, H, Hkv, d, fmt):
    s = Sparse([1, 3, 0, 20, 2], [300, 33, 40, 530, 1], H, Hkv, d, blocks, seed=d, page=page, fmt=fmt, heads_first=page == 64)
    lists = s.lists()
    s.check_attention(lists.cpu(), *s.attend(lists))


@pytest.mark.parametrize("fmt", FORMATS)
def test_long_lists_are_split_and_joined(fmt):
    s = Sparse([1], [9001], 8, 2, 128, 90, 1, 2, page=32, fmt=fmt)
    lists = s.lists()
    s.check_attention(lists.cpu(), *s.attend(lists))


@pytest.mark.parametrize("fmt", FORMATS)
def test_lists_of_everything_are_the_whole(fmt):
    """Lists that hold all blocks: as exact as the attention over the whole cache, in particular
    rows without a position give O = 0, LSE = -inf."""
    s = Sparse([1, 3, 5, 20], [300, 2, 0, 530], 8, 2, 128, 40, fmt=fmt)
    out, lse = s.attend(s.lists())
    pm.check_attention(s.c, out, lse)


def test_lists_of_any_numbers_read_no_other_sequence():
    """Entries outside of a row's blocks stand for the nearest block."""
    s = Sparse([1, 2], [300, 500], 8, 2, 128, 6)
    lists = s.lists()
    wild = lists.clone()
    wild[..., 0], wild[..., -1] = -2 ** 31, 2 ** 31 - 1
    near = lists.clone()
    near[..., 0] = 0
    for t, b, pos in s.rows():
        near[t, :, -1] = pos // 16
    a, b = s.attend(wild), s.attend(near)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_rows_past_the_last_sequence_are_left_alone():
    s = Sparse([1, 4], [300, 500], 8, 2, 128, 6, pad_rows=3)
    lists = s.lists()
    assert (lists[5:] == -7).all()
    out, lse = s.attend(lists)
    assert torch.isnan(out[5:]).all() and torch.isnan(lse[:, 5:]).all()
    s.check_attention(lists.cpu(), out, lse)


def test_strided_lists_and_bounds():
    s = Sparse([1, 4], [300, 500], 8, 2, 128, 6)
    want = s.lists()
    wide = torch.zeros(2, 9, 10, dtype=torch.int32, device="cuda")
    view = wide[:, 1:6, 2:8].transpose(0, 1)
    code = torch.zeros(2, 3, s.c.num_pages, 160, dtype=torch.int8, device="cuda")[:, :2, :, 16:144].permute(2, 0, 1, 3)
    exp = torch.zeros(2, s.c.num_pages, dtype=torch.uint8, device="cuda").t()
    code.copy_(s.bounds.code)
    exp.copy_(s.bounds.exp)
    bd.bd_block_select(s.plan, s.c.q.cuda(), bd.BlockBounds(code, exp), view)
    torch.cuda.synchronize()
    assert torch.equal(view, want) and (wide[:, 0] == 0).all() and (wide[:, 6:] == 0).all() and (wide[..., 8:] == 0).all()
    a, b = s.attend(want), s.attend(view)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("fmt", FORMATS)
def test_nan_in_unlisted_blocks_stays_there(fmt):
    """What no row's list names may hold anything."""
    s = Sparse([2], [640], 8, 2, 128, 5, fmt=fmt, junk=0.0)
    lists = s.lists()
    want = s.attend(lists)
    used = {j for r in lists.cpu().flatten().tolist() for j in [r]}
    for j in set(range(40)) - used:
        p = s.c.pages[0][j]
        for t in (s.c.k, s.c.v, s.c.ke, s.c.ve):
            if t is not None:
                t.view(torch.uint8)[p] = 255
    got = s.attend(lists)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_same_bits_every_time_and_on_streams():
    s = Sparse([1, 1, 30], [9000, 500, 3000], 8, 2, 128, 20, 1, 2, page=32)
    lists = s.lists()
    want = s.attend(lists)
    q = s.c.q.cuda()
    torch.cuda.synchronize()
    for _ in range(3):
        st = torch.cuda.Stream()
        out, lse, got = bd.sparse_attn(s.plan, q, s.c.cache, s.bounds, stream=st)
        torch.cuda.current_stream().wait_stream(st)
        assert torch.equal(got, lists) and torch.equal(out.cpu(), want[0]) and torch.equal(lse.cpu(), want[1])


@pytest.mark.parametrize("fmt", FORMATS)
def test_captured_steps_replay(fmt):
    """Append, bounds, selection and attention of a decode step in one graph, replayed over three
    steps: the bits of eager calls with a synchronisation after each."""
    H, Hkv, d, P, f = 8, 2, 128, 16, torch.rand(64, generator=torch.Generator().manual_seed(0))
    kv0, pages = [5000, 250, 30], [list(range(320)), list(range(320, 340)), list(range(340, 345))]
    c = pm.Case([0], [345 * P], H, Hkv, d, fmt=fmt, junk=0.0)
    rope = bd.Rope(f, device="cuda")

    def plan_of(i):
        return bd.PagedPlan([1, 1, 1], [n + i for n in kv0], pages, H, Hkv, d, page_size=P, num_pages=c.num_pages, fmt=c.cache.fmt,
                            blocks=12, first=1, recent=2)

    start = [t.clone() if t is not None else None for t in (c.k, c.v, c.ke, c.ve)]
    bounds = bd.BlockBounds.empty(c.cache)
    all_ = bd.PagedPlan(kv0, kv0, pages, H, Hkv, d, page_size=P, num_pages=c.num_pages, fmt=c.cache.fmt).upload("cuda")
    bd.bd_block_bounds(all_, c.cache, bounds)
    b0 = (bounds.code.clone(), bounds.exp.clone())
    g = torch.Generator().manual_seed(2)
    rows = [[torch.randn(3, h, d, generator=g).bfloat16().cuda() for h in (H, Hkv, Hkv)] for _ in range(3)]
    q, k, v = (t.clone() for t in rows[0])
    out, lse = torch.zeros_like(q), torch.zeros(H, 3, device="cuda")
    lists = torch.zeros(3, Hkv, 12, dtype=torch.int32, device="cuda")
    plan = plan_of(1)
    ws = torch.empty(bd.bd_paged_attn_workspace(plan), dtype=torch.uint8, device="cuda")

    def calls(p, sync=lambda: None):
        for op_ in (lambda: bd.bd_cache_append(p, q, k, v, rope, c.cache, q), lambda: bd.bd_block_bounds(p, c.cache, bounds),
                    lambda: bd.bd_block_select(p, q, bounds, lists), lambda: bd.bd_sparse_attn(p, q, c.cache, lists, out, lse, ws)):
            op_()
            sync()

    def reset():
        for t, t0 in zip((c.k, c.v, c.ke, c.ve), start):
            if t is not None:
                t.view(torch.uint8).copy_(t0.view(torch.uint8))
        bounds.code.copy_(b0[0])
        bounds.exp.copy_(b0[1])

    def feed(i):
        for t, x in zip((q, k, v), rows[i]):
            t.copy_(x)

    want = []
    for i in range(3):
        feed(i)
        calls(plan_of(1 + i).upload("cuda"), torch.cuda.synchronize)
        want.append([t.clone() for t in (q, out, lse, lists, bounds.code, bounds.exp)])
    reset()
    buf = torch.zeros(plan.nbytes // 4 + 4096, dtype=torch.int32, device="cuda")
    plan.upload(buffer=buf)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(plan)
    reset()
    for i in range(3):
        nxt = plan_of(1 + i)
        assert nxt.key() == plan.key()
        nxt.upload(buffer=buf)
        feed(i)
        graph.replay()
        torch.cuda.synchronize()
        bd.bd_check_status(nxt)
        assert all(torch.equal(a, b) for a, b in zip((q, out, lse, lists, bounds.code, bounds.exp), want[i])), i


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 300])
def test_scores_of_the_largest_codes_are_exact(new, d):
    """Codes of +-127 throughout but for single ones: sums that differ by one, the largest there are."""
    s = Sparse([new], [700], 4, 1, d, 5, 0, 1, junk=0.0)
    s.c.q[:] = 127.0
    s.c.q[:, 1:] = -127.0
    g = torch.Generator().manual_seed(0)
    code = torch.full((s.c.num_pages, 1, 2, d), 127, dtype=torch.int8)
    code[:, :, 0] = -127
    for p in range(s.c.num_pages):
        code[p, 0, :, int(torch.randint(0, d, (1,), generator=g))] -= torch.tensor([-(p % 3), p % 5], dtype=torch.int8)
    s.bounds.code.copy_(code)
    s.bounds.exp[:] = 127
    assert torch.equal(s.lists().cpu(), s.want_lists())


def test_bounds_of_values_far_below_the_largest():
    """floor and ceil of what 2^-e takes below the least float: -1 and 1, not 0."""
    c = pm.Case([32], [32], 4, 1, 64, page=16, junk=0.0)
    k = c.k_new.clone()
    k[:, 0, 0] = 2.0 ** 60
    k[:16, 0, 1], k[:16, 0, 2], k[:16, 0, 3] = -2.0 ** -120, 2.0 ** -120, 2.0 ** -133
    k[16:, 0, 1], k[16:, 0, 2], k[16:, 0, 3] = -2.0 ** -133, -0.0, 0.0
    bd.bd_cache_write(c.plan, k.cuda(), k.cuda(), c.cache)
    b = bd.BlockBounds.empty(c.cache)
    bd.bd_block_bounds(c.plan, c.cache, b)
    torch.cuda.synchronize()
    for j in range(2):
        p = c.pages[0][j]
        lo, hi, e = ob.bounds(k[16 * j:16 * j + 16, 0])
        assert b.exp[p, 0].item() == e and torch.equal(b.code[p, 0].cpu(), torch.stack([lo, hi])), j


def test_captured_bounds_replay_over_pages_of_two_sequences():
    """A step whose two sequences enter one page, under a graph captured with one whose do not: the
    page's bounds are of the most rows of it that are used."""
    c = pm.Case([64], [64], 4, 2, 64, page=16, junk=0.0)
    p = c.pages[0]

    def step(kv, pages):
        return bd.PagedPlan([1, 1], kv, pages, 4, 2, 64, page_size=16, num_pages=c.num_pages)

    b = bd.BlockBounds.empty(c.cache)
    plan = step([20, 24], [[p[0], p[1]], [p[2], p[3]]])
    buf = torch.zeros(plan.nbytes // 4, dtype=torch.int32, device="cuda")
    plan.upload(buffer=buf)
    bd.bd_block_bounds(plan, c.cache, b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bd.bd_block_bounds(plan, c.cache, b)
    K = c.rows(0)[0]
    for kv in ([20, 24], [24, 20], [31, 32]):
        nxt = step(kv, [[p[0], p[1]], [p[2], p[1]]])
        assert nxt.key() == plan.key()
        nxt.upload(buffer=buf)
        b.code.fill_(99)
        b.exp.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        for g in range(2):
            lo, hi, e = ob.bounds(K[16:max(kv), g])
            assert b.exp[p[1], g] == e and torch.equal(b.code[p[1], g].cpu(), torch.stack([lo, hi])), (kv, g)
        assert all((b.code[x] == 99).all() and (b.exp[x] == 9).all() for x in (p[0], p[2], p[3]))


def test_blocks_without_bounds_are_listed():
    """Bounds that nobody made: such a block is listed before all whose bounds are known."""
    s = Sparse([2], [640], 4, 2, 64, 6, 1, 2, junk=0.0)
    fresh = bd.BlockBounds.empty(s.c.cache)
    known = [p for j, p in enumerate(s.c.pages[0]) if j not in (7, 31)]
    fresh.code[known], fresh.exp[known] = s.bounds.code[known], s.bounds.exp[known]
    s.bounds = fresh
    got = s.lists().cpu()
    assert torch.equal(got, s.want_lists()) and all({0, 7, 31, 38, 39} <= set(r.tolist()) for r in got.flatten(0, 1))


@pytest.mark.parametrize("size", [-80, 0, 80])
def test_any_byte_is_a_number(size):
    """Bytes that bd_block_bounds does not write count as the nearest that it does, whatever q."""
    s = Sparse([3], [1200], 4, 2, 64, 9, 0, 1, junk=0.0)
    s.c.q *= 2.0 ** size
    g = torch.Generator().manual_seed(1)
    exp = torch.randint(0, 255, s.bounds.exp.shape, generator=g).to(torch.uint8)
    s.bounds.exp.copy_(exp)
    s.bounds.code[::3] = 0
    got = s.lists().cpu()
    s.bounds.exp.copy_(exp.clamp(77, 177))
    assert torch.equal(got, s.want_lists())
