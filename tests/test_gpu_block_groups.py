"""GPU lists of block selection where several new rows of a sequence select together, where CTAs
take more than one group, and where clusters do, against a plain oracle (whole numbers: equal)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

bd = pytest.importorskip("block_causal_varlen_gb300")
# header words of a sparse plan (csrc/paged_plan.h)
SEL_ROWS, NSELG, SEL_SPLIT = 40, 42, 43
CTAS = 152 * 8      # the most that a launch has


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bd.load()


class Lists:
    """Random bounds of random pages, and q: selection reads no cache."""

    def __init__(self, new, kv, H, Hkv, d, blocks, first=0, recent=1, page=16, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.new, self.kv, self.H, self.Hkv, self.d, self.page = new, kv, H, Hkv, d, page
        self.blocks, self.first, self.recent = blocks, first, recent
        cut = np.cumsum([0] + [-(-n // page) for n in kv])
        n = int(cut[-1]) + 1
        order = np.random.default_rng(seed).permutation(n)
        self.pages = [order[cut[b]:cut[b + 1]] for b in range(len(kv))]
        self.plan = bd.PagedPlan(new, kv, self.pages, H, Hkv, d, page_size=page, num_pages=n, blocks=blocks, first=first,
                                 recent=recent).upload("cuda")
        self.code = torch.randint(-127, 128, (n, Hkv, 2, d), generator=g).sort(2)[0].to(torch.int8)
        self.exp = torch.randint(117, 122, (n, Hkv), generator=g).to(torch.uint8)
        twin = torch.randint(0, n, (n,), generator=g)       # blocks of equal bounds, and odd ones
        some = torch.rand(n, generator=g) < 0.3
        self.code[some], self.exp[some] = self.code[twin[some]], self.exp[twin[some]]
        self.exp[torch.rand(n, Hkv, generator=g) < 0.02] = 255
        self.q = torch.randn(sum(new) + 2, H, d, generator=g).bfloat16()
        self.q[::7, 0] = 0
        self.q[3::11, -1, 5] = float("nan")
        self.q[2::5] *= 2.0 ** 70
        self.bounds = bd.BlockBounds(self.code.cuda(), self.exp.cuda())

    def run(self, plan=None, out=None):
        if out is None:
            out = torch.full((self.q.shape[0], self.Hkv, self.blocks), -7, dtype=torch.int32, device="cuda")
        bd.bd_block_select(plan or self.plan, self.q.cuda(), self.bounds, out)
        torch.cuda.synchronize()
        return out

    def want(self):
        """The definition, row by row in 64 bits; rows past the last sequence are left alone."""
        H, Hkv, P = self.H, self.Hkv, self.page
        G = H // Hkv
        out = torch.full((self.q.shape[0], Hkv, self.blocks), -7, dtype=torch.int32)
        q = self.q.cuda().double()
        ok = torch.isfinite(q).all(-1)
        # (powers on the device are off by a rounding, which a tie does not forgive)
        two = torch.tensor([2.0 ** i for i in range(-300, 301)], dtype=torch.float64, device="cuda")
        q = torch.where(ok[..., None], q, torch.zeros_like(q))
        top = q.abs().amax(-1)
        e = torch.full_like(top, -50)
        for i in range(-50, 50):
            e = torch.where(top > 127 * 2.0 ** i, i + 1, e)
        c = torch.round(q * two[(300 - e).long()][..., None]).clamp(-127, 127).unflatten(1, (Hkv, G))
        e = e.unflatten(1, (Hkv, G))
        end = 0
        for n, kv, pages in zip(self.new, self.kv, self.pages):
            at = torch.from_numpy(np.asarray(pages, dtype=np.int64))
            lo, hi = (self.code[at, :, i].cuda().double().transpose(0, 1) for i in range(2))       # [Hkv, blocks, d]
            eb = self.exp[at].cuda().double().t()
            end += n
            for t in range(end - n, end):
                nblk = max(0, (kv - end + t) // P + 1)      # its position is kv - end + t
                if nblk <= self.blocks:
                    out[t] = torch.tensor(list(range(nblk)) + [-1] * (self.blocks - nblk))
                    continue
                x = c[t][:, :, None]                                                              # [Hkv, G, 1, d]
                s = torch.maximum(x * lo[:, None, :nblk], x * hi[:, None, :nblk]).sum(-1)
                s = (s * two[(e[t][..., None] + eb[:, None, :nblk] + 173).long()]).amax(1)
                s[eb[:, :nblk] == 255] = 1e300
                s[:, :self.first] = s[:, nblk - self.recent:] = float("inf")
                best = torch.sort(s, dim=1, descending=True, stable=True)[1][:, :self.blocks]
                out[t] = best.sort(1)[0].int().cpu()
        return out


@pytest.mark.parametrize("H,Hkv,d,rows", [(32, 8, 128, 8), (8, 8, 64, 8), (40, 8, 64, 8), (20, 4, 256, 4), (24, 8, 128, 8),
                                          (4, 4, 128, 4), (4, 2, 128, 2), (64, 8, 256, 4)])
@pytest.mark.parametrize("blocks,first,recent", [(9, 1, 2), (3, 1, 2), (40, 0, 1)])
def test_rows_that_select_together(blocks, first, recent, H, Hkv, d, rows):
    """Groups that end with their sequence, rows without a position or with fewer blocks than a list
    holds in a group with others, heads that do not fill the columns."""
    s = Lists([301, 37, 1, 0, 26, 19], [900, 500, 333, 50, 12, 700], H, Hkv, d, blocks, first, recent, seed=d + H)
    assert s.plan.host[SEL_ROWS] == rows
    assert torch.equal(s.run().cpu(), s.want())


@pytest.mark.parametrize("blocks", [5, 60])
def test_a_cta_takes_one_group_after_another(blocks):
    """More groups and heads than CTAs: rows of 400 sequences."""
    s = Lists([1 + (i % 3 == 0) for i in range(400)], [20 + 7 * (i % 120) for i in range(400)], 8, 4, 128, blocks)
    assert s.plan.host[SEL_ROWS] == 8 and s.plan.host[NSELG] * 4 > CTAS
    assert torch.equal(s.run().cpu(), s.want())


def test_a_cta_takes_one_row_after_another():
    """Rows of so many blocks that each selects by itself, more of them than CTAs."""
    s = Lists([160], [66000], 8, 8, 64, 33, 1, 2)
    assert s.plan.host[SEL_ROWS] == 1 and s.plan.host[SEL_SPLIT] == 1 and s.plan.host[NSELG] * 8 > CTAS
    assert torch.equal(s.run().cpu(), s.want())


def test_captured_clusters_replay_over_more_rows():
    """Captured with one row, replayed with 19: each cluster takes several."""
    s = Lists([1] * 19, [9000 + 40 * i for i in range(18)] + [30], 8, 2, 128, 12, 1, 2)
    pool = s.plan.num_pages
    plan = bd.PagedPlan([1], [9000], [s.pages[0]], 8, 2, 128, page_size=16, num_pages=pool, blocks=12, first=1, recent=2)
    assert plan.host[SEL_SPLIT] == 4 and plan.key() == s.plan.key()
    buf = torch.zeros(s.plan.nbytes // 4, dtype=torch.int32, device="cuda")
    plan.upload(buffer=buf)
    q, out = s.q.cuda(), torch.full((21, 2, 12), -7, dtype=torch.int32, device="cuda")
    bd.bd_block_select(plan, q, s.bounds, out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bd.bd_block_select(plan, q, s.bounds, out)
    s.plan.upload(buffer=buf)
    out.fill_(-7)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), s.want())
