"""GPU parity of attention over e4m3 caches whose V rows differ in size as far as the format
goes, and of few-rows blocks of 17 to 48 pairs under the bound of their own rounding."""
import math

import pytest
import torch

from oracle import paged as op

pytestmark = pytest.mark.gpu

bd = pytest.importorskip("block_causal_varlen_gb300")
pu = pytest.importorskip("paged_util")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bd.load()


def check(case, out, lse, span=0, zeros=False):
    """Against the oracle under pu.tolerances, where P is fp16 for all sequences that the
    few-rows kernel takes (up to 48 pairs of a K/V head). span: V's exponents reach as far from
    zero; the running maximum includes them there, so a score's distance from it and the
    sum's logarithm reach span + 8 + 24 (a margin of 2^8, 2^24 keys): their roundings and the
    logarithm's error relative to itself are within 2^-22 of that each (2^-24 for the
    roundings; 2^-22 is the approximate logarithm's bound), as is that of their sum. zeros: V has
    zero rows, which count as codes of exponent -60: a weight is within 2^-32 of theirs, 2^-60 at
    most, times a code of at most 448 for each key."""
    at = 0
    for b, (n, kv) in enumerate(zip(case.new, case.kv)):
        k, v = case.rows(b)
        o_ref, l_ref, A, big = op.attention(case.q[at:at + n], k, v, kv, case.causal)
        pairs = n * case.H // case.Hkv
        tol_o, tol_l = pu.tolerances(case.d, max(kv, 1), A, big, case.fmt, 1 if pairs <= 48 else pairs)
        if span:
            more = 3 * 2.0 ** -22 * (span + 32)
            tol_l, tol_o = tol_l + more, tol_o + A * 2 * more
        if zeros:
            tol_o = tol_o + kv * 448 * 2.0 ** -92
        got, gl = out[at:at + n].double(), lse[:, at:at + n].double()
        assert torch.isfinite(got).all() and torch.isfinite(gl).all()
        bad = (gl - l_ref).abs() > tol_l
        assert not bad.any(), (b, n, kv, "LSE", gl[bad][:3].tolist(), l_ref[bad][:3].tolist())
        bad = (got - o_ref).abs() > tol_o
        assert not bad.any(), (b, n, kv, "O", got[bad][:3].tolist(), o_ref[bad][:3].tolist())
        at += n


def spread(new, kv, d, score, e, large, codes=None):
    """Every row scores `score` with all keys but those at `large`, which score 0 and whose V is
    448 2^e (a random sign in each column); the other rows of V are zeros, of exponent -60 as
    bd_cache_write has it."""
    c = pu.Case(new, kv, 4, 1, d, page=32, fmt="e4m3", junk=0.0)
    c.q = torch.zeros_like(c.q)
    c.q[..., 0] = math.sqrt(d)
    k, v = torch.zeros(c.kd.shape, dtype=torch.float64), torch.zeros(c.kd.shape, dtype=torch.float64)
    k[..., 0] = score
    sign = torch.randint(0, 2, v.shape, generator=torch.Generator().manual_seed(d)).double() * 2 - 1
    for n, pg in zip(kv, c.pages):
        for at in large:
            at = min(n - 1, int(at * n))
            k[pg[at // 32], at % 32] = 0
            v[pg[at // 32], at % 32] = 448.0 * 2.0 ** e * sign[pg[at // 32], at % 32]
    (kc, ke), (vc, ve) = op.quantise(k), op.quantise(v)
    c.kd, c.vd = op.dequantise(kc, ke), op.dequantise(vc, ve)
    c.k, c.v = kc.cuda().view(torch.float8_e4m3fn), vc.cuda().view(torch.float8_e4m3fn)
    c.ke, c.ve = ke.cuda(), ve.cuda()
    c.cache = bd.PagedCache(c.k, c.v, c.ke, c.ve)
    return c


# one piece; joins by warps (two to four parts), by CTAs (many); three blocks; tiles whole and split
SHAPES = [([1], [100]), ([1] * 100, [1000] * 100), ([1], [4096]), ([12], [700]), ([12], [9000]), ([15], [300]), ([15], [9000])]


@pytest.mark.parametrize("new,kv", SHAPES)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("large", [(0.0,), (0.5,), (1.0,), (0.1, 0.9)])
def test_large_rows_beside_zeros(large, d, new, kv):
    c = spread(new, kv, d, -5.5, 60, [1 - max(new) / min(kv) if x == 1.0 else x for x in large])
    check(c, *pu.run_attention(c), span=60)


@pytest.mark.parametrize("new", [1, 15])
@pytest.mark.parametrize("e,score", [(50, -12.0), (60, 1.75), (20, -9.0), (-20, -3.0)])
def test_large_rows_in_a_long_context(e, score, new):
    c = spread([new], [65536], 128, score, e, [0.6])
    check(c, *pu.run_attention(c), span=60)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new,kv", [([1], [21]), ([3, 12], [400, 3000])])
@pytest.mark.parametrize("vmag", [(-40, -30), (-7, 15), (30, 58)])
def test_most_rows_zeros(vmag, new, kv, d):
    """Peaked scores that mostly fall on zero rows of V, as bd_cache_write stores them."""
    c = pu.Case(new, kv, 8, 2, d, page=32, fmt="e4m3", seed=d, vmag=vmag, kmag=(-3, 1), qscale=8.0)
    codes, ve = c.v.view(torch.uint8).cpu(), c.ve.cpu()
    zero = (torch.rand(ve.shape, generator=torch.Generator().manual_seed(d)) < 0.9) & c.used[..., None]
    codes[zero], ve[zero] = 0, 67
    c.v.view(torch.uint8).copy_(codes.cuda())
    c.ve.copy_(ve.cuda())
    c.vd = op.dequantise(codes, ve)
    check(c, *pu.run_attention(c), span=60, zeros=True)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new,kv", [([5], [40]), ([6, 8], [9, 600]), ([9, 12], [20, 3000]), ([11], [12001])])
def test_few_rows_of_17_to_48_pairs(new, kv, d):
    """Within the bound of a P in fp16."""
    c = pu.Case(new, kv, 8, 2, d, page=32, fmt="e4m3", seed=d + len(new))
    check(c, *pu.run_attention(c))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new,kv", [([1], [200]), ([2, 12], [3000, 400])])
@pytest.mark.parametrize("gap", [3, 12, 24])
def test_zeros_of_a_high_byte(gap, new, kv, d):
    """A cache filled by other means: every third row of V is zeros with an exponent `gap` above
    the largest other one's. Weights are then good to 2^-32 of the largest p 2^e, that of such a
    row or not, times a code of at most 448 each."""
    c = pu.Case(new, kv, 4, 1, d, page=32, fmt="e4m3", seed=gap, vmag=(-2, 2))
    codes, ve = c.v.view(torch.uint8).cpu(), c.ve.cpu()
    top = int(ve[c.used].max())
    zero = torch.zeros(c.num_pages, 32, dtype=torch.bool)
    zero[:, ::3] = True
    zero &= c.used
    codes[zero], ve[zero] = 0, top + gap
    c.v.view(torch.uint8).copy_(codes.cuda())
    c.ve.copy_(ve.cuda())
    c.vd = op.dequantise(codes, ve)
    out, lse = pu.run_attention(c)
    at = 0
    for b, (n, m) in enumerate(zip(c.new, c.kv)):
        k, v = c.rows(b)
        e = op.rows_of(ve, m, c.pages[b], 32)[:, 0].double() - 127
        o_ref, l_ref, A, big = op.attention(c.q[at:at + n], k, v, m)
        tol_o, tol_l = pu.tolerances(d, m, A, big, "e4m3", 1)
        # p of every (row, head, key), and the largest weight of a row
        s = torch.einsum("ihd,jd->ihj", c.q[at:at + n].double(), k[:, 0]) / math.sqrt(d)
        s = s.masked_fill((torch.arange(m) > m - n + torch.arange(n)[:, None])[:, None], -math.inf)
        w = (torch.softmax(s, -1) * 2.0 ** e).amax(-1)
        more = 3 * 2.0 ** -22 * (40 + 32)        # as in check(): exponents up to 40 from zero
        tol_o = tol_o + A * 2 * more + m * 448 * 2.0 ** -32 * w[..., None]
        tol_l = tol_l + more
        assert ((out[at:at + n].double() - o_ref).abs() <= tol_o).all()
        assert ((lse[:, at:at + n].double() - l_ref).abs() <= tol_l).all()
        at += n
