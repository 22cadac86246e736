"""GPU parity of appends of so many rows that a group of lanes takes several heads: every
format and pairing, against the float64 oracle, a write of the turned K, and appends of few rows."""
import numpy as np
import pytest
import torch

from oracle import rope as orope

pytestmark = pytest.mark.gpu

bd = pytest.importorskip("block_causal_varlen_gb300")
FORMATS = {"bf16": bd.BD_CACHE_BF16, "e4m3": bd.BD_CACHE_E4M3, "e2m1": bd.BD_CACHE_E2M1}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bd.load()


def heads_of_a_group(T, H, Hkv, d):
    """As csrc/cache_append.cu counts them."""
    return min(16, max(1, T * (H + 2 * Hkv) * (d // 8) // (152 * 2048)))


def pool(fmt, n, P, Hkv, d):
    """A pool of bytes that no append writes, head-first."""
    def part(width, dtype):
        return torch.full((n, Hkv, P, width), 77, dtype=torch.uint8, device="cuda").view(dtype).transpose(1, 2)

    if fmt == "bf16":
        return bd.PagedCache(*(part(2 * d, torch.bfloat16) for _ in range(2)))
    if fmt == "e4m3":
        return bd.PagedCache(*(part(d, torch.float8_e4m3fn) for _ in range(2)), *(part(1, torch.uint8)[..., 0] for _ in range(2)))
    return bd.PagedCache(*(part(d // 2, torch.uint8) for _ in range(2)), *(part(d // 16, torch.uint8) for _ in range(2)))


def same(a, b):
    return all(x is None or torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))
               for x, y in ((a.k, b.k), (a.v, b.v), (a.k_exp, b.k_exp), (a.v_exp, b.v_exp)))


def check_turned(got, x, pos, f, interleaved):
    """Half a step of bf16 (2^-8 relative) and 2^-21 of the pair's length, as the header states it."""
    want = orope.turn(x, pos, f, interleaved)
    tol = want.abs() * 2.0 ** -8 + orope.lengths(x, f, interleaved) * 2.0 ** -21 + 1e-38
    assert not ((got.double() - want).abs() > tol).any()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("H,Hkv,d,r,T,per", [(20, 5, 128, 128, 2301, 3), (40, 20, 128, 96, 4005, 16), (9, 3, 64, 64, 6501, 2),
                                             (10, 2, 256, 256, 3617, 5), (33, 11, 64, 16, 7011, 9)])
def test_groups_of_several_heads(T, per, H, Hkv, d, r, interleaved, fmt):
    assert heads_of_a_group(T, H, Hkv, d) == per
    P = 64
    new, kv = [T - 1000, 0, 990, 10], [T - 1000 + 37, 20, 990, 4]          # the last rows: some without a position
    cut = np.cumsum([0] + [-(-n // P) for n in kv])
    n = int(cut[-1]) + 1
    order = np.random.default_rng(d).permutation(n)
    pages = [order[cut[b]:cut[b + 1]] for b in range(4)]

    def plan(heads, new=new, kv=kv, pages=pages):
        return bd.PagedPlan(new, kv, pages, heads, Hkv, d, page_size=P, num_pages=n, fmt=FORMATS[fmt]).upload("cuda")

    g = torch.Generator(device="cuda").manual_seed(r)
    big = torch.randn(T + 2, (H + 2 * Hkv) * d, generator=g, device="cuda").bfloat16()
    q, k, v = (big[:, a * d:b * d].view(T + 2, b - a, d) for a, b in ((0, H), (H, H + Hkv), (H + Hkv, H + 2 * Hkv)))
    f = (1.0 / 10000.0 ** (torch.arange(0, r, 2, dtype=torch.float64) / r)).float()
    rope = bd.Rope(f, interleaved=interleaved, device="cuda")
    many, few, written = (pool(fmt, n, P, Hkv, d) for _ in range(3))
    out = torch.full((T + 2, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    bd.bd_cache_append(plan(H), q, k, v, rope, many, out)
    assert (out[T:] == 7).all()
    # a few rows at a time: groups of one head
    part, step = torch.full_like(out, 7.0), 61
    at = 0
    for b in range(4):
        for i in range(0, new[b], step):
            m, end = min(step, new[b] - i), kv[b] - new[b] + min(i + step, new[b])
            if end >= 0:
                assert heads_of_a_group(m, H, Hkv, d) == 1
                rows = slice(at + i, at + i + m)
                bd.bd_cache_append(plan(H, [m], [end], [pages[b]]), q[rows], k[rows], v[rows], rope, few, part[rows])
        at += new[b]
    assert torch.equal(out, part) and same(many, few)
    # a write of K turned as q of a call
    kt = torch.empty(T + 2, Hkv, d, dtype=torch.bfloat16, device="cuda")
    bd.bd_cache_append(plan(Hkv), k, k, v, rope, few, kt)
    bd.bd_cache_write(plan(H), kt, v, written)
    torch.cuda.synchronize()
    assert same(many, written)
    pos = [e - m + i for m, e in zip(new, kv) for i in range(m)]
    some = [0, 1, 5, 777, T - 1001, T - 1000, T - 11, T - 10, T - 5, T - 4, T - 1]
    for got, x in ((out, q), (kt, k)):
        check_turned(got[some].cpu(), x[some].cpu(), [pos[i] for i in some], f, interleaved)
    stays = [i for i in some if pos[i] < 0]
    assert stays and torch.equal(out[stays], q[stays])


@pytest.mark.parametrize("fmt", FORMATS)
def test_groups_of_several_heads_in_place(fmt):
    """q turned where it stands."""
    T, H, Hkv, d, P = 2301, 20, 5, 128, 64
    plan = bd.PagedPlan([T], [T], [list(range(36))], H, Hkv, d, page_size=P, num_pages=36, fmt=FORMATS[fmt]).upload("cuda")
    g = torch.Generator(device="cuda").manual_seed(0)
    q, k, v = (torch.randn(T, h, d, generator=g, device="cuda").bfloat16() for h in (H, Hkv, Hkv))
    rope = bd.Rope(torch.rand(64, generator=torch.Generator().manual_seed(0)), device="cuda")
    a, b, out = pool(fmt, 36, P, Hkv, d), pool(fmt, 36, P, Hkv, d), torch.empty_like(q)
    bd.bd_cache_append(plan, q, k, v, rope, a, out)
    bd.bd_cache_append(plan, q, k, v, rope, b, q)
    torch.cuda.synchronize()
    assert torch.equal(q, out) and same(a, b)
