"""Host side of 4-bit caches, rotated appends and selected blocks (CPU): validation, what sparse
plans hold, rotation phases against exact arithmetic, the binding's refusals, and the kernels'
place behind the grids in front of them."""
import ctypes
import os
import re
from fractions import Fraction

import numpy as np
import pytest
import torch

bd = pytest.importorskip("block_causal_varlen_gb300")
from block_causal_varlen_gb300 import _abi  # noqa: E402
from oracle import blocks as ob  # noqa: E402
from oracle import paged_e2m1 as o4  # noqa: E402
from oracle import rope as orope  # noqa: E402

by = ctypes.byref
DEV = ctypes.c_void_p(4096)     # never read: every refusal below comes before a launch
# header words behind those of test_paged_plan (csrc/paged_plan.h)
POS, TOUCH, NTOUCH, BOUNDS_OK, BLOCKS, FIRST, RECENT, ROWPG, SEL_CAP, SEL_ROWS, SELG, NSELG, SEL_SPLIT = range(31, 44)
OFF_PAGES, DEC, NDEC = 18, 22, 23


def make(new, kv, H=8, Hkv=2, d=128, page=16, fmt=bd.BD_CACHE_E2M1, **kw):
    cut = np.cumsum([0] + [-(-n // page) for n in kv])
    pages = [list(range(cut[b], cut[b + 1])) for b in range(len(kv))]
    return bd.PagedPlan(new, kv, pages, H, Hkv, d, page_size=page, num_pages=max(1, int(cut[-1])), fmt=fmt, **kw)


def tensor(rows, heads, d, ptr=1 << 21):
    return _abi.bd_tensor(ptr, 0, 0, heads * d, d, rows, 0)


def cache_of(plan, **kw):
    c = _abi.bd_paged_cache()
    width = {bd.BD_CACHE_BF16: plan.d, bd.BD_CACHE_E4M3: plan.d, bd.BD_CACHE_E2M1: plan.d // 2}[plan.fmt]
    for t in (c.k, c.v):
        t.ptr, t.rows, t.stride_head, t.stride_row = 1 << 20, plan.page_size, width, width * plan.Hkv
        t.stride_b = width * plan.Hkv * plan.page_size
    n = plan.d // 16 if plan.fmt == bd.BD_CACHE_E2M1 else 1
    c.k_exp = c.v_exp = 1 << 23
    c.exp_stride_head, c.exp_stride_row, c.exp_stride_page = n, n * plan.Hkv, n * plan.Hkv * plan.page_size
    c.fmt, c.num_pages = plan.fmt, plan.num_pages
    for k, v in kw.items():
        setattr(c, k, v)
    return c


# ------------------------------------------------------------------ the 4-bit format

def test_an_e2m1_cache_needs_scales_and_their_alignment():
    lib = bd.load()
    for d, al in ((64, 4), (128, 8), (256, 8)):
        plan = make([3], [40], d=d)
        kv = tensor(3, 2, d)

        def write(**kw):
            return lib.bd_cache_write(plan.host_ptr, DEV, by(kv), by(kv), by(cache_of(plan, **kw)), None)

        n = d // 16
        assert write(k_exp=None) == _abi.BD_ERR_ARG and write(v_exp=None) == _abi.BD_ERR_ARG
        assert write(k_exp=(1 << 23) + al // 2) == _abi.BD_ERR_ALIGN
        assert write(exp_stride_row=2 * n + al // 2) == _abi.BD_ERR_ALIGN
        assert write(exp_stride_head=n + al // 2) == _abi.BD_ERR_ALIGN
        assert write(exp_stride_page=2 * n * 16 + al // 2) == _abi.BD_ERR_ALIGN
        assert write(exp_stride_row=0) == _abi.BD_ERR_ARG
        assert write(exp_stride_row=2 ** 31 // 16) == _abi.BD_ERR_UNSUPPORTED
        assert write(fmt=bd.BD_CACHE_E4M3) == _abi.BD_ERR_PLAN


def test_binding_refuses_other_e2m1_pools():
    z = torch.zeros(4, 16, 2, 64, dtype=torch.uint8)
    s = torch.zeros(4, 16, 2, 8, dtype=torch.uint8)
    assert bd.PagedCache(z, z, s, s).d == 128 and bd.PagedCache(z, z, s, s).fmt == bd.BD_CACHE_E2M1
    for bad in (None, s[..., :4], s.float(), torch.zeros(4, 16, 2, 16, dtype=torch.uint8)[..., ::2]):
        with pytest.raises(ValueError, match="scales"):
            bd.PagedCache(z, z, bad, s)
        with pytest.raises(ValueError, match="scales"):
            bd.PagedCache(z, z, s, bad)
    with pytest.raises(ValueError, match="strides"):
        bd.PagedCache(z, z, s, torch.zeros(4, 2, 16, 8, dtype=torch.uint8).transpose(1, 2))
    with pytest.raises(ValueError, match="half of a head dim"):
        bd.PagedCache(z[..., :12], z[..., :12], s, s)


def test_oracle_quantiser_follows_the_definition():
    g = torch.Generator().manual_seed(0)
    x = (torch.randn(500, 32, generator=g) * 2.0 ** torch.randint(-20, 18, (500, 1), generator=g)).bfloat16()
    codes, scales = o4.quantise(x)
    y = o4.dequantise(codes, scales)
    s = o4.scales_of(scales).repeat_interleave(16, -1)
    top = x.double().abs().unflatten(-1, (-1, 16)).amax(-1)
    assert ((top <= 6 * o4.scales_of(scales)) | (scales == 226)).all()
    assert ((top > 6 * o4.SCALES[(scales.long() - 1)]) | (scales == 8)).all()
    grid = torch.cat([o4.E2M1, -o4.E2M1])
    near = (x.double()[..., None] - grid * s[..., None]).abs().amin(-1)
    assert torch.equal((x.double() - y).abs(), near)
    assert torch.equal(y, y.bfloat16().double()) and torch.equal(y, y.half().double())   # exact in either


# ------------------------------------------------------------------ rotation

def test_phases_are_turns_to_64_bits():
    f = [0.0, 1.0, 0.5, 1e-6, 123.456, -0.3, 2.0 ** -40, 1e9, 3.1e-5, 500000.0 ** (-62 / 64)]
    got = bd.bd_rope_phases(f)
    for x, p in zip(f, got):
        turns = Fraction(x) / (2 * orope._PI)
        turns -= turns.__floor__()
        off = (int(p) - int(turns * 2 ** 64)) % 2 ** 64
        assert min(off, 2 ** 64 - off) <= 2 ** 64 * (2.0 ** -62 + abs(x) * 2.0 ** -100) + 4096, (x, off)
    for bad in ([float("nan")], [float("inf")]):
        with pytest.raises(bd.BDError, match="finite"):
            bd.bd_rope_phases(bad)
    assert len(bd.bd_rope_phases([])) == 0


@pytest.mark.parametrize("sign", [1, -1])
def test_phases_of_either_sign_are_off_by_units(sign):
    """Two terms cut at 2^-64, and 2^-106 of the frequency: 1 / 2 pi is held to 2^-109, and the product's
    second part, below |f| 2^-55, is rounded twice to 53 bits. No more for negative frequencies, or where
    that second part is negative."""
    g = np.random.default_rng(0)
    f = sign * np.concatenate([np.exp(g.uniform(-25, 25, 600)), 500000.0 ** -(np.arange(64) / 64), 2.0 ** np.arange(-60, 60, 3.0)])
    for x, p in zip(f, bd.bd_rope_phases(f)):
        turns = Fraction(float(x)) / (2 * orope._PI)
        off = (int(p) - (turns - turns.__floor__()) * 2 ** 64) % 2 ** 64
        assert min(off, 2 ** 64 - off) <= 2 + abs(x) * 2.0 ** -42, (x, float(off))


def test_append_refusals():
    lib = bd.load()
    plan = make([3], [40])
    q, kv, c = tensor(3, 8, 128), tensor(3, 2, 128), cache_of(plan)

    def append(dim=128, inter=0, phase=1 << 22, rope=True, q=q, out=q, k=kv, cache=c, p=plan):
        r = _abi.bd_rope(phase, dim, inter, 1.0, 0)
        return lib.bd_cache_append(p.host_ptr, DEV, by(q) if q else None, by(k), by(kv), by(r) if rope else None, by(cache),
                                   by(out) if out else None, None)

    A = _abi.BD_ERR_ARG
    assert append(rope=False) == A and append(phase=None) == A and append(phase=(1 << 22) + 4) == A
    for dim in (0, -16, 24, 144):
        assert append(dim=dim) == A
    assert append(inter=2) == A
    assert append(q=None) == A and append(out=None) == A
    assert append(q=tensor(2, 8, 128)) == A and append(out=tensor(2, 8, 128)) == A and append(k=tensor(2, 2, 128)) == A
    assert append(q=tensor(3, 8, 128, ptr=(1 << 21) + 8)) == _abi.BD_ERR_ALIGN
    free = make([3], [40], causal=False)
    assert append(p=free, cache=cache_of(free)) == _abi.BD_ERR_PLAN
    both = bd.PagedPlan([1, 1], [20, 20], [[0, 1], [2, 1]], 8, 2, 128, page_size=16, num_pages=3, fmt=bd.BD_CACHE_E2M1)
    assert append(p=both, cache=cache_of(both)) == _abi.BD_ERR_PLAN


def test_binding_refuses_other_ropes():
    with pytest.raises(ValueError, match="vector"):
        bd.Rope(torch.zeros(2, 8), device="cpu")
    with pytest.raises(ValueError, match="vector"):
        bd.Rope([], device="cpu")
    r = bd.Rope(torch.ones(8), interleaved=True, scale=0.5)
    assert (r.dim, r.interleaved, r.scale, r.phase.device.type) == (16, True, 0.5, "cpu")
    z = torch.zeros(4, 16, 2, 128, dtype=torch.bfloat16)
    plan = make([3], [40], fmt=bd.BD_CACHE_BF16)
    q = torch.zeros(3, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(RuntimeError, match="not uploaded"):
        bd.bd_cache_append(plan, q, q, q, r, bd.PagedCache(z[:3], z[:3]), q)
    plan.upload("cpu")
    with pytest.raises(ValueError, match="together"):
        bd.bd_cache_append(plan, q, q, q, r, bd.PagedCache(z[:3], z[:3]))
    with pytest.raises(TypeError, match="CUDA"):
        bd.bd_cache_append(plan, q, q, q, r, bd.PagedCache(z[:3], z[:3]), q)


# ------------------------------------------------------------------ selected blocks

def test_sparse_refusals():
    A = _abi.BD_ERR_ARG
    for kw in (dict(blocks=2, first=2), dict(blocks=1, recent=2), dict(blocks=4097), dict(blocks=4, recent=0),
               dict(blocks=4, first=-1), dict(blocks=-1), dict(blocks=4, causal=False)):
        with pytest.raises(bd.BDError) as e:
            make([1], [100], **kw)
        assert e.value.status == A, kw
    P = 16
    pages = [np.zeros(16385, dtype=np.int32)]
    bd.PagedPlan([1], [16384 * P], pages, 8, 2, 128, page_size=P, num_pages=1, blocks=4)
    with pytest.raises(bd.BDError, match="blocks") as e:
        bd.PagedPlan([1], [16384 * P + 1], pages, 8, 2, 128, page_size=P, num_pages=1, blocks=4)
    assert e.value.status == _abi.BD_ERR_UNSUPPORTED
    lib, n = bd.load(), ctypes.c_size_t()
    s = _abi.bd_sparse_desc(4, 0, 1, 0)
    assert lib.bd_sparse_plan_bytes(None, by(s), by(n)) == A
    assert lib.bd_sparse_plan_bytes(by(_abi.bd_paged_desc()), None, by(n)) == A


def test_a_plan_without_lists_has_no_first_or_recent_blocks():
    for kw in (dict(first=1), dict(recent=2), dict(recent=0)):
        with pytest.raises(ValueError, match="blocks="):
            make([1], [100], **kw)
    make([1], [100], first=0, recent=1)


def test_sparse_calls_refuse_other_plans_bounds_and_lists():
    lib = bd.load()
    dense, plan = make([3], [400]), make([3], [400], blocks=4)
    q, ws = tensor(3, 8, 128), ctypes.c_void_p(1 << 22)
    bounds = _abi.bd_bounds(1 << 20, 2 * 2 * 128, 2 * 128, 128, 1 << 21, 2, 1, plan.num_pages, 0)
    lists = _abi.bd_blocks(1 << 20, 8, 4, 3, 0)

    def edit(x, **kw):
        y = type(x)()
        ctypes.memmove(by(y), by(x), ctypes.sizeof(x))
        for k, v in kw.items():
            setattr(y, k, v)
        return y

    def sparse(p=plan, b=lists):
        return lib.bd_sparse_attn(p.host_ptr, DEV, by(q), by(cache_of(p)), by(b) if b else None, by(q), None, ws, 1 << 40, None)

    def select(p=plan, x=bounds, b=lists, q=q):
        return lib.bd_block_select(p.host_ptr, DEV, by(q), by(x) if x else None, by(b) if b else None, None)

    def update(p=plan, x=bounds):
        return lib.bd_block_bounds(p.host_ptr, DEV, by(cache_of(p)), by(x) if x else None, None)

    A, P, L = _abi.BD_ERR_ARG, _abi.BD_ERR_PLAN, _abi.BD_ERR_ALIGN
    assert sparse(p=dense) == P and select(p=dense) == P
    assert lib.bd_paged_attn(plan.host_ptr, DEV, by(q), by(cache_of(plan)), by(q), None, ws, 1 << 40, None) == P
    for call in (sparse, select):
        assert call(b=None) == A and call(b=edit(lists, ptr=None)) == A and call(b=edit(lists, ptr=(1 << 20) + 2)) == A
        assert call(b=edit(lists, rows=2)) == A and call(b=edit(lists, stride_head=3)) == A and call(b=edit(lists, stride_row=3)) == A
    for call in (select, update):
        assert call(x=None) == A and call(x=edit(bounds, code=None)) == A and call(x=edit(bounds, exp=None)) == A
        assert call(x=edit(bounds, num_pages=plan.num_pages + 1)) == P
        assert call(x=edit(bounds, code=(1 << 20) + 8)) == L and call(x=edit(bounds, stride_bound=136)) == L
        assert call(x=edit(bounds, stride_bound=112)) == A and call(x=edit(bounds, stride_head=112)) == A
        assert call(x=edit(bounds, exp_stride_page=0)) == A and call(x=edit(bounds, stride_page=-512)) == A
    assert select(q=tensor(2, 8, 128)) == A
    free = make([3], [400], causal=False)
    assert update(p=free, x=edit(bounds, num_pages=free.num_pages)) == P
    both = bd.PagedPlan([1, 1], [20, 24], [[0, 1], [2, 1]], 8, 2, 128, page_size=16, num_pages=3, fmt=bd.BD_CACHE_E2M1)
    assert both.host[15] and not both.host[BOUNDS_OK]     # rows of their own, a page in common
    assert update(p=both, x=edit(bounds, num_pages=3)) == P


def test_binding_refuses_other_lists_and_bounds():
    plan = make([3], [400], fmt=bd.BD_CACHE_BF16, blocks=4)
    z = torch.zeros(25, 16, 2, 128, dtype=torch.bfloat16)
    cache, q = bd.PagedCache(z, z), torch.zeros(3, 8, 128, dtype=torch.bfloat16)
    b = bd.BlockBounds.empty(cache)
    assert b.code.shape == (25, 2, 2, 128) and b.exp.shape == (25, 2)
    with pytest.raises(ValueError, match="int8"):
        bd.BlockBounds(b.code.to(torch.uint8), b.exp)
    with pytest.raises(ValueError, match="exponents"):
        bd.BlockBounds(b.code, b.exp[:, :1])
    lists = torch.zeros(3, 2, 4, dtype=torch.int32)
    with pytest.raises(RuntimeError, match="not uploaded"):
        bd.bd_block_select(plan, q, b, lists)
    plan.upload("cpu")
    with pytest.raises(TypeError, match="CUDA"):
        bd.bd_block_select(plan, q, b, lists)
    with pytest.raises(TypeError, match="dtype"):
        bd.bd_sparse_attn(plan, q, cache, lists.long(), q)
    with pytest.raises(ValueError, match="heads of"):
        bd.bd_block_bounds(plan, cache, bd.BlockBounds(b.code[:, :1], b.exp[:, :1]))
    dense = make([3], [400], fmt=bd.BD_CACHE_BF16).upload("cpu")
    with pytest.raises(ValueError, match="not a sparse plan"):
        bd.sparse_attn(dense, q, cache, b)


def test_bounds_start_as_those_of_unknown_blocks():
    z = torch.zeros(25, 16, 2, 128, dtype=torch.bfloat16)
    assert (bd.BlockBounds.empty(bd.PagedCache(z, z)).exp == 255).all()


LAYOUTS = [([1], [1]), ([1], [5000]), ([3], [2]), ([5, 0, 1], [0, 7, 90]), ([1, 17, 0, 200, 1], [5000, 17, 40, 333, 16])]


@pytest.mark.parametrize("new,kv", LAYOUTS)
@pytest.mark.parametrize("H,Hkv", [(8, 2), (40, 1), (4, 4)])
@pytest.mark.parametrize("blocks,page", [(1, 16), (7, 16), (3, 64)])
def test_sparse_pieces_cover_every_rows_keys(new, kv, H, Hkv, blocks, page):
    plan = make(new, kv, H, Hkv, page=page, blocks=blocks)
    w, G = plan.host, H // Hkv
    pos = [n - q + i for q, n in zip(new, kv) for i in range(q)]
    assert w[w[POS]:w[POS] + plan.T].tolist() == [max(p, -1) for p in pos]
    cut = np.cumsum([0] + [-(-n // page) for n in kv])
    seq = [b for b, q in enumerate(new) for _ in range(q)]
    assert w[w[ROWPG]:w[ROWPG] + plan.T].tolist() == [w[OFF_PAGES] + cut[b] for b in seq]
    touched = [cut[b] + j for b in range(len(kv)) if new[b]
               for j in range(max(0, kv[b] - new[b]) // page, -(-kv[b] // page))]
    assert w[w[TOUCH]:w[TOUCH] + w[NTOUCH]].tolist() == touched
    seen = {}
    for i in range(w[NDEC]):
        p = w[w[DEC] + 12 * i:w[DEC] + 12 * i + 12].tolist()
        q0, qlen, kvlen, pages, hkv, row0, nrows, k0, k1, _, _, nblk = p
        n = 0 if pos[q0] < 0 else pos[q0] // page + 1
        keys = 0 if n == 0 else (min(n, blocks) - 1) * page + pos[q0] % page + 1
        assert qlen == 1 and kvlen == keys and nblk == n and pages == w[OFF_PAGES] + cut[seq[q0]]
        for r in range(row0, row0 + nrows):
            seen.setdefault((q0, hkv, r), []).append((k0, k1))
    assert len(seen) == plan.T * H
    for (t, _, r), parts in seen.items():
        parts.sort()
        n = 0 if pos[t] < 0 else (min(pos[t] // page + 1, blocks) - 1) * page + pos[t] % page + 1
        assert r < G and parts[0][0] == 0 and parts[-1][1] == n
        assert all(a[1] == b[0] for a, b in zip(parts, parts[1:]))


def test_groups_of_rows_are_of_one_sequence_and_cover_all():
    plan = make([300, 1, 37], [5000, 90, 4000], blocks=9)
    w = plan.host
    assert w[SEL_ROWS] > 1
    rows = []
    for t, n in w[w[SELG]:w[SELG] + 2 * w[NSELG]].reshape(-1, 2).tolist():
        assert 1 <= n <= w[SEL_ROWS] and not any(t < c < t + n for c in (300, 301))
        rows += range(t, t + n)
    assert rows == list(range(338))
    assert make([1] * 4, [900] * 4, blocks=9).host[SEL_ROWS] == 1
    # one row of more than 512 blocks is shared out to a cluster where it finds SMs
    for B, kv, want in ((1, 8000, 1), (1, 9000, 4), (19, 9000, 4), (20, 9000, 2), (38, 9000, 2), (39, 9000, 1)):
        plan = make([1] * B, [kv] * B, blocks=9)
        assert plan.host[SEL_ROWS] == 1 and plan.host[SEL_SPLIT] == want, (B, kv)


def test_key_covers_the_lists():
    base = dict(new=[1, 1], kv=[5000, 333])
    plans = [make(**base), make(**base, blocks=4), make(**base, blocks=5), make(**base, blocks=4, first=1),
             make(**base, blocks=4, recent=2), make([1, 1], [9000, 333], blocks=4)]
    assert len({p.key() for p in plans}) == len(plans)
    assert make([1, 1], [5008, 334], blocks=4).key() == plans[1].key()


def test_key_leaves_out_which_pages_new_rows_enter():
    """Steps that differ in it replay under one graph: sequences with new rows in a page of both, new
    rows without a position. A page that two sequences enter is listed once, with the most rows."""
    def step(new, kv, pages, **kw):
        return bd.PagedPlan(new, kv, pages, 8, 2, 128, page_size=16, num_pages=4, **kw)

    for kw in ({}, dict(blocks=4)):
        apart = step([1, 1], [20, 24], [[0, 1], [2, 3]], **kw)
        for kv in ([20, 24], [24, 20]):
            both = step([1, 1], kv, [[0, 1], [2, 1]], **kw)
            w = both.host
            assert w[BOUNDS_OK] == 0 and apart.host[BOUNDS_OK] == 1 and both.key() == apart.key()
            assert w[w[TOUCH]:w[TOUCH] + w[NTOUCH]].tolist() == [1 if kv[0] > kv[1] else 3]
    none, some = (step([3], [n], [[0]]) for n in (0, 3))
    assert none.host[NTOUCH] == 0 and some.host[NTOUCH] == 1
    some, more = step([3], [2], [[0]]), step([3], [16], [[0]])
    assert some.key() == more.key()


def test_oracle_scores_bound_the_products():
    """A block's score is at least q . k of every key, up to q's rounding: a sanity check of the
    definition."""
    g = torch.Generator().manual_seed(0)
    k, q = torch.randn(16, 64, generator=g).bfloat16(), torch.randn(3, 64, generator=g).bfloat16()
    lo, hi, e = ob.bounds(k)
    best = (q.double() @ k.double().t()).max().item()
    slack = (q.double().abs().amax(-1) / 64 * k.double().abs().amax()).max().item() / 2 * 64
    assert ob.score(q, lo, hi, e) >= best - slack


# ------------------------------------------------------------------ order on a stream

def test_the_new_kernels_wait_before_their_first_read():
    csrc = os.path.join(os.path.dirname(bd.__file__), "csrc")
    names = []
    for f in ("cache_append.cu", "block_select.cu"):
        s = re.sub(r"//[^\n]*", "", open(os.path.join(csrc, f)).read())
        for m in re.finditer(r"__global__ void.*?(\w+_kernel)\(", s, re.S):
            names.append(m.group(1))
            body = s[s.index("{", s.index(") {", m.end())):]
            early = body[:body.index("grid_wait();")]
            assert not re.search(r"\bplan\[|\bphase\[|->|__ld[cg]\w*\(|\bcp\.async", early), m.group(1)
            assert early[early.rfind("\n"):].strip() == ""
    assert set(names) == {"bd_cache_append_kernel", "bd_block_bounds_kernel", "bd_block_select_kernel"}


def test_tile_warps_meet_where_waits_have_a_limit():
    """A warp whose wait ran out leaves its loop: no other may wait for it without a limit. The tile
    kernel's threads meet in barriers before its warps take their roles, and when all have ended."""
    s = open(os.path.join(os.path.dirname(bd.__file__), "csrc", "paged_tile.cu")).read()
    s = re.sub(r"//[^\n]*", "", s)
    roles = s[s.index("if (warp == 0)", s.index("bd_paged_tile_kernel(")):s.index("launch_tile_t(")]
    last = roles.rindex("__syncthreads()")
    assert not re.search(r"named_bar_sync|__syncthreads|bar\.sync", roles[:last])
    assert not re.search(r"\bfor \(|mbar_wait\(", roles[last:])
