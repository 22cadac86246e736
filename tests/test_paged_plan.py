"""Host side of the paged K/V cache (CPU): validation, the plan blob's contents against
plain recomputation, and the binding's refusals."""
import ctypes

import numpy as np
import pytest
import torch

bd = pytest.importorskip("block_causal_varlen_gb300")
from block_causal_varlen_gb300 import _abi  # noqa: E402
from oracle import paged as op  # noqa: E402

# header words and record layouts (csrc/paged_plan.h)
WORDS = ("MAGIC VERSION WORDS B H HKV D G PAGE PAGE_SHIFT NUM_PAGES FMT CAUSAL T KV_TOTAL WRITE_OK SCALE OFF_TOK "
         "OFF_PAGES NPAGES OFF_PGROW OFF_PGCNT OFF_DEC NDEC NDECM DECM_WIDE DEC_LIVE DEC_ROWS OFF_TILE NTILE NTILEM").split()
PIECE = ("Q0", "QLEN", "KVLEN", "PAGES", "HKV", "ROW0", "NROWS", "K0", "K1", "SLOT", "T0", "R1")
MERGE = ("SLOT0", "N", "Q0", "HKV", "ROW0", "NROWS", "R0", "R1")
CTAS = {"DEC": 304, "TILE": 152}


def header(plan):
    return {n: int(plan.host[i]) for i, n in enumerate(WORDS)}


def lists(plan, kind):
    """(pieces of every CTA, merges) of the kind's work list."""
    h, w = header(plan), plan.host
    n_ctas = CTAS[kind]
    rec = 64 if kind == "DEC" else 64 + CTAS["DEC"] * (16 + 8)
    at, n = h[f"OFF_{kind}"], h[f"N{kind}"]
    assert at % 4 == 0
    pieces = [dict(zip(PIECE, w[at + 12 * i:at + 12 * i + 12].tolist())) for i in range(n)]
    ctas, end = [], 0
    for c in range(n_ctas):
        r = w[rec + 16 * c:rec + 16 * c + 16].tolist()
        ctas.append(pieces[r[0]:r[1]])
        if r[1] > r[0]:
            assert r[0] == end and r[4:] == w[at + 12 * r[0]:at + 12 * r[0] + 12].tolist()
            end = r[1]
    assert end == n
    mo = rec + n_ctas * 16
    merges = [dict(zip(MERGE, w[mo + 8 * i:mo + 8 * i + 8].tolist())) for i in range(h[f"N{kind}M"])]
    return ctas, merges


def make(new, kv, H=8, Hkv=2, d=128, page=16, causal=True, pages=None, num_pages=None, fmt=bd.BD_CACHE_BF16):
    if pages is None:
        cut = np.cumsum([0] + [-(-n // page) for n in kv])
        order = np.random.default_rng(3).permutation(int(cut[-1]) + 1)
        pages = [order[cut[b]:cut[b + 1]].tolist() for b in range(len(kv))]
        num_pages = int(cut[-1]) + 1
    return bd.PagedPlan(new, kv, pages, H, Hkv, d, page_size=page, num_pages=num_pages, fmt=fmt, causal=causal), pages


LAYOUTS = [([1], [1]), ([1], [4096]), ([0], [77]), ([3], [2]), ([5], [0]), ([1] * 64, list(range(0, 6400, 100))),
           ([1, 17, 0, 200, 1], [5000, 17, 40, 333, 16]), ([700], [900]), ([1, 1], [200000, 3])]


@pytest.mark.parametrize("new,kv", LAYOUTS)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,Hkv", [(8, 2), (10, 2), (4, 4), (40, 1)])
def test_every_row_meets_every_key_once(new, kv, causal, H, Hkv):
    """Over all pieces of both lists, each (new row, head) is covered by exactly the keys
    it may see: its piece ranges tile [0, last visible key of the block)."""
    plan, _ = make(new, kv, H, Hkv, causal=causal)
    G = H // Hkv
    q0 = np.cumsum([0] + list(new))
    seen = {}
    for kind, unit in (("DEC", 32), ("TILE", 128)):
        ctas, merges = lists(plan, kind)
        pieces = [p for c in ctas for p in c]
        slots = sorted(p["SLOT"] for p in pieces if p["SLOT"] >= 0)
        assert slots == list(range(len(slots))) and len(slots) <= 2 * CTAS[kind]
        joined = {}
        for m in merges:
            assert m["N"] >= 2
            for s in range(m["SLOT0"], m["SLOT0"] + m["N"]):
                assert s not in joined
                joined[s] = m
        assert sorted(joined) == slots
        for p in pieces:
            b = int(np.searchsorted(q0, p["Q0"], side="right") - 1)
            while new[b] == 0:
                b -= 1
            assert p["QLEN"] == new[b] and p["KVLEN"] == kv[b] and p["Q0"] == q0[b]
            assert p["K0"] % unit == 0 and 0 < p["NROWS"] and p["ROW0"] + p["NROWS"] <= new[b] * G
            if p["SLOT"] >= 0:
                m = joined[p["SLOT"]]
                assert all(m[x] == p[x] for x in ("Q0", "HKV", "ROW0", "NROWS"))
            seen.setdefault((b, p["HKV"], p["ROW0"], p["NROWS"]), []).append((p["K0"], p["K1"], p["SLOT"]))
    rows = set()
    for (b, g, r0, n), parts in seen.items():
        for r in range(r0, r0 + n):
            assert (b, g, r) not in rows
            rows.add((b, g, r))
        parts.sort(key=lambda x: (x[0], x[2]))
        last = (r0 + n - 1) // G
        want = max(0, kv[b] - new[b] + last + 1) if causal else kv[b]
        assert parts[0][0] == 0 and parts[-1][1] == want
        assert all(a[1] == c[0] and a[2] + 1 == c[2] for a, c in zip(parts, parts[1:]))
        assert (len(parts) == 1) == (parts[0][2] == -1)
    assert len(rows) == sum(new) * H


def test_work_is_spread_evenly():
    """One long sequence fills the SMs; the longest stretch of a ragged batch is at most
    one key unit and one piece's cost over an even share."""
    for new, kv in (([1], [40000]), ([1] * 64, [int(500 * 1.05 ** i) for i in range(64)])):
        plan, _ = make(new, kv, 32, 8)
        ctas, _ = lists(plan, "DEC")
        load = [sum(-(-(p["K1"] - p["K0"]) // 32) + 6 for p in c) for c in ctas]
        assert max(load) <= sum(load) / len(ctas) + 8, (max(load), sum(load) / len(ctas))


def test_short_contexts_are_not_cut():
    """Blocks that a CTA reads about as fast as a join takes stay whole: no join is launched."""
    for new, kv, d, cut in (([1], [128], 128, False), ([1], [128], 256, False), ([1], [256], 256, True), ([1], [2000], 128, True),
                            ([1] * 8, [200] * 8, 64, False), ([1, 1], [100, 5000], 128, True)):
        plan, _ = make(new, kv, 32, 8, d)
        assert (header(plan)["NDECM"] > 0) == cut, (kv, d)


@pytest.mark.parametrize("Hkv,gang", [(1, 1), (3, 3), (7, 7), (10, 10), (24, 12), (29, 1), (32, 16), (64, 16), (128, 16), (320, 20)])
def test_heads_go_in_gangs(Hkv, gang):
    """Any number of K/V heads: everything is covered, at most 4 CTAs are left over, and a
    gang's CTAs have the same blocks and keys of neighbouring heads."""
    new, kv = [1, 2, 0, 1, 1], [3000, 47, 5, 1, 900]
    for causal in (True, False):
        test_every_row_meets_every_key_once(new, kv, causal, Hkv, Hkv)
    plan, _ = make(new, kv, Hkv, Hkv)
    ctas, _ = lists(plan, "DEC")
    assert 304 % gang <= 4
    for c in range(0, 304 - 304 % gang, gang):
        for g in range(1, gang):
            a, b = ([{k: v for k, v in p.items() if k not in ("HKV", "SLOT")} for p in ctas[c + i]] for i in (0, g))
            assert a == b and [p["HKV"] + g for p in ctas[c]] == [p["HKV"] for p in ctas[c + g]]
    load = [sum(-(-(p["K1"] - p["K0"]) // 32) + 8 for p in c) for c in ctas]
    assert max(load) <= sum(load) / (304 - 304 % gang) + 10


def test_tiles_are_cut_only_where_it_helps():
    """Many equal blocks are given out whole; a few long ones are spread over the SMs."""
    plan, _ = make([64] * 152, [64] * 152, 8, 2)
    ctas, merges = lists(plan, "TILE")
    assert not merges and max(len(c) for c in ctas) == 2
    plan, _ = make([64], [60000], 8, 2)
    ctas, merges = lists(plan, "TILE")
    load = [sum(-(-(p["K1"] - p["K0"]) // 128) + 1 for p in c) for c in ctas]
    assert merges and max(load) <= sum(load) / len(ctas) + 3


@pytest.mark.parametrize("new,kv", LAYOUTS)
def test_rows_and_pages(new, kv):
    plan, pages = make(new, kv)
    h, w = header(plan), plan.host
    assert w[h["OFF_TOK"]:h["OFF_TOK"] + h["T"]].tolist() == op.slots(new, kv, pages, 16)
    want_pg, want_row, want_n, at = [], [], [], 0
    for n, pg in zip(kv, pages):
        for j in range(0, n, 16):
            want_pg.append(pg[j // 16])
            want_row.append(at + j)
            want_n.append(min(16, n - j))
        at += n
    np_ = h["NPAGES"]
    assert np_ == len(want_pg) and h["KV_TOTAL"] == at
    assert w[h["OFF_PAGES"]:h["OFF_PAGES"] + np_].tolist() == want_pg
    assert w[h["OFF_PGROW"]:h["OFF_PGROW"] + np_].tolist() == want_row
    assert w[h["OFF_PGCNT"]:h["OFF_PGCNT"] + np_].tolist() == want_n
    assert h["WRITE_OK"] == 1


def test_table_form_of_the_pages_gives_the_same_blob():
    a, pages = make([1, 2, 0], [40, 33, 5])
    table = np.full((3, 9), -7)          # entries past the last used page may hold anything
    for b, pg in enumerate(pages):
        table[b, :len(pg)] = pg
    b = bd.PagedPlan([1, 2, 0], [40, 33, 5], table, 8, 2, 128, page_size=16, num_pages=a.num_pages)
    assert np.array_equal(a.host, b.host)


def test_sequences_writing_the_same_row_are_found():
    ok = bd.PagedPlan([1, 1], [20, 20], [[0, 1], [0, 2]], 8, 2, 128, page_size=16, num_pages=3)   # a shared prefix page
    assert header(ok)["WRITE_OK"] == 1
    both = bd.PagedPlan([1, 1], [20, 20], [[0, 1], [2, 1]], 8, 2, 128, page_size=16, num_pages=3)
    assert header(both)["WRITE_OK"] == 0
    twice = bd.PagedPlan([20], [20], [[1, 1]], 8, 2, 128, page_size=16, num_pages=3)              # a page listed twice
    assert header(twice)["WRITE_OK"] == 0
    beside = bd.PagedPlan([1, 3], [17, 19], [[0, 1], [2, 1]], 8, 2, 128, page_size=16, num_pages=3)
    assert header(beside)["WRITE_OK"] == 0
    later = bd.PagedPlan([1, 1], [17, 18], [[0, 1], [2, 1]], 8, 2, 128, page_size=16, num_pages=3)
    assert header(later)["WRITE_OK"] == 1


def _bad(match, status, **kw):
    a = dict(q_len=[1, 1], kv_len=[20, 5], pages=[[0, 1], [2]], H=8, Hkv=2, d=128, page_size=16, num_pages=4)
    a.update(kw)
    with pytest.raises(bd.BDError, match=match) as e:
        bd.PagedPlan(**a)
    assert e.value.status == status


def test_plan_refusals():
    A, U, Cp = _abi.BD_ERR_ARG, _abi.BD_ERR_UNSUPPORTED, _abi.BD_ERR_CAPACITY
    _bad("page 4", A, pages=[[0, 4], [2]])
    _bad("page -1", A, pages=[[0, -1], [2]])
    _bad("pages listed", A, pages=[[0], [2]])
    _bad("negative", A, q_len=[-1, 1])
    _bad("negative", A, kv_len=[20, -5])
    _bad("head dim", U, d=96)
    _bad("multiple", U, H=9)
    _bad("multiple", U, H=2 * 129)
    _bad("positive", A, H=0)
    _bad("page_size", U, page_size=8)
    _bad("page_size", U, page_size=24)
    _bad("page_size", U, page_size=2048)
    _bad("num_pages", A, num_pages=0)
    _bad("2\\^31", Cp, num_pages=2 ** 27, page_size=16)
    _bad("format", A, fmt=2)
    _bad("positive", A, q_len=[], kv_len=[], pages=[])
    _bad("2\\^31", Cp, q_len=[2 ** 30, 1])
    with pytest.raises(ValueError, match="one entry"):
        bd.PagedPlan([1], [1, 2], [[0], [1]], 8, 2, 128, page_size=16, num_pages=4)
    # page entries past the used ones are not looked at
    bd.PagedPlan([1], [16], [[0, 99]], 8, 2, 128, page_size=16, num_pages=4)


def test_c_entry_points_refuse_nulls_and_foreign_blobs():
    lib = bd.load()
    n = ctypes.c_size_t()
    assert lib.bd_paged_plan_bytes(None, ctypes.byref(n)) == _abi.BD_ERR_ARG
    plan, _ = make([1], [40])
    assert lib.bd_paged_attn_workspace(plan.host_ptr, None) == _abi.BD_ERR_ARG
    assert lib.bd_paged_attn_workspace(None, ctypes.byref(n)) == _abi.BD_ERR_ARG
    other = bd.Plan([[0, 200, 350, 512]], 512, 2, 4, 4, 64)
    assert lib.bd_paged_attn_workspace(other.host_ptr, ctypes.byref(n)) == _abi.BD_ERR_PLAN
    need = ctypes.c_size_t()
    assert lib.bd_attn_bwd_workspace(plan.host_ptr, ctypes.byref(need)) == _abi.BD_ERR_PLAN
    c = _abi.bd_paged_cache()
    t = _abi.bd_tensor()
    dev = ctypes.c_void_p(4096)     # never read: every refusal below comes before a launch
    assert lib.bd_cache_write(plan.host_ptr, None, ctypes.byref(t), ctypes.byref(t), ctypes.byref(c), None) == _abi.BD_ERR_ARG
    assert lib.bd_cache_write(plan.host_ptr, dev, ctypes.byref(t), ctypes.byref(t), None, None) == _abi.BD_ERR_ARG
    c.fmt = 1
    assert lib.bd_cache_write(plan.host_ptr, dev, ctypes.byref(t), ctypes.byref(t), ctypes.byref(c), None) == _abi.BD_ERR_PLAN
    c.fmt, c.num_pages = 0, plan.num_pages + 1
    assert lib.bd_paged_attn(plan.host_ptr, dev, ctypes.byref(t), ctypes.byref(c), ctypes.byref(t), None, None, 0,
                             None) == _abi.BD_ERR_PLAN
    c.num_pages, c.k.rows, c.v.rows = plan.num_pages, 16, 16
    assert lib.bd_cache_read(plan.host_ptr, dev, ctypes.byref(c), ctypes.byref(t), ctypes.byref(t), None) == _abi.BD_ERR_ARG


def _fake_cache(plan, **kw):
    """A bd_paged_cache with made-up addresses, for refusals that come before any launch."""
    c = _abi.bd_paged_cache()
    for t in (c.k, c.v):
        t.ptr, t.rows, t.stride_head, t.stride_row = 1 << 20, plan.page_size, plan.d, plan.d * plan.Hkv
        t.stride_b = plan.d * plan.Hkv * plan.page_size
    c.fmt, c.num_pages = plan.fmt, plan.num_pages
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _fake(rows, heads, d, ptr=1 << 21):
    return _abi.bd_tensor(ptr, 0, 0, heads * d, d, rows, 0)


def test_c_entry_points_check_alignment_rows_and_workspace():
    lib, dev = bd.load(), ctypes.c_void_p(4096)
    plan, _ = make([3], [40])
    by = ctypes.byref
    q, kv = _fake(3, 8, 128), _fake(3, 2, 128)

    def attn(q=q, out=q, cache=None, lse=None, ws=1 << 22, n=1 << 40):
        return lib.bd_paged_attn(plan.host_ptr, dev, by(q), by(cache or _fake_cache(plan)), by(out),
                                 by(lse) if lse else None, ctypes.c_void_p(ws), n, None)

    assert attn(q=_fake(2, 8, 128)) == _abi.BD_ERR_ARG                     # fewer rows than new rows
    assert attn(out=_fake(2, 8, 128)) == _abi.BD_ERR_ARG
    assert attn(q=_fake(3, 8, 128, ptr=(1 << 21) + 8)) == _abi.BD_ERR_ALIGN
    assert attn(ws=None) == _abi.BD_ERR_ARG and attn(ws=(1 << 22) + 16) == _abi.BD_ERR_ARG
    assert attn(n=16) == _abi.BD_ERR_CAPACITY
    assert attn(lse=_abi.bd_rowstat(None, 0, 0, 3)) == _abi.BD_ERR_ARG
    assert attn(lse=_abi.bd_rowstat(1 << 23, 0, 0, 2)) == _abi.BD_ERR_ARG  # heads' rows overlap
    odd = _fake_cache(plan)
    odd.k.stride_row = 2 * 128 + 4
    assert attn(cache=odd) == _abi.BD_ERR_ALIGN
    assert lib.bd_cache_write(plan.host_ptr, dev, by(_fake(2, 2, 128)), by(kv), by(_fake_cache(plan)), None) == _abi.BD_ERR_ARG
    assert lib.bd_cache_read(plan.host_ptr, dev, by(_fake_cache(plan)), by(_fake(39, 2, 128)), by(_fake(40, 2, 128)),
                             None) == _abi.BD_ERR_ARG
    e4, _ = make([3], [40], fmt=bd.BD_CACHE_E4M3)
    assert lib.bd_cache_write(e4.host_ptr, dev, by(kv), by(kv), by(_fake_cache(e4)), None) == _abi.BD_ERR_ARG  # no exponents
    free, _ = make([3], [40], causal=False)
    assert lib.bd_cache_write(free.host_ptr, dev, by(kv), by(kv), by(_fake_cache(free)), None) == _abi.BD_ERR_PLAN
    both = bd.PagedPlan([1, 1], [20, 20], [[0, 1], [2, 1]], 8, 2, 128, page_size=16, num_pages=3)
    assert lib.bd_cache_write(both.host_ptr, dev, by(kv), by(kv), by(_fake_cache(both)), None) == _abi.BD_ERR_PLAN


def test_binding_refusals():
    z = torch.zeros(4, 16, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="pages, page_size"):
        bd.PagedCache(z[0], z[0])
    with pytest.raises(ValueError, match="differ"):
        bd.PagedCache(z, z[:, :8])
    with pytest.raises(TypeError, match="dtype"):
        bd.PagedCache(z.float(), z.float())
    with pytest.raises(ValueError, match="no exponents"):
        bd.PagedCache(z, z, torch.zeros(4, 16, 2, dtype=torch.uint8))
    f = z.to(torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="exponents"):
        bd.PagedCache(f, f)
    e = torch.zeros(4, 16, 2, dtype=torch.uint8)
    with pytest.raises(ValueError, match="strides"):
        bd.PagedCache(f, f, e, torch.zeros(4, 2, 16, dtype=torch.uint8).transpose(1, 2))
    cache = bd.PagedCache(z, z)
    plan, _ = make([3], [40], num_pages=4, pages=[[0, 1, 2]])
    q = torch.zeros(3, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(RuntimeError, match="not uploaded"):
        bd.bd_paged_attn(plan, q, cache, q)
    plan.upload("cpu")      # a host copy stands in: the refusals below come before a launch
    with pytest.raises(TypeError, match="dtype"):
        bd.bd_paged_attn(plan, q.float(), cache, q)
    with pytest.raises(TypeError, match="CUDA"):
        bd.bd_paged_attn(plan, q, cache, q)
    with pytest.raises(TypeError, match="CUDA"):
        bd.bd_cache_write(plan, q, q, cache)
    with pytest.raises(ValueError, match="heads of"):
        bd.bd_cache_read(plan, bd.PagedCache(z[:, :, :1], z[:, :, :1]), q, q)


def test_key_follows_what_a_captured_call_holds():
    a, _ = make([1, 1], [5000, 333])
    b, _ = make([1, 1], [5001, 334], num_pages=a.num_pages, pages=[list(range(313)), list(range(313, 334))])
    assert a.key() == b.key() and bd.bd_paged_attn_workspace(a) == bd.bd_paged_attn_workspace(b)
    c, _ = make([1, 1], [5, 7], num_pages=a.num_pages, pages=[[0], [1]])            # nothing to join
    d, _ = make([1, 1], [5000, 333], causal=False)
    e, _ = make([1, 1], [5000, 333], H=4)
    assert len({a.key(), c.key(), d.key(), e.key()}) == 4


def test_oracle_quantiser_matches_torch_rounding():
    """The oracle's nearest-code search against torch's own e4m3 conversion, on values
    within range, and the definition of the exponent."""
    g = torch.Generator().manual_seed(0)
    x = torch.cat([torch.randn(64, 64, generator=g) * 2.0 ** torch.randint(-20, 20, (64, 1), generator=g),
                   torch.zeros(1, 64), torch.full((1, 64), 448.0), torch.full((1, 64), 449.0)]).bfloat16()
    codes, exps = op.quantise(x)
    e = exps.double() - 127
    top = x.double().abs().amax(-1)
    assert ((top <= 448 * 2.0 ** e) | (e == 60)).all() and ((top > 448 * 2.0 ** (e - 1)) | (e == -60)).all()
    want = (x.double() * 2.0 ** -e[:, None]).float().to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(codes, want)
    back = op.dequantise(codes, exps)
    assert torch.equal(back, back.bfloat16().double()), "values read back are exact in bf16"
    assert ((back - x.double()).abs() <= top[:, None] * 2.0 ** -4).all()
    bad = torch.ones(2, 64, dtype=torch.bfloat16)
    bad[0, 3], bad[1, 5] = float("inf"), float("nan")
    codes, exps = op.quantise(bad)
    assert (codes == 127).all() and (exps == 255).all() and torch.isnan(op.dequantise(codes, exps)).all()


def test_oracle_attention_matches_the_chunk_oracle():
    """New rows over cached rows = the last rows of a causal document."""
    import oracle
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(50, h, 64, generator=g).bfloat16() for h in (4, 2, 2))
    o, lse = oracle.attention_fwd(q, k, v, [0, 50])
    got, gl, _, _ = op.attention(q[43:], k, v, 50)
    assert torch.allclose(got, o[43:].double(), atol=1e-12) and torch.allclose(gl, lse[:, 43:].double(), atol=1e-12)


def test_lengths_and_pages_are_whole_numbers_in_range():
    for bad in ([1.5], [2 ** 32], np.array([2 ** 40])):
        with pytest.raises(ValueError, match="whole"):
            bd.PagedPlan([1], bad, [[0, 1]], 8, 2, 128, page_size=16, num_pages=4)
        with pytest.raises(ValueError, match="whole"):
            bd.PagedPlan([1], [16], [bad], 8, 2, 128, page_size=16, num_pages=4)
    a = bd.PagedPlan(np.array([1], np.int64), torch.tensor([17]), [torch.tensor([2, 0])], 8, 2, 128, page_size=16, num_pages=4)
    b = bd.PagedPlan([1], [17], [[2, 0]], 8, 2, 128, page_size=16, num_pages=4)
    assert np.array_equal(a.host, b.host)


@pytest.mark.parametrize("name", ["H", "Hkv", "d", "page_size", "num_pages", "fmt"])
def test_sizes_are_whole_numbers_in_range(name):
    a = dict(H=8, Hkv=2, d=128, page_size=16, num_pages=4, fmt=0)
    bd.PagedPlan([1], [17], [[0, 1]], **{**a, name: np.int64(a[name])})
    for bad in (a[name] + 2 ** 32, a[name] + 0.5, [a[name]]):
        with pytest.raises(ValueError, match=name):
            bd.PagedPlan([1], [17], [[0, 1]], **{**a, name: bad})


def test_no_lengths_past_the_kernels_arithmetic():
    """A page may be listed again and again: kv_len is bounded by itself, not by the pool."""
    n = 2 ** 31 - 1
    pages = np.zeros((1, 2 ** 21), np.int32)
    with pytest.raises(bd.BDError) as e:
        bd.PagedPlan([1], [n], pages, 8, 2, 128, page_size=1024, num_pages=4)
    assert e.value.status == _abi.BD_ERR_CAPACITY


def test_a_blob_too_small_is_refused():
    plan, pages = make([300, 1], [300, 5000])
    q, kv, flat = (np.array(x, np.int32) for x in ([300, 1], [300, 5000], sum(pages, [])))
    offs = np.array([0, len(pages[0]), len(flat)], np.int32)
    p32 = ctypes.POINTER(ctypes.c_int32)
    desc = _abi.bd_paged_desc(2, 8, 2, 128, 16, plan.num_pages, 0, 1, *[x.ctypes.data_as(p32) for x in (q, kv, flat, offs)])
    need = bd.bd_paged_plan_bytes(desc)
    blob = np.full(need // 4 + 16, 7, np.int32)
    at = blob.ctypes.data + (-blob.ctypes.data % 64)
    lib = bd.load()
    assert lib.bd_paged_plan_build(ctypes.byref(desc), ctypes.c_void_p(at), need - 4) == _abi.BD_ERR_CAPACITY
    assert (blob == 7).all()
    assert lib.bd_paged_plan_build(ctypes.byref(desc), ctypes.c_void_p(at + 4), need) == _abi.BD_ERR_ARG      # alignment
    assert lib.bd_paged_plan_build(ctypes.byref(desc), ctypes.c_void_p(at), need) == 0
    off = (at - blob.ctypes.data) // 4
    assert np.array_equal(blob[off:off + len(plan.host)], plan.host) and len(plan.host) * 4 <= need


_C = r"""
#include <stdio.h>
#include <string.h>
#include "bd_paged.h"
int main(void) {
  const int32_t q[2] = {1, 3}, kv[2] = {40, 17}, pages[5] = {4, 0, 2, 1, 3}, offs[3] = {0, 3, 5}, bad[5] = {4, 0, 9, 1, 3};
  bd_paged_desc d;
  size_t n = 0;
  static int32_t blob[1 << 16];
  uint64_t key = 0;
  memset(&d, 0, sizeof d);
  d.B = 2; d.H = 8; d.Hkv = 2; d.d = 128; d.page_size = 16; d.num_pages = 5; d.fmt = BD_CACHE_E4M3; d.causal = 1;
  d.q_len = q; d.kv_len = kv; d.pages = pages; d.page_offsets = offs;
  if (bd_paged_plan_bytes(&d, &n) != BD_OK || n > sizeof blob) { printf("error %s\n", bd_last_error()); return 1; }
  if (bd_paged_plan_build(&d, (void*)(((size_t)blob + 15) & ~(size_t)15), sizeof blob - 16) != BD_OK) return 1;
  if (bd_paged_plan_key((void*)(((size_t)blob + 15) & ~(size_t)15), &key) != BD_OK || key == 0) return 1;
  d.pages = bad;
  printf("reject %d\n", (int)bd_paged_plan_bytes(&d, &n));
  printf("sizeof %u %u\n", (unsigned)sizeof(bd_paged_cache), (unsigned)sizeof(bd_paged_desc));
  return 0;
}
"""


def test_c99_consumer(tmp_path):
    """The header is plain C99, the structs have the binding's sizes, and a C program
    plans and is refused like the binding."""
    import os
    import shutil
    import subprocess
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("no C compiler")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src, exe = tmp_path / "p.c", tmp_path / "p"
    src.write_text(_C)
    subprocess.run([cc, "-std=c99", "-pedantic", "-Wall", "-Werror", "-I", os.path.join(root, "include"), str(src), "-o", str(exe),
                    _abi.LIB_PATH, f"-Wl,-rpath,{os.path.dirname(_abi.LIB_PATH)}"], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert out == ["reject", str(_abi.BD_ERR_ARG), "sizeof", str(ctypes.sizeof(_abi.bd_paged_cache)),
                   str(ctypes.sizeof(_abi.bd_paged_desc))]
