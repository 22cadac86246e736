"""Cases for a paged K/V cache held in 4 bits, for appending rotated rows to a cache, and for
attention over the blocks of a cache that a cheap score selects.

The operators, for sequence b with q_b new rows of kv_b rows in the cache, new row i at
position p = kv_b - q_b + i:

* an e2m1 cache holds, for every 16 values of a (row, head), a scale s = (1 + m/8) 2^(e - 15) by
  its byte 8 e + m, the smallest byte of [8, 226] that has max|x| <= 6 s (226 where none has),
  and the codes of x / s rounded to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (ties to the even
  code), saturating at 6; two codes a byte, the even element's in the low half.
* append: K and q are turned by their position first: with f the pair's frequency,
  (x, y) -> scale (x cos(p f) - y sin(p f), y cos(p f) + x sin(p f)); the pairs are (c, c + r/2)
  or (2 c, 2 c + 1) of the first r elements of a head, the others stay. Rotated rows are bf16
  rows, which then enter the cache as those of a plain write do.
* write, read, attention: as for the other formats (perf/operators.py).
* sparse attention over blocks (the pages of a sequence): a block of a K/V head is described by
  the least and the greatest value of every element of its keys, in 8 bits: lo = floor(min 2^-e),
  hi = ceil(max 2^-e), e the smallest integer of [-50, 50] with max|.| <= 127 2^e (50 where none
  has; codes saturate). q is held in 8 bits too, rn(q 2^-e), e by the same rule for every head. A
  block's score for a head is sum_c max(q_c lo_c, q_c hi_c) times both powers of two, for a group
  the largest of its heads'. New row i attends, for every K/V head, `blocks` of the blocks up to
  its own: the first `first`, the last `recent` (its own among them), and those of the largest
  scores (ties: the lowest index); all, if there are no more. Lists ascend and end in -1.
"""
import math
import random

import numpy as np
import torch

own = False


def _case(name, op, fmt, B, new, ctx, heads, page, heads_first=False, layout=1, rot=0, pairs=False, blocks=0, first=1, recent=1):
    """One case: `new` = (lo, hi) new rows of a sequence, `ctx` = (lo, hi) rows cached before them,
    heads = (H, Hkv, d), rot = rotated elements of a head, pairs: of neighbours."""
    return {"name": name, "op": op, "fmt": fmt, "B": B, "new_lo": new[0], "new_hi": new[1], "ctx_lo": ctx[0],
            "ctx_hi": ctx[1], "H": heads[0], "Hkv": heads[1], "d": heads[2], "page": page, "heads_first": heads_first,
            "layout": layout, "rot": rot, "pairs": pairs, "blocks": blocks, "first": first, "recent": recent}


def listed():
    return [
        # a decode step's rows of a few sequences are turned and stored: pure launch latency
        _case("append bf16 step", "append", "bf16", 8, (1, 1), (100, 8000), (32, 8, 128), 64, rot=128),
        # packed prompts of a few hundred to eight thousand rows are turned, q too, and enter a cache
        _case("append bf16 prompts", "append", "bf16", 8, (300, 8000), (0, 300), (32, 8, 128), 64, rot=128),
        # the same into 8 bits, half of each head turned by neighbouring pairs, then read back as bf16 rows for a prefill
        _case("append e4m3 prompts", "append", "e4m3", 6, (64, 2048), (0, 300), (16, 8, 128), 16, True, rot=64, pairs=True),
        # a whole decode step of a layer over a 4-bit cache: the new rows enter it, and attend
        _case("step e2m1", "step", "e2m1", 16, (1, 1), (300, 6000), (32, 8, 128), 64, rot=128),
        # a long prefill step enters a 4-bit cache, sequences continuing in the middle of a page
        _case("write e2m1 prompts", "write", "e2m1", 12, (500, 8000), (0, 3000), (32, 8, 128), 64, True),
        # one long document is read back from a 4-bit cache as bf16 rows
        _case("read e2m1 long", "read", "e2m1", 1, (0, 0), (49152, 49152), (32, 8, 128), 64),
        # a single user's decode step: little to read, latency counts
        _case("decode e2m1 one", "attn", "e2m1", 1, (1, 1), (4095, 4095), (32, 8, 128), 16),
        # a full decode batch with contexts of every length
        _case("decode e2m1 batch", "attn", "e2m1", 64, (1, 1), (500, 16000), (32, 8, 128), 64, True),
        # a serving step that mixes drafted rows with prompt chunks, head dim 256
        _case("mixed e2m1 d256", "attn", "e2m1", 10, (1, 700), (60, 8000), (16, 4, 256), 32, False, 22),
        # one chunk of a long prompt over what is cached already
        _case("chunk e2m1", "attn", "e2m1", 1, (4096, 4096), (12288, 12288), (32, 8, 128), 64, True),
        # a decode step over long contexts, each row over 2048 keys that the blocks' bounds pick
        _case("sparse bf16 decode", "sparse", "bf16", 16, (1, 1), (4000, 60000), (32, 8, 128), 64, True, blocks=32, recent=2),
        # a chunk of a prompt whose rows each pick their blocks, 4-bit cache
        _case("sparse e2m1 chunk", "sparse", "e2m1", 2, (200, 500), (6000, 16000), (16, 4, 128), 32, blocks=24),
    ]


def _logint(r, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    if hi <= lo:
        return lo
    a = max(lo, 1)
    v = int(round(math.exp(r.uniform(math.log(a), math.log(hi)))))
    return min(hi, max(lo, v))


def lengths(case):
    """(new rows, cached rows with them) of every sequence."""
    r = random.Random(case["layout"])
    q = [_logint(r, case["new_lo"], case["new_hi"]) for _ in range(case["B"])]
    return q, [x + _logint(r, case["ctx_lo"], case["ctx_hi"]) for x in q]


# what a drawn case may cost at most: the largest listed ones
MOST_CACHE = 350_000 * 8 * 128 * 2      # cached values of K and V
MOST_ROWS = 30_000 * 48 * 128           # values of the new rows of q, K and V
MOST_PADDED = 64 * 16001 * 8 * 128      # values of K in a batch padded to its longest sequence
MOST_SCORES = 32 * 4096 * 16384         # scores of a batch padded to its longest chunk and sequence
MOST_GATHERED = 700 * 4 * 24 * 32 * 128  # values of K that rows of their own blocks take


def draw(rng):
    while True:
        op = rng.choice(["append", "append", "step", "write", "read", "attn", "attn", "attn", "sparse", "sparse"])
        H, Hkv, d = rng.choice([(32, 8, 128), (16, 8, 128), (32, 8, 64), (4, 4, 64), (32, 8, 256), (10, 2, 128), (8, 1, 128),
                                (24, 8, 256)])
        B = _logint(rng, 1, 64)
        ctx_hi = _logint(rng, 1, 30000)
        ctx_lo = min(ctx_hi, _logint(rng, 1, 2000))
        if op == "read":
            new = (0, 0)
        elif rng.random() < 0.5 or op == "step":
            new = (1, rng.choice([1, 1, 1, 2, 5, 8]))
        else:
            hi = _logint(rng, 2, 300 if op == "sparse" else 4096)
            new = (_logint(rng, 1, hi), hi)
        fmt = "e2m1" if op in ("write", "read", "attn", "step") else rng.choice(["bf16", "e4m3", "e2m1"])
        page = rng.choice([16, 32, 64, 128])
        rot = rng.choice([d, d, d // 2, 16]) if op in ("append", "step") else 0
        first, recent = rng.choice([0, 1, 2]), rng.choice([1, 1, 2])
        blocks = max(first + recent, _logint(rng, 3, 64)) if op == "sparse" else 0
        c = _case("", op, fmt, B, new, (ctx_lo, ctx_hi), (H, Hkv, d), page, rng.random() < 0.5, rng.randrange(1 << 20), rot,
                  rng.random() < 0.5, blocks, first, recent)
        del c["name"]
        q, kv = lengths(c)
        padded = B * max(kv) * Hkv * d
        if (2 * sum(kv) * Hkv * d > MOST_CACHE or padded > MOST_PADDED or sum(q) * (H + 2 * Hkv) * d > MOST_ROWS
                or (op in ("attn", "step") and B * H * max(q) * max(kv) > MOST_SCORES)
                or (op == "sparse" and sum(q) * Hkv * blocks * page * d > MOST_GATHERED)):
            continue
        return c


def _row_bytes(case):
    """Bytes of one head's K (or V) of a cached row."""
    d = case["d"]
    return {"bf16": 2 * d, "e4m3": d + 1, "e2m1": d // 2 + d // 16}[case["fmt"]]


def work(case):
    q, kv = lengths(case)
    H, Hkv, d, op, P = case["H"], case["Hkv"], case["d"], case["op"], case["page"]
    cached = 2 * Hkv * _row_bytes(case)                  # bytes of one row of K and V in the cache
    plain = 2 * Hkv * d * 2                              # and as bf16
    rows_q = sum(q) * H * d * 2
    pairs = sum(a * b - a * (a - 1) // 2 for a, b in zip(q, kv))
    attn = {"bytes": sum(kv) * cached + 2 * rows_q + sum(q) * H * 4, "flops": 4 * d * H * pairs}
    if op == "write":
        return {"bytes": sum(q) * (plain + cached), "flops": 0}
    if op == "read":
        return {"bytes": sum(kv) * (plain + cached), "flops": 0}
    if op == "attn":
        return attn
    turn = 6 * sum(q) * (H + Hkv) * case["rot"] // 2
    if op == "step":
        return {"bytes": attn["bytes"] + rows_q + sum(q) * (plain + cached), "flops": attn["flops"] + turn}
    if op == "append":
        back = 0 if case["fmt"] == "bf16" else sum(kv) * (plain + cached)
        return {"bytes": 2 * rows_q + sum(q) * (plain + cached) + back, "flops": turn}
    n = [min(case["blocks"], (p // P) + 1) for a, b in zip(q, kv) for p in range(b - a, b)]
    seen = sum(((k - 1) * P + p % P + 1) for k, p in zip(n, [p for a, b in zip(q, kv) for p in range(b - a, b)]))
    nblk, touched = sum(-(-b // P) for b in kv), sum((b - 1) // P - (b - a) // P + 1 for a, b in zip(q, kv))
    keys = Hkv * min(seen, sum(kv))                      # keys of one head that some row attends, at most
    return {"bytes": keys * 2 * _row_bytes(case) + touched * P * Hkv * _row_bytes(case) + (nblk + touched) * Hkv * (2 * d + 1)
            + 2 * rows_q + sum(q) * H * 4 + sum(q) * Hkv * case["blocks"] * 4,
            "flops": 4 * d * H * seen + 4 * d * H * sum(p // P + 1 for a, b in zip(q, kv) for p in range(b - a, b))}


# ------------------------------------------------------------------ the formats

def _pow2(e):
    """2^e for whole numbers e of [-126, 127], in 32 bits (pow and ldexp may be a step off)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _scales(device):
    """The values of the scale bytes 0..226 of an e2m1 cache."""
    b = torch.arange(227, device=device, dtype=torch.float64)
    e, m = torch.div(b, 8, rounding_mode="floor"), torch.remainder(b, 8)
    return torch.where(e == 0, m / 8 * 2.0 ** -14, (1 + m / 8) * torch.pow(2.0, e - 15)).float()


def _quantise4(x):
    """Packed codes [..., d / 2] and scale bytes [..., d / 16] of x, as defined at the top."""
    table = _scales(x.device)
    g = x.float().unflatten(-1, (-1, 16))
    byte = (8 + torch.searchsorted(6 * table[8:], g.abs().amax(-1))).clamp(max=226)
    y = g.abs().double() / table.double()[byte][..., None]
    code = ((y > 0.25).int() + (y >= 0.75).int() + (y > 1.25).int() + (y >= 1.75).int() + (y > 2.5).int() + (y >= 3.5).int()
            + (y > 5).int() + torch.signbit(g).int() * 8).flatten(-2)
    return (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8), byte.to(torch.uint8)


def _values4(codes, scale):
    """The values that packed codes and their scale bytes stand for, in 32 bits."""
    mag = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    both = torch.cat([mag, -mag])
    c = codes.int()
    x = torch.stack([both[c & 15], both[c >> 4]], -1).flatten(-2)
    return (x.unflatten(-1, (-1, 16)) * _scales(codes.device)[scale.int()][..., None]).flatten(-2)


def _quantise8(x):
    """e4m3 codes and exponent bytes of x [..., d]: e the smallest integer of [-60, 60] with
    max|x| <= 448 2^e, codes rn(x 2^-e)."""
    amax = x.float().abs().amax(-1)
    f, E = torch.frexp(amax)                             # amax = f 2^E, f in [0.5, 1); 448 = 0.875 2^9
    e = torch.where(amax == 0, -60, E - 9 + (f > 0.875)).clamp(-60, 60)
    y = (x.float() * _pow2(-e)[..., None]).clamp(-448, 448)
    return y.to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _store(st, name, page, row, x):
    """bf16 rows x into the cache, in its format."""
    fmt = st["case"]["fmt"]
    if fmt == "bf16":
        st[name][page, row] = x
    else:
        codes, s = _quantise8(x) if fmt == "e4m3" else _quantise4(x)
        st[name].view(torch.uint8)[page, row] = codes.view(torch.uint8)
        st[name + "_s"][page, row] = s


def _load(st, name, page, row):
    """Cached rows in 32 bits."""
    fmt = st["case"]["fmt"]
    if fmt == "bf16":
        return st[name][page, row].float()
    c, s = st[name].view(torch.uint8)[page, row], st[name + "_s"][page, row]
    return _values4(c, s) if fmt == "e2m1" else c.view(torch.float8_e4m3fn).float() * _pow2(s.int() - 127)[..., None]


def _pow8(amax):
    """The smallest e of [-50, 50] with amax <= 127 2^e."""
    f, E = torch.frexp(amax)                             # 127 = 0.9921875 2^7
    return torch.where(amax == 0, -50, E - 7 + (f > 0.9921875)).clamp(-50, 50)


def _bounds_of(k, count):
    """lo / hi codes [n, Hkv, 2, d] and exponent bytes of blocks of keys k [n, P, Hkv, d], `count` of which are there."""
    gone = (torch.arange(k.shape[1], device=k.device) >= count[:, None])[..., None, None]
    lo, hi = k.masked_fill(gone, math.inf).amin(1), k.masked_fill(gone, -math.inf).amax(1)
    e = _pow8(torch.maximum(lo.abs(), hi.abs()).amax(-1))
    f = _pow2(-e)[..., None]
    both = torch.stack([(lo * f).floor(), (hi * f).ceil()], 2)
    return both.clamp(-127, 127).to(torch.int8), (e + 127).to(torch.uint8)


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    q, kv = lengths(case)
    B, H, Hkv, d, P, op = case["B"], case["H"], case["Hkv"], case["d"], case["page"], case["op"]
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    npages = [-(-n // P) for n in kv]
    total = sum(npages) + 3                              # a few pages belong to nobody
    order = np.random.default_rng(seed).permutation(total).astype(np.int32)
    cut = np.cumsum([0] + npages)
    pages = [order[cut[b]:cut[b + 1]] for b in range(B)]
    shape = (total, Hkv, P, d) if case["heads_first"] else (total, P, Hkv, d)

    def rows_first(x):
        return x.transpose(1, 2) if case["heads_first"] else x          # [page, row, head, ...] either way

    st = {"case": case, "k_s": None, "v_s": None}
    for name in ("k", "v"):
        x = torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)
        if op == "sparse" and name == "k":               # keys of a block have something in common
            x = x + torch.randn(total, Hkv, d, generator=g, device=dev, dtype=torch.bfloat16).unsqueeze(2 if case["heads_first"] else 1)
        if case["fmt"] != "bf16":
            # rows of different sizes, so that scales differ
            mag = torch.exp2(torch.randint(-3, 4, shape[:3], generator=g, device=dev).float())
            x = x * (mag if name == "v" else mag.clamp(max=2))[..., None].to(x.dtype)
            x, s = _quantise8(x) if case["fmt"] == "e4m3" else _quantise4(x)
            st[name + "_s"] = rows_first(s)
        st[name] = rows_first(x)
    T = sum(q)
    if T:
        # the rows of a fused projection, as they come: the heads of q, then k, then v
        qkv = torch.randn(T, (H + 2 * Hkv) * d, generator=g, device=dev, dtype=torch.bfloat16)
        st["q"] = qkv[:, :H * d].view(T, H, d)
        st["k_new"] = qkv[:, H * d:(H + Hkv) * d].view(T, Hkv, d)
        st["v_new"] = qkv[:, (H + Hkv) * d:].view(T, Hkv, d)
    if case["rot"]:
        r = case["rot"]
        st["inv_freq"] = (1.0 / 500000.0 ** (torch.arange(0, r, 2, dtype=torch.float64) / r)).float().to(dev)
        st["q_turned"] = torch.empty(T, H, d, device=dev, dtype=torch.bfloat16)
    # where things are, for the plain form
    table = np.zeros((B, max(npages)), dtype=np.int64)
    for b in range(B):
        table[b, :npages[b]] = pages[b]
    st["table"] = torch.from_numpy(table).to(dev)
    st["q_len"], st["kv_len"] = torch.tensor(q, device=dev), torch.tensor(kv, device=dev)
    st["max_q"], st["max_kv"] = max(q), max(kv)
    for key, n in (("new", q), ("row", kv)):
        st[key + "_seq"] = torch.from_numpy(np.repeat(np.arange(B), n)).to(dev)
        st[key + "_idx"] = torch.from_numpy(np.concatenate([np.arange(x) for x in n])).to(dev)
    if op == "read" or (op == "append" and case["fmt"] != "bf16"):
        st["k_out"] = torch.empty(sum(kv), Hkv, d, device=dev, dtype=torch.bfloat16)
        st["v_out"] = torch.empty_like(st["k_out"])
    if op in ("attn", "step", "sparse"):
        st["out"] = torch.empty(T, H, d, device=dev, dtype=torch.bfloat16)
        st["lse"] = torch.empty(H, T, device=dev, dtype=torch.float32)
    if op == "sparse":
        # every block's bounds as earlier steps left them; those of the blocks that new rows enter come with the step
        page = torch.arange(total, device=dev)
        st["bounds"] = torch.empty(total, Hkv, 2, d, device=dev, dtype=torch.int8)
        st["bounds_exp"] = torch.empty(total, Hkv, device=dev, dtype=torch.uint8)
        for p in page.split(max(1, (1 << 27) // (P * Hkv * d))):
            x = _load(st, "k", p, slice(None))
            st["bounds"][p], st["bounds_exp"][p] = _bounds_of(x, torch.full_like(p, P))
        touched = [(b, j) for b in range(B) for j in range((kv[b] - q[b]) // P, npages[b])]
        st["touched"] = torch.tensor([int(pages[b][j]) for b, j in touched], device=dev)
        st["touched_rows"] = torch.tensor([min(P, kv[b] - j * P) for b, j in touched], device=dev)
        st["blocks"] = torch.empty(T, Hkv, case["blocks"], device=dev, dtype=torch.int32)
    if own:
        import block_causal_varlen_gb300 as bd

        st["cache"] = bd.PagedCache(st["k"], st["v"], st["k_s"], st["v_s"])
        more = {"blocks": case["blocks"], "first": case["first"], "recent": case["recent"]} if op == "sparse" else {}
        st["plan"] = bd.PagedPlan(q, kv, pages, H, Hkv, d, page_size=P, num_pages=total, fmt=st["cache"].fmt, **more).upload(dev)
        if case["rot"]:
            st["rope"] = bd.Rope(st["inv_freq"], interleaved=case["pairs"])
        if op == "sparse":
            st["block_bounds"] = bd.BlockBounds(st["bounds"], st["bounds_exp"])
        if op in ("attn", "step", "sparse"):
            st["workspace"] = torch.empty(bd.bd_paged_attn_workspace(st["plan"]), device=dev, dtype=torch.uint8)
    return st


# ------------------------------------------------------------------ the framework's calls

def _run_own(st):
    import block_causal_varlen_gb300 as bd

    op = st["case"]["op"]
    if op == "write":
        bd.bd_cache_write(st["plan"], st["k_new"], st["v_new"], st["cache"])
    if op in ("append", "step"):
        bd.bd_cache_append(st["plan"], st["q"], st["k_new"], st["v_new"], st["rope"], st["cache"], st["q_turned"])
    if "k_out" in st:
        bd.bd_cache_read(st["plan"], st["cache"], st["k_out"], st["v_out"])
    if op in ("attn", "step"):
        q = st["q"] if op == "attn" else st["q_turned"]
        bd.bd_paged_attn(st["plan"], q, st["cache"], st["out"], st["lse"], st["workspace"])
    if op == "sparse":
        bd.bd_block_bounds(st["plan"], st["cache"], st["block_bounds"])
        bd.bd_block_select(st["plan"], st["q"], st["block_bounds"], st["blocks"])
        bd.bd_sparse_attn(st["plan"], st["q"], st["cache"], st["blocks"], st["out"], st["lse"], st["workspace"])


# ------------------------------------------------------------------ the plain form

def _turn(st, x, pos):
    """Rows x [T, heads, d] turned by their positions (angles, and values next to a rounding's border: 64 bits)."""
    r = st["case"]["rot"]
    a = pos.double()[:, None] * st["inv_freq"].double()
    c, s = a.cos()[:, None], a.sin()[:, None]
    y = x.double()
    if st["case"]["pairs"]:
        u, v = y[..., 0:r:2], y[..., 1:r:2]
        t = torch.stack([u * c - v * s, v * c + u * s], -1).flatten(-2)
    else:
        u, v = y[..., :r // 2], y[..., r // 2:r]
        t = torch.cat([u * c - v * s, v * c + u * s], -1)
    return torch.cat([t, y[..., r:]], -1).to(torch.bfloat16)


def _places(st, key, pos):
    P = st["case"]["page"]
    return st["table"][st[key + "_seq"], pos // P], pos % P


def _padded_q(st, x):
    """Rows [T, heads, ...] padded to the longest chunk: [B, max_q, heads, ...]."""
    q = torch.zeros(st["case"]["B"], st["max_q"], *x.shape[1:], device=x.device, dtype=x.dtype)
    q[st["new_seq"], st["new_idx"]] = x
    return q


def _softmax_sum(s, v):
    """exp(s - max) v / sum and log sum exp(s) over the last axis of s, 0 and -inf where there is nothing."""
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    return (p @ v) / torch.where(total == 0, 1.0, total), (m + total.log())[..., 0]


def _attend(st, q):
    case = st["case"]
    B, H, Hkv, d, P = case["B"], case["H"], case["Hkv"], case["d"], case["page"]
    G, nq = H // Hkv, st["max_q"]
    q = _padded_q(st, q.float()).view(B, nq, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * nq, d)
    k, v = (_load(st, n, st["table"], slice(None)).flatten(1, 2)[:, :st["max_kv"]].transpose(1, 2) for n in ("k", "v"))
    s = (q @ k.transpose(2, 3)).mul_(1 / math.sqrt(d)).view(B, Hkv, G, nq, -1)
    i = torch.arange(nq, device=s.device)[None, :, None]
    j = torch.arange(s.shape[-1], device=s.device)[None, None, :]
    last = (st["kv_len"] - st["q_len"])[:, None, None] + i
    s.masked_fill_((j > last)[:, None, None], -math.inf)
    o, lse = _softmax_sum(s.view(B, Hkv, G * nq, -1), v)
    st["out"].copy_(o.view(B, Hkv, G, nq, d).permute(0, 3, 1, 2, 4).reshape(B, nq, H, d)[st["new_seq"], st["new_idx"]])
    st["lse"].copy_(lse.view(B, H, nq).permute(1, 0, 2)[:, st["new_seq"], st["new_idx"]])


def _select(st, pos):
    """The blocks of every new row and K/V head."""
    case = st["case"]
    B, H, Hkv, d, P, n = case["B"], case["H"], case["Hkv"], case["d"], case["page"], case["blocks"]
    G, nq = H // Hkv, st["max_q"]
    x = st["q"].float()
    eq = _pow8(x.abs().amax(-1))                                        # [T, H]
    x = _padded_q(st, (x * _pow2(-eq)[..., None]).round().clamp(-127, 127))
    x = x.view(B, nq, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * nq, d)
    b = st["bounds"][st["table"]].float()                               # [B, blocks, Hkv, 2, d]
    lo, hi = b[:, :, :, 0].permute(0, 2, 3, 1), b[:, :, :, 1].permute(0, 2, 3, 1)
    s = x.clamp(min=0) @ hi + x.clamp(max=0) @ lo                       # whole numbers below 2^24
    s = s.view(B, Hkv, G, nq, -1)[st["new_seq"], :, :, st["new_idx"]]   # [T, Hkv, G, blocks]
    eb = st["bounds_exp"][st["table"]].int() - 127                      # [B, blocks, Hkv]
    e = eq.view(-1, Hkv, G, 1) + eb.transpose(1, 2)[st["new_seq"]][:, :, None]
    s = (s * _pow2(e)).amax(2)
    j, last = torch.arange(s.shape[-1], device=s.device), (pos // P)[:, None, None]
    s = s.masked_fill((j < case["first"]) | (j > last - case["recent"]), math.inf).masked_fill(j > last, -math.inf)
    at = s.sort(dim=-1, descending=True, stable=True)[1][..., :n]
    at = torch.where(at > last, s.shape[-1], at).sort(-1)[0]            # what is not there goes to the end
    at = torch.where(at == s.shape[-1], -1, at)
    st["blocks"].fill_(-1)
    st["blocks"][..., :at.shape[-1]] = at


def _attend_blocks(st, pos):
    case = st["case"]
    H, Hkv, d, P = case["H"], case["Hkv"], case["d"], case["page"]
    T, at = len(pos), st["blocks"].long()
    page = st["table"][st["new_seq"][:, None, None], at.clamp(min=0)]                # [T, Hkv, n]
    rows = torch.arange(P, device=page.device)
    heads = torch.arange(Hkv, device=page.device)[:, None, None]

    def gathered(name):
        fmt, x = case["fmt"], st[name].view(torch.uint8) if case["fmt"] != "bf16" else st[name]
        c = x[page[..., None], rows, heads]                                         # [T, Hkv, n, P, ...]
        if fmt == "bf16":
            c = c.float()
        else:
            s = st[name + "_s"][page[..., None], rows, heads]
            c = _values4(c, s) if fmt == "e2m1" else c.view(torch.float8_e4m3fn).float() * _pow2(s.int() - 127)[..., None]
        return c.flatten(2, 3)

    s = (st["q"].float().view(T, Hkv, H // Hkv, d) @ gathered("k").transpose(2, 3)).mul_(1 / math.sqrt(d))
    there = (at[..., None] >= 0) & (at[..., None] * P + rows <= pos[:, None, None, None])
    s.masked_fill_(~there.flatten(2)[:, :, None], -math.inf)
    o, lse = _softmax_sum(s, gathered("v"))
    st["out"].copy_(o.reshape(T, H, d))
    st["lse"].copy_(lse.reshape(T, H).t())


def _run_plain(st):
    op = st["case"]["op"]
    if op != "read":
        pos = st["kv_len"][st["new_seq"]] - st["q_len"][st["new_seq"]] + st["new_idx"]
        place = _places(st, "new", pos)
    q = st.get("q")
    if op in ("append", "step"):
        q = _turn(st, q, pos)
        st["q_turned"].copy_(q)
        _store(st, "k", *place, _turn(st, st["k_new"], pos))
        _store(st, "v", *place, st["v_new"])
    if op == "write":
        _store(st, "k", *place, st["k_new"])
        _store(st, "v", *place, st["v_new"])
    if "k_out" in st:
        place = _places(st, "row", st["row_idx"])
        st["k_out"].copy_(_load(st, "k", *place))
        st["v_out"].copy_(_load(st, "v", *place))
    if op in ("attn", "step"):
        _attend(st, q)
    if op == "sparse":
        k = _load(st, "k", st["touched"], slice(None))
        st["bounds"][st["touched"]], st["bounds_exp"][st["touched"]] = _bounds_of(k, st["touched_rows"])
        _select(st, pos)
        _attend_blocks(st, pos)


def run(st):
    if own:
        _run_own(st)
    else:
        _run_plain(st)
    op = st["case"]["op"]
    names = {"write": ("k", "v", "k_s", "v_s"), "read": ("k_out", "v_out"), "attn": ("out", "lse"), "step": ("out", "lse", "q_turned"),
             "append": ("q_turned",) + (("k_out", "v_out") if "k_out" in st else ("k", "v")),
             "sparse": ("out", "lse", "blocks", "bounds", "bounds_exp")}[op]
    return {n: st[n] for n in names}


# ------------------------------------------------------------------ from the definitions, in 64 bits

def _powers(lo, hi, device):
    """2^lo .. 2^hi in 64 bits, not by the device's pow."""
    return torch.tensor([2.0 ** e for e in range(lo, hi + 1)], device=device, dtype=torch.float64)


# the magnitudes of the codes in their order
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
_E4M3 = [m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127]


def _nearest(y, grid):
    """Codes of the nearest magnitudes of `grid` to y >= 0 (ties to the even code)."""
    grid = torch.tensor(grid, device=y.device, dtype=torch.float64)
    mid = (grid[1:] + grid[:-1]) / 2
    lo, hi = torch.searchsorted(mid, y), torch.searchsorted(mid, y, right=True)   # differ at a tie
    code = torch.where(lo % 2 == 0, lo, hi)
    return code, grid[code]


def _exact_store(x, fmt):
    """(values, scale bytes, e2m1 codes) that rows x [..., d] of 64 bits are stored as."""
    x = x.to(torch.bfloat16).double()
    if fmt == "e4m3":
        top = x.abs().amax(-1, keepdim=True)
        powers = _powers(-60, 60, x.device)
        e = (top > 448.0 * powers).sum(-1).clamp(max=120) - 60
        s = powers[e + 60][..., None]
        return torch.copysign(_nearest(x.abs() / s, _E4M3)[1], x) * s, e + 127, None
    g = x.unflatten(-1, (-1, 16))
    top, byte = g.abs().amax(-1), torch.full(g.shape[:-1], 8, device=x.device)
    for b in range(8, 226):
        byte += top > 6 * (1 + b % 8 / 8) * 2.0 ** (b // 8 - 15)
    s = ((1 + (byte % 8).double() / 8) * _powers(-15, 16, x.device)[torch.div(byte, 8, rounding_mode="floor")])[..., None]
    code, mag = _nearest(g.abs() / s, _E2M1)
    return (torch.copysign(mag, g) * s).flatten(-2), byte, (code + 8 * torch.signbit(g)).flatten(-2)


def _exact_cached(st, page, row, name):
    """Cached rows as they stand, in 64 bits."""
    fmt, x = st["case"]["fmt"], st[name]
    if fmt == "bf16":
        return x[page, row].double()
    s = st[name + "_s"][page, row].long()
    c = x.view(torch.uint8)[page, row]
    if fmt == "e4m3":
        return c.view(torch.float8_e4m3fn).double() * _powers(-127, 128, c.device)[s][..., None]
    grid = torch.tensor(_E2M1 + [-m for m in _E2M1], device=c.device, dtype=torch.float64)
    y = torch.empty(*c.shape[:-1], 2 * c.shape[-1], device=c.device, dtype=torch.float64)
    y[..., 0::2], y[..., 1::2] = grid[c.long() % 16], grid[c.long() // 16]
    return y * ((1 + (s % 8).double() / 8) * _powers(-15, 16, c.device)[torch.div(s, 8, rounding_mode="floor")]).repeat_interleave(16, -1)


def _exact_turn(x, pos, inv_freq, r, pairs):
    """Each pair as a complex number times e^(i p f), in 64 bits."""
    y = x.double().clone()
    a, b = (slice(0, r, 2), slice(1, r, 2)) if pairs else (slice(0, r // 2), slice(r // 2, r))
    angle = torch.outer(pos.double(), inv_freq.double())[:, None]
    z = torch.complex(y[..., a], y[..., b]) * torch.polar(torch.ones_like(angle), angle)
    y[..., a], y[..., b] = z.real, z.imag
    return y


def _exact_attend(q, K, V, hidden):
    """O and LSE of q [n, d] over K, V [m, d]."""
    s = torch.where(hidden, -math.inf, q @ K.t() / math.sqrt(q.shape[-1]))
    z = torch.logsumexp(s, -1)
    return torch.exp(s - z[:, None]) @ V, z


def _exact_blocks(q, lo, hi, eb, last, case):
    """The blocks of one row and K/V head: q [G, d] and the bounds of blocks 0..last in 64 bits."""
    n = last + 1
    if n <= case["blocks"]:
        return list(range(n))
    powers = _powers(-50, 50, q.device)
    eq = (q.abs().amax(-1, keepdim=True) > 127 * powers).sum(-1).clamp(max=100)
    c = torch.round(q / powers[eq][:, None]).clamp(-127, 127)
    s = torch.maximum(c[:, None] * lo, c[:, None] * hi).sum(-1) * powers[eq][:, None] * powers[eb + 50]
    s = s.amax(0).tolist()
    keep = set(range(case["first"])) | set(range(n - case["recent"], n))
    order = sorted((j for j in range(n) if j not in keep), key=lambda j: (-s[j], j))
    return sorted(keep | set(order[:case["blocks"] - len(keep)]))


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    q, kv = lengths(case)
    B, H, Hkv, d, P, op, fmt = (case[n] for n in ("B", "H", "Hkv", "d", "page", "op", "fmt"))
    dev, at, want = st["table"].device, np.cumsum([0] + q), {}
    if op == "sparse" and sum(q) * Hkv > 3000:
        return None

    def where(b, n):
        p = torch.arange(n, device=dev)
        return st["table"][b][torch.div(p, P, rounding_mode="floor")], torch.remainder(p, P)

    if op in ("append", "step", "write"):
        stored = {n: st[n].double() if fmt == "bf16" else None for n in ("k", "v")}
        bits = {n: [st[n].clone(), st[n + "_s"].clone()] for n in ("k", "v")} if op == "write" else None
        rows = {"k": [], "v": []}
        turned = torch.zeros(sum(q), H, d, device=dev, dtype=torch.float64)
        for b in range(B):
            page, row = where(b, kv[b])
            pos = torch.arange(kv[b] - q[b], kv[b], device=dev)
            for name in ("k", "v"):
                x = st[name + "_new"][at[b]:at[b + 1]]
                if op != "write" and name == "k":
                    x = _exact_turn(x, pos, st["inv_freq"], case["rot"], case["pairs"])
                if fmt == "bf16":
                    stored[name][page[kv[b] - q[b]:], row[kv[b] - q[b]:]] = x.double()
                    continue
                x, s, c = _exact_store(x.double(), fmt)
                if op == "write":
                    bits[name][0][page[kv[b] - q[b]:], row[kv[b] - q[b]:]] = (c[..., 0::2] + 16 * c[..., 1::2]).to(torch.uint8)
                    bits[name][1][page[kv[b] - q[b]:], row[kv[b] - q[b]:]] = s.to(torch.uint8)
                else:
                    full = _exact_cached(st, page, row, name)
                    full[kv[b] - q[b]:] = x
                    rows[name].append(full)
            if op != "write":
                turned[at[b]:at[b + 1]] = _exact_turn(st["q"][at[b]:at[b + 1]], pos, st["inv_freq"], case["rot"], case["pairs"])
        if op == "write":
            return {"k": bits["k"][0], "v": bits["v"][0], "k_s": bits["k"][1], "v_s": bits["v"][1]}
        want["q_turned"] = turned
        if op == "append":
            # (a turned K next to the border of two codes has no value of its own in 8 or 4 bits: V has, and bf16 rows)
            want.update(stored if fmt == "bf16" else {"k_out": None, "v_out": torch.cat(rows["v"])})
            return want
    if op == "read":
        return {n + "_out": torch.cat([_exact_cached(st, *where(b, kv[b]), n) for b in range(B)]) for n in ("k", "v")}
    out = torch.zeros(sum(q), H, d, device=dev, dtype=torch.float64)
    lse = torch.full((H, sum(q)), -math.inf, device=dev, dtype=torch.float64)
    if op == "sparse":
        lists = torch.full((sum(q), Hkv, case["blocks"]), -1, dtype=torch.int32)
        bounds, bexp = st["bounds"].clone(), st["bounds_exp"].clone()
        powers = _powers(-50, 50, dev)
    for b in range(B):
        page, row = where(b, kv[b])
        if op == "step":
            K, V = rows["k"][b], rows["v"][b]
            Q = turned[at[b]:at[b + 1]].to(torch.bfloat16).double()
        else:
            K, V = _exact_cached(st, page, row, "k"), _exact_cached(st, page, row, "v")
            Q = st["q"][at[b]:at[b + 1]].double()
        if op != "sparse":
            hidden = torch.arange(kv[b], device=dev)[None] > kv[b] - q[b] + torch.arange(q[b], device=dev)[:, None]
            for h in range(H):
                out[at[b]:at[b + 1], h], lse[h, at[b]:at[b + 1]] = _exact_attend(Q[:, h], K[:, h * Hkv // H], V[:, h * Hkv // H], hidden)
            continue
        for j in range((kv[b] - q[b]) // P, (kv[b] - 1) // P + 1):
            x = K[j * P:min(kv[b], j * P + P)]
            lo, hi = x.min(0)[0], x.max(0)[0]
            e = (torch.maximum(lo.abs(), hi.abs()).amax(-1, keepdim=True) > 127 * powers).sum(-1).clamp(max=100)
            s = powers[e][:, None]
            n = int(st["table"][b, j])
            bounds[n, :, 0], bounds[n, :, 1] = (lo / s).floor().clamp(-127, 127).to(torch.int8), (hi / s).ceil().clamp(-127, 127).to(torch.int8)
            bexp[n] = (e + 77).to(torch.uint8)
        mine = st["table"][b][:-(-kv[b] // P)]
        B8, E8 = bounds[mine].double(), bexp[mine].long() - 127
        for i in range(q[b]):
            t, pos = at[b] + i, kv[b] - q[b] + i
            for g in range(Hkv):
                heads, m = slice(g * (H // Hkv), (g + 1) * (H // Hkv)), pos // P + 1
                pick = _exact_blocks(Q[i, heads], B8[:m, g, 0], B8[:m, g, 1], E8[:m, g], pos // P, case)
                lists[t, g, :len(pick)] = torch.tensor(pick, dtype=torch.int32)
                keys = (torch.tensor(pick, device=dev)[:, None] * P + torch.arange(P, device=dev)).flatten()
                keys = keys[keys <= pos]
                none = torch.zeros(1, 1, dtype=torch.bool, device=dev)
                out[t, heads], lse[heads, t] = _exact_attend(Q[i, heads], K[keys, g], V[keys, g], none)
    want.update({"out": out, "lse": lse})
    if op == "sparse":
        want.update({"blocks": lists.to(dev), "bounds": bounds, "bounds_exp": bexp})
    return want
