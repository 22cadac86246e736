"""Cases for the paged K/V cache: writing new rows into it, reading sequences back
out of it, and attention of a chunk of new rows (one row up to a whole prompt) over it.

The operators, for sequence b with q_b new rows of kv_b rows in the cache:

* write: row i of the sequence's new rows goes to cache position kv_b - q_b + i, i.e.
  to row ``position % page`` of the sequence's page ``position // page``. A bf16 cache
  holds the values; an e4m3 cache holds, for every (row, head), a power of two 2^e with
  e the smallest integer in [-60, 60] that has max|x| <= 448 2^e (60 where none has)
  and the codes rn(x 2^-e), saturating at 448; e is kept as the byte e + 127.
* read: rows [0, kv_b) of every sequence, packed back to back, as bf16.
* attention: new row i sees the cache positions j <= kv_b - q_b + i;
  O_i = sum_j softmax_j(q_i . k_j / sqrt(d)) v_j and LSE_i = log sum_j exp(q_i . k_j / sqrt(d)),
  query head h reading K/V head h // (H / Hkv). A row that sees nothing gives O = 0, LSE = -inf.
"""
import math
import random

import numpy as np
import torch

own = False


def _case(name, op, fmt, B, new, ctx, heads, page, heads_first=False, layout=1):
    """One case: `new` = (lo, hi) new rows of a sequence, `ctx` = (lo, hi) rows cached before
    them, heads = (H, Hkv, d)."""
    return {"name": name, "op": op, "fmt": fmt, "B": B, "new_lo": new[0], "new_hi": new[1], "ctx_lo": ctx[0],
            "ctx_hi": ctx[1], "H": heads[0], "Hkv": heads[1], "d": heads[2], "page": page,
            "heads_first": heads_first, "layout": layout}


def listed():
    return [
        # a decode step of a few sequences stores its one new row each: pure launch latency
        _case("write e4m3 step", "write", "e4m3", 8, (1, 1), (100, 8000), (32, 8, 128), 64),
        # packed prompts of a few hundred to two thousand rows enter a bf16 cache
        _case("write bf16 prompts", "write", "bf16", 6, (64, 2048), (0, 300), (32, 8, 128), 16),
        # a long prefill step enters an 8-bit cache, sequences continuing in the middle of a page
        _case("write e4m3 prompts", "write", "e4m3", 12, (500, 8000), (0, 3000), (32, 8, 128), 64, True),
        # a few short sequences of a small model leave the cache (moved to another worker, or recomputed from)
        _case("read bf16 short", "read", "bf16", 5, (0, 0), (17, 700), (4, 4, 64), 16),
        # one long document is read back from an 8-bit cache as bf16 rows
        _case("read e4m3 long", "read", "e4m3", 1, (0, 0), (49152, 49152), (32, 8, 128), 64, True),
        # a single user's decode step: little to read, latency counts
        _case("decode bf16 one", "attn", "bf16", 1, (1, 1), (4095, 4095), (32, 8, 128), 16),
        # a full decode batch with contexts of every length
        _case("decode bf16 batch", "attn", "bf16", 64, (1, 1), (500, 16000), (32, 8, 128), 64, True),
        # the same kind of batch over an 8-bit cache, two query heads to a K/V head
        _case("decode e4m3 batch", "attn", "e4m3", 64, (1, 1), (500, 16000), (16, 8, 128), 64),
        # a few drafted rows of each sequence are attended at once, head dim 256
        _case("drafts bf16 d256", "attn", "bf16", 16, (3, 6), (300, 8000), (32, 8, 256), 32, True),
        # one chunk of a long prompt over what is cached already
        _case("chunk bf16", "attn", "bf16", 1, (4096, 4096), (12288, 12288), (32, 8, 128), 64, True),
        # a serving step that mixes decode rows with prompt chunks, 8-bit cache
        _case("mixed e4m3", "attn", "e4m3", 10, (1, 1024), (60, 8000), (32, 8, 128), 64, False, 22),
        # small ragged chunks of a small model without grouped heads
        _case("chunk bf16 small", "attn", "bf16", 4, (30, 250), (0, 300), (4, 4, 64), 16),
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
MOST_PADDED = 64 * 16001 * 8 * 128      # values of K in a batch padded to its longest sequence
MOST_SCORES = 32 * 4096 * 16384         # scores of a batch padded to its longest chunk and sequence


def draw(rng):
    while True:
        op = rng.choice(["write", "read", "attn", "attn", "attn"])
        H, Hkv, d = rng.choice([(32, 8, 128), (16, 8, 128), (32, 8, 64), (4, 4, 64), (32, 8, 256), (10, 2, 128), (8, 1, 128),
                                (24, 8, 256)])
        B = _logint(rng, 1, 64)
        ctx_hi = _logint(rng, 1, 30000)
        ctx_lo = min(ctx_hi, _logint(rng, 1, 2000))
        if op == "read":
            new = (0, 0)
        elif rng.random() < 0.5:
            new = (1, rng.choice([1, 1, 1, 2, 5, 8]))
        else:
            hi = _logint(rng, 2, 4096)
            new = (_logint(rng, 1, hi), hi)
        c = _case("", op, rng.choice(["bf16", "e4m3"]), B, new, (ctx_lo, ctx_hi), (H, Hkv, d),
                  rng.choice([16, 32, 64, 128]), rng.random() < 0.5, rng.randrange(1 << 20))
        del c["name"]
        q, kv = lengths(c)
        if (2 * sum(kv) * Hkv * d <= MOST_CACHE and B * max(kv) * Hkv * d <= MOST_PADDED
                and (op != "attn" or B * H * max(q) * max(kv) <= MOST_SCORES)):
            return c


def _esize(case):
    return 2 if case["fmt"] == "bf16" else 1


def work(case):
    q, kv = lengths(case)
    H, Hkv, d = case["H"], case["Hkv"], case["d"]
    scale = 0 if case["fmt"] == "bf16" else 1
    cached = 2 * Hkv * (d * _esize(case) + scale)        # bytes of one row of K and V in the cache
    plain = 2 * Hkv * d * 2                              # and as bf16
    if case["op"] == "write":
        return {"bytes": sum(q) * (plain + cached), "flops": 0}
    if case["op"] == "read":
        return {"bytes": sum(kv) * (plain + cached), "flops": 0}
    pairs = sum(a * b - a * (a - 1) // 2 for a, b in zip(q, kv))
    return {"bytes": sum(kv) * cached + sum(q) * H * (2 * d * 2 + 4), "flops": 4 * d * H * pairs}


def quantise(x):
    """e4m3 codes and exponents of x [..., d], as defined at the top."""
    amax = x.float().abs().amax(-1)
    f, E = torch.frexp(amax)                             # amax = f 2^E, f in [0.5, 1); 448 = 0.875 2^9
    e = torch.where(amax == 0, -60, E - 9 + (f > 0.875)).clamp(-60, 60)
    y = torch.ldexp(x.float(), -e[..., None]).clamp(-448, 448)
    return y.to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def prepare(case, seed):
    q, kv = lengths(case)
    B, H, Hkv, d, P = case["B"], case["H"], case["Hkv"], case["d"], case["page"]
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    npages = [-(-n // P) for n in kv]
    total = sum(npages) + 3                              # a few pages belong to nobody
    order = np.random.default_rng(seed).permutation(total).astype(np.int32)
    cut = np.cumsum([0] + npages)
    pages = [order[cut[b]:cut[b + 1]] for b in range(B)]
    shape = (total, Hkv, P, d) if case["heads_first"] else (total, P, Hkv, d)

    def pool():
        x = torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)
        return x.transpose(1, 2) if case["heads_first"] else x       # [page, row, head, d] either way

    k, v = pool(), pool()
    st = {"case": case, "k": k, "v": v, "k_exp": None, "v_exp": None}
    if case["fmt"] == "e4m3":
        # rows of different sizes, so that every row has an exponent of its own
        for name, x in (("k", k), ("v", v)):
            mag = torch.exp2(torch.randint(-3, 4, x.shape[:3], generator=g, device=dev).float())
            x = x * (mag if name == "v" else mag.clamp(max=2))[..., None].to(x.dtype)
            st[name], st[name + "_exp"] = quantise(x)
    T = sum(q)
    if T:
        # the rows of a fused projection, as they come: the heads of q, then k, then v
        qkv = torch.randn(T, (H + 2 * Hkv) * d, generator=g, device=dev, dtype=torch.bfloat16)
        st["q"] = qkv[:, :H * d].view(T, H, d)
        st["k_new"] = qkv[:, H * d:(H + Hkv) * d].view(T, Hkv, d)
        st["v_new"] = qkv[:, (H + Hkv) * d:].view(T, Hkv, d)
    # where things are, for the plain form
    table = np.zeros((B, max(npages)), dtype=np.int64)
    for b in range(B):
        table[b, :npages[b]] = pages[b]
    st["table"] = torch.from_numpy(table).to(dev)
    st["q_len"], st["kv_len"] = torch.tensor(q, device=dev), torch.tensor(kv, device=dev)
    st["max_q"], st["max_kv"] = max(q), max(kv)
    seq = np.repeat(np.arange(B), q if T else kv)
    idx = np.concatenate([np.arange(n) for n in (q if T else kv)])
    st["seq"], st["idx"] = torch.from_numpy(seq).to(dev), torch.from_numpy(idx).to(dev)
    if case["op"] == "read":
        st["k_out"] = torch.empty(sum(kv), Hkv, d, device=dev, dtype=torch.bfloat16)
        st["v_out"] = torch.empty_like(st["k_out"])
    if case["op"] == "attn":
        st["out"] = torch.empty(T, H, d, device=dev, dtype=torch.bfloat16)
        st["lse"] = torch.empty(H, T, device=dev, dtype=torch.float32)
    if own:
        import block_causal_varlen_gb300 as bd

        st["cache"] = bd.PagedCache(st["k"], st["v"], st["k_exp"], st["v_exp"])
        st["plan"] = bd.PagedPlan(q, kv, pages, H, Hkv, d, page_size=P, num_pages=total, fmt=st["cache"].fmt).upload(dev)
        if case["op"] == "attn":
            st["workspace"] = torch.empty(bd.bd_paged_attn_workspace(st["plan"]), device=dev, dtype=torch.uint8)
    return st


def _rows(st, name):
    """Every sequence's cached rows in 32 bits, padded to the longest: [B, max_kv, Hkv, d]."""
    if st[name + "_exp"] is None:
        x = st[name][st["table"]].flatten(1, 2)[:, :st["max_kv"]].float()
    else:
        x = st[name].view(torch.uint8)[st["table"]].flatten(1, 2)[:, :st["max_kv"]].view(torch.float8_e4m3fn).float()
        e = st[name + "_exp"][st["table"]].flatten(1, 2)[:, :st["max_kv"]]
        x = torch.ldexp(x, (e.int() - 127)[..., None])
    return x


def _run_own(st):
    import block_causal_varlen_gb300 as bd

    op = st["case"]["op"]
    if op == "write":
        bd.bd_cache_write(st["plan"], st["k_new"], st["v_new"], st["cache"])
    elif op == "read":
        bd.bd_cache_read(st["plan"], st["cache"], st["k_out"], st["v_out"])
    else:
        bd.bd_paged_attn(st["plan"], st["q"], st["cache"], st["out"], st["lse"], st["workspace"])


def _run_plain(st):
    case = st["case"]
    op, P = case["op"], case["page"]
    if op == "write":
        pos = st["kv_len"][st["seq"]] - st["q_len"][st["seq"]] + st["idx"]
        page, row = st["table"][st["seq"], pos // P], pos % P
        for name in ("k", "v"):
            if case["fmt"] == "bf16":
                st[name][page, row] = st[name + "_new"]
            else:
                codes, e = quantise(st[name + "_new"])
                st[name].view(torch.uint8)[page, row] = codes.view(torch.uint8)
                st[name + "_exp"][page, row] = e
    elif op == "read":
        page, row = st["table"][st["seq"], st["idx"] // P], st["idx"] % P
        for name in ("k", "v"):
            x = st[name].view(torch.uint8 if case["fmt"] == "e4m3" else torch.bfloat16)[page, row]
            if case["fmt"] == "e4m3":
                x = torch.ldexp(x.view(torch.float8_e4m3fn).float(), (st[name + "_exp"][page, row].int() - 127)[..., None])
            st[name + "_out"].copy_(x)
    else:
        B, H, Hkv, d = case["B"], case["H"], case["Hkv"], case["d"]
        G, nq = H // Hkv, st["max_q"]
        q = torch.zeros(B, nq, H, d, device=st["q"].device)
        q[st["seq"], st["idx"]] = st["q"].float()
        q = q.view(B, nq, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * nq, d)
        k, v = _rows(st, "k").transpose(1, 2), _rows(st, "v").transpose(1, 2)
        s = (q @ k.transpose(2, 3)).mul_(1 / math.sqrt(d)).view(B, Hkv, G, nq, -1)
        i = torch.arange(nq, device=s.device)[None, :, None]
        j = torch.arange(s.shape[-1], device=s.device)[None, None, :]
        last = (st["kv_len"] - st["q_len"])[:, None, None] + i
        s.masked_fill_((j > last)[:, None, None], -math.inf)
        m = s.amax(-1, keepdim=True)
        m = torch.where(m == -math.inf, 0.0, m)
        p = s.sub_(m).exp_()
        total = p.sum(-1, keepdim=True)
        o = (p.view(B, Hkv, G * nq, -1) @ v).view(B, Hkv, G, nq, d) / torch.where(total == 0, 1.0, total)
        lse = (m + total.log())[..., 0]                                  # [B, Hkv, G, nq]
        st["out"].copy_(o.permute(0, 3, 1, 2, 4).reshape(B, nq, H, d)[st["seq"], st["idx"]])
        st["lse"].copy_(lse.permute(1, 2, 0, 3).reshape(H, B, nq)[:, st["seq"], st["idx"]])


def run(st):
    if own:
        _run_own(st)
    else:
        _run_plain(st)
    op = st["case"]["op"]
    if op == "write":
        return {n: st[n] for n in ("k", "v", "k_exp", "v_exp") if st[n] is not None}
    if op == "read":
        return {"k": st["k_out"], "v": st["v_out"]}
    return {"out": st["out"], "lse": st["lse"]}


def _positions(table, n, P):
    """Page and row of positions [0, n) of one sequence."""
    pos = torch.arange(n, device=table.device)
    return table[torch.div(pos, P, rounding_mode="floor")], torch.remainder(pos, P)


def _exact_rows(st, b, n, name):
    """Rows [0, n) of sequence b in 64 bits: [n, Hkv, d]."""
    page, row = _positions(st["table"][b], n, st["case"]["page"])
    if st[name + "_exp"] is None:
        return st[name][page, row].double()
    codes = st[name].view(torch.uint8)[page, row].view(torch.float8_e4m3fn).double()
    return codes * torch.pow(2.0, st[name + "_exp"][page, row].double() - 127.0)[..., None]


# the 127 finite e4m3 magnitudes, in the order of their codes
_GRID = [m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127]


def _exact_quantise(x):
    """The nearest code of every value from the list of all codes (ties to the even code)."""
    x = x.double()
    top = x.abs().amax(-1, keepdim=True)
    powers = torch.pow(2.0, torch.arange(-60, 61, device=x.device, dtype=torch.float64))
    e = (top > 448.0 * powers).sum(-1).clamp(max=120) - 60
    y = x.abs() / torch.pow(2.0, e.double())[..., None]
    grid = torch.tensor(_GRID, device=x.device, dtype=torch.float64)
    mid = (grid[1:] + grid[:-1]) / 2
    lo, hi = torch.searchsorted(mid, y), torch.searchsorted(mid, y, right=True)   # differ at a tie
    code = torch.where(lo % 2 == 0, lo, hi)
    return torch.copysign(grid[code], x), e + 127


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    q, kv = lengths(case)
    H, Hkv, d, P = case["H"], case["Hkv"], case["d"], case["page"]
    if case["op"] == "read":
        return {n: torch.cat([_exact_rows(st, b, kv[b], n) for b in range(case["B"])]) for n in ("k", "v")}
    at = np.cumsum([0] + q)
    if case["op"] == "write":
        want = {}
        for name in ("k", "v"):
            vals = st[name].double() if case["fmt"] == "bf16" else st[name].view(torch.uint8).clone().view(torch.float8_e4m3fn).double()
            exps = None if st[name + "_exp"] is None else st[name + "_exp"].clone()
            for b in range(case["B"]):
                page, row = _positions(st["table"][b], kv[b], P)
                page, row = page[kv[b] - q[b]:], row[kv[b] - q[b]:]
                x = st[name + "_new"][at[b]:at[b + 1]]
                if exps is None:
                    vals[page, row] = x.double()
                else:
                    y, e = _exact_quantise(x)
                    vals[page, row], exps[page, row] = y, e.to(torch.uint8)
            want[name] = vals
            if exps is not None:
                want[name + "_exp"] = exps
        return want
    out = torch.zeros(sum(q), H, d, device="cuda", dtype=torch.float64)
    lse = torch.full((H, sum(q)), -math.inf, device="cuda", dtype=torch.float64)
    for b in range(case["B"]):
        K, V = _exact_rows(st, b, kv[b], "k"), _exact_rows(st, b, kv[b], "v")
        seen = kv[b] - q[b] + 1 + torch.arange(q[b], device="cuda")      # keys that row i sees
        hidden = torch.arange(kv[b], device="cuda")[None] >= seen[:, None]
        for h in range(H):
            s = st["q"][at[b]:at[b + 1], h].double() @ K[:, h * Hkv // H].t() / math.sqrt(d)
            s = torch.where(hidden, -math.inf, s)
            z = torch.logsumexp(s, -1)
            out[at[b]:at[b + 1], h] = torch.exp(s - z[:, None]) @ V[:, h * Hkv // H]
            lse[h, at[b]:at[b + 1]] = z
    return {"out": out, "lse": lse}
