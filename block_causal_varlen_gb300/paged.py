"""Paged K/V cache: the binding of include/bd_paged.h.

Tensor layouts (all strided views are accepted; the head dim is contiguous):
    cache k, v     bf16 or e4m3 codes [pages, page_size, Hkv, d], or e2m1 codes, two a byte,
                   uint8 [pages, page_size, Hkv, d / 2]; either may be a view of a head-first
                   pool [pages, Hkv, page_size, ...]
    k_exp, v_exp   uint8 [pages, page_size, Hkv] exponents of an e4m3 cache, or
                   uint8 [pages, page_size, Hkv, d / 16] scales of an e2m1 cache
    q, out         bf16 [rows, H, d], rows >= T: the new rows of all sequences, packed
    k, v (new)     bf16 [rows, Hkv, d]
    lse            fp32 [H, rows]
    bounds         int8 [pages, Hkv, 2, d] and uint8 [pages, Hkv]: what block selection goes by
    blocks         int32 [rows, Hkv, blocks]: the blocks that a new row attends
"""
from __future__ import annotations

import ctypes as C
import struct

import numpy as np
import torch

from . import _abi
from ._abi import (BD_CACHE_BF16, BD_CACHE_E2M1, BD_CACHE_E4M3, bd_bounds, bd_paged_cache, bd_paged_desc, bd_rope,
                   bd_sparse_desc, bd_tensor, check, load)

__all__ = ["PagedCache", "PagedPlan", "bd_paged_plan_bytes", "bd_paged_plan_build", "bd_paged_plan_key",
           "bd_cache_write", "bd_cache_read", "bd_paged_attn_workspace", "bd_paged_attn", "paged_attn",
           "BD_CACHE_BF16", "BD_CACHE_E4M3", "BD_CACHE_E2M1", "Rope", "bd_rope_phases", "bd_cache_append",
           "bd_sparse_plan_bytes", "bd_sparse_plan_build", "BlockBounds", "bd_block_bounds", "bd_block_select",
           "bd_sparse_attn", "sparse_attn"]

_P32 = C.POINTER(C.c_int32)


def bd_paged_plan_bytes(desc: bd_paged_desc) -> int:
    """Bytes of the plan blob of a descriptor (validates it)."""
    n = C.c_size_t()
    check(load().bd_paged_plan_bytes(C.byref(desc), C.byref(n)))
    return n.value


def bd_paged_plan_build(desc: bd_paged_desc, blob_ptr: int, nbytes: int) -> None:
    """Build the plan blob into host memory at ``blob_ptr``."""
    check(load().bd_paged_plan_build(C.byref(desc), C.c_void_p(blob_ptr), nbytes))


def bd_sparse_plan_bytes(desc: bd_paged_desc, sparse: bd_sparse_desc) -> int:
    """Bytes of the plan blob of a sparse plan (validates both descriptors)."""
    n = C.c_size_t()
    check(load().bd_sparse_plan_bytes(C.byref(desc), C.byref(sparse), C.byref(n)))
    return n.value


def bd_sparse_plan_build(desc: bd_paged_desc, sparse: bd_sparse_desc, blob_ptr: int, nbytes: int) -> None:
    """Build the blob of a sparse plan into host memory at ``blob_ptr``."""
    check(load().bd_sparse_plan_build(C.byref(desc), C.byref(sparse), C.c_void_p(blob_ptr), nbytes))


class PagedCache:
    """One layer's K/V pool as the library takes it; the tensors' dtype says its format
    (bfloat16, float8_e4m3fn with exponents, uint8 with scales: e2m1). The tensors stay the
    caller's; they are kept alive here, and their addresses are fixed for this object."""

    def __init__(self, k, v, k_exp=None, v_exp=None):
        for t, n in ((k, "k"), (v, "v")):
            if t.dim() != 4 or t.stride(3) != 1:
                raise ValueError(f"cache {n}: expected [pages, page_size, Hkv, d] with d contiguous, got {tuple(t.shape)}")
        if v.shape != k.shape or v.dtype != k.dtype or v.device != k.device:
            raise ValueError("cache k and v differ in shape, dtype or device")
        if k.dtype == torch.bfloat16:
            self.fmt = BD_CACHE_BF16
            if k_exp is not None or v_exp is not None:
                raise ValueError("a bf16 cache has no exponents")
        elif k.dtype == torch.float8_e4m3fn:
            self.fmt = BD_CACHE_E4M3
            for t, n in ((k_exp, "k_exp"), (v_exp, "v_exp")):
                if t is None or t.dtype != torch.uint8 or t.shape != k.shape[:3] or t.device != k.device:
                    raise ValueError(f"{n}: an e4m3 cache needs uint8 exponents [pages, page_size, Hkv] on its device")
            if any(n > 1 and a != b for n, a, b in zip(k.shape, k_exp.stride(), v_exp.stride())):
                raise ValueError("k_exp and v_exp must have the same strides")
        elif k.dtype == torch.uint8:
            self.fmt = BD_CACHE_E2M1
            if k.shape[3] % 8:
                raise ValueError(f"cache of {k.shape[3]} bytes of codes a head, expected half of a head dim of 64, 128 or 256")
            for t, n in ((k_exp, "k_exp"), (v_exp, "v_exp")):
                if (t is None or t.dtype != torch.uint8 or t.shape != (*k.shape[:3], k.shape[3] // 8) or t.device != k.device
                        or t.stride(3) != 1):
                    raise ValueError(f"{n}: an e2m1 cache needs uint8 scales [pages, page_size, Hkv, d / 16] on its device, "
                                     "those of a head contiguous")
            if any(n > 1 and a != b for n, a, b in zip(k.shape[:3], k_exp.stride(), v_exp.stride())):
                raise ValueError("k_exp and v_exp must have the same strides")
        else:
            raise TypeError(f"cache dtype {k.dtype}, expected bfloat16, float8_e4m3fn or uint8 (e2m1 codes)")
        self.k, self.v, self.k_exp, self.v_exp = k, v, k_exp, v_exp
        self.num_pages, self.page_size, self.Hkv, self.d = k.shape
        if self.fmt == BD_CACHE_E2M1:
            self.d *= 2
        self.device = k.device
        st = [bd_tensor(t.data_ptr(), t.stride(0), 0, t.stride(1), t.stride(2), t.shape[1], 0) for t in (k, v)]
        es = k_exp.stride() if k_exp is not None else (0, 0, 0)
        ep = [t.data_ptr() if t is not None else None for t in (k_exp, v_exp)]
        self._c = bd_paged_cache(st[0], st[1], ep[0], ep[1], es[0], es[1], es[2], self.fmt, self.num_pages)
        self._addr = C.addressof(self._c)
        self._index = k.get_device()


def _ints(x, name):
    """x as int32, if it is whole numbers in range."""
    a = np.asarray(x)
    if a.size and (a.dtype.kind not in "iu" or a.min() < -2 ** 31 or a.max() >= 2 ** 31):
        raise ValueError(f"{name}: expected whole numbers of 32 bits")
    return np.ascontiguousarray(a, dtype=np.int32)


def _int(x, name):
    if type(x) is int and 0 <= x < 2 ** 31:
        return x
    if np.ndim(x) != 0:
        raise ValueError(f"{name}: expected one number")
    return int(_ints(x, name)[0])


def _placed(device):
    """``device`` as tensors on it say it: "cuda" is the current device."""
    device = torch.device(device)
    if device.type == "cuda" and device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    return device


class PagedPlan:
    """Host plan blob of one step over a paged cache, and its device copy.

    ``q_len``, ``kv_len``: new rows of every sequence, and its cached rows with them;
    ``pages``: a page list per sequence, or an integer table [B, max_pages]. With ``blocks``
    the plan is a sparse one: every new row attends that many blocks (pages) of its sequence,
    the ``first`` and the ``recent`` last ones always among them (bd_block_select,
    bd_sparse_attn).
    """

    def __init__(self, q_len, kv_len, pages, H, Hkv, d, page_size, num_pages, fmt=BD_CACHE_BF16, causal=True, blocks=0,
                 first=0, recent=1):
        q, kv = _ints(q_len, "q_len"), _ints(kv_len, "kv_len")
        H, Hkv, d, fmt = _int(H, "H"), _int(Hkv, "Hkv"), _int(d, "d"), _int(fmt, "fmt")
        page_size, num_pages = _int(page_size, "page_size"), _int(num_pages, "num_pages")
        if q.ndim != 1 or q.shape != kv.shape or len(pages) != len(q):
            raise ValueError("q_len, kv_len and pages must have one entry per sequence")
        if isinstance(pages, np.ndarray) and pages.ndim == 2:
            flat = _ints(pages, "pages").reshape(-1)
            offs = np.arange(len(q) + 1, dtype=np.int64) * pages.shape[1]
        else:
            lists = [np.asarray(x).reshape(-1) for x in pages]
            offs = np.cumsum([0] + [x.size for x in lists])
            some = [x for x in lists if x.size]
            flat = _ints(np.concatenate(some) if some else (), "pages")
        if offs[-1] >= 2 ** 31:
            raise ValueError("page lists of more than 2^31 entries")
        offs = np.ascontiguousarray(offs, dtype=np.int32)
        self.B, self.H, self.Hkv, self.d = len(q), H, Hkv, d
        self.page_size, self.num_pages, self.fmt, self.causal = page_size, num_pages, fmt, bool(causal)
        self.T, self.kv_total = int(q.sum(dtype=np.int64)), int(kv.sum(dtype=np.int64))
        desc = bd_paged_desc(self.B, H, Hkv, d, page_size, num_pages, fmt, int(self.causal), q.ctypes.data_as(_P32),
                             kv.ctypes.data_as(_P32), flat.ctypes.data_as(_P32), offs.ctypes.data_as(_P32))
        self.blocks = _int(blocks, "blocks")
        first, recent = _int(first, "first"), _int(recent, "recent")
        if not self.blocks and (first, recent) != (0, 1):
            raise ValueError("first and recent are of a sparse plan: build it with blocks=...")
        sparse = bd_sparse_desc(self.blocks, first, recent, 0) if self.blocks else None
        self.nbytes = bd_sparse_plan_bytes(desc, sparse) if sparse else bd_paged_plan_bytes(desc)
        self._raw = np.empty(self.nbytes // 4 + 16, dtype=np.int32)
        off = (-self._raw.ctypes.data % 64) // 4
        self.host = self._raw[off:off + self.nbytes // 4]
        if sparse:
            bd_sparse_plan_build(desc, sparse, self.host.ctypes.data, self.nbytes)
        else:
            bd_paged_plan_build(desc, self.host.ctypes.data, self.nbytes)
        self.host = self.host[:int(self.host[2])]       # the words in use (csrc/paged_plan.h: PH_WORDS)
        self._host_ptr = self.host.ctypes.data
        self.dev = self._dev_ptr = None
        self._index, self._own = -1, False
        self._streams = set()       # raw streams that the allocator knows to use the plan's own memory
        ws = C.c_size_t()
        check(load().bd_paged_attn_workspace(self._host_ptr, C.byref(ws)))
        self._workspace = ws.value

    @property
    def host_ptr(self):
        return C.c_void_p(self._host_ptr)

    @property
    def dev_ptr(self):
        if self._dev_ptr is None:
            raise RuntimeError("plan not uploaded: call .upload(device)")
        return C.c_void_p(self._dev_ptr)

    def upload(self, device="cuda", non_blocking=False, buffer=None):
        """Copy the plan blob to device memory (once per step): into memory of its own,
        or into ``buffer``, an int32 device tensor that a captured graph reads (see
        bd_paged_plan_key; nbytes / 4 words always suffice). Memory of its own stays the
        plan's until the calls made with it have run, on whichever streams; ``buffer`` is
        the caller's to keep, and so is a plan whose own memory a captured graph reads."""
        src = torch.from_numpy(self.host)
        if buffer is not None:
            if buffer.dtype != torch.int32 or buffer.dim() != 1 or not buffer.is_contiguous() or not buffer.is_cuda:
                raise TypeError("buffer: expected a contiguous 1-D int32 CUDA tensor")
            if buffer.numel() < src.numel():
                raise ValueError(f"buffer of {buffer.numel()} words, the plan has {src.numel()}")
            self.dev, self._own = buffer[:src.numel()], False
        elif not self._own or self.dev.device != _placed(device):
            self.dev, self._own = torch.empty_like(src, device=device), True
            self._streams = {_raw_stream(self.dev.get_device())} if self.dev.is_cuda else set()
        self._dev_ptr, self._index = self.dev.data_ptr(), self.dev.get_device()
        if self.dev.is_cuda:
            self._used_on(_raw_stream(self._index), None)
        self.dev.copy_(src, non_blocking=non_blocking)
        return self

    def _used_on(self, raw, stream):
        """Work is about to be queued on ``stream`` (None: the current one) that uses the device
        copy: its own memory is not to be given to others before that has run."""
        if self._own and raw not in self._streams:
            self.dev.record_stream(torch.cuda.current_stream(self._index) if stream is None else stream)
            self._streams.add(raw)

    def key(self) -> int:
        """See bd_paged_plan_key."""
        return bd_paged_plan_key(self)


def bd_paged_plan_key(plan: PagedPlan) -> int:
    """Plans of equal keys may replace each other under a captured graph (see
    include/bd_paged.h)."""
    n = C.c_uint64()
    check(load().bd_paged_plan_key(plan._host_ptr, C.byref(n)))
    return n.value


def bd_paged_attn_workspace(plan: PagedPlan) -> int:
    """Workspace bytes of bd_paged_attn."""
    return plan._workspace


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


# The device calls take their structs as packed bytes and every pointer as an address: half
# the binding's cost of a small call otherwise goes into ctypes structures.
_tensor = struct.Struct("PqqqqiI").pack        # bd_tensor
_rowstat = struct.Struct("Pqqq").pack          # bd_rowstat
_entries = {}
_BF16 = torch.bfloat16


def _entry(name):
    f = _entries.get(name)
    if f is None:
        lib = load()
        f = lib[name]  # a function object of its own
        args = getattr(lib, name).argtypes
        f.restype, f.argtypes = C.c_int32, [C.c_size_t if a is C.c_size_t else C.c_void_p for a in args]
        _entries[name] = f
    return f


def _refuse(t, name, dtype, idx):
    """Says what is wrong with a tensor's type or place."""
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if not t.is_cuda:
        raise TypeError(f"{name}: must be a CUDA tensor")
    raise ValueError(f"{name}: on {t.device}, the plan was uploaded to cuda:{idx}")


def _rows3(t, name, heads, d, rows, idx):
    """A packed [rows, heads, d] bf16 tensor as the ABI's strided tensor (its bytes). The C ABI
    carries neither dtypes nor head counts, so they are checked here."""
    if t.dtype is not _BF16 or t.get_device() != idx or idx < 0:
        _refuse(t, name, _BF16, idx)
    n, h, c = t.shape if t.dim() == 3 else (-1, 0, 0)
    if h != heads or c != d or n < rows:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected [{rows} or more, {heads}, {d}]")
    row, head, one = t.stride()
    if one != 1:
        raise ValueError(f"{name}: head dim must be contiguous")
    return _tensor(t.data_ptr(), 0, 0, row, head, n, 0)


def _device(plan, cache):
    """The device of a call: that of the plan's device copy, which must be the cache's
    (heads and head dim of the cache are checked too; the ABI does not carry them)."""
    if plan._dev_ptr is None:
        raise RuntimeError("plan not uploaded: call .upload(device)")
    if cache._index != plan._index:
        raise ValueError(f"cache: on {cache.device}, the plan was uploaded to {plan.dev.device}")
    if cache.Hkv != plan.Hkv or cache.d != plan.d:
        raise ValueError(f"cache of {cache.Hkv} heads of {cache.d}, the plan was built for {plan.Hkv} of {plan.d}")
    return plan._index


def _call(fn, plan, idx, stream, *args):
    s = _raw_stream(idx) if stream is None else stream.cuda_stream
    plan._used_on(s, stream)
    if torch.cuda.current_device() == idx:
        st = fn(*args, s)
    else:
        with torch.cuda.device(idx):
            st = fn(*args, s)
    if st < 0:
        check(st)


def bd_cache_write(plan: PagedPlan, k, v, cache: PagedCache, stream=None):
    """Store the new rows' K and V at their cache positions (see include/bd_paged.h)."""
    idx = _device(plan, cache)
    tk = _rows3(k, "k", plan.Hkv, plan.d, plan.T, idx)
    tv = _rows3(v, "v", plan.Hkv, plan.d, plan.T, idx)
    _call(_entry("bd_cache_write"), plan, idx, stream, plan._host_ptr, plan._dev_ptr, tk, tv, cache._addr)


def bd_rope_phases(inv_freq) -> np.ndarray:
    """Frequencies (radians a position, host numbers) as the kernels take them: uint64 turns a
    position, modulo 1, in units of 2^-64 (see include/bd_paged.h)."""
    f = np.ascontiguousarray(inv_freq, dtype=np.float64).reshape(-1)
    out = np.empty(f.size, dtype=np.uint64)
    check(load().bd_rope_phases(f.ctypes.data_as(C.POINTER(C.c_double)), f.size, out.ctypes.data_as(C.POINTER(C.c_uint64))))
    return out


class Rope:
    """A position rotation of the first 2 * len(inv_freq) elements of a head: pair i turns by
    inv_freq[i] radians a position. ``interleaved``: pairs (2 i, 2 i + 1) instead of
    (i, i + len(inv_freq)); ``scale``: a factor of the turned elements. Made once (the
    frequencies go through host memory), for the device of ``inv_freq`` or ``device``. Its
    memory stays its own until the calls made with it have run, on whichever streams; what a
    captured graph uses is the caller's to keep."""

    def __init__(self, inv_freq, interleaved=False, scale=1.0, device=None):
        if isinstance(inv_freq, torch.Tensor):
            device = inv_freq.device if device is None else device
            inv_freq = inv_freq.detach().double().cpu().numpy()
        if np.ndim(inv_freq) != 1 or np.size(inv_freq) == 0:
            raise ValueError("inv_freq: expected a vector, one frequency for each pair")
        phase = bd_rope_phases(inv_freq)
        self.dim, self.interleaved, self.scale = 2 * phase.size, bool(interleaved), float(scale)
        self.phase = torch.from_numpy(phase.view(np.int64)).to("cuda" if device is None else device)
        self._c = bd_rope(self.phase.data_ptr(), self.dim, int(self.interleaved), self.scale, 0)
        self._addr = C.addressof(self._c)
        self._index = self.phase.get_device()
        self._streams = {_raw_stream(self._index)} if self.phase.is_cuda else set()   # that the allocator knows

    def _used_on(self, raw, stream):
        """As PagedPlan._used_on."""
        if raw not in self._streams:
            self.phase.record_stream(torch.cuda.current_stream(self._index) if stream is None else stream)
            self._streams.add(raw)


def bd_cache_append(plan: PagedPlan, q, k, v, rope: Rope, cache: PagedCache, q_out=None, stream=None):
    """bd_cache_write of K turned by its positions, and of V as it is; q (or None) turned into
    q_out, which may be q itself (see include/bd_paged.h)."""
    idx = _device(plan, cache)
    if rope._index != idx:
        raise ValueError(f"rope: on {rope.phase.device}, the plan was uploaded to cuda:{idx}")
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out come together")
    tq = _rows3(q, "q", plan.H, plan.d, plan.T, idx) if q is not None else None
    to = _rows3(q_out, "q_out", plan.H, plan.d, plan.T, idx) if q is not None else None
    tk = _rows3(k, "k", plan.Hkv, plan.d, plan.T, idx)
    tv = _rows3(v, "v", plan.Hkv, plan.d, plan.T, idx)
    rope._used_on(_raw_stream(idx) if stream is None else stream.cuda_stream, stream)
    _call(_entry("bd_cache_append"), plan, idx, stream, plan._host_ptr, plan._dev_ptr, tq, tk, tv, rope._addr, cache._addr, to)


def bd_cache_read(plan: PagedPlan, cache: PagedCache, k, v, stream=None):
    """The cached rows of every sequence, packed in batch order (see include/bd_paged.h)."""
    idx = _device(plan, cache)
    tk = _rows3(k, "k", plan.Hkv, plan.d, plan.kv_total, idx)
    tv = _rows3(v, "v", plan.Hkv, plan.d, plan.kv_total, idx)
    _call(_entry("bd_cache_read"), plan, idx, stream, plan._host_ptr, plan._dev_ptr, cache._addr, tk, tv)


def _attend(name, plan, q, cache, out, lse, workspace, stream, *more):
    idx = _device(plan, cache)
    tq = _rows3(q, "q", plan.H, plan.d, plan.T, idx)
    to = _rows3(out, "out", plan.H, plan.d, plan.T, idx)
    tl = None
    if lse is not None:
        if lse.dtype is not torch.float32 or lse.get_device() != idx:
            _refuse(lse, "lse", torch.float32, idx)
        s = lse.shape
        if len(s) != 2 or s[0] != plan.H or s[1] < plan.T or (s[1] > 1 and lse.stride(1) != 1):
            raise ValueError(f"lse: expected [{plan.H}, {plan.T} or more] with rows contiguous, got {tuple(s)}")
        tl = _rowstat(lse.data_ptr(), 0, 0, lse.stride(0))
    wp, wn = None, 0
    if workspace is None and plan._workspace:
        with torch.cuda.stream(stream):      # memory of the stream that uses it
            workspace = torch.empty(plan._workspace, dtype=torch.uint8, device=plan.dev.device)
    if workspace is not None:
        if workspace.get_device() != idx:
            raise ValueError(f"workspace: on {workspace.device}, the plan was uploaded to cuda:{idx}")
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        wp, wn = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _call(_entry(name), plan, idx, stream, plan._host_ptr, plan._dev_ptr, tq, cache._addr, *more, to, tl, wp, wn)


def bd_paged_attn(plan: PagedPlan, q, cache: PagedCache, out, lse=None, workspace=None, stream=None):
    """O and LSE of the new rows over the cache (see include/bd_paged.h). Without a
    workspace one is allocated for the call."""
    _attend("bd_paged_attn", plan, q, cache, out, lse, workspace, stream)


def _outputs(plan, q, stream):
    with torch.cuda.stream(stream):      # memory of the stream that writes it
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        lse = torch.empty(plan.H, q.shape[0], dtype=torch.float32, device=q.device)
        blocks = torch.empty(q.shape[0], plan.Hkv, plan.blocks, dtype=torch.int32, device=q.device) if plan.blocks else None
    if stream is not None:
        for t in (out, lse) if blocks is None else (out, lse, blocks):  # and of the caller's, which reads it
            t.record_stream(torch.cuda.current_stream(q.device))
    return out, lse, blocks


def paged_attn(plan: PagedPlan, q, cache: PagedCache, stream=None):
    """Allocate O and LSE and run bd_paged_attn; returns (out, lse). Rows past the new ones
    are not written."""
    out, lse, _ = _outputs(plan, q, stream)
    bd_paged_attn(plan, q, cache, out, lse, stream=stream)
    return out, lse


# ---------------------------------------------------------------- selected blocks

class BlockBounds:
    """The bounds of a pool's blocks as the library takes them: ``code`` int8 [pages, Hkv, 2, d],
    ``exp`` uint8 [pages, Hkv]. The tensors stay the caller's and are kept alive here."""

    def __init__(self, code, exp):
        if code.dim() != 4 or code.shape[2] != 2 or code.dtype != torch.int8 or code.stride(3) != 1:
            raise ValueError(f"bounds: expected int8 [pages, Hkv, 2, d] with d contiguous, got {code.dtype} {tuple(code.shape)}")
        if exp.dtype != torch.uint8 or exp.shape != code.shape[:2] or exp.device != code.device:
            raise ValueError("bounds: expected uint8 exponents [pages, Hkv] on the codes' device")
        self.code, self.exp = code, exp
        self.num_pages, self.Hkv, _, self.d = code.shape
        s, e = code.stride(), exp.stride()
        self._c = bd_bounds(code.data_ptr(), s[0], s[1], s[2], exp.data_ptr(), e[0], e[1], self.num_pages, 0)
        self._addr = C.addressof(self._c)
        self._index = code.get_device()

    @classmethod
    def empty(cls, cache: PagedCache):
        """Bounds for a cache's pool; a block's are there once bd_block_bounds has seen its rows. Until
        then its byte is 255: a block of which nothing is known outscores the others."""
        return cls(torch.zeros(cache.num_pages, cache.Hkv, 2, cache.d, dtype=torch.int8, device=cache.device),
                   torch.full((cache.num_pages, cache.Hkv), 255, dtype=torch.uint8, device=cache.device))


def _check_bounds(plan, bounds, idx):
    if bounds._index != idx:
        raise ValueError(f"bounds: on {bounds.code.device}, the plan was uploaded to cuda:{idx}")
    if bounds.Hkv != plan.Hkv or bounds.d != plan.d:
        raise ValueError(f"bounds of {bounds.Hkv} heads of {bounds.d}, the plan was built for {plan.Hkv} of {plan.d}")


_blocks = struct.Struct("PqqiI").pack          # bd_blocks


def _lists(t, plan, idx):
    """The rows' lists as the ABI's struct (its bytes)."""
    if t.dtype is not torch.int32 or t.get_device() != idx:
        _refuse(t, "blocks", torch.int32, idx)
    s = t.shape
    if not plan.blocks:
        raise ValueError("not a sparse plan: build it with blocks=...")
    if len(s) != 3 or s[0] < plan.T or s[1] != plan.Hkv or s[2] != plan.blocks or (s[2] > 1 and t.stride(2) != 1):
        raise ValueError(f"blocks: expected [{plan.T} or more, {plan.Hkv}, {plan.blocks}] with lists contiguous, got {tuple(s)}")
    return _blocks(t.data_ptr(), t.stride(0), t.stride(1), s[0], 0)


def bd_block_bounds(plan: PagedPlan, cache: PagedCache, bounds: BlockBounds, stream=None):
    """Bounds of the blocks that hold new rows, from the cache (see include/bd_paged.h)."""
    idx = _device(plan, cache)
    _check_bounds(plan, bounds, idx)
    _call(_entry("bd_block_bounds"), plan, idx, stream, plan._host_ptr, plan._dev_ptr, cache._addr, bounds._addr)


def bd_block_select(plan: PagedPlan, q, bounds: BlockBounds, blocks, stream=None):
    """The blocks that each new row attends, int32 [rows, Hkv, plan.blocks] (see include/bd_paged.h)."""
    if plan._dev_ptr is None:
        raise RuntimeError("plan not uploaded: call .upload(device)")
    idx = plan._index
    _check_bounds(plan, bounds, idx)
    tq = _rows3(q, "q", plan.H, plan.d, plan.T, idx)
    _call(_entry("bd_block_select"), plan, idx, stream, plan._host_ptr, plan._dev_ptr, tq, bounds._addr, _lists(blocks, plan, idx))


def bd_sparse_attn(plan: PagedPlan, q, cache: PagedCache, blocks, out, lse=None, workspace=None, stream=None):
    """O and LSE of the new rows over their listed blocks (see include/bd_paged.h). Without a
    workspace one is allocated for the call."""
    _attend("bd_sparse_attn", plan, q, cache, out, lse, workspace, stream, _lists(blocks, plan, _device(plan, cache)))


def sparse_attn(plan: PagedPlan, q, cache: PagedCache, bounds: BlockBounds, stream=None):
    """Select the new rows' blocks and attend over them; returns (out, lse, blocks). The bounds of
    the blocks that new rows entered are brought up to date first."""
    out, lse, blocks = _outputs(plan, q, stream)
    if blocks is None:
        raise ValueError("not a sparse plan: build it with blocks=...")
    bd_block_bounds(plan, cache, bounds, stream=stream)
    bd_block_select(plan, q, bounds, blocks, stream=stream)
    bd_sparse_attn(plan, q, cache, blocks, out, lse, stream=stream)
    return out, lse, blocks
