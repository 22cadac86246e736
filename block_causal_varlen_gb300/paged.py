"""Paged K/V cache: the binding of include/bd_paged.h.

Tensor layouts (all strided views are accepted; the head dim is contiguous):
    cache k, v     bf16 or e4m3 codes [pages, page_size, Hkv, d], either may be a view
                   of a head-first pool [pages, Hkv, page_size, d]
    k_exp, v_exp   uint8 [pages, page_size, Hkv], e4m3 caches only
    q, out         bf16 [rows, H, d], rows >= T: the new rows of all sequences, packed
    k, v (new)     bf16 [rows, Hkv, d]
    lse            fp32 [H, rows]
"""
from __future__ import annotations

import ctypes as C
import struct

import numpy as np
import torch

from . import _abi
from ._abi import BD_CACHE_BF16, BD_CACHE_E4M3, bd_paged_cache, bd_paged_desc, bd_tensor, check, load

__all__ = ["PagedCache", "PagedPlan", "bd_paged_plan_bytes", "bd_paged_plan_build", "bd_paged_plan_key",
           "bd_cache_write", "bd_cache_read", "bd_paged_attn_workspace", "bd_paged_attn", "paged_attn",
           "BD_CACHE_BF16", "BD_CACHE_E4M3"]

_P32 = C.POINTER(C.c_int32)


def bd_paged_plan_bytes(desc: bd_paged_desc) -> int:
    """Bytes of the plan blob of a descriptor (validates it)."""
    n = C.c_size_t()
    check(load().bd_paged_plan_bytes(C.byref(desc), C.byref(n)))
    return n.value


def bd_paged_plan_build(desc: bd_paged_desc, blob_ptr: int, nbytes: int) -> None:
    """Build the plan blob into host memory at ``blob_ptr``."""
    check(load().bd_paged_plan_build(C.byref(desc), C.c_void_p(blob_ptr), nbytes))


class PagedCache:
    """One layer's K/V pool as the library takes it. The tensors stay the caller's;
    they are kept alive here, and their addresses are fixed for this object."""

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
        else:
            raise TypeError(f"cache dtype {k.dtype}, expected bfloat16 or float8_e4m3fn")
        self.k, self.v, self.k_exp, self.v_exp = k, v, k_exp, v_exp
        self.num_pages, self.page_size, self.Hkv, self.d = k.shape
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
    ``pages``: a page list per sequence, or an integer table [B, max_pages].
    """

    def __init__(self, q_len, kv_len, pages, H, Hkv, d, page_size, num_pages, fmt=BD_CACHE_BF16, causal=True):
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
        self.nbytes = bd_paged_plan_bytes(desc)
        self._raw = np.empty(self.nbytes // 4 + 16, dtype=np.int32)
        off = (-self._raw.ctypes.data % 64) // 4
        self.host = self._raw[off:off + self.nbytes // 4]
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
    if t.dtype is not torch.bfloat16 or t.get_device() != idx or idx < 0:
        _refuse(t, name, torch.bfloat16, idx)
    s = t.shape
    if len(s) != 3 or s[1] != heads or s[2] != d or s[0] < rows:
        raise ValueError(f"{name}: shape {tuple(s)}, expected [{rows} or more, {heads}, {d}]")
    st = t.stride()
    if st[2] != 1:
        raise ValueError(f"{name}: head dim must be contiguous")
    return _tensor(t.data_ptr(), 0, 0, st[0], st[1], s[0], 0)


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


def bd_cache_read(plan: PagedPlan, cache: PagedCache, k, v, stream=None):
    """The cached rows of every sequence, packed in batch order (see include/bd_paged.h)."""
    idx = _device(plan, cache)
    tk = _rows3(k, "k", plan.Hkv, plan.d, plan.kv_total, idx)
    tv = _rows3(v, "v", plan.Hkv, plan.d, plan.kv_total, idx)
    _call(_entry("bd_cache_read"), plan, idx, stream, plan._host_ptr, plan._dev_ptr, cache._addr, tk, tv)


def bd_paged_attn(plan: PagedPlan, q, cache: PagedCache, out, lse=None, workspace=None, stream=None):
    """O and LSE of the new rows over the cache (see include/bd_paged.h). Without a
    workspace one is allocated for the call."""
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
    _call(_entry("bd_paged_attn"), plan, idx, stream, plan._host_ptr, plan._dev_ptr, tq, cache._addr, to, tl, wp, wn)


def paged_attn(plan: PagedPlan, q, cache: PagedCache, stream=None):
    """Allocate O and LSE and run bd_paged_attn; returns (out, lse). Rows past the new ones
    are not written."""
    with torch.cuda.stream(stream):      # memory of the stream that writes it
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        lse = torch.empty(plan.H, q.shape[0], dtype=torch.float32, device=q.device)
    if stream is not None:
        for t in (out, lse):             # and of the caller's, which reads it
            t.record_stream(torch.cuda.current_stream(q.device))
    bd_paged_attn(plan, q, cache, out, lse, stream=stream)
    return out, lse
