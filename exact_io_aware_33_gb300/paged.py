"""The paged 8-bit key/value cache: appending rotated keys and values, and attention over it.

Binding of ``fa_paged_append`` and ``fa_paged_attn`` (``include/fa.h`` states the operators). A serving
step is two calls on one ``PagedCache`` and one ``PagedBatch``:

    cache = fa.PagedCache.empty(num_pages, num_heads, page_size, d)
    batch = fa.PagedBatch(block_table, kv_lens, cu_q, max_q=..., max_kv=...)   # or cu_q=None: decode
    q = fa.fa_paged_append(cache, batch, k, v, q=q, rope=(cos, sin))
    o, lse = fa.fa_paged_attn(cache, batch, q)

Both objects only hold tensors of the caller and their checked sizes, so a decode loop makes them once
and updates ``kv_lens`` and ``block_table`` in place between steps (``copy_``, ``add_``, indexing). Other
tensors take a new object: attributes cannot be set, and a call refuses a tensor whose memory has moved
since (``resize_``, ``set_``, ``.data``). The calls can be captured into a
CUDA graph and replayed that way. All tensors of a call must be on one device, which need not be the
current one. With ``stream`` the work is queued there and outputs and workspaces belong to that stream;
tensors of other streams must be ready, and kept, by the caller.

The calls' own checks and allocations are in csrc/paged_binding.cpp.
"""

from __future__ import annotations

import ctypes
import math

_PAGE_SIZES = (16, 32, 64, 128)

# Set with the first object: the package loads neither torch nor the libraries by itself.
torch = _lib = _native = _current = None


def _load():
    global torch, _lib, _native, _current
    if torch is None:
        import torch as t

        from . import _check, load_library
        lib = load_library()
        try:
            from . import _paged_native as native
        except ImportError as e:
            raise ImportError(f"the Python binding of the paged cache and of packed sequences is not built ({e}); run "
                              "`python -m exact_io_aware_33_gb300.build` or __graft_entry__.build() first") from e
        native.set_fail(_check)
        _lib, _native, _current = lib, native, t._C._cuda_getDevice
        torch = t


class _CacheStruct(ctypes.Structure):
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("num_pages", ctypes.c_int), ("num_heads", ctypes.c_int),
                ("page_size", ctypes.c_int), ("d", ctypes.c_int)]


class _BatchStruct(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("kv_lens", ctypes.c_void_p), ("cu_q", ctypes.c_void_p),
                ("B", ctypes.c_int), ("T", ctypes.c_int), ("max_q", ctypes.c_int),
                ("max_pages", ctypes.c_int), ("max_kv", ctypes.c_int)]


def _require(t, name, dtype, dim, device=None):
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.dim() == dim and (
            t.device == device if device is not None else t.is_cuda):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path exists)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions, got {t.dim()}")
    raise ValueError(f"{name} is on {t.device}, expected {device}")


class _Fixed:
    """An object whose attributes stay as they are once ``_address``, of the C struct made from them, is set."""

    def _refuse(self, name):
        if "_address" in self.__dict__:
            raise AttributeError(f"{type(self).__name__}.{name} cannot be changed: make a new {type(self).__name__}")

    def __setattr__(self, name, value):
        self._refuse(name)
        super().__setattr__(name, value)

    def __delattr__(self, name):
        self._refuse(name)
        super().__delattr__(name)


class PagedCache(_Fixed):
    """A pool of e4m3 pages [num_pages, num_heads, page_size, d] with fp32 scales [num_pages, num_heads]."""

    def __init__(self, k_pages, v_pages, k_scales, v_scales):
        _load()
        _require(k_pages, "k_pages", torch.float8_e4m3fn, 4)
        dev = k_pages.device
        _require(v_pages, "v_pages", torch.float8_e4m3fn, 4, dev)
        P, H, page, d = k_pages.shape
        if page not in _PAGE_SIZES:
            raise ValueError(f"page size {page} is not one of {_PAGE_SIZES}")
        if d not in (64, 128):
            raise ValueError(f"head size {d} is not 64 or 128")
        if v_pages.shape != k_pages.shape:
            raise ValueError(f"v_pages has shape {tuple(v_pages.shape)}, expected {tuple(k_pages.shape)}")
        for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
            _require(t, name, torch.float32, 2, dev)
            if tuple(t.shape) != (P, H):
                raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(P, H)}")
        for name, t in (("k_pages", k_pages), ("v_pages", v_pages), ("k_scales", k_scales),
                        ("v_scales", v_scales)):
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
        self.k_pages, self.v_pages, self.k_scales, self.v_scales = k_pages, v_pages, k_scales, v_scales
        self.num_pages, self.num_heads, self.page_size, self.d = P, H, page, d
        self.device = dev
        self._index = dev.index
        self._scale = 1.0 / math.sqrt(d)
        self._held = (k_pages, v_pages, k_scales, v_scales)
        self._struct = _CacheStruct(k_pages.data_ptr(), v_pages.data_ptr(), k_scales.data_ptr(),
                                    v_scales.data_ptr(), P, H, page, d)
        self._address = ctypes.addressof(self._struct)

    @classmethod
    def empty(cls, num_pages: int, num_heads: int, page_size: int, d: int, device="cuda"):
        """A new pool. Its contents do not matter: only what was appended is ever read."""
        _load()
        shape = (num_pages, num_heads, page_size, d)
        pages = [torch.empty(shape, dtype=torch.float8_e4m3fn, device=device) for _ in range(2)]
        scales = [torch.empty(shape[:2], dtype=torch.float32, device=device) for _ in range(2)]
        return cls(*pages, *scales)


class PagedBatch(_Fixed):
    """The sequences of a step: their pages, lengths (new tokens included) and packed rows.

    ``cu_q`` None: one new token per sequence. ``max_q`` bounds the new tokens of a sequence, ``max_kv``
    their lengths (0: what the block table can hold); both are host numbers, no tensor is read back."""

    def __init__(self, block_table, kv_lens, cu_q=None, max_q: int = 1, max_kv: int = 0):
        _load()
        _require(block_table, "block_table", torch.int32, 2)
        dev = block_table.device
        _require(kv_lens, "kv_lens", torch.int32, 1, dev)
        B, max_pages = block_table.shape
        if kv_lens.shape[0] != B:
            raise ValueError(f"kv_lens has {kv_lens.shape[0]} entries, block_table {B} rows")
        if cu_q is not None:
            _require(cu_q, "cu_q", torch.int32, 1, dev)
            if cu_q.shape[0] != B + 1:
                raise ValueError(f"cu_q has {cu_q.shape[0]} entries, expected {B + 1}")
        elif max_q != 1:
            raise ValueError("max_q must be 1 without cu_q")
        if not (1 <= max_q < 2 ** 31 and 0 <= max_kv < 2 ** 31 and max_pages < 2 ** 31):
            raise ValueError("max_q must be at least 1 and max_kv at least 0, all sizes below 2^31")
        for name, t in (("block_table", block_table), ("kv_lens", kv_lens), ("cu_q", cu_q)):
            if t is not None and not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
        self.block_table, self.kv_lens, self.cu_q = block_table, kv_lens, cu_q
        self.B, self.max_pages, self.max_q, self.max_kv = B, max_pages, int(max_q), int(max_kv)
        self.device = dev
        self._index = dev.index
        self._held = (block_table, kv_lens, cu_q)
        # (the rows of a call's tensors take the place of T there)
        self._struct = _BatchStruct(block_table.data_ptr(), kv_lens.data_ptr(),
                                    0 if cu_q is None else cu_q.data_ptr(), B, B, self.max_q, max_pages, self.max_kv)
        self._address = ctypes.addressof(self._struct)


def _elsewhere(device, stream):
    """Where a call allocates and launches when not as things stand: `stream`, or the tensors' own device."""
    if stream is None:
        return torch.cuda.device(device)
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, expected {device}")
    return torch.cuda.stream(stream)


def fa_paged_append(cache: PagedCache, batch: PagedBatch, k, v, q=None, rope=None, interleaved: bool = False,
                    q_out=None, stream=None):
    """Writes k and v [T, num_heads, d] to the batch's pages, keys rotated; returns the rotated queries.

    ``rope`` is (cos, sin), fp32 [max_pos, rot / 2] each, or None. Without ``q`` the result is None. Rows
    of a new ``q_out`` behind the last sequence, or without a position, are not written."""
    index = cache._index
    if stream is not None or _current() != index:
        with _elsewhere(cache.device, stream):
            return fa_paged_append(cache, batch, k, v, q, rope, interleaved, q_out)
    if batch._index != index:
        raise ValueError(f"the batch is on {batch.device}, the cache on {cache.device}")
    if q is None and q_out is not None:
        raise ValueError("q_out without q")
    cos, sin = (None, None) if rope is None else rope
    return _native.append(cache._address, cache._held, batch._address, batch._held, index, k, v, q, cos, sin, interleaved, q_out)


def fa_paged_attn_workspace_bytes(cache: PagedCache, batch: PagedBatch, Hq: int) -> int:
    """Workspace bytes of fa_paged_attn with these arguments; they do not depend on the number of rows."""
    if _current() != cache._index:
        with _elsewhere(cache.device, None):
            return fa_paged_attn_workspace_bytes(cache, batch, Hq)
    return _lib.fa_paged_attn_workspace_bytes(cache._address, batch._address, Hq)


def fa_paged_attn(cache: PagedCache, batch: PagedBatch, q, window: int = 0, scale: float | None = None,
                  out=None, lse=None, workspace=None, stream=None):
    """Causal attention of q [T, Hq, d] over the batch's cached tokens; (o bf16 [T, Hq, d], lse fp32 [T, Hq]).

    Rows of a new ``out`` behind the last sequence are not written. Without ``workspace`` one is allocated
    where the call needs it."""
    index = cache._index
    if stream is not None or _current() != index:
        with _elsewhere(cache.device, stream):
            return fa_paged_attn(cache, batch, q, window, scale, out, lse, workspace)
    if batch._index != index:
        raise ValueError(f"the batch is on {batch.device}, the cache on {cache.device}")
    return _native.attn(cache._address, cache._held, batch._address, batch._held, index, q, window,
                        cache._scale if scale is None else scale, out, lse, workspace)
