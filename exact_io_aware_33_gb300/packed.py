"""Packed sequences: attention with grouped heads and its gradients, and rotary positions with several axes.

Bindings of ``fa_rope_axes``, ``fa_packed_fwd`` and ``fa_packed_bwd`` (``include/fa.h`` states the operators). The rows
of a call's sequences lie one after another in tensors [T, heads, d], which may be slices of a fused projection; ``cu``
(int32 [B + 1], on the device) marks where each sequence begins. A layer's step and its gradients:

    q, k = fa.fa_rope_axes(q, k, positions, (cos, sin), sections=(16, 24, 24))
    o, lse = fa.fa_packed_fwd(q, k, v, cu, causal=True)

    dq, dk, dv = fa.fa_packed_bwd(q, k, v, o, lse, do, cu, causal=True)
    dq, dk = fa.fa_rope_axes(dq, dk, positions, (cos, sin), sections=(16, 24, 24), inverse=True)

All tensors of a call must be on one device, which need not be the current one. With ``stream`` the work
is queued there and outputs belong to that stream; tensors of other streams must be ready, and kept, by
the caller. The calls can be captured into a CUDA graph and replayed; nothing is kept between calls.

The calls' own checks and allocations are in csrc/packed_binding.h.
"""

from __future__ import annotations

import functools

from . import paged as _paged


def _ready(q, stream):
    """The extension module when the call can be made as things stand; None when it must be made elsewhere."""
    if _paged._native is None:
        _paged._load()
    if not isinstance(q, _paged.torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    if stream is not None or (q.is_cuda and _paged._current() != q.get_device()):
        return None
    return _paged._native


def _elsewhere(q, stream):
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor (no CPU path exists)")
    return _paged._elsewhere(q.device, stream)


@functools.lru_cache(maxsize=64)
def _axes(sections, axis_of) -> bytes:
    """The axis of each pair, from its sections or as given."""
    if (sections is None) == (axis_of is None):
        raise ValueError("give either sections (pairs on each axis) or axis_of (the axis of each pair)")
    if axis_of is None:
        if any(n < 0 for n in sections):
            raise ValueError(f"sections {sections} has a negative count")
        axis_of = [a for a, n in enumerate(sections) for _ in range(n)]
    if any(a < 0 or a > 255 for a in axis_of):
        raise ValueError("axes are numbered from 0 to 255")
    return bytes(axis_of)


def fa_rope_axes(q, k, positions, rope, sections=None, axis_of=None, interleaved: bool = False,
                 inverse: bool = False, q_out=None, k_out=None, stream=None):
    """q [T, Hq, d] and k [T, Hk, d] (or None) turned by positions with several axes; returns (q, k).

    ``positions`` is int32 [axes, T]; ``rope`` is (cos, sin), fp32 [max_pos, rot / 2] each. Pair i of the
    first rot channels takes column i of the tables at the token's position on its axis: ``sections`` says
    how many pairs in a row are on each axis, ``axis_of`` names every pair's. ``inverse`` turns the other
    way: the gradient. ``q_out`` and ``k_out`` may be ``q`` and ``k`` themselves."""
    native = _ready(q, stream)
    if native is None:
        with _elsewhere(q, stream):
            return fa_rope_axes(q, k, positions, rope, sections, axis_of, interleaved, inverse, q_out, k_out)
    axes = _axes(None if sections is None else tuple(sections), None if axis_of is None else tuple(axis_of))
    cos, sin = rope
    return native.rope(q, k, positions, cos, sin, axes, interleaved, inverse, q_out, k_out)


def fa_packed_fwd_workspace_bytes(B: int, T: int, Hq: int, Hkv: int, d: int) -> int:
    """Workspace bytes of fa_packed_fwd for B sequences in T rows."""
    if _paged._native is None:
        _paged._load()
    return _paged._lib.fa_packed_fwd_workspace_bytes(B, T, Hq, Hkv, d)


def fa_packed_fwd(q, k, v, cu, causal: bool = False, window: int = 0, scale: float | None = None, out=None,
                  lse=None, workspace=None, stream=None):
    """Attention of each sequence's rows over its own; (o bf16 [T, Hq, d], lse fp32 [T, Hq]).

    q [T, Hq, d], k and v [T, Hkv, d], bf16; query head h reads key head h / (Hq / Hkv). Rows of a new
    ``out`` outside the sequences are not written. Without ``workspace`` one is allocated where the call
    needs it."""
    native = _ready(q, stream)
    if native is None:
        with _elsewhere(q, stream):
            return fa_packed_fwd(q, k, v, cu, causal, window, scale, out, lse, workspace)
    return native.packed_fwd(q, k, v, cu, causal, window, scale, out, lse, workspace)


def fa_packed_bwd_workspace_bytes(B: int, T: int, Hq: int, Hkv: int, d: int) -> int:
    """Workspace bytes of fa_packed_bwd for B sequences in T rows."""
    if _paged._native is None:
        _paged._load()
    return _paged._lib.fa_packed_bwd_workspace_bytes(B, T, Hq, Hkv, d)


def fa_packed_bwd(q, k, v, o, lse, do, cu, causal: bool = False, window: int = 0, scale: float | None = None,
                  dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Gradients of fa_packed_fwd, given its results ``o`` and ``lse``; (dq, dk, dv), bf16.

    ``dq``, ``dk`` and ``dv`` may be slices of the gradient of a fused projection. Rows of new ones outside
    the sequences are not written."""
    native = _ready(q, stream)
    if native is None:
        with _elsewhere(q, stream):
            return fa_packed_bwd(q, k, v, o, lse, do, cu, causal, window, scale, dq, dk, dv, workspace)
    return native.packed_bwd(q, k, v, o, lse, do, cu, causal, window, scale, dq, dk, dv, workspace)
