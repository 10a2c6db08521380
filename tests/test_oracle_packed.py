"""The plain packed operators against facts about them, and the host checks of the library's (no device touched)."""

import ctypes

import numpy as np
import pytest
import torch

import exact_io_aware_33_gb300 as fa
from oracle import packed, paged


# ------------------------------------------------------------------ rotary positions
def angles(n, half):
    x = np.arange(n)[:, None] * 10000.0 ** (-np.arange(half) / half)
    return np.cos(x), np.sin(x)


@pytest.mark.parametrize("interleaved", [False, True])
def test_the_rotation_is_complex_multiplication_on_each_axis(interleaved):
    rng = np.random.default_rng(1)
    T, H, d, half = 9, 3, 64, 24
    x, pos = rng.standard_normal((T, H, d)), rng.integers(0, 50, (3, T))
    axis_of = rng.integers(0, 3, half)
    cos, sin = angles(50, half)
    y = packed.rope(x, pos, axis_of, cos, sin, interleaved, dtype=np.float64)
    for t in range(T):
        for i in range(half):
            ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            z = (x[t, :, ia] + 1j * x[t, :, ib]) * np.exp(1j * pos[axis_of[i], t] * 10000.0 ** (-i / half))
            assert np.allclose(y[t, :, ia] + 1j * y[t, :, ib], z, atol=1e-12)
    assert np.array_equal(y[..., 2 * half:], x[..., 2 * half:])
    back = packed.rope(y, pos, axis_of, cos, sin, interleaved, inverse=True, dtype=np.float64)
    assert np.allclose(back, x, atol=1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
def test_one_axis_is_the_rotation_of_the_paged_cache(interleaved):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((5, 2, 64)).astype(np.float32)
    cos, sin = (a.astype(np.float32) for a in angles(40, 32))
    pos = np.array([[3, 39, 0, 7, 7]])
    y = packed.rope(x, pos, [0] * 32, cos, sin, interleaved)
    for t, p in enumerate(pos[0]):
        assert np.array_equal(y[t], paged.rotate(x[t], cos[p], sin[p], interleaved))


def test_the_inverse_rotation_is_the_gradient():
    rng = np.random.default_rng(3)
    x, w = rng.standard_normal((2, 3, 1, 16))
    pos, axis_of = rng.integers(0, 30, (2, 3)), [0, 1, 1, 0]
    cos, sin = angles(30, 4)
    f = lambda z: float((packed.rope(z, pos, axis_of, cos, sin, True, dtype=np.float64) * w).sum())  # noqa: E731
    g = packed.rope(w, pos, axis_of, cos, sin, True, inverse=True, dtype=np.float64)
    for at in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[at] = 1e-6
        assert abs((f(x + e) - f(x - e)) / 2e-6 - g[at]) < 1e-8


@pytest.fixture(scope="module")
def lib():
    from exact_io_aware_33_gb300 import build
    build.build()
    return fa.load_library()


P = 0x100000  # never dereferenced: checks fail first


def _rope(lib, q=P, qs=512, qo=P + 0x100000, qos=512, Hq=4, k=P + 0x200000, ks=256, ko=P + 0x300000, kos=256, Hk=2,
          positions=P, axes=3, T=8, axis_of=None, cos=P, sin=P, max_pos=100, rot=128, d=128):
    a = (ctypes.c_ubyte * max(rot // 2, 1))(*(axis_of or [0] * (rot // 2)))
    return lib.fa_rope_axes(q, qs, qo, qos, Hq, k, ks, ko, kos, Hk, positions, axes, T, ctypes.addressof(a), cos, sin,
                            max_pos, rot, d, 0, 0, None)


@pytest.mark.parametrize("kw,code", [
    (dict(d=96), fa.FA_ERR_UNSUPPORTED), (dict(d=512), fa.FA_ERR_UNSUPPORTED), (dict(rot=24), fa.FA_ERR_UNSUPPORTED),
    (dict(rot=144), fa.FA_ERR_INVALID), (dict(rot=-16), fa.FA_ERR_INVALID), (dict(T=-1), fa.FA_ERR_INVALID),
    (dict(Hq=-1), fa.FA_ERR_INVALID), (dict(Hk=-1), fa.FA_ERR_INVALID), (dict(axes=0), fa.FA_ERR_INVALID),
    (dict(max_pos=0), fa.FA_ERR_INVALID), (dict(max_pos=-5), fa.FA_ERR_INVALID),
    (dict(q=0), fa.FA_ERR_INVALID), (dict(k=0), fa.FA_ERR_INVALID), (dict(qo=0), fa.FA_ERR_INVALID),
    (dict(ko=0), fa.FA_ERR_INVALID), (dict(q=P + 8), fa.FA_ERR_INVALID), (dict(ko=P + 0x300004), fa.FA_ERR_INVALID),
    (dict(cos=0), fa.FA_ERR_INVALID), (dict(sin=P + 4), fa.FA_ERR_INVALID), (dict(positions=0), fa.FA_ERR_INVALID),
    (dict(positions=P + 2), fa.FA_ERR_INVALID), (dict(qs=511), fa.FA_ERR_INVALID), (dict(qs=516), fa.FA_ERR_INVALID),
    (dict(ks=248), fa.FA_ERR_INVALID), (dict(kos=8), fa.FA_ERR_INVALID),
    (dict(axis_of=[0] * 63 + [3]), fa.FA_ERR_INVALID),
    # outputs that meet an input or each other
    (dict(qo=P + 1024), fa.FA_ERR_INVALID), (dict(qo=P, qos=1024), fa.FA_ERR_INVALID),
    (dict(ko=P), fa.FA_ERR_INVALID), (dict(qo=P + 0x200000), fa.FA_ERR_INVALID),
    (dict(qo=P + 0x300000), fa.FA_ERR_INVALID), (dict(ko=P + 0x200000 + 512), fa.FA_ERR_INVALID),
    # nothing to do
    (dict(T=0, q=0, k=0), fa.FA_OK), (dict(Hq=0, Hk=0, q=0, k=0), fa.FA_OK)])
def test_rope_refusals(lib, kw, code):
    assert _rope(lib, **kw) == code


@pytest.mark.parametrize("kw", [
    dict(), dict(qo=P, ko=P + 0x200000), dict(T=1, qo=P, qos=1024),
    # slices of one projection (queries, keys, values of a token side by side), in place and to such slices
    dict(qs=1024, ks=1024, qos=1024, kos=1024, k=P + 1024, qo=P, ko=P + 1024),
    dict(qs=1024, ks=1024, qos=1024, kos=1024, k=P + 1024, ko=P + 0x100000 + 1024),
    dict(Hk=0, k=0, ko=0), dict(rot=0, positions=0, cos=0, sin=0)])
def test_rope_accepts(lib, kw):
    # (there is no device here, or the pointers are no memory of its: the checks before the device passed)
    if torch.cuda.is_available():
        pytest.skip("would launch on pointers that are none")
    assert _rope(lib, **kw) in (fa.FA_ERR_LAUNCH, fa.FA_ERR_UNSUPPORTED)


def test_rope_binding_refusals():
    q = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    rope, pos = (torch.zeros(8, 32), torch.zeros(8, 32)), torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        fa.fa_rope_axes(q, q, pos, rope, sections=(16, 16))
    with pytest.raises(TypeError, match="Tensor"):
        fa.fa_rope_axes(None, q, pos, rope, sections=(16, 16))
    axes = fa.packed._axes
    assert axes((2, 0, 3), None) == bytes([0, 0, 2, 2, 2]) and axes(None, (1, 0)) == bytes([1, 0])
    for bad in ((None, None), ((1,), (0,)), ((2, -1), None), (None, (0, 256)), (None, (0, -1))):
        with pytest.raises(ValueError):
            axes(*bad)


# ------------------------------------------------------------------ attention
def test_one_sequence_with_heads_of_its_own_is_the_general_oracle():
    from oracle import general
    rng = np.random.default_rng(4)
    q, k, v, do = rng.standard_normal((4, 11, 2, 8))
    for causal, window in ((True, 0), (False, 0), (True, 3)):
        o, lse = packed.forward(q, k, v, [0, 11], causal, 0.3, window)
        g = packed.backward(q, k, v, o, lse, do, [0, 11], causal, 0.3, window)
        for h in range(2):
            want, want_lse = general.forward_head(q[:, h], k[:, h], v[:, h], causal, 0.3, window)
            assert np.array_equal(o[:, h], want) and np.array_equal(lse[:, h], want_lse)
            for a, b in zip(g, general.backward_head(q[:, h], k[:, h], v[:, h], want, want_lse, do[:, h], causal, 0.3, window)):
                assert np.array_equal(a[:, h], b)


def test_gradients_of_shared_heads_and_separate_sequences_against_differences():
    rng = np.random.default_rng(5)
    T, cu, w = 8, [1, 4, 4, 7], 2                    # rows 0 and 7 are no sequence's
    x = [rng.standard_normal((T, h, 4)) for h in (4, 2, 2)]
    do = rng.standard_normal((T, 4, 4))
    loss = lambda *a: float(np.nansum(packed.forward(*a, cu, True, 0.5, w)[0] * do))  # noqa: E731
    o, lse = packed.forward(*x, cu, True, 0.5, w)
    assert np.isnan(o[[0, 7]]).all() and not np.isnan(o[1:7]).any()
    for i, g in enumerate(packed.backward(*x, o, lse, do, cu, True, 0.5, w)):
        assert np.isnan(g[[0, 7]]).all()
        for at in np.ndindex(x[i].shape):
            moved = [[y.copy() for y in x] for _ in range(2)]
            moved[0][i][at] += 1e-5
            moved[1][i][at] -= 1e-5
            want = (loss(*moved[0]) - loss(*moved[1])) / 2e-5
            assert abs(want - (0.0 if at[0] in (0, 7) else g[at])) < 1e-8, (i, at)


def _far(i):
    return P + i * 0x100000


def _fwd(lib, q=_far(0), qs=512, k=_far(1), ks=256, v=_far(2), vs=256, cu=P, B=3, T=8, Hq=4, Hkv=2, d=128, causal=1,
         window=0, scale=0.1, o=_far(3), lse=P, ws=0, ws_bytes=0):
    return lib.fa_packed_fwd(q, qs, k, ks, v, vs, cu, B, T, Hq, Hkv, d, causal, window, scale, o, lse, ws, ws_bytes, None)


def _bwd(lib, q=_far(0), qs=512, k=_far(1), ks=256, v=_far(2), vs=256, o=_far(3), lse=P, do=_far(4), dos=512, cu=P, B=3, T=8,
         Hq=4, Hkv=2, d=128, causal=1, window=0, scale=0.1, dq=_far(5), dqs=512, dk=_far(6), dks=256, dv=_far(7), dvs=256,
         ws=_far(8), ws_bytes=1 << 20):
    return lib.fa_packed_bwd(q, qs, k, ks, v, vs, o, lse, do, dos, cu, B, T, Hq, Hkv, d, causal, window, scale, dq, dqs,
                             dk, dks, dv, dvs, ws, ws_bytes, None)


SHARED = [
    (dict(d=96), fa.FA_ERR_UNSUPPORTED), (dict(d=256), fa.FA_ERR_UNSUPPORTED),
    (dict(Hq=258, Hkv=2, qs=258 * 128), fa.FA_ERR_UNSUPPORTED),
    (dict(Hq=5), fa.FA_ERR_INVALID), (dict(Hq=0), fa.FA_ERR_INVALID), (dict(Hkv=0), fa.FA_ERR_INVALID),
    (dict(Hkv=-2), fa.FA_ERR_INVALID), (dict(B=-1), fa.FA_ERR_INVALID), (dict(T=-1), fa.FA_ERR_INVALID),
    (dict(T=2 ** 29 - 1), fa.FA_ERR_INVALID), (dict(T=2 ** 30, Hq=1, Hkv=1), fa.FA_ERR_INVALID),
    (dict(B=2 ** 30), fa.FA_ERR_INVALID),
    (dict(scale=-1.0), fa.FA_ERR_INVALID), (dict(scale=float("nan")), fa.FA_ERR_INVALID),
    (dict(scale=float("inf")), fa.FA_ERR_INVALID), (dict(window=-1), fa.FA_ERR_INVALID),
    (dict(window=5, causal=0), fa.FA_ERR_INVALID),
    (dict(q=0), fa.FA_ERR_INVALID), (dict(k=P + 8), fa.FA_ERR_INVALID), (dict(v=0), fa.FA_ERR_INVALID),
    (dict(o=0), fa.FA_ERR_INVALID), (dict(lse=0), fa.FA_ERR_INVALID), (dict(lse=P + 2), fa.FA_ERR_INVALID),
    (dict(cu=0), fa.FA_ERR_INVALID), (dict(cu=P + 1), fa.FA_ERR_INVALID),
    (dict(qs=504), fa.FA_ERR_INVALID), (dict(qs=516), fa.FA_ERR_INVALID), (dict(ks=248), fa.FA_ERR_INVALID),
    (dict(vs=2 ** 38), fa.FA_ERR_INVALID),
    (dict(B=0, q=0, cu=0), fa.FA_OK), (dict(T=0, q=0, cu=0), fa.FA_OK)]


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(o=_far(0)), fa.FA_ERR_INVALID), (dict(o=_far(1) + 512), fa.FA_ERR_INVALID),
    (dict(o=_far(2) - 512), fa.FA_ERR_INVALID)])
def test_packed_fwd_refusals(lib, kw, code):
    assert _fwd(lib, **kw) == code


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(do=0), fa.FA_ERR_INVALID), (dict(dos=8), fa.FA_ERR_INVALID), (dict(dq=0), fa.FA_ERR_INVALID),
    (dict(dk=P + 8), fa.FA_ERR_INVALID), (dict(dvs=252), fa.FA_ERR_INVALID),
    (dict(ws=0), fa.FA_ERR_WORKSPACE), (dict(ws=_far(8) + 128), fa.FA_ERR_WORKSPACE), (dict(ws_bytes=100), fa.FA_ERR_WORKSPACE),
    # outputs that meet an input or each other
    (dict(dq=_far(0)), fa.FA_ERR_INVALID), (dict(dk=_far(1)), fa.FA_ERR_INVALID), (dict(dv=_far(4)), fa.FA_ERR_INVALID),
    (dict(dq=_far(3) + 1024), fa.FA_ERR_INVALID), (dict(dk=_far(7)), fa.FA_ERR_INVALID),
    (dict(dv=_far(5) + 512), fa.FA_ERR_INVALID)])
def test_packed_bwd_refusals(lib, kw, code):
    assert _bwd(lib, **kw) == code


@pytest.mark.parametrize("call,kw", [
    (_fwd, dict()), (_fwd, dict(window=2 ** 31 - 1)),
    # slices of one projection, and gradients into slices of another
    (_fwd, dict(qs=1024, ks=1024, vs=1024, k=_far(0) + 1024, v=_far(0) + 1536)),
    (_bwd, dict()),
    (_bwd, dict(qs=1024, ks=1024, vs=1024, k=_far(0) + 1024, v=_far(0) + 1536, dqs=1024, dks=1024, dvs=1024,
                dk=_far(5) + 1024, dv=_far(5) + 1536))])
def test_packed_accepts(lib, call, kw):
    if torch.cuda.is_available():
        pytest.skip("would launch on pointers that are none")
    assert call(lib, **kw) in (fa.FA_ERR_LAUNCH, fa.FA_ERR_UNSUPPORTED)


def test_packed_workspace(lib):
    n = lib.fa_packed_fwd_workspace_bytes
    assert n(1, 100, 4, 2, 64) == 0                         # every item has a CTA
    # a list of entries of 2 x 32 tokens, 16 bytes each
    assert n(8, 20000, 32, 8, 128) == 16 + 16 * (20000 // 64 + 8)
    for bad in ((-1, 8, 4, 2, 64), (1, 8, 5, 2, 64), (1, 8, 4, 2, 65), (0, 8, 4, 2, 64), (1, 0, 4, 2, 64)):
        assert n(*bad) == 0 and lib.fa_packed_bwd_workspace_bytes(*bad) == 0
    m = lib.fa_packed_bwd_workspace_bytes
    assert m(1, 100, 4, 2, 64) == 100 * 4 * 8 + 128         # two statistics a row, to a multiple of 256
    assert m(8, 20000, 32, 8, 128) >= 20000 * 32 * 8 + 16 * (20000 // 128 + 20000 // 32 + 16)


def test_packed_binding_refusals():
    q = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        fa.fa_packed_fwd(q, q, q, cu)
    with pytest.raises(ValueError, match="CUDA"):
        fa.fa_packed_bwd(q, q, q, q, torch.zeros(3, 2), q, cu)
    for call in (lambda: fa.fa_packed_fwd([1], q, q, cu), lambda: fa.fa_packed_bwd(None, q, q, q, q, q, cu)):
        with pytest.raises(TypeError, match="Tensor"):
            call()
