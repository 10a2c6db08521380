"""The plain paged cache against facts about e4m3 and against dense attention, and the binding's host checks."""

import ctypes
import math

import numpy as np
import pytest
import torch

import exact_io_aware_33_gb300 as fa
from oracle import dense, paged


def test_every_code_has_the_value_that_torch_gives_it():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes.copy()).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(paged.E4M3, want, equal_nan=True)


def test_encode_rounds_to_nearest_even():
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.standard_normal(4000) * s for s in (1e-3, 1e-2, 1.0, 60.0)]).astype(np.float32)
    x = np.clip(x, -448, 448)
    pos = paged.E4M3[:127]
    mids = ((pos[:-1] + pos[1:]) / 2).astype(np.float32)   # every tie
    x = np.concatenate([x, mids, -mids, pos.astype(np.float32)])
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(paged.encode(x), want)
    assert np.array_equal(paged.encode(paged.E4M3[:127]), np.arange(127))
    assert list(paged.encode([np.inf, -np.inf, 1e9, np.nan])) == [126, 254, 126, 127]


@pytest.mark.parametrize("amax,want", [(448.0, 1.0), (448.5, 2.0), (224.0, 0.5), (1.0, 2.0 ** -8), (1.75, 2.0 ** -8),
                                       (1.7500001, 2.0 ** -7), (2.0 ** -133, 2.0 ** -126), (0.0, 1.0)])
def test_scales_are_the_smallest_power_of_two(amax, want):
    assert paged.scale_of(amax) == want


def test_rotation_keeps_pairs_lengths_and_relative_angles():
    rng = np.random.default_rng(2)
    for interleaved in (False, True):
        x, y = rng.standard_normal((2, 64))
        ang = lambda p: p * 10000.0 ** (-np.arange(16) / 16)  # noqa: E731
        at = lambda v, p: paged.rotate(v, np.cos(ang(p)), np.sin(ang(p)), interleaved, np.float64)  # noqa: E731
        assert math.isclose(np.linalg.norm(at(x, 77)), np.linalg.norm(x), rel_tol=1e-12)
        assert np.array_equal(at(x, 77)[32:], x[32:])
        assert math.isclose(at(x, 10) @ at(y, 3), at(x, 107) @ at(y, 100), rel_tol=1e-9)


def test_a_growing_scale_rounds_the_older_codes_again():
    c = paged.Cache(np.zeros((1, 1, 16, 64)), np.zeros((1, 1, 16, 64)), np.ones((1, 1)), np.ones((1, 1)))
    table = [[0]]
    x = np.full((1, 1, 64), 1.0)
    c.append(table, [1], [0, 1], x, x)
    assert c.scales["k"][0, 0] == 2.0 ** -8
    c.append(table, [2], [0, 1], 100 * x, 100 * x)
    assert c.scales["k"][0, 0] == 0.25
    assert np.all(c.read("k", [0], 2)[0, :, 0] == [1.0, 96.0 if paged.E4M3[paged.encode(400.0)] == 384 else 104.0])
    c.append(table, [3], [0, 1], x, x)   # smaller values do not shrink the scale
    assert c.scales["k"][0, 0] == 0.25


def test_attend_is_dense_attention_over_what_is_read():
    rng = np.random.default_rng(3)
    P, H, page, d, n = 4, 2, 16, 64, 40
    codes = [paged.encode(rng.standard_normal((P, H, page, d)) * 50) for _ in range(2)]
    scales = [2.0 ** rng.integers(-8, -4, (P, H)) for _ in range(2)]
    c = paged.Cache(codes[0], codes[1], scales[0], scales[1])
    table = [[2, 0, 3]]
    q = rng.standard_normal((n, H, d)).astype(np.float32)  # the dense oracle reads its inputs as float32
    o, lse = c.attend(table, [n], [0, n], q, 0.125)
    k, v = c.read("k", table[0], n), c.read("v", table[0], n)
    as_t = lambda x: torch.from_numpy(np.ascontiguousarray(x))[None]  # noqa: E731
    want, want_lse = dense.forward(as_t(q.transpose(1, 0, 2)), as_t(k), as_t(v), True, 0.125)
    assert np.allclose(o, want[0].transpose(1, 0, 2), atol=1e-12)
    assert np.allclose(lse, want_lse[0].T, atol=1e-12)


# ------------------------------------------------------------------ host checks, no device touched
@pytest.fixture(scope="module")
def lib():
    from exact_io_aware_33_gb300 import build
    build.build()
    return fa.load_library()


P = 0x100000  # never dereferenced: every call below fails its checks first or is empty


def _cache(**kw):
    from exact_io_aware_33_gb300.paged import _CacheStruct
    f = dict(k_pages=P, v_pages=P, k_scales=P, v_scales=P, num_pages=8, num_heads=2, page_size=16, d=64)
    f.update(kw)
    return _CacheStruct(**f)


def _batch(**kw):
    from exact_io_aware_33_gb300.paged import _BatchStruct
    f = dict(block_table=P, kv_lens=P, cu_q=P, B=2, T=9, max_q=8, max_pages=4, max_kv=0)
    f.update(kw)
    return _BatchStruct(**f)


def _attn(lib, c, b, q=P, stride=4 * 64, o=P + 0x10000, lse=P, Hq=4, window=0, scale=0.125, ws=0, bytes_=0):
    return lib.fa_paged_attn(ctypes.addressof(c) if c else 0, ctypes.addressof(b) if b else 0, q, stride, o, lse, Hq,
                             window, scale, ws, bytes_, 0)


def _append(lib, c, b, k=P, ks=2 * 64, v=P, vs=2 * 64, q=P, qs=4 * 64, qo=P + 0x10000, qos=4 * 64, Hq=4, cos=P, sin=P,
            max_pos=9, rot=64):
    return lib.fa_paged_append(ctypes.addressof(c) if c else 0, ctypes.addressof(b) if b else 0, k, ks, v, vs, q, qs,
                               qo, qos, Hq, cos, sin, max_pos, rot, 0, 0)


BOTH = [
    (dict(d=96), {}, fa.FA_ERR_UNSUPPORTED),
    (dict(d=256), {}, fa.FA_ERR_UNSUPPORTED),
    (dict(page_size=48), {}, fa.FA_ERR_UNSUPPORTED),
    (dict(page_size=256), {}, fa.FA_ERR_UNSUPPORTED),
    (dict(num_heads=0), {}, fa.FA_ERR_INVALID),
    (dict(num_pages=0), {}, fa.FA_ERR_INVALID),
    (dict(num_pages=1 << 30, num_heads=4), {}, fa.FA_ERR_INVALID),
    (dict(k_pages=0), {}, fa.FA_ERR_INVALID),
    (dict(v_pages=P + 8), {}, fa.FA_ERR_INVALID),
    (dict(k_scales=0), {}, fa.FA_ERR_INVALID),
    (dict(v_scales=P + 2), {}, fa.FA_ERR_INVALID),
    ({}, dict(B=-1), fa.FA_ERR_INVALID),
    ({}, dict(T=-3), fa.FA_ERR_INVALID),
    ({}, dict(max_q=0), fa.FA_ERR_INVALID),
    ({}, dict(max_kv=-1), fa.FA_ERR_INVALID),
    ({}, dict(max_pages=0), fa.FA_ERR_INVALID),
    ({}, dict(max_pages=1 << 28), fa.FA_ERR_INVALID),
    ({}, dict(block_table=0), fa.FA_ERR_INVALID),
    ({}, dict(kv_lens=P + 1), fa.FA_ERR_INVALID),
    ({}, dict(cu_q=0), fa.FA_ERR_INVALID),              # one token per sequence, but nine rows for two
    ({}, dict(cu_q=0, T=2), fa.FA_ERR_INVALID),         # ... and max_q is not 1
    ({}, dict(B=0), fa.FA_OK),
    ({}, dict(T=0), fa.FA_OK),
]


@pytest.mark.parametrize("c,b,code", BOTH)
def test_cache_and_batch_are_checked_on_the_host(lib, c, b, code):
    assert _attn(lib, _cache(**c), _batch(**b)) == code
    assert _append(lib, _cache(**c), _batch(**b)) == code


def test_missing_structs_are_refused(lib):
    assert _attn(lib, None, _batch()) == fa.FA_ERR_INVALID
    assert _append(lib, _cache(), None) == fa.FA_ERR_INVALID
    assert lib.fa_paged_attn_workspace_bytes(0, 0, 4) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(Hq=3), fa.FA_ERR_INVALID), (dict(Hq=0), fa.FA_ERR_INVALID), (dict(window=-1), fa.FA_ERR_INVALID),
    (dict(scale=math.nan), fa.FA_ERR_INVALID), (dict(scale=-1.0), fa.FA_ERR_INVALID), (dict(q=0), fa.FA_ERR_INVALID),
    (dict(q=P + 2), fa.FA_ERR_INVALID), (dict(o=0), fa.FA_ERR_INVALID), (dict(lse=0), fa.FA_ERR_INVALID),
    (dict(stride=4 * 64 - 8), fa.FA_ERR_INVALID), (dict(stride=4 * 64 + 4), fa.FA_ERR_INVALID),
    (dict(), fa.FA_ERR_WORKSPACE), (dict(ws=P + 16, bytes_=1 << 30), fa.FA_ERR_WORKSPACE),
    (dict(ws=P, bytes_=64), fa.FA_ERR_WORKSPACE)])
def test_attention_arguments_are_checked_on_the_host(lib, kw, code):
    assert _attn(lib, _cache(), _batch(max_pages=100000), **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(k=0), fa.FA_ERR_INVALID), (dict(v=P + 4), fa.FA_ERR_INVALID), (dict(ks=2 * 64 - 8), fa.FA_ERR_INVALID),
    (dict(vs=2 * 64 + 1), fa.FA_ERR_INVALID), (dict(Hq=-1), fa.FA_ERR_INVALID), (dict(q=0), fa.FA_ERR_INVALID),
    (dict(qo=0), fa.FA_ERR_INVALID), (dict(qs=8), fa.FA_ERR_INVALID), (dict(qos=12), fa.FA_ERR_INVALID),
    (dict(rot=80), fa.FA_ERR_INVALID), (dict(rot=-16), fa.FA_ERR_INVALID), (dict(rot=24), fa.FA_ERR_UNSUPPORTED),
    (dict(cos=0), fa.FA_ERR_INVALID), (dict(sin=P + 4), fa.FA_ERR_INVALID), (dict(max_pos=0), fa.FA_ERR_INVALID)])
def test_append_arguments_are_checked_on_the_host(lib, kw, code):
    assert _append(lib, _cache(), _batch(), **kw) == code


@pytest.mark.parametrize("d,max_q,max_kv", [(64, 5, 4096), (128, 4, 2048), (128, 64, 2048), (64, 300, 900), (128, 16, 512)])
@pytest.mark.parametrize("B,heads", [(1, 1), (3, 8), (16, 4), (48, 8)])
def test_the_workspace_does_not_depend_on_the_rows(lib, d, max_q, max_kv, B, heads):
    c = _cache(page_size=64, num_heads=heads, d=d, num_pages=100)
    need = {lib.fa_paged_attn_workspace_bytes(ctypes.addressof(c), ctypes.addressof(_batch(
        B=B, T=T, max_q=max_q, max_pages=200, max_kv=max_kv)), 4 * heads) for T in (1, B, B * max_q // 2, B * max_q)}
    assert len(need) == 1


ROW = 4 * 64 * 2  # bytes of a query row; nine rows


@pytest.mark.parametrize("o,stride,code", [
    (P, 256, fa.FA_ERR_WORKSPACE),                 # in place: past this check
    (P, 512, fa.FA_ERR_INVALID),                   # ... but the rows lie apart
    (P + ROW, 256, fa.FA_ERR_INVALID), (P - 8 * ROW, 256, fa.FA_ERR_INVALID), (P + 8 * ROW, 256, fa.FA_ERR_INVALID),
    (P + 9 * ROW, 256, fa.FA_ERR_WORKSPACE), (P - 9 * ROW, 256, fa.FA_ERR_WORKSPACE)])
def test_attention_output_may_be_the_queries_or_apart_from_them(lib, o, stride, code):
    assert _attn(lib, _cache(), _batch(max_pages=100000), o=o, stride=stride) == code


@pytest.mark.parametrize("kw", [
    dict(qo=P + ROW), dict(qo=P - ROW), dict(qo=P, qos=512), dict(qo=P, qs=512),
    # slices of a fused projection of 8 heads: queries 0..3, keys 4..5, values 6..7
    dict(qs=512, qos=512, ks=512, vs=512, k=P + ROW, v=P + ROW + ROW // 2, qo=P + 16),
    dict(qs=512, qos=512, ks=512, vs=512, k=P + ROW, v=P + ROW + ROW // 2, qo=P + ROW),
    dict(qs=512, qos=512, ks=512, vs=512, k=P + ROW, v=P + ROW + ROW // 2, qo=P - 16),
    dict(qo=P + 0x10000, k=P + 0x10000 + 8 * ROW), dict(qo=P + 0x10000, v=P + 0x10000 - 8 * 256)])
def test_rotated_queries_may_not_overlap_the_inputs(lib, kw):
    assert _append(lib, _cache(), _batch(), **kw) == fa.FA_ERR_INVALID


def test_workspace(lib):
    c, b = _cache(page_size=64, num_heads=2), _batch(B=3, T=3, cu_q=0, max_q=1, max_pages=100000)
    need = lib.fa_paged_attn_workspace_bytes(ctypes.addressof(c), ctypes.addressof(b), 8)
    # the states of two pieces of 8 rows (d + 1 floats each) for several CTAs on each of at least 100 SMs
    assert need >= 200 * 2 * 8 * (64 + 1) * 4
    b.max_kv = 100   # so little that a cluster takes each sequence and head
    assert lib.fa_paged_attn_workspace_bytes(ctypes.addressof(c), ctypes.addressof(b), 8) == 0
    assert lib.fa_paged_attn_workspace_bytes(ctypes.addressof(c), ctypes.addressof(b), 7) == 0  # heads do not divide


def test_the_library_builds_without_pytorch(lib, monkeypatch, tmp_path):
    from exact_io_aware_33_gb300 import build
    monkeypatch.setattr(build, "_has_torch", lambda: False)
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "binding.so"))
    monkeypatch.setattr(build, "_binding_flags", lambda: pytest.fail("the binding's flags need PyTorch"))
    assert build.build() == build.LIB
    assert not (tmp_path / "binding.so").exists()


@pytest.fixture
def fake_build(monkeypatch, tmp_path):
    """build.py with compilers that only write down what they were asked for; g++ fails on request."""
    from exact_io_aware_33_gb300 import build
    tool = tmp_path / "bin" / "tool"
    tool.parent.mkdir()
    tool.write_text(f'''#!/bin/sh
echo "$0 $@" >> {tmp_path}/log
if [ "${{0##*/}}" = g++ ] && [ -e {tmp_path}/fail ]; then echo no such header; exit 1; fi
while [ $# -gt 0 ]; do [ "$1" = -o ] && touch "$2"; shift; done
''')
    tool.chmod(0o755)
    for name in ("nvcc", "g++"):
        (tmp_path / "bin" / name).symlink_to(tool)
        monkeypatch.setattr(build, {"nvcc": "nvcc", "g++": "cxx"}[name], lambda p=str(tmp_path / "bin" / name): p)
    for name, value in (("BUILD", "obj"), ("LIB", "libfa.so"), ("BINDING", "binding.so")):
        monkeypatch.setattr(build, name, str(tmp_path / value))

    def asked(word):  # command lines with the word since the last look
        log = tmp_path / "log"
        lines = log.read_text().splitlines() if log.exists() else []
        log.write_text("")
        return [x for x in lines if word in x]
    return build, tmp_path, asked


def test_the_library_is_built_where_the_binding_is_not(fake_build, monkeypatch, capsys):
    build, tmp, asked = fake_build
    assert build.build() == build.LIB and (tmp / "binding.so").exists()
    (tmp / "fail").touch()
    (tmp / "libfa.so").unlink()
    assert build.build(force=True) == build.LIB
    assert (tmp / "libfa.so").exists()
    assert not (tmp / "binding.so").exists()                     # the old one does not fit any more
    assert "no such header" in capsys.readouterr().err
    (tmp / "fail").unlink()
    assert build.build() == build.LIB and (tmp / "binding.so").exists()
    for name in ("cxx", "_binding_flags"):                       # no g++; a PyTorch that cannot be imported
        with monkeypatch.context() as m:
            def missing(*_):
                raise (RuntimeError if name == "cxx" else ImportError)(f"{name} is missing")
            m.setattr(build, name, missing)
            (tmp / "libfa.so").unlink()
            assert build.build(force=True) == build.LIB and (tmp / "libfa.so").exists()
            assert not (tmp / "binding.so").exists() and f"{name} is missing" in capsys.readouterr().err


def test_the_binding_is_built_again_for_another_pytorch(fake_build, monkeypatch):
    build, tmp, asked = fake_build
    build.build()
    assert len(asked("g++")) == 2    # compiled and linked
    build.build()
    assert asked("") == []           # nothing to do
    monkeypatch.setattr(build, "_binding_stamp", lambda: "another one")
    build.build()
    assert len(asked("g++")) == 2
    build.build()
    assert asked("") == []


def test_a_failing_cuda_source_is_still_an_error(fake_build, monkeypatch):
    build, tmp, asked = fake_build
    monkeypatch.setattr(build, "nvcc", lambda: "/bin/false")
    with pytest.raises(RuntimeError, match="nvcc failed"):
        build.build()


@pytest.fixture
def on_the_cpu(lib, monkeypatch):
    """A PagedCache and a PagedBatch of CPU tensors, for what can be refused before a device is looked at."""
    monkeypatch.setattr(fa.paged, "_require", lambda *a: None)
    pages = [torch.zeros(4, 2, 16, 64, dtype=torch.float8_e4m3fn) for _ in range(2)]
    cache = fa.PagedCache(*pages, torch.ones(4, 2), torch.ones(4, 2))
    ints = lambda *shape: torch.zeros(shape, dtype=torch.int32)  # noqa: E731
    return cache, fa.PagedBatch(ints(3, 4), ints(3), ints(4), max_q=2)


def test_what_a_cache_and_a_batch_hold_cannot_be_exchanged(on_the_cpu):
    cache, batch = on_the_cpu
    for obj, names in ((cache, ("k_pages", "v_scales", "page_size", "d", "_address")),
                       (batch, ("block_table", "kv_lens", "cu_q", "max_kv", "max_q", "B"))):
        for name in names:
            before = getattr(obj, name)
            with pytest.raises(AttributeError, match=name):
                setattr(obj, name, before)
            with pytest.raises(AttributeError, match=name):
                delattr(obj, name)
            assert getattr(obj, name) is before


@pytest.mark.parametrize("which,name,n_fields", [(0, n, 4) for n in ("k_pages", "v_pages", "k_scales", "v_scales")]
                         + [(1, n, 3) for n in ("block_table", "kv_lens", "cu_q")])
def test_tensors_whose_memory_has_moved_are_refused(on_the_cpu, which, name, n_fields):
    cache, batch = on_the_cpu
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    def attn():
        return fa.paged._native.attn(cache._address, cache._held, batch._address, batch._held, 0, q, 0, 0.125, None, None, None)
    def append():
        return fa.paged._native.append(cache._address, cache._held, batch._address, batch._held, 0, q, q, None, None, None,
                                       False, None)
    for call in (attn, append):   # as they are, the calls get as far as q
        with pytest.raises(ValueError, match="CUDA"):
            call()
    t = getattr((cache, batch)[which], name)
    t.data = t.detach().clone()
    for call in (attn, append):
        with pytest.raises(ValueError, match=f"{name} has moved"):
            call()


def test_binding_refuses_cpu_tensors():
    pages = torch.zeros(4, 2, 16, 64, dtype=torch.float8_e4m3fn)
    scales = torch.ones(4, 2)
    with pytest.raises(ValueError, match="CUDA"):
        fa.PagedCache(pages, pages, scales, scales)
    with pytest.raises(ValueError, match="CUDA"):
        fa.PagedBatch(torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
