"""Packed rows on the GPU: fa_rope_axes against the float64 oracle.

Tolerances, derived from the arithmetic:

* rope: each product and sum is rounded to float32 by definition and the result to bf16; compared bit for bit.
"""

import numpy as np
import pytest

from oracle import packed

torch = pytest.importorskip("torch")
fa = pytest.importorskip("exact_io_aware_33_gb300")

pytestmark = pytest.mark.gpu


def done(code=None):
    torch.cuda.synchronize()
    assert fa.fa_get_last_device_status() == (fa.FA_OK if code is None else code)


def randn(rng, *shape, size=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * size).astype(np.float32)).to(torch.bfloat16)


# ------------------------------------------------------------------ rotary positions
def tables(n, half):
    x = np.arange(n)[:, None] * 10000.0 ** (-np.arange(half) / half)
    return np.cos(x).astype(np.float32), np.sin(x).astype(np.float32)


def want_rope(x, pos, axis_of, cos, sin, interleaved, inverse):
    y = packed.rope(x.float().numpy(), pos, axis_of, cos, sin, interleaved, inverse)
    return torch.from_numpy(y).to(torch.bfloat16)


ROPE = [
    # T, Hq, Hk, d, sections, interleaved, inverse
    (1, 1, 1, 64, (32,), False, False),
    (1, 32, 8, 128, (16, 24, 24), False, False),
    (2, 5, 0, 128, (32, 32), True, False),
    (7, 12, 4, 64, (11, 11, 10), False, True),        # sections that cut the groups of eight pairs
    (33, 3, 1, 64, (3, 13), True, True),              # half of each head
    (1000, 40, 1, 128, (20, 20, 20, 4), False, False),
    (517, 8, 8, 256, (100, 28), False, False),
    (300, 71, 70, 128, (8,), True, False),            # more heads than a block has places for
    (64, 300, 2, 64, (16, 0, 16), False, True),
    (4099, 16, 16, 64, (16, 16), True, True),
]


@pytest.mark.parametrize("T,Hq,Hk,d,sections,interleaved,inverse", ROPE)
def test_rope(T, Hq, Hk, d, sections, interleaved, inverse):
    rng = np.random.default_rng(T + Hq)
    half, n = sum(sections), 97
    pos = rng.integers(0, n, (len(sections), T)).astype(np.int32)
    pos[:, -1] = n - 1
    cos, sin = tables(n, half)
    axis_of = [a for a, m in enumerate(sections) for _ in range(m)]
    # queries and keys lie in one projection, with something behind them
    whole = randn(rng, T, (Hq + Hk) * d + 16)
    q, k = whole[:, :Hq * d].view(T, Hq, d), whole[:, Hq * d:(Hq + Hk) * d].view(T, Hk, d)
    on = whole.cuda()
    qg, kg = on[:, :Hq * d].view(T, Hq, d), on[:, Hq * d:(Hq + Hk) * d].view(T, Hk, d)
    args = (torch.from_numpy(pos).cuda(), (torch.from_numpy(cos).cuda(), torch.from_numpy(sin).cuda()))
    a, b = fa.fa_rope_axes(qg, kg if Hk else None, *args, sections=sections, interleaved=interleaved, inverse=inverse)
    done()
    want_q = want_rope(q, pos, axis_of, cos, sin, interleaved, inverse)
    want_k = want_rope(k, pos, axis_of, cos, sin, interleaved, inverse) if Hk else None
    assert torch.equal(a.cpu(), want_q)
    assert (b is None) if not Hk else torch.equal(b.cpu(), want_k)
    assert torch.equal(on.cpu(), whole)
    # in place, and the axes named one by one
    c, _ = fa.fa_rope_axes(qg, kg if Hk else None, *args, axis_of=axis_of, interleaved=interleaved, inverse=inverse,
                           q_out=qg, k_out=kg if Hk else None)
    done()
    assert c is qg and torch.equal(qg.cpu(), want_q)
    assert not Hk or torch.equal(kg.cpu(), want_k)
    assert torch.equal(on[:, (Hq + Hk) * d:].cpu(), whole[:, (Hq + Hk) * d:])


def test_rope_axes_in_any_order_and_not_finite_values():
    rng = np.random.default_rng(5)
    T, H, d = 50, 3, 128
    pos = rng.integers(0, 60, (3, T)).astype(np.int32)
    axis_of = rng.integers(0, 3, 64).tolist()
    cos, sin = tables(60, 64)
    q = randn(rng, T, H, d)
    q[3, 1, 5], q[4, 2, 64], q[5, 0, 0] = float("inf"), float("nan"), -float("inf")
    got, _ = fa.fa_rope_axes(q.cuda(), None, torch.from_numpy(pos).cuda(), (torch.from_numpy(cos).cuda(),
                             torch.from_numpy(sin).cuda()), axis_of=axis_of)
    done()
    want = want_rope(q, pos, axis_of, cos, sin, False, False)
    assert torch.equal(got.cpu().isnan(), want.isnan())
    assert torch.equal(got.cpu().nan_to_num(), want.nan_to_num())


def test_rope_positions_out_of_range_are_reported():
    q = torch.ones(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    cos, sin = (torch.from_numpy(x).cuda() for x in tables(10, 32))
    pos = torch.tensor([[0, 10, 9, -1], [1, 2, 3, 4]], dtype=torch.int32, device="cuda")
    got, _ = fa.fa_rope_axes(q, None, pos, (cos, sin), sections=(16, 16))
    done(fa.FA_ERR_INDEX)
    want, _ = fa.fa_rope_axes(q, None, pos.clamp(0, 9), (cos, sin), sections=(16, 16))
    done()
    assert torch.equal(got, want)


def test_rope_is_the_paged_append_s_rotation():
    rng = np.random.default_rng(6)
    T, H, d = 37, 4, 128
    q, k = randn(rng, T, H, d).cuda(), randn(rng, T, H, d).cuda()
    cos, sin = (torch.from_numpy(x).cuda() for x in tables(64, 64))
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    batch = fa.PagedBatch(ints([[2, 0, 1]]), ints([T + 5]), ints([0, T]), max_q=T)
    caches = [fa.PagedCache.empty(3, H, 16, d) for _ in range(2)]
    for c in caches:
        for t in (c.k_pages, c.v_pages):
            t.view(torch.uint8).zero_()
        for t in (c.k_scales, c.v_scales):
            t.fill_(1)
    turned = fa.fa_paged_append(caches[0], batch, k, k, q=q, rope=(cos, sin))
    pos = torch.arange(5, T + 5, dtype=torch.int32, device="cuda")[None].contiguous()
    got, _ = fa.fa_rope_axes(q, None, pos, (cos, sin), sections=(64,))
    done()
    assert torch.equal(got, turned)


def test_rope_captured_on_a_stream_and_off_the_current_one():
    rng = np.random.default_rng(7)
    T, Hq, Hk, d = 65, 8, 2, 64
    q, k = randn(rng, T, Hq, d).cuda(), randn(rng, T, Hk, d).cuda()
    cos, sin = (torch.from_numpy(x).cuda() for x in tables(200, 32))
    pos = torch.from_numpy(rng.integers(0, 200, (2, T)).astype(np.int32)).cuda()
    call = lambda **kw: fa.fa_rope_axes(q, k, pos, (cos, sin), sections=(20, 12), **kw)  # noqa: E731
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    a, b = call(stream=s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        x, y = call()
    pos.copy_(torch.from_numpy(rng.integers(0, 200, (2, T)).astype(np.int32)))
    c, e = call()
    g.replay()
    done()
    assert torch.equal(x, c) and torch.equal(y, e) and not torch.equal(a, c)
