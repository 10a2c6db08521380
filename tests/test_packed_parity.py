"""Packed sequences on the GPU: fa_rope_axes, fa_packed_fwd and fa_packed_bwd against the float64 oracle.

Tolerances, derived from the arithmetic:

* rope: each product and sum is rounded to float32 by definition and the result to bf16; compared bit for bit.
* o: one rounding to bf16 (2^-8 of the value), and P rounded to bf16 (2^-8 of each weight: at most 2^-8 A with A =
  sum_j p_j |v_j|). Float32 sums of S err by at most 128 * 2^-24 sum_c |q_c k_c|, below 2^-11 in the exponent here
  (sum |q_c k_c| scale <= 64), and exponentials and sums by less than 2^-12: together below 2^-10 A.
  Bound: 2^-8 |o| + (2^-8 + 2^-10) A.
* gradients, of the same o and lse on both sides: one rounding to bf16 (2^-8 of the value); P and dS rounded to bf16
  (2^-8 of each) and P's own error from S (below 2^-10 of it, as above): (2^-8 + 2^-10) A with A the sum of the
  absolute terms, sum P |dO| for dV and scale sum |dS| |k| or |q| for dQ and dK; and dP - D, whose 128-term float32 sums
  err by at most 2^-17 of the sums of their absolute terms each: 2^-16 B with B = scale sum P (|dO| |v| + |dO| |o|) |k|
  or |q|.
* lse: the error of S enters it unchanged: 128 * 2^-24 * 64 = 4.9e-4 at the very most. Bound: 5e-4.
"""

import math

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


# ------------------------------------------------------------------ attention
class Rows:
    """q, k and v of packed sequences, side by side in one tensor; `lead` rows before the sequences and `trail` behind
    them are no sequence's and hold NaN."""

    def __init__(self, lens, Hq, Hkv, d, seed, lead=0, trail=0):
        rng = self.rng = np.random.default_rng(seed)
        self.Hq, self.Hkv, self.d, self.G = Hq, Hkv, d, Hq // Hkv
        self.cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32) + lead
        self.T = int(self.cu[-1]) + trail
        self.inside = np.zeros(self.T, dtype=bool)
        self.inside[self.cu[0]:self.cu[-1]] = True
        self.whole = randn(rng, self.T, (Hq + 2 * Hkv) * d + 8)
        self.whole[~torch.from_numpy(self.inside)] = float("nan")
        self.q, self.k, self.v = self.views(self.whole)

    def views(self, whole):
        a, b = self.Hq * self.d, self.Hkv * self.d
        return (whole[:, :a].view(self.T, self.Hq, self.d), whole[:, a:a + b].view(self.T, self.Hkv, self.d),
                whole[:, a + b:a + 2 * b].view(self.T, self.Hkv, self.d))

    def on_gpu(self):
        return self.views(self.whole.cuda()), torch.from_numpy(self.cu).cuda()


def f64(*xs):
    return [x.float().cpu().double().numpy() for x in xs]


def check_fwd(rows, o, lse, causal, scale, window, which=None):
    """Against the oracle in the sequences `which` (all); rows outside the sequences are not looked at."""
    cu = rows.cu
    q, k, v = f64(rows.q, rows.k, rows.v)
    o, lse = f64(o, lse)
    for b in range(len(cu) - 1) if which is None else which:
        at = slice(cu[b], cu[b + 1])
        n = cu[b + 1] - cu[b]
        one = np.array([0, n])
        want, want_lse = packed.forward(q[at], k[at], v[at], one, causal, scale, window)
        A, _ = packed.forward(q[at], k[at], np.abs(v[at]), one, causal, scale, window)
        err = np.abs(o[at] - want) - 2.0 ** -8 * np.abs(want)
        assert n == 0 or (err <= (2.0 ** -8 + 2.0 ** -10) * A).all(), (b, (err / A).max())
        assert (np.abs(lse[at] - want_lse) <= 5e-4).all(), b


FWD = [
    # lens, Hq, Hkv, d, causal, window
    ([1], 1, 1, 64, True, 0),
    ([1], 2, 1, 128, False, 0),
    ([1, 2, 127, 128, 129], 2, 2, 128, True, 0),
    ([255, 256, 257, 0, 3], 1, 1, 64, True, 0),
    ([255, 256, 257, 0, 3], 2, 1, 64, False, 0),
    ([300, 41], 8, 2, 128, True, 0),              # four heads on one, a tile of 32 tokens
    ([300, 41], 6, 2, 128, False, 0),             # three: 42 tokens and two rows over
    ([77, 513], 10, 2, 64, True, 0),
    ([130, 64], 14, 2, 128, True, 0),             # seven: 18 tokens, two rows over
    ([45], 71, 1, 64, True, 0),                   # one token's heads fill a tile half
    ([19, 20], 128, 1, 128, False, 0),
    ([200, 300], 4, 4, 64, True, 1),              # a window of the row itself
    ([500, 129, 700], 4, 2, 128, True, 130),
    ([500, 129, 700], 3, 1, 64, True, 200),
    ([640], 2, 2, 128, True, 127),
    ([640], 2, 2, 64, True, 2 ** 31 - 1),         # as long as there is: none
    ([2100], 8, 1, 128, True, 1000),
    ([1500, 700], 12, 12, 64, False, 0),
    ([3, 1, 4, 1, 5, 9, 2, 6] * 60, 2, 2, 64, True, 0),       # more items than CTAs
    ([33, 0, 100, 7] * 60, 4, 2, 128, True, 0),
    ([33, 0, 100, 7] * 60, 4, 2, 64, False, 0),
    ([1500, 1, 2300, 129], 24, 8, 128, True, 0),
    ([1500, 1, 2300, 129], 24, 12, 64, True, 300),
]


@pytest.mark.parametrize("lens,Hq,Hkv,d,causal,window", FWD)
def test_packed_fwd(lens, Hq, Hkv, d, causal, window):
    rows = Rows(lens, Hq, Hkv, d, seed=sum(lens) + Hq + d, lead=3 if len(lens) > 2 else 0, trail=5)
    (q, k, v), cu = rows.on_gpu()
    out = torch.full((rows.T, Hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((rows.T, Hq), 7.0, device="cuda")
    o, l = fa.fa_packed_fwd(q, k, v, cu, causal=causal, window=window, out=out, lse=lse)
    done()
    assert o is out and l is lse
    check_fwd(rows, o, l, causal, 1 / math.sqrt(d), window)
    outside = torch.from_numpy(~rows.inside).cuda()
    assert (o[outside] == 7).all() and (l[outside] == 7).all()
    again, l2 = fa.fa_packed_fwd(q, k, v, cu, causal=causal, window=window)
    done()
    inside = ~outside
    assert torch.equal(again[inside], o[inside]) and torch.equal(l2[inside], l[inside])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale", [0.0, 1e-30, 1.0])
def test_packed_fwd_scales(d, scale):
    rows = Rows([150, 40], 4, 2, d, seed=d)
    rows.whole *= 0.25                            # (scale 1: sums |q_c k_c| stay below 64)
    (q, k, v), cu = rows.on_gpu()
    o, lse = fa.fa_packed_fwd(q, k, v, cu, causal=True, scale=scale)
    done()
    check_fwd(rows, o, lse, True, scale, 0)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d,G", [(64, 1), (64, 4), (128, 1), (128, 3)])
def test_packed_fwd_what_is_not_finite_stays_in_its_sequence(d, G, causal):
    rows = Rows([100, 60, 200, 90, 300], 2 * G, 2, d, seed=d + G, lead=2, trail=4)
    for b, bad in ((1, float("nan")), (3, float("inf"))):
        rows.whole[rows.cu[b]:rows.cu[b + 1]] = bad
    (q, k, v), cu = rows.on_gpu()
    o, lse = fa.fa_packed_fwd(q, k, v, cu, causal=causal)
    done()
    check_fwd(rows, o, lse, causal, 1 / math.sqrt(d), 0, which=(0, 2, 4))
    assert o[rows.cu[1]:rows.cu[2]].isnan().all()


def test_packed_fwd_large_scores():
    # one key outweighs the others by far, and rows whose maximum grows from tile to tile
    rows = Rows([400], 2, 2, 64, seed=3)
    rows.k[:] = 0
    rows.q[:] = 0
    rows.q[..., 0] = 1
    rows.k[:, :, 0] = torch.arange(400).to(torch.bfloat16)[:, None]
    (q, k, v), cu = rows.on_gpu()
    for causal in (False, True):
        o, lse = fa.fa_packed_fwd(q, k, v, cu, causal=causal, scale=1.0)
        done()
        check_fwd(rows, o, lse, causal, 1.0, 0)


def test_packed_fwd_borders_out_of_range_are_reported():
    rows = Rows([50, 60], 2, 2, 64, seed=4)
    (q, k, v), _ = rows.on_gpu()
    for bad in ([0, 50, 200], [-4, 50, 110], [0, 60, 50], [0, 110, 0, 110, 0, 110]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        fa.fa_packed_fwd(q, k, v, cu, causal=True)
        done(fa.FA_ERR_INDEX)
    good = torch.tensor([0, 50, 110], dtype=torch.int32, device="cuda")
    o, lse = fa.fa_packed_fwd(q, k, v, torch.tensor([0, 50, 200], dtype=torch.int32, device="cuda"), causal=True)
    done(fa.FA_ERR_INDEX)
    want, _ = fa.fa_packed_fwd(q, k, v, good, causal=True)
    done()
    assert torch.equal(o, want)                   # clamped to the rows there are


def test_packed_fwd_too_many_overlapping_rows_for_the_list():
    # borders that fall and rise again name more rows than there are: the list holds what fits
    rows = Rows([700] * 4, 2, 2, 64, seed=5)
    (q, k, v), _ = rows.on_gpu()
    cu = torch.tensor([0, 2800] * 300, dtype=torch.int32, device="cuda")
    fa.fa_packed_fwd(q, k, v, cu, causal=True)
    done(fa.FA_ERR_INDEX)


@pytest.mark.parametrize("B,at", [(100, 50), (3000, 2500), (70000, 69999)])
def test_borders_that_fall_make_no_work(B, at):
    """Thousands of sequences that each hold all rows would be hours of work: a list of them stays empty."""
    T = 100000
    q, out = (torch.ones(T, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    outs, lse = [torch.full_like(q, 3) for _ in range(3)], torch.full((T, 2), 7.0, device="cuda")
    for cu in ([0, T] * (B // 2), [T // 2] * at + [0] + [T] * (B - at)):
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        fa.fa_packed_fwd(q, q, q, cu, out=out, lse=lse, causal=True)
        done(fa.FA_ERR_INDEX)
        fa.fa_packed_bwd(q, q, q, q, torch.zeros_like(lse), q, cu, dq=outs[0], dk=outs[1], dv=outs[2])
        done(fa.FA_ERR_INDEX)
        assert (out == 1).all() and (lse == 7).all() and all((x == 3).all() for x in outs)


def test_packed_fwd_of_nothing():
    for T, B in ((0, 1), (5, 0)):
        q = torch.zeros(T, 2, 64, dtype=torch.bfloat16, device="cuda")
        o, lse = fa.fa_packed_fwd(q, q, q, torch.zeros(B + 1, dtype=torch.int32, device="cuda"), causal=True)
        assert o.shape == (T, 2, 64) and lse.shape == (T, 2)
    q = torch.ones(300, 2, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 3)
    for B in (3, 700):                            # sequences of nothing, with and without a list
        fa.fa_packed_fwd(q, q, q, torch.full((B + 1,), 9, dtype=torch.int32, device="cuda"), out=out)
        done()
        assert (out == 3).all()


@pytest.mark.parametrize("lens", [[200, 130], [200, 3, 0, 130] * 50])
def test_packed_fwd_captured_with_new_borders_and_on_a_stream(lens):
    rows = Rows(lens, 4, 2, 64, seed=6)
    (q, k, v), cu = rows.on_gpu()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    a, _ = fa.fa_packed_fwd(q, k, v, cu, causal=True, stream=s)
    s.synchronize()
    check_fwd(rows, a, torch.zeros(0), True, 0.125, 0, which=())
    b, _ = fa.fa_packed_fwd(q, k, v, cu, causal=True)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = fa.fa_packed_fwd(q, k, v, cu, causal=True)
    rows.cu[1:-1] = np.sort(rows.rng.integers(0, rows.T, len(lens) - 1))
    cu.copy_(torch.from_numpy(rows.cu))
    g.replay()
    done()
    assert torch.equal(a, b)
    check_fwd(rows, o, lse, True, 0.125, 0)


# ------------------------------------------------------------------ gradients
def check_bwd(rows, o, lse, do, grads, causal, scale, window, which=None):
    cu, G = rows.cu, rows.G
    q, k, v = f64(rows.q, rows.k, rows.v)
    o, lse, do = f64(o, lse, do)
    got = dict(zip(("dq", "dk", "dv"), f64(*grads)))
    for b in range(len(cu) - 1) if which is None else which:
        at, n = slice(cu[b], cu[b + 1]), cu[b + 1] - cu[b]
        if n == 0:
            continue
        want = dict(zip(("dq", "dk", "dv"), packed.backward(q[at], k[at], v[at], o[at], lse[at], do[at], np.array([0, n]),
                                                            causal, scale, window)))
        bound = {x: 2.0 ** -8 * np.abs(want[x]) for x in want}
        far = np.arange(n)[:, None] - np.arange(n)
        seen = ((far >= 0) if causal else True) & ((far < window) if window else True)
        for h in range(rows.Hq):
            qh, kh, vh, oh, dh = q[at, h], k[at, h // G], v[at, h // G], o[at, h], do[at, h]
            p = np.where(seen, np.exp(np.where(seen, scale * (qh @ kh.T) - lse[at, h][:, None], 0)), 0)
            ds = np.abs(p * (dh @ vh.T - (dh * oh).sum(-1)[:, None]))
            off = p * (np.abs(dh) @ np.abs(vh).T + (np.abs(dh) * np.abs(oh)).sum(-1)[:, None])
            each = scale * ((2.0 ** -8 + 2.0 ** -10) * ds + 2.0 ** -16 * off)
            bound["dq"][:, h] += each @ np.abs(kh)
            bound["dk"][:, h // G] += each.T @ np.abs(qh)
            bound["dv"][:, h // G] += (2.0 ** -8 + 2.0 ** -10) * (p.T @ np.abs(dh))
        for x in want:
            err = np.abs(got[x][at] - want[x])
            assert (err <= bound[x]).all(), (b, x, (err / np.maximum(bound[x], 1e-300)).max())


def forward_for(rows, causal, scale, window):
    """The forward's results, from the oracle, where there are sequences; NaN elsewhere."""
    o, lse = packed.forward(*f64(rows.q, rows.k, rows.v), rows.cu, causal, scale, window)
    return torch.from_numpy(o).to(torch.bfloat16), torch.from_numpy(lse).float()


BWD = [
    # lens, Hq, Hkv, d, causal, window
    ([1], 1, 1, 64, True, 0),
    ([1], 2, 1, 128, False, 0),
    ([1, 2, 127, 128, 129], 2, 2, 128, True, 0),
    ([255, 256, 257, 0, 3], 1, 1, 64, True, 0),
    ([255, 256, 257, 0, 3], 2, 1, 64, False, 0),
    ([300, 41], 8, 2, 128, True, 0),
    ([300, 41], 6, 2, 128, False, 0),
    ([77, 513], 10, 2, 64, True, 0),
    ([130, 64], 14, 2, 128, True, 0),
    ([45], 71, 1, 64, True, 0),
    ([19, 20], 128, 1, 128, False, 0),
    ([200, 300], 4, 4, 64, True, 1),
    ([500, 129, 700], 4, 2, 128, True, 130),
    ([500, 129, 700], 3, 1, 64, True, 200),
    ([640], 2, 2, 128, True, 127),
    ([640], 2, 2, 64, True, 2 ** 31 - 1),
    ([1100], 8, 1, 128, True, 400),
    ([1000, 700], 3, 3, 64, False, 0),
    ([3, 1, 4, 1, 5, 9, 2, 6] * 60, 2, 2, 64, True, 0),
    ([33, 0, 100, 7] * 60, 4, 2, 128, True, 0),
    ([33, 0, 100, 7] * 60, 4, 2, 64, False, 0),
    ([1200, 1, 900, 129], 12, 4, 128, True, 0),
    ([1200, 1, 900, 129], 8, 4, 64, True, 300),
]


@pytest.mark.parametrize("lens,Hq,Hkv,d,causal,window", BWD)
def test_packed_bwd(lens, Hq, Hkv, d, causal, window):
    rows = Rows(lens, Hq, Hkv, d, seed=sum(lens) + Hq + d, lead=3 if len(lens) > 2 else 0, trail=5)
    scale = 1 / math.sqrt(d)
    o, lse = forward_for(rows, causal, scale, window)
    wide = randn(rows.rng, rows.T, Hq * d + 64)
    wide[~torch.from_numpy(rows.inside)] = float("nan")
    do = wide[:, :Hq * d].view(rows.T, Hq, d)
    (q, k, v), cu = rows.on_gpu()
    args = (q, k, v, o.cuda(), lse.cuda(), wide.cuda()[:, :Hq * d].view(rows.T, Hq, d), cu)
    # into one gradient of the projection that q, k and v are slices of
    whole = torch.full_like(rows.whole, 7).cuda()
    outs = rows.views(whole)
    got = fa.fa_packed_bwd(*args, causal=causal, window=window, dq=outs[0], dk=outs[1], dv=outs[2])
    done()
    assert all(a is b for a, b in zip(got, outs))
    check_bwd(rows, o, lse, do, got, causal, scale, window)
    assert (whole[torch.from_numpy(~rows.inside).cuda()] == 7).all() and (whole[:, -8:] == 7).all()
    again = fa.fa_packed_bwd(*args, causal=causal, window=window)
    done()
    inside = torch.from_numpy(rows.inside).cuda()
    for a, b in zip(again, got):
        assert torch.equal(a[inside], b[inside])


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d,G", [(64, 1), (64, 4), (128, 1), (128, 3)])
def test_packed_bwd_what_is_not_finite_stays_in_its_sequence(d, G, causal):
    rows = Rows([100, 60, 200, 90, 300], 2 * G, 2, d, seed=d + G, lead=2, trail=4)
    scale = 1 / math.sqrt(d)
    o, lse = forward_for(rows, causal, scale, 0)
    do = randn(rows.rng, rows.T, 2 * G, d)
    for b, bad in ((1, float("nan")), (3, float("inf"))):
        at = slice(int(rows.cu[b]), int(rows.cu[b + 1]))
        for x in (rows.whole, o, lse, do):
            x[at] = bad
    (q, k, v), cu = rows.on_gpu()
    got = fa.fa_packed_bwd(q, k, v, o.cuda(), lse.cuda(), do.cuda(), cu, causal=causal)
    done()
    check_bwd(rows, o, lse, do, got, causal, scale, 0, which=(0, 2, 4))
    assert all(x[rows.cu[1]:rows.cu[2]].isnan().all() for x in got)


@pytest.mark.parametrize("d,G", [(64, 1), (64, 5), (128, 1), (128, 8)])
@pytest.mark.parametrize("lens,causal,window", [([1] * 300, False, 0), ([1, 0, 1], True, 0), ([70, 300, 1], True, 1)])
def test_packed_bwd_where_each_row_sees_one_key(lens, causal, window, d, G):
    """The softmax of one score does not depend on it: dq and dk are zero, and dv is dO, summed over the group."""
    rows = Rows(lens, 2 * G, 2, d, seed=d + G)
    (q, k, v), cu = rows.on_gpu()
    do = randn(rows.rng, rows.T, 2 * G, d)
    o, lse = fa.fa_packed_fwd(q, k, v, cu, causal=causal, window=window)
    dq, dk, dv = fa.fa_packed_bwd(q, k, v, o, lse, do.cuda(), cu, causal=causal, window=window)
    done()
    assert not dq.any() and not dk.any()
    check_bwd(rows, o.cpu(), lse.cpu(), do, (dq, dk, dv), causal, 1 / math.sqrt(d), window)


@pytest.mark.parametrize("d", [64, 128])
def test_packed_bwd_against_differences(d):
    """The loss sum(o dO) of the GPU's own forward, along a direction, against the GPU's gradients.

    Both ends of a difference carry o's rounding and P's (2^-8 of o at most each, so of o's size a deviation of 2^-8 /
    sqrt(3) each, independent over the elements): the difference deviates by 2 * 2^-8 / sqrt(3) norm(o dO). Six of these;
    and 2^-6 of the norm of the gradient's terms for their own roundings (2^-7) and the third derivative: a step of h in
    each channel moves a score by about h, and h^2 / 6 < 2^-10."""
    rows = Rows([90, 200], 4, 2, d, seed=d)
    do = randn(rows.rng, rows.T, 4, d).cuda()
    (q, k, v), cu = rows.on_gpu()
    o, lse = fa.fa_packed_fwd(q, k, v, cu, causal=True)
    grads = fa.fa_packed_bwd(q, k, v, o, lse, do, cu, causal=True)
    done()
    h = 1 / 16
    for i, x in enumerate((q, k, v)):
        step = randn(rows.rng, *x.shape).cuda().sign() * h
        ends = [(x.float() + s * step.float()).to(torch.bfloat16) for s in (1, -1)]
        moved = (ends[0].double() - ends[1].double())
        loss = []
        for e in ends:
            args = [q, k, v]
            args[i] = e
            loss.append(float((fa.fa_packed_fwd(*args, cu, causal=True)[0].double() * do.double()).sum()))
        got, want = loss[0] - loss[1], float((grads[i].double() * moved).sum())
        noise = 2 * 2.0 ** -8 / math.sqrt(3) * float((o.double() * do.double()).norm())
        size = float((grads[i].double() * moved).norm())
        assert abs(got - want) <= 6 * noise + 2.0 ** -6 * size, (i, got, want, noise, size)


def test_packed_bwd_borders_out_of_range_are_reported():
    rows = Rows([50, 60], 2, 2, 64, seed=4)
    (q, k, v), _ = rows.on_gpu()
    o, lse = (x.cuda() for x in forward_for(rows, True, 0.125, 0))
    for bad in ([0, 50, 200], [-4, 50, 110], [0, 60, 50], [0, 110] * 200):
        fa.fa_packed_bwd(q, k, v, o, lse, o, torch.tensor(bad, dtype=torch.int32, device="cuda"), causal=True)
        done(fa.FA_ERR_INDEX)


def test_packed_bwd_of_nothing():
    q = torch.ones(300, 2, 64, dtype=torch.bfloat16, device="cuda")
    lse, out = torch.zeros(300, 2, device="cuda"), [torch.full_like(q, 3) for _ in range(3)]
    for B in (3, 700):
        cu = torch.full((B + 1,), 9, dtype=torch.int32, device="cuda")
        fa.fa_packed_bwd(q, q, q, q, lse, q, cu, dq=out[0], dk=out[1], dv=out[2])
        done()
        assert all((x == 3).all() for x in out)
    e = q[:0]
    assert all(x.shape == (0, 2, 64) for x in fa.fa_packed_bwd(e, e, e, e, lse[:0], e, cu))


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("d,Hq,Hkv,window", [(64, 6, 2, 0), (128, 8, 2, 50)])
def test_a_layer_and_its_gradients_in_one_graph(d, Hq, Hkv, window):
    """Rotation, attention and both backwards on slices of one projection, eagerly, then captured and replayed with
    other lengths and inputs."""
    lens = [70, 1, 0, 190, 33]
    rows = Rows(lens, Hq, Hkv, d, seed=d)
    half = d // 2
    cos, sin = tables(64, half)
    sections = (half // 4, half // 4, half // 2)
    axis_of = [a for a, m in enumerate(sections) for _ in range(m)]
    pos = rows.rng.integers(0, 64, (3, rows.T)).astype(np.int32)
    whole, posg, cu = rows.whole.cuda(), torch.from_numpy(pos).cuda(), torch.from_numpy(rows.cu).cuda()
    rope = (torch.from_numpy(cos).cuda(), torch.from_numpy(sin).cuda())
    do = randn(rows.rng, rows.T, Hq, d).cuda()
    back = torch.zeros_like(whole)
    q, k, v = rows.views(whole)
    dq, dk, dv = rows.views(back)

    def layer():
        a, b = fa.fa_rope_axes(q, k, posg, rope, sections=sections)
        o, lse = fa.fa_packed_fwd(a, b, v, cu, causal=True, window=window)
        fa.fa_packed_bwd(a, b, v, o, lse, do, cu, causal=True, window=window, dq=dq, dk=dk, dv=dv)
        fa.fa_rope_axes(dq, dk, posg, rope, sections=sections, inverse=True, q_out=dq, k_out=dk)
        return a, b, o, lse

    def check(a, b, o, lse):
        done()
        now = Rows.__new__(Rows)
        now.__dict__.update(rows.__dict__)
        now.q, now.k, now.v = (x.cpu() for x in (a, b, v))
        check_fwd(now, o, lse, True, 1 / math.sqrt(d), window)
        turned = [want_rope(x.cpu(), pos, axis_of, cos, sin, False, False) for x in (q, k)]
        assert torch.equal(a.cpu(), turned[0]) and torch.equal(b.cpu(), turned[1])
        grads = fa.fa_packed_bwd(a, b, v, o, lse, do, cu, causal=True, window=window)
        check_bwd(now, o, lse, do, grads, True, 1 / math.sqrt(d), window)
        assert torch.equal(dq.cpu(), want_rope(grads[0].cpu(), pos, axis_of, cos, sin, False, True))
        assert torch.equal(dk.cpu(), want_rope(grads[1].cpu(), pos, axis_of, cos, sin, False, True))
        assert torch.equal(dv, grads[2])

    check(*layer())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = layer()
    rows.cu[1:-1] = np.sort(rows.rng.integers(0, rows.T, len(lens) - 1))
    cu.copy_(torch.from_numpy(rows.cu))
    whole.copy_(randn(rows.rng, *whole.shape))
    g.replay()
    check(*outs)


def test_a_prompt_and_its_answer_with_positions_of_several_axes():
    """The prompt: rotation, attention over its own rows, its keys and values into the pages. Then token by token:
    rotation, append, attention over the pages."""
    from test_paged_parity import World, check_attn, check_cache
    lens, Hq, Hkv, d, sections = [45, 1, 130], 8, 2, 128, (16, 24, 24)
    rows = Rows(lens, Hq, Hkv, d, seed=31)
    w = World([n + 4 for n in lens], Hkv, 16, d, seed=32)
    cache, cos_sin = w.to_gpu(), tables(200, 64)
    rope = tuple(torch.from_numpy(x).cuda() for x in cos_sin)
    axis_of = [a for a, m in enumerate(sections) for _ in range(m)]
    turned = lambda x, pos: want_rope(x, pos, axis_of, *cos_sin, False, False)  # noqa: E731

    def rotated(q, k, pos):
        a, b = fa.fa_rope_axes(q, k, torch.from_numpy(pos).cuda(), rope, sections=sections)
        assert torch.equal(a.cpu(), turned(q.cpu(), pos)) and torch.equal(b.cpu(), turned(k.cpu(), pos))
        return a, b

    (q, k, v), cu = rows.on_gpu()
    a, b = rotated(q, k, w.rng.integers(0, 200, (3, rows.T)).astype(np.int32))
    o, lse = fa.fa_packed_fwd(a, b, v, cu, causal=True)
    w.lens = lens
    host, batch = w.batch(lens)
    fa.fa_paged_append(cache, batch, b, v)
    done()
    rows.q, rows.k = a.cpu(), b.cpu()
    check_fwd(rows, o, lse, True, 1 / math.sqrt(d), 0)
    w.oracle.append(w.table, lens, host, rows.k.float().numpy(), rows.v.float().numpy())
    check_cache(w, cache)
    for step in range(1, 5):
        w.lens = [n + step for n in lens]
        host, batch = w.batch([1, 1, 1])
        q, k, v = (randn(w.rng, 3, h, d).cuda() for h in (Hq, Hkv, Hkv))
        a, b = rotated(q, k, w.rng.integers(0, 200, (3, 3)).astype(np.int32))
        fa.fa_paged_append(cache, batch, b, v)
        o, lse = fa.fa_paged_attn(cache, batch, a)
        done()
        w.oracle.append(w.table, w.lens, host, b.cpu().float().numpy(), v.cpu().float().numpy())
        check_cache(w, cache)
        check_attn(w, host, o, lse, a.cpu(), 1 / math.sqrt(d))


# ------------------------------------------------------------------ layouts, sizes, calls at once
def backward_of(rows, o, lse, do, causal, window, **kw):
    (q, k, v), cu = rows.on_gpu()
    return fa.fa_packed_bwd(q, k, v, o.cuda(), lse.cuda(), do.cuda(), cu, causal=causal, window=window, **kw)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale", [0.0, 1e-30, 1.0])
def test_packed_bwd_scales(d, scale):
    rows = Rows([150, 40], 4, 2, d, seed=d + 1)
    rows.whole *= 0.25
    o, lse = forward_for(rows, True, scale, 0)
    do = randn(rows.rng, rows.T, 4, d)
    got = backward_of(rows, o, lse, do, True, 0, scale=scale)
    done()
    check_bwd(rows, o, lse, do, got, True, scale, 0)


@pytest.mark.parametrize("d", [64, 128])
def test_rows_at_odd_distances_and_bases(d):
    """Bases that are multiples of 16 bytes and of nothing more, row distances that are odd multiples of 16 bytes."""
    rows = Rows([90, 3, 200], 6, 2, d, seed=d + 2, trail=2)
    scale = 1 / math.sqrt(d)
    o, lse = forward_for(rows, True, scale, 0)
    do = randn(rows.rng, rows.T, 6, d)

    def apart(x, lead, extra):
        T, H, _ = x.shape
        flat = torch.full((lead + T * (H * d + extra),), 7.0, dtype=torch.bfloat16, device="cuda")
        view = flat[lead:].view(T, H * d + extra)[:, :H * d].view(T, H, d)
        view.copy_(x)
        return view, flat

    q, k, v, g = (apart(x, *at)[0] for x, at in ((rows.q, (8, 8)), (rows.k, (24, 40)), (rows.v, (40, 24)), (do, (56, 8))))
    outs = [apart(torch.full_like(x, 7.0), *at) for x, at in ((rows.q, (8, 24)), (rows.k, (8, 8)), (rows.v, (24, 40)))]
    cu = torch.from_numpy(rows.cu).cuda()
    og = torch.full((8 + o.numel(),), 7.0, dtype=torch.bfloat16, device="cuda")[8:].view(o.shape)
    got, l = fa.fa_packed_fwd(q, k, v, cu, causal=True, out=og)
    check_fwd(rows, got, l, True, scale, 0)
    og.copy_(o)
    before = [flat.clone() for _, flat in outs]
    grads = fa.fa_packed_bwd(q, k, v, og, lse.cuda(), g, cu, causal=True, dq=outs[0][0], dk=outs[1][0], dv=outs[2][0])
    done()
    check_bwd(rows, o, lse, do, grads, True, scale, 0)
    for (view, flat), was in zip(outs, before):      # and nothing between the rows or behind them
        view[rows.cu[0]:rows.cu[-1]] = 7.0
        assert torch.equal(flat, was)


class Slice:
    """Rows [lo, hi) of tensors on the GPU, as `Rows` of one sequence."""

    def __init__(self, q, k, v, lo, hi):
        self.q, self.k, self.v = (x[lo:hi].cpu() for x in (q, k, v))
        self.cu, self.T = np.array([0, hi - lo]), hi - lo
        self.Hq, self.G = q.shape[1], q.shape[1] // k.shape[1]


@pytest.mark.parametrize("layout", ["many rows", "far rows"])
def test_offsets_past_32_bits(layout):
    """More than 2^31 elements: of many rows of many heads, and of rows that lie far apart."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    d, n = 128, 100
    if layout == "many rows":
        Hq, Hkv, B, wide = 128, 2, 1400, 0
    else:
        Hq, Hkv, B, wide = 4, 2, 6, 1 << 22
    T = B * n
    whole = torch.empty(T, wide or Hq * d, dtype=torch.bfloat16, device="cuda")
    assert whole.numel() > 2 ** 31
    q = whole[:, -Hq * d:].view(T, Hq, d)
    q.normal_(generator=gen)
    k, v = (torch.empty(T, Hkv, d, dtype=torch.bfloat16, device="cuda").normal_(generator=gen) for _ in range(2))
    do = torch.empty(T, Hq, d, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    cu = torch.arange(0, T + 1, n, dtype=torch.int32, device="cuda")
    cos, sin = tables(50, d // 2)
    pos = (torch.arange(T, dtype=torch.int32, device="cuda") % 50)[None].contiguous()
    last = q[-n:].cpu()
    a, b = fa.fa_rope_axes(q, k, pos, (torch.from_numpy(cos).cuda(), torch.from_numpy(sin).cuda()), sections=(d // 2,),
                           q_out=q)
    assert torch.equal(q[-n:].cpu(), want_rope(last, pos[:, -n:].cpu().numpy(), [0] * (d // 2), cos, sin, False, False))
    o, lse = fa.fa_packed_fwd(q, b, v, cu, causal=True)
    grad = torch.empty_like(whole)[:, :Hq * d].view(T, Hq, d)
    grads = fa.fa_packed_bwd(q, b, v, o, lse, do, cu, causal=True, dq=grad)
    done()
    for lo in (0, T - n):
        at = slice(lo, lo + n)
        one = Slice(q, b, v, lo, lo + n)
        check_fwd(one, o[at], lse[at], True, 1 / math.sqrt(d), 0)
        check_bwd(one, o[at].cpu(), lse[at].cpu(), do[at].cpu(), [x[at] for x in grads], True, 1 / math.sqrt(d), 0)


def test_heads_past_32_bits():
    """One token with so many heads that a row has more than 2^31 elements."""
    H, d = (1 << 24) + 8, 128
    gen = torch.Generator(device="cuda").manual_seed(2)
    q, k, v, do = (torch.empty(1, H, d, dtype=torch.bfloat16, device="cuda").normal_(generator=gen) for _ in range(4))
    assert q.numel() > 2 ** 31
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    o, lse = fa.fa_packed_fwd(q, k, v, cu)
    grads = fa.fa_packed_bwd(q, k, v, o, lse, do, cu)
    done()
    assert torch.equal(o, v)                     # its own key alone
    for at in (slice(0, 4), slice(H - 4, H)):
        one = Slice(q[:, at], k[:, at], v[:, at], 0, 1)
        check_fwd(one, o[:, at], lse[:, at], False, 1 / math.sqrt(d), 0)
        check_bwd(one, o[:, at].cpu(), lse[:, at].cpu(), do[:, at].cpu(), [x[:, at] for x in grads], False, 1 / math.sqrt(d), 0)


def test_two_streams_with_workspaces_of_their_own():
    both = []
    for i, (lens, Hq, d) in enumerate((([700, 3, 1200, 40] * 3, 8, 128), ([33, 2000, 500, 0] * 3, 12, 64))):
        rows = Rows(lens, Hq, 4, d, seed=40 + i)
        (q, k, v), cu = rows.on_gpu()
        do = randn(rows.rng, rows.T, Hq, d).cuda()
        o, lse = fa.fa_packed_fwd(q, k, v, cu, causal=True)
        want = (o, lse, *fa.fa_packed_bwd(q, k, v, o, lse, do, cu, causal=True))
        both.append((q, k, v, o, lse, do, cu, want, torch.cuda.Stream()))
    done()
    outs = []
    for _ in range(4):
        for q, k, v, o, lse, do, cu, _, s in both:
            outs.append((*fa.fa_packed_fwd(q, k, v, cu, causal=True, stream=s),
                         *fa.fa_packed_bwd(q, k, v, o, lse, do, cu, causal=True, stream=s)))
    done()
    for i, got in enumerate(outs):
        assert all(torch.equal(a, b) for a, b in zip(got, both[i % 2][7]))


def test_two_graphs_with_one_workspace_in_turn():
    rows = [Rows(lens, 4, 2, 64, seed=50 + i) for i, lens in enumerate(([300, 5, 600, 0] * 40, [90] * 160))]
    ws = torch.empty(max(f(160, r.T, 4, 2, 64) for r in rows for f in (fa.fa_packed_fwd_workspace_bytes,
                                                                      fa.fa_packed_bwd_workspace_bytes)),
                     dtype=torch.uint8, device="cuda").fill_(255)
    made = []
    for r in rows:
        (q, k, v), cu = r.on_gpu()
        do = randn(r.rng, r.T, 4, 64).cuda()

        def step(q=q, k=k, v=v, cu=cu, do=do, **kw):
            o, lse = fa.fa_packed_fwd(q, k, v, cu, causal=True, **kw)
            return (o, lse, *fa.fa_packed_bwd(q, k, v, o, lse, do, cu, causal=True, **kw))

        want = step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = step(workspace=ws)
        made.append((g, got, want, (q, k, v, cu, do)))
    for _ in range(3):
        for g, got, want, _ in made:
            for x in got:
                x.zero_()
            g.replay()
            done()
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_arguments_that_the_binding_refuses():
    T, Hq, Hkv, d = 40000, 4, 2, 64
    q, do = (torch.zeros(T, Hq, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k, v = (torch.zeros(T, Hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(T, Hq, device="cuda")
    fwd = lambda **kw: fa.fa_packed_fwd(**{**dict(q=q, k=k, v=v, cu=cu, causal=True), **kw})  # noqa: E731
    bwd = lambda **kw: fa.fa_packed_bwd(**{**dict(q=q, k=k, v=v, o=o, lse=lse, do=do, cu=cu, causal=True), **kw})  # noqa: E731
    for call in (fwd, bwd):
        for kw in (dict(q=q.half()), dict(k=k.float()), dict(cu=cu.long())):
            with pytest.raises(TypeError):
                call(**kw)
        for kw in (dict(q=q[0]), dict(k=k[1:]), dict(v=v[:, :1]), dict(v=v[:, :, :32]), dict(cu=cu.cpu()), dict(cu=cu[:0]),
                   dict(cu=cu[None]), dict(k=k.cpu()), dict(q=q.transpose(0, 1)), dict(window=2 ** 40),
                   dict(workspace=torch.empty(1 << 24, dtype=torch.uint8))):
            with pytest.raises(ValueError):
                call(**kw)
        for kw in (dict(q=q[:, :3]), dict(window=-1), dict(causal=False, window=3), dict(scale=float("nan")),
                   dict(scale=-0.5), dict(k=k[:1].expand(T, Hkv, d)),
                   dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
            with pytest.raises((fa.FAError, ValueError)):     # (three heads: o has not three, says the binding)
                call(**kw)
    for kw in (dict(out=q[:, :, :32]), dict(out=torch.empty(T, 2 * Hq, d, dtype=torch.bfloat16, device="cuda")[:, ::2]),
               dict(lse=lse[:, :2]), dict(out=torch.empty(T, 2 * Hq * d, dtype=torch.bfloat16, device="cuda")[:, :Hq * d].view(T, Hq, d))):
        with pytest.raises(ValueError):
            fwd(**kw)
    for kw in (dict(out=q), dict(out=torch.empty_like(q).flatten()[4:], causal=False)):
        with pytest.raises((fa.FAError, ValueError)):
            fwd(**kw)
    for kw in (dict(o=torch.empty(T, 2 * Hq * d, dtype=torch.bfloat16, device="cuda")[:, :Hq * d].view(T, Hq, d)),
               dict(lse=lse.double()), dict(lse=lse.t()), dict(do=do[:5]), dict(dq=q[:, :2]), dict(dk=k.float())):
        with pytest.raises((ValueError, TypeError)):
            bwd(**kw)
    for kw in (dict(dq=q), dict(dk=k, dv=torch.empty_like(v)), dict(dq=do), dict(dk=torch.empty_like(k), dv=None, dq=o)):
        with pytest.raises(fa.FAError):
            bwd(**kw)
    same = torch.empty_like(k)
    with pytest.raises(fa.FAError):
        bwd(dk=same, dv=same)
    done()
