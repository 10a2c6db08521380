"""Packed sequences on the GPU where calls are legal and rare: hand-offs under load, values, scales and lengths at the
ends of their ranges. Against the float64 oracle, with the bounds of test_packed_parity.py, or for equal bits."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
fa = pytest.importorskip("exact_io_aware_33_gb300")

from test_packed_parity import Rows, backward_of, check_bwd, check_fwd, done, forward_for, randn  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,G", [(64, 1), (64, 3), (128, 1), (128, 4)])
def test_rows_past_a_sequence_are_zeros_before_they_are_multiplied(d, G):
    """Every second sequence holds NaN, so that the last tiles of the others reach into it, on every SM and again and
    again: the others' bits are those of a call in which it holds zeros."""
    lens = np.random.default_rng(d + G).integers(1, 300, 400).tolist()
    rows = Rows(lens, 2 * G, 2, d, seed=d + G)
    do = randn(rows.rng, rows.T, 2 * G, d)
    kept = np.zeros(rows.T, dtype=bool)
    for b in range(0, len(lens), 2):
        kept[rows.cu[b]:rows.cu[b + 1]] = True
    kept = torch.from_numpy(kept).cuda()
    (q, k, v), cu = rows.on_gpu()
    x = [t.clone() for t in (q, k, v, do.cuda())]
    results = []
    for other in (0.0, float("nan")):
        for t in x:
            t[~kept] = other
        for _ in range(1 if other == 0 else 20):
            o, lse = fa.fa_packed_fwd(*x[:3], cu, causal=True)
            results.append([t[kept] for t in (o, lse, *fa.fa_packed_bwd(*x[:3], o, lse, x[3], cu, causal=True))])
    done()
    for got in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(results[0], got))


# ------------------------------------------------------------------ scales
@pytest.mark.parametrize("d", [64, 128])
def test_the_largest_queries_with_the_smallest_scales(d):
    """The scale takes the queries' size back: powers of two, so the bits are those of queries and a scale of usual size
    (dq's times the size). At 2^100 dq is no normal number where it is below 2^-26, as where a row sees one key and dq
    is the rounding of nothing: to the nearest multiple of 2^-133 it errs by up to 2^-134, which is 2^-34 times the size,
    and the other side by up to 2^-9 of 2^-26: together less than 2^-33."""
    rows = Rows([150, 40], 4, 2, d, seed=d)
    (q, k, v), cu = rows.on_gpu()
    do = randn(rows.rng, rows.T, 4, d).cuda()
    o, lse = fa.fa_packed_fwd(q, k, v, cu, causal=True, scale=0.125)
    dq, dk, dv = fa.fa_packed_bwd(q, k, v, o, lse, do, cu, causal=True, scale=0.125)
    done()
    check_fwd(rows, o, lse, True, 0.125, 0)
    check_bwd(rows, o, lse, do, (dq, dk, dv), True, 0.125, 0)
    for size in (2.0 ** 100, 2.0 ** 120):
        large = (q.float() * size).to(torch.bfloat16)
        got, got_lse = fa.fa_packed_fwd(large, k, v, cu, causal=True, scale=0.125 / size)
        done()
        assert torch.equal(got, o) and torch.equal(got_lse, lse)
        if size > 2.0 ** 100:                     # (sums of dS q would leave float32's range)
            continue
        grads = fa.fa_packed_bwd(large, k, v, o, lse, do, cu, causal=True, scale=0.125 / size)
        done()
        err = (grads[0].double() * size - dq.double()).abs()
        assert (err <= torch.where(dq.double().abs() <= 2.0 ** -26, 2.0 ** -33, 0.0)).all()
        assert torch.equal(grads[1], dk) and torch.equal(grads[2], dv)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale", [0.0, 1e-42])
def test_scales_of_nothing_weigh_all_keys_alike_whatever_the_queries(d, scale):
    rows = Rows([150, 40], 4, 2, d, seed=d)
    rows.q *= 2.0 ** 115                          # (scores times 1e-42: below 1e-5)
    (q, k, v), cu = rows.on_gpu()
    o, lse = fa.fa_packed_fwd(q, k, v, cu, causal=True, scale=scale)
    done()
    check_fwd(rows, o, lse, True, scale, 0)
    o, lse = forward_for(rows, True, 0.0, 0)
    do = randn(rows.rng, rows.T, 4, d)
    got = backward_of(rows, o, lse, do, True, 0, scale=0.0)
    done()
    check_bwd(rows, o, lse, do, got, True, 0.0, 0)
    assert not got[0].any() and not got[1].any()


# ------------------------------------------------------------------ rows that see one key
ONE_KEY = [([40, 1, 200, 1, 1, 129], True, 0), ([40, 1, 200, 1, 1, 129], True, 1), ([300, 1, 70, 1], False, 0), ([1] * 300, False, 0)]


@pytest.mark.parametrize("lens,causal,window", ONE_KEY)
@pytest.mark.parametrize("d,G", [(64, 1), (64, 3), (128, 1), (128, 8)])
def test_gradients_that_are_not_finite_where_a_row_sees_one_key(lens, causal, window, d, G):
    """dS = P (dO . v - D) is NaN there as elsewhere: an infinity less itself, or a NaN."""
    rows = Rows(lens, 2 * G, 2, d, seed=d + G)
    scale = 1 / math.sqrt(d)
    o, lse = forward_for(rows, causal, scale, window)
    do = randn(rows.rng, rows.T, 2 * G, d)
    hurt = [b for b in range(len(lens)) if b % 2 == 1 or lens[b] == 200]
    alone = [int(rows.cu[b]) for b in hurt if causal or lens[b] == 1]     # rows that see their own key alone
    for i, t in enumerate(alone):
        do[t, ::G, i % d] = (float("nan"), float("inf"), -float("inf"))[i % 3]
    dq, dk, dv = backward_of(rows, o, lse, do, causal, window)
    done()
    for t in alone:
        assert dq[t, ::G].isnan().all() and dk[t].isnan().all(), t
        assert not dv[t].isfinite().all()
    check_bwd(rows, o, lse, do, (dq, dk, dv), causal, scale, window,
              which=[b for b in range(len(lens)) if not rows.cu[b] in alone])


@pytest.mark.parametrize("lens,causal,window", ONE_KEY + [([33, 0, 100, 7] * 60, True, 0)])
@pytest.mark.parametrize("d,G", [(64, 1), (64, 3), (128, 1), (128, 8)])
def test_gradients_of_attention_in_parts(lens, causal, window, d, G):
    """o and lse of rows that see more keys than this call's, as where a row's keys are divided among calls: rows that
    see one key here have a gradient too."""
    rows = Rows(lens, 2 * G, 2, d, seed=d + G, trail=3)
    scale = 1 / math.sqrt(d)
    o, lse = forward_for(rows, causal, scale, window)
    part = torch.from_numpy(rows.rng.uniform(0.2, 0.9, lse.shape)).float()         # of a row's weight, here
    o = (part[..., None] * o.float() + (1 - part[..., None]) * randn(rows.rng, *o.shape).float()).to(torch.bfloat16)
    lse = lse - part.log()
    do = randn(rows.rng, rows.T, 2 * G, d)
    got = backward_of(rows, o, lse, do, causal, window)
    done()
    check_bwd(rows, o, lse, do, got, causal, scale, window)


# ------------------------------------------------------------------ NaN
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 150)])
@pytest.mark.parametrize("d,G", [(64, 1), (64, 3), (128, 1), (128, 8)])
def test_a_key_of_nan_reaches_the_lse_of_the_rows_that_see_it(causal, window, d, G):
    rows = Rows([100, 400, 60], 2 * G, 2, d, seed=d + G)
    at = 100 + 210
    rows.k[at, 1, 3] = float("nan")               # of the second key head
    (q, k, v), cu = rows.on_gpu()
    o, lse = fa.fa_packed_fwd(q, k, v, cu, causal=causal, window=window)
    done()
    t = torch.arange(rows.T, device="cuda")
    seen = (t >= (at if causal else 100)) & (t < (min(at + window, 500) if window else 500))
    want = torch.zeros(rows.T, 2 * G, dtype=torch.bool, device="cuda")
    want[:, G:] = seen[:, None]
    assert torch.equal(lse.isnan(), want) and not lse.isinf().any()
    assert torch.equal(o.isnan().all(-1), want) and torch.equal(o.isnan().any(-1), want)


# ------------------------------------------------------------------ lengths, streams
@pytest.mark.parametrize("lens,Hq,Hkv,d,causal,window", [
    ([2600], 2, 1, 64, True, 0), ([2600], 2, 1, 128, True, 0), ([2311, 40], 1, 1, 64, False, 0), ([2311, 40], 3, 1, 128, False, 0),
    ([3001], 2, 2, 64, True, 900), ([3001], 4, 1, 128, True, 900)])
def test_gradients_of_long_sequences(lens, Hq, Hkv, d, causal, window):
    rows = Rows(lens, Hq, Hkv, d, seed=d + Hq)
    scale = 1 / math.sqrt(d)
    o, lse = forward_for(rows, causal, scale, window)
    do = randn(rows.rng, rows.T, Hq, d)
    got = backward_of(rows, o, lse, do, causal, window)
    done()
    check_bwd(rows, o, lse, do, got, causal, scale, window)


@pytest.mark.parametrize("lens", [[200, 130], [200, 3, 0, 130] * 50])
def test_a_call_on_a_stream_against_the_oracle(lens):
    rows = Rows(lens, 4, 2, 64, seed=6)
    (q, k, v), cu = rows.on_gpu()
    do = randn(rows.rng, rows.T, 4, 64)
    dog = do.cuda()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    o, lse = fa.fa_packed_fwd(q, k, v, cu, causal=True, stream=s)
    grads = fa.fa_packed_bwd(q, k, v, o, lse, dog, cu, causal=True, stream=s)
    done()
    check_fwd(rows, o, lse, True, 0.125, 0)
    check_bwd(rows, o, lse, do, grads, True, 0.125, 0)


def test_borders_that_fall_and_rise_again_write_nothing_where_there_is_a_list():
    rows = Rows([700] * 4, 2, 2, 64, seed=5)
    (q, k, v), _ = rows.on_gpu()
    cu = torch.tensor([0, 2800] * 300, dtype=torch.int32, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((2800, 2), 7.0, device="cuda")
    fa.fa_packed_fwd(q, k, v, cu, causal=True, out=out, lse=lse)
    done(fa.FA_ERR_INDEX)
    assert (out == 7).all() and (lse == 7).all()


@pytest.mark.parametrize("window", [0, 1])
@pytest.mark.parametrize("bad", [[0, 1, 2, 200], [-4, 1, 2, 110], [0, 60, 50], [109, 300, 400], [0, 110, 0, 110, 109, 110], [-1, 0, 1]])
def test_borders_out_of_range_where_rows_see_one_key(bad, window):
    """Reported, and clamped: what lies outside the rows there are is neither read nor written."""
    rows = Rows([110], 4, 2, 64, seed=4)
    (q, k, v), _ = rows.on_gpu()
    o, lse = (x.cuda() for x in forward_for(rows, True, 0.125, 0))
    cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
    outs = [torch.full((130, h, 64), 7.0, dtype=torch.bfloat16, device="cuda") for h in (4, 2, 2)]
    fa.fa_packed_bwd(q, k, v, o, lse, o, cu, causal=True, window=window, dq=outs[0][:110], dk=outs[1][:110], dv=outs[2][:110])
    done(fa.FA_ERR_INDEX)
    assert all((x[110:] == 7).all() for x in outs)
    if bad == sorted(bad):                        # the rows that the clamped borders leave
        cu = cu.clamp(0, 110)
        want = fa.fa_packed_bwd(q, k, v, o, lse, o, cu, causal=True, window=window)
        done()
        at = slice(int(cu[0]), int(cu[-1]))
        assert all(torch.equal(a[at], b[at]) for a, b in zip(outs, want))
