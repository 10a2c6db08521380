"""Packed sequences on the GPU where calls are legal and rare: hand-offs under load, values, scales and lengths at the
ends of their ranges. Against the float64 oracle, with the bounds of test_packed_parity.py, or for equal bits."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
fa = pytest.importorskip("exact_io_aware_33_gb300")

from test_packed_parity import Rows, done, randn  # noqa: E402

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
