"""The paged 8-bit cache on the GPU: fa_paged_append and fa_paged_attn against the float64 oracle.

Tolerances, derived from the arithmetic:

* Codes and scales of the append are compared bit for bit: the rotation rounds each product and sum to
  float32 by definition, and everything after it is exact but the one rounding to e4m3. Rotated queries
  are the same float32 numbers rounded to bf16, also bit for bit.
* o: one rounding to bf16 (2^-8 of the value), P rounded to f16 (2^-11 of each weight, so at most
  2^-11 * max |v| over the row), and float32 sums: at most 2^-24 per addition over up to 4096 keys, and
  2^-22 per exponential (the hardware's), together below 2^-11 * max |v|. Bound: 2^-8 |o| + 2^-10 max |v|.
* lse: float32 products and sums of S. |S| in log2 units is below B = scale log2(e) max|q.k| bound;
  the 128-term sums err by at most 128 * 2^-24 * sum |q_c k_c| and that error enters the lse unchanged:
  with sum |q_c k_c| scale <= 64 here, 64 * 128 * 2^-24 = 4.9e-4 at the very most. Bound: 5e-4.
"""

import math

import numpy as np
import pytest

from oracle import paged

torch = pytest.importorskip("torch")
fa = pytest.importorskip("exact_io_aware_33_gb300")

pytestmark = pytest.mark.gpu


class World:
    """A pool, its oracle, and sequences with pages handed out in no order. Unused slots hold NaN codes."""

    def __init__(self, lens, H, page, d, seed, max_pages=None, fill=0x7F):
        rng = self.rng = np.random.default_rng(seed)
        self.H, self.page, self.d = H, page, d
        need = [-(-n // page) for n in lens]
        self.P = sum(need) + 2
        self.max_pages = max_pages or max(need + [1])
        perm = rng.permutation(self.P)
        self.table = np.full((len(lens), self.max_pages), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.lens = list(lens)
        shape = (self.P, H, page, d)
        codes = [np.full(shape, fill, dtype=np.uint8) for _ in range(2)]
        scales = [np.full((self.P, H), np.nan) for _ in range(2)]
        self.oracle = paged.Cache(*codes, *scales)

    def fill(self, spread=0):
        """Every token of every sequence cached: codes over the whole range, scales of many sizes."""
        rng, o = self.rng, self.oracle
        for name in ("k", "v"):
            for b, n in enumerate(self.lens):
                for i in range(-(-n // self.page)):
                    p, m = self.table[b, i], min(self.page, n - i * self.page)
                    s = 2.0 ** rng.integers(-8 - spread, -6 + spread, self.H)
                    o.scales[name][p] = s
                    o.codes[name][p, :, :m] = paged.encode(rng.standard_normal((self.H, m, self.d)) * 100)
        return self

    def to_gpu(self):
        o = self.oracle
        pages = [torch.from_numpy(o.codes[n].copy()).cuda().view(torch.float8_e4m3fn) for n in ("k", "v")]
        scales = [torch.from_numpy(o.scales[n].astype(np.float32)).cuda() for n in ("k", "v")]
        return fa.PagedCache(*pages, *scales)

    def batch(self, news, **kw):
        cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        kw.setdefault("max_q", max(list(news) + [1]))
        return cu, fa.PagedBatch(torch.from_numpy(self.table).cuda(),
                                 torch.tensor(self.lens, dtype=torch.int32, device="cuda"),
                                 torch.from_numpy(cu).cuda(), **kw)


def bf16(rng, *shape, size=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * size).astype(np.float32)).to(torch.bfloat16)


def done():
    torch.cuda.synchronize()
    assert fa.fa_get_last_device_status() == fa.FA_OK


def check_attn(w, cu, o, lse, q, scale, window=0):
    want, want_lse = w.oracle.attend(w.table, w.lens, cu, q.float().numpy(), scale, window)
    o, lse = o.float().cpu().double().numpy(), lse.cpu().double().numpy()
    G = q.shape[1] // w.H
    for b, n in enumerate(w.lens):
        size = np.nan_to_num(np.abs(w.oracle.read("v", w.table[b], n))).max(-1) if n else None  # [H, n]
        for r in range(cu[b], cu[b + 1]):
            p = n - cu[b + 1] + r
            lo = max(p - window + 1, 0) if window else 0
            top = np.repeat(size[:, lo:p + 1].max(-1), G)[:, None] if p >= lo else 0.0  # max |v| that the row sees
            assert np.array_equal(np.isnan(o[r]), np.isnan(want[r])), (b, r)
            err = np.nan_to_num(np.abs(o[r] - want[r]) - 2.0 ** -8 * np.abs(want[r]))
            assert (err <= 2.0 ** -10 * top).all(), (b, r, (err / np.maximum(top, 1e-300)).max())
            none = np.isneginf(want_lse[r])
            assert np.array_equal(none, np.isneginf(lse[r])), (b, r)
            assert (np.abs(lse[r][~none] - want_lse[r][~none]) <= 5e-4).all(), (b, r)


# ------------------------------------------------------------------ attention
DECODE = [
    # lens, Hq, Hkv, d, page
    ([1], 4, 4, 64, 16),
    ([1, 2, 15, 16, 17], 8, 2, 128, 16),
    ([64, 63, 65, 300], 6, 2, 64, 32),
    ([1000, 0, 127, 129], 8, 1, 128, 64),         # a sequence of nothing; eight rows
    ([1000, 513], 32, 2, 128, 128),               # sixteen rows
    ([700], 40, 1, 64, 16),                       # three row tiles
    ([4096, 5, 2049], 12, 12, 64, 64),
    ([2500, 1], 5, 1, 128, 32),
    ([333], 3, 3, 128, 16),
    ([0, 0], 4, 2, 64, 16),
]
STREAM = 1 << 20  # a length bound that large always divides the work among the SMs


@pytest.mark.parametrize("max_kv", [0, STREAM])
@pytest.mark.parametrize("lens,Hq,Hkv,d,page", DECODE)
def test_one_token_per_sequence(lens, Hq, Hkv, d, page, max_kv):
    w = World(lens, Hkv, page, d, seed=sum(lens) + Hq, max_pages=STREAM // page if max_kv else None).fill()
    q = bf16(w.rng, len(lens), Hq, d)
    cu = np.arange(len(lens) + 1)
    batch = fa.PagedBatch(torch.from_numpy(w.table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                          max_kv=max_kv)
    o, lse = fa.fa_paged_attn(w.to_gpu(), batch, q.cuda())
    done()
    check_attn(w, cu, o, lse, q, 1 / math.sqrt(d))


SEVERAL = [
    # lens, news, Hq, Hkv, d, page, window
    ([100, 40], [5, 1], 12, 4, 64, 16, 0),
    ([200, 200, 33], [3, 0, 8], 8, 2, 128, 32, 0),          # a sequence without rows
    ([70, 3], [70, 3], 4, 4, 128, 64, 0),                   # fresh prompts
    ([130, 257], [129, 200], 4, 2, 64, 128, 0),
    ([5, 2], [8, 4], 4, 1, 64, 16, 0),                      # more rows than tokens: the first see nothing
    ([0, 40], [4, 2], 4, 1, 64, 16, 0),                     # ... and all of a sequence's
    ([500, 90], [40, 90], 8, 2, 128, 16, 17),               # windows
    ([500, 90], [4, 1], 8, 8, 64, 64, 1),                   # ... of the own key alone
    ([1500], [2], 16, 1, 128, 64, 1000),
    ([1100, 1], [300, 1], 6, 6, 64, 32, 64),
    ([640], [256], 8, 1, 128, 64, 0),                       # 2048 rows of one key head
    ([200] * 40, [1, 2, 3, 0] * 10, 4, 2, 64, 16, 0),       # more sequences than a warp has lanes
]


@pytest.mark.parametrize("max_kv", [0, STREAM])
@pytest.mark.parametrize("lens,news,Hq,Hkv,d,page,window", SEVERAL)
def test_several_tokens_per_sequence(lens, news, Hq, Hkv, d, page, window, max_kv):
    w = World(lens, Hkv, page, d, seed=sum(lens) + sum(news) + window,
              max_pages=STREAM // page if max_kv else None).fill()
    cu, batch = w.batch(news, max_kv=max_kv)
    q = bf16(w.rng, int(cu[-1]), Hq, d)
    o, lse = fa.fa_paged_attn(w.to_gpu(), batch, q.cuda(), window=window)
    done()
    check_attn(w, cu, o, lse, q, 1 / math.sqrt(d), window)


@pytest.mark.parametrize("max_pages", [None, STREAM // 16])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 3, 2 ** 31 - 100])
@pytest.mark.parametrize("lens,news,Hq", [([5, 2], [8, 4], 4), ([5, 2], [8, 4], 1), ([500, 2], [560, 4], 4)])
def test_a_window_longer_than_every_position(lens, news, Hq, window, max_pages):
    # rows without a position, whose window would begin below the int range; rows and chunks
    w = World(lens, 1, 16, 64, seed=13, max_pages=max_pages).fill()
    cu, batch = w.batch(news)
    q = bf16(w.rng, sum(news), Hq, 64)
    o, lse = fa.fa_paged_attn(w.to_gpu(), batch, q.cuda(), window=window)
    done()
    check_attn(w, cu.tolist(), o, lse, q, 0.125, window)


@pytest.mark.parametrize("max_kv", [0, STREAM])
@pytest.mark.parametrize("news", [[1, 1], [40, 33]])
def test_scales_of_very_different_sizes(news, max_kv):
    # pages whose scales lie up to 2^24 apart: the largest values decide the output, but every row that
    # sees only small ones keeps its relative precision (the bound is relative to the row's largest value)
    for seed in range(4):
        w = World([120, 75], 2, 16, 64, seed=seed, max_pages=STREAM // 16 if max_kv else None).fill()
        big = 2.0 ** w.rng.integers(-12, 12, w.oracle.scales["v"].shape)
        w.oracle.scales["v"] *= big
        w.oracle.scales["k"] *= 2.0 ** w.rng.integers(-3, 2, big.shape)
        cu, batch = w.batch(news)
        q = bf16(w.rng, int(cu[-1]), 4, 64)
        o, lse = fa.fa_paged_attn(w.to_gpu(), batch, q.cuda())
        done()
        check_attn(w, cu, o, lse, q, 0.125)


@pytest.mark.parametrize("max_kv", [0, STREAM])
@pytest.mark.parametrize("news", [[1], [150]])
def test_values_near_the_ends_of_the_float_range(news, max_kv):
    # one page's values some 2^180 above the others': the weights' references for numerators and
    # denominators lie as far apart, and a row that does not see that page must not notice it
    for where in (0, 3, 9):
        w = World([150], 1, 16, 64, seed=where, max_pages=STREAM // 16 if max_kv else None).fill()
        w.oracle.scales["v"][:] = 2.0 ** -90
        w.oracle.scales["v"][w.table[0, where]] = 2.0 ** 90
        cu, batch = w.batch(news)
        q = bf16(w.rng, news[0], 4, 64)
        o, lse = fa.fa_paged_attn(w.to_gpu(), batch, q.cuda())
        done()
        check_attn(w, cu, o, lse, q, 0.125)


@pytest.mark.parametrize("max_pages", [3, STREAM // 32])
def test_a_scale_need_not_be_a_power_of_two(max_pages):
    w = World([90, 31], 2, 32, 128, seed=4, max_pages=max_pages).fill()
    for name in ("k", "v"):
        w.oracle.scales[name] = (w.oracle.scales[name] * w.rng.uniform(1, 2, w.oracle.scales[name].shape)
                                 ).astype(np.float32).astype(np.float64)
    cu, batch = w.batch([2, 31])
    q = bf16(w.rng, int(cu[-1]), 4, 128)
    o, lse = fa.fa_paged_attn(w.to_gpu(), batch, q.cuda())
    done()
    check_attn(w, cu, o, lse, q, 1 / math.sqrt(128))


@pytest.mark.parametrize("scale", [0.0, 1e-3, 0.3])
def test_other_softmax_scales(scale):
    w = World([90, 31], 2, 32, 64, seed=5).fill()
    cu, batch = w.batch([2, 31])
    q = bf16(w.rng, int(cu[-1]), 4, 64)
    o, lse = fa.fa_paged_attn(w.to_gpu(), batch, q.cuda(), scale=scale)
    done()
    check_attn(w, cu, o, lse, q, scale)


@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** -20, 2.0 ** 30])
def test_queries_of_any_size(size):
    # the scale takes the size back, exactly
    w = World([150], 2, 16, 64, seed=6).fill()
    cu, batch = w.batch([3])
    q = bf16(w.rng, 3, 4, 64)
    cache = w.to_gpu()
    want = fa.fa_paged_attn(cache, batch, q.cuda(), scale=0.125)
    got = fa.fa_paged_attn(cache, batch, (q.float() * size).to(torch.bfloat16).cuda(), scale=0.125 / size)
    done()
    assert torch.equal(want[0], got[0])
    assert (want[1] - got[1]).abs().max().item() <= 5e-4


@pytest.mark.parametrize("size", [2.0 ** 100, 2.0 ** 120])
@pytest.mark.parametrize("news,Hq", [([3], 4), ([3], 12), ([100], 4)])
def test_the_largest_queries_with_the_smallest_scales(news, Hq, size):
    # the scale takes the size back, exactly; the few-row kernel with 8 and 16 rows, and the chunk kernel
    w = World([150], 2, 16, 64, seed=16).fill()
    cu, batch = w.batch(news)
    q = bf16(w.rng, news[0], Hq, 64)
    cache = w.to_gpu()
    want = fa.fa_paged_attn(cache, batch, q.cuda(), scale=0.125)
    got = fa.fa_paged_attn(cache, batch, (q.float() * size).to(torch.bfloat16).cuda(), scale=0.125 / size)
    done()
    check_attn(w, cu, *want, q, 0.125)
    assert torch.equal(want[0], got[0])
    assert (want[1] - got[1]).abs().max().item() <= 5e-4


@pytest.mark.parametrize("max_pages", [13, STREAM // 16])
@pytest.mark.parametrize("news", [[1], [20], [150]])
def test_nan_codes_reach_the_rows_that_see_them_and_no_others(news, max_pages):
    n = 200
    w = World([n], 1, 16, 64, seed=7, max_pages=max_pages).fill()
    rows = news[0]
    # the last key, one that half of the rows see, and one that all rows see, next to keys that they do not
    spots = ((n - 1, 5), (n - rows // 2 - 1, 60), ((n - rows) // 16 * 16 - 1, 17))
    for j, c in spots:
        w.oracle.codes["v"][w.table[0, j // 16], 0, j % 16, c] = 0x7F if c == 5 else 0xFF
    cu, batch = w.batch(news)
    q = bf16(w.rng, rows, 4, 64)
    o, lse = fa.fa_paged_attn(w.to_gpu(), batch, q.cuda())
    done()
    assert torch.isfinite(lse).all()
    o = o.float().cpu().numpy()
    for i in range(rows):
        p = n - rows + i
        want = {c for j, c in spots if j <= p}
        got = set(np.nonzero(np.isnan(o[i]).any(0))[0])
        assert got == want, (i, got, want)


@pytest.mark.parametrize("max_pages", [None, STREAM // 16])
@pytest.mark.parametrize("window", [0, 100, 256])
@pytest.mark.parametrize("rows,Hq", [(1, 4), (20, 2), (150, 1), (300, 4)])
def test_nan_codes_anywhere_in_a_long_sequence(rows, Hq, window, max_pages):
    # at both edges of the first and the last row's windows, in between, and in a slot behind the length
    n = 700
    w = World([n], 1, 16, 64, seed=14, max_pages=max_pages).fill()
    first = n - rows
    edges = {0, 15, 16, 40, first, first + 1, n - 1, n - 17, (first + n) // 2}
    if window:
        edges |= {max(x, 0) for p in (first, n - 1) for x in (p - window, p - window + 1, p - window + 17)}
    spots = [(j, (7 * i) % 64) for i, j in enumerate(sorted(edges)) if j < n]
    for j, c in spots:
        w.oracle.codes["v"][w.table[0, j // 16], 0, j % 16, c] = 0xFF
    cu, batch = w.batch([rows])
    q = bf16(w.rng, rows, Hq, 64)
    o, lse = fa.fa_paged_attn(w.to_gpu(), batch, q.cuda(), window=window)
    done()
    assert torch.isfinite(lse).all()
    o = o.float().cpu().numpy()
    for i in range(rows):
        p = n - rows + i
        want = {c for j, c in spots if j <= p and (window == 0 or j > p - window)}
        assert {c for c in range(64) if np.isnan(o[i, :, c]).any()} == want, (i, want)
        assert all(np.isnan(o[i, :, c]).all() for c in want)


@pytest.mark.parametrize("lens,news,Hq,Hkv,d", [
    ([8189] * 8, [1] * 8, 32, 8, 128), ([4093] * 16, [3] * 16, 12, 4, 64),
    ([2045] * 4, [2045] * 4, 8, 8, 128), ([333] * 24, [333] * 24, 12, 12, 64)])
def test_what_lies_behind_a_length_costs_no_time(lens, news, Hq, Hkv, d):
    # The same work whatever the slots behind the lengths hold: the ratio is 1 but for the timer's few per
    # cent. (Rows that had to be mended for NaN codes there took 3 to 66 times as long.)
    w = World(lens, 1, 64, d, seed=15)
    shape = (w.P, Hkv, 64, d)
    k, v = (torch.randint(0, 0x70, shape, dtype=torch.uint8, device="cuda") for _ in range(2))
    scales = [torch.full(shape[:2], 2.0 ** -8, device="cuda") for _ in range(2)]
    caches = []
    for byte in (0, 0x7F):
        x = v.clone()
        for b, n in enumerate(lens):
            x[w.table[b, n // 64], :, n % 64:] = byte
        caches.append(fa.PagedCache(k.view(torch.float8_e4m3fn), x.view(torch.float8_e4m3fn), *scales))
    cu, batch = w.batch(news)
    q = bf16(w.rng, int(cu[-1]), Hq, d).cuda()
    times, outs = [[], []], [None, None]
    for _ in range(15):
        for i, cache in enumerate(caches):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            fa.fa_paged_attn(cache, batch, q)
            a.record()
            for _ in range(4):
                outs[i] = fa.fa_paged_attn(cache, batch, q)
            b.record()
            torch.cuda.synchronize()
            times[i].append(a.elapsed_time(b))
    assert fa.fa_get_last_device_status() == fa.FA_OK
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert min(times[1]) <= 1.3 * min(times[0]), (min(times[0]), min(times[1]))


@pytest.mark.parametrize("max_pages", [3, STREAM // 16])
@pytest.mark.parametrize("heads", [2, 8])
def test_a_key_with_nan_gives_nan_to_the_rows_that_see_it(heads, max_pages):
    w = World([40], 1, 16, 64, seed=8, max_pages=max_pages).fill()
    w.oracle.codes["k"][w.table[0, 36 // 16], 0, 36 % 16, 3] = 0x7F
    cu, batch = w.batch([8])
    o, lse = fa.fa_paged_attn(w.to_gpu(), batch, bf16(w.rng, 8, heads, 64).cuda())
    done()
    seen = torch.arange(32, 40) >= 36
    assert torch.isnan(o.cpu()).all(-1).all(-1).equal(seen) and torch.isnan(lse.cpu()).all(-1).equal(seen)
    assert torch.isfinite(o[:4]).all()


@pytest.mark.parametrize("max_pages", [4, STREAM // 16])
@pytest.mark.parametrize("Hq", [4, 32])
def test_rows_outside_every_sequence_stay_as_they_were(Hq, max_pages):
    w = World([50, 20], 2, 16, 64, seed=9, max_pages=max_pages).fill()
    cu, batch = w.batch([3, 2])
    T = 9
    q = bf16(w.rng, T, Hq, 64)
    out = torch.full((T, Hq, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, Hq), 7.0, device="cuda")
    fa.fa_paged_attn(w.to_gpu(), batch, q.cuda(), out=out, lse=lse)
    done()
    assert (out[5:] == 7).all() and (lse[5:] == 7).all()
    check_attn(w, cu, out[:5], lse[:5], q[:5], 0.125)


def test_strided_queries_and_the_same_bits_again():
    w = World([300, 77], 2, 32, 128, seed=10).fill()
    cu, batch = w.batch([4, 9])
    wide = bf16(w.rng, 13, 10, 128).cuda()
    q = wide[:, 3:7]
    cache = w.to_gpu()
    a = fa.fa_paged_attn(cache, batch, q)
    b = fa.fa_paged_attn(cache, batch, q.contiguous())
    done()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    check_attn(w, cu, *a, q.cpu(), 1 / math.sqrt(128))


@pytest.mark.parametrize("max_kv", [1, 100, 0])
def test_the_length_bound_only_divides_the_work(max_kv):
    w = World([900, 3], 2, 64, 64, seed=11, max_pages=40).fill()
    cu, batch = w.batch([1, 1], max_kv=max_kv)
    q = bf16(w.rng, 2, 4, 64)
    o, lse = fa.fa_paged_attn(w.to_gpu(), batch, q.cuda())
    done()
    check_attn(w, cu, o, lse, q, 0.125)


@pytest.mark.parametrize("lens,news,Hq,Hkv,d", [
    ([381, 130], [1, 1], 25, 25, 128),             # clusters of three, five, six and seven
    ([320], [1], 30, 30, 128),
    ([765], [1], 25, 25, 128),
    ([430], [1], 13, 13, 128),
    ([1500, 1490, 3, 700, 1], [1] * 5, 32, 32, 128),   # more tiles per CTA than its ring holds
    ([2000, 1100], [5, 3], 60, 30, 64),
    ([3000, 1], [2, 1], 48, 6, 128),
    ([2100] * 3, [1] * 3, 24, 24, 64)])
def test_clusters_of_any_size(lens, news, Hq, Hkv, d):
    w = World(lens, Hkv, 64, d, seed=62).fill()
    cu, batch = w.batch(news)
    q = bf16(w.rng, sum(news), Hq, d)
    o, lse = fa.fa_paged_attn(w.to_gpu(), batch, q.cuda())
    done()
    check_attn(w, cu, o, lse, q, d ** -0.5)


@pytest.mark.parametrize("lens,news,max_pages", [([300, 70], [1, 1], None), ([300, 2000], [2, 3], 5000),
                                                 ([900, 2500], [300, 200], 5000)])
def test_the_output_may_take_the_queries_place(lens, news, max_pages):
    # the cluster, streaming and chunk forms
    w = World(lens, 2, 16, 128, seed=61, max_pages=max_pages).fill()
    cu, batch = w.batch(news)
    cache = w.to_gpu()
    q = bf16(w.rng, sum(news), 16, 128).cuda()
    want, want_lse = fa.fa_paged_attn(cache, batch, q)
    o, lse = fa.fa_paged_attn(cache, batch, q, out=q)
    done()
    assert o is q and torch.equal(o, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("seed", range(24))
def test_random_batches(seed):
    rng = np.random.default_rng(1000 + seed)
    d, page, H = int(rng.choice([64, 128])), int(rng.choice([16, 32, 64, 128])), int(rng.choice([1, 2, 3, 5]))
    Hq = H * int(rng.choice([1, 2, 3, 4, 8, 16]))
    lens = rng.integers(0, int(rng.choice([20, 200, 900])), int(rng.choice([1, 2, 5, 17]))).tolist()
    most = int(rng.choice([2, 10, 150]))  # new tokens, some of which may have no position
    news = rng.integers(0, most, len(lens)).tolist()
    news[0] += 1
    w = World(lens, H, page, d, seed=seed, max_pages=int(rng.choice([60, 5000]))).fill()
    cu, batch = w.batch(news, max_kv=int(rng.choice([0, max(lens)])))
    window = int(rng.choice([0, 0, 1, 100]))
    q = bf16(w.rng, sum(news), Hq, d)
    cache = w.to_gpu()
    o, lse = fa.fa_paged_attn(cache, batch, q.cuda(), window=window)
    o2, lse2 = fa.fa_paged_attn(cache, batch, q.cuda(), window=window)
    done()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    check_attn(w, cu, o, lse, q, d ** -0.5, window)


def test_shared_pages_may_be_read_by_several_sequences():
    w = World([64, 64], 2, 16, 64, seed=12).fill()
    w.table[1, :3] = w.table[0, :3]  # a common beginning
    cu, batch = w.batch([1, 2])
    q = bf16(w.rng, 3, 4, 64)
    o, lse = fa.fa_paged_attn(w.to_gpu(), batch, q.cuda())
    done()
    check_attn(w, cu, o, lse, q, 0.125)


@pytest.mark.parametrize("rows,heads", [(1, 4), (4, 4), (64, 4)])
def test_a_long_sequence_is_cut_into_many_parts(rows, heads):
    # a few items over all SMs: up to one part per CTA of each item to join
    n = 20011
    w = World([n, 130], 1, 128, 128, seed=51 + rows).fill()
    cu, batch = w.batch([rows, 1])
    q = bf16(w.rng, int(cu[-1]), heads, 128)
    o, lse = fa.fa_paged_attn(w.to_gpu(), batch, q.cuda())
    done()
    check_attn(w, cu, o, lse, q, 1 / math.sqrt(128))


def test_a_prompt_among_single_tokens():
    lens = [300, 1, 77, 513, 40, 1000, 2]
    news = [1, 1, 1, 300, 40, 1, 2]
    w = World(lens, 2, 64, 64, seed=52, max_pages=STREAM // 64).fill()
    cu, batch = w.batch(news)
    q = bf16(w.rng, int(cu[-1]), 8, 64)
    o, lse = fa.fa_paged_attn(w.to_gpu(), batch, q.cuda())
    done()
    check_attn(w, cu, o, lse, q, 0.125)


@pytest.mark.parametrize("news_of,Hq", [(lambda b: 1, 2), (lambda b: b % 4, 2), (lambda b: b % 3, 24)])
def test_many_sequences(news_of, Hq):
    B = 700
    news = [news_of(b) for b in range(B)]
    lens = [1 + (b * 37) % 90 for b in range(B)]
    w = World(lens, 1, 16, 64, seed=53).fill()
    cu, batch = w.batch(news)
    q = bf16(w.rng, int(cu[-1]), Hq, 64)
    o, lse = fa.fa_paged_attn(w.to_gpu(), batch, q.cuda())
    done()
    check_attn(w, cu, o, lse, q, 0.125)


@pytest.mark.parametrize("rows,Hq", [(1, 2), (9, 2), (40, 8)])
def test_pages_before_the_window_may_be_gone(rows, Hq):
    n, window = 700, 100
    for max_pages in (None, STREAM // 16):
        w = World([n], 1, 16, 64, seed=54, max_pages=max_pages).fill()
        keep = w.table.copy()
        w.table[0, :(n - rows - window + 1) // 16] = -1     # handed back to the pool
        cu, batch = w.batch([rows])
        q = bf16(w.rng, rows, Hq, 64)
        o, lse = fa.fa_paged_attn(w.to_gpu(), batch, q.cuda(), window=window)
        done()
        w.table = keep
        check_attn(w, cu, o, lse, q, 0.125, window)


def test_a_chunk_captured_once_and_replayed():
    w = World([900, 350], 2, 32, 128, seed=55).fill()
    q = bf16(w.rng, 240, 8, 128)
    cache, gpu = w.to_gpu(), q.cuda()
    cu, batch = w.batch([200, 40])
    whole = list(w.lens)
    ws = torch.empty(fa.fa_paged_attn_workspace_bytes(cache, batch, 8), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fa.fa_paged_attn(cache, batch, gpu, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = fa.fa_paged_attn(cache, batch, gpu, workspace=ws)
    for lens in (whole, [640, 41], [200, 350]):
        batch.kv_lens.copy_(torch.tensor(lens))
        graph.replay()
        done()
        w.lens = lens
        check_attn(w, cu, o, lse, q, 1 / math.sqrt(128))


def test_two_streams_with_workspaces_of_their_own():
    worlds = [World([5000, 1200], 2, 64, 128, seed=56 + i).fill() for i in range(2)]
    calls = []
    for i, w in enumerate(worlds):
        news = [1, 1] if i == 0 else [100, 60]
        cu, batch = w.batch(news)
        q = bf16(w.rng, int(cu[-1]), 8, 128)
        calls.append((w, cu, batch, q, w.to_gpu(), q.cuda(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(4):
        outs = [fa.fa_paged_attn(c[4], c[2], c[5], stream=c[6]) for c in calls]
    done()
    for c, (o, lse) in zip(calls, outs):
        check_attn(c[0], c[1], o, lse, c[3], 1 / math.sqrt(128))


# ------------------------------------------------------------------ append
def angles(n, rot):
    a = np.arange(n)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def check_cache(w, cache):
    for name, pages, scales in (("k", cache.k_pages, cache.k_scales), ("v", cache.v_pages, cache.v_scales)):
        got = pages.view(torch.uint8).cpu().numpy()
        assert np.array_equal(got, w.oracle.codes[name]), (name, np.argwhere(got != w.oracle.codes[name])[:5])
        assert np.array_equal(scales.cpu().double().numpy(), w.oracle.scales[name], equal_nan=True), name


def check_queries(w, cu, got, q, cos, sin, interleaved):
    got = got.float().cpu().numpy()
    for b, n in enumerate(w.lens):
        for i in range(cu[b + 1] - cu[b]):
            p = n - (cu[b + 1] - cu[b]) + i
            if p < 0:
                continue
            x = q[cu[b] + i].float().numpy()
            x = x if cos is None else paged.rotate(x, cos[p], sin[p], interleaved)
            want = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).float().numpy()
            assert np.array_equal(got[cu[b] + i], want), (b, i)


APPEND = [
    # lens, news, Hq, Hkv, d, page, rot, interleaved
    ([1], [1], 4, 2, 64, 16, 64, False),
    ([1, 17, 16, 33], [1, 1, 1, 1], 8, 2, 128, 16, 128, False),
    ([5, 300], [1, 1], 6, 3, 64, 128, 32, True),
    ([40, 16], [40, 16], 8, 2, 128, 16, 128, True),
    ([100, 31, 64], [7, 31, 0], 12, 12, 64, 32, 64, False),       # odd beginnings; a sequence without rows
    ([500], [300], 32, 8, 128, 64, 64, False),
    ([300, 129], [299, 2], 4, 5, 128, 128, 16, True),             # an odd number of key heads
    ([70], [70], 0, 1, 64, 64, 0, False),                         # no queries, no rotation
    ([2, 0], [5, 3], 4, 2, 64, 16, 64, False),                    # rows without a position
    ([0, 3], [1, 1], 4, 2, 128, 32, 128, False),                  # a padded decode batch
]


@pytest.mark.parametrize("lens,news,Hq,Hkv,d,page,rot,interleaved", APPEND)
def test_append_matches_bit_for_bit(lens, news, Hq, Hkv, d, page, rot, interleaved):
    w = World(lens, Hkv, page, d, seed=sum(lens) + d + page)
    # what the sequences held before
    old = [max(n - m, 0) for n, m in zip(lens, news)]
    kv = [w.rng.standard_normal((sum(old), Hkv, d)) for _ in range(2)]
    w.oracle.append(w.table, old, np.concatenate([[0], np.cumsum(old)]), *kv)
    cache = w.to_gpu()
    cu, batch = w.batch(news)
    if all(m == 1 for m in news):
        batch = fa.PagedBatch(batch.block_table, batch.kv_lens)
    T = int(cu[-1])
    # slices of a fused projection; some tokens much larger than what their pages hold
    wide = bf16(w.rng, T, Hq + 2 * Hkv, d) * torch.from_numpy(4.0 ** w.rng.integers(-1, 3, (T, 1, 1))).to(torch.bfloat16)
    q, k, v = wide[:, :Hq], wide[:, Hq:Hq + Hkv], wide[:, Hq + Hkv:]
    gpu = wide.cuda()
    cos, sin = angles(max(lens) + 1, rot) if rot else (None, None)
    rope = tuple(torch.from_numpy(x).cuda() for x in (cos, sin)) if rot else None
    got = fa.fa_paged_append(cache, batch, gpu[:, Hq:Hq + Hkv], gpu[:, Hq + Hkv:], q=gpu[:, :Hq] if Hq else None,
                             rope=rope, interleaved=interleaved)
    done()
    w.oracle.append(w.table, lens, cu, k.float().numpy(), v.float().numpy(), cos, sin, interleaved)
    check_cache(w, cache)
    if Hq:
        check_queries(w, cu, got, q, cos, sin, interleaved)
    # the same call again changes nothing: the tokens are where they were
    fa.fa_paged_append(cache, batch, gpu[:, Hq:Hq + Hkv], gpu[:, Hq + Hkv:], rope=rope, interleaved=interleaved)
    done()
    if all(n >= m for n, m in zip(lens, news)):
        check_cache(w, cache)


def test_a_ragged_batch_whose_blocks_look_for_their_sequences():
    # one long sequence among many short ones: most of a rectangular grid would be empty
    news = [1] * 20 + [700] + [2] * 20 + [0, 0, 3]
    lens = [n + 5 for n in news]
    w = World(lens, 2, 16, 64, seed=21)
    old = [5] * len(lens)
    kv = [w.rng.standard_normal((sum(old), 2, 64)) for _ in range(2)]
    w.oracle.append(w.table, old, np.arange(len(lens) + 1) * 5, *kv)
    cache = w.to_gpu()
    cu, batch = w.batch(news)
    k, v = (bf16(w.rng, int(cu[-1]) + 4, 2, 64) for _ in range(2))  # and rows behind the last sequence
    fa.fa_paged_append(cache, batch, k.cuda(), v.cuda())
    done()
    w.oracle.append(w.table, lens, cu, k.float().numpy(), v.float().numpy())
    check_cache(w, cache)


def test_append_token_by_token_as_scales_grow():
    w = World([40], 2, 16, 128, seed=22)
    cache = w.to_gpu()
    table = torch.from_numpy(w.table).cuda()
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    batch = fa.PagedBatch(table, lens)
    for n in range(1, 41):
        lens.fill_(n)
        k, v = (bf16(w.rng, 1, 2, 128, size=1.3 ** (n % 23)) for _ in range(2))
        fa.fa_paged_append(cache, batch, k.cuda(), v.cuda())
        w.oracle.append(w.table, [n], [0, 1], k.float().numpy(), v.float().numpy())
    done()
    check_cache(w, cache)


def test_values_that_are_not_finite():
    w = World([16], 1, 16, 64, seed=23)
    cache = w.to_gpu()
    cu, batch = w.batch([16])
    k, v = bf16(w.rng, 16, 1, 64), bf16(w.rng, 16, 1, 64)
    v[3, 0, 5], v[4, 0, 6], k[5, 0, 7], v[6, 0, 0] = math.inf, -math.inf, math.nan, math.nan
    fa.fa_paged_append(cache, batch, k.cuda(), v.cuda())
    done()
    w.oracle.append(w.table, [16], cu, k.float().numpy(), v.float().numpy())
    for name, pages in (("k", cache.k_pages), ("v", cache.v_pages)):
        got = pages.float().cpu().numpy()
        assert np.array_equal(got, paged.E4M3[w.oracle.codes[name]].astype(np.float32), equal_nan=True)
    assert torch.isfinite(cache.k_scales[w.table[0, 0]]).all()


@pytest.mark.parametrize("size", [1e-38, 2.0 ** -126, 1e30, 3e38])
def test_values_of_any_size(size):
    w = World([20], 1, 16, 64, seed=24)
    cache = w.to_gpu()
    cu, batch = w.batch([20])
    k, v = (bf16(w.rng, 20, 1, 64).clamp(-1, 1) * size for _ in range(2))
    fa.fa_paged_append(cache, batch, k.cuda(), v.cuda())
    done()
    w.oracle.append(w.table, [20], cu, k.float().numpy(), v.float().numpy())
    check_cache(w, cache)


def test_queries_may_be_rotated_in_place():
    w = World([30], 2, 16, 64, seed=25)
    cu, batch = w.batch([30])
    cos, sin = angles(30, 64)
    rope = (torch.from_numpy(cos).cuda(), torch.from_numpy(sin).cuda())
    wide = bf16(w.rng, 30, 8, 64)
    gpu = wide.cuda()
    cache = w.to_gpu()
    got = fa.fa_paged_append(cache, batch, gpu[:, 4:6], gpu[:, 6:], q=gpu[:, :4], rope=rope, q_out=gpu[:, :4])
    done()
    assert got.data_ptr() == gpu.data_ptr()
    check_queries(w, cu, got, wide[:, :4], cos, sin, False)
    assert torch.equal(gpu[:, 4:].cpu(), wide[:, 4:])


# ------------------------------------------------------------------ together
def test_a_conversation():
    # a prompt, then chunks and single tokens: each step appended and attended as a model's layer does
    Hq, H, d, page = 8, 2, 64, 16
    steps = [([37, 5], [37, 5]), ([38, 6], [1, 1]), ([39, 30], [1, 24]), ([45, 31], [6, 1]), ([46, 32], [1, 1])]
    w = World(steps[-1][0], H, page, d, seed=31)
    cache = w.to_gpu()
    cos, sin = angles(64, d)
    rope = (torch.from_numpy(cos).cuda(), torch.from_numpy(sin).cuda())
    for lens, news in steps:
        w.lens = lens
        cu, batch = w.batch(news)
        T = int(cu[-1])
        q, k, v = bf16(w.rng, T, Hq, d), bf16(w.rng, T, H, d), bf16(w.rng, T, H, d)
        qr = fa.fa_paged_append(cache, batch, k.cuda(), v.cuda(), q=q.cuda(), rope=rope)
        o, lse = fa.fa_paged_attn(cache, batch, qr)
        done()
        w.oracle.append(w.table, lens, cu, k.float().numpy(), v.float().numpy(), cos, sin)
        check_cache(w, cache)
        check_attn(w, cu, o, lse, qr.cpu(), 0.125)


def test_a_decode_step_captured_once_and_replayed():
    Hq, H, d, page, B = 8, 2, 128, 16, 3
    w = World([90, 47, 33], H, page, d, seed=32)
    start = [40, 15, 0]
    kv = [w.rng.standard_normal((sum(start), H, d)) for _ in range(2)]
    w.oracle.append(w.table, start, [0, 40, 55, 55], *kv)
    cache = w.to_gpu()
    cos, sin = angles(128, d)
    rope = (torch.from_numpy(cos).cuda(), torch.from_numpy(sin).cuda())
    lens = torch.tensor(start, dtype=torch.int32, device="cuda")
    batch = fa.PagedBatch(torch.from_numpy(w.table).cuda(), lens)
    q, k, v = (torch.zeros(B, h, d, dtype=torch.bfloat16, device="cuda") for h in (Hq, H, H))
    ws = torch.empty(fa.fa_paged_attn_workspace_bytes(cache, batch, Hq), dtype=torch.uint8, device="cuda")

    def step():
        lens.add_(1)
        return fa.fa_paged_attn(cache, batch, fa.fa_paged_append(cache, batch, k, v, q=q, rope=rope), workspace=ws)

    codes = cache.k_pages.view(torch.uint8).clone(), cache.v_pages.view(torch.uint8).clone()
    scales = cache.k_scales.clone(), cache.v_scales.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = step()
    # back to the beginning
    lens.copy_(torch.tensor(start))
    cache.k_pages.view(torch.uint8).copy_(codes[0])
    cache.v_pages.view(torch.uint8).copy_(codes[1])
    cache.k_scales.copy_(scales[0])
    cache.v_scales.copy_(scales[1])
    for i in range(1, 31):
        new = [bf16(w.rng, B, h, d) for h in (Hq, H, H)]
        for dst, src in zip((q, k, v), new):
            dst.copy_(src)
        graph.replay()
        now = [n + i for n in start]
        w.oracle.append(w.table, now, [0, 1, 2, 3], new[1].float().numpy(), new[2].float().numpy(), cos, sin)
    done()
    w.lens = now
    check_cache(w, cache)
    turned = torch.stack([torch.from_numpy(paged.rotate(new[0][b].float().numpy(), cos[n - 1], sin[n - 1], False))
                          for b, n in enumerate(now)]).to(torch.bfloat16)
    check_attn(w, [0, 1, 2, 3], o, lse, turned, 1 / math.sqrt(d))


def test_another_stream():
    w = World([3000, 1700], 4, 64, 128, seed=33).fill()
    cu, batch = w.batch([1, 1])
    q = bf16(w.rng, 2, 16, 128)
    cache, gpu = w.to_gpu(), q.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, lse = fa.fa_paged_attn(cache, batch, gpu, stream=side)
    side.synchronize()
    done()
    check_attn(w, cu, o, lse, q, 1 / math.sqrt(128))


def test_more_than_two_to_the_31_bytes_of_pages():
    # page ids whose byte offsets need more than 32 bits, in reading and in writing
    P, H, page, d = 140_000, 2, 128, 64
    cache = fa.PagedCache.empty(P, H, page, d)
    ids = [P - 1, 131_073, 3]
    w = World([300], H, page, d, seed=34).fill()
    lens = torch.tensor([300], dtype=torch.int32, device="cuda")
    table = torch.tensor([ids], dtype=torch.int32, device="cuda")
    for name, pages, scales in (("k", cache.k_pages, cache.k_scales), ("v", cache.v_pages, cache.v_scales)):
        for i, p in enumerate(ids):
            pages.view(torch.uint8)[p] = torch.from_numpy(w.oracle.codes[name][w.table[0, i]]).cuda()
            scales[p] = torch.from_numpy(w.oracle.scales[name][w.table[0, i]].astype(np.float32)).cuda()
    batch = fa.PagedBatch(table, lens)
    q, k, v = bf16(w.rng, 1, 4, d), bf16(w.rng, 1, H, d), bf16(w.rng, 1, H, d)
    fa.fa_paged_append(cache, batch, k.cuda(), v.cuda())
    o, lse = fa.fa_paged_attn(cache, batch, q.cuda())
    done()
    w.oracle.append(w.table, [300], [0, 1], k.float().numpy(), v.float().numpy())
    check_attn(w, [0, 1], o, lse, q, 0.125)


# ------------------------------------------------------------------ what the device finds out of range
def test_indices_out_of_range_are_reported_and_touch_nothing():
    w = World([40, 40], 2, 16, 64, seed=41).fill()
    q = bf16(w.rng, 2, 4, 64).cuda()
    k, v = bf16(w.rng, 2, 2, 64).cuda(), bf16(w.rng, 2, 2, 64).cuda()
    for bad in (-1, w.P, 2 ** 31 - 1, -2 ** 31):
        cache = w.to_gpu()
        table = torch.from_numpy(w.table).cuda()
        table[1, 2] = bad           # the page that the new token goes to, and the last one read
        batch = fa.PagedBatch(table, torch.tensor([40, 40], dtype=torch.int32, device="cuda"))
        o, lse = fa.fa_paged_attn(cache, batch, q)
        torch.cuda.synchronize()
        assert fa.fa_get_last_device_status() == fa.FA_ERR_INDEX
        assert fa.fa_get_last_device_status() == fa.FA_OK    # reading clears it
        whole = World.__new__(World)
        whole.__dict__.update(w.__dict__, lens=w.lens[:1])
        check_attn(whole, [0, 1], o[:1], lse[:1], q[:1].cpu(), 0.125)   # the other sequence is untouched
        before = cache.k_pages.view(torch.uint8).clone()
        fa.fa_paged_append(cache, batch, k, v)
        torch.cuda.synchronize()
        assert fa.fa_get_last_device_status() == fa.FA_ERR_INDEX
        changed = (cache.k_pages.view(torch.uint8) != before).flatten(1).any(1).nonzero().flatten().tolist()
        assert changed == [int(w.table[0, 2])]
    # a chunk: 20 rows of each sequence, the second sequence's last page bad
    long_table = torch.full((2, STREAM // 16), -1, dtype=torch.int32)
    long_table[:, :3] = torch.from_numpy(w.table)
    long_table[1, 2] = w.P
    batch = fa.PagedBatch(long_table.cuda(), torch.tensor([40, 40], dtype=torch.int32, device="cuda"),
                          torch.tensor([0, 20, 40], dtype=torch.int32, device="cuda"), max_q=20)
    many = bf16(w.rng, 40, 4, 64)
    o, lse = fa.fa_paged_attn(w.to_gpu(), batch, many.cuda())
    torch.cuda.synchronize()
    assert fa.fa_get_last_device_status() == fa.FA_ERR_INDEX
    check_attn(whole, [0, 20], o[:20], lse[:20], many[:20], 0.125)
    # absent keys take no part: the rows of sequence 1 see its first 32 keys, up to their own position
    part = World.__new__(World)
    part.__dict__.update(w.__dict__, lens=[32], table=w.table[1:])
    check_attn(part, [0, 12], o[20:32], lse[20:32], many[20:32], 0.125)
    check_attn(part, [0, 1], o[39:], lse[39:], many[39:], 0.125)
    for lens in ([40, -5], [40, 10 ** 6]):
        batch = fa.PagedBatch(torch.from_numpy(w.table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"))
        fa.fa_paged_attn(w.to_gpu(), batch, q)
        torch.cuda.synchronize()
        assert fa.fa_get_last_device_status() == fa.FA_ERR_INDEX
    for cu in ([0, 5, 2], [-3, 1, 2], [0, 1, 100]):
        batch = fa.PagedBatch(torch.from_numpy(w.table).cuda(), torch.tensor([40, 40], dtype=torch.int32, device="cuda"),
                              torch.tensor(cu, dtype=torch.int32, device="cuda"), max_q=2)
        fa.fa_paged_attn(w.to_gpu(), batch, q)
        fa.fa_paged_append(w.to_gpu(), batch, k, v)
        torch.cuda.synchronize()
        assert fa.fa_get_last_device_status() == fa.FA_ERR_INDEX
    cos, sin = (torch.from_numpy(x).cuda() for x in angles(39, 64))   # position 39 has no angles
    batch = fa.PagedBatch(torch.from_numpy(w.table).cuda(), torch.tensor([40, 30], dtype=torch.int32, device="cuda"))
    fa.fa_paged_append(w.to_gpu(), batch, k, v, rope=(cos, sin))
    torch.cuda.synchronize()
    assert fa.fa_get_last_device_status() == fa.FA_ERR_INDEX


def test_arguments_that_the_binding_refuses():
    w = World([20, 20], 2, 16, 64, seed=42, max_pages=100000).fill()   # a long table: a workspace is needed
    cache = w.to_gpu()
    cu, batch = w.batch([2, 1])
    q = bf16(w.rng, 3, 4, 64).cuda()
    k = bf16(w.rng, 3, 2, 64).cuda()
    for bad in (q.float(), q.half()):
        with pytest.raises(TypeError):
            fa.fa_paged_attn(cache, batch, bad)
    for bad in (q[:, :, :32], q.transpose(0, 1), q.expand(3, 4, 64).transpose(1, 2)):
        with pytest.raises((ValueError, fa.FAError)):
            fa.fa_paged_attn(cache, batch, bad)
    with pytest.raises(fa.FAError):
        fa.fa_paged_attn(cache, batch, q[:, :3])          # 3 heads over 2
    with pytest.raises(fa.FAError):
        fa.fa_paged_attn(cache, batch, q, window=-1)
    with pytest.raises(fa.FAError):
        fa.fa_paged_attn(cache, batch, q, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        fa.fa_paged_append(cache, batch, k, k[:2])
    with pytest.raises(ValueError):
        fa.fa_paged_append(cache, batch, k[:, :1], k[:, :1])
    with pytest.raises(ValueError):
        fa.fa_paged_append(cache, batch, k, k, q=q[:2])
    with pytest.raises(ValueError):
        fa.PagedBatch(batch.block_table, batch.kv_lens[:1])
    with pytest.raises(ValueError):
        fa.PagedBatch(batch.block_table, batch.kv_lens, max_q=2)
    with pytest.raises(ValueError):
        fa.PagedBatch(batch.block_table, batch.kv_lens, batch.cu_q, max_q=2 ** 32 + 1)
    with pytest.raises(ValueError):
        fa.fa_paged_append(cache, batch, k, k, q_out=q)
    with pytest.raises(fa.FAError):
        fa.fa_paged_attn(cache, batch, q[:2], out=q[1:])      # outputs over another row's queries
    with pytest.raises(fa.FAError):
        fa.fa_paged_append(cache, batch, k, k.clone(), q=k.clone(), q_out=k)  # rotated queries over the keys
    with pytest.raises(TypeError):
        fa.PagedBatch(batch.block_table.long(), batch.kv_lens)
    with pytest.raises(ValueError):
        fa.fa_paged_attn(cache, fa.PagedBatch(batch.block_table, batch.kv_lens), q)   # 3 rows for 2 sequences
    done()
