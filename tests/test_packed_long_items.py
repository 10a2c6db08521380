"""Packed sequences so long that one item of work takes longer than a wait may, on the GPU.

A build of the library whose waits give up after 5 ms instead of a second (never part of libfa.so) stands for sequences
two hundred times as long. A role that has nothing to do until an item ends, the gradients' write-back or the softmax of
a tile that holds no rows, has to wait as long as the others get on with it; every other wait spans a few steps of a
microsecond. Where one gave up, the status would say FA_ERR_TIMEOUT, and outputs would be missing.
"""

import ctypes
import os

import pytest

torch = pytest.importorskip("torch")
fa = pytest.importorskip("exact_io_aware_33_gb300")

from test_packed_parity import done  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def impatient():
    from exact_io_aware_33_gb300 import build as b
    where = os.path.join(b.BUILD, "short_wait_test")
    return fa.load_library(b.build(extra_flags=["-DFA_WAIT_BUDGET_NS=5000000ull"], out_dir=where,
                                   lib_path=os.path.join(where, "libfa_short_wait_test.so")))


def inputs(n, Hq, Hkv, d):
    gen = torch.Generator(device="cuda").manual_seed(n)
    return [torch.empty(n, h, d, dtype=torch.bfloat16, device="cuda").normal_(generator=gen) for h in (Hq, Hkv, Hkv, Hq)]


def at(x):
    return x.data_ptr(), x.stride(0)


def test_a_tile_without_rows_waits_for_the_next_item(impatient):
    n, d = (1 << 21) + 64, 128                    # the last two tiles of 128 tokens: 64 rows in one, none in the other
    q, k, v, _ = inputs(n, 1, 1, d)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    want, want_lse = fa.fa_packed_fwd(q, k, v, cu, causal=True)
    done()
    o, lse = torch.zeros_like(want), torch.zeros_like(want_lse)
    ws = torch.empty(fa.fa_packed_fwd_workspace_bytes(1, n, 1, 1, d), dtype=torch.uint8, device="cuda")
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert impatient.fa_packed_fwd(*at(q), *at(k), *at(v), cu.data_ptr(), 1, n, 1, 1, d, 1, 0, d ** -0.5, o.data_ptr(),
                                   lse.data_ptr(), ws.data_ptr(), ws.numel(), stream) == fa.FA_OK
    assert impatient.fa_get_last_device_status() == fa.FA_OK
    assert torch.equal(o, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("d", [64, 128])
def test_the_write_back_waits_for_a_long_item(impatient, d):
    n, Hq = 20000, 128                            # a token of 128 heads makes a step: 20000 steps for the first keys
    q, k, v, do = inputs(n, Hq, 1, d)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    o, lse = fa.fa_packed_fwd(q, k, v, cu, causal=True)
    want = fa.fa_packed_bwd(q, k, v, o, lse, do, cu, causal=True)
    done()
    got = [torch.zeros_like(x) for x in want]
    ws = torch.empty(fa.fa_packed_bwd_workspace_bytes(1, n, Hq, 1, d), dtype=torch.uint8, device="cuda")
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert impatient.fa_packed_bwd(*at(q), *at(k), *at(v), o.data_ptr(), lse.data_ptr(), *at(do), cu.data_ptr(), 1, n, Hq, 1,
                                   d, 1, 0, d ** -0.5, *at(got[0]), *at(got[1]), *at(got[2]), ws.data_ptr(), ws.numel(),
                                   stream) == fa.FA_OK
    assert impatient.fa_get_last_device_status() == fa.FA_OK
    assert all(torch.equal(a, b) for a, b in zip(got, want))
