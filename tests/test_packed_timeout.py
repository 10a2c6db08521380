"""The bounded waits of the packed attention kernels, on the GPU, without a fault.

The test-only variant of the library (see test_timeout_path.py; never part of libfa.so) never loads the last tile of
the first item of each CTA, so the warps that wait for it give up after the variant's 20 ms, raise the CTA's abort flag,
and every role winds down. The status says FA_ERR_TIMEOUT once, and the product library's results in the same process
are right. With few rows every CTA finds its own item; with many sequences the items come from a list.
"""

import ctypes
import math
import time

import pytest

torch = pytest.importorskip("torch")
fa = pytest.importorskip("exact_io_aware_33_gb300")

from test_packed_parity import Rows, check_bwd, check_fwd, done, forward_for, randn  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def timeout_lib():
    from exact_io_aware_33_gb300 import build as b
    return fa.load_library(b.build_timeout_test_variant())


def runs_out(lib, call):
    torch.cuda.synchronize()
    assert fa.fa_get_last_device_status() == fa.FA_OK
    t0 = time.perf_counter()
    assert call() == fa.FA_OK  # launched; the failure shows in the status word
    status = lib.fa_get_last_device_status()  # synchronises the device
    elapsed = time.perf_counter() - t0
    assert status == fa.FA_ERR_TIMEOUT
    assert elapsed < 10.0, f"the wind-down took {elapsed:.2f} s"
    assert lib.fa_get_last_device_status() == fa.FA_OK  # read once, then cleared
    assert fa.fa_get_last_device_status() == fa.FA_OK   # the product library's word is its own


@pytest.mark.parametrize("lens", [[300, 150], [140, 3, 90, 200] * 50])
@pytest.mark.parametrize("d", [64, 128])
def test_waits_run_out_and_the_context_survives(timeout_lib, d, lens):
    rows = Rows(lens, 4, 2, d, seed=d + len(lens))
    scale = 1 / math.sqrt(d)
    (q, k, v), cu = rows.on_gpu()
    B, T, Hq, Hkv = len(lens), rows.T, 4, 2
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    at = lambda x: (x.data_ptr(), x.stride(0))  # noqa: E731
    o, lse = torch.empty(T, Hq, d, dtype=torch.bfloat16, device="cuda"), torch.empty(T, Hq, device="cuda")
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    sizes = (cu.data_ptr(), B, T, Hq, Hkv, d, 1, 0, scale)
    runs_out(timeout_lib, lambda: timeout_lib.fa_packed_fwd(*at(q), *at(k), *at(v), *sizes, o.data_ptr(), lse.data_ptr(),
                                                            ws.data_ptr(), ws.numel(), stream))
    o, lse = forward_for(rows, True, scale, 0)
    og, lg, do = o.cuda(), lse.cuda(), randn(rows.rng, T, Hq, d)
    dog = do.cuda()
    dq, dk, dv = torch.empty_like(og), *(torch.empty(T, Hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    runs_out(timeout_lib, lambda: timeout_lib.fa_packed_bwd(*at(q), *at(k), *at(v), og.data_ptr(), lg.data_ptr(), *at(dog),
                                                            *sizes, *at(dq), *at(dk), *at(dv), ws.data_ptr(), ws.numel(),
                                                            stream))
    got, got_lse = fa.fa_packed_fwd(q, k, v, cu, causal=True)
    grads = fa.fa_packed_bwd(q, k, v, og, lg, dog, cu, causal=True)
    done()
    check_fwd(rows, got, got_lse, True, scale, 0)
    check_bwd(rows, o, lse, do, grads, True, scale, 0)
