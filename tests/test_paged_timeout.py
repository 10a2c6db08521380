"""The bounded waits of the paged attention kernels, on the GPU, without a fault.

The test-only variant of the library (see test_timeout_path.py; never part of libfa.so) never loads the
last tile of a sequence, so the warps that wait for it give up after the variant's 20 ms, raise the
CTA's abort flag, and every role winds down. Each form is run once: clusters, streaming, chunks. The
status says FA_ERR_TIMEOUT once, and the product library's results in the same process are right.
"""

import ctypes
import time

import pytest

torch = pytest.importorskip("torch")
fa = pytest.importorskip("exact_io_aware_33_gb300")

from test_paged_parity import STREAM, World, bf16, check_attn, done  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def timeout_lib():
    from exact_io_aware_33_gb300 import build as b
    return fa.load_library(b.build_timeout_test_variant())


@pytest.mark.parametrize("rows,heads,max_kv", [(1, 4, 0), (1, 4, STREAM), (9, 2, STREAM), (300, 4, STREAM)])
@pytest.mark.parametrize("d", [64, 128])
def test_wait_runs_out_and_the_context_survives(timeout_lib, d, rows, heads, max_kv):
    w = World([500], 2, 64, d, seed=d + rows, max_pages=STREAM // 64 if max_kv else None).fill()
    cu, batch = w.batch([rows])
    q = bf16(w.rng, rows, heads, d)
    cache, gpu = w.to_gpu(), q.cuda()
    o = torch.empty_like(gpu)
    lse = torch.empty(rows, heads, device="cuda")
    c_batch = type(batch._struct).from_buffer_copy(batch._struct)
    c_batch.T = rows
    struct = ctypes.addressof(c_batch)
    need = timeout_lib.fa_paged_attn_workspace_bytes(cache._address, struct, heads)
    ws = torch.zeros(max(need, 1), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert fa.fa_get_last_device_status() == fa.FA_OK

    t0 = time.perf_counter()
    rc = timeout_lib.fa_paged_attn(cache._address, struct, gpu.data_ptr(), heads * d, o.data_ptr(), lse.data_ptr(),
                                   heads, 0, d ** -0.5, ws.data_ptr(), need,
                                   ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == fa.FA_OK  # launched; the failure shows in the status word
    status = timeout_lib.fa_get_last_device_status()  # synchronises the device
    elapsed = time.perf_counter() - t0
    assert status == fa.FA_ERR_TIMEOUT
    assert elapsed < 10.0, f"the wind-down took {elapsed:.2f} s"
    assert timeout_lib.fa_get_last_device_status() == fa.FA_OK  # read once, then cleared
    assert fa.fa_get_last_device_status() == fa.FA_OK           # the product library's word is its own

    o, lse = fa.fa_paged_attn(cache, batch, gpu)
    done()
    check_attn(w, cu, o, lse, q, d ** -0.5)


def run_out(timeout_lib, w, cu, batch, q):
    """One call of the variant on a World: launched, then FA_ERR_TIMEOUT within a few seconds."""
    rows, heads, d = q.shape
    cache, gpu = w.to_gpu(), q.cuda()
    o, lse = torch.empty_like(gpu), torch.empty(rows, heads, device="cuda")
    c_batch = type(batch._struct).from_buffer_copy(batch._struct)
    c_batch.T = rows
    struct = ctypes.addressof(c_batch)
    need = timeout_lib.fa_paged_attn_workspace_bytes(cache._address, struct, heads)
    ws = torch.zeros(max(need, 1), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    assert timeout_lib.fa_paged_attn(cache._address, struct, gpu.data_ptr(), heads * d, o.data_ptr(), lse.data_ptr(),
                                     heads, 0, d ** -0.5, ws.data_ptr(), need,
                                     ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == fa.FA_OK
    status = timeout_lib.fa_get_last_device_status()
    assert time.perf_counter() - t0 < 10.0
    return status


# Many sequences, each longer than a CTA's ring: the loading warp is in the middle of its work, waiting
# for a free stage, when the flag goes up, and has to leave it with all its lanes at once.
@pytest.mark.parametrize("lens,news,heads,max_kv", [
    ([2100, 1900, 2000, 1700] * 12, [1] * 48, 4, STREAM),
    ([2100, 3, 1900, 0, 2000] * 8, [3, 1, 4, 0, 2] * 8, 8, STREAM),
    ([2100, 3, 1900, 0, 2000] * 4, [1] * 20, 4, 0)])
@pytest.mark.parametrize("d", [64, 128])
def test_a_long_batch_winds_down(timeout_lib, d, lens, news, heads, max_kv):
    w = World(lens, 2, 64, d, seed=d + len(lens), max_pages=STREAM // 64 if max_kv else None).fill()
    cu, batch = w.batch(news)
    q = bf16(w.rng, sum(news), heads, d)
    assert run_out(timeout_lib, w, cu, batch, q) == fa.FA_ERR_TIMEOUT
    assert timeout_lib.fa_get_last_device_status() == fa.FA_OK
    o, lse = fa.fa_paged_attn(w.to_gpu(), batch, q.cuda())
    done()
    check_attn(w, cu, o, lse, q, d ** -0.5)


@pytest.mark.parametrize("rows", [1, 300])
def test_a_bad_index_does_not_hide_a_timeout(timeout_lib, rows):
    w = World([500], 2, 64, 64, seed=rows, max_pages=STREAM // 64).fill()
    cu, batch = w.batch([rows])
    cache, q = w.to_gpu(), bf16(w.rng, rows, 4, 64).cuda()
    kv = torch.zeros(rows, 2, 64, dtype=torch.bfloat16, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(rows, 4, device="cuda")
    batch.block_table[0, 2] = w.P    # the append finds this page out of range, and so does the attention
    c_batch = type(batch._struct).from_buffer_copy(batch._struct)
    c_batch.T = rows
    struct, stream = ctypes.addressof(c_batch), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    ws = torch.zeros(timeout_lib.fa_paged_attn_workspace_bytes(cache._address, struct, 4), dtype=torch.uint8, device="cuda")

    def append():
        assert timeout_lib.fa_paged_append(cache._address, struct, kv.data_ptr(), 128, kv.data_ptr(), 128, 0, 0, 0, 0, 0,
                                           0, 0, 0, 0, 0, stream) == fa.FA_OK

    def attend():
        assert timeout_lib.fa_paged_attn(cache._address, struct, q.data_ptr(), 256, o.data_ptr(), lse.data_ptr(), 4, 0,
                                         0.125, ws.data_ptr(), ws.numel(), stream) == fa.FA_OK

    batch.kv_lens.fill_(2 * 64 + rows)    # the new tokens begin on that page
    append()
    assert timeout_lib.fa_get_last_device_status() == fa.FA_ERR_INDEX
    for calls in ((attend, append), (append, attend)):
        for call in calls:
            call()
        assert timeout_lib.fa_get_last_device_status() == fa.FA_ERR_TIMEOUT
        assert timeout_lib.fa_get_last_device_status() == fa.FA_OK
