"""Host checks of the packed calls that tests/test_oracle_packed.py does not make (no device touched)."""

import os
import subprocess
import sys

import pytest

import exact_io_aware_33_gb300 as fa
from test_oracle_packed import _bwd, _far, _fwd, _rope, lib  # noqa: F401


@pytest.mark.parametrize("kw", [
    dict(lse=_far(5)), dict(lse=_far(5) + 4096), dict(lse=_far(6) - 16), dict(lse=_far(7) + 8 * 512 - 4),
    dict(cu=_far(5) + 512), dict(cu=_far(6) - 4), dict(cu=_far(7) + 8 * 512 - 4),
    # in a row, or across the end of the gap between two
    dict(dqs=1024, lse=_far(5) + 2048 + 1024 - 4), dict(dqs=1024, lse=_far(5) + 2048 - 64),
    dict(dks=1024, cu=_far(6) + 2048 + 512 - 4), dict(dvs=1024, cu=_far(7) + 2048 - 8)])
def test_gradients_that_meet_the_statistics_or_the_borders_are_refused(lib, kw):  # noqa: F811
    assert _bwd(lib, **kw) == fa.FA_ERR_INVALID


@pytest.mark.parametrize("kw", [
    dict(lse=_far(5) - 128), dict(lse=_far(5) + 8 * 1024), dict(cu=_far(6) - 16), dict(cu=_far(6) + 8 * 512),
    # between two rows (128 bytes of lse, 16 of cu), or behind the last one's
    dict(dqs=1024, lse=_far(5) + 1024), dict(dqs=1024, lse=_far(5) + 2048 - 128), dict(dks=1024, cu=_far(6) + 2048 - 16),
    dict(dvs=1024, cu=_far(7) + 7 * 2048 + 512)])
def test_gradients_beside_the_statistics_or_the_borders_are_not(lib, kw):  # noqa: F811
    # the code that a call which passes its checks gives where there is no device to launch on
    if fa.fa_get_last_device_status() != fa.FA_ERR_LAUNCH:
        pytest.skip("would launch on pointers that are none")
    assert _bwd(lib, **kw) == fa.FA_ERR_LAUNCH


@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_scales_whose_product_with_log2_e_is_no_number_are_refused(lib, call):  # noqa: F811
    # scores are scaled in units of log2: 3.4e38 / 1.4427 is the largest scale
    for scale in (2.4e38, 3.4e38):
        assert call(lib, scale=scale) == fa.FA_ERR_INVALID


# What a call that passes its checks gives where there is no device to launch on.
@pytest.mark.parametrize("call,kw", [
    (_fwd, dict()), (_fwd, dict(scale=2.3e38)), (_fwd, dict(scale=0.0)), (_fwd, dict(d=64, qs=256, ks=128, vs=128)),
    (_bwd, dict()), (_bwd, dict(scale=2.3e38)), (_bwd, dict(scale=0.0)),
    (_bwd, dict(d=64, qs=256, ks=128, vs=128, dos=256, dqs=256, dks=128, dvs=128)),
    (_rope, dict()), (_rope, dict(rot=64, d=64, qs=256, qos=256, ks=128, kos=128)), (_rope, dict(rot=64, d=256, qs=1024,
                                                                                    qos=1024, ks=512, kos=512))])
def test_calls_as_they_are_meant_pass_their_checks(lib, call, kw):  # noqa: F811
    if fa.fa_get_last_device_status() != fa.FA_ERR_LAUNCH:
        pytest.skip("would launch on pointers that are none")
    assert call(lib, **kw) == fa.FA_ERR_LAUNCH


def test_packed_calls_say_what_is_missing_where_there_is_no_binding():
    code = """
import sys
import torch
import exact_io_aware_33_gb300 as fa
sys.modules["exact_io_aware_33_gb300._paged_native"] = None    # an import that fails
q, cu = torch.zeros(1, 1, 64, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
for call in (lambda: fa.fa_packed_fwd(q, q, q, cu), lambda: fa.fa_packed_bwd_workspace_bytes(1, 1, 1, 1, 64),
             lambda: fa.fa_rope_axes(q, q, cu[None, :1], (q, q), sections=(32,)), lambda: fa.PagedCache.empty(1, 1, 16, 64)):
    try:
        call()
    except ImportError as e:
        assert "packed sequences" in str(e) and "paged cache" in str(e) and "build()" in str(e), e
    else:
        raise AssertionError("no ImportError")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
