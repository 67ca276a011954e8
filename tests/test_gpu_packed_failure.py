"""Failure detection of the ragged prefill without a fault: its copies are left out, so every wait runs out within its
bound, the launch ends by itself with device error 1, and the next call on the same context is right."""
import pytest
import torch

from tests import ragged_reference as R
from tests.test_gpu_ragged import SCALE, _cu, _prefill, _prefill_inputs

pytestmark = pytest.mark.gpu

WAIT_TIMEOUT = 1


@pytest.fixture(scope="module")
def L():
    from mla_latent_kv_fp8_gb300 import build
    build.build()
    from mla_latent_kv_fp8_gb300 import _lib
    _lib.lib()
    assert _lib.mla_device_error() == 0
    return _lib


@pytest.mark.parametrize("lq,lk,H,n_splits,causal,cap", [
    ([77], [77], 1, 1, 1, 0.0),              # items in halves
    ([100, 30], [2000, 700], 2, 5, 1, 0.0),  # the same, split: the join follows
    ([2048], [2048], 12, 1, 0, 0.0),         # whole items
    ([300], [2300], 1, 2, 0, 20.0),          # with a cap, split
    ([20] * 40, [50] * 40, 2, 1, 1, 0.0),    # more than 32 sequences
])
def test_waits_that_run_out_are_reported(L, lq, lk, H, n_splits, causal, cap):
    x = _prefill_inputs(lq, lk, H, 17)
    L.mla_test_stall_copies(True)
    try:
        _prefill(L, x, lq, lk, n_splits, cap, causal)
        torch.cuda.synchronize()             # the launch ends by itself
        assert L.mla_device_error() == WAIT_TIMEOUT
    finally:
        L.mla_test_stall_copies(False)
    assert L.mla_device_error() == 0         # reading the word cleared it
    out, lse = _prefill(L, x, lq, lk, n_splits, cap, causal)
    torch.cuda.synchronize()
    assert L.mla_device_error() == 0
    R.assert_prefill(out, lse, R.prefill(*x, _cu(lq), _cu(lk), SCALE, cap, bool(causal)), what="after a reported timeout")
