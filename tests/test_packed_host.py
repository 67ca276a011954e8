"""Host-side checks of the packed operators (no GPU needed), beside those of test_ragged_host.py."""
import pytest

from tests.test_ragged_host import L, _prefill  # noqa: F401 (L is a fixture)


@pytest.mark.parametrize("scale,status", [(2.0 ** 21, 2), (2.0 ** 100, 2), (3e38, 2), (float("inf"), 1)])
@pytest.mark.parametrize("cap", [0.0, 2.0 ** -10])
def test_prefill_refuses_scales_whose_scores_fp32_cannot_hold(L, scale, status, cap):  # noqa: F811
    assert _prefill(L, sm=scale, cap=cap) == status
    assert "sm_scale" in L.mla_last_error()
