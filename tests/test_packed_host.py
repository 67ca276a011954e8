"""Host-side checks of the packed operators (no GPU needed), beside those of test_ragged_host.py."""
import pytest

from tests.test_ragged_host import F32, L, _prefill, _strided  # noqa: F401 (L is a fixture)


@pytest.mark.parametrize("scale,status", [(2.0 ** 21, 2), (2.0 ** 100, 2), (3e38, 2), (float("inf"), 1)])
@pytest.mark.parametrize("cap", [0.0, 2.0 ** -10])
def test_prefill_refuses_scales_whose_scores_fp32_cannot_hold(L, scale, status, cap):  # noqa: F811
    assert _prefill(L, sm=scale, cap=cap) == status
    assert "sm_scale" in L.mla_last_error()


@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("window", [0, 1, 5000])
def test_automatic_splits_leave_the_longest_part_four_blocks(L, causal, window):  # noqa: F811
    """The longest item's blocks of 128 keys (for items of 256 or of 128 rows), cut into the automatic count: the longest
    part has four at least."""
    for B in (1, 2, 17, 1000):
        for H in (1, 3, 12, 96):
            for max_q in (1, 128, 129, 700, 5000, 70000):
                for max_k in (1, 500, 600, 1664, 9000, 70000, 1 << 20):
                    n = L.mla_prefill_auto_splits(B * max_q, B, H, max_q, max_k, causal, window, 152)
                    assert 1 <= n <= 256
                    longest = 0
                    for rows in (128, 256):
                        keys = min(max_k, window + min(max_q, rows)) if window else max_k
                        longest = max(longest, -(-(-(-keys // 128)) // n))
                    assert n == 1 or longest >= 4


def test_tensors_without_elements_are_contiguous(L):  # noqa: F811
    """An lse [5, 0] of a call without heads, its strides as torch gives them (1, 1)."""
    assert _prefill(L, H=0, lse=_strided([5, 0], [1, 1], F32)) == 0
    assert _prefill(L, lse=_strided([5, 3], [1, 1], F32)) == 2      # with elements they have to be
