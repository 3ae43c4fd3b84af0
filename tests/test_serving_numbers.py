"""The serving binding's checks of numbers that the C fields would cut (CPU)."""
import pytest

from sparse_kv_cache_kmax_b200 import binding as B


def test_windows_past_32_bits_are_refused():
    """The C field would keep the low half: 2³² + 5 would hide all but five tokens."""
    for window in (2 ** 31, 2 ** 32 + 5, -1, -2 ** 31):
        with pytest.raises(ValueError):
            B.make_score_mod(window=window)
    assert B.make_score_mod(window=2 ** 31 - 1).window == 2 ** 31 - 1 and B.make_score_mod(window=None).window == 0
