"""Host side of the paged cache's records: what a KvCache may be made of."""
import pytest

import fp4_spectral_split_amd as M


def test_tensor_scales_of_a_cache_are_positive_numbers():
    good = M.KvCache.empty("nvfp4", 2, 16, 1, 64, "cpu", 2.0 ** -126, 3e38)
    assert float(good.k.tensor_scale) == 2.0 ** -126 and not good.v.codes.any()
    for bad in (0.0, -0.01, float("nan"), float("inf"), 1e-45, 1e39):
        for pair in ((bad, 0.01), (0.01, bad)):
            with pytest.raises(M.MetisError):
                M.KvCache.empty("nvfp4", 2, 16, 1, 64, "cpu", *pair)
