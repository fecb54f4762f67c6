"""Frequencies scaled by parts, against the formula in 64 bits (no GPU needed)."""
import math

import numpy as np
import pytest


@pytest.mark.parametrize("dims, base, scale, context, slow, fast", [
    (128, 10000.0, 8.0, 4096.0, 1.0, 32.0), (128, 500000.0, 8.0, 8192.0, 1.0, 4.0), (64, 10000.0, 40.0, 4096.0, 0.0, 2.0),
    (48, 1000000.0, 1.5, 32768.0, 7.25, 7.5), (2, 10000.0, 4.0, 4096.0, 1.0, 32.0)])
def test_the_mixed_part(dims, base, scale, context, slow, fast):
    import kv_cache_eviction_split_gb300 as kv
    kv.build()
    kv.load()
    w, factor = kv.kv_rotary_frequencies(dims, base, "parts", scale, context, slow, fast)
    plain = base ** (-2.0 * np.arange(dims // 2) / dims)
    turns = context * plain / (2 * math.pi)
    keep = np.clip((turns - slow) / (fast - slow), 0.0, 1.0)
    if dims > 2 and fast > 2 * slow:
        assert ((keep > 0) & (keep < 1)).any()
    # one rounding to fp32, and a few of 64 bits of the mix
    np.testing.assert_allclose(w, plain * (keep + (1 - keep) / scale), rtol=2.0 ** -24 + 2.0 ** -48)
    assert abs(factor - (0.1 * math.log(scale) + 1)) <= 2.0 ** -23
