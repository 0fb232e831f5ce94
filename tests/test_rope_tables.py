"""Frequency tables whose ramp reaches past their last pair."""
import math

import pytest


@pytest.mark.parametrize("rot", [64, 128, 20])
@pytest.mark.parametrize("original_len", [2048, 65536, 131072, 1 << 20])
@pytest.mark.parametrize("factor", [4.0, 8.0])
def test_blend_over_long_contexts(rot, original_len, factor):
    """The straight line runs to the pair index that turns `low` times, in the table
    or behind it: a pair that turns more often is never slowed by the whole factor."""
    import torch
    import dynamic_block_sparse_tiled_b200 as bl
    base = 10000.0
    got, mscale = bl.rope_frequencies(rot, base=base, scaling="blend", factor=factor, original_len=original_len,
                                      device="cpu")
    assert math.isclose(mscale, 0.1 * math.log(factor) + 1.0)
    # pair i turns original_len / (2 pi) base^(-2 i / rot) times
    index = lambda turns: math.log(original_len / (2 * math.pi * turns)) / math.log(base) * rot / 2  # noqa: E731
    first, last = max(math.floor(index(32.0)), 0), math.ceil(index(1.0))
    for i in range(rot // 2):
        plain = base ** (-2.0 * i / rot)
        slowed = min(max((i - first) / (last - first), 0.0), 1.0)
        want = plain * (1.0 - slowed) + plain / factor * slowed
        assert math.isclose(float(got[i]), want, rel_tol=1e-12), i
        if original_len * plain / (2 * math.pi) > 1.0:
            assert float(got[i]) > plain / factor * (1 + 1e-9), i
    assert got.dtype == torch.float64
