"""Yarn scaling as rope_frequencies states it."""
import math

import pytest


@pytest.mark.parametrize("length", [1, 2, 5, 6, 7, 16, 60, 201, 202, 4096, 1 << 20])
@pytest.mark.parametrize("rope,axes", [(2, 1), (8, 1), (64, 1), (96, 3), (256, 1)])
@pytest.mark.parametrize("slow", [0.5, 1.0, 4.0])
def test_yarn_scales_pairs_of_few_turns(rope, axes, length, slow):
    """Pairs of at most beta_slow turns within the length are slowed by the whole factor, those of at
    least beta_fast are as they were, and none by more or less than that."""
    import video_dit_block_b200 as sba
    plain = sba.rope_frequencies(rope, axes=axes).inv_freq
    yarn = sba.rope_frequencies(rope, axes=axes, scaling="yarn", factor=4.0, original_length=length, beta_slow=slow)
    for f, p in zip(yarn.inv_freq, plain):
        turns = length * p / (2 * math.pi)
        if turns <= slow * (1 - 1e-12):
            assert f == pytest.approx(p / 4, rel=1e-12), (turns, f / p)
        if turns >= 32 * (1 + 1e-12):
            assert f == pytest.approx(p, rel=1e-12), (turns, f / p)
        assert p / 4 * (1 - 1e-12) <= f <= p * (1 + 1e-12)


@pytest.mark.parametrize("base", [0.5, 1.0, 1e-3])
def test_yarn_refuses_a_base_of_at_most_one(base):
    """Its frequencies do not fall with the pair, and the ramp runs over pairs of falling ones."""
    import video_dit_block_b200 as sba
    with pytest.raises(ValueError):
        sba.rope_frequencies(64, base=base, scaling="yarn", factor=2.0)
