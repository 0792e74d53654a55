"""lora_rope_inv_freq's lengthened frequencies against numbers worked out by hand (host only)."""
import numpy as np

import weight_patches_gb300 as wpg


def test_yarn_ramp_is_linear_in_the_pairs_index():
    # 64 of base 10000, 4096 positions: the index that turns 32 times is 64 ln(4096 / 64 pi) / (2 ln 10000) = 10.47, the one that
    # turns once 22.51, so the ramp goes from 10 to 23
    base, one = wpg.lora_rope_inv_freq(64)
    yarn, factor = wpg.lora_rope_inv_freq(64, scaling="yarn", scale=8.0, original_length=4096)
    ramp = np.clip((np.arange(32) - 10) / 13, 0, 1)
    assert np.allclose((yarn / base).numpy(), 1 - ramp * (1 - 1 / 8), rtol=1e-14)


def test_yarn_ramp_within_the_head():
    # a short context: index 32 turns would lie below 0, a long one with few pairs: the end is cut to rot - 1
    base, _ = wpg.lora_rope_inv_freq(16)
    share = (wpg.lora_rope_inv_freq(16, scaling="yarn", scale=4.0, original_length=64)[0] / base).numpy()
    # 32 turns: 16 ln(64 / 64 pi) / (2 ln 10000) < 0; one: 2.02, so from 0 to 3
    assert np.allclose(share, 1 - np.clip(np.arange(8) / 3, 0, 1) * 0.75, rtol=1e-14)
    # one turn: 16 ln(1e9 / 2 pi) / 18.42 = 16.4, cut to 15; 32 turns 13.4, so 13: no pair of 8 reaches the ramp
    share = (wpg.lora_rope_inv_freq(16, scaling="yarn", scale=4.0, original_length=10 ** 9)[0] / base).numpy()
    assert np.all(share == 1)
