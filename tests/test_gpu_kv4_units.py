"""The unit in which the 4-bit decode attention rounds its weights, over runs of many tiles.

A warp takes a run of 64-key tiles, so a request is made long enough that every run has nine tiles or more: one period of
16 tiles, the keys all zero (the logits are gain * bias), repeated.  The expected output is the float64 softmax over one
period.  Tolerances as in test_gpu_kv4.py."""
import math

import numpy as np
import pytest
import torch

from learned_token_pruning_b200 import synth, tokengate as tg
from oracle import kv4_oracle as K
from test_gpu_kv4 import Batch, _dev, _i32

pytestmark = pytest.mark.gpu
DEV = "cuda"
TILE, TILES = 64, 16
ROWS = TILE * TILES
SHAPES = [(16, 8, 128), (6, 2, 64), (8, 1, 128), (3, 1, 128)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", SHAPES)
@pytest.mark.parametrize("shift", [112, 116, 120, 123])
def test_a_tiny_weight_times_a_huge_value_counts(shift, hq, hkv, d, dtype):
    # weights of 2^-shift (normal floats) on values 2^shift times the others': equal contributions.  Logits of
    # 120 in base 2 are off by at most 3 * 120 * 2^-24, which the tolerance of 1e-4 holds
    b = Batch([150, 20], hq, hkv, d, 16, dtype, seed=51)
    b.gain[:] = 1.0
    b.temp[:] = 2.0 ** -4
    for s, n in ((0, 150), (150, 20)):
        few = s + np.arange(3, n, 17)
        b.bias[few] = -shift * math.log(2)
        b.v[few] = synth.round_to(np.clip(b.v[few], -2, 2) * np.float32(2.0 ** shift), "bf16")
    b.store()
    b.go()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", SHAPES)
def test_negative_scales_negate_what_the_codes_stand_for(hq, hkv, d, dtype):
    # the pools are the caller's memory, and a scale has a sign
    b = Batch([300, 70], hq, hkv, d, 16, dtype, seed=50)
    s, page, row = b.slots[:300], b.slots[:300] // 16, b.slots[:300] % 16
    pick = np.random.default_rng(3).random((300, hkv, d // 32)) < 0.4
    for scales, x in ((b.cache.v_scales, b.v), (b.cache.k_scales, b.k)):
        at = scales[_dev(page).long(), :, _dev(row).long()]            # [300, hkv, d / 32]
        scales[_dev(page).long(), :, _dev(row).long()] = torch.where(_dev(pick), -at, at)
        x[:300] *= np.where(np.repeat(pick, 32, -1), -1, 1)
    b.go()
