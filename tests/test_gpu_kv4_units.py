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


def _long(hq, hkv, d, dtype, bias, factor, gain, seed, same=False):
    """Attention over one request: `bias` [TILES, TILE] and value factors [TILES] of a period, repeated until every warp's
    run has nine tiles; the result against the softmax over one period."""
    rng = np.random.default_rng(seed)
    runs = torch.cuda.get_device_properties(0).multi_processor_count * 12
    n = -(-9 * runs // (hkv * TILES))
    v = rng.standard_normal((1 if same else TILE, hkv, d)) + (2.0 if same else 0.0)
    v = np.broadcast_to(v, (TILE, hkv, d)).astype(np.float32)
    v = synth.round_to((v[None] * np.asarray(factor, np.float32)[:, None, None, None]).reshape(ROWS, hkv, d), "bf16")
    bias = np.asarray(bias, np.float32).reshape(ROWS)
    page = 64
    pages = n * ROWS // page
    cache = tg.KV4Cache.zeros(pages, page, hkv, d)
    dv = _dev(v.reshape(ROWS, hkv * d), torch.bfloat16).repeat(n, 1)
    slots = torch.arange(n * ROWS, dtype=torch.int32, device=DEV)
    tg.tg_kv4_store(cache, torch.zeros_like(dv), dv, _dev(bias).repeat(n), slots)
    dt = synth.torch_dtype(dtype)
    q = synth.round_to(rng.standard_normal((1, hq * d)).astype(np.float32), dtype)
    out, lse = torch.full((1, hq * d), 7.0, dtype=dt, device=DEV), torch.full((1, hq), 7.0, device=DEV)
    gain, temp = np.asarray(gain, np.float32), np.ones(hq, np.float32)
    ws = torch.full((tg.kv4_decode_workspace_bytes(hq, hkv, d),), 0xA5, dtype=torch.uint8, device=DEV)
    tg.tg_kv4_decode_attention(cache, _dev(q, dt), torch.arange(pages, dtype=torch.int32, device=DEV)[None], _i32([n * ROWS]),
                               _dev(gain), _dev(temp), None, d ** -0.5, out, ws, lse)
    assert tg.tg_check_device_error() == 0
    val, zero = K.kv4_quantize(v)[0], np.zeros((ROWS, hkv, d))
    want, wl = K.kv4_decode_attention(q.reshape(hq, d), zero, val, bias, gain, temp, 1.0, d ** -0.5)
    size, _ = K.kv4_decode_attention(q.reshape(hq, d), zero, np.abs(val), bias, gain, temp, 1.0, d ** -0.5)
    half, slack = (2.0 ** -8, 2.0 ** -10) if dtype == "bf16" else (2.0 ** -24, 1e-4)
    err = np.abs(out.float().cpu().numpy().reshape(hq, d) - want)
    tol = half * np.abs(want) + slack * size
    assert (err <= tol).all(), (float((err / tol).max()), float((err / np.maximum(size, 1e-30)).max()))
    np.testing.assert_allclose(lse[0].cpu().numpy(), wl + math.log(n), rtol=1e-4, atol=1e-4)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", SHAPES)
@pytest.mark.parametrize("steps", [(12, 24), (12, 24, 36), (4, 8, 12, 16, 20, 24, 28, 32)])
def test_masked_rows_that_grow_from_tile_to_tile_leave_the_others_exact(steps, hq, hkv, d, dtype):
    # each masked tile's values are a step larger than the last one's: no step may raise the unit without a weight
    bias = np.random.default_rng(5).standard_normal((TILES, TILE))
    factor = np.ones(TILES)
    for i, e in enumerate(steps):
        bias[3 + i], factor[3 + i] = -250.0, 2.0 ** e
    _long(hq, hkv, d, dtype, bias, factor, np.ones(hq), 60)


@pytest.mark.parametrize("hq,hkv,d", SHAPES)
@pytest.mark.parametrize("step", [6, 8, 12])
def test_one_step_of_masked_rows_leaves_the_small_weights_their_digits(step, hq, hkv, d):
    # one key of weight 1 and 959 of 2^-14 with the same values: what rounding does to one of them it does to all
    bias = np.full((TILES, TILE), -14 * math.log(2) - 0.3)
    bias[0, 0] = 0.0
    factor = np.ones(TILES)
    bias[4], factor[4] = -250.0, 2.0 ** step
    _long(hq, hkv, d, "f32", bias, factor, np.ones(hq), 61, same=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", SHAPES)
def test_the_unit_comes_down_as_the_reference_rises(hq, hkv, d, dtype):
    # logits rise by 11 (base 2) from tile to tile while the values shrink by 2^10: the last tiles carry the output
    bias = np.random.default_rng(6).standard_normal((TILES, TILE)) * 0.5
    factor = np.ones(TILES)
    for j in range(6):
        bias[j] -= 11 * (6 - j) * math.log(2)
        factor[j] = 2.0 ** (10 * (6 - j))
    _long(hq, hkv, d, dtype, bias, factor, np.ones(hq), 62)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", SHAPES)
def test_a_neighbouring_heads_products_leave_a_heads_weights_their_digits(hq, hkv, d, dtype):
    # odd heads meet large products in the first tile, which the last one's logits make nothing of; the even
    # heads give all their weight to the tiles between
    bias = np.random.default_rng(7).standard_normal((TILES, TILE)) * 0.5
    factor = np.ones(TILES)
    bias[0], factor[0] = -200 * math.log(2), 2.0 ** 40
    bias[-1] = -400 * math.log(2)
    gain = np.where(np.arange(hq) % (hq // hkv) % 2 == 0, 1.0, -0.3)
    _long(hq, hkv, d, dtype, bias, factor, gain, 63)


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
