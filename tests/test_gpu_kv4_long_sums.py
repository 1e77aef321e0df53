"""Attention with fp32 queries over runs of a thousand tiles: the sums must not drift with the number of additions.

One page of rows, named by every entry of the table, so that the expected output is the float64 softmax over that page
whatever the length.  Tolerance, in steps of 2^-24 of A = sum softmax |v|: a tile's eight matrix instructions cut their sums
(2 steps each), one addition a tile of the run, under 100 more joining warps and parts, and 50 for the weights themselves
(logits below 8 in base 2 off by 3 roundings, the exponential by 4 steps, two parts of 11 bits, numerator and denominator)."""
import math

import numpy as np
import pytest
import torch

from learned_token_pruning_b200 import tokengate as tg
from oracle import kv4_oracle as K
from test_gpu_kv4 import DEV, _dev, _i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,d,page", [(2, 1, 64, 128), (2, 1, 128, 64), (8, 1, 128, 128), (3, 1, 128, 128)])
def test_sums_of_a_thousand_tiles(hq, hkv, d, page):
    rng = np.random.default_rng(d + hq)
    tiles = 1000
    rows = tiles * 64 * 8 * torch.cuda.get_device_properties(0).multi_processor_count
    n = rows // page
    v = (np.abs(rng.standard_normal((page, hkv, d))) + 0.5).astype(np.float32)
    bias = rng.standard_normal(page).astype(np.float32)
    cache = tg.KV4Cache.zeros(1, page, hkv, d)
    dv = _dev(v.reshape(page, hkv * d))
    tg.tg_kv4_store(cache, torch.zeros_like(dv), dv, _dev(bias), torch.arange(page, dtype=torch.int32, device=DEV))
    q, one = rng.standard_normal((1, hq * d)).astype(np.float32), np.ones(hq, np.float32)
    out, lse = torch.empty(1, hq * d, device=DEV), torch.empty(1, hq, device=DEV)
    ws = torch.full((tg.kv4_decode_workspace_bytes(hq, hkv, d),), 0xA5, dtype=torch.uint8, device=DEV)
    tg.tg_kv4_decode_attention(cache, _dev(q), torch.zeros(1, n, dtype=torch.int32, device=DEV), _i32([rows]), _dev(one),
                               _dev(one), None, d ** -0.5, out, ws, lse)
    assert tg.tg_check_device_error() == 0
    val = K.kv4_quantize(v)[0]
    want, wl = K.kv4_decode_attention(q.reshape(hq, d), np.zeros_like(val), val, bias, one, one, 1.0, d ** -0.5)
    err = np.abs(out.cpu().numpy().reshape(hq, d) - want)
    tol = (16 + tiles + 100 + 50) * 2.0 ** -24 * np.abs(want)          # v > 0: A is the output
    assert (err <= tol).all(), float((err / np.abs(want)).max())
    np.testing.assert_allclose(lse[0].cpu().numpy(), wl + math.log(n), rtol=1e-5)
