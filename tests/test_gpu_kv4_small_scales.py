"""Rows of the smallest magnitudes into the 4-bit cache, against the oracle's single rounding in 64 bits (exact)."""
import numpy as np
import pytest
import torch

from learned_token_pruning_b200 import tokengate as tg
from oracle import kv4_oracle as K
from test_gpu_kv4 import DEV, I32, _dev

pytestmark = pytest.mark.gpu


def test_store_scales_below_the_smallest_normal_number_round_once():
    # fp32 rows whose largest value over 6 lies just beside the middle of two bf16 numbers below 2^-126: the quotient
    # does not fit fp32 there, so it must not be rounded twice
    u = 2.0 ** -149
    rows = []
    for i in list(range(12)) + [31, 32, 62, 63, 125, 126, 127]:
        for step in (-1, 0, 1):
            top = 6 * (2 * i + 1) * 2.0 ** -134 + step * u
            rows.append(np.concatenate([[top], top * np.linspace(-1, 1, 31)]))
    x = np.tile(np.array(rows).astype(np.float32), (1, 2))
    n = len(x)
    cache = tg.KV4Cache.zeros(-(-n // 16), 16, 1, 64)
    slots = torch.arange(n, dtype=I32, device=DEV)
    tg.tg_kv4_store(cache, _dev(x), _dev(x), None, slots)
    k, v = torch.empty(n, 64, device=DEV), torch.empty(n, 64, device=DEV)
    tg.tg_kv4_load(cache, slots, k, v)
    want = K.kv4_quantize(x)[0]
    np.testing.assert_array_equal(k.cpu().numpy(), want)
    np.testing.assert_array_equal(v.cpu().numpy(), want)
