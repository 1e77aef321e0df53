"""The norm-weight gradients of tg_qk_norm_rope_backward, with a bound that one lost row breaks.

A lane adds the terms of its warp's passes, five exchanges at most join the warp, eight additions the block, and the
second kernel adds ceil(blocks / 32) partials and then 32: n additions in line, each 2^-24 of the sum of magnitudes.  A
term g x r itself is within 24 such steps (cosine and sine 4, the rotation 3, r 8, the products 3, and room)."""
import numpy as np
import pytest
import torch

from learned_token_pruning_b200 import synth, tokengate as tg
from oracle import kv4_oracle as K
from test_gpu_qk_rope import EPS, THETA, _dev, _inputs, _pair, _views

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("m,hq,hkv,d,dtype", [(3001, 16, 8, 128, "bf16"), (2999, 6, 2, 64, "f32"), (593, 16, 8, 128, "bf16"),
                                              (1187, 10, 2, 128, "bf16"), (5000, 5, 1, 128, "f32"), (310, 40, 33, 128, "f32"),
                                              (8256, 4, 2, 64, "bf16")])
def test_weight_gradients_hold_every_row(m, hq, hkv, d, dtype):
    x, pos, wq, wk, rng = _inputs(m, hq, hkv, d, dtype, m)
    dt = synth.torch_dtype(dtype)
    dy = [rng.standard_normal((m, h, d)).astype(np.float32) for h in (hq, hkv)]
    _, q, k = _views(x, hq, hkv, d, dt)
    qi, ki = torch.empty(m, hq * d, dtype=dt, device=DEV), torch.empty(m, hkv * d, dtype=dt, device=DEV)
    ws = torch.full((tg.qk_rope_backward_workspace_bytes(m, d),), 0xA5, dtype=torch.uint8, device=DEV)
    dw = [torch.full((d,), 9.0, device=DEV) for _ in range(2)]
    tg.tg_qk_norm_rope_backward(q, k, d, _dev(pos), _dev(wq), _dev(wk), EPS, THETA, _dev(dy[0].reshape(m, -1)),
                                _dev(dy[1].reshape(m, -1)), qi, ki, ws, dw_q=dw[0], dw_k=dw[1])
    torch.cuda.synchronize()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    passes = -(-hq * d // 512) + -(-hkv * d // 512)
    n = -(-m // (16 * sms)) * passes + 5 + 8 + -(-2 * sms // 32) + 32
    for got, rows, w, g in ((dw[0], x[:, :hq], wq, dy[0]), (dw[1], x[:, hq:hq + hkv], wk, dy[1])):
        rows = rows.astype(np.float64)
        back = K.rope(g.astype(np.float64), -pos.astype(np.float64), THETA)
        r = 1 / np.sqrt(np.mean(rows ** 2, -1, keepdims=True) + EPS)
        terms = (back * rows * r).sum(1)                                   # [m, d]
        want = K.qk_norm_rope_backward(rows, w, pos, THETA, EPS, g, True)[1]
        np.testing.assert_allclose(terms.sum(0), want, rtol=0, atol=1e-9 * m)
        tol = (n + 24) * 2.0 ** -24 * np.sum(_pair(back, d) * np.abs(rows) * r, axis=(0, 1))
        err = np.abs(got.cpu().numpy() - want)
        assert (err <= tol).all(), float((err / tol).max())
        # the bound is sharp enough: the oracle without any one row leaves it
        assert (np.abs(terms) > 2 * tol).any(1).all()
