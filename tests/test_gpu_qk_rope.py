"""tg_qk_norm_rope and its gradients against the float64 oracle.

Tolerances.  bf16 out: half a step, 2^-8 of the value.  fp32 arithmetic, per pair (a, b) of the normalised row: the
sum of D squares (8 in line, 3 exchanges), 1/sqrt, two products and the rotation are at most 24 roundings of 2^-24,
cosine and sine of the reduced angle are off by at most 2^-22 (the remainder's rounding, 2^-23 of pi, and 2 ulp), so
|error| <= 2^-18 (|a| + |b|).  Gradients: the same with g in the place of the row, and r |x| |mean(g w x)| r^2 beside it;
dw sums m * heads such terms in at most 2^13 additions of partial sums, each 2^-24 of the sum of magnitudes."""
import numpy as np
import pytest
import torch

from learned_token_pruning_b200 import synth, tokengate as tg
from oracle import kv4_oracle as K

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS, THETA = 1e-6, 1e6
SLACK = 2.0 ** -18


def _half(dtype):
    return 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24


def _inputs(m, hq, hkv, d, dtype, seed, far=131072):
    rng = np.random.default_rng(seed)
    x = synth.round_to(rng.standard_normal((m, hq + 2 * hkv, d)).astype(np.float32), dtype)
    pos = np.sort(rng.integers(0, far, m)).astype(np.int32)
    return x, pos, rng.uniform(0.5, 1.5, d).astype(np.float32), rng.uniform(0.5, 1.5, d).astype(np.float32), rng


def _dev(a, dt=None):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV, dt)


def _pair(y, d):
    """|a| + |b| of every rotated pair, for both of its places."""
    s = np.abs(y[..., :d // 2]) + np.abs(y[..., d // 2:])
    return np.concatenate([s, s], -1)


def _views(x, hq, hkv, d, dt):
    buf = _dev(x.reshape(x.shape[0], -1), dt)
    return buf, buf[:, :hq * d], buf[:, hq * d:(hq + hkv) * d]


def _check_forward(m, hq, hkv, d, dtype, seed, norm=True, weights=True, in_place=False, pos=None):
    x, p, wq, wk, _ = _inputs(m, hq, hkv, d, dtype, seed)
    pos = p if pos is None else pos
    dt = synth.torch_dtype(dtype)
    buf, q, k = _views(x, hq, hkv, d, dt)
    qo, ko = (q, k) if in_place else (torch.full((m, hq * d), 7.0, dtype=dt, device=DEV),
                                      torch.full((m, hkv * d), 7.0, dtype=dt, device=DEV))
    tg.tg_qk_norm_rope(q, k, d, _dev(pos), _dev(wq) if weights else None, _dev(wk) if weights else None, EPS, THETA, qo, ko,
                       qk_norm=norm)
    torch.cuda.synchronize()
    for got, rows, w in ((qo, x[:, :hq], wq), (ko, x[:, hq:hq + hkv], wk)):
        w = w if weights else None
        want = K.qk_norm_rope(rows, w, pos, THETA, EPS, norm)
        flat = K.rms_norm(rows, w, EPS) if norm else rows.astype(np.float64)
        tol = _half(dtype) * np.abs(want) + SLACK * _pair(flat, d)
        err = np.abs(got.float().cpu().numpy().reshape(want.shape) - want)
        assert (err <= tol).all(), float((err / np.maximum(tol, 1e-30)).max())
    if in_place:   # the values next to q and k are not touched
        np.testing.assert_array_equal(buf[:, (hq + hkv) * d:].float().cpu().numpy(), x[:, hq + hkv:].reshape(m, -1))
    return qo.clone(), ko.clone()


@pytest.mark.parametrize("m", [1, 2, 9, 64, 257])
@pytest.mark.parametrize("hq,hkv,d", [(16, 8, 128), (4, 2, 64), (6, 2, 64), (5, 1, 128), (1, 1, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_forward(m, hq, hkv, d, dtype):
    _check_forward(m, hq, hkv, d, dtype, seed=m + hq)


@pytest.mark.parametrize("norm,weights,in_place", [(False, True, False), (True, False, False), (True, True, True),
                                                   (False, False, True)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_forward_variants(norm, weights, in_place, dtype):
    _check_forward(37, 16, 8, 128, dtype, seed=3, norm=norm, weights=weights, in_place=in_place)


def test_forward_prompt_rows_take_whole_rows_per_warp():
    a = _check_forward(4160, 16, 8, 128, "bf16", seed=5)
    b = _check_forward(4160, 16, 8, 128, "bf16", seed=5, in_place=True)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_forward_negative_and_far_positions():
    # up to 2^26 the fp64 angle keeps 2^-26 of a radian; both sides form it the same way
    pos = np.array([-5, -1, 0, 1, 2 ** 20, 2 ** 26], np.int32)
    _check_forward(6, 4, 2, 128, "f32", seed=6, pos=pos)


def test_forward_zero_rows_and_zero_sized_call():
    d = 64
    q = torch.zeros(3, 4 * d, device=DEV)
    k = torch.zeros(3, 2 * d, device=DEV)
    qo, ko = torch.ones_like(q), torch.ones_like(k)
    pos = torch.arange(3, dtype=torch.int32, device=DEV)
    tg.tg_qk_norm_rope(q, k, d, pos, None, None, EPS, THETA, qo, ko)
    assert not qo.any() and not ko.any()     # a row of zeros stays one: eps keeps the norm finite
    tg.tg_qk_norm_rope(q[:0], k[:0], d, pos[:0], None, None, EPS, THETA, qo[:0], ko[:0])


def _check_backward(m, hq, hkv, d, dtype, seed, norm=True, weights=True, sums=True, in_place=False):
    x, pos, wq, wk, rng = _inputs(m, hq, hkv, d, dtype, seed)
    dt = synth.torch_dtype(dtype)
    dy = [rng.standard_normal((m, h, d)).astype(np.float32) for h in (hq, hkv)]
    buf, q, k = _views(x, hq, hkv, d, dt)
    qi, ki = (q, k) if in_place else _views(np.zeros_like(x), hq, hkv, d, dt)[1:]
    need = tg.qk_rope_backward_workspace_bytes(m, d)
    ws = torch.full((need,), 0xA5, dtype=torch.uint8, device=DEV) if sums else None
    dw = [torch.full((d,), 9.0, device=DEV) for _ in range(2)] if sums else [None, None]
    tg.tg_qk_norm_rope_backward(q, k, d, _dev(pos), _dev(wq) if weights else None, _dev(wk) if weights else None, EPS, THETA,
                                _dev(dy[0].reshape(m, -1)), _dev(dy[1].reshape(m, -1)), qi, ki, ws, dw_q=dw[0], dw_k=dw[1],
                                qk_norm=norm)
    torch.cuda.synchronize()
    for got, gw, rows, w, g in ((qi, dw[0], x[:, :hq], wq, dy[0]), (ki, dw[1], x[:, hq:hq + hkv], wk, dy[1])):
        w = w if weights else None
        dx, want_w = K.qk_norm_rope_backward(rows, w, pos, THETA, EPS, g, norm)
        back = K.rope(g.astype(np.float64), -pos.astype(np.float64), THETA)
        size = _pair(back, d)
        if norm:
            r = 1 / np.sqrt(np.mean(rows.astype(np.float64) ** 2, -1, keepdims=True) + EPS)
            wv = np.ones(d) if w is None else w.astype(np.float64)
            size = r * np.abs(wv) * size + np.abs(rows) * r ** 3 * np.mean(np.abs(wv * size * rows), -1, keepdims=True)
        tol = _half(dtype) * np.abs(dx) + SLACK * size
        err = np.abs(got.float().cpu().numpy().reshape(dx.shape) - dx)
        assert (err <= tol).all(), float((err / np.maximum(tol, 1e-30)).max())
        if sums and norm:
            mag = np.sum(_pair(back, d) * np.abs(rows) * r, axis=(0, 1))
            np.testing.assert_array_less(np.abs(gw.cpu().numpy() - want_w), (SLACK + m * (hq + hkv) ** 0.5 * 2.0 ** -24) * mag + 1e-30)
        elif sums:
            assert not gw.any()
    return [t.clone() for t in (qi, ki, *dw) if t is not None]


@pytest.mark.parametrize("m", [1, 3, 8, 65])
@pytest.mark.parametrize("hq,hkv,d", [(16, 8, 128), (4, 2, 64), (6, 2, 64), (5, 1, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward(m, hq, hkv, d, dtype):
    _check_backward(m, hq, hkv, d, dtype, seed=m * 3 + hq)


@pytest.mark.parametrize("norm,weights,sums,in_place", [(False, True, True, False), (True, False, True, False),
                                                        (True, True, False, False), (True, True, True, True),
                                                        (False, True, False, False)])
def test_backward_variants(norm, weights, sums, in_place):
    _check_backward(41, 16, 8, 128, "bf16", 11, norm=norm, weights=weights, sums=sums, in_place=in_place)


def test_backward_prompt_rows_and_reruns_are_identical():
    a = _check_backward(3001, 16, 8, 128, "bf16", 12)
    b = _check_backward(3001, 16, 8, 128, "bf16", 12)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("m,hq,hkv,d,dtype", [(593, 16, 8, 128, "bf16"), (1187, 10, 2, 128, "bf16"), (2999, 6, 2, 64, "f32"),
                                              (700, 70, 7, 64, "bf16"), (310, 40, 33, 128, "f32")])
def test_rows_cut_into_parts(m, hq, hkv, d, dtype):
    # a row's passes shared by several warps, the last part shorter, q and k in one part
    _check_forward(m, hq, hkv, d, dtype, seed=m)
    _check_backward(m, hq, hkv, d, dtype, seed=m + 1)


def test_backward_against_differences_of_the_forward():
    # central differences of the CUDA forward in fp32, along random directions
    m, hq, hkv, d, h = 5, 2, 1, 64, 2.0 ** -6
    x, pos, wq, wk, rng = _inputs(m, hq, hkv, d, "f32", 13, far=100)
    dy = [_dev(rng.standard_normal((m, n * d)).astype(np.float32)) for n in (hq, hkv)]
    dirs = [_dev(rng.standard_normal((m, n * d)).astype(np.float32)) for n in (hq, hkv)]
    q, k = [_dev(t.reshape(m, -1)) for t in (x[:, :hq], x[:, hq:hq + hkv])]
    pos, wq, wk = _dev(pos), _dev(wq), _dev(wk)

    def f(q_, k_, wq_, wk_):
        qo, ko = torch.empty_like(q), torch.empty_like(k)
        tg.tg_qk_norm_rope(q_, k_, d, pos, wq_, wk_, EPS, THETA, qo, ko)
        return float((qo.double() * dy[0]).sum() + (ko.double() * dy[1]).sum())

    qi, ki, dwq, dwk = torch.empty_like(q), torch.empty_like(k), torch.empty(d, device=DEV), torch.empty(d, device=DEV)
    ws = torch.empty(tg.qk_rope_backward_workspace_bytes(m, d), dtype=torch.uint8, device=DEV)
    tg.tg_qk_norm_rope_backward(q, k, d, pos, wq, wk, EPS, THETA, dy[0], dy[1], qi, ki, ws, dw_q=dwq, dw_k=dwk)
    # third-order term of the difference: h^2 / 6 of a third derivative of about the size of the sum itself
    got = float((qi.double() * dirs[0]).sum() + (ki.double() * dirs[1]).sum())
    num = (f(q + h * dirs[0], k + h * dirs[1], wq, wk) - f(q - h * dirs[0], k - h * dirs[1], wq, wk)) / (2 * h)
    size = float((qi.double() * dirs[0]).abs().sum() + (ki.double() * dirs[1]).abs().sum())
    assert abs(got - num) <= (h * h + 2.0 ** -12) * size
    v = _dev(rng.standard_normal(d).astype(np.float32))
    num = (f(q, k, wq + h * v, wk + h * v) - f(q, k, wq - h * v, wk - h * v)) / (2 * h)
    got = float(((dwq + dwk).double() * v).sum())
    assert abs(got - num) <= (h * h + 2.0 ** -12) * float(((dwq.abs() + dwk.abs()).double() * v.abs()).sum())


def test_backward_zero_rows_zeroes_the_weight_gradients():
    d = 64
    e = lambda n: torch.empty(0, n * d, device=DEV)
    dwq, dwk = torch.ones(d, device=DEV), torch.ones(d, device=DEV)
    tg.tg_qk_norm_rope_backward(e(2), e(1), d, torch.empty(0, dtype=torch.int32, device=DEV), None, None, EPS, THETA, e(2), e(1),
                                e(2), e(1), None, dw_q=dwq, dw_k=dwk)
    assert not dwq.any() and not dwk.any()


def test_forward_and_backward_in_a_replayed_graph():
    m, hq, hkv, d = 20, 16, 8, 128
    x, pos, wq, wk, rng = _inputs(m, hq, hkv, d, "bf16", 14)
    dt = torch.bfloat16
    buf, q, k = _views(x, hq, hkv, d, dt)
    pos, wq, wk = _dev(pos), _dev(wq), _dev(wk)
    dq, dk = [torch.randn(m, n * d, device=DEV) for n in (hq, hkv)]
    ws = torch.empty(tg.qk_rope_backward_workspace_bytes(m, d), dtype=torch.uint8, device=DEV)
    e = lambda: [torch.empty(m, hq * d, dtype=dt, device=DEV), torch.empty(m, hkv * d, dtype=dt, device=DEV)]

    def call(o):
        tg.tg_qk_norm_rope(q, k, d, pos, wq, wk, EPS, THETA, o[0], o[1])
        tg.tg_qk_norm_rope_backward(q, k, d, pos, wq, wk, EPS, THETA, dq, dk, o[2], o[3], ws, dw_q=o[4], dw_k=o[5])

    new = lambda: e() + e() + [torch.empty(d, device=DEV), torch.empty(d, device=DEV)]
    eager, held = new(), new()
    call(held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(held)
    for _ in range(2):
        buf.normal_()
        pos.add_(3)
        graph.replay()
        call(eager)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, held))
    del graph
