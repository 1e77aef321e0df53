"""Pins of the 4-bit cache oracle, and host-side checks of its entry points (CPU)."""
import ctypes
import itertools
import math

import numpy as np
import pytest
import torch

from learned_token_pruning_b200 import build, synth, tokengate as tg
from oracle import kv4_oracle as K


@pytest.fixture(scope="module")
def L():
    build.build()
    return tg.lib()


# ------------------------------------------------------------------ pins
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("d", [64, 128])
def test_qk_norm_rope_and_gradients_against_autograd_and_differences(d, norm):
    rng = np.random.default_rng(d)
    m, h, theta, eps = 3, 2, 1e6, 1e-6
    x, dy, w = rng.standard_normal((m, h, d)), rng.standard_normal((m, h, d)), rng.uniform(0.5, 1.5, d)
    pos = np.array([0, 7, 131071])
    xt, wt = torch.tensor(x, requires_grad=True), torch.tensor(w, requires_grad=True)
    y = torch.nn.functional.rms_norm(xt, (d,), wt, eps) if norm else xt + 0 * wt
    ang = torch.tensor(pos, dtype=torch.float64)[:, None] * theta ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
    z = torch.complex(y[..., :d // 2], y[..., d // 2:]) * torch.polar(torch.ones_like(ang), ang)[:, None]
    out = torch.cat((z.real, z.imag), -1)
    np.testing.assert_allclose(K.qk_norm_rope(x, w, pos, theta, eps, norm), out.detach().numpy(), atol=1e-9)
    out.backward(torch.tensor(dy))
    dx, dw = K.qk_norm_rope_backward(x, w, pos, theta, eps, dy, norm)
    np.testing.assert_allclose(dx, xt.grad.numpy(), atol=1e-9)
    np.testing.assert_allclose(dw, wt.grad.numpy(), atol=1e-9)
    f = lambda x_, w_: float(np.sum(K.qk_norm_rope(x_, w_, pos, theta, eps, norm) * dy))
    for at in [(0, 0, 3), (1, 1, d - 1), (2, 0, d // 2)]:
        e = np.zeros_like(x)
        e[at] = 1e-6
        assert (f(x + e, w) - f(x - e, w)) / 2e-6 == pytest.approx(dx[at], rel=1e-5, abs=1e-6)
    e = np.zeros(d)
    e[5] = 1e-6
    assert (f(x, w + e) - f(x, w - e)) / 2e-6 == pytest.approx(dw[5], rel=1e-5, abs=1e-6)


def test_round_bf16_is_torchs():
    rng = np.random.default_rng(0)
    a = (rng.standard_normal(5000) * 10.0 ** rng.uniform(-38, 38, 5000)).astype(np.float32)
    a = np.concatenate([a, np.float32([0, 1e-40, 9.2e-41, 1e-45, 257 / 256, 259 / 256])])
    np.testing.assert_array_equal(K.round_bf16(a), synth.round_to(a, "bf16").astype(np.float64))


def test_quantize_against_brute_force_over_all_levels():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((40, 64)).astype(np.float32) * 10.0 ** rng.uniform(-3, 3, (40, 1))
    val, scale, code = K.kv4_quantize(synth.round_to(x.astype(np.float32), "bf16"))
    x = synth.round_to(x.astype(np.float32), "bf16").astype(np.float64)
    signed = np.concatenate([K.LEVELS, -K.LEVELS])
    for r, g in itertools.product(range(40), range(2)):
        grp, s = x[r, 32 * g:32 * g + 32], scale[r, g]
        assert s == synth.round_to(np.float32([np.abs(grp).max() / 6]), "bf16")[0]
        best = np.abs(grp[:, None] - signed * s).min(1)
        np.testing.assert_allclose(np.abs(val[r, 32 * g:32 * g + 32] - grp), best, rtol=1e-9, atol=0)
        np.testing.assert_array_equal(signed[code[r, 32 * g:32 * g + 32]] * s, val[r, 32 * g:32 * g + 32])


def test_quantize_ties_and_special_groups():
    # scale 1 (largest magnitude 6): every border goes to the even code
    x = np.zeros(32)
    x[:8] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5]
    x[8:15] = -x[1:8]
    val, scale, code = K.kv4_quantize(x)
    assert scale[0] == 1
    np.testing.assert_array_equal(code[:15], [7, 0, 2, 2, 4, 4, 6, 6, 8, 10, 10, 12, 12, 14, 14])
    for bad in (np.inf, -np.inf, np.nan):
        x[20] = bad
        val, scale, code = K.kv4_quantize(x)
        assert np.isnan(val).all() and np.isnan(scale[0]) and not code.any()
    val, scale, code = K.kv4_quantize(np.zeros(32))
    assert not val.any() and scale[0] == 0 and not code.any()


@pytest.mark.parametrize("d", [64, 128])
def test_pack_puts_every_nibble_in_one_place(d):
    for row in range(5):
        seen = np.zeros(d, int)
        for i in range(d):
            c = np.zeros(d, int)
            c[i] = 15
            b = K.kv4_pack(c, row)
            (at,) = np.nonzero(b)
            assert len(at) == 1 and b[at[0]] in (15, 240)
            seen[2 * at[0] + (b[at[0]] == 240)] += 1
        assert (seen == 1).all()
    # the units a decode lane needs are neighbours: dimensions 4r .. 4r+3 of every group
    c = np.arange(d) // 4 % 16
    b = K.kv4_pack(c, 0)
    for r in range(8):
        part = b[2 * r * (d // 32):2 * (r + 1) * (d // 32)]
        units = [(int(x) & 15) for x in part]
        assert units == [v % 16 for g in range(d // 32) for v in (8 * g + r, 8 * g + r)]


def test_decode_attention_masks_and_empty_requests():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((4, 64)), rng.standard_normal((6, 2, 64)), rng.standard_normal((6, 2, 64))
    bias = rng.standard_normal(6)
    bias[[1, 4]] = -np.inf
    k[1] = np.nan
    v[4] = np.inf
    gain, temp = rng.uniform(0.5, 2, 4), rng.uniform(0.8, 1.2, 4)
    out, lse = K.kv4_decode_attention(q, k, v, bias, gain, temp, 0.9, 0.125)
    keep = [0, 2, 3, 5]
    for h in range(4):
        x = temp[h] * 0.9 * 0.125 * (k[keep, h // 2] @ q[h]) + gain[h] * bias[keep]
        p = np.exp(x - x.max())
        np.testing.assert_allclose(out[h], p / p.sum() @ v[keep, h // 2], rtol=1e-12)
        assert lse[h] == pytest.approx(math.log(np.exp(x).sum()), rel=1e-12)
    out, lse = K.kv4_decode_attention(q, k, v, np.full(6, -np.inf), gain, temp, 0.9, 0.125)
    assert not out.any() and np.isneginf(lse).all()
    out, lse = K.kv4_decode_attention(q, k[:0], v[:0], None, gain, temp, 0.9, 0.125)
    assert not out.any() and np.isneginf(lse).all()


def test_page_tables_by_hand():
    # pages of 4; request 0 holds 5 rows (pages 7, 2), request 1 3 rows (page 9), request 2 none
    tables = np.full((3, 3), -1)
    tables[0, :2], tables[1, 0] = [7, 2], 9
    free = np.array([4, 5, 6, -1, -1])
    got = K.page_tables([5, 3, 0], [2, 3, 1], None, 4, tables, free, 3, 8)
    lens, tab, fr, top, slots, start = got
    assert lens == [7, 6, 1] and top == 1 and start == [0, 2, 5, 6]
    assert slots == [2 * 4 + 1, 2 * 4 + 2, 9 * 4 + 3, 6 * 4, 6 * 4 + 1, 5 * 4, -1, -1]
    assert tab[1, 1] == 6 and tab[2, 0] == 5 and (tables[1, 1], tables[2, 0]) == (-1, -1)
    # request 0 done: pages 7, 2 go back and are taken from the top
    lens, tab, fr, top, slots, start = K.page_tables([5, 3, 0], [0, 2, 5], [1, 0, 0], 4, tables, free, 3, 7)
    assert lens == [0, 5, 5] and list(fr[:5]) == [4, 5, 6, 7, 2] and top == 2
    assert tab[1, 1] == 2 and list(tab[2, :2]) == [7, 6]
    assert K.page_tables([5, 3, 0], [0, 2, 16], None, 4, tables, free, 3, 99) is None    # past the table
    assert K.page_tables([5, 3, 0], [0, 6, 5], None, 4, tables, free, 3, 10) is None     # slots too short
    assert K.page_tables([5, 3, 0], [0, 6, 9], None, 4, tables, free, 3, 99) is None     # five pages wanted, three free


# ------------------------------------------------------------------ refusals on the host
P = ctypes.c_void_p(256)  # non-null and aligned: validation fails before it is dereferenced
OFF = ctypes.c_void_p(260)


def _cache(**kw):
    d = dict(k_codes=256, v_codes=256, k_scales=256, v_scales=256, bias=256, num_pages=10, page_rows=16, hkv=8,
             head_dim=128)
    d.update(kw)
    return ctypes.byref(tg.KV4CacheStruct(**d))


def test_page_tables_validation(L):
    f = L.tg_page_tables

    def call(lens=P, new=P, rel=None, nreq=4, page=16, tab=P, mp=8, free=P, cap=32, nf=P, lo=P, nfo=P, slots=P, ns=4, rs=P):
        return f(lens, new, rel, nreq, page, tab, mp, free, cap, nf, lo, nfo, slots, ns, rs, None)

    assert call(lens=None) == 1 and call(new=None) == 1 and call(tab=None) == 1 and call(lo=None) == 1
    assert call(nf=None) == 1 and call(nfo=None) == 1 and call(rs=None) == 1 and call(slots=None) == 1
    assert call(free=None) == 1
    assert call(nreq=-1) == 1 and call(page=0) == 1 and call(mp=0) == 1 and call(cap=-1) == 1 and call(ns=-1) == 1
    assert call(nreq=4097) == 4
    assert call(page=1 << 20, mp=1 << 11) == 4 and call(page=1 << 15, mp=(1 << 15) + 1) == 4
    assert call(ns=(1 << 30) + 1) == 4


def test_qk_rope_validation(L):
    f, b = L.tg_qk_norm_rope, L.tg_qk_norm_rope_backward

    def call(q=P, ldq=2048, k=P, ldk=1024, dt=1, m=10, hq=16, hkv=8, d=128, pos=P, eps=1e-6, theta=1e6, qo=P, ldqo=2048,
             ko=P, ldko=1024):
        return f(q, ldq, k, ldk, dt, m, hq, hkv, d, pos, P, P, 1, eps, theta, qo, ldqo, ko, ldko, None)

    assert call(q=None) == 1 and call(k=None) == 1 and call(qo=None) == 1 and call(ko=None) == 1 and call(pos=None) == 1
    assert call(m=-1) == 1 and call(hq=0) == 1 and call(hkv=0) == 1 and call(dt=5) == 1
    assert call(eps=-1.0) == 1 and call(eps=math.nan) == 1 and call(theta=0.0) == 1 and call(theta=math.inf) == 1
    assert call(d=96) == 4 and call(m=1 << 31) == 4
    assert call(ldq=2047) == 2 and call(ldko=1000) == 2
    assert call(q=OFF, qo=P) == 3 and call(ldk=1028) == 3
    assert call(ldqo=4096) == 2                               # in place with another leading dimension
    assert call(m=0) == 0                                     # nothing to do

    def back(m=10, ws=P, wsb=1 << 20, dq=P, dk=P, dwq=P, dwk=P, norm=1, dqi=P, lddq=2048, d=128):
        return b(P, 2048, P, 1024, 1, m, 16, 8, d, P, P, P, norm, 1e-6, 1e6, dq, dk, dqi, lddq, P, 1024, dwq, dwk, ws, wsb,
                 None)

    assert back(dq=None) == 1 and back(dk=None) == 1 and back(dqi=None) == 1
    assert back(dq=OFF) == 3 and back(ws=OFF) == 3
    need = tg.qk_rope_backward_workspace_bytes(10, 128)
    assert need > 0 and back(wsb=need - 1) == 5 and back(ws=None) == 5
    assert back(d=32) == 4 and back(lddq=100) == 2
    assert tg.qk_rope_backward_workspace_bytes(0, 128) == 0 and tg.qk_rope_backward_workspace_bytes(5, 96) == 0


def test_kv4_rows_validation(L):
    for f in (lambda c, k=P, ldk=1024, v=P, ldv=1024, dt=1, n=5, s=P: L.tg_kv4_store(c, k, ldk, v, ldv, dt, n, None, s, None),
              lambda c, k=P, ldk=1024, v=P, ldv=1024, dt=1, n=5, s=P: L.tg_kv4_load(c, s, n, k, ldk, v, ldv, dt, None, None)):
        assert f(None) == 1 and f(_cache(k_codes=None)) == 1 and f(_cache(v_scales=None)) == 1
        assert f(_cache(num_pages=0)) == 1 and f(_cache(hkv=0)) == 1
        for page in (0, 8, 48, 256):
            assert f(_cache(page_rows=page)) == 1
        assert f(_cache(head_dim=96)) == 4 and f(_cache(num_pages=1 << 27)) == 4
        assert f(_cache(v_codes=264)) == 3 and f(_cache(bias=260)) == 3
        c = _cache()
        assert f(c, k=None) == 1 and f(c, v=None) == 1 and f(c, s=None) == 1 and f(c, dt=2) == 1 and f(c, n=-1) == 1
        assert f(c, ldk=1000) == 2 and f(c, ldv=1023) == 2
        assert f(c, k=OFF) == 3 and f(c, ldv=1028) == 3
        assert f(c, n=1 << 31) == 4
        assert f(c, n=0) == 0


def test_kv4_decode_validation(L):
    f = L.tg_kv4_decode_attention
    ws_need = tg.kv4_decode_workspace_bytes(16, 8, 128)
    assert ws_need > 0
    assert tg.kv4_decode_workspace_bytes(16, 6, 128) == 0 and tg.kv4_decode_workspace_bytes(16, 1, 128) == 0
    assert tg.kv4_decode_workspace_bytes(16, 8, 96) == 0

    def call(c=None, q=P, ldq=2048, dt=1, tab=P, mp=4, lens=P, nreq=3, hq=16, gain=P, temp=P, out=P, ldo=2048, ws=P,
             wsb=1 << 30, flags=0):
        return f(c or _cache(), q, ldq, dt, tab, mp, lens, nreq, hq, gain, temp, None, 0.1, out, ldo, None, ws, wsb, flags,
                 None)

    assert call(q=None) == 1 and call(out=None) == 1 and call(tab=None) == 1 and call(lens=None) == 1
    assert call(gain=None) == 1 and call(temp=None) == 1
    assert call(flags=2) == 1 and call(dt=3) == 1 and call(nreq=-1) == 1 and call(mp=0) == 1
    assert call(hq=12) == 1                                   # not a multiple of the KV heads
    assert call(hq=72, ldq=9216, ldo=9216) == 4               # nine query heads per KV head
    assert call(nreq=4097) == 4 and call(mp=1 << 28) == 4 and call(mp=(1 << 26) + 1) == 4
    assert call(nreq=4096, mp=1 << 20) == 4                   # more work than 32 bits count
    assert call(c=_cache(page_rows=20)) == 1 and call(c=_cache(head_dim=32)) == 4
    assert call(ldq=2040) == 2 and call(ldo=100) == 2
    assert call(q=OFF) == 3 and call(ws=OFF) == 3 and call(ldo=2052) == 3
    assert call(ws=None) == 5 and call(wsb=ws_need - 1) == 5
    assert call(nreq=0) == 0


def test_binding_refuses_what_the_library_cannot_see(L):
    z = torch.zeros
    i32 = torch.int32
    with pytest.raises(tg.TokenGateError):   # CPU tensors
        tg.KV4Cache(z(2, 2, 16, 64, dtype=torch.uint8), z(2, 2, 16, 64, dtype=torch.uint8),
                    z(2, 2, 16, 4, dtype=torch.bfloat16), z(2, 2, 16, 4, dtype=torch.bfloat16))
    with pytest.raises(tg.TokenGateError):
        tg.tg_page_tables(z(3, dtype=i32), z(3, dtype=i32), None, 16, z(3, 4, dtype=i32), z(9, dtype=i32), z(1, dtype=i32),
                          z(3, dtype=i32), z(1, dtype=i32), z(3, dtype=i32), z(4, dtype=i32))
    with pytest.raises(tg.TokenGateError):   # one table row too few
        tg.tg_page_tables(z(3, dtype=i32), z(3, dtype=i32), None, 16, z(2, 4, dtype=i32), z(9, dtype=i32), z(1, dtype=i32),
                          z(3, dtype=i32), z(1, dtype=i32), z(3, dtype=i32), z(4, dtype=i32))
    with pytest.raises(tg.TokenGateError):   # half a head
        tg.tg_qk_norm_rope(z(3, 96), z(3, 64), 64, z(3, dtype=i32), None, None, 1e-6, 1e6, z(3, 96), z(3, 64))
