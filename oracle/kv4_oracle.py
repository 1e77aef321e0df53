"""CPU oracle of the paged 4-bit cache operators and of the q/k norm + rotation
with its gradients -- TEST INFRASTRUCTURE, float64 numpy and plain Python loops.
Shares no code with the CUDA path.  Pins: tests/test_oracle_kv4.py.
"""
from __future__ import annotations

from typing import Optional

import numpy as np

from .tokengate_oracle import gated_decode_attention, rms_norm, rope

F64 = np.float64
LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def page_tables(lens, new_rows, release, page_rows, tables, free_pages, n_free, nslots):
    """One call of the page-table builder on copies: (lens, tables, free_pages, n_free, slots, row_start), or None
    where the call has to be refused."""
    lens, new = [int(x) for x in lens], [int(x) for x in new_rows]
    tables, free = np.array(tables), np.array(free_pages)
    most = tables.shape[1] * page_rows
    pages = lambda n: -(-n // page_rows)
    top = int(n_free)
    if any(x < 0 or x > most for x in lens) or any(x < 0 for x in new) or top < 0:
        return None
    back = []
    for r, n in enumerate(lens):
        if release is not None and release[r]:
            back += list(tables[r, :pages(n)])
            lens[r] = 0
    if top + len(back) > len(free):
        return None
    free[top:top + len(back)] = back
    top += len(back)
    if any(n + a > most for n, a in zip(lens, new)) or sum(new) > nslots:
        return None
    if sum(pages(n + a) - pages(n) for n, a in zip(lens, new)) > top:
        return None
    slots, start = [], [0]
    for r, add in enumerate(new):
        for t in range(add):
            at = lens[r] + t
            if at % page_rows == 0:
                top -= 1
                tables[r, at // page_rows] = free[top]
            slots.append(int(tables[r, at // page_rows]) * page_rows + at % page_rows)
        start.append(len(slots))
        lens[r] += add
    slots += [-1] * (nslots - len(slots))
    return lens, tables, free, top, slots, start


def qk_norm_rope(x, w: Optional[np.ndarray], pos, theta: float, eps: float, norm: bool = True) -> np.ndarray:
    """x [m, heads, D]: per-head RMSNorm (optional), then rotate-half rotation."""
    x = np.asarray(x, F64)
    return rope(rms_norm(x, w, eps) if norm else x, np.asarray(pos), theta)


def qk_norm_rope_backward(x, w: Optional[np.ndarray], pos, theta: float, eps: float, dy, norm: bool = True):
    """Gradients (dx, dw) for upstream dy; dw is zero without the norm."""
    x, dy = np.asarray(x, F64), np.asarray(dy, F64)
    g = rope(dy, -np.asarray(pos, F64), theta)   # the rotation's transpose is the rotation back
    if not norm:
        return g, np.zeros(x.shape[-1])
    w = np.ones(x.shape[-1]) if w is None else np.asarray(w, F64)
    r = 1.0 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    dw = np.sum(g * x * r, axis=tuple(range(x.ndim - 1)))
    dx = r * g * w - x * r ** 3 * np.mean(g * w * x, -1, keepdims=True)
    return dx, dw


def round_bf16(a) -> np.ndarray:
    """float64 -> nearest bf16 (ties to even), as float64; finite input in bf16's normal and subnormal range."""
    a = np.asarray(a, F64)
    m, e = np.frexp(a)
    step = np.ldexp(1.0, np.maximum(e - 8, -133))
    return np.rint(a / step) * step


def kv4_quantize(x):
    """x [..., D] -> (values the 4-bit row stands for, scales [..., D/32], codes 0..15 [..., D])."""
    x = np.asarray(x, F64)
    y = x.reshape(x.shape[:-1] + (x.shape[-1] // 32, 32))
    finite = np.isfinite(y).all(-1)
    z = np.where(finite[..., None], y, 0.0)
    scale = round_bf16(np.abs(z).max(-1) / 6.0)
    s = np.where(scale > 0, scale, 1.0)[..., None]
    ratio = np.abs(z) / s
    dist = np.abs(ratio[..., None] - LEVELS) + np.where(np.arange(8) % 2 == 1, 1e-12, 0.0)  # a tie goes to the even code
    code = np.argmin(dist, -1)
    code = np.where(scale[..., None] > 0, code, 0)
    val = np.where(np.signbit(z), -1.0, 1.0) * LEVELS[code] * scale[..., None]
    val = np.where(finite[..., None], val, np.nan)
    scale = np.where(finite, scale, np.nan)
    code = np.where(finite[..., None] & (scale[..., None] > 0), code + 8 * np.signbit(z), 0)
    return val.reshape(x.shape), scale, code.reshape(x.shape)


def kv4_pack(codes, row: int) -> np.ndarray:
    """Codes [D] of page row `row` -> its D / 2 stored bytes."""
    d = len(codes)
    out = np.zeros(d // 2, np.uint8)
    for i, c in enumerate(codes):
        g, r, j = i // 32, i % 32 // 4, i % 4
        b = 2 * (r * (d // 32) + g) + j // 2
        if d == 128 and row % 4 >= 2:
            b ^= 32
        out[b] |= int(c) << (4 * (j % 2))
    return out


def kv4_decode_attention(q, k, v, bias, head_gain, head_temp, ratio: float, sm_scale: float):
    """One request: q [hq, D], k/v [length, hkv, D] (values), bias [length] or None.  Keys with bias -inf are left
    out; returns (out, lse), zeros and -inf where no key is left."""
    length = k.shape[0]
    keep = np.ones(length, bool) if bias is None else ~np.isneginf(np.asarray(bias, F64))
    hq, d = q.shape
    if not keep.any():
        return np.zeros((hq, d)), np.full(hq, -np.inf)
    return gated_decode_attention(q, k[keep], v[keep], None if bias is None else np.asarray(bias)[keep], head_gain,
                                  head_temp, ratio, sm_scale, return_lse=True)
