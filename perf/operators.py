"""The paged 4-bit KV cache operators and the query/key norm + rotation, as measured work.

Operators (entry points of learned_token_pruning_b200.tokengate):
  tables   tg_page_tables: page tables and slot maps built on the device from request lengths
  rotate   tg_qk_norm_rope: per-head RMSNorm of q and k and the position rotation in one pass
  rotate_b tg_qk_norm_rope_backward: its gradients (inputs and both norm weights)
  store    tg_kv4_store, then tg_kv4_load: rows into the 4-bit cache, and the values it stands for
  attend   tg_kv4_decode_attention: one new token per request over its 4-bit cache

run() computes them in plain torch operations, or with `own` set through the library.

The 4-bit cache: a row of a KV head holds head_dim E2M1 codes (sign, 2 exponent bits, 1 mantissa
bit: 0, .5, 1, 1.5, 2, 3, 4, 6) and one bf16 scale for each 32 dimensions.  Byte b of the row's
natural order holds dimension 2b in its low half and 2b + 1 in its high half; the two bytes of
dimensions 32g + 4r .. 32g + 4r + 3 are stored as the 16-bit unit r * (head_dim / 32) + g.  With
head_dim 128, rows 2 and 3 of every four rows of a page hold their two halves swapped.
"""
import math
import random

import torch

own = False

DEV = "cuda"
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
MIDS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)   # halfway between neighbouring levels
THETA, EPS = 1.0e6, 1.0e-6
WS_BYTES = 8 << 20                                 # scratch a program keeps for these calls

HEADS = {"16/8x128": (16, 8, 128), "4/2x64": (4, 2, 64), "6/2x64": (6, 2, 64), "8/1x128": (8, 1, 128),
         "4/4x128": (4, 4, 128), "10/2x128": (10, 2, 128)}


def listed():
    return [
        # one new token for each of a batch of running requests, a few of them just finished
        {"name": "tables, a decode step", "op": "tables", "nreq": 64, "page": 64, "len": 8321, "new": 1, "done": 8},
        # a wave of prompts admitted at once, pages of 16 rows
        {"name": "tables, prompts admitted", "op": "tables", "nreq": 1000, "page": 16, "len": 0, "new": 261, "done": 0},
        # the new tokens of a small batch, between the projections and attention
        {"name": "rotate, a decode step", "op": "rotate", "m": 16, "heads": "16/8x128", "dtype": "bf16", "norm": True},
        # the kept rows of the 128K-token prompt
        {"name": "rotate, kept rows of 128K", "op": "rotate", "m": 8256, "heads": "16/8x128", "dtype": "bf16", "norm": True},
        # training on the kept rows of the 16K-token prompt, after the attention backward
        {"name": "rotate backward, 16K", "op": "rotate_b", "m": 2064, "heads": "16/8x128", "dtype": "bf16", "norm": True},
        # full precision, small heads, an odd number of rows
        {"name": "rotate backward, fp32", "op": "rotate_b", "m": 501, "heads": "4/2x64", "dtype": "f32", "norm": True},
        # the kept rows of one prompt enter the cache
        {"name": "store, kept rows of 128K", "op": "store", "rows": 8256, "heads": "16/8x128", "page": 64, "dtype": "bf16"},
        # a decode step's new rows, fp32 activations
        {"name": "store, a decode step", "op": "store", "rows": 33, "heads": "6/2x64", "page": 16, "dtype": "f32"},
        # one request over the kept rows of the 16K-token prompt and its generated ones: latency
        {"name": "attend, one request, 16K", "op": "attend", "nreq": 1, "len": 2129, "heads": "16/8x128", "page": 64, "dtype": "bf16"},
        # a ragged batch, requests of up to the 128K-token prompt's kept rows
        {"name": "attend, ragged batch", "op": "attend", "nreq": 33, "len": 8321, "heads": "16/8x128", "page": 16, "dtype": "bf16"},
        # the unpruned cache of the 128K-token prompt
        {"name": "attend, unpruned 128K", "op": "attend", "nreq": 1, "len": 131137, "heads": "16/8x128", "page": 128, "dtype": "bf16"},
        # full precision queries, small heads, an odd group, lengths off the page size
        {"name": "attend, fp32", "op": "attend", "nreq": 5, "len": 997, "heads": "6/2x64", "page": 32, "dtype": "f32"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(("tables", "rotate", "rotate_b", "store", "attend", "attend"))
    page = rng.choice((16, 32, 64, 128))
    heads = rng.choice(sorted(HEADS))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op == "tables":
        nreq = _log(rng, 1, 1000)
        step = rng.random() < 0.5
        return {"op": op, "nreq": nreq, "page": page, "len": _log(rng, 1, 8321) if step else 0,
                "new": 1 if step else _log(rng, 2, 261), "done": rng.randrange(0, nreq // 4 + 1) if step else 0}
    if op in ("rotate", "rotate_b"):
        return {"op": op, "m": _log(rng, 1, 8256 if op == "rotate" else 4160), "heads": heads, "dtype": dtype,
                "norm": rng.random() < 0.8}
    if op == "store":
        return {"op": op, "rows": _log(rng, 1, 8256), "heads": heads, "page": page, "dtype": dtype}
    nreq = _log(rng, 1, 64)
    return {"op": op, "nreq": nreq, "len": _log(rng, 1, 131137 // nreq), "heads": heads, "page": page, "dtype": dtype}


# ------------------------------------------------------------------------------------------ sizes
def _lengths(case):
    """Rows each request already has: the first the longest, the others spread below it, one of a larger batch empty."""
    n, top = case["nreq"], case["len"]
    r = random.Random(n * 1000003 + top)
    v = [top] + [r.randint(min(1, top), top) for _ in range(n - 1)]
    if n >= 8:
        v[n // 2] = 0
    return v


def _new_rows(case):
    n, new = case["nreq"], case["new"]
    r = random.Random(n * 7919 + new)
    # the requests that have finished (the first ones) get no more rows
    return [0 if i < case["done"] else new if new == 1 else r.randint(0, new) for i in range(n)]


def _pages(rows, page):
    return -(-rows // page)


def work(case):
    op = case["op"]
    if op == "tables":
        lens, new = _lengths(case), _new_rows(case)
        kept = [0 if i < case["done"] else x for i, x in enumerate(lens)]
        back = sum(_pages(x, case["page"]) for x in lens[:case["done"]])
        taken = sum(_pages(a + b, case["page"]) - _pages(a, case["page"]) for a, b in zip(kept, new))
        # lengths, new rows and flags in; lengths, row starts, slots out; pages moved between list and tables
        return {"bytes": 17 * case["nreq"] + 4 * sum(new) + 8 * (back + taken) + 12, "flops": 0}
    hq, hkv, d = HEADS[case["heads"]]
    if op == "attend":
        rows, e = sum(_lengths(case)), 2 if case["dtype"] == "bf16" else 4
        row = 2 * hkv * (d // 2 + d // 32 * 2) + 4        # K and V codes and scales, the key's bias
        return {"bytes": rows * row + case["nreq"] * hq * (2 * d * e + 4), "flops": 4 * rows * hq * d}
    e = 2 if case["dtype"] == "bf16" else 4
    if op == "store":
        n = case["rows"] * hkv * d * 2                   # K and V values
        cache = n // 2 + n // 16
        return {"bytes": n * e + 2 * cache + n * 4 + case["rows"] * 16, "flops": 3 * n}
    n = case["m"] * (hq + hkv) * d
    if op == "rotate":
        return {"bytes": 2 * n * e + case["m"] * 4, "flops": 8 * n}
    return {"bytes": 2 * n * e + 4 * n + case["m"] * 4, "flops": 16 * n}


# ----------------------------------------------------------------------------------------- inputs
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    normal = lambda *s: torch.randn(*s, generator=g, device=DEV)
    uniform = lambda lo, hi, n: torch.rand(n, generator=g, device=DEV) * (hi - lo) + lo
    op = case["op"]
    s = {"op": op, "ws": torch.zeros(WS_BYTES, dtype=torch.uint8, device=DEV)}
    if op == "tables":
        lens, new, page = _lengths(case), _new_rows(case), case["page"]
        most = max(_pages(a + b, page) for a, b in zip(lens, new)) + 1
        held = [_pages(x, page) for x in lens]
        total = sum(held) + sum(_pages(b, page) + 1 for b in new) + 5
        order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
        tables = torch.full((case["nreq"], most), -1, dtype=torch.int32, device=DEV)
        col = torch.arange(most, device=DEV)
        mine = col < _ints(held)[:, None]
        tables[mine] = order[:sum(held)]
        n_free = total - sum(held)
        free = torch.full((total,), -1, dtype=torch.int32, device=DEV)
        free[:n_free] = order[sum(held):]
        done = torch.zeros(case["nreq"], dtype=torch.uint8, device=DEV)
        done[:case["done"]] = 1
        s.update(page=page, lens=_ints(lens), new=_ints(new), done=done, tables=tables, free=free,
                 n_free=_ints([n_free]), nslots=sum(new) + 3)
        s.update(lens_out=torch.empty_like(s["lens"]), n_free_out=torch.empty_like(s["n_free"]),
                 slots=torch.empty(s["nslots"], dtype=torch.int32, device=DEV),
                 row_start=torch.empty(case["nreq"] + 1, dtype=torch.int32, device=DEV))
        return s
    hq, hkv, d = HEADS[case["heads"]]
    dt = _dtype(case)
    s.update(hq=hq, hkv=hkv, d=d, dt=dt)
    if op in ("rotate", "rotate_b"):
        m = case["m"]
        qkv = normal(m, (hq + 2 * hkv) * d).to(dt)        # the fused projection's output
        # original positions of kept rows of a prompt eight times as long
        pos = torch.randperm(8 * m + 64, generator=g, device=DEV)[:m].sort().values.to(torch.int32)
        s.update(q=qkv[:, :hq * d], k=qkv[:, hq * d:(hq + hkv) * d], pos=pos, norm=case["norm"],
                 wq=uniform(0.5, 1.5, d), wk=uniform(0.5, 1.5, d))
        if op == "rotate":
            s.update(q_out=torch.empty(m, hq * d, dtype=dt, device=DEV), k_out=torch.empty(m, hkv * d, dtype=dt, device=DEV))
        else:
            s.update(dq=normal(m, hq * d), dk=normal(m, hkv * d) * 2, dq_in=torch.empty(m, hq * d, dtype=dt, device=DEV),
                     dk_in=torch.empty(m, hkv * d, dtype=dt, device=DEV),
                     dwq=torch.empty(d, device=DEV), dwk=torch.empty(d, device=DEV))
        return s
    page = case["page"]
    if op == "store":
        n = case["rows"]
        npages = _pages(n, page) + 2
        kv = normal(n, 2 * hkv * d) * (0.25 + 2 * torch.rand(2 * hkv * d, generator=g, device=DEV))  # channels of unlike size
        kv = kv.to(dt)
        s.update(k=kv[:, :hkv * d], v=kv[:, hkv * d:], bias=normal(n),
                 slots=torch.randperm(npages * page, generator=g, device=DEV)[:n].to(torch.int32))
        s.update(_pools(npages, page, hkv, d))
        s.update(k_back=torch.empty(n, hkv * d, device=DEV), v_back=torch.empty(n, hkv * d, device=DEV),
                 bias_back=torch.empty(n, device=DEV))
        return s
    lens = _lengths(case)
    held = [_pages(x, page) for x in lens]
    most, npages = max(held + [1]) + 1, sum(held) + 2
    tables = torch.full((case["nreq"], most), -1, dtype=torch.int32, device=DEV)
    tables[torch.arange(most, device=DEV) < _ints(held)[:, None]] = \
        torch.randperm(npages, generator=g, device=DEV)[:sum(held)].to(torch.int32)
    s.update(_pools(npages, page, hkv, d))
    channel = 0.25 + 2 * torch.rand(2, hkv, 1, d, generator=g, device=DEV)
    for i, what in enumerate(("k", "v")):
        x = (normal(npages, hkv, page, d) * channel[i]).to(torch.bfloat16)
        scale, code = _quantize(x.float())
        s[what + "_codes"].copy_(_pack(code))
        s[what + "_scales"].copy_(scale)
        del x, scale, code
    s["bias_pool"].copy_(normal(npages, page))
    s.update(lens=_ints(lens), tables=tables, q=normal(case["nreq"], hq * d).to(dt), gain=uniform(0.5, 2, hq),
             temp=uniform(0.8, 1.2, hq), ratio=uniform(0.6, 1, case["nreq"]), scale=1 / math.sqrt(d),
             out=torch.empty(case["nreq"], hq * d, dtype=dt, device=DEV), lse=torch.empty(case["nreq"], hq, device=DEV))
    return s


def _pools(npages, page, hkv, d):
    u8 = lambda: torch.zeros(npages, hkv, page, d // 2, dtype=torch.uint8, device=DEV)
    sc = lambda: torch.zeros(npages, hkv, page, d // 32, dtype=torch.bfloat16, device=DEV)
    return {"k_codes": u8(), "v_codes": u8(), "k_scales": sc(), "v_scales": sc(),
            "bias_pool": torch.zeros(npages, page, device=DEV)}


# ------------------------------------------------------------------------------------- plain forms
def _quantize(x):
    """fp32 [..., d] -> bf16 scales [..., d / 32] and codes 0 .. 15 [..., d]: scale = max / 6, codes by nearest, ties to even."""
    y = x.unflatten(-1, (-1, 32))
    scale = (y.abs().amax(-1) / 6).to(torch.bfloat16)
    s = scale.float()[..., None]
    a = y.abs()
    code = torch.zeros(y.shape, dtype=torch.uint8, device=x.device)
    for i, m in enumerate(MIDS):   # the border above code i; a value on it goes to the even one
        code += (a > m * s) if i % 2 == 0 else (a >= m * s)
    code = torch.where(s > 0, code, 0) + (y < 0).to(torch.uint8) * 8
    return scale, code.flatten(-2)


def _swap(b):
    """Swaps the halves of rows 2 and 3 of every four, where a row is 64 bytes."""
    if b.shape[-1] != 64:
        return b
    odd = torch.arange(b.shape[-2], device=b.device)[:, None] & 2
    return torch.where(odd > 0, b.roll(32, -1), b)


def _pack(code):
    """Codes [..., page rows, d] -> bytes [..., page rows, d / 2] in the cache's order."""
    b = code[..., 0::2] | (code[..., 1::2] << 4)
    return _swap(b.unflatten(-1, (-1, 8, 2)).transpose(-3, -2).flatten(-3))


def _level(code):
    return torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=code.device)[code.int()]


def _values(codes, scales):
    """What the rows of whole pages stand for, fp32 [..., page rows, d]."""
    b = _swap(codes).unflatten(-1, (8, -1, 2)).transpose(-3, -2).flatten(-3)
    v = _level(torch.stack((b & 15, b >> 4), -1).flatten(-2))
    return (v.unflatten(-1, (-1, 32)) * scales.float()[..., None]).flatten(-2)


def _angles(pos, d):
    inv = THETA ** (-torch.arange(0, d, 2, dtype=torch.float64, device=pos.device) / d)
    a = pos.double()[:, None] * inv
    return a.cos().float()[:, None], a.sin().float()[:, None]


def _plain_tables(s):
    page, lens, new, nreq = s["page"], s["lens"].long(), s["new"].long(), s["lens"].numel()
    done, tables, free = s["done"].bool(), s["tables"].clone(), s["free"].clone()
    col = torch.arange(tables.shape[1], device=DEV)
    held = (lens + page - 1) // page
    back = tables[(col < held[:, None]) & done[:, None]]                   # by request, then by page
    n_free = s["n_free"].long()
    free[n_free + torch.arange(back.numel(), device=DEV)] = back
    n_free = n_free + back.numel()
    lens = torch.where(done, 0, lens)
    held = (lens + page - 1) // page
    after = (lens + new + page - 1) // page
    fresh = (col >= held[:, None]) & (col < after[:, None])
    taken = free[n_free - 1 - torch.arange(int(fresh.sum()), device=DEV)]
    tables[fresh] = taken
    start = torch.zeros(nreq + 1, dtype=torch.long, device=DEV)
    start[1:] = new.cumsum(0)
    rows = torch.arange(s["nslots"], device=DEV)
    r = torch.searchsorted(start, rows, right=True) - 1
    real = rows < start[-1]
    r = torch.where(real, r, 0)
    at = torch.where(real, lens[r] + rows - start[r], 0)
    slots = torch.where(real, tables[r, at // page].long() * page + at % page, -1)
    i32 = torch.int32
    return {"tables": tables, "free": free, "n_free": (n_free - taken.numel()).to(i32), "lens": (lens + new).to(i32),
            "slots": slots.to(i32), "row_start": start.to(i32)}


def _plain_rotate(x, heads, d, pos, w, norm):
    y = x.float().unflatten(-1, (heads, d))
    if norm:
        y = y * (y.square().mean(-1, keepdim=True) + EPS).rsqrt() * w
    c, sn = _angles(pos, d)
    a, b = y[..., :d // 2], y[..., d // 2:]
    return torch.cat((a * c - b * sn, b * c + a * sn), -1).flatten(-2)


def _plain_rotate_b(x, heads, d, pos, w, norm, dy):
    x = x.float().unflatten(-1, (heads, d))
    c, sn = _angles(pos, d)
    dy = dy.unflatten(-1, (heads, d))
    a, b = dy[..., :d // 2], dy[..., d // 2:]
    g = torch.cat((a * c + b * sn, b * c - a * sn), -1)
    if not norm:
        return g.flatten(-2), torch.zeros(d, device=DEV)
    r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    dw = (g * x * r).double().sum((0, 1)).float()
    g = g * w
    return (r * g - x * r.pow(3) * (g * x).mean(-1, keepdim=True)).flatten(-2), dw


def _plain_attend(s):
    nreq, page, hkv, d = s["lens"].numel(), s["k_codes"].shape[2], s["hkv"], s["d"]
    group = s["hq"] // hkv
    at = s["tables"].clamp(min=0).long()
    rows = at.shape[1] * page
    take = lambda c, sc: _values(c[at], sc[at]).transpose(2, 3).reshape(nreq, rows, hkv, d)
    q = s["q"].float().reshape(nreq, hkv, group, d)
    x = torch.einsum("rhgd,rlhd->rhgl", q, take(s["k_codes"], s["k_scales"]))
    x = x * s["temp"].reshape(hkv, group, 1) * (s["ratio"] * s["scale"])[:, None, None, None]
    bias = s["bias_pool"][at].reshape(nreq, 1, 1, rows)
    x = x + s["gain"].reshape(hkv, group, 1) * bias
    live = torch.arange(rows, device=DEV) < s["lens"][:, None]
    x = torch.where(live[:, None, None], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = (x - torch.where(top == -math.inf, 0.0, top)).exp()
    total = p.sum(-1, keepdim=True)
    v = torch.where(live[..., None, None], take(s["v_codes"], s["v_scales"]), 0.0)
    o = torch.einsum("rhgl,rlhd->rhgd", p, v) / torch.where(total > 0, total, 1.0)
    lse = (top + total.log()).reshape(nreq, -1)
    return {"out": o.reshape(nreq, -1).to(s["dt"]), "lse": torch.where(total.reshape(nreq, -1) > 0, lse, -math.inf)}


def _cache(s):
    """The library's handle of the state's cache, made once as a program would."""
    if "cache" not in s:
        from learned_token_pruning_b200 import tokengate as tg
        s["cache"] = tg.KV4Cache(s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"], s["bias_pool"])
    return s["cache"]


def run(s):
    op = s["op"]
    if own:
        from learned_token_pruning_b200 import tokengate as tg
    if op == "tables":
        if own:
            tg.tg_page_tables(s["lens"], s["new"], s["done"], s["page"], s["tables"], s["free"], s["n_free"], s["lens_out"],
                              s["n_free_out"], s["slots"], s["row_start"])
            return {"tables": s["tables"], "free": s["free"], "n_free": s["n_free_out"], "lens": s["lens_out"],
                    "slots": s["slots"], "row_start": s["row_start"]}
        return _plain_tables(s)
    hq, hkv, d = s["hq"], s["hkv"], s["d"]
    if op == "rotate":
        if own:
            tg.tg_qk_norm_rope(s["q"], s["k"], d, s["pos"], s["wq"], s["wk"], EPS, THETA, s["q_out"], s["k_out"], qk_norm=s["norm"])
            return {"q": s["q_out"], "k": s["k_out"]}
        return {"q": _plain_rotate(s["q"], hq, d, s["pos"], s["wq"], s["norm"]).to(s["dt"]),
                "k": _plain_rotate(s["k"], hkv, d, s["pos"], s["wk"], s["norm"]).to(s["dt"])}
    if op == "rotate_b":
        if own:
            tg.tg_qk_norm_rope_backward(s["q"], s["k"], d, s["pos"], s["wq"], s["wk"], EPS, THETA, s["dq"], s["dk"], s["dq_in"],
                                        s["dk_in"], s["ws"], dw_q=s["dwq"], dw_k=s["dwk"], qk_norm=s["norm"])
            return {"dq": s["dq_in"], "dk": s["dk_in"], "dwq": s["dwq"], "dwk": s["dwk"]}
        dq, dwq = _plain_rotate_b(s["q"], hq, d, s["pos"], s["wq"], s["norm"], s["dq"])
        dk, dwk = _plain_rotate_b(s["k"], hkv, d, s["pos"], s["wk"], s["norm"], s["dk"])
        return {"dq": dq.to(s["dt"]), "dk": dk.to(s["dt"]), "dwq": dwq, "dwk": dwk}
    if op == "store":
        if own:
            tg.tg_kv4_store(_cache(s), s["k"], s["v"], s["bias"], s["slots"])
            tg.tg_kv4_load(_cache(s), s["slots"], s["k_back"], s["v_back"], s["bias_back"])
            return {"k": s["k_back"], "v": s["v_back"], "bias": s["bias_back"]}
        back = {}
        for what in ("k", "v"):
            scale, code = _quantize(s[what].float())
            back[what] = (_level(code).unflatten(-1, (-1, 32)) * scale.float()[..., None]).flatten(-2)
        return {**back, "bias": s["bias"].clone()}
    if own:
        tg.tg_kv4_decode_attention(_cache(s), s["q"], s["tables"], s["lens"], s["gain"], s["temp"], s["ratio"], s["scale"],
                                   s["out"], s["ws"], s["lse"], flags=tg.TG_WS_KEPT_ZERO)
        return {"out": s["out"], "lse": s["lse"]}
    return _plain_attend(s)


# ------------------------------------------------------------------------------------- in 64 bits
def _near(x):
    """Values that the 4-bit row stands for, by the distance to every level (ties to the even code)."""
    y = x.double().unflatten(-1, (-1, 32))
    scale = (y.abs().amax(-1, keepdim=True) / 6).float().to(torch.bfloat16).double()
    level = torch.tensor(LEVELS, dtype=torch.float64, device=x.device)
    odd = torch.arange(8, device=x.device) % 2 * 1e-12
    ratio = y.abs() / torch.where(scale > 0, scale, 1.0)
    best = torch.stack([(ratio - level[i]).abs() + odd[i] for i in range(8)], -1).argmin(-1)
    return (level[best] * y.sign() * scale).flatten(-2)


def _row_values(codes, scales):
    """Pages [..., page rows, d / 2] unpacked dimension by dimension, in 64 bits."""
    d = codes.shape[-1] * 2
    dim = torch.arange(d, device=codes.device)
    g, r, j = dim // 32, dim % 32 // 4, dim % 4
    byte = (r * (d // 32) + g) * 2 + j // 2
    row = torch.arange(codes.shape[-2], device=codes.device)[:, None]
    at = torch.where(row % 4 >= 2, byte ^ 32, byte) if d == 128 else byte.expand(row.numel(), d)
    c = codes.long().gather(-1, at.expand(*codes.shape[:-1], d)) >> (4 * (dim % 2)) & 15
    e, m = c >> 1 & 3, c & 1
    v = torch.where(e > 0, (1 + 0.5 * m) * torch.pow(2.0, (e - 1).double()), 0.5 * m.double())
    return v * (1 - 2 * (c >> 3)).double() * scales.double().index_select(-1, g)


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op == "tables":
        return None
    hq, hkv, d = HEADS[case["heads"]]
    if op == "store":
        return {"k": _near(s["k"]), "v": _near(s["v"]), "bias": s["bias"].double()}
    if op == "attend":
        outs, lses = [], []
        for r, n in enumerate(_lengths(case)):
            at = s["tables"][r, :_pages(n, case["page"])].long()
            out, lse = [], []
            for h in range(hq):
                kv = h // (hq // hkv)
                k = _row_values(s["k_codes"][at, kv], s["k_scales"][at, kv]).reshape(-1, d)[:n]
                v = _row_values(s["v_codes"][at, kv], s["v_scales"][at, kv]).reshape(-1, d)[:n]
                q = s["q"][r, h * d:(h + 1) * d].double()
                x = (k @ q) * s["temp"][h].double() * s["ratio"][r].double() * s["scale"] \
                    + s["gain"][h].double() * s["bias_pool"][at].reshape(-1)[:n].double()
                z = torch.logsumexp(x, 0) if n else torch.tensor(-math.inf, dtype=torch.float64, device=DEV)
                out.append((x - z).exp() @ v if n else torch.zeros(d, dtype=torch.float64, device=DEV))
                lse.append(z)
            outs.append(torch.cat(out))
            lses.append(torch.stack(lse))
        return {"out": torch.stack(outs), "lse": torch.stack(lses)}
    # the norm and the rotation as a complex product, gradients by automatic differentiation
    freq = torch.exp(torch.arange(d // 2, dtype=torch.float64, device=DEV) * (-2 * math.log(THETA) / d))
    turn = torch.polar(torch.ones(case["m"], d // 2, dtype=torch.float64, device=DEV), s["pos"].double()[:, None] * freq)[:, None]

    def one(x, w, heads):
        y = x.reshape(-1, heads, d)
        if case["norm"]:
            y = w * y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / d + EPS)
        z = torch.complex(y[..., :d // 2], y[..., d // 2:]) * turn
        return torch.cat((z.real, z.imag), -1).flatten(1)

    found = {}
    for what, heads in (("q", hq), ("k", hkv)):
        x = s[what].double().clone().requires_grad_(True)
        w = s["w" + what].double().requires_grad_(True)
        y = one(x, w, heads)
        if op == "rotate":
            found[what] = y.detach()
            continue
        y.backward(s["d" + what].double())
        found["d" + what] = x.grad
        found["dw" + what] = w.grad if w.grad is not None else torch.zeros_like(w)
    return found
