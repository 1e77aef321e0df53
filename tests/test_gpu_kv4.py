"""The paged 4-bit cache on the GPU against the float64 oracle: page tables (exact), rows in and out (exact), decode
attention, and a run of all of them as a batch of requests is decoded.

Attention tolerances, per output dimension with A = sum_c softmax_c |v_c| (>= |out|): rounding the output, 2^-8 |out|
in bf16 (2^-24 in fp32); bf16: weights rounded to 11 bits, 2^-11 A, and as much again for the logits (fp32 sums of
D products, under 2^-12 for logits below 2^8) and the exponentials; fp32: 1e-4 A, the bound of the contiguous
decode's fp32 path (fp32 sums of up to 128 products of size 8 in the exponent are off by 128 * 8 * 2^-24 = 6e-5)."""
import math

import numpy as np
import pytest
import torch

from learned_token_pruning_b200 import synth, tokengate as tg
from oracle import kv4_oracle as K

pytestmark = pytest.mark.gpu
DEV = "cuda"
I32 = torch.int32


def _i32(v):
    return torch.tensor(v, dtype=I32, device=DEV)


def _dev(a, dt=None):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV, dt)


# ---------------------------------------------------------------------------------------------- page tables
def _tables_case(nreq, page, seed, top_len, new, done=0, spare=3):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, top_len + 1, nreq)
    add = rng.integers(0, new + 1, nreq)
    held = -(-lens // page)
    most = int((-(-(lens + add) // page)).max(initial=0)) + 1
    total = int(held.sum() + (-(-(lens + add) // page) - held).sum()) + spare
    order = rng.permutation(total).astype(np.int32)
    tables = np.full((nreq, most), -1, np.int32)
    at = 0
    for r in range(nreq):
        tables[r, :held[r]] = order[at:at + held[r]]
        at += held[r]
    free = np.full(total + 2, -1, np.int32)
    free[:total - at] = order[at:]
    rel = np.zeros(nreq, np.uint8)
    rel[rng.permutation(nreq)[:done]] = 1
    return lens.astype(np.int32), add.astype(np.int32), rel, tables, free, total - at, int(add.sum()) + 2


def _tables_call(case, page, release=True, in_place=False):
    lens, add, rel, tables, free, nf, ns = case
    n = len(lens)
    t = dict(lens=_i32(lens.tolist()), new=_i32(add.tolist()), rel=_dev(rel) if release else None, tables=_dev(tables),
             free=_dev(free), nf=_i32([nf]), slots=torch.full((ns,), 99, dtype=I32, device=DEV),
             start=torch.full((n + 1,), 99, dtype=I32, device=DEV))
    t["lo"], t["nfo"] = (t["lens"], t["nf"]) if in_place else (torch.full_like(t["lens"], 99), torch.full_like(t["nf"], 99))
    t["call"] = lambda: tg.tg_page_tables(t["lens"], t["new"], t["rel"], page, t["tables"], t["free"], t["nf"], t["lo"],
                                          t["nfo"], t["slots"], t["start"])
    return t


def _tables_same(t, want):
    lens, tables, free, top, slots, start = want
    for got, w in ((t["lo"], lens), (t["tables"], tables), (t["free"], free), (t["nfo"], [top]), (t["slots"], slots),
                   (t["start"], start)):
        np.testing.assert_array_equal(got.cpu().numpy(), np.array(w, np.int32).reshape(got.shape))


@pytest.mark.parametrize("nreq,page,top_len,new,done", [
    (1, 16, 0, 1, 0), (1, 16, 16, 1, 0), (3, 64, 200, 3, 1), (64, 64, 500, 1, 9), (33, 16, 100, 300, 33), (7, 7, 50, 20, 2),
    (700, 32, 64, 5, 100), (513, 16, 0, 261, 0), (4096, 128, 300, 2, 1000), (5, 16, 40, 0, 5), (2, 1, 9, 9, 1)])
@pytest.mark.parametrize("in_place", [False, True])
def test_page_tables(nreq, page, top_len, new, done, in_place):
    case = _tables_case(nreq, page, nreq + page, top_len, new, done)
    want = K.page_tables(case[0], case[1], case[2], page, case[3], case[4], case[5], case[6])
    t = _tables_call(case, page, in_place=in_place)
    t["call"]()
    assert tg.tg_check_device_error() == 0
    _tables_same(t, want)


@pytest.mark.parametrize("nreq,page,top_len,new,done", [(300, 16, 10, 150, 20), (1000, 16, 0, 261, 0), (1000, 64, 8321, 1, 30),
                                                        (60, 32, 5, 900, 7)])
def test_page_tables_slots_in_runs_of_several_lengths(nreq, page, top_len, new, done):
    test_page_tables(nreq, page, top_len, new, done, False)


def test_page_tables_without_a_release_vector_and_without_requests():
    case = _tables_case(9, 16, 1, 60, 4)
    t = _tables_call(case, 16, release=False)
    t["call"]()
    assert tg.tg_check_device_error() == 0
    _tables_same(t, K.page_tables(case[0], case[1], None, 16, *case[3:6], case[6]))
    none = (np.zeros(0, np.int32), np.zeros(0, np.int32), np.zeros(0, np.uint8), np.zeros((0, 4), np.int32),
            np.arange(3, dtype=np.int32), 3, 5)
    t = _tables_call(none, 16)
    t["call"]()
    assert tg.tg_check_device_error() == 0
    assert (t["slots"] == -1).all() and int(t["start"][0]) == 0 and int(t["nfo"]) == 3


@pytest.mark.parametrize("what", ["pages", "table", "slots", "negative length", "long length", "negative new", "free count",
                                  "free list"])
def test_page_tables_refuses_on_the_device_and_changes_nothing(what):
    page = 16
    lens, add, rel, tables, free, nf, ns = _tables_case(40, page, 2, 100, 9, done=3)
    if what == "pages":
        nf = 0
        rel[:] = 0
        add[:] = 20
        tables = np.concatenate([tables, np.full((40, 3), -1, np.int32)], 1)
        ns = 900
    elif what == "table":
        add[7] = 10000
        ns = 20000
    elif what == "slots":
        ns = int(add.sum()) - 1
    elif what == "negative length":
        lens[11] = -1
    elif what == "long length":
        lens[11] = tables.shape[1] * page + 1
    elif what == "negative new":
        add[39] = -2
    elif what == "free count":
        nf = -1
    else:
        nf = len(free) + 1
    assert K.page_tables(lens, add, rel, page, tables, free, nf, ns) is None
    t = _tables_call((lens, add, rel, tables, free, nf, ns), page)
    t["call"]()
    with pytest.raises(tg.TokenGateError) as e:
        tg.tg_check_device_error()
    assert e.value.status == 8
    assert (t["slots"] == -1).all() and (t["start"] == 0).all()
    np.testing.assert_array_equal(t["tables"].cpu().numpy(), tables)
    np.testing.assert_array_equal(t["free"].cpu().numpy(), free)
    np.testing.assert_array_equal(t["lo"].cpu().numpy(), lens)
    assert int(t["nfo"]) == nf
    assert tg.tg_check_device_error() == 0


def test_page_tables_follow_a_batch_through_a_replayed_graph():
    nreq, page, steps = 6, 16, 40
    tables = np.full((nreq, 5), -1, np.int32)
    free = np.arange(40, dtype=np.int32)[::-1].copy()
    lens, top = [0] * nreq, 40
    t = _tables_call((np.zeros(nreq, np.int32), np.ones(nreq, np.int32), np.zeros(nreq, np.uint8), tables, free, top, 40), page,
                     in_place=True)
    add, rel = t["new"], t["rel"]
    add.zero_()
    t["call"]()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t["call"]()
    rng = np.random.default_rng(4)
    for s in range(steps):
        n = rng.integers(0, 4, nreq)
        d = (rng.random(nreq) < 0.15) | (np.array(lens) > 60)
        add.copy_(_i32(n.tolist()))
        rel.copy_(_dev(d.astype(np.uint8)))
        want = K.page_tables(lens, n, d, page, tables, free, top, 40)
        graph.replay()
        assert tg.tg_check_device_error() == 0
        _tables_same(t, want)
        lens, tables, free, top = want[:4]
    del graph


# ---------------------------------------------------------------------------------------------- rows in and out
def _pool_rows(cache, slots):
    """(stored K bytes, K scales) of slots, on the host."""
    p = cache.page_rows
    return [(cache.k_codes[s // p, :, s % p].cpu().numpy(), cache.k_scales[s // p, :, s % p].float().cpu().numpy()) for s in slots]


@pytest.mark.parametrize("rows", [1, 5, 130])
@pytest.mark.parametrize("hkv,d,page", [(8, 128, 64), (2, 64, 16), (1, 128, 128), (3, 64, 32)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_store_and_load_are_exact(rows, hkv, d, page, dtype):
    rng = np.random.default_rng(rows + d)
    pages = -(-rows // page) + 2
    kv = (rng.standard_normal((2, rows, hkv, d)) * 10 ** rng.uniform(-2, 2, (2, 1, hkv, d))).astype(np.float32)
    # borders between codes: with 6 s present, multiples of s / 4 hit them exactly
    kv[0, 0, 0, :32] = np.float32(0.5) * np.r_[6, np.arange(31) * 0.25 - 3].astype(np.float32)
    kv[1, -1, -1, 32:64] = 0.0
    kv[0, -1, -1, 32:64] = np.float32(1e-40)
    kv = synth.round_to(kv, dtype)
    bias = rng.standard_normal(rows).astype(np.float32)
    slots = rng.permutation(pages * page)[:rows].astype(np.int32)
    cache = tg.KV4Cache.zeros(pages, page, hkv, d)
    dt = synth.torch_dtype(dtype)
    buf = _dev(np.concatenate([np.zeros((rows, 8 * hkv)), kv[0].reshape(rows, -1), kv[1].reshape(rows, -1)], 1), dt)
    w = hkv * d
    tg.tg_kv4_store(cache, buf[:, 8 * hkv:8 * hkv + w], buf[:, 8 * hkv + w:], _dev(bias), _dev(slots))
    val = [K.kv4_quantize(x) for x in kv]
    for (code, scale), r in list(zip(_pool_rows(cache, slots), range(rows)))[:7]:
        np.testing.assert_array_equal(scale, val[0][1][r])
        for h in range(hkv):
            np.testing.assert_array_equal(code[h], K.kv4_pack(val[0][2][r, h], slots[r] % page))
    for out in (torch.float32, torch.bfloat16):
        back = torch.full((rows, 2 * w + 8), 3.0, dtype=out, device=DEV)
        b = torch.empty(rows, device=DEV)
        tg.tg_kv4_load(cache, _dev(slots), back[:, :w], back[:, w:2 * w], b)
        want = np.concatenate([v[0].reshape(rows, -1) for v in val], 1)
        want = want if out == torch.float32 else synth.round_to(want.astype(np.float32), "bf16")
        np.testing.assert_array_equal(back[:, :2 * w].float().cpu().numpy(), want)
        assert (back[:, 2 * w:] == 3).all()
        np.testing.assert_array_equal(b.cpu().numpy(), bias)
    assert tg.tg_check_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("top", [6.0, 1.0, 5.34375, 0.0703125, 3.0e38, 7e-31, 3e-38, 2.0 ** -128])
def test_store_every_value_below_a_largest_one(dtype, top):
    # the bf16 values from top down over eight powers of two, their neighbours in fp32, and the borders
    # themselves: every code is the exact nearest, ties to even
    top = synth.round_to(np.float32([top]), "bf16")[0]
    bits = np.float32(top).view(np.uint32) >> 16
    x = (np.arange(bits, max(int(bits) - 8 * 128, 0), -1, dtype=np.uint32) << 16).view(np.float32)
    s = K.round_bf16(np.float64(top) / 6)
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]) * s
    x = np.concatenate([x, mids.astype(np.float32)])
    if dtype == "f32":
        x = np.concatenate([x, np.nextafter(x, np.float32(0)), np.nextafter(x, np.float32(np.inf))])
        x = x[x <= top]
    x = synth.round_to(x, dtype)
    n = -(-len(x) // 31)
    body = np.zeros(31 * n, np.float32)
    body[:len(x)] = x
    rows = np.concatenate([np.full((n, 1), top, np.float32), body.reshape(n, 31) * np.where(np.arange(31) % 3 == 0, -1, 1)], 1)
    rows = np.tile(rows.astype(np.float32), (1, 2))           # two groups of a head
    cache = tg.KV4Cache.zeros(-(-n // 16), 16, 1, 64)
    d = _dev(rows, synth.torch_dtype(dtype))
    slots = torch.arange(n, dtype=I32, device=DEV)
    tg.tg_kv4_store(cache, d, d, None, slots)
    k, v = torch.empty(n, 64, device=DEV), torch.empty(n, 64, device=DEV)
    tg.tg_kv4_load(cache, slots, k, v)
    want = K.kv4_quantize(rows)[0]
    np.testing.assert_array_equal(k.cpu().numpy(), want)
    np.testing.assert_array_equal(v.cpu().numpy(), want)


def test_store_non_finite_groups_read_back_as_nan_and_leave_their_neighbours():
    x = torch.randn(4, 128, device=DEV)
    x[0, 3], x[1, 40], x[2, 100] = math.inf, -math.inf, math.nan
    cache = tg.KV4Cache.zeros(1, 16, 1, 128, bias=False)
    slots = _i32([3, 2, 9, 4])
    tg.tg_kv4_store(cache, x, x, None, slots)
    k, v, b = torch.empty_like(x), torch.empty_like(x), torch.ones(4, device=DEV)
    tg.tg_kv4_load(cache, slots, k, v, b)
    want = K.kv4_quantize(x.cpu().numpy())[0]
    np.testing.assert_array_equal(k.cpu().numpy(), want)
    np.testing.assert_array_equal(v.cpu().numpy(), want)
    assert np.isnan(want).sum() == 96 and not b.any()      # a cache without biases gives zeros


def test_store_leaves_out_negative_slots_and_load_leaves_their_rows():
    cache = tg.KV4Cache.zeros(2, 16, 2, 64)
    x = torch.randn(5, 128, device=DEV, dtype=torch.bfloat16)
    slots = _i32([4, -1, 31, -7, 0])
    tg.tg_kv4_store(cache, x, x, None, slots)
    touched = (cache.k_codes != 0).any(-1).any(1).flatten().nonzero().flatten().tolist()
    assert touched == [0, 4, 31]
    k, v = torch.full_like(x, 5), torch.full_like(x, 5)
    tg.tg_kv4_load(cache, slots, k, v)
    assert (k[[1, 3]] == 5).all() and (v[[1, 3]] == 5).all() and not (k[[0, 2, 4]] == 5).any()
    assert tg.tg_check_device_error() == 0


def test_slots_past_the_cache_are_left_out_and_reported():
    cache = tg.KV4Cache.zeros(2, 16, 2, 64)
    x = torch.randn(3, 128, device=DEV)
    for slots in ([1, 32, 2], [1, 2 ** 31 - 1, 2]):
        tg.tg_kv4_store(cache, x, x, None, _i32(slots))
        with pytest.raises(tg.TokenGateError) as e:
            tg.tg_check_device_error()
        assert e.value.status == 8
        k, v = torch.full_like(x, 5), torch.full_like(x, 5)
        tg.tg_kv4_load(cache, _i32(slots), k, v)
        with pytest.raises(tg.TokenGateError):
            tg.tg_check_device_error()
        assert (k[1] == 5).all() and not (k[[0, 2]] == 5).any()


# ---------------------------------------------------------------------------------------------- decode attention
class Batch:
    """Requests of the given lengths in a cache with shuffled pages, garbage everywhere else."""

    def __init__(self, lens, hq, hkv, d, page, dtype, seed, bias=True, spread=0.0, extra_pages=1):
        rng = np.random.default_rng(seed)
        self.lens, self.hq, self.hkv, self.d, self.page, self.dtype = list(lens), hq, hkv, d, page, dtype
        held = [-(-n // page) for n in lens]
        pages = sum(held) + extra_pages
        order = rng.permutation(pages).astype(np.int32)
        most = max(held + [1])
        self.tables = np.full((len(lens), most), -9, np.int32)   # entries past a request are never read
        at = 0
        for r, n in enumerate(held):
            self.tables[r, :n] = order[at:at + n]
            at += n
        self.cache = tg.KV4Cache.zeros(pages, page, hkv, d, bias=bias)
        # rows of no request: codes of all ones, NaN scales, NaN biases
        for t in (self.cache.k_codes, self.cache.v_codes):
            t.fill_(0xFF)
        for t in (self.cache.k_scales, self.cache.v_scales):
            t.fill_(math.nan)
        if bias:
            self.cache.bias.fill_(math.nan)
        rows = sum(lens)
        self.k = synth.round_to((rng.standard_normal((rows, hkv, d)) * 2 ** rng.uniform(-spread, spread, (rows, hkv, 1))).astype(np.float32), "bf16")
        self.v = synth.round_to((rng.standard_normal((rows, hkv, d)) * 2 ** rng.uniform(-spread, spread, (rows, hkv, 1))).astype(np.float32), "bf16")
        self.bias = rng.standard_normal(rows).astype(np.float32) if bias else None
        self.slots = np.concatenate([self.tables[r, np.arange(n) // page] * page + np.arange(n) % page
                                     for r, n in enumerate(lens)] or [np.zeros(0)]).astype(np.int32)
        self.q = synth.round_to(rng.standard_normal((len(lens), hq * d)).astype(np.float32), dtype)
        self.gain, self.temp = rng.uniform(0.5, 2, hq).astype(np.float32), rng.uniform(0.8, 1.2, hq).astype(np.float32)
        self.ratio = rng.uniform(0.6, 1, len(lens)).astype(np.float32)
        self.scale = 1 / math.sqrt(d)
        self.store()
        self.ws = torch.full((tg.kv4_decode_workspace_bytes(hq, hkv, d),), 0xA5, dtype=torch.uint8, device=DEV)

    def store(self):
        n = sum(self.lens)
        w = self.hkv * self.d
        tg.tg_kv4_store(self.cache, _dev(self.k.reshape(n, w), torch.bfloat16), _dev(self.v.reshape(n, w), torch.bfloat16),
                        None if self.bias is None else _dev(self.bias), _dev(self.slots))

    def want(self, r):
        s = sum(self.lens[:r])
        sl = slice(s, s + self.lens[r])
        k, v = K.kv4_quantize(self.k[sl])[0], K.kv4_quantize(self.v[sl])[0]
        b = None if self.bias is None else self.bias[sl]
        q = self.q[r].reshape(self.hq, self.d)
        ratio = 1.0 if self.ratio is None else float(self.ratio[r])
        out, lse = K.kv4_decode_attention(q, k, v, b, self.gain, self.temp, ratio, self.scale)
        size, _ = K.kv4_decode_attention(q, k, np.abs(v), b, self.gain, self.temp, ratio, self.scale)
        return out, lse, size

    def run(self, out=None, lse=True, flags=0, q=None):
        dt = synth.torch_dtype(self.dtype)
        n = len(self.lens)
        out = torch.full((n, self.hq * self.d), 7.0, dtype=dt, device=DEV) if out is None else out
        ls = torch.full((n, self.hq), 7.0, device=DEV) if lse else None
        tg.tg_kv4_decode_attention(self.cache, _dev(self.q, dt) if q is None else q, _dev(self.tables), _i32(self.lens),
                                   _dev(self.gain), _dev(self.temp), None if self.ratio is None else _dev(self.ratio),
                                   self.scale, out, self.ws, ls, flags=flags)
        return out, ls

    def check(self, out, lse, only=None):
        got = out.float().cpu().numpy()
        half, slack = (2.0 ** -8, 2.0 ** -10) if self.dtype == "bf16" else (2.0 ** -24, 1e-4)
        for r in range(len(self.lens)) if only is None else only:
            want, wl, size = self.want(r)
            err = np.abs(got[r].reshape(want.shape) - want)
            tol = half * np.abs(want) + slack * size
            assert (err <= tol).all(), (r, self.lens[r], float((err / np.maximum(tol, 1e-30)).max()))
            if lse is not None:
                np.testing.assert_allclose(lse[r].cpu().numpy(), wl, rtol=1e-4, atol=1e-4)

    def go(self, only=None):
        out, lse = self.run()
        assert tg.tg_check_device_error() == 0
        self.check(out, lse, only)
        return out, lse


LENS = [1, 0, 15, 16, 17, 63, 64, 65, 2, 128, 129, 300, 0, 777]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("hq,hkv,d", [(16, 8, 128), (4, 2, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_ragged_batch(page, hq, hkv, d, dtype):
    Batch(LENS, hq, hkv, d, page, dtype, seed=page + d).go()


@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 128), (4, 4, 64), (6, 2, 64), (3, 1, 128), (8, 2, 128), (10, 2, 128), (6, 1, 64),
                                      (14, 2, 64), (8, 1, 128), (8, 1, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_head_groups(hq, hkv, d, dtype):
    Batch([517, 40, 1], hq, hkv, d, 32, dtype, seed=hq * 10 + d).go()


@pytest.mark.parametrize("length", [1, 64, 2129, 8321])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_one_request(length, dtype):
    Batch([length], 16, 8, 128, 64, dtype, seed=length).go()


@pytest.mark.parametrize("hq,hkv", [(16, 8), (8, 1)])
def test_attention_long_request_beside_short_ones(hq, hkv):
    Batch([3, 40001, 100], hq, hkv, 128, 128, "bf16", seed=8).go()


def test_attention_many_requests():
    b = Batch([(i * 37) % 83 for i in range(600)], 4, 2, 64, 16, "bf16", seed=9)
    b.go(only=range(0, 600, 13))


def test_attention_most_requests():
    b = Batch([i % 3 for i in range(4096)], 2, 1, 64, 16, "bf16", seed=10)
    b.go(only=list(range(0, 4096, 97)) + [4095])


def test_attention_no_requests_is_a_no_op():
    b = Batch([5], 4, 2, 64, 16, "bf16", seed=1)
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=DEV)
    tg.tg_kv4_decode_attention(b.cache, z(0, 256), torch.zeros(0, 3, dtype=I32, device=DEV), _i32([]), _dev(b.gain),
                               _dev(b.temp), None, 0.1, z(0, 256), b.ws)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_rows_of_unlike_size(dtype):
    # rows whose largest values span 2^20: the small ones' weights and values must not be lost to a common scale
    b = Batch([700, 90], 16, 8, 128, 16, dtype, seed=12, spread=10.0)
    b.k /= np.abs(b.k).max((1, 2), keepdims=True) / 3
    b.k = synth.round_to(b.k, "bf16")
    b.store()
    b.go()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_without_biases_and_ratios(dtype):
    b = Batch([130, 7], 16, 8, 128, 32, dtype, seed=13, bias=False)
    b.ratio = None
    b.go()


def test_attention_masked_keys_reach_nothing():
    # keys with bias -inf whose rows hold NaN, a request with every key masked, the type's lowest value as a mask
    b = Batch([200, 33, 70], 16, 8, 128, 16, "bf16", seed=14)
    rng = np.random.default_rng(1)
    off = rng.permutation(200)[:60]
    b.bias[off] = -np.inf
    b.k[off[:20]], b.v[off[20:40]] = np.nan, np.inf
    b.bias[200:233] = -np.inf
    b.k[200:210] = np.nan
    b.bias[240:300:3] = -3.4e38       # finite: such keys weigh nothing next to others
    b.bias[233:240] = -3.4e38
    b.store()
    out, lse = b.go()
    assert not out[1].any() and torch.isneginf(lse[1]).all()


def test_attention_every_key_at_the_lowest_finite_bias():
    # -3.4e38 for every key: softmax is over equal huge logits, which swallow the content term
    b = Batch([40], 4, 2, 64, 16, "bf16", seed=15)
    b.bias[:] = -1e38
    b.gain[:] = 1.0
    b.store()
    out, lse = b.run()
    v = K.kv4_quantize(b.v)[0]
    want = np.repeat(v.mean(0), 2, 0).reshape(-1)
    size = np.repeat(np.abs(v).mean(0), 2, 0).reshape(-1)
    assert (np.abs(out[0].float().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * size).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", [(16, 8, 128), (6, 2, 64), (8, 1, 128)])
def test_attention_every_key_at_the_types_lowest_value(hq, hkv, d, dtype):
    # gain * bias passes the largest float in base 2 (and for gains above 1 in any base): the logits
    # are equal all the same, and the output is the mean of the values
    b = Batch([130, 9], hq, hkv, d, 16, dtype, seed=40)
    b.bias[:] = np.finfo(np.float32).min
    b.gain[:] = np.linspace(0.5, 2.0, hq)
    b.store()
    out, lse = b.run()
    half, slack = (2.0 ** -8, 2.0 ** -10) if dtype == "bf16" else (2.0 ** -24, 1e-4)
    for r, rows in ((0, slice(0, 130)), (1, slice(130, 139))):
        v = np.repeat(K.kv4_quantize(b.v[rows])[0], hq // hkv, 1)
        err = np.abs(out[r].float().cpu().numpy().reshape(hq, d) - v.mean(0))
        assert (err <= half * np.abs(v.mean(0)) + slack * np.abs(v).mean(0)).all()
    assert torch.isfinite(lse).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_lowest_value_under_a_negative_gain_takes_all_the_weight(dtype):
    b = Batch([100], 4, 2, 64, 16, dtype, seed=41)
    b.gain[:] = [-1.0, 1.0, -2.0, 0.5]
    b.bias[:] = 0.0
    b.bias[30:40] = np.finfo(np.float32).min
    b.store()
    out, _ = b.run()
    v = np.repeat(K.kv4_quantize(b.v)[0][30:40], 2, 1)
    got = out[0].float().cpu().numpy().reshape(4, 64)
    for h in (0, 2):
        assert (np.abs(got[h] - v[:, h].mean(0)) <= 2.0 ** -8 * np.abs(v[:, h].mean(0)) + 2.0 ** -10 * np.abs(v[:, h]).mean(0)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", [(16, 8, 128), (6, 2, 64), (8, 1, 128), (3, 1, 128)])
@pytest.mark.parametrize("low", [-3.4e38, -300.0])
def test_attention_huge_values_behind_a_finite_mask_leave_the_others_exact(low, hq, hkv, d, dtype):
    # rows without weight must not set the unit that the others' weights are rounded in
    b = Batch([200, 31], hq, hkv, d, 16, dtype, seed=42)
    b.gain[:] = 1.0
    off = np.random.default_rng(2).permutation(231)[:40]
    b.bias[off] = low
    b.v[off] = synth.round_to(b.v[off] * np.float32(2.0 ** 90 if low < -1e38 else 2.0 ** 60), "bf16")
    b.store()
    b.go()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", [(16, 8, 128), (6, 2, 64), (10, 2, 128)])
def test_attention_whole_tiles_of_huge_values_behind_a_finite_mask(hq, hkv, d, dtype):
    b = Batch([1500, 700], hq, hkv, d, 32, dtype, seed=44)
    b.gain[:] = 1.0
    for s in (0, 640, 1500 + 128):
        b.bias[s:s + 192] = -250.0
        b.v[s:s + 192] = synth.round_to(b.v[s:s + 192] * np.float32(2.0 ** 50), "bf16")
    b.store()
    b.go()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_huge_values_whose_weight_a_later_key_takes(dtype):
    b = Batch([260, 500], 16, 8, 128, 64, dtype, seed=43)
    b.gain[:] = 1.0
    for s, n in ((0, 260), (260, 500)):
        b.v[s:s + 70] = synth.round_to(b.v[s:s + 70] * np.float32(2.0 ** 40), "bf16")
        b.bias[s + n - 60:s + n] += 120.0
    b.store()
    b.go()


def test_attention_nan_in_a_live_row_reaches_its_own_request_only():
    b = Batch([50, 60], 4, 2, 64, 16, "bf16", seed=16)
    b.v[7, 0, :32] = np.nan            # request 0, KV head 0, dimensions 0..31
    b.store()
    out, lse = b.run()
    got = out.float().reshape(2, 4, 64)
    assert got[0, :2, :32].isnan().all() and not got[0, :2, 32:].isnan().any() and not got[0, 2:].isnan().any()
    b.check(out, lse, only=[1])


def test_attention_strided_rows_and_rows_behind_the_batch():
    b = Batch([90, 0, 17], 16, 8, 128, 64, "bf16", seed=17)
    big = torch.full((5, 16 * 128 + 64), 3.0, dtype=torch.bfloat16, device=DEV)
    qbuf = torch.zeros(3, 16 * 128 + 512, dtype=torch.bfloat16, device=DEV)
    qbuf[:, 256:256 + 2048] = _dev(b.q, torch.bfloat16)
    out, lse = b.run(out=big[:3, 32:32 + 2048], q=qbuf[:, 256:256 + 2048])
    b.check(out, lse)
    assert (big[3:] == 3).all() and (big[:, :32] == 3).all() and (big[:, 32 + 2048:] == 3).all()


def test_attention_reruns_are_identical_and_the_workspace_is_reused():
    b = Batch([5000, 3, 801], 16, 8, 128, 64, "bf16", seed=18)
    c = Batch([1300], 4, 1, 64, 16, "f32", seed=19)
    first = b.run()
    c.ws = b.ws if b.ws.numel() >= c.ws.numel() else c.ws
    c.go()
    again = b.run()
    assert all(torch.equal(x, y) for x, y in zip(first, again))
    b.check(*again)
    # a workspace kept at zero: no memset, any number of calls, lengths changing in between
    b.ws = torch.zeros_like(b.ws)
    for cut in (5000, 100, 2500, 5000):
        b.lens[0] = cut
        out, lse = b.run(flags=tg.TG_WS_KEPT_ZERO)
    assert tg.tg_check_device_error() == 0
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


def test_attention_pages_shared_by_requests():
    # a common prefix: two requests name the same pages
    b = Batch([64, 64], 4, 2, 64, 16, "bf16", seed=20)
    b.tables[1, :3] = b.tables[0, :3]
    b.k[64:112], b.v[64:112], b.bias[64:112] = b.k[:48], b.v[:48], b.bias[:48]
    b.go()


@pytest.mark.parametrize("bad", ["page", "negative page", "length", "negative length"])
def test_attention_bad_pages_and_lengths_are_reported_and_stay_inside(bad):
    b = Batch([100, 40, 60], 4, 2, 64, 16, "bf16", seed=21)
    if bad == "page":
        b.tables[1, 1] = 2 ** 30
    elif bad == "negative page":
        b.tables[1, 0] = -1
    elif bad == "length":
        b.lens[1] = b.tables.shape[1] * 16 + 1
    else:
        b.lens[1] = -4
    out, lse = b.run()
    with pytest.raises(tg.TokenGateError) as e:
        tg.tg_check_device_error()
    assert e.value.status == 8
    if "length" in bad:
        assert not out[1].any() and torch.isneginf(lse[1]).all()
    b.lens[1] = 40
    b.check(out, lse, only=[0, 2])
    b.tables[1] = np.where(b.tables[1] < 0, -9, b.tables[1])
    assert tg.tg_check_device_error() == 0


def test_attention_on_a_side_stream_and_two_at_once():
    a, b = Batch([3000, 50], 16, 8, 128, 64, "bf16", seed=22), Batch([900, 900], 8, 1, 128, 16, "bf16", seed=23)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(s1):
            ra = a.run()
        with torch.cuda.stream(s2):
            rb = b.run()
    torch.cuda.synchronize()
    assert tg.tg_check_device_error() == 0
    a.check(*ra)
    b.check(*rb)


def test_attention_replayed_graph_follows_the_lengths():
    b = Batch([700, 20, 300], 16, 8, 128, 64, "bf16", seed=24)
    dt = torch.bfloat16
    q, tables, lens = _dev(b.q, dt), _dev(b.tables), _i32(b.lens)
    gain, temp, ratio = _dev(b.gain), _dev(b.temp), _dev(b.ratio)
    out, lse = torch.empty(3, 2048, dtype=dt, device=DEV), torch.empty(3, 16, device=DEV)
    other = torch.empty_like(out)
    call = lambda o: tg.tg_kv4_decode_attention(b.cache, q, tables, lens, gain, temp, ratio, b.scale, o, b.ws, lse)
    call(out)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]   # two graphs, one workspace, replayed in turn
    for g, o in zip(graphs, (out, other)):
        with torch.cuda.graph(g):
            call(o)
    full, k, v, bias = list(b.lens), b.k, b.v, b.bias
    for cut in ([700, 20, 300], [1, 0, 299], [513, 20, 64]):
        lens.copy_(_i32(cut))
        for g, o in zip(graphs, (out, other)):
            o.fill_(7)
            g.replay()
            torch.cuda.synchronize()
            keep = np.concatenate([np.arange(c) + s for c, s in zip(cut, np.cumsum([0] + full[:-1]))])
            b.lens, b.k, b.v, b.bias = cut, k[keep], v[keep], bias[keep]
            b.check(o, lse)
    assert tg.tg_check_device_error() == 0
    del graphs


def test_attention_cache_offsets_past_32_bits():
    # 66048 pages of 128 rows x 8 heads x 64 bytes: codes reach 4.3 GB; a request at the far end
    pages, page, hkv, d = 66048, 128, 8, 128
    cache = tg.KV4Cache.zeros(pages, page, hkv, d)
    b = Batch([300, 5], 16, hkv, d, page, "bf16", seed=25)
    used = sorted({int(x) for x in b.tables.flatten() if x >= 0})
    for name in ("k_codes", "v_codes", "k_scales", "v_scales", "bias"):
        getattr(cache, name)[pages - 20:] = getattr(b.cache, name)[0]
    for i, p in enumerate(used):
        b.tables[b.tables == p] = -100 - i
    for i in range(len(used)):
        b.tables[b.tables == -100 - i] = pages - 1 - i
    b.slots = np.concatenate([b.tables[r, np.arange(n) // page] * page + np.arange(n) % page
                              for r, n in enumerate(b.lens)]).astype(np.int32)
    b.cache = cache
    b.store()
    b.go()
    k, v = torch.empty(305, hkv * d, device=DEV), torch.empty(305, hkv * d, device=DEV)
    tg.tg_kv4_load(cache, _dev(b.slots), k, v)
    np.testing.assert_array_equal(k.cpu().numpy().reshape(b.k.shape), K.kv4_quantize(b.k)[0])


def test_attention_agrees_with_the_contiguous_decode_on_the_same_values():
    # the two decode paths on the values the 4-bit rows stand for (bf16 holds them up to half a step)
    b = Batch([1500], 16, 8, 128, 64, "bf16", seed=26)
    out, lse = b.go()
    k, v = [torch.empty(1500, 1024, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    tg.tg_kv4_load(b.cache, _dev(b.slots), k, v)
    other = torch.empty(16, 128, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(tg.decode_workspace_bytes(1500, 16, 8, 128), dtype=torch.uint8, device=DEV)
    tg.tg_gated_decode_attention(_dev(b.q, torch.bfloat16).reshape(16, 128), k, v, 128, _dev(b.bias), _dev(b.gain),
                                 _dev(b.temp), float(b.ratio[0]), b.scale, other, ws)
    np.testing.assert_allclose(out.float().cpu().numpy().reshape(16, 128), other.float().cpu().numpy(), atol=2e-2, rtol=1e-2)
