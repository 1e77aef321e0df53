"""Steps of a batch in which some requests take no part: slots by request, idle requests keep what they hold, the others go
on.  Against the float64 oracle; tolerances as in test_gpu_paged_batch.py."""
import numpy as np
import pytest
import torch

from learned_token_pruning_b200 import pipeline, synth, tokengate as tg
from oracle import kv4_oracle as K
from test_gpu_kv4 import DEV, I32, _dev, _i32
from test_gpu_paged_batch import Model

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------------ page tables by request
@pytest.mark.parametrize("nreq,page", [(1, 16), (7, 1), (64, 64), (1000, 16), (4096, 128), (33, 48)])
@pytest.mark.parametrize("in_place", [False, True])
def test_slots_by_request_are_the_packed_ones_in_their_places(nreq, page, in_place):
    rng = np.random.default_rng(nreq + page)
    lens = rng.integers(0, 3 * page + 1, nreq)
    new, rel = (rng.random(nreq) < 0.7).astype(np.int32), (rng.random(nreq) < 0.2).astype(np.uint8)
    held = -(-lens // page)
    total = int(held.sum()) + nreq + 2
    order = rng.permutation(total).astype(np.int32)
    tables = np.full((nreq, 5), -1, np.int32)
    at = 0
    for r in range(nreq):
        tables[r, :held[r]] = order[at:at + held[r]]
        at += held[r]
    free = np.full(total, -1, np.int32)
    free[:total - at] = order[at:]
    want = K.page_tables(lens, new, rel, page, tables, free, total - at, nreq)
    t = dict(lens=_i32(lens.tolist()), tables=_dev(tables), free=_dev(free), n_free=_i32([total - at]))
    lo, nfo = (t["lens"], t["n_free"]) if in_place else (torch.full((nreq,), 9, dtype=I32, device=DEV), _i32([9]))
    slots, start = torch.full((nreq,), 9, dtype=I32, device=DEV), torch.full((nreq + 1,), 9, dtype=I32, device=DEV)
    tg.tg_page_tables_by_request(t["lens"], _dev(new), _dev(rel), page, t["tables"], t["free"], t["n_free"], lo, nfo, slots,
                                 start if in_place else None)
    assert tg.tg_check_device_error() == 0
    wl, wt, wf, top, packed, ws = want
    assert lo.tolist() == wl and int(nfo) == top
    np.testing.assert_array_equal(t["tables"].cpu().numpy(), wt)
    np.testing.assert_array_equal(t["free"].cpu().numpy()[:top], wf[:top])
    assert slots.tolist() == [packed[ws[r]] if new[r] else -1 for r in range(nreq)]
    assert start.tolist() == (ws if in_place else [9] * (nreq + 1))


@pytest.mark.parametrize("new", [[1, 2, 0], [1, -1, 0], [1, 1, 1]])
def test_more_than_one_row_or_too_few_pages_are_refused(new):
    lens, tables, free, n_free = _i32([16, 3, 16]), _i32([[0, -1], [1, -1], [2, -1]]), _i32([3]), _i32([1])
    slots, start = torch.full((3,), 7, dtype=I32, device=DEV), torch.full((4,), 7, dtype=I32, device=DEV)
    tg.tg_page_tables_by_request(lens, _i32(new), None, 16, tables, free, n_free, lens, n_free, slots, start)
    with pytest.raises(tg.TokenGateError) as e:
        tg.tg_check_device_error()
    assert e.value.status == 8
    assert slots.tolist() == [-1] * 3 and start.tolist() == [0] * 4 and lens.tolist() == [16, 3, 16] and int(n_free) == 1


# ------------------------------------------------------------------------------------------------ steps
@pytest.mark.parametrize("hq,hkv,d,page,dtype", [(16, 8, 128, 16, "bf16"), (6, 2, 64, 32, "f32")])
@pytest.mark.parametrize("graph", [False, True])
def test_idle_requests_keep_their_rows_and_the_others_go_on(hq, hkv, d, page, dtype, graph):
    rng = np.random.default_rng(hq + 1)
    nreq, cap, dt = 5, 5 * page, synth.torch_dtype(dtype)
    gain, temp = rng.uniform(0.5, 2, hq).astype(np.float32), rng.uniform(0.8, 1.2, hq).astype(np.float32)
    wq, wk = rng.uniform(0.5, 1.5, d).astype(np.float32), rng.uniform(0.5, 1.5, d).astype(np.float32)
    b = pipeline.PagedDecodeBatch(nreq, cap, 30, page, hq=hq, hkv=hkv, head_dim=d, head_gain=_dev(gain), head_temp=_dev(temp),
                                  w_q_norm=_dev(wq), w_k_norm=_dev(wk), dtype=dt, device=DEV)
    model = Model(nreq, hkv, d)

    def admit(rows, release=None):
        n = sum(rows)
        k, v = [synth.round_to(rng.standard_normal((n, hkv, d)).astype(np.float32), dtype) for _ in range(2)]
        bias = rng.standard_normal(n).astype(np.float32)
        at = 0
        for r, m in enumerate(rows):
            if release is not None and release[r]:
                model.drop(r)
            model.add(r, k[at:at + m], v[at:at + m], bias[at:at + m])
            at += m
        b.admit(_i32(rows), _dev(k.reshape(n, -1), dt), _dev(v.reshape(n, -1), dt), _dev(bias),
                None if release is None else _dev(np.array(release, np.uint8)))

    def step(live, check=True):
        assert b.live.tolist() == live
        before = b.lens.tolist()
        qkv = synth.round_to(rng.standard_normal((nreq, hq + 2 * hkv, d)).astype(np.float32), dtype)
        b.qkv.copy_(_dev(qkv.reshape(nreq, -1)))
        b.pos.copy_(_i32(rng.integers(0, 131072, nreq).tolist()))
        out = b.replay() if graph else b.step()
        assert tg.tg_check_device_error() == 0
        assert b.lens.tolist() == [x + y for x, y in zip(before, live)]
        assert [s >= 0 for s in b.slots.tolist()] == [x == 1 for x in live]
        q, k = b.q.float().cpu().numpy().reshape(nreq, hq, d), b.k.float().cpu().numpy().reshape(nreq, hkv, d)
        got = out.float().cpu().numpy().reshape(nreq, hq, d)
        half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
        for r in range(nreq):
            if not live[r]:
                continue
            model.add(r, k[r:r + 1], qkv[r:r + 1, hq + hkv:], np.zeros(1, np.float32))
            if not check:
                continue
            args = (model.bias[r], gain, temp, 1.0, d ** -0.5)
            want, lse = K.kv4_decode_attention(q[r], model.k[r], model.v[r], *args)
            size, _ = K.kv4_decode_attention(q[r], model.k[r], np.abs(model.v[r]), *args)
            tol = half * np.abs(want) + (2.0 ** -10 if dtype == "bf16" else 1e-4) * size
            assert (np.abs(got[r] - want) <= tol).all(), r
            np.testing.assert_allclose(b.lse[r].cpu().numpy(), lse, rtol=1e-4, atol=1e-4)

    assert b.live.tolist() == [0] * 5
    admit([37, 5, cap, 1, 0])                # request 2 holds all it may, request 4 nothing
    b.live[2] = 0
    for i in range(3):
        step([1, 1, 0, 1, 0])
    b.live[1] = 0                            # one in the middle pauses
    for i in range(page + 2):                # past a page border of the others
        step([1, 0, 0, 1, 0], check=i in (0, page + 1))
    b.live[1] = 1
    b.live[0] = 0
    step([0, 1, 0, 1, 0])                    # its rows are as they were
    admit([0, 0, 9, 0, 12], release=[1, 0, 1, 0, 0])    # 0 ends, 2 gives its place to another prompt, 4 begins
    for i in range(2):
        step([0, 1, 1, 1, 1])
    assert int(b.n_free) == 30 - sum(-(-n // page) for n in b.lens.tolist())


def test_a_refused_admission_leaves_the_live_requests_as_they_were():
    b = pipeline.PagedDecodeBatch(3, 64, 3, 16, hq=4, hkv=2, head_dim=64, head_gain=torch.ones(4, device=DEV),
                                  head_temp=torch.ones(4, device=DEV), device=DEV)
    kv = torch.randn(100, 128, device=DEV, dtype=torch.bfloat16)
    b.admit(_i32([16, 0, 16]), kv[:32], kv[:32], torch.zeros(32, device=DEV))
    b.live[2] = 0
    assert tg.tg_check_device_error() == 0
    b.admit(_i32([0, 60, 30]), kv[:90], kv[:90], torch.zeros(90, device=DEV))
    with pytest.raises(tg.TokenGateError):
        tg.tg_check_device_error()
    assert b.live.tolist() == [1, 0, 0] and b.lens.tolist() == [16, 0, 16]


def test_capturing_a_full_batch_reports_nothing_and_changes_nothing():
    b = pipeline.PagedDecodeBatch(2, 32, 3, 16, hq=4, hkv=2, head_dim=64, head_gain=torch.ones(4, device=DEV),
                                  head_temp=torch.ones(4, device=DEV), device=DEV)
    kv = torch.randn(48, 128, device=DEV, dtype=torch.bfloat16)
    b.admit(torch.tensor([32, 16], dtype=torch.int32, device=DEV), kv, kv, torch.zeros(48, device=DEV))
    state = [t.clone() for t in (b.lens, b.tables, b.free_pages, b.n_free, b.qkv, b.cache.k_codes, b.cache.bias)]
    b.capture()
    assert tg.tg_check_device_error() == 0
    for t, old in zip((b.lens, b.tables, b.free_pages, b.n_free, b.qkv, b.cache.k_codes, b.cache.bias), state):
        assert torch.equal(t, old)
