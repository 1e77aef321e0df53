"""A batch of requests decoded over the paged 4-bit cache: every step's page tables, rotated rows, stored rows and
attention together, through pipeline.PagedDecodeBatch, against the float64 oracle on the same inputs."""
import numpy as np
import pytest
import torch

from learned_token_pruning_b200 import pipeline, synth, tokengate as tg
from oracle import kv4_oracle as K

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Model:
    """The oracle's side of a batch: what every request's cache stands for."""

    def __init__(self, nreq, hkv, d):
        self.k, self.v = [[np.zeros((0, hkv, d))] * nreq for _ in range(2)]
        self.bias = [np.zeros(0, np.float32)] * nreq
        self.k, self.v = list(self.k), list(self.v)

    def add(self, r, k, v, bias):
        self.k[r] = np.concatenate([self.k[r], K.kv4_quantize(k)[0]])
        self.v[r] = np.concatenate([self.v[r], K.kv4_quantize(v)[0]])
        self.bias[r] = np.concatenate([self.bias[r], bias])

    def drop(self, r):
        self.k[r], self.v[r], self.bias[r] = self.k[r][:0], self.v[r][:0], self.bias[r][:0]


@pytest.mark.parametrize("hq,hkv,d,page,dtype", [(16, 8, 128, 16, "bf16"), (6, 2, 64, 32, "f32")])
@pytest.mark.parametrize("graph", [False, True])
def test_a_batch_decodes_as_the_oracle_does(hq, hkv, d, page, dtype, graph):
    rng = np.random.default_rng(hq)
    nreq, dt = 4, synth.torch_dtype(dtype)
    dev = lambda a, t=None: torch.from_numpy(np.ascontiguousarray(a)).to(DEV, t)
    gain, temp = rng.uniform(0.5, 2, hq).astype(np.float32), rng.uniform(0.8, 1.2, hq).astype(np.float32)
    wq, wk = rng.uniform(0.5, 1.5, d).astype(np.float32), rng.uniform(0.5, 1.5, d).astype(np.float32)
    b = pipeline.PagedDecodeBatch(nreq, 150, 40, page, hq=hq, hkv=hkv, head_dim=d, head_gain=dev(gain), head_temp=dev(temp),
                                  w_q_norm=dev(wq), w_k_norm=dev(wk), dtype=dt, device=DEV)
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
        b.admit(dev(np.array(rows, np.int32)), dev(k.reshape(n, -1), dt), dev(v.reshape(n, -1), dt), dev(bias),
                None if release is None else dev(np.array(release, np.uint8)))

    def step(check):
        qkv = synth.round_to(rng.standard_normal((nreq, hq + 2 * hkv, d)).astype(np.float32), dtype)
        pos = rng.integers(0, 131072, nreq).astype(np.int32)
        ratio = rng.uniform(0.6, 1, nreq).astype(np.float32)
        b.qkv.copy_(dev(qkv.reshape(nreq, -1)))
        b.pos.copy_(dev(pos))
        b.ratio.copy_(dev(ratio))
        out = b.replay() if graph else b.step()
        assert tg.tg_check_device_error() == 0
        # q and k as the kernel left them: against the oracle within its rounding, then taken as they are
        q, k = b.q.float().cpu().numpy().reshape(nreq, hq, d), b.k.float().cpu().numpy().reshape(nreq, hkv, d)
        half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
        for got, rows, w in ((q, qkv[:, :hq], wq), (k, qkv[:, hq:hq + hkv], wk)):
            want = K.qk_norm_rope(rows, w, pos, 1e6, 1e-6)
            flat = np.abs(K.rms_norm(rows, w, 1e-6))
            pair = flat[..., :d // 2] + flat[..., d // 2:]
            assert (np.abs(got - want) <= half * np.abs(want) + 2.0 ** -18 * np.concatenate([pair, pair], -1)).all()
        got = out.float().cpu().numpy().reshape(nreq, hq, d)
        for r in range(nreq):
            model.add(r, k[r:r + 1], qkv[r:r + 1, hq + hkv:], np.zeros(1, np.float32))
            if not check:
                continue
            args = (model.bias[r], gain, temp, float(ratio[r]), d ** -0.5)
            want, lse = K.kv4_decode_attention(q[r], model.k[r], model.v[r], *args)
            size, _ = K.kv4_decode_attention(q[r], model.k[r], np.abs(model.v[r]), *args)
            tol = half * np.abs(want) + (2.0 ** -10 if dtype == "bf16" else 1e-4) * size
            assert (np.abs(got[r] - want) <= tol).all(), r
            np.testing.assert_allclose(b.lse[r].cpu().numpy(), lse, rtol=1e-4, atol=1e-4)

    admit([37, 5, 70, 1])
    for i in range(20):          # pages fill up and new ones are taken
        step(check=i in (0, 11, 19))
    admit([0, 33, 0, 16], release=[0, 1, 0, 1])   # two requests done, two prompts in their place
    for i in range(6):
        step(check=i in (0, 5))
    assert b.lens.tolist() == [63, 39, 96, 22]
    held = sum(-(-n // page) for n in b.lens.tolist())
    assert int(b.n_free) == 40 - held


def test_a_step_without_free_pages_is_reported_and_leaves_the_lengths():
    b = pipeline.PagedDecodeBatch(2, 64, 2, 16, hq=4, hkv=2, head_dim=64, head_gain=torch.ones(4, device=DEV),
                                  head_temp=torch.ones(4, device=DEV), device=DEV)
    kv = torch.randn(32, 128, device=DEV, dtype=torch.bfloat16)
    b.admit(torch.tensor([16, 16], dtype=torch.int32, device=DEV), kv, kv, torch.zeros(32, device=DEV))
    assert tg.tg_check_device_error() == 0
    b.step()
    with pytest.raises(tg.TokenGateError) as e:
        tg.tg_check_device_error()
    assert e.value.status == 8 and b.lens.tolist() == [16, 16] and int(b.n_free) == 0
    assert (b.slots == -1).all()


def test_training_chain_attention_backward_into_the_norm_and_rotation():
    # gradients of the projection's q and k through gated attention and the norm + rotation: the two backward
    # calls in a row against the oracle's chain in 64 bits (fp32 path: 1e-4 of the largest gradient each)
    from oracle import tokengate_oracle as O
    m, hq, hkv, d = 65, 4, 2, 64
    rng = np.random.default_rng(5)
    x = rng.standard_normal((m, hq + hkv, d)).astype(np.float32)
    v, dout = rng.standard_normal((m, hkv, d)).astype(np.float32), rng.standard_normal((m, hq, d)).astype(np.float32)
    bias, ratio = rng.standard_normal(m).astype(np.float32), rng.uniform(0.6, 1, m).astype(np.float32)
    gain, temp = rng.uniform(0.5, 2, hq).astype(np.float32), rng.uniform(0.8, 1.2, hq).astype(np.float32)
    wq, wk = rng.uniform(0.5, 1.5, d).astype(np.float32), rng.uniform(0.5, 1.5, d).astype(np.float32)
    pos = np.sort(rng.integers(0, 16384, m)).astype(np.int32)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    flat = lambda a: dev(a.reshape(m, -1))
    qx, kx = flat(x[:, :hq]), flat(x[:, hq:])
    q, k = torch.empty_like(qx), torch.empty_like(kx)
    tg.tg_qk_norm_rope(qx, kx, d, dev(pos), dev(wq), dev(wk), 1e-6, 1e6, q, k)
    out, lse = torch.empty_like(q), torch.empty(hq, m, device=DEV)
    att = (dev(bias), dev(gain), dev(temp), dev(ratio), d ** -0.5)
    tg.tg_gated_attention(q, k, flat(v), d, *att, out, lse)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(k)
    ws = torch.empty(tg.attention_backward_workspace_bytes(m, hq, hkv, d), dtype=torch.uint8, device=DEV)
    tg.tg_gated_attention_backward(q, k, flat(v), out, flat(dout), d, *att, lse, dq, dk, dv, ws)
    dqx, dkx, dwq, dwk = torch.empty_like(q), torch.empty_like(k), torch.empty(d, device=DEV), torch.empty(d, device=DEV)
    ws = torch.empty(tg.qk_rope_backward_workspace_bytes(m, d), dtype=torch.uint8, device=DEV)
    tg.tg_qk_norm_rope_backward(qx, kx, d, dev(pos), dev(wq), dev(wk), 1e-6, 1e6, dq, dk, dqx, dkx, ws, dw_q=dwq, dw_k=dwk)
    assert tg.tg_check_device_error() == 0
    qo, ko = [K.qk_norm_rope(r, w, pos, 1e6, 1e-6) for r, w in ((x[:, :hq], wq), (x[:, hq:], wk))]
    g = O.gated_attention_backward(qo, ko, v, bias, gain, temp, ratio, d ** -0.5, dout)
    for dy, rows, w, got, gw in ((g["dq"], x[:, :hq], wq, dqx, dwq), (g["dk"], x[:, hq:], wk, dkx, dwk)):
        dx, dw = K.qk_norm_rope_backward(rows, w, pos, 1e6, 1e-6, dy)
        np.testing.assert_allclose(got.cpu().numpy().reshape(dx.shape), dx, atol=2e-4 * np.abs(dx).max(), rtol=0)
        np.testing.assert_allclose(gw.cpu().numpy(), dw, atol=2e-4 * np.abs(dw).max(), rtol=0)


def test_admission_on_a_side_stream_keeps_its_slots():
    # the slots' memory must not go to other work of the current stream before the side stream has used it
    n, hkv, d = 300, 2, 64
    ones = torch.ones(4, device=DEV)
    b = pipeline.PagedDecodeBatch(2, 400, 60, 16, hq=4, hkv=hkv, head_dim=d, head_gain=ones, head_temp=ones, device=DEV)
    k, v = [torch.randint(-6, 7, (n, hkv * d), device=DEV).to(torch.bfloat16) for _ in range(2)]
    k[:, ::32] = v[:, ::32] = 6            # scale 1: the stored values are the nearest codes
    new, bias = torch.tensor([n - 7, 7], dtype=torch.int32, device=DEV), torch.zeros(n, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)      # the side stream is behind
    b.admit(new, k, v, bias, stream=side)
    other = [torch.full((n,), -1, dtype=torch.int32, device=DEV) for _ in range(8)]
    torch.cuda.synchronize()
    assert tg.tg_check_device_error() == 0 and all((t == -1).all() for t in other)
    rows = torch.cat([torch.arange(n - 7), torch.arange(7)])
    tables = b.tables.cpu()
    slots = torch.cat([tables[0, rows[:n - 7] // 16], tables[1, rows[n - 7:] // 16]]) * 16 + rows % 16
    got = [torch.empty(n, hkv * d, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    tg.tg_kv4_load(b.cache, slots.to(torch.int32).to(DEV), *got)
    for t, x in zip(got, (k, v)):
        want = K.kv4_quantize(x.float().cpu().numpy().reshape(n, hkv, d))[0].reshape(n, -1)
        np.testing.assert_array_equal(t.float().cpu().numpy(), want)
