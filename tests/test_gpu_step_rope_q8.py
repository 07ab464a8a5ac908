"""AttentionStep with rotary positions and over an 8-bit cache: chunked prefill, decode and two streams, as served.

What a step stores is checked against the 64-bit definitions (bf16: half a step, 2^-8,
plus the fp32 rotation; 8 bits: at most one rounding when a value is stored and one per
growth of its block's scale, each half a step of at most 32 * 2^x, and the scales grow
once or twice here), its attention against the fp64 oracle on the stored values.
"""
import numpy as np
import pytest
import torch

import oracle
import workloads as W
from helpers import to_dev
from oracle import append as A
from q8_helpers import bf16_bits, close

pytestmark = pytest.mark.gpu


class Served:
    """Two to three requests that grow step by step over a shared pool of pages."""

    def __init__(self, cpsa, q8, rope, hq=8, hkv=2, d=128, P=16, n=3, most=400, two_stream=False, tokens=600):
        self.cpsa, self.q8, self.hq, self.hkv, self.d, self.P, self.n = cpsa, q8, hq, hkv, d, P, n
        rng = self.rng = np.random.default_rng(7)
        blocks = (most + P - 1) // P
        self.table = rng.permutation(n * blocks).reshape(n, blocks).astype(np.int32)
        kind = torch.float8_e4m3fn if q8 else torch.bfloat16
        raw = torch.uint8 if q8 else torch.int16
        self.kc = torch.full((n * blocks, hkv, P, d), 0x7F if q8 else 0x7FC0, dtype=raw, device="cuda").view(kind)
        self.vc = self.kc.clone()
        self.scales = {}
        if q8:
            sc = torch.full((n * blocks, hkv, P // min(16, P)), 255, dtype=torch.uint8, device="cuda")
            self.scales = dict(k_scale=sc, v_scale=sc.clone())
        self.rope = cpsa.rope_table(most, 64, device="cuda") if rope else None
        self.step = cpsa.AttentionStep(n, tokens, hq, hkv, d, max_kv_splits=4, two_stream=two_stream, kv_dtype=kind,
                                       rope=self.rope, length_threshold=16, balance_threshold=1.0)
        self.len = [0] * n
        self.k = [np.zeros((0, hkv, d)) for _ in range(n)]
        self.v = [np.zeros((0, hkv, d)) for _ in range(n)]

    def inputs(self, qlen):
        T = sum(qlen)
        qkv = torch.from_numpy(self.rng.standard_normal((T, (self.hq + 2 * self.hkv) * self.d)).astype(np.float32))
        qkv = qkv.to(torch.bfloat16).cuda()
        cut = [self.hq * self.d, (self.hq + self.hkv) * self.d]
        q, k, v = (x.unflatten(1, (-1, self.d)) for x in (qkv[:, :cut[0]], qkv[:, cut[0]:cut[1]], qkv[:, cut[1]:]))
        if self.rope is None:
            q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        pos = np.concatenate([np.arange(n, n + c) for n, c in zip(self.len, qlen)]).astype(np.int64)
        req = np.repeat(np.arange(self.n), qlen)
        slots = (self.table[req, pos // self.P].astype(np.int64) * self.P + pos % self.P)
        return q, k, v, pos, slots

    def go(self, qlen, two_stream=False):
        q, k, v, pos, slots = self.inputs(qlen)
        seq = [n + c for n, c in zip(self.len, qlen)]
        out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        more = dict(self.scales)
        if self.rope is not None:
            more["positions"] = to_dev(pos)
        run = self.step.run_two_stream if two_stream else self.step.run
        split = run(q, k, v, to_dev(slots), self.kc, self.vc, to_dev(np.array(qlen, np.int32)),
                    to_dev(np.array(seq, np.int32)), to_dev(self.table), out, **more)
        torch.cuda.synchronize()
        assert self.step.read_errors() == 0
        self.check(q, k, v, pos, qlen, seq, out)
        self.len = seq
        return split

    def held(self, cache, scale):
        return (A.values(cache.view(torch.uint8).cpu().numpy(), scale.cpu().numpy()) if self.q8
                else cache.double().cpu().numpy())

    def check(self, q, k, v, pos, qlen, seq, out):
        k64, v64, q64 = (x.double().cpu().numpy() for x in (k, v, q))
        if self.rope is not None:
            tab = self.rope.cpu().numpy()
            k64, q64 = A.rotate(k64, pos, tab, False), A.rotate(q64, pos, tab, False)
            qr = self.step.q_rot[:q.shape[0]]
            assert np.all(np.abs(qr.double().cpu().numpy() - q64) <= 2.0 ** -8 * np.abs(q64) + 2.0 ** -18)
            q = qr
        kh, vh = self.held(self.kc, self.scales.get("k_scale")), self.held(self.vc, self.scales.get("v_scale"))
        at = 0
        vmax = []
        for r, c in enumerate(qlen):
            self.k[r] = np.concatenate([self.k[r], k64[at:at + c]])
            self.v[r] = np.concatenate([self.v[r], v64[at:at + c]])
            at += c
            j = np.arange(seq[r])
            for want, held, sc in ((self.k[r], kh, "k_scale"), (self.v[r], vh, "v_scale")):
                got = held[self.table[r, j // self.P], :, j % self.P]
                if self.q8:
                    x = self.scales[sc].cpu().numpy()[self.table[r, j // self.P], :, j % self.P // min(16, self.P)]
                    bound = 32 * 2.0 ** (x.astype(np.float64) - 127)[..., None]
                else:
                    bound = 2.0 ** -8 * np.abs(want) + 2.0 ** -18
                assert np.all(np.abs(got - want) <= bound)
            m = np.abs(vh[self.table[r, j // self.P], :, j % self.P]).max((0, 2)) if len(j) else np.zeros(self.hkv)
            vmax += [np.repeat(m, self.hq // self.hkv)] * c
        ref = oracle.paged_attention(bf16_bits(q.double().cpu().numpy()), bf16_bits(kh), bf16_bits(vh),
                                     np.array(qlen, np.int32), np.array(seq, np.int32), self.table)
        close(out.double().cpu().numpy(), ref, np.array(vmax)[..., None])


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("rope", [False, True])
def test_prefill_in_chunks_then_decode(cuda_lib, q8, rope):
    s = Served(cuda_lib, q8, rope)
    for qlen in ([130, 1, 40], [70, 33, 1], [1, 1, 1], [1, 128, 1], [1, 1, 1], [2, 1, 3]):
        s.go(qlen)


@pytest.mark.parametrize("P", [8, 64])
@pytest.mark.parametrize("d", [64, 128])
def test_other_pages_and_heads(cuda_lib, P, d):
    s = Served(cuda_lib, True, True, hq=7, hkv=1, d=d, P=P)
    for qlen in ([100, 1, 9], [1, 1, 1], [50, 60, 70]):
        s.go(qlen)


@pytest.mark.parametrize("q8", [False, True])
def test_two_streams(cuda_lib, q8):
    s = Served(cuda_lib, q8, True, n=4, two_stream=True)
    used = [s.go(qlen, two_stream=True) for qlen in ([100, 40, 60, 90], [64, 64, 64, 64], [1, 1, 1, 1])]
    assert used == [True, True, False]


def test_a_step_replayed_from_a_graph_agrees_with_eager(cuda_lib):
    """Append and attention captured together, replayed on new inputs: the buffers of a decode step."""
    a, b = Served(cuda_lib, True, True), Served(cuda_lib, True, True)
    for s in (a, b):
        s.go([150, 40, 80])
    q, k, v, pos, slots = a.inputs([1, 1, 1])
    b.inputs([1, 1, 1])
    buf = {n: x.clone() for n, x in dict(q=q, k=k, v=v, slots=to_dev(slots), pos=to_dev(pos)).items()}
    lens = to_dev(np.ones(3, np.int32))
    seq = to_dev(np.array([n + 1 for n in a.len], np.int32))
    out = torch.zeros(3, 8, 128, dtype=torch.bfloat16, device="cuda")

    def step(s, o):
        s.step.run(buf["q"], buf["k"], buf["v"], buf["slots"], s.kc, s.vc, lens, seq, to_dev_table[s], o,
                   positions=buf["pos"], **s.scales)

    to_dev_table = {a: to_dev(a.table), b: to_dev(b.table)}
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(a, out)
    side.synchronize()
    step(b, torch.zeros_like(out))
    with torch.cuda.graph(g, stream=side):
        step(a, out)
    for i in range(3):
        x = torch.from_numpy(a.rng.standard_normal((3, 12, 128)).astype(np.float32)).to(torch.bfloat16).cuda()
        buf["q"].copy_(x[:, :8])
        buf["k"].copy_(x[:, 8:10] * 2.0 ** i)
        buf["v"].copy_(x[:, 10:])
        pos = np.array([n + 1 + i for n in a.len])
        buf["pos"].copy_(torch.from_numpy(pos))
        buf["slots"].copy_(torch.from_numpy(a.table[np.arange(3), pos // 16].astype(np.int64) * 16 + pos % 16))
        seq.copy_(torch.from_numpy((pos + 1).astype(np.int32)))
        want = torch.zeros_like(out)
        step(b, want)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert torch.equal(a.kc.view(torch.uint8), b.kc.view(torch.uint8))
        assert torch.equal(a.scales["k_scale"], b.scales["k_scale"])


def test_refusals(cuda_lib):
    with pytest.raises(cuda_lib.CpsaError, match="fuses"):
        cuda_lib.AttentionStep(1, 8, 8, 2, 128, fused_kv_write=True, kv_dtype=torch.float8_e4m3fn)
    with pytest.raises(cuda_lib.CpsaError, match="kv_dtype"):
        cuda_lib.AttentionStep(1, 8, 8, 2, 128, kv_dtype=torch.float16)
    s = Served(cuda_lib, True, True)
    q, k, v, pos, slots = s.inputs([3, 0, 0])
    lens = to_dev(np.array([3, 0, 0], np.int32))
    args = (q, k, v, to_dev(slots), s.kc, s.vc, lens, lens, to_dev(s.table), torch.zeros_like(q).contiguous())
    with pytest.raises(cuda_lib.CpsaError, match="positions"):
        s.step.run(*args, **s.scales)
    with pytest.raises(cuda_lib.CpsaError, match="k_scale"):
        s.step.run(*args, positions=to_dev(pos))
    plain = cuda_lib.AttentionStep(3, 8, 8, 2, 128)
    with pytest.raises(cuda_lib.CpsaError, match="positions"):
        plain.run(*args, positions=to_dev(pos))


@pytest.mark.parametrize("rot", [16, 64, 128])
def test_rope_table_is_the_64_bit_one_rounded(cuda_lib, rot):
    t = cuda_lib.rope_table(40000, rot, base=500000.0, device="cuda").cpu().numpy()
    angle = np.arange(40000)[:, None] * 500000.0 ** (-np.arange(0, rot, 2) / rot)
    want = np.concatenate([np.cos(angle), np.sin(angle)], 1)
    # fp32's half step, and 64-bit angles of up to 40000 off by 2^-53 of themselves a few times over
    assert np.all(np.abs(t - want) <= 2.0 ** -24 * np.abs(want) + 40000 * 2.0 ** -50)
