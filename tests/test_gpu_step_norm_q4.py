"""AttentionStep with head norms and over a 4-bit cache: chunked prefill, decode, two streams and a graph, as served, and
the cached tokens handed on to a bf16 cache.

What a step stores is checked against the 64-bit definitions: a token's 4-bit numbers are rounded once, when it is
stored (q4_helpers.check_group_values), bf16 ones by half a step, 2^-8; norm and rotation in fp32 are within 2^-20 (see
test_gpu_q4_append.py). Its attention is checked against the fp64 oracle on the stored values.
"""
import numpy as np
import pytest
import torch

import oracle
from helpers import to_dev
from oracle import append as A
from oracle import q4
from q4_helpers import check_group_values
from q8_helpers import bf16_bits, close
from test_gpu_rope_append import pair_size

pytestmark = pytest.mark.gpu
EPS = 1e-5


class Served:
    """Requests that grow step by step over a shared pool of pages."""

    def __init__(self, cpsa, bits=4, rope=64, norm=True, hq=8, hkv=2, d=128, P=16, n=3, most=400, two_stream=False, seed=7):
        self.cpsa, self.bits, self.hq, self.hkv, self.d, self.P, self.n = cpsa, bits, hq, hkv, d, P, n
        rng = self.rng = np.random.default_rng(seed)
        blocks = (most + P - 1) // P
        self.table = rng.permutation(n * blocks).reshape(n, blocks).astype(np.int32)
        pages, self.scales = n * blocks, {}
        if bits == 4:
            self.kc = torch.full((pages, hkv, P, d // 2), 0x77, dtype=torch.uint8, device="cuda").view(torch.float4_e2m1fn_x2)
            sc = torch.full((pages, hkv, P, d // 16), 255, dtype=torch.uint8, device="cuda")
            self.scales = dict(k_scale=sc, v_scale=sc.clone())
        elif bits == 8:
            self.kc = torch.full((pages, hkv, P, d), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
            sc = torch.full((pages, hkv, P // min(16, P)), 255, dtype=torch.uint8, device="cuda")
            self.scales = dict(k_scale=sc, v_scale=sc.clone())
        else:
            self.kc = torch.full((pages, hkv, P, d), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.vc = torch.empty_like(self.kc)
        self.vc.view(torch.uint8).copy_(self.kc.view(torch.uint8))
        self.rope = cpsa.rope_table(most, rope, device="cuda") if rope else None
        self.weights = tuple(torch.from_numpy((1 + 0.2 * rng.standard_normal(d)).astype(np.float32)).cuda()
                             for _ in range(2)) if norm else None
        more = dict(q_norm=self.weights[0], k_norm=self.weights[1], norm_eps=EPS) if norm else {}
        self.step = cpsa.AttentionStep(n, 700, hq, hkv, d, max_kv_splits=4, two_stream=two_stream, kv_dtype=self.kc.dtype,
                                       rope=self.rope, length_threshold=16, balance_threshold=1.0, **more)
        self.len = [0] * n
        self.k = [np.zeros((0, hkv, d)) for _ in range(n)]
        self.v = [np.zeros((0, hkv, d)) for _ in range(n)]

    def inputs(self, qlen):
        T = sum(qlen)
        qkv = torch.from_numpy(self.rng.standard_normal((T, (self.hq + 2 * self.hkv) * self.d)).astype(np.float32))
        qkv = (2 * qkv).to(torch.bfloat16).cuda()
        cut = [self.hq * self.d, (self.hq + self.hkv) * self.d]
        q, k, v = (x.unflatten(1, (-1, self.d)) for x in (qkv[:, :cut[0]], qkv[:, cut[0]:cut[1]], qkv[:, cut[1]:]))
        if self.rope is None and self.weights is None:
            q = q.contiguous()
        pos = np.concatenate([np.arange(n, n + c) for n, c in zip(self.len, qlen)]).astype(np.int64)
        req = np.repeat(np.arange(self.n), qlen)
        slots = self.table[req, pos // self.P].astype(np.int64) * self.P + pos % self.P
        return q, k, v, pos, slots

    def more(self, pos):
        return dict(self.scales, **({} if self.rope is None else {"positions": to_dev(pos)}))

    def go(self, qlen, two_stream=False):
        q, k, v, pos, slots = self.inputs(qlen)
        seq = [n + c for n, c in zip(self.len, qlen)]
        out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        run = self.step.run_two_stream if two_stream else self.step.run
        split = run(q, k, v, to_dev(slots), self.kc, self.vc, to_dev(np.array(qlen, np.int32)),
                    to_dev(np.array(seq, np.int32)), to_dev(self.table), out, **self.more(pos))
        torch.cuda.synchronize()
        assert self.step.read_errors() == 0
        self.check(q, k, v, pos, qlen, seq, out)
        self.len = seq
        return split

    def held(self, cache, scale):
        raw = cache.view(torch.uint8).cpu().numpy()
        if self.bits == 4:
            return q4.values(raw, scale.cpu().numpy())
        return A.values(raw, scale.cpu().numpy()) if self.bits == 8 else cache.double().cpu().numpy()

    def wanted(self, x, weight, pos):
        """(normed and rotated, how far off in fp32)"""
        x = x.double().cpu().numpy()
        if self.weights is not None:
            x = q4.head_norm(x, weight.cpu().numpy(), EPS)
        if self.rope is None:
            return x, 2.0 ** -20 * np.abs(x) * (self.weights is not None)
        tol = 2.0 ** -20 * np.maximum(np.abs(x), pair_size(x, self.rope.shape[1], False))
        return A.rotate(x, pos, self.rope.cpu().numpy(), False), tol

    def check(self, q, k, v, pos, qlen, seq, out):
        wq, wk = self.weights or (None, None)
        k64, k_tol = self.wanted(k, wk, pos)
        q64, q_tol = self.wanted(q, wq, pos)
        v64 = v.double().cpu().numpy()
        if self.step.q_rot is not None:
            qr = self.step.q_rot[:q.shape[0]]
            assert np.all(np.abs(qr.double().cpu().numpy() - q64) <= 2.0 ** -8 * np.abs(q64) + 2 * q_tol)
            q = qr
        kh, vh = self.held(self.kc, self.scales.get("k_scale")), self.held(self.vc, self.scales.get("v_scale"))
        at, vmax = 0, []
        for r, c in enumerate(qlen):
            new = np.arange(self.len[r], seq[r])
            page, off = self.table[r, new // self.P], new % self.P
            for want, tol, cache, name, all_held in ((k64, k_tol, self.kc, "k_scale", kh), (v64, 0 * k_tol, self.vc, "v_scale", vh)):
                want, tol = want[at:at + c], tol[at:at + c]
                if self.bits == 4:
                    check_group_values(want, tol, cache.view(torch.uint8).cpu().numpy()[page, :, off],
                                       self.scales[name].cpu().numpy()[page, :, off])
                elif self.bits == 16:
                    assert np.all(np.abs(all_held[page, :, off] - want) <= 2.0 ** -8 * np.abs(want) + 2 * tol)
            at += c
            j = np.arange(seq[r])
            m = np.abs(vh[self.table[r, j // self.P], :, j % self.P]).max((0, 2)) if len(j) else np.zeros(self.hkv)
            vmax += [np.repeat(m, self.hq // self.hkv)] * c
        ref = oracle.paged_attention(bf16_bits(q.double().cpu().numpy()), bf16_bits(kh), bf16_bits(vh),
                                     np.array(qlen, np.int32), np.array(seq, np.int32), self.table)
        close(out.double().cpu().numpy(), ref, np.array(vmax)[..., None])


@pytest.mark.parametrize("bits,rope,norm", [(4, 128, True), (4, 0, True), (4, 64, False), (4, 0, False), (8, 64, True),
                                            (16, 128, True), (16, 0, True)])
def test_prefill_in_chunks_then_decode(cuda_lib, bits, rope, norm):
    s = Served(cuda_lib, bits, rope, norm)
    for qlen in ([130, 1, 40], [70, 33, 1], [1, 1, 1], [1, 128, 1], [1, 1, 1], [2, 1, 3]):
        s.go(qlen)


@pytest.mark.parametrize("P", [8, 64])
@pytest.mark.parametrize("d", [64, 128])
def test_other_pages_and_heads(cuda_lib, P, d):
    s = Served(cuda_lib, hq=7, hkv=1, d=d, P=P)
    for qlen in ([100, 1, 9], [1, 1, 1], [50, 60, 70]):
        s.go(qlen)


@pytest.mark.parametrize("bits", [4, 16])
def test_two_streams(cuda_lib, bits):
    s = Served(cuda_lib, bits, n=4, two_stream=True)
    used = [s.go(qlen, two_stream=True) for qlen in ([100, 40, 60, 90], [64, 64, 64, 64], [1, 1, 1, 1])]
    assert used == [True, True, False]


def test_a_step_replayed_from_a_graph_agrees_with_eager(cuda_lib):
    """Append and attention captured together, replayed on new inputs: the buffers of a decode step."""
    a, b = Served(cuda_lib), Served(cuda_lib)
    for s in (a, b):
        s.go([150, 40, 80])
    q, k, v, pos, slots = a.inputs([1, 1, 1])
    buf = {n: x.clone() for n, x in dict(q=q, k=k, v=v, slots=to_dev(slots), pos=to_dev(pos)).items()}
    lens, seq = to_dev(np.ones(3, np.int32)), to_dev(np.array([n + 1 for n in a.len], np.int32))
    out = torch.zeros(3, 8, 128, dtype=torch.bfloat16, device="cuda")
    table = {s: to_dev(s.table) for s in (a, b)}

    def step(s, o):
        s.step.run(buf["q"], buf["k"], buf["v"], buf["slots"], s.kc, s.vc, lens, seq, table[s], o, positions=buf["pos"],
                   **s.scales)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(a, out)
    side.synchronize()
    step(b, torch.zeros_like(out))
    g = torch.cuda.CUDAGraph()
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


def test_cached_tokens_handed_on_to_a_bf16_cache(cuda_lib):
    """Read back and written into a bf16 cache, a request's attention goes on there: the same values, another kernel."""
    s = Served(cuda_lib, hq=8, hkv=8)
    s.go([200, 30, 77])
    n = 200
    j = np.arange(n)
    slots = to_dev(s.table[0, j // 16].astype(np.int64) * 16 + j % 16)
    k, v = (torch.empty(n, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cuda_lib.cpp_kv_cache_read_q4(s.kc, s.vc, *s.scales.values(), slots, k, v, err)
    kc, vc = (torch.zeros(13, 8, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cuda_lib.cpp_kv_cache_write(k, v, torch.arange(n, device="cuda"), kc, vc, err)
    kh = s.held(s.kc, s.scales["k_scale"])[s.table[0, j // 16], :, j % 16]
    assert np.array_equal(k.double().cpu().numpy(), kh)
    q = torch.from_numpy(s.rng.standard_normal((1, 8, 128)).astype(np.float32)).to(torch.bfloat16).cuda()
    lens, seq = to_dev(np.array([1], np.int32)), to_dev(np.array([n], np.int32))
    table = {4: to_dev(s.table[:1]), 16: torch.arange(13, dtype=torch.int32, device="cuda").view(1, -1)}
    ws = torch.empty(cuda_lib.cpp_attn_workspace_bytes(1, 1, 8, 8, 128, 8), dtype=torch.uint8, device="cuda")
    a, b = torch.zeros_like(q), torch.zeros_like(q)
    cuda_lib.cpp_chunked_prefill_attn_q4(q, s.kc, s.vc, *s.scales.values(), lens, seq, table[4], a, ws, err)
    cuda_lib.cpp_chunked_prefill_attn(q, kc, vc, lens, seq, table[16], b, ws, err)
    vmax = v.abs().amax((0, 2)).double().cpu().numpy()
    # each within half a bf16 step of the output and 2^-8 of the largest value (see q8_helpers.py)
    gap = np.abs(a.double().cpu().numpy() - b.double().cpu().numpy())[0]
    assert np.all(gap <= 2 * (2.0 ** -8 * np.abs(b.double().cpu().numpy()[0]) + 2.0 ** -7 * vmax[:, None]))
    assert cuda_lib.cpp_read_device_error(err) == 0


def test_refusals(cuda_lib):
    w = torch.ones(128, device="cuda")
    with pytest.raises(cuda_lib.CpsaError, match="fuses"):
        cuda_lib.AttentionStep(1, 8, 8, 2, 128, fused_kv_write=True, kv_dtype=torch.float4_e2m1fn_x2)
    with pytest.raises(cuda_lib.CpsaError, match="fuses"):
        cuda_lib.AttentionStep(1, 8, 8, 2, 128, fused_kv_write=True, q_norm=w, k_norm=w)
    with pytest.raises(cuda_lib.CpsaError, match="go together"):
        cuda_lib.AttentionStep(1, 8, 8, 2, 128, q_norm=w)
    s = Served(cuda_lib)
    q, k, v, pos, slots = s.inputs([3, 0, 0])
    lens = to_dev(np.array([3, 0, 0], np.int32))
    args = (q, k, v, to_dev(slots), s.kc, s.vc, lens, lens, to_dev(s.table), torch.zeros_like(q).contiguous())
    with pytest.raises(cuda_lib.CpsaError, match="k_scale"):
        s.step.run(*args, positions=to_dev(pos))
    with pytest.raises(cuda_lib.CpsaError, match="positions"):
        s.step.run(*args, **s.scales)
    with pytest.raises(cuda_lib.CpsaError, match="must be torch.uint8 or torch.float4"):
        wrong = s.kc.view(torch.uint8).view(torch.int8)
        s.step.run(q, k, v, to_dev(slots), wrong, wrong, *args[6:], **s.more(pos))
