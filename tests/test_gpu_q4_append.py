"""The 4-bit append, head norms and the 4-bit cache's read on the GPU against their 64-bit definitions (oracle/q4.py).

Tolerances before a value's one rounding to its output's type (fp32 roundings are half steps of 2^-24):
  rotated          2^-22 (|a| + |b|), as in test_gpu_rope_append.py
  head norm        the sum of squares of positive terms passes at most 16 / 2 + 1 + 3 + 1 additions and a division by
                   head_dim (exact), eps is one more: 14 * 2^-24 of it, halved by the root; the reciprocal root is off
                   by at most two last places, 4 * 2^-24, and the two products round once each: 13 * 2^-24 < 2^-20 of
                   the value, and with its rotation's 3 * 2^-24 at most 2^-20 (|a| + |b|)
What is neither normed nor rotated is exact before its rounding, and then codes and scales are those of the definition.
bf16 adds half a step, 2^-8 of the value; 4 bits: q4_helpers.check_group_values.
"""
import numpy as np
import pytest
import torch

from oracle import append as A
from oracle import q4
from q4_helpers import check_group_values
from test_gpu_rope_append import RUNS, SHAPES, Case, bf16, check_q8, pair_size, q8_cache, wide

pytestmark = pytest.mark.gpu

MORE_SHAPES = SHAPES + [
    (3, 2, 128, 16, 48, False),      # halves of a group in different places of two threads
    (2, 2, 64, 32, 48, False),
    (2, 1, 128, 64, 112, False),
    (2, 1, 128, 16, 96, True),
    (2, 3, 64, 16, 0, True),
]


def q4_cache(c):
    shape = (c.pages, c.hkv, c.P)
    cache = torch.from_numpy(c.rng.integers(0, 256, (*shape, c.d // 2)).astype(np.uint8)).cuda()
    scale = torch.from_numpy(c.rng.integers(0, 256, (*shape, c.d // 16)).astype(np.uint8)).cuda()
    return cache, scale


def weights(c):
    return tuple(torch.from_numpy((1 + 0.3 * c.rng.standard_normal(c.d)).astype(np.float32)).cuda() for _ in range(2))


def check_q4(c, x, tol, cache, scale, cache0, scale0):
    """One of k and v: the places written, and nothing else."""
    _, w = c.live()
    page, off = c.slots[w] // c.P, c.slots[w] % c.P
    got, gs = cache.view(torch.uint8).cpu().numpy(), scale.cpu().numpy()
    check_group_values(x[w], tol[w], got[page, :, off], gs[page, :, off])
    got[page, :, off], gs[page, :, off] = cache0[page, :, off], scale0[page, :, off]
    assert np.array_equal(got, cache0) and np.array_equal(gs, scale0), "other places of the cache changed"


def numpied(*tensors):
    return [t.view(torch.uint8).cpu().numpy() for t in tensors]


@pytest.mark.parametrize("runs", RUNS)
@pytest.mark.parametrize("shape", MORE_SHAPES, ids=str)
def test_q4_append(cuda_lib, shape, runs):
    hq, hkv, d, P, rot, inter = shape
    c = Case(21, hq, hkv, d, P, 1024 // P, rot, RUNS[runs])
    (kc, ks), (vc, vs) = q4_cache(c), q4_cache(c)
    was = numpied(kc, ks, vc, vs)
    q_out = bf16(c.rng, (c.T, hq, d)).cuda()
    before = q_out.clone()
    q, k, v, pos, cs, slots = c.args()
    cuda_lib.cpp_rope_kv_cache_write_q4(q, k, v, pos, cs, slots, kc.view(torch.float4_e2m1fn_x2), vc, ks, vs, q_out, c.err,
                                        interleaved=inter)
    c.check_q(q_out, before, inter)
    check_q4(c, c.expected(k, inter), 2.0 ** -22 * pair_size(wide(k), rot, inter), kc, ks, was[0], was[1])
    check_q4(c, wide(v), np.zeros(v.shape), vc, vs, was[2], was[3])
    assert cuda_lib.cpp_read_device_error(c.err) == 0


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("runs", ["one", "decode", "mixed"])
@pytest.mark.parametrize("shape", MORE_SHAPES, ids=str)
def test_norm_append(cuda_lib, shape, runs, bits):
    hq, hkv, d, P, rot, inter = shape
    eps = 1e-5
    c = Case(22, hq, hkv, d, P, 1024 // P, rot, RUNS[runs], gain=3.0)
    qw, kw = weights(c)
    q_out = bf16(c.rng, (c.T, hq, d)).cuda()
    before = q_out.clone()
    q, k, v, pos, cs, slots = c.args()
    qn, kn = (q4.head_norm(wide(x), wide(w), eps) for x, w in ((q, qw), (k, kw)))
    q_ref, k_ref = (A.rotate(x, c.pos, c.table, inter) for x in (qn, kn))
    q_tol, k_tol = (2.0 ** -20 * np.maximum(np.abs(x), pair_size(x, rot, inter)) for x in (qn, kn))
    ok, w = c.live()
    page, off = c.slots[w] // P, c.slots[w] % P
    more = dict(eps=eps, interleaved=inter)
    if bits == 16:
        kc, vc = (bf16(c.rng, (c.pages, hkv, P, d)).cuda() for _ in range(2))
        k0, v0 = wide(kc), wide(vc)
        cuda_lib.cpp_norm_rope_kv_cache_write(q, k, v, qw, kw, pos, cs, slots, kc, vc, q_out, c.err, **more)
        got = wide(kc)
        assert np.all(np.abs(got[page, :, off] - k_ref[w]) <= (2.0 ** -8 * np.abs(k_ref) + 2 * k_tol)[w])
        got[page, :, off] = k0[page, :, off]
        v0[page, :, off] = wide(v)[w]
        assert np.array_equal(got, k0) and np.array_equal(wide(vc), v0)
    else:
        (kc, ks), (vc, vs) = (q8_cache if bits == 8 else q4_cache)(c), (q8_cache if bits == 8 else q4_cache)(c)
        was = numpied(kc, ks, vc, vs)
        fn = cuda_lib.cpp_norm_rope_kv_cache_write_q8 if bits == 8 else cuda_lib.cpp_norm_rope_kv_cache_write_q4
        fn(q, k, v, qw, kw, pos, cs, slots, kc, vc, ks, vs, q_out, c.err, **more)
        if bits == 8:
            sl = np.where(w, c.slots, -1)
            check_q8(c, k_ref, True, 2 * k_tol, kc, ks, was[0], was[1], sl)
            check_q8(c, wide(v), False, 0 * k_tol, vc, vs, was[2], was[3], sl)
        else:
            check_q4(c, k_ref, k_tol, kc, ks, was[0], was[1])
            check_q4(c, wide(v), 0 * k_tol, vc, vs, was[2], was[3])
    got = wide(q_out)
    assert np.all((np.abs(got - q_ref) <= 2.0 ** -8 * np.abs(q_ref) + 2 * q_tol)[ok])
    assert torch.equal(q_out.cpu().view(torch.int16)[~ok], before.cpu().view(torch.int16)[~ok])
    assert cuda_lib.cpp_read_device_error(c.err) == 0


def test_norm_of_zero_tiny_and_huge_heads(cuda_lib):
    """A zero head stays zero, eps counts beside tiny ones, one large column does not drown the rest's digits."""
    d, eps = 128, 1e-6
    x = torch.zeros(5, 1, d)
    x[1] = 1e-5
    x[2] = torch.linspace(-1, 1, d) * 1e15
    x[3, 0, 7] = 3e4
    x[3, 0, 8:] = 1.0
    x[4, 0, 3] = float("nan")
    x = x.to(torch.bfloat16).cuda()
    w = torch.linspace(0.5, 2, d, device="cuda")
    kc, vc = (torch.zeros(1, 1, 8, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q_out, err = torch.zeros_like(x), torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = torch.arange(5, device="cuda")
    cuda_lib.cpp_norm_rope_kv_cache_write(x, x, x, w, w, None, None, slots, kc, vc, q_out, err, eps=eps)
    want = q4.head_norm(wide(x)[:4], wide(w), eps)
    for got in (wide(q_out)[:, 0], wide(kc)[0, 0, :5]):
        assert np.all(np.abs(got[:4] - want[:, 0]) <= (2.0 ** -8 + 2.0 ** -20) * np.abs(want[:, 0]))
        assert np.all(np.isnan(got[4]))
    assert torch.equal(vc[0, 0, :5].view(torch.int16), x[:, 0].view(torch.int16))


@pytest.mark.parametrize("d", [64, 128])
def test_q4_values_of_every_size(cuda_lib, d):
    """Groups from the smallest bf16 to the largest, ties of scales and codes, zeros, infinities and NaN."""
    rng = np.random.default_rng(23)
    inf, nan = float("inf"), float("nan")
    rows = [np.zeros(d), np.full(d, -0.0), np.full(d, 3.38e38), np.full(d, 1e-40)]
    for e in range(-30, 20):
        rows.append(rng.standard_normal(d) * 2.0 ** e)
    for s in (1.0, 1.125, 1.875, 0.234375, 2.0 ** -17, 5 * 2.0 ** -17):       # ties between codes under the scale s
        rows.append(s * rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -2.5, -5.0, 6.0], d))
        rows[-1][::16] = 6 * s
    rows += [np.full(d, 6 * (1 + m / 16) * 2.0 ** e) for m in range(16) for e in (-3, 0)]   # ties between scales
    for bad in (inf, -inf, nan):
        rows.append(rng.standard_normal(d))
        rows[-1][rng.integers(0, d)] = bad
    x = torch.from_numpy(np.array(rows, np.float32)).to(torch.bfloat16)[:, None].contiguous().cuda()
    n, P = len(rows), 8
    pages = n // P + 1
    kc = torch.full((pages, 1, P, d // 2), 0x5A, dtype=torch.uint8, device="cuda")
    ks = torch.full((pages, 1, P, d // 16), 77, dtype=torch.uint8, device="cuda")
    vc, vs = kc.clone(), ks.clone()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cuda_lib.cpp_rope_kv_cache_write_q4(None, x, x, None, None, torch.arange(n, device="cuda"), kc, vc, ks, vs, None, err)
    code, scale = q4.quantised(wide(x)[:, 0])
    for c, s in ((kc, ks), (vc, vs)):
        c, s = c.cpu().numpy().reshape(-1, d // 2), s.cpu().numpy().reshape(-1, d // 16)
        assert np.array_equal(s[:n], scale)
        got = q4.unpacked(c[:n])
        same = (got == code) | ((got & 7 == 0) & (code & 7 == 0)) | np.repeat(scale == 255, 16, 1)
        assert same.all()
        assert np.all(c[n:] == 0x5A) and np.all(s[n:] == 77)


def test_flags_and_skipped_tokens(cuda_lib):
    """Positions and slots out of range are flagged and skipped, padding is skipped, the rest is done."""
    runs = [(0, 3, 0), (1024, 1, 5), (20, 2, 600), (30, 1, -1), (-7, 1, 9), (40, 2, 598), (1 << 40, 1, 4), (50, 1, 1 << 40)]
    c = Case(24, 4, 2, 64, 16, 64, 48, runs)
    qw, kw = weights(c)
    for norm in (False, True):
        (kc, ks), (vc, vs) = q4_cache(c), q4_cache(c)
        was = numpied(vc, vs)
        q_out = bf16(c.rng, (c.T, 4, 64)).cuda()
        before = q_out.clone()
        q, k, v, pos, cs, slots = c.args()
        if norm:
            cuda_lib.cpp_norm_rope_kv_cache_write_q4(q, k, v, qw, kw, pos, cs, slots, kc, vc, ks, vs, q_out, c.err)
            ok = torch.from_numpy(c.live()[0])
            assert torch.equal(q_out.cpu().view(torch.int16)[~ok], before.cpu().view(torch.int16)[~ok])
        else:
            cuda_lib.cpp_rope_kv_cache_write_q4(q, k, v, pos, cs, slots, kc, vc, ks, vs, q_out, c.err)
            c.check_q(q_out, before, False)
        check_q4(c, wide(v), np.zeros(v.shape), vc, vs, was[0], was[1])
        assert cuda_lib.cpp_read_device_error(c.err) == cuda_lib.DEV_SLOT_OUT_OF_RANGE | cuda_lib.DEV_POSITION_OUT_OF_RANGE


@pytest.mark.parametrize("bits", [16, 8, 4])
def test_strided_contiguous_and_in_place_agree(cuda_lib, bits):
    c = Case(25, 14, 2, 128, 16, 64, 96, RUNS["mixed"])
    qw, kw = weights(c)
    q, k, v, pos, cs, slots = c.args()
    outs = []
    for form in ("strided", "contiguous", "in place"):
        qq, kk, vv = (q, k, v) if form == "strided" else (q.contiguous(), k.contiguous(), v.contiguous())
        q_out = qq if form == "in place" else torch.empty(c.T, 14, 128, dtype=torch.bfloat16, device="cuda")
        held = [torch.zeros(64, 2, 16, 64 if bits == 4 else 128, dtype=torch.bfloat16 if bits == 16 else torch.uint8,
                            device="cuda") for _ in range(2)]
        if bits < 16:
            held += [torch.full((64, 2, 1) if bits == 8 else (64, 2, 16, 8), 120, dtype=torch.uint8, device="cuda")
                     for _ in range(2)]
        fn = {16: cuda_lib.cpp_norm_rope_kv_cache_write, 8: cuda_lib.cpp_norm_rope_kv_cache_write_q8,
              4: cuda_lib.cpp_norm_rope_kv_cache_write_q4}[bits]
        fn(qq, kk, vv, qw, kw, pos, cs, slots, *held, q_out, c.err)
        outs.append([q_out, *held])
    ok = torch.from_numpy(c.live()[0]).cuda()
    for o in outs[1:]:
        assert torch.equal(o[0][ok], outs[0][0][ok])
        assert all(torch.equal(a, b) for a, b in zip(o[1:], outs[0][1:]))


def test_append_and_read_captured_on_another_stream_and_replayed(cuda_lib):
    c = Case(26, 8, 2, 128, 16, 64, 128, RUNS["prompt"])
    q, k, v, pos, cs, slots = c.args()
    qw, kw = weights(c)
    shape = (64, 2, 16)

    def buffers():
        return [torch.zeros(*shape, n, dtype=torch.uint8, device="cuda") for n in (64, 64, 8, 8)] + [
            torch.zeros(c.T, 8, 128, dtype=torch.bfloat16, device="cuda")] + [
            torch.zeros(c.T, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]

    def go(b):
        cuda_lib.cpp_norm_rope_kv_cache_write_q4(q, k, v, qw, kw, pos, cs, slots, *b[:5], c.err)
        cuda_lib.cpp_kv_cache_read_q4(*b[:4], slots, *b[5:], c.err)

    a, b = buffers(), buffers()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        go(b)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        go(b)
    fresh = bf16(c.rng, (c.T, 12 * 128)).cuda()
    q.copy_(fresh[:, :1024].unflatten(1, (8, 128)))
    k.copy_(fresh[:, 1024:1280].unflatten(1, (2, 128)))
    v.copy_(fresh[:, 1280:].unflatten(1, (2, 128)))
    g.replay()
    torch.cuda.synchronize()
    go(a)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_slots_in_any_order(cuda_lib):
    n, P = 40, 16
    rng = np.random.default_rng(27)
    k, v = (bf16(rng, (n, 2, 64)).cuda() for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = rng.permutation(4 * P)[:n]
    held = [torch.zeros(4, 2, P, m, dtype=torch.uint8, device="cuda") for m in (32, 32, 4, 4)]
    cuda_lib.cpp_rope_kv_cache_write_q4(None, k, v, None, None, torch.from_numpy(slots).cuda(), *held, None, err)
    got = [x.cpu().numpy()[slots // P, :, slots % P] for x in held]
    check_group_values(wide(k), np.zeros(k.shape), got[0], got[2])
    check_group_values(wide(v), np.zeros(v.shape), got[1], got[3])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("P", [8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("T", [1, 2, 15, 17, 300])
def test_read(cuda_lib, T, P, d):
    """Any slots, some twice, some of padding, some past the cache, all scale bytes but those beyond bf16."""
    rng = np.random.default_rng(1000 * T + P + d)
    pages, hkv = 512 // P, 3
    held = [rng.integers(0, 256, (pages, hkv, P, n)).astype(np.uint8) for n in (d // 2, d // 2)]
    held += [rng.integers(0, 248, (pages, hkv, P, n)).astype(np.uint8) for n in (d // 16, d // 16)]
    held[2][0, 0, 0, :] = 255
    slots = rng.integers(0, 512, T)
    slots[T // 2:] = np.where(rng.random(T - T // 2) < 0.2, -1, slots[T // 2:])
    slots[0] = 0
    if T > 2:
        slots[1], slots[2] = 512, 1 << 50
    k, v = (torch.full((T, hkv, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cuda_lib.cpp_kv_cache_read_q4(*(torch.from_numpy(x).cuda() for x in held), torch.from_numpy(slots).cuda(), k, v, err)
    live = (slots >= 0) & (slots < 512)
    at, off = slots[live] // P, slots[live] % P
    for got, codes, scale in ((k, held[0], held[2]), (v, held[1], held[3])):
        want = np.full((T, hkv, d), 7.0)
        x = q4.values(codes[at, :, off], scale[at, :, off])
        # in f16 on the way: exact below 65504 (scales of the append), infinite behind it
        want[live] = np.where(np.abs(x) >= 65520, np.where(x < 0, -np.inf, np.inf), x)
        assert np.array_equal(wide(got), want, equal_nan=True)
    assert cuda_lib.cpp_read_device_error(err) == (cuda_lib.DEV_SLOT_OUT_OF_RANGE if T > 2 else 0)


@pytest.mark.parametrize("d", [64, 128])
def test_read_into_tensors_on_16_byte_boundaries(cuda_lib, d):
    """k and v 16 bytes behind a 32-byte boundary: the same values, and nothing beside them."""
    rng = np.random.default_rng(29)
    T, hkv, P = 37, 2, 16
    held = [torch.from_numpy(rng.integers(0, 227, (8, hkv, P, n)).astype(np.uint8)).cuda()
            for n in (d // 2, d // 2, d // 16, d // 16)]
    slots = torch.from_numpy(rng.integers(0, 8 * P, T)).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    n = T * hkv * d
    whole = [torch.full((n + 16,), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    shifted = [x[8:8 + n].view(T, hkv, d) for x in whole]
    plain = [torch.empty(T, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    assert all(x.data_ptr() % 32 == 16 for x in shifted)
    cuda_lib.cpp_kv_cache_read_q4(*held, slots, *shifted, err)
    cuda_lib.cpp_kv_cache_read_q4(*held, slots, *plain, err)
    assert all(torch.equal(a, b) for a, b in zip(shifted, plain))
    assert all(bool((x[:8] == 3).all()) and bool((x[8 + n:] == 3).all()) for x in whole)


def test_q4_cache_beyond_32_bit_offsets(cuda_lib):
    P, hkv, d = 16, 8, 128
    pages = (1 << 32) // (P * hkv * d // 2) + 3
    held = [torch.zeros(pages, hkv, P, n, dtype=torch.uint8, device="cuda") for n in (d // 2, d // 2, d // 16, d // 16)]
    rng = np.random.default_rng(28)
    n = 20
    k, v = (bf16(rng, (n, hkv, d)).cuda() for _ in range(2))
    slots = torch.arange(n, device="cuda") + (pages - 2) * P
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cuda_lib.cpp_rope_kv_cache_write_q4(None, k, v, None, None, slots, *held, None, err)
    got = [x[-2:].cpu().numpy().transpose(0, 2, 1, 3).reshape(2 * P, hkv, -1)[:n] for x in held]
    check_group_values(wide(k), np.zeros(k.shape), got[0], got[2])
    check_group_values(wide(v), np.zeros(v.shape), got[1], got[3])
    assert all(int((x[:-2] != 0).sum()) == 0 for x in held)
    kb, vb = torch.zeros_like(k), torch.zeros_like(v)
    cuda_lib.cpp_kv_cache_read_q4(*held, slots, kb, vb, err)
    assert np.array_equal(wide(kb), q4.values(got[0], got[2])) and np.array_equal(wide(vb), q4.values(got[1], got[3]))
    assert cuda_lib.cpp_read_device_error(err) == 0


def test_calls_of_another_device_are_refused(cuda_lib, monkeypatch):
    """Tensors are on device 0; with another device current the calls do not run."""
    k = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    held = [torch.zeros(2, 2, 16, n, dtype=torch.uint8, device="cuda") for n in (32, 32, 4, 4)]
    slots = torch.zeros(2, dtype=torch.int64, device="cuda")
    w = torch.ones(64, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    s = torch.cuda.default_stream(0)
    with pytest.raises(cuda_lib.CpsaError, match="cuda:"):
        cuda_lib.cpp_rope_kv_cache_write_q4(None, k, k, None, None, slots, *held, None, err, stream=s)
    with pytest.raises(cuda_lib.CpsaError, match="cuda:"):
        cuda_lib.cpp_norm_rope_kv_cache_write_q4(None, k, k, None, w, None, None, slots, *held, None, err, stream=s)
    with pytest.raises(cuda_lib.CpsaError, match="cuda:"):
        cuda_lib.cpp_kv_cache_read_q4(*held, slots, k, k.clone(), err, stream=s)


def test_no_tokens(cuda_lib):
    z = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    held = [torch.zeros(2, 2, 16, n, dtype=torch.uint8, device="cuda") for n in (32, 32, 4, 4)]
    slots = torch.zeros(0, dtype=torch.int64, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cuda_lib.cpp_rope_kv_cache_write_q4(z, z, z, None, None, slots, *held, z, err)
    cuda_lib.cpp_kv_cache_read_q4(*held, slots, z, z.clone(), err)
    assert not any(x.any() for x in held)
