"""The rotary KV appends on the GPU against their 64-bit definitions (oracle/append.py).

Tolerances. A rotated value is formed in fp32 from a c and b s: two products and a
sum, each off by at most 2^-24 of its size, so it is within 3 * 2^-24 (|a c| + |b s|)
<= 2^-22 (|a| + |b|) of the exact one. bf16 then adds half a step, 2^-8 of the value.
An e4m3 byte is within half a step of value / 2^x, plus that fp32 error / 2^x (which
can also move a value over the border between two bytes). What is not rotated (v,
columns from rotary dim on) is exact before its one rounding.
"""
import numpy as np
import pytest
import torch

from oracle import append as A

pytestmark = pytest.mark.gpu


def table(top, rot, rng):
    angle = np.arange(top)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)[None]
    return np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)


def bf16(rng, shape, gain=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * gain).astype(np.float32)).to(torch.bfloat16)


def wide(x):
    return x.double().cpu().numpy()


def pair_size(x, rot, interleaved):
    """|a| + |b| of every column's pair (0 where nothing is rotated)."""
    out = np.zeros_like(x)
    a = np.abs(x)
    for i in range(rot // 2):
        m, n = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        out[..., m] = out[..., n] = a[..., m] + a[..., n]
    return out


def same_bytes(got, want):
    """Equal bytes, every NaN byte counting as one."""
    nan = (got & 127) == 127
    return np.array_equal(nan, (want & 127) == 127) and np.array_equal(got[~nan], want[~nan])


class Case:
    """One call's inputs: `runs` lists (slot of the first token, tokens, first position)."""

    def __init__(self, seed, hq, hkv, d, P, pages, rot, runs, top=600, fused=True, gain=1.0):
        rng = np.random.default_rng(seed)
        self.hq, self.hkv, self.d, self.P, self.pages, self.rot = hq, hkv, d, P, pages, rot
        slots = [np.arange(s, s + n) if s >= 0 else np.full(n, s) for s, n, _ in runs]
        pos = [np.arange(p, p + n) if p >= 0 else np.full(n, p) for _, n, p in runs]
        self.slots, self.pos = np.concatenate(slots).astype(np.int64), np.concatenate(pos).astype(np.int64)
        T = len(self.slots)
        self.T = T
        self.table = table(top, rot, rng) if rot else None
        if fused:
            qkv = bf16(rng, (T, (hq + 2 * hkv) * d), gain).cuda()
            self.q = qkv[:, :hq * d].unflatten(1, (hq, d))
            self.k = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
            self.v = qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
        else:
            self.q, self.k, self.v = (bf16(rng, (T, h, d), gain).cuda() for h in (hq, hkv, hkv))
        self.rng = rng
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def args(self):
        cs = None if self.table is None else torch.from_numpy(self.table).cuda()
        pos = None if self.table is None else torch.from_numpy(self.pos).cuda()
        return self.q, self.k, self.v, pos, cs, torch.from_numpy(self.slots).cuda()

    def expected(self, x, interleaved):
        return A.rotate(wide(x), self.pos, self.table, interleaved)

    def live(self):
        ok = np.ones(self.T, bool) if self.table is None else (self.pos >= 0) & (self.pos < self.table.shape[0])
        return ok, ok & (self.slots >= 0) & (self.slots < self.pages * self.P)

    def check_q(self, q_out, before, interleaved):
        ok, _ = self.live()
        want, got = self.expected(self.q, interleaved), wide(q_out)
        tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -21 * pair_size(wide(self.q), self.rot, interleaved)
        assert np.all((np.abs(got - want) <= tol)[ok])
        assert torch.equal(q_out.cpu().view(torch.int16)[~ok], before.cpu().view(torch.int16)[~ok])
        plain = want[..., self.rot:][ok]
        assert np.array_equal(got[..., self.rot:][ok], plain)


SHAPES = [
    # hq, hkv, d, page, rot, interleaved
    (32, 8, 128, 16, 128, False),
    (8, 2, 128, 128, 128, True),
    (6, 3, 128, 8, 64, False),
    (14, 2, 64, 32, 32, True),
    (4, 4, 64, 256, 64, False),
    (5, 1, 64, 8, 16, False),
    (1, 1, 128, 64, 0, False),
]
# (first slot, tokens, first position); page numbers are multiplied in below
RUNS = {
    "one": [(5, 1, 77)],
    "decode": [(8 * i + (3 * i) % 8, 1, 11 * i) for i in range(21)],
    "prompt": [(0, 131, 0)],
    "middle": [(13, 70, 13)],
    "mixed": [(512 + 9, 1, 400), (640, 1, 0), (3, 45, 3), (256, 33, 0), (-1, 3, -1), (700, 2, 60)],
    "late": [(1, 1, 1)] * 1 + [(16 * i + 7, 1, 5) for i in range(2, 9)] + [(256 + 1, 60, 21)],
}


@pytest.mark.parametrize("runs", RUNS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_bf16_append(cuda_lib, shape, runs):
    hq, hkv, d, P, rot, inter = shape
    c = Case(1, hq, hkv, d, P, 1024 // P, rot, RUNS[runs])
    kc = bf16(c.rng, (c.pages, hkv, P, d)).cuda()
    vc = bf16(c.rng, (c.pages, hkv, P, d)).cuda()
    k0, v0 = wide(kc), wide(vc)
    q_out = bf16(c.rng, (c.T, hq, d)).cuda()
    before = q_out.clone()
    q, k, v, pos, cs, slots = c.args()
    cuda_lib.cpp_rope_kv_cache_write(q, k, v, pos, cs, slots, kc, vc, q_out, c.err, interleaved=inter)
    c.check_q(q_out, before, inter)
    _, w = c.live()
    page, off = c.slots[w] // P, c.slots[w] % P
    want = c.expected(k, inter)[w]
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -21 * pair_size(wide(k), rot, inter)[w]
    got = wide(kc)
    assert np.all(np.abs(got[page, :, off] - want) <= tol)
    v0[page, :, off] = wide(v)[w]
    assert np.array_equal(wide(vc), v0)
    got[page, :, off] = k0[page, :, off]
    assert np.array_equal(got, k0), "other places of the cache changed"
    assert cuda_lib.cpp_read_device_error(c.err) == 0


def check_q8(c, x, moved, tol_in, cache, scale, cache0, scale0, slots=None):
    """One of k and v: against the oracle run on the same bytes."""
    want, wscale = cache0.copy(), scale0.copy()
    slots = c.slots if slots is None else slots
    y = A.append_q8(x, slots, want, wscale)
    got, gscale = cache.view(torch.uint8).cpu().numpy(), scale.view(torch.uint8).cpu().numpy()
    assert np.array_equal(gscale, wscale)
    fixed = np.ones(got.shape[:3], bool)
    sb = min(16, c.P)
    row = {(int(s) // c.P, int(s) % c.P): t for t, s in enumerate(slots) if s >= 0}
    for (page, h, off), t in y.items():
        fixed[page, h, off] = False
        val = A.VALUES[got[page, h, off]]
        fin = np.isfinite(t)
        assert np.array_equal(np.isnan(val), ~fin)
        slack = tol_in[row[(page, off)], h] * 2.0 ** (127 - int(wscale[page, h, off // sb]))
        t = np.clip(t[fin], -448, 448)
        assert np.all(np.abs(val[fin] - t) <= A.half_step(np.abs(t) + slack[fin]) + slack[fin])
        if not moved:
            assert same_bytes(got[page, h, off], want[page, h, off])
    assert same_bytes(got[fixed], want[fixed]), "bytes of other places"


def q8_cache(c):
    """Random bytes and scales around those of normal data."""
    shape = (c.pages, c.hkv, c.P, c.d)
    cache = torch.from_numpy(c.rng.standard_normal(shape).astype(np.float32) * 100).clamp(-448, 448)
    cache = cache.to(torch.float8_e4m3fn).cuda()
    scale = torch.from_numpy(c.rng.integers(116, 123, (c.pages, c.hkv, c.P // min(16, c.P))).astype(np.uint8)).cuda()
    return cache, scale


@pytest.mark.parametrize("runs", RUNS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_q8_append(cuda_lib, shape, runs):
    hq, hkv, d, P, rot, inter = shape
    c = Case(2, hq, hkv, d, P, 1024 // P, rot, RUNS[runs])
    (kc, ks), (vc, vs) = q8_cache(c), q8_cache(c)
    was = [x.view(torch.uint8).cpu().numpy() for x in (kc, ks, vc, vs)]
    q_out = bf16(c.rng, (c.T, hq, d)).cuda()
    before = q_out.clone()
    q, k, v, pos, cs, slots = c.args()
    cuda_lib.cpp_rope_kv_cache_write_q8(q, k, v, pos, cs, slots, kc, vc, ks, vs, q_out, c.err, interleaved=inter)
    c.check_q(q_out, before, inter)
    _, w = c.live()
    slots_w = np.where(w, c.slots, -1)
    tol = 2.0 ** -21 * pair_size(wide(k), rot, inter)
    check_q8(c, c.expected(k, inter), rot > 0, tol, kc, ks, was[0], was[1], slots_w)
    check_q8(c, wide(v), False, 0 * tol, vc, vs, was[2], was[3], slots_w)
    assert cuda_lib.cpp_read_device_error(c.err) == 0


@pytest.mark.parametrize("P", [8, 16, 64])
def test_q8_filled_token_by_token(cuda_lib, P):
    """Decode: one token a call, ever larger and then smaller, from an unwritten cache."""
    rng = np.random.default_rng(3)
    hkv, d, pages = 3, 128, 128 // P
    kc = torch.full((pages, hkv, P, d), 0x7F, dtype=torch.uint8, device="cuda")
    ks = torch.full((pages, hkv, P // min(16, P)), 255, dtype=torch.uint8, device="cuda")
    vc, vs = kc.clone(), ks.clone()
    want = [x.cpu().numpy().copy() for x in (kc, ks, vc, vs)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for t in range(41):
        k, v = (bf16(rng, (1, hkv, d), 4.0 ** ((t * 7) % 5 - 2)).cuda() for _ in range(2))
        slot = torch.tensor([t], device="cuda")
        cuda_lib.cpp_rope_kv_cache_write_q8(None, k, v, None, None, slot, kc, vc, ks, vs, None, err)
        A.append_q8(wide(k), [t], want[0], want[1])
        A.append_q8(wide(v), [t], want[2], want[3])
    for got, exp in zip((kc, ks, vc, vs), want):
        assert same_bytes(got.cpu().numpy(), exp)
    # and in one call: every block has the scale of its own largest value, none was rounded twice
    assert cuda_lib.cpp_read_device_error(err) == 0


@pytest.mark.parametrize("d", [64, 128])
def test_q8_values_at_the_ends_of_the_range(cuda_lib, d):
    """Zeros, the smallest and largest bf16, infinities and NaN, one kind a block."""
    inf, nan, big = float("inf"), float("nan"), 3.38e38
    rows = [[0.0, -0.0], [1e-38, -3e-39], [big, -big], [inf, 1.0], [nan, -2.0], [inf, nan], [448.0, 2 ** -6],
            [449.0, 2 ** -6], [2 ** -30, 2 ** 30], [-inf, 0.0]]
    x = torch.tensor(rows).to(torch.bfloat16).repeat(1, d // 2)[:, None].contiguous().cuda()
    P = 16
    slots = np.arange(len(rows)) * P + (np.arange(len(rows)) == 3) * 4
    kc = torch.full((len(rows), 1, P, d), 0x38, dtype=torch.uint8, device="cuda")
    ks = torch.full((len(rows), 1, 1), 100, dtype=torch.uint8, device="cuda")
    vc, vs = kc.clone(), ks.clone()
    want, wscale = kc.cpu().numpy().copy(), ks.cpu().numpy().copy()
    A.append_q8(wide(x), slots, want, wscale)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cuda_lib.cpp_rope_kv_cache_write_q8(None, x, x, None, None, torch.from_numpy(slots).cuda(), kc, vc, ks, vs, None, err)
    for c, s in ((kc, ks), (vc, vs)):
        assert np.array_equal(s.cpu().numpy(), wscale)
        assert same_bytes(c.cpu().numpy(), want)


def test_q8_growth_by_many_steps(cuda_lib):
    """A block's scale grows by 0 to 60 steps at once: its bytes are rounded as if from their values."""
    P, d, n = 16, 64, 61
    rng = np.random.default_rng(4)
    kc = torch.from_numpy(rng.integers(0, 256, (n, 1, P, d)).astype(np.uint8)).cuda()
    ks = torch.full((n, 1, 1), 100, dtype=torch.uint8, device="cuda")
    vc, vs = kc.clone(), ks.clone()
    want, wscale = kc.cpu().numpy().copy(), ks.cpu().numpy().copy()
    x = torch.zeros(n, 1, d)
    x[:, 0, 3] = 448.0 * 2.0 ** torch.arange(-27, n - 27)
    x = x.to(torch.bfloat16).cuda()
    slots = np.arange(n) * P + 5
    A.append_q8(wide(x), slots, want, wscale)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cuda_lib.cpp_rope_kv_cache_write_q8(None, x, x, None, None, torch.from_numpy(slots).cuda(), kc, vc, ks, vs, None, err)
    assert wscale.min() == 100 and wscale.max() == 160
    for c, s in ((kc, ks), (vc, vs)):
        assert np.array_equal(s.cpu().numpy(), wscale)
        assert same_bytes(c.cpu().numpy(), want)


@pytest.mark.parametrize("q8", [False, True])
def test_flags_and_skipped_tokens(cuda_lib, q8):
    """Positions and slots out of range are flagged and skipped, padding is skipped, the rest is done."""
    runs = [(0, 3, 0), (1024, 1, 5), (20, 2, 600), (30, 1, -1), (-7, 1, 9), (40, 2, 598), (1 << 40, 1, 4)]
    c = Case(5, 4, 2, 64, 16, 64, 64, runs)
    q_out = bf16(c.rng, (c.T, 4, 64)).cuda()
    before = q_out.clone()
    q, k, v, pos, cs, slots = c.args()
    _, w = c.live()
    sl = np.where(w, c.slots, -1)
    if q8:
        (kc, ks), (vc, vs) = q8_cache(c), q8_cache(c)
        was = [x.view(torch.uint8).cpu().numpy() for x in (vc, vs)]
        cuda_lib.cpp_rope_kv_cache_write_q8(q, k, v, pos, cs, slots, kc, vc, ks, vs, q_out, c.err)
        check_q8(c, wide(v), False, np.zeros((c.T, 2, 64)), vc, vs, was[0], was[1], sl)
    else:
        kc, vc = (bf16(c.rng, (64, 2, 16, 64)).cuda() for _ in range(2))
        want = wide(vc)
        cuda_lib.cpp_rope_kv_cache_write(q, k, v, pos, cs, slots, kc, vc, q_out, c.err)
        want[sl[w] // 16, :, sl[w] % 16] = wide(v)[w]
        assert np.array_equal(wide(vc), want)
    c.check_q(q_out, before, False)
    flags = cuda_lib.cpp_read_device_error(c.err)
    assert flags == cuda_lib.DEV_SLOT_OUT_OF_RANGE | cuda_lib.DEV_POSITION_OUT_OF_RANGE


@pytest.mark.parametrize("q8", [False, True])
def test_no_position_outside_the_table_is_looked_up(cuda_lib, q8):
    """Positions far behind and far before the table, between tokens that are done: their rows of it are not read."""
    runs = [(0, 2, 0), (18, 1, 1 << 40), (19, 1, -(1 << 40)), (20, 5, 1), (40, 1, (1 << 62) + 5), (41, 1, -1), (42, 3, 2)]
    c = Case(11, 4, 2, 128, 16, 64, 128, runs, top=6)
    q_out = bf16(c.rng, (c.T, 4, 128)).cuda()
    before = q_out.clone()
    q, k, v, pos, cs, slots = c.args()
    _, w = c.live()
    sl = np.where(w, c.slots, -1)
    (kc, ks), (vc, vs) = q8_cache(c), q8_cache(c)
    if q8:
        was = [x.view(torch.uint8).cpu().numpy() for x in (vc, vs)]
        cuda_lib.cpp_rope_kv_cache_write_q8(q, k, v, pos, cs, slots, kc, vc, ks, vs, q_out, c.err)
        check_q8(c, wide(v), False, np.zeros((c.T, 2, 128)), vc, vs, was[0], was[1], sl)
    else:
        kc, vc = (bf16(c.rng, (64, 2, 16, 128)).cuda() for _ in range(2))
        want = wide(vc)
        cuda_lib.cpp_rope_kv_cache_write(q, k, v, pos, cs, slots, kc, vc, q_out, c.err)
        want[sl[w] // 16, :, sl[w] % 16] = wide(v)[w]
        assert np.array_equal(wide(vc), want)
    c.check_q(q_out, before, False)
    assert cuda_lib.cpp_read_device_error(c.err) == cuda_lib.DEV_POSITION_OUT_OF_RANGE


@pytest.mark.parametrize("q8", [False, True])
def test_strided_contiguous_and_in_place_agree(cuda_lib, q8):
    c = Case(6, 14, 2, 128, 16, 64, 96, RUNS["mixed"])
    q, k, v, pos, cs, slots = c.args()
    outs = []
    for form in ("strided", "contiguous", "in place"):
        qq, kk, vv = (q, k, v) if form == "strided" else (q.contiguous(), k.contiguous(), v.contiguous())
        q_out = qq if form == "in place" else torch.empty(c.T, 14, 128, dtype=torch.bfloat16, device="cuda")
        kc = torch.zeros(64, 2, 16, 128, dtype=torch.uint8 if q8 else torch.bfloat16, device="cuda")
        vc = kc.clone()
        if q8:
            ks = torch.full((64, 2, 1), 120, dtype=torch.uint8, device="cuda")
            vs = ks.clone()
            cuda_lib.cpp_rope_kv_cache_write_q8(qq, kk, vv, pos, cs, slots, kc, vc, ks, vs, q_out, c.err)
            outs.append([q_out, kc, vc, ks, vs])
        else:
            cuda_lib.cpp_rope_kv_cache_write(qq, kk, vv, pos, cs, slots, kc, vc, q_out, c.err)
            outs.append([q_out, kc, vc])
    ok = torch.from_numpy(c.live()[0]).cuda()
    for o in outs[1:]:
        assert torch.equal(o[0][ok], outs[0][0][ok])
        assert all(torch.equal(a, b) for a, b in zip(o[1:], outs[0][1:]))


@pytest.mark.parametrize("q8", [False, True])
def test_captured_on_another_stream_and_replayed(cuda_lib, q8):
    c = Case(7, 8, 2, 128, 16, 64, 128, RUNS["prompt"])
    q, k, v, pos, cs, slots = c.args()
    kc = torch.zeros(64, 2, 16, 128, dtype=torch.uint8 if q8 else torch.bfloat16, device="cuda")
    sc = torch.full((64, 2, 1), 120, dtype=torch.uint8, device="cuda")

    def go(kc, vc, ks, vs, out):
        if q8:
            cuda_lib.cpp_rope_kv_cache_write_q8(q, k, v, pos, cs, slots, kc, vc, ks, vs, out, c.err)
        else:
            cuda_lib.cpp_rope_kv_cache_write(q, k, v, pos, cs, slots, kc, vc, out, c.err)

    a = [kc.clone(), kc.clone(), sc.clone(), sc.clone(), torch.zeros_like(q.contiguous())]
    b = [x.clone() for x in a]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        go(*b)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        go(*b)
    fresh = bf16(c.rng, (c.T, 12 * 128)).cuda()
    q.copy_(fresh[:, :1024].unflatten(1, (8, 128)))
    k.copy_(fresh[:, 1024:1280].unflatten(1, (2, 128)))
    v.copy_(fresh[:, 1280:].unflatten(1, (2, 128)))
    g.replay()
    torch.cuda.synchronize()
    go(*a)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_slots_in_any_order(cuda_lib):
    """bf16: any order. 8 bits: every token a block of its own, descending."""
    n, P = 40, 16
    rng = np.random.default_rng(8)
    k, v = (bf16(rng, (n, 2, 64)).cuda() for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = rng.permutation(n)
    kc, vc = (torch.zeros(4, 2, P, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cuda_lib.cpp_rope_kv_cache_write(None, k, v, None, None, torch.from_numpy(slots).cuda(), kc, vc, None, err)
    assert np.array_equal(wide(vc)[slots // P, :, slots % P], wide(v))
    slots = np.arange(n)[::-1].copy() * P
    kc, vc = (torch.zeros(n, 2, P, 64, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(n, 2, 1, dtype=torch.uint8, device="cuda") for _ in range(2))
    want, wscale = vc.cpu().numpy().copy(), vs.cpu().numpy().copy()
    cuda_lib.cpp_rope_kv_cache_write_q8(None, k, v, None, None, torch.from_numpy(slots).cuda(), kc, vc, ks, vs, None, err)
    A.append_q8(wide(v), slots, want, wscale)
    assert same_bytes(vc.cpu().numpy(), want) and np.array_equal(vs.cpu().numpy(), wscale)


def test_duplicate_and_scattered_slots_touch_nothing_else(cuda_lib):
    """The documented unspecified cases: only the blocks that are named change."""
    P = 16
    slots = np.array([3, 3, 5, 40, 4, 41, 3, 40, 7])
    rng = np.random.default_rng(9)
    k = bf16(rng, (len(slots), 2, 128)).cuda()
    kc = torch.from_numpy(rng.integers(0, 127, (8, 2, P, 128)).astype(np.uint8)).cuda()
    ks = torch.full((8, 2, 1), 110, dtype=torch.uint8, device="cuda")
    vc, vs = kc.clone(), ks.clone()
    was = kc.clone()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cuda_lib.cpp_rope_kv_cache_write_q8(None, k, k, None, None, torch.from_numpy(slots).cuda(), kc, vc, ks, vs, None, err)
    others = [p for p in range(8) if p not in (0, 2)]
    for c, s in ((kc, ks), (vc, vs)):
        assert torch.equal(c[others], was[others]) and bool((s[others] == 110).all())


@pytest.mark.parametrize("q8", [False, True])
def test_cache_beyond_32_bit_offsets(cuda_lib, q8):
    """Places behind 2^32 bytes (and elements) of a cache."""
    P, hkv, d = 16, 8, 128
    pages = (1 << 32) // (P * hkv * d) + 3
    kind = torch.uint8 if q8 else torch.bfloat16
    kc = torch.zeros(pages, hkv, P, d, dtype=kind, device="cuda")
    vc = torch.zeros_like(kc)
    rng = np.random.default_rng(10)
    n = 20
    k, v = (bf16(rng, (n, hkv, d)).cuda() for _ in range(2))
    slots = np.arange(n) + (pages - 2) * P
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (None, k, v, None, None, torch.from_numpy(slots).cuda(), kc, vc)
    if q8:
        ks, vs = (torch.zeros(pages, hkv, 1, dtype=torch.uint8, device="cuda") for _ in range(2))
        cuda_lib.cpp_rope_kv_cache_write_q8(*args, ks, vs, None, err)
        want, wscale = vc[-2:].cpu().numpy() * 0, vs[-2:].cpu().numpy() * 0
        A.append_q8(wide(v), slots - (pages - 2) * P, want, wscale)
        assert same_bytes(vc[-2:].cpu().numpy(), want) and np.array_equal(vs[-2:].cpu().numpy(), wscale)
    else:
        cuda_lib.cpp_rope_kv_cache_write(*args, None, err)
        got = wide(vc[-2:]).transpose(0, 2, 1, 3).reshape(-1, hkv, d)
        assert np.array_equal(got[:n], wide(v))
    assert int((vc[:-2].view(torch.uint8) != 0).sum()) == 0
    assert cuda_lib.cpp_read_device_error(err) == 0


def test_no_tokens(cuda_lib):
    z = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    kc = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = torch.zeros(0, dtype=torch.int64, device="cuda")
    cuda_lib.cpp_rope_kv_cache_write(z, z, z, None, None, slots, kc, kc.clone(), z, err)
    assert not kc.any()
