"""Keys of the rotary appends, and their block scales, where the tokens around them are skipped, come in
another order, or lie behind 2^32 bytes (tolerances: test_gpu_rope_append.py)."""
import numpy as np
import pytest
import torch

from oracle import append as A
from test_gpu_rope_append import Case, bf16, check_q8, pair_size, q8_cache, same_bytes, wide

pytestmark = pytest.mark.gpu

SKIPPED = {
    "flagged and padded": (64, 600, [(0, 3, 0), (1024, 1, 5), (20, 2, 600), (30, 1, -1), (-7, 1, 9), (40, 2, 598),
                                     (1 << 40, 1, 4)]),
    "far outside the table": (128, 6, [(0, 2, 0), (18, 1, 1 << 40), (19, 1, -(1 << 40)), (20, 5, 1),
                                       (40, 1, (1 << 62) + 5), (41, 1, -1), (42, 3, 2)]),
    # behind a block's last token of the call, at a window's end, in front of the next block's
    "between blocks": (128, 50, [(16, 2, 16), (18, 1, -1), (32, 11, 32), (-2, 2, 9), (43, 1, 1 << 33), (48, 9, 40),
                                 (60, 1, 50), (64, 1, 3), (-1, 3, -1), (85, 4, 20)]),
}


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("kind", SKIPPED)
def test_keys_beside_skipped_tokens(cuda_lib, kind, q8, inter):
    d, top, runs = SKIPPED[kind]
    c = Case(21, 4, 2, d, 16, 64, d, runs, top=top)
    q_out = bf16(c.rng, (c.T, 4, d)).cuda()
    before = q_out.clone()
    q, k, v, pos, cs, slots = c.args()
    ok, w = c.live()
    # rows of the table for the tokens that are done alone
    c.pos = np.where(ok, c.pos, 0)
    want = c.expected(k, inter)
    tol = 2.0 ** -21 * pair_size(wide(k), d, inter)
    sl = np.where(w, c.slots, -1)
    if q8:
        (kc, ks), (vc, vs) = q8_cache(c), q8_cache(c)
        was = [x.view(torch.uint8).cpu().numpy() for x in (kc, ks, vc, vs)]
        cuda_lib.cpp_rope_kv_cache_write_q8(q, k, v, pos, cs, slots, kc, vc, ks, vs, q_out, c.err, interleaved=inter)
        check_q8(c, want, True, tol, kc, ks, was[0], was[1], sl)
        check_q8(c, wide(v), False, 0 * tol, vc, vs, was[2], was[3], sl)
    else:
        kc, vc = (bf16(c.rng, (64, 2, 16, d)).cuda() for _ in range(2))
        k0, v0 = wide(kc), wide(vc)
        cuda_lib.cpp_rope_kv_cache_write(q, k, v, pos, cs, slots, kc, vc, q_out, c.err, interleaved=inter)
        got, (page, off) = wide(kc), (sl[w] // 16, sl[w] % 16)
        assert np.all(np.abs(got[page, :, off] - want[w]) <= 2.0 ** -8 * np.abs(want[w]) + tol[w])
        got[page, :, off] = k0[page, :, off]
        assert np.array_equal(got, k0), "other places of the k cache changed"
        v0[page, :, off] = wide(v)[w]
        assert np.array_equal(wide(vc), v0)
    assert torch.equal(q_out.cpu().view(torch.int16)[~ok], before.cpu().view(torch.int16)[~ok])


def test_keys_with_slots_in_any_order(cuda_lib):
    n, P = 40, 16
    rng = np.random.default_rng(22)
    k, v = (bf16(rng, (n, 2, 64)).cuda() for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = rng.permutation(n)
    kc, vc = (torch.zeros(4, 2, P, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cuda_lib.cpp_rope_kv_cache_write(None, k, v, None, None, torch.from_numpy(slots).cuda(), kc, vc, None, err)
    want = np.zeros(kc.shape)
    want[slots // P, :, slots % P] = wide(k)
    assert np.array_equal(wide(kc), want)
    slots = np.arange(n)[::-1].copy() * P
    kc, vc = (torch.zeros(n, 2, P, 64, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(n, 2, 1, dtype=torch.uint8, device="cuda") for _ in range(2))
    want, wscale = kc.cpu().numpy().copy(), ks.cpu().numpy().copy()
    cuda_lib.cpp_rope_kv_cache_write_q8(None, k, v, None, None, torch.from_numpy(slots).cuda(), kc, vc, ks, vs, None, err)
    A.append_q8(wide(k), slots, want, wscale)
    assert same_bytes(kc.cpu().numpy(), want) and np.array_equal(ks.cpu().numpy(), wscale)
    assert cuda_lib.cpp_read_device_error(err) == 0


@pytest.mark.parametrize("q8", [False, True])
def test_keys_beyond_32_bit_offsets(cuda_lib, q8):
    P, hkv, d = 16, 8, 128
    pages = (1 << 32) // (P * hkv * d) + 3
    kc = torch.zeros(pages, hkv, P, d, dtype=torch.uint8 if q8 else torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    rng = np.random.default_rng(23)
    n = 20
    k, v = (bf16(rng, (n, hkv, d)).cuda() for _ in range(2))
    slots = np.arange(n) + (pages - 2) * P
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (None, k, v, None, None, torch.from_numpy(slots).cuda(), kc, vc)
    if q8:
        ks, vs = (torch.zeros(pages, hkv, 1, dtype=torch.uint8, device="cuda") for _ in range(2))
        cuda_lib.cpp_rope_kv_cache_write_q8(*args, ks, vs, None, err)
        want, wscale = kc[-2:].cpu().numpy() * 0, ks[-2:].cpu().numpy() * 0
        A.append_q8(wide(k), slots - (pages - 2) * P, want, wscale)
        assert same_bytes(kc[-2:].cpu().numpy(), want) and np.array_equal(ks[-2:].cpu().numpy(), wscale)
        assert not bool(ks[:-2].any())
    else:
        cuda_lib.cpp_rope_kv_cache_write(*args, None, err)
        got = wide(kc[-2:]).transpose(0, 2, 1, 3).reshape(-1, hkv, d)
        assert np.array_equal(got[:n], wide(k)) and not got[n:].any()
    assert not bool(kc[:-2].view(torch.uint8).any())
    assert cuda_lib.cpp_read_device_error(err) == 0
