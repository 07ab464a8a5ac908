"""GPU parity of cpp_chunked_prefill_attn_q4 against the fp64 oracle (tolerances: q4_helpers.py, q8_helpers.py)."""
import numpy as np
import pytest
import torch

import workloads as W
from helpers import to_dev, to_dev_bf16
from oracle import q4
from q4_helpers import check, draw, reference, run
from q8_helpers import bf16_bits, close

pytestmark = pytest.mark.gpu


def spec(hist, qlen, hq=8, hkv=2, d=128, P=16, seed=1, **kw):
    return W.BatchSpec(hist=hist, qlen=qlen, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, page_size=P, seed=seed, **kw)


HEADS = [(4, 4), (8, 2), (32, 8), (6, 2), (16, 1), (14, 2), (12, 12), (1, 1)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", HEADS)
def test_heads_and_dims_mixed(cuda_lib, d, hq, hkv):
    check(cuda_lib, spec([130, 0, 7, 333], [200, 129, 1, 1], hq, hkv, d, seed=100 + hq + d))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", HEADS)
def test_heads_and_dims_decode(cuda_lib, d, hq, hkv):
    check(cuda_lib, spec([0, 1, 14, 15, 16, 17, 1200, 64], [1] * 8, hq, hkv, d, seed=150 + hq + d))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("P", [8, 16, 32, 64, 128, 256])
def test_page_sizes(cuda_lib, P, d):
    check(cuda_lib, spec([300, 1000, 0, 7], [77, 1, 260, 1], P=P, d=d, seed=200 + P, extra_pages=5))


@pytest.mark.parametrize("P", [8, 16, 256])
@pytest.mark.parametrize("n", [1, 2, 3, 15, 16, 17, 127, 128, 129, 255, 257])
def test_one_request_without_history(cuda_lib, n, P):
    check(cuda_lib, spec([0], [n], P=P, seed=300 + n))


@pytest.mark.parametrize("h", [1, 100, 127, 128, 129, 2047])
@pytest.mark.parametrize("n", [1, 2, 64, 130])
def test_one_request_with_history(cuda_lib, n, h):
    check(cuda_lib, spec([h], [n], hq=4, hkv=1, P=32, seed=400 + n + h))


def test_ragged_mixed_batch(cuda_lib):
    """Decode rows first, then chunks with ragged tails, a zero-length request inside."""
    check(cuda_lib, spec([900, 33, 4000, 0, 511, 512, 513, 0, 77], [1, 1, 1, 2, 128, 127, 129, 0, 383], hq=32, hkv=8,
                         seed=500))


@pytest.mark.parametrize("splits", [1, 2, 8, 32])
def test_long_history_splits(cuda_lib, splits):
    check(cuda_lib, spec([9000, 5000, 6000], [1, 150, 1], seed=600 + splits), max_kv_splits=splits)


@pytest.mark.parametrize("hkv", [1, 4, 8])
def test_long_single_rows(cuda_lib, hkv):
    """One decode row of 20001 keys, as a step of one user over a long context."""
    check(cuda_lib, spec([20000], [1], hq=4 * hkv, hkv=hkv, seed=650))


def test_small_workspace_clamps_the_splits(cuda_lib):
    s = spec([9000, 5000], [1, 150], seed=700)
    small = cuda_lib.cpp_attn_workspace_min_bytes(2, 151, 8, 2, 128, 8)
    check(cuda_lib, s, workspace_bytes=small, expect_flags=cuda_lib.DEV_SPLITS_CLAMPED)


@pytest.mark.parametrize("d,hq,hkv", [(128, 8, 2), (64, 14, 2), (128, 24, 24), (128, 16, 1)])
@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 128, 129, 1000, 5000])
def test_one_row_plans_itself(cuda_lib, n, d, hq, hkv):
    """One decode row: its splits, and one split where the workspace has no room for partial results."""
    s = spec([n - 1], [1], hq, hkv, d, P=32, seed=720 + n)
    for splits in (1, 3, 8, 32):
        check(cuda_lib, s, max_kv_splits=splits)
    small = cuda_lib.cpp_attn_workspace_min_bytes(1, 1, hq, hkv, d, 8)
    check(cuda_lib, s, workspace_bytes=small, expect_flags=cuda_lib.DEV_SPLITS_CLAMPED)


def test_one_row_that_is_refused_and_one_right_after(cuda_lib):
    """A single decode row's lengths that cannot be: flagged, its output left alone; the workspace serves the next call."""
    b, caches = draw(spec([700], [1], hq=8, hkv=2, seed=740))
    kc, ks, vc, vs = (to_dev(x) for x in caches)
    ws = torch.full((cuda_lib.cpp_attn_workspace_bytes(1, 1, 8, 2, 128, 8),), 0xAB, dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((1, 8, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    ref, vmax = reference(b, caches)
    q, bt = to_dev_bf16(b.q), to_dev(b.block_table)
    for ql, sl, want in ((2, 701, cuda_lib.DEV_TOKENS_MISMATCH), (0, 701, cuda_lib.DEV_TOKENS_MISMATCH),
                         (1, 0, cuda_lib.DEV_SEQ_LT_QUERY), (1, 1 << 20, cuda_lib.DEV_SEQ_GT_TABLE), (1, 701, 0),
                         (-3, 701, cuda_lib.DEV_TOKENS_MISMATCH), (1, -5, cuda_lib.DEV_SEQ_LT_QUERY)):
        out.fill_(5.0)
        lens = [torch.tensor([x], dtype=torch.int32, device="cuda") for x in (ql, sl)]
        cuda_lib.cpp_chunked_prefill_attn_q4(q, kc, vc, ks, vs, *lens, bt, out, ws, err)
        assert cuda_lib.cpp_read_device_error(err) == want
        if want:
            assert bool((out == 5.0).all())
        else:
            close(out.double().cpu().numpy(), ref, vmax)


@pytest.mark.parametrize("scale", [0.02, 1.0])
def test_custom_scale(cuda_lib, scale):
    check(cuda_lib, spec([300, 40, 90], [130, 70, 1], seed=800), scale=scale)


@pytest.mark.parametrize("spread", [24, 60])
def test_scales_far_apart(cuda_lib, spread):
    """Groups between 2^-3 and 2^3, 2^-7 and 2^7 of the usual scale: the largest keys and values dominate."""
    check(cuda_lib, spec([400, 700, 33], [150, 1, 1], seed=900 + spread), spread=spread)


@pytest.mark.parametrize("centre", [1, 226])
def test_scales_at_the_ends(cuda_lib, centre):
    """The smallest and the largest scales that the append stores (scores stay ordinary through the softmax scale)."""
    b, (kc, ks, vc, vs) = draw(spec([200, 600], [130, 1], seed=950 + centre))
    _, (_, ends, _, _) = draw(spec([200, 600], [130, 1], seed=950 + centre), centre=centre, spread=3)
    caches = (kc, ks, vc, ends)
    got, flags = run(cuda_lib, b, caches)
    ref, vmax = reference(b, caches)
    close(got, ref, vmax)
    caches, sc = (kc, ends, vc, vs), float(np.float32(0.3 / q4.SCALES[centre] / np.sqrt(128)))
    got, flags = run(cuda_lib, b, caches, scale=sc)
    ref, vmax = reference(b, caches, scale=sc)
    close(got, ref, vmax)


@pytest.mark.parametrize("kind", ["tiny", "huge", "one column"])
def test_queries_of_any_size(cuda_lib, kind):
    """Query rows far from 1: the softmax scale brings the scores back, or a single key wins."""
    b, caches = draw(spec([150, 300], [140, 1], seed=970))
    q = (b.q.astype(np.uint32) << 16).view(np.float32).copy()
    scale = 0.0
    if kind == "tiny":
        q, scale = q * np.float32(2.0 ** -90), float(2.0 ** 90 / np.sqrt(128))
    elif kind == "huge":
        q, scale = q * np.float32(2.0 ** 60), float(2.0 ** -60 / np.sqrt(128))
    else:
        q[..., 1:] *= np.float32(2.0 ** -20)
    q = bf16_bits(q.astype(np.float64))
    got, flags = run(cuda_lib, b, caches, scale=scale, q=q)
    assert flags == 0
    ref, vmax = reference(b, caches, scale=scale, q=q)
    close(got, ref, vmax, kind)


def test_scales_that_rise_and_fall_along_the_sequence(cuda_lib):
    """Value scales from 2^-8 up to 2^8 of the usual one along the keys, and down again."""
    b, (kc, ks, vc, vs) = draw(spec([1000, 1000], [200, 1], seed=980))
    for r in range(2):
        for j in range(int(b.seq_lens[r])):
            vs[b.block_table[r, j // 16], :, j % 16] = 106 + int(64 * np.sin(j / 90.0))
    caches = (kc, ks, vc, vs)
    got, flags = run(cuda_lib, b, caches)
    ref, vmax = reference(b, caches)
    assert flags == 0
    close(got, ref, vmax)


@pytest.mark.parametrize("q1", [1, 40])
def test_one_key_wins_with_small_values(cuda_lib, q1):
    """A row whose probability is all on a key of values 2^12 below the others': its output keeps its own precision."""
    b, (kc, ks, vc, vs) = draw(spec([600], [q1], hq=2, hkv=2, seed=990))
    q = np.zeros((q1, 2, 128))
    q[:, :, 5] = 64.0
    kc[:, :, :, 2] &= 0x0F                          # column 5, the high half of byte 2: zero
    page = b.block_table[0, 3]
    kc[page, :, 4, 2] |= 0x70                       # but for one key's 6
    ks[page, :, 4, 0] = 112
    vs[page] = 10
    q = bf16_bits(q)
    caches = (kc, ks, vc, vs)
    got, flags = run(cuda_lib, b, caches, q=q)
    ref, _ = reference(b, caches, q=q)
    assert flags == 0
    # the score is 64 * 6 * 0.5 / sqrt(128) = 16.97, the other 639 keys' probabilities e^-16.97 of values up to 3
    assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -9) * 640 * 3 * np.exp(-16.9))


@pytest.mark.parametrize("bad", [0, 5, 9])
def test_nan_in_a_live_place(cuda_lib, bad):
    """A NaN key poisons the rows that see it and no others; a NaN value its 16 columns of the rows that see it (and,
    as documented, may poison those columns of earlier rows of their request), no other column or request."""
    b, (kc, ks, vc, vs) = draw(spec([0, 100], [150, 1], hq=2, hkv=1, seed=1000 + bad))
    vs[b.block_table[0, (100 + bad) // 16], 0, (100 + bad) % 16, 3] = 255
    ks[b.block_table[0, (120 + bad) // 16], 0, (120 + bad) % 16, 1] = 255
    got, _ = run(cuda_lib, b, (kc, ks, vc, vs))
    nan = np.isnan(got)
    assert nan[120 + bad:150].all() and nan[100 + bad:120 + bad, :, 48:64].all()
    assert not nan[:120 + bad][..., np.r_[:48, 64:128]].any() and not nan[150:].any()


def test_scales_of_zero(cuda_lib):
    """Scale byte 0 (no number of the append's) holds zeros: scores of zero, values of zero."""
    b, (kc, ks, vc, vs) = draw(spec([70, 300], [60, 1], seed=1050))
    ks[ks != 255] = 0
    caches = (kc, ks, vc, vs)
    got, flags = run(cuda_lib, b, caches)
    ref, vmax = reference(b, caches)
    close(got, ref, vmax)
    vs[vs != 255] = 0
    got, _ = run(cuda_lib, b, caches)
    assert not got.any()


def test_two_calls_alike_and_with_another_workspace(cuda_lib):
    b, caches = draw(spec([3000, 9000, 20], [300, 1, 90], hq=32, hkv=8, seed=1100))
    a, _ = run(cuda_lib, b, caches)
    c, _ = run(cuda_lib, b, caches, workspace_bytes=(64 << 20) +
               cuda_lib.cpp_attn_workspace_bytes(3, 391, 32, 8, 128, 8))
    assert np.array_equal(a, c)


def test_invalid_pages_and_lengths_are_flagged(cuda_lib):
    b, caches = draw(spec([300, 40, 500, 200], [130, 1, 1, 60], seed=1200))
    bt = b.block_table.copy()
    bt[0, 2], bt[2, 5] = b.num_pages, -5
    got, flags = run(cuda_lib, b, caches, block_table=bt)
    assert flags == cuda_lib.DEV_PAGE_OUT_OF_RANGE
    ref, vmax = reference(b, caches)
    keep = np.r_[130, 132:192]
    close(got[keep], ref[keep], vmax[keep])
    b.seq_lens[1] = 0
    _, flags = run(cuda_lib, b, caches)
    assert flags == cuda_lib.DEV_SEQ_LT_QUERY
    b.seq_lens[1] = 1 << 20
    _, flags = run(cuda_lib, b, caches)
    assert flags == cuda_lib.DEV_SEQ_GT_TABLE
    b.query_lens[1] = 3
    b.seq_lens[1] = 41
    got, flags = run(cuda_lib, b, caches)
    assert flags == cuda_lib.DEV_TOKENS_MISMATCH and np.isnan(got).all()


@pytest.mark.parametrize("hist,qlen", [([2000], [300]), ([900, 5000, 64], [1, 1, 200]), ([5000] * 3, [1] * 3)])
def test_captured_and_replayed_on_another_stream(cuda_lib, hist, qlen):
    b, caches = draw(spec(hist, qlen, hq=8, hkv=4, seed=1300))
    T = b.num_tokens
    want, _ = run(cuda_lib, b, caches)
    kc, ks, vc, vs = (to_dev(x) for x in caches)
    q, lens = to_dev_bf16(b.q), [to_dev(x) for x in (b.query_lens, b.seq_lens, b.block_table)]
    ws = torch.empty(cuda_lib.cpp_attn_workspace_bytes(len(hist), T, 8, 4, 128, 8), dtype=torch.uint8, device="cuda")
    out = torch.empty(T, 8, 128, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    args = (q, kc, vc, ks, vs, *lens, out, ws, err)
    cuda_lib.cpp_chunked_prefill_attn_q4(*args, stream=s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        cuda_lib.cpp_chunked_prefill_attn_q4(*args)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(out.double().cpu().numpy(), want)
    assert cuda_lib.cpp_read_device_error(err) == 0


def test_two_graphs_that_share_a_workspace(cuda_lib):
    """Replayed in turn: neither the work lists nor the merge counters of one disturb the other."""
    batches = [draw(spec([3000], [300], hq=8, hkv=2, seed=1350)), draw(spec([2000, 900, 5000], [260, 1, 1], seed=1351))]
    want = [run(cuda_lib, *x)[0] for x in batches]
    size = max(cuda_lib.cpp_attn_workspace_bytes(len(b.spec.qlen), b.num_tokens, 8, 2, 128, 8) for b, _ in batches)
    ws = torch.full((size,), 0xAB, dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    jobs = []
    for b, caches in batches:
        kc, ks, vc, vs = (to_dev(x) for x in caches)
        out = torch.zeros(b.num_tokens, 8, 128, dtype=torch.bfloat16, device="cuda")
        args = (to_dev_bf16(b.q), kc, vc, ks, vs, to_dev(b.query_lens), to_dev(b.seq_lens), to_dev(b.block_table), out,
                ws, err)
        torch.cuda.synchronize()
        cuda_lib.cpp_chunked_prefill_attn_q4(*args, stream=side)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            cuda_lib.cpp_chunked_prefill_attn_q4(*args)
        jobs.append((g, out, args))
    for i in (0, 1, 1, 0, 1, 0, 0):
        g, out, _ = jobs[i]
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(out.double().cpu().numpy(), want[i])
    assert cuda_lib.cpp_read_device_error(err) == 0


def test_calls_of_another_device_are_refused(cuda_lib, monkeypatch):
    """Tensors and streams that are not the current device's (here: a current device that is not theirs)."""
    from chunked_prefill_paged_slot_gb300 import _lib
    b, caches = draw(spec([20], [3], hq=2, hkv=2, seed=1360))
    kc, ks, vc, vs = (to_dev(x) for x in caches)
    q = to_dev_bf16(b.q)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    monkeypatch.setattr(_lib.torch.cuda, "current_device", lambda: 1)
    with pytest.raises(cuda_lib.CpsaError, match="the current device is cuda:1"):
        cuda_lib.cpp_chunked_prefill_attn_q4(q, kc, vc, ks, vs, to_dev(b.query_lens), to_dev(b.seq_lens),
                                             to_dev(b.block_table), q.clone(), kc, err, stream=s)
    with pytest.raises(cuda_lib.CpsaError, match="the current device is cuda:1"):
        cuda_lib.cpp_rope_kv_cache_write_q4(None, q, q, None, None, to_dev(b.slot_mapping), kc, vc, ks, vs, None, err,
                                            stream=s)
    monkeypatch.undo()
    with pytest.raises(cuda_lib.CpsaError, match="q is on cuda:0, the current device is cuda:1"):
        _lib._ptr(q, torch.bfloat16, "q", 1)


def test_two_streams_with_their_own_workspaces(cuda_lib):
    one, two = draw(spec([3000, 100], [200, 1], seed=1400)), draw(spec([100, 4000, 5000], [150, 1, 1], seed=1401))
    want = [run(cuda_lib, *x)[0] for x in (one, two)]
    jobs = []
    for b, caches in (one, two):
        B, T = len(b.spec.qlen), b.num_tokens
        kc, ks, vc, vs = (to_dev(x) for x in caches)
        out = torch.empty(T, 8, 128, dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(cuda_lib.cpp_attn_workspace_bytes(B, T, 8, 2, 128, 8), dtype=torch.uint8, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        jobs.append((torch.cuda.Stream(), (to_dev_bf16(b.q), kc, vc, ks, vs, to_dev(b.query_lens), to_dev(b.seq_lens),
                                           to_dev(b.block_table), out, ws, err), out))
    torch.cuda.synchronize()
    for _ in range(20):
        for s, args, _ in jobs:
            cuda_lib.cpp_chunked_prefill_attn_q4(*args, stream=s)
    torch.cuda.synchronize()
    for (_, _, out), w in zip(jobs, want):
        assert np.array_equal(out.double().cpu().numpy(), w)


@pytest.mark.parametrize("qlen", [1, 130])
def test_pages_beyond_32_bit_offsets(cuda_lib, qlen):
    """The same sequence at the end of a cache of more than 2^32 bytes."""
    b, (kc, ks, vc, vs) = draw(spec([300], [qlen], hq=8, hkv=8, seed=1500))
    want, _ = run(cuda_lib, b, (kc, ks, vc, vs))
    n = kc.shape[0]
    pages = (1 << 32) // (8 * 16 * 64) + n
    big = []
    for x in (kc, ks, vc, vs):
        y = torch.zeros((pages, *x.shape[1:]), dtype=torch.uint8, device="cuda")
        y[pages - n:] = to_dev(x)
        big.append(y)
    out = torch.empty(qlen, 8, 128, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(cuda_lib.cpp_attn_workspace_bytes(1, qlen, 8, 8, 128, 8), dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    bt = np.where(b.block_table >= 0, b.block_table + pages - n, -1).astype(np.int32)
    cuda_lib.cpp_chunked_prefill_attn_q4(to_dev_bf16(b.q), big[0], big[2], big[1], big[3], to_dev(b.query_lens),
                                         to_dev(b.seq_lens), to_dev(bt), out, ws, err)
    assert np.array_equal(out.double().cpu().numpy(), want)


def test_random_batches(cuda_lib):
    rng = np.random.default_rng(1600)
    for i in range(12):
        n = int(rng.integers(1, 9))
        hist = [int(rng.integers(0, 1500)) * int(rng.integers(0, 2)) for _ in range(n)]
        qlen = [1 if rng.random() < 0.5 else int(rng.integers(0, 300)) for _ in range(n)]
        if not sum(qlen):
            qlen[0] = 2
        hq, hkv = HEADS[int(rng.integers(len(HEADS)))]
        check(cuda_lib, spec(hist, qlen, hq, hkv, int(rng.choice([64, 128])), int(rng.choice([8, 16, 32, 64, 128, 256])),
                             seed=1600 + i), spread=int(rng.integers(0, 30)))


def test_no_tokens(cuda_lib):
    q = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    c = torch.zeros(2, 2, 16, 32, dtype=torch.uint8, device="cuda")
    sc = torch.zeros(2, 2, 16, 4, dtype=torch.uint8, device="cuda")
    i32 = torch.zeros(0, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cuda_lib.cpp_chunked_prefill_attn_q4(q, c, c, sc, sc, i32, i32, i32.view(0, 0), q, c.view(-1), err)
    assert cuda_lib.cpp_read_device_error(err) == 0
