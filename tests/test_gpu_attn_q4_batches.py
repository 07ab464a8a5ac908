"""Batches over an 4-bit cache in which every CTA works off several items, against the fp64
oracle (tolerances: q4_helpers.py): decode batches of more items than SMs for every number of
kv heads an item can hold, rows of one key beside rows of several splits, and mixed batches
of more requests and tokens than one warp plans."""
import numpy as np
import pytest

import workloads as W
from q4_helpers import check, draw, reference, run
from q8_helpers import close

pytestmark = pytest.mark.gpu


def rows(n, seed, long=3000):
    """Lengths before the new token: a third of 0 to 19, most of the rest to 700, every eighth to `long`."""
    rng = np.random.default_rng(seed)
    kind = np.arange(n) % 8
    return [int(rng.integers(0, 20)) if k in (1, 4, 6) else int(rng.integers(1025, long)) if k == 7
            else int(rng.integers(0, 700)) for k in kind]


# (rows, q heads, kv heads): items of 8, 4, 2 and 1 kv heads; groups of up to 8 q heads and above
DECODE = [(400, 16, 8), (170, 72, 8), (200, 16, 4), (110, 24, 12), (160, 48, 4), (180, 14, 2), (120, 24, 6),
          (170, 24, 2), (330, 4, 1), (120, 9, 3), (170, 16, 1)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,hq,hkv", DECODE)
def test_decode_batches_of_several_items_a_cta(cuda_lib, n, hq, hkv, d):
    P = (8, 16, 32, 64, 256)[(n + hq + hkv) % 5]
    check(cuda_lib, W.BatchSpec(hist=rows(n, n + hq), qlen=[1] * n, num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                                page_size=P, seed=4000 + n + hq + d), spread=12)


@pytest.mark.parametrize("splits", [1, 3, 32])
def test_decode_batch_split_otherwise(cuda_lib, splits):
    n = 200
    check(cuda_lib, W.BatchSpec(hist=rows(n, 7, long=6000), qlen=[1] * n, num_q_heads=8, num_kv_heads=4, head_dim=128,
                                page_size=16, seed=4100), max_kv_splits=splits)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(32, 8), (14, 2), (4, 4), (24, 2)])
def test_mixed_batches_of_many_requests(cuda_lib, hq, hkv, d):
    """30 decode rows, a request without new tokens and 14 chunks: several units a CTA, in turn with short ones."""
    rng = np.random.default_rng(hq + d)
    qlen = [1] * 30 + [0] + [int(x) for x in rng.integers(2, 420, 14)]
    hist = rows(30, hq) + [5] + [int(x) * int(rng.integers(0, 2)) for x in rng.integers(1, 900, 14)]
    check(cuda_lib, W.BatchSpec(hist=hist, qlen=qlen, num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                                page_size=(16, 64)[d == 64], seed=4200 + hq), spread=20)


@pytest.mark.parametrize("d,hq,hkv", [(128, 16, 4), (64, 7, 1)])
def test_more_tokens_than_one_warp_plans(cuda_lib, d, hq, hkv):
    """A few requests of more than 8192 tokens together (sampled rows), and decode rows."""
    qlen = [1, 4000, 1, 3777, 700, 1]
    b, caches = draw(W.BatchSpec(hist=[2000, 0, 17, 300, 1111, 0], qlen=qlen, num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                                 page_size=32, seed=4300 + hq))
    got, flags = run(cuda_lib, b, caches)
    assert flags == 0 and np.all(np.isfinite(got))
    at = np.r_[0, 1:4001:37, 4000, 4001, 4002:7779:41, 7778, 7779:8479:13, 8478, 8479]
    ref, vmax = reference(b, caches, rows=at)
    close(got[at], ref, vmax)


@pytest.mark.parametrize("n,hq,hkv,d", [(1500, 4, 1, 64), (1100, 6, 6, 128), (2100, 2, 2, 64)])
def test_more_rows_than_one_pass_of_the_plan(cuda_lib, n, hq, hkv, d):
    """Decode rows beside requests without tokens, more than 1024 requests; one row much longer than the others."""
    rng = np.random.default_rng(n)
    hist, qlen = [int(x) for x in rng.integers(0, 130, n)], [1] * n
    hist[n // 2] = 9000
    for i in range(5, n, 97):
        qlen[i] = 0
    check(cuda_lib, W.BatchSpec(hist=hist, qlen=qlen, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, page_size=16,
                                seed=4400 + n))


@pytest.mark.parametrize("n,hq,hkv", [(160, 8, 8), (60, 12, 6), (90, 16, 1)])
@pytest.mark.parametrize("prompts", [0, 2])
def test_rows_in_whole_where_partials_do_not_fit(cuda_lib, n, hq, hkv, prompts):
    hist, qlen = rows(n, n) + [300] * prompts, [1] * n + [140] * prompts
    T = n + 140 * prompts
    small = cuda_lib.cpp_attn_workspace_min_bytes(n + prompts, T, hq, hkv, 128, 8)
    check(cuda_lib, W.BatchSpec(hist=hist, qlen=qlen, num_q_heads=hq, num_kv_heads=hkv, head_dim=128, page_size=32,
                                seed=4500 + n), workspace_bytes=small, expect_flags=cuda_lib.DEV_SPLITS_CLAMPED)


@pytest.mark.parametrize("splits", [1, 2, 8])
def test_rows_of_equal_and_of_one_length(cuda_lib, splits):
    """Runs that end where rows do, and rows of one key."""
    for hist in ([127] * 304, [0] * 200, [4095] * 80, [63] * 151 + [20000]):
        check(cuda_lib, W.BatchSpec(hist=hist, qlen=[1] * len(hist), num_q_heads=8, num_kv_heads=8, head_dim=64,
                                    page_size=64, seed=4600 + len(hist)), max_kv_splits=splits)


def test_invalid_rows_among_many(cuda_lib):
    """Rows that are refused take no part; the others come out as they should."""
    n = 120
    b, caches = draw(W.BatchSpec(hist=rows(n, 3), qlen=[1] * n, num_q_heads=8, num_kv_heads=8, head_dim=128, page_size=16,
                                 seed=4700))
    ref, vmax = reference(b, caches)
    b.seq_lens[7] = 0
    b.seq_lens[50] = 1 << 20
    got, flags = run(cuda_lib, b, caches)
    assert flags == cuda_lib.DEV_SEQ_LT_QUERY | cuda_lib.DEV_SEQ_GT_TABLE
    keep = np.delete(np.arange(n), [7, 50])
    close(got[keep], ref[keep], vmax[keep])
    assert np.isnan(got[[7, 50]]).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(32, 8), (8, 8), (48, 8), (72, 8), (16, 16), (12, 4)])
def test_few_rows_with_fewer_heads_an_item(cuda_lib, hq, hkv, d):
    """Rows few enough that an item holds 4, 2 or 1 of the heads that one of more rows would: each number of
    rows with each number of splits has its own, up to the one row more that has all of them."""
    for n, splits in ((1, 1), (1, 8), (2, 32), (3, 8), (4, 2), (5, 8), (9, 8), (10, 8), (19, 4), (37, 1), (38, 2)):
        check(cuda_lib, W.BatchSpec(hist=rows(n, n + hq, long=4000), qlen=[1] * n, num_q_heads=hq, num_kv_heads=hkv,
                                    head_dim=d, page_size=(16, 64, 256)[(n + hkv) % 3], seed=4600 + n + hq + d),
              max_kv_splits=splits, spread=12)


def test_a_few_rows_beside_a_chunk(cuda_lib):
    check(cuda_lib, W.BatchSpec(hist=[5000, 3, 900, 0], qlen=[1, 1, 300, 1], num_q_heads=32, num_kv_heads=8,
                                head_dim=128, page_size=16, seed=4700))
