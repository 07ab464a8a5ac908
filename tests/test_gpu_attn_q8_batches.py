"""Batches over an 8-bit cache in which every CTA works off several items, against the fp64
oracle (tolerances: q8_helpers.py): decode batches of more items than SMs for every number of
kv heads an item can hold, rows of one key beside rows of several splits, and mixed batches
of more requests and tokens than one warp plans."""
import numpy as np
import pytest

import workloads as W
from q8_helpers import check, close, draw, reference, run

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
                                page_size=P, seed=3000 + n + hq + d), spread=2)


@pytest.mark.parametrize("splits", [1, 3, 32])
def test_decode_batch_split_otherwise(cuda_lib, splits):
    n = 200
    check(cuda_lib, W.BatchSpec(hist=rows(n, 7, long=6000), qlen=[1] * n, num_q_heads=8, num_kv_heads=4, head_dim=128,
                                page_size=16, seed=3100), max_kv_splits=splits)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(32, 8), (14, 2), (4, 4), (24, 2)])
def test_mixed_batches_of_many_requests(cuda_lib, hq, hkv, d):
    """30 decode rows, a request without new tokens and 14 chunks: several units a CTA, in turn with short ones."""
    rng = np.random.default_rng(hq + d)
    qlen = [1] * 30 + [0] + [int(x) for x in rng.integers(2, 420, 14)]
    hist = rows(30, hq) + [5] + [int(x) * int(rng.integers(0, 2)) for x in rng.integers(1, 900, 14)]
    check(cuda_lib, W.BatchSpec(hist=hist, qlen=qlen, num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                                page_size=(16, 64)[d == 64], seed=3200 + hq), spread=3)


@pytest.mark.parametrize("d,hq,hkv", [(128, 16, 4), (64, 7, 1)])
def test_more_tokens_than_one_warp_plans(cuda_lib, d, hq, hkv):
    """A few requests of more than 8192 tokens together (sampled rows), and decode rows."""
    qlen = [1, 4000, 1, 3777, 700, 1]
    b, caches = draw(W.BatchSpec(hist=[2000, 0, 17, 300, 1111, 0], qlen=qlen, num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                                 page_size=32, seed=3300 + hq))
    got, flags = run(cuda_lib, b, caches)
    assert flags == 0 and np.all(np.isfinite(got))
    at = np.r_[0, 1:4001:37, 4000, 4001, 4002:7779:41, 7778, 7779:8479:13, 8478, 8479]
    ref, vmax = reference(b, caches, rows=at)
    close(got[at], ref, vmax)
