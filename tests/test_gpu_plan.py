"""Work lists of batches on both sides of the plan's choices (one warp, a warp a request, the block; a thread a run
boundary): checked by the attention that runs over them, against the fp64 oracle."""
import numpy as np
import pytest

import q4_helpers
import q8_helpers
import workloads as W
from helpers import compare, oracle_caches, run_gpu_batch

import oracle

pytestmark = pytest.mark.gpu


def spec(hist, qlen, hq=4, hkv=2, d=64, P=16, seed=1):
    return W.BatchSpec(hist=list(hist), qlen=list(qlen), num_q_heads=hq, num_kv_heads=hkv, head_dim=d, page_size=P, seed=seed)


def check_bf16(cpsa, s, max_kv_splits=8):
    b = W.make_batch(s)
    got, flags, _, _ = run_gpu_batch(cpsa, b, max_kv_splits=max_kv_splits)
    assert flags == 0
    compare(got, oracle.paged_attention(b.q, *oracle_caches(b), b.query_lens, b.seq_lens, b.block_table), what=str(s))


CHECKS = {"bf16": check_bf16, "8 bit": lambda c, s, **kw: q8_helpers.check(c, s, **kw),
          "4 bit": lambda c, s, **kw: q4_helpers.check(c, s, **kw)}


@pytest.mark.parametrize("kind", CHECKS)
@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 31, 32, 33, 40])
@pytest.mark.parametrize("where", ["first", "last", "middle"])
def test_one_large_chunk_beside_decode_rows(cuda_lib, n, where, kind):
    """The units of one request, cut by most of the run boundaries, ahead of the others' entries, behind and between them."""
    r = np.random.default_rng(n)
    hist, qlen = [int(x) for x in r.integers(0, 300, n - 1)], [1] * (n - 1)
    at = {"first": 0, "last": n - 1, "middle": n // 2}[where]
    hist.insert(at, 700)
    qlen.insert(at, 900)
    CHECKS[kind](cuda_lib, spec(hist, qlen, hq=8, hkv=8, seed=20 + n))


@pytest.mark.parametrize("kind", CHECKS)
@pytest.mark.parametrize("splits", [1, 8])
@pytest.mark.parametrize("n", [2, 3, 4, 9, 32, 33, 70])
def test_ragged_prompts(cuda_lib, n, splits, kind):
    """Prompts and chunks of any length, requests without tokens among them, units whole and cut."""
    r = np.random.default_rng(100 + n)
    qlen = [int(x) for x in r.integers(0, 3, n) * r.integers(1, 6000 // n, n)]
    qlen[0], qlen[-1] = 2, 0
    hist = [int(x) for x in r.integers(0, 2, n) * r.integers(0, 900, n)]
    CHECKS[kind](cuda_lib, spec(hist, qlen, hq=6, hkv=3, seed=200 + n), max_kv_splits=splits)


@pytest.mark.parametrize("kind", CHECKS)
@pytest.mark.parametrize("n", [3, 4, 32, 33])
def test_many_units_a_token(cuda_lib, n, kind):
    """Chunks of a few tokens and many heads: a unit for every two or three rows."""
    CHECKS[kind](cuda_lib, spec([50 + i for i in range(n)], [2 + i % 3 for i in range(n)], hq=64, hkv=64, seed=300 + n))


@pytest.mark.parametrize("kind", CHECKS)
def test_more_requests_than_a_block_has_threads(cuda_lib, kind):
    """The second thousand of requests goes on where the first ended, inside a run."""
    r = np.random.default_rng(7)
    qlen = [int(x) for x in r.choice([0, 1, 1, 2, 3], 1100)]
    qlen[1020:1030] = [150] * 10
    CHECKS[kind](cuda_lib, spec([int(x) for x in r.integers(0, 40, 1100)], qlen, hq=2, hkv=1, seed=400))
