"""Work lists of batches on both sides of the plan's choices (one warp, a warp a request, the block; a thread a run
boundary): checked by the attention that runs over them, against the fp64 oracle."""
import numpy as np
import pytest
import torch

import q4_helpers
import q8_helpers
import workloads as W
from helpers import bf16_tensor_to_f64, compare, oracle_caches, run_gpu_batch, to_dev, to_dev_bf16

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


@pytest.mark.parametrize("hist,qlen", [([100, 900, 0, 40, 700, 0], [1, 300, 5, 1, 200, 129]), ([100, 900, 40], [1, 300, 77])])
def test_captured_and_replayed_with_other_lengths(cuda_lib, hist, qlen):
    """The lists are made anew by every replay: the same requests in another order, with two calls at once on two streams."""
    batches = [W.make_batch(spec(hist[i:] + hist[:i], qlen[i:] + qlen[:i], hq=8, hkv=4, seed=500 + i)) for i in range(3)]
    b0, T, B = batches[0], sum(qlen), len(qlen)
    blocks = max(b.block_table.shape[1] for b in batches)
    pages = max(b.num_pages for b in batches)
    sets = []
    for _ in range(2):
        sets.append(dict(q=torch.zeros(T, 8, 64, dtype=torch.bfloat16, device="cuda"), kc=torch.zeros(pages, 4, 16, 64, dtype=torch.bfloat16, device="cuda"),
                         vc=torch.zeros(pages, 4, 16, 64, dtype=torch.bfloat16, device="cuda"), ql=torch.zeros(B, dtype=torch.int32, device="cuda"),
                         sl=torch.zeros(B, dtype=torch.int32, device="cuda"), bt=torch.zeros(B, blocks, dtype=torch.int32, device="cuda"),
                         out=torch.zeros(T, 8, 64, dtype=torch.bfloat16, device="cuda"), err=torch.zeros(1, dtype=torch.int32, device="cuda"),
                         ws=torch.empty(cuda_lib.cpp_attn_workspace_bytes(B, T, 8, 4, 64, 8), dtype=torch.uint8, device="cuda"),
                         stream=torch.cuda.Stream(), graph=torch.cuda.CUDAGraph()))

    def fill(x, b):
        kc, vc = oracle_caches(b)
        x["q"].copy_(to_dev_bf16(b.q))
        x["kc"][:b.num_pages].copy_(to_dev_bf16(kc))
        x["vc"][:b.num_pages].copy_(to_dev_bf16(vc))
        x["ql"].copy_(to_dev(b.query_lens))
        x["sl"].copy_(to_dev(b.seq_lens))
        x["bt"].fill_(-1)[:, :b.block_table.shape[1]].copy_(to_dev(b.block_table))
        x["out"].fill_(float("nan"))
        return oracle.paged_attention(b.q, kc, vc, b.query_lens, b.seq_lens, b.block_table)

    for x in sets:
        fill(x, b0)
        torch.cuda.synchronize()
        with torch.cuda.graph(x["graph"], stream=x["stream"]):
            cuda_lib.cpp_chunked_prefill_attn(x["q"], x["kc"], x["vc"], x["ql"], x["sl"], x["bt"], x["out"], x["ws"], x["err"])
    for i in range(3):
        refs = [fill(x, batches[(i + k) % 3]) for k, x in enumerate(sets)]
        torch.cuda.synchronize()
        for x in sets:
            with torch.cuda.stream(x["stream"]):
                x["graph"].replay()
        torch.cuda.synchronize()
        for x, ref in zip(sets, refs):
            assert cuda_lib.cpp_read_device_error(x["err"]) == 0
            compare(bf16_tensor_to_f64(x["out"]), ref)
