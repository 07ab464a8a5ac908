"""Pages outside the cache: flagged, and their keys and values count as zeros, whatever else the call reads. The oracle
takes the same batch with a page of zeros in their place; nothing of what a kernel had in hand before shows."""
import dataclasses

import numpy as np
import pytest
import torch

import oracle
import q4_helpers
import q8_helpers
import workloads as W
from helpers import bf16_tensor_to_f64, to_dev, to_dev_bf16
from q8_helpers import close

pytestmark = pytest.mark.gpu

HEADS = [(32, 8, 128), (16, 4, 128), (8, 2, 64), (6, 3, 128), (16, 1, 64), (1, 1, 128), (24, 8, 64)]


class bf16_helpers:
    """draw, run and reference over a bf16 cache, as q8_helpers and q4_helpers have them."""

    @staticmethod
    def draw(spec):
        b = W.make_batch(spec, with_history=False)
        seen = np.zeros((b.num_pages, spec.page_size), bool)
        for r, n in enumerate(b.seq_lens):
            j = np.arange(n)
            seen[b.block_table[r, j // spec.page_size], j % spec.page_size] = True
        rng, caches = np.random.default_rng(spec.seed), []
        for _ in "kv":
            c = W.randn_bf16(rng, (b.num_pages, spec.num_kv_heads, spec.page_size, spec.head_dim))
            c.transpose(0, 2, 1, 3)[~seen] = W.BF16_NAN_SENTINEL
            caches.append(c)
        return b, caches

    @staticmethod
    def run(cpsa, batch, caches, max_kv_splits=8, block_table=None):
        s, T = batch.spec, batch.num_tokens
        ws = torch.empty(cpsa.cpp_attn_workspace_bytes(len(s.qlen), T, s.num_q_heads, s.num_kv_heads, s.head_dim,
                                                       max_kv_splits), dtype=torch.uint8, device="cuda")
        out = torch.full((T, s.num_q_heads, s.head_dim), float("nan"), dtype=torch.bfloat16, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        cpsa.cpp_chunked_prefill_attn(to_dev_bf16(batch.q), *map(to_dev_bf16, caches), to_dev(batch.query_lens),
                                      to_dev(batch.seq_lens), to_dev(block_table), out, ws, err,
                                      max_kv_splits=max_kv_splits)
        return bf16_tensor_to_f64(out), cpsa.cpp_read_device_error(err)

    @staticmethod
    def reference(batch, caches):
        s = batch.spec
        ref = oracle.paged_attention(batch.q, *caches, batch.query_lens, batch.seq_lens, batch.block_table)
        v64, vmax = W.bf16_bits_to_f32(caches[1]).astype(np.float64), []
        for r, (ql, n) in enumerate(zip(batch.query_lens, batch.seq_lens)):
            j = np.arange(n)
            m = np.abs(v64[batch.block_table[r, j // s.page_size], :, j % s.page_size]).max((0, 2))
            vmax += [np.repeat(m, s.num_q_heads // s.num_kv_heads)] * int(ql)
        return ref, np.array(vmax)[..., None]


def with_zero_page(batch, caches, bad):
    """(the batch's table with the entries `bad` [(request, page number, what stands there)], the batch and caches that
    the oracle takes: a page of zeros more, which those entries name)."""
    table, zeros = batch.block_table.copy(), batch.block_table.copy()
    for r, i, x in bad:
        table[r, i], zeros[r, i] = x, batch.num_pages
    more = [np.concatenate([c, np.zeros_like(c[:1])]) for c in caches]
    return table, dataclasses.replace(batch, block_table=zeros, num_pages=batch.num_pages + 1), more


def bad_entries(batch):
    """Of every second request the first page, the last and every third in between."""
    s, out = batch.spec, []
    for r in range(0, len(s.qlen), 2):
        n = -(-int(batch.seq_lens[r]) // s.page_size)
        out += [(r, i, (batch.num_pages, -1, -5, 2 ** 31 - 1, -2 ** 31)[(r + i) % 5]) for i in range(n) if i % 3 == 0 or i == n - 1]
    return out


def check(cpsa, helpers, spec, max_kv_splits=8):
    b, caches = helpers.draw(spec)
    table, bz, cz = with_zero_page(b, caches, bad_entries(b))
    got, flags = helpers.run(cpsa, b, caches, max_kv_splits=max_kv_splits, block_table=table)
    assert flags == cpsa.DEV_PAGE_OUT_OF_RANGE
    ref, vmax = helpers.reference(bz, cz)
    seen = np.broadcast_to(vmax > 0, ref.shape).any((1, 2))     # rows with a page: of the others nothing but zeros is due
    assert not ref[~seen].any() and not got[~seen].any()
    if seen.any():
        close(got[seen], ref[seen], vmax[seen], str(spec))


@pytest.mark.parametrize("P", [8, 16, 64, 256])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_4_bit_decode_rows(cuda_lib, hq, hkv, d, P):
    """Rows of several lengths, so that a stage has held another row's places before; behind the ends stands NaN."""
    spec = W.BatchSpec(hist=[2999, 700, 1500, 60, 5000], qlen=[1] * 5, num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                       page_size=P, seed=10 + hq + P)
    check(cuda_lib, q4_helpers, spec)
    check(cuda_lib, q4_helpers, spec, max_kv_splits=1)


@pytest.mark.parametrize("n", [1, 40, 900, 6000])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_4_bit_single_row(cuda_lib, hq, hkv, d, n):
    check(cuda_lib, q4_helpers, W.BatchSpec(hist=[n - 1], qlen=[1], num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                                            page_size=16, seed=40 + hq + n))


@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_4_bit_chunks_beside_decode_rows(cuda_lib, hq, hkv, d):
    check(cuda_lib, q4_helpers, W.BatchSpec(hist=[700, 300, 33, 0, 900], qlen=[130, 1, 1, 200, 1], num_q_heads=hq,
                                            num_kv_heads=hkv, head_dim=d, page_size=16, seed=70 + hq))


def test_4_bit_many_rows(cuda_lib):
    """Enough rows for equal runs a CTA, each over several rows."""
    r = np.random.default_rng(5)
    check(cuda_lib, q4_helpers, W.BatchSpec(hist=[int(x) for x in r.integers(1, 900, 200)], qlen=[1] * 200, num_q_heads=8,
                                            num_kv_heads=2, head_dim=128, page_size=16, seed=90))


@pytest.mark.parametrize("P", [8, 16, 64, 256])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_8_bit_decode_rows(cuda_lib, hq, hkv, d, P):
    check(cuda_lib, q8_helpers, W.BatchSpec(hist=[2999, 700, 1500, 60, 5000], qlen=[1] * 5, num_q_heads=hq,
                                            num_kv_heads=hkv, head_dim=d, page_size=P, seed=110 + hq + P))


@pytest.mark.parametrize("n", [1, 40, 900, 6000])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_8_bit_single_row(cuda_lib, hq, hkv, d, n):
    check(cuda_lib, q8_helpers, W.BatchSpec(hist=[n - 1], qlen=[1], num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                                            page_size=16, seed=140 + hq + n))


@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_8_bit_chunks_beside_decode_rows(cuda_lib, hq, hkv, d):
    check(cuda_lib, q8_helpers, W.BatchSpec(hist=[700, 300, 33, 0, 900], qlen=[130, 1, 1, 200, 1], num_q_heads=hq,
                                            num_kv_heads=hkv, head_dim=d, page_size=16, seed=170 + hq))


@pytest.mark.parametrize("P", [8, 16, 64, 256])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_bf16_decode_rows(cuda_lib, hq, hkv, d, P):
    spec = W.BatchSpec(hist=[2999, 700, 1500, 60, 5000], qlen=[1] * 5, num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                       page_size=P, seed=210 + hq + P)
    check(cuda_lib, bf16_helpers, spec)
    check(cuda_lib, bf16_helpers, spec, max_kv_splits=1)


@pytest.mark.parametrize("n", [1, 40, 900, 6000])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_bf16_single_row(cuda_lib, hq, hkv, d, n):
    check(cuda_lib, bf16_helpers, W.BatchSpec(hist=[n - 1], qlen=[1], num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                                              page_size=16, seed=240 + hq + n))


@pytest.mark.parametrize("P", [8, 16, 64, 256])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_bf16_chunks_beside_decode_rows(cuda_lib, hq, hkv, d, P):
    check(cuda_lib, bf16_helpers, W.BatchSpec(hist=[700, 300, 33, 0, 900], qlen=[130, 1, 1, 200, 1], num_q_heads=hq,
                                              num_kv_heads=hkv, head_dim=d, page_size=P, seed=270 + hq + P))


@pytest.mark.parametrize("P", [16, 128])
@pytest.mark.parametrize("helpers", [bf16_helpers, q8_helpers, q4_helpers], ids=["bf16", "8 bit", "4 bit"])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_one_long_chunk(cuda_lib, hq, hkv, d, helpers, P):
    """One request, which plans itself; its tiles' slots are used many times over."""
    check(cuda_lib, helpers, W.BatchSpec(hist=[2500], qlen=[333], num_q_heads=hq, num_kv_heads=hkv, head_dim=d, page_size=P,
                                         seed=300 + hq + P))


@pytest.mark.parametrize("P", [8, 16, 128])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_fused_write(cuda_lib, hq, hkv, d, P):
    """With the KV write fused: the history's bad pages count as zeros, the new rows are the call's own, also where the table
    has a bad page for them."""
    spec = W.BatchSpec(hist=[700, 300, 33, 0, 900], qlen=[130, 1, 1, 200, 1], num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                       page_size=P, seed=400 + hq + P)
    b, caches = bf16_helpers.draw(spec)
    table = b.block_table.copy()
    whole = dataclasses.replace(b, block_table=b.block_table.copy())
    more = []
    for n, (r, i, x) in enumerate(bad_entries(b)):          # a page of zeros for each
        table[r, i], whole.block_table[r, i] = x, b.num_pages + n
        more.append(np.zeros_like(caches[0][:1]))
    ref_caches = [np.concatenate([c] + more) for c in caches]
    at = np.concatenate([[0], np.cumsum(spec.qlen)])
    for r, (h, n) in enumerate(zip(spec.hist, spec.qlen)):
        j = np.arange(h, h + n)
        for c, new in zip(ref_caches, (b.k, b.v)):
            c[whole.block_table[r, j // P], :, j % P] = new[at[r]:at[r + 1]]
    T, s = b.num_tokens, spec
    ws = torch.empty(cuda_lib.cpp_attn_workspace_bytes(5, T, hq, hkv, d, 8), dtype=torch.uint8, device="cuda")
    out = torch.full((T, hq, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kc, vc = map(to_dev_bf16, caches)
    cuda_lib.cpp_chunked_prefill_attn_write_kv(to_dev_bf16(b.q), to_dev_bf16(b.k), to_dev_bf16(b.v), to_dev(b.slot_mapping),
                                               kc, vc, to_dev(b.query_lens), to_dev(b.seq_lens), to_dev(table), out, ws, err)
    got = bf16_tensor_to_f64(out)
    assert cuda_lib.cpp_read_device_error(err) == cuda_lib.DEV_PAGE_OUT_OF_RANGE
    ref, vmax = bf16_helpers.reference(whole, ref_caches)
    close(got, ref, vmax, str(spec))
