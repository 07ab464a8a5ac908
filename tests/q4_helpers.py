"""Seeded batches over a 4-bit cache, their run and their check (no arithmetic of the method here).

A stored number (code * scale) is exact in bf16, so the fp64 oracle for bf16 caches takes the
very values that the 4-bit cache holds. Tolerance of attention: as in q8_helpers.py.
"""
from __future__ import annotations

import numpy as np
import torch

import oracle
import workloads as W
from helpers import bf16_tensor_to_f64, to_dev, to_dev_bf16
from oracle import q4
from q8_helpers import bf16_bits, close


def check_group_values(x, tol, cache, scale):
    """cache [..., d / 2], scale [..., d / 16] bytes against the exact values x [..., d], each known to within tol before
    its rounding: the scale is that of an amax so far off at most, a code within half a step (and that tol) of value / scale."""
    g = lambda a: a.reshape(-1, q4.GROUP)
    x, tol, code, byte = g(x), g(np.broadcast_to(tol, x.shape)), g(q4.unpacked(cache)), scale.reshape(-1)
    for v, t, c, b in zip(x, tol, code, byte):
        if not np.all(np.isfinite(v)):
            assert b == q4.NAN_SCALE
            continue
        amax, off = np.abs(v).max(), t.max()
        assert q4.to_scale(max(amax - off, 0.0)) <= b <= q4.to_scale(amax + off), (amax, b)
        s = q4.SCALES[b]
        got = np.where(c & 8, -1.0, 1.0) * q4.CODES[c & 7]
        y, d = np.clip(v / s, -6, 6), t / s
        size = np.abs(y) + d
        half = np.where(size <= 2, 0.25, np.where(size <= 4, 0.5, 1.0))
        assert np.all(np.abs(got - y) <= half + d), (v, got * s)
        if off == 0:
            assert np.array_equal(got, [(-1 if k & 8 else 1) * q4.CODES[k & 7] for k in (q4.to_code(z / s) for z in v)])


def draw_cache(rng, batch, centre=106, spread=5, spoil=True):
    """Random codes and scale bytes (centre +- spread); places behind the sequences are NaN (scale 255)."""
    s = batch.spec
    shape = (batch.num_pages, s.num_kv_heads, s.page_size)
    cache = rng.integers(0, 256, (*shape, s.head_dim // 2)).astype(np.uint8)
    scale = rng.integers(max(1, centre - spread), min(q4.MAX_SCALE, centre + spread) + 1,
                         (*shape, s.head_dim // q4.GROUP)).astype(np.uint8)
    if spoil:
        seen = np.zeros((batch.num_pages, s.page_size), bool)
        for r, n in enumerate(batch.seq_lens):
            j = np.arange(n)
            seen[batch.block_table[r, j // s.page_size], j % s.page_size] = True
        scale.transpose(0, 2, 1, 3)[~seen] = 255
    return cache, scale


def run(cpsa, batch, caches, max_kv_splits=8, workspace_bytes=None, scale=0.0, block_table=None, q=None):
    """One call; returns (out float64, device flags)."""
    s = batch.spec
    T, B = batch.num_tokens, len(s.qlen)
    if workspace_bytes is None:
        workspace_bytes = cpsa.cpp_attn_workspace_bytes(B, T, s.num_q_heads, s.num_kv_heads, s.head_dim, max_kv_splits)
    ws = torch.full((workspace_bytes,), 0xAB, dtype=torch.uint8, device="cuda")
    out = torch.full((T, s.num_q_heads, s.head_dim), float("nan"), dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kc, ks, vc, vs = (to_dev(x) for x in caches)
    bt = batch.block_table if block_table is None else block_table
    cpsa.cpp_chunked_prefill_attn_q4(to_dev_bf16(batch.q if q is None else q), kc, vc, ks, vs, to_dev(batch.query_lens),
                                     to_dev(batch.seq_lens), to_dev(bt), out, ws, err, scale=scale,
                                     max_kv_splits=max_kv_splits)
    torch.cuda.synchronize()
    return bf16_tensor_to_f64(out), cpsa.cpp_read_device_error(err)


def reference(batch, caches, scale=0.0, q=None, rows=None):
    """(float64 rows, per row and q head the largest |v| of its keys)."""
    s = batch.spec
    k64, v64 = q4.values(caches[0], caches[1]), q4.values(caches[2], caches[3])
    ref = oracle.paged_attention(batch.q if q is None else q, bf16_bits(k64), bf16_bits(v64), batch.query_lens,
                                 batch.seq_lens, batch.block_table, scale=scale, rows=rows)
    vmax = []
    for r, (ql, n) in enumerate(zip(batch.query_lens, batch.seq_lens)):
        j = np.arange(n)
        v = v64[batch.block_table[r, j // s.page_size], :, j % s.page_size]
        m = np.abs(v).max((0, 2)) if n else np.zeros(s.num_kv_heads)
        vmax += [np.repeat(m, s.num_q_heads // s.num_kv_heads)] * int(ql)
    vmax = np.array(vmax)
    return ref, (vmax if rows is None else vmax[rows])[..., None]


def draw(spec, seed=None, **kw):
    b = W.make_batch(spec, with_history=False)
    rng = np.random.default_rng(spec.seed if seed is None else seed)
    kc, ks = draw_cache(rng, b, **kw)
    vc, vs = draw_cache(rng, b, **kw)
    return b, (kc, ks, vc, vs)


def check(cpsa, spec, max_kv_splits=8, workspace_bytes=None, scale=0.0, expect_flags=0, **kw):
    b, caches = draw(spec, **kw)
    got, flags = run(cpsa, b, caches, max_kv_splits=max_kv_splits, workspace_bytes=workspace_bytes, scale=scale)
    assert flags == expect_flags, f"device flags {flags:#x}"
    ref, vmax = reference(b, caches, scale=scale)
    close(got, ref, vmax, str(spec))
