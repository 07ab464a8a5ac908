"""Seeded batches over an 8-bit cache, their run and their check (no arithmetic of the method here).

A stored value, e4m3 byte * 2^x, is exact in bf16, so the fp64 oracle for bf16
caches takes the very values that the 8-bit cache holds.

Tolerance: the output is off by half a bf16 step, 2^-8 |o|; a merged partial was
rounded once to bf16, 2^-8 of at most the largest |v| that the row sees; each
probability once to 16 bits, and the row's sum is not, at most 2^-9 of that v; the
scores' fp32 sums move the probabilities by far less, 2^-10 taken for them.
"""
from __future__ import annotations

import numpy as np
import torch

import oracle
import workloads as W
from helpers import bf16_tensor_to_f64, to_dev, to_dev_bf16
from oracle import append as A


def bf16_bits(x64):
    """bf16 bits of float64 values that bf16 holds exactly."""
    x = x64.astype(np.float32)
    bits = x.view(np.uint32)
    assert np.array_equal(x.astype(np.float64), x64, equal_nan=True) and not np.any(bits[np.isfinite(x)] & 0xffff)
    out = (bits >> 16).astype(np.uint16)
    out[np.isnan(x)] = 0x7FC0
    return out


def draw_cache(rng, batch, centre=120, spread=1, spoil=True):
    """Random bytes and scale bytes (centre +- spread); places behind the sequences are NaN, unstarted blocks 255."""
    s = batch.spec
    P, sb = s.page_size, min(16, s.page_size)
    byte = np.array([A.to_byte(v) for v in np.linspace(-448, 448, 4097)], np.uint8)
    shape = (batch.num_pages, s.num_kv_heads, P, s.head_dim)
    draw = np.clip(rng.standard_normal(shape) * 100, -448, 448)
    cache = byte[np.rint((draw + 448) / 896 * 4096).astype(np.int64)]
    scale = rng.integers(centre - spread, centre + spread + 1, (batch.num_pages, s.num_kv_heads, P // sb)).astype(np.uint8)
    if spoil:
        seen = np.zeros((batch.num_pages, P), bool)
        for r, n in enumerate(batch.seq_lens):
            j = np.arange(n)
            seen[batch.block_table[r, j // P], j % P] = True
        cache.transpose(0, 2, 1, 3)[~seen] = 0x7F
        scale.transpose(0, 2, 1)[~seen.reshape(-1, P // sb, sb).any(2)] = 255
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
    cpsa.cpp_chunked_prefill_attn_q8(to_dev_bf16(batch.q if q is None else q), kc, vc, ks, vs, to_dev(batch.query_lens),
                                     to_dev(batch.seq_lens), to_dev(bt), out, ws, err, scale=scale,
                                     max_kv_splits=max_kv_splits)
    torch.cuda.synchronize()
    return bf16_tensor_to_f64(out), cpsa.cpp_read_device_error(err)


def reference(batch, caches, scale=0.0, q=None, rows=None):
    """(float64 rows, per row and q head the largest |v| of its keys)."""
    s = batch.spec
    k64, v64 = A.values(caches[0], caches[1]), A.values(caches[2], caches[3])
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


def close(got, ref, vmax, what=""):
    assert np.all(np.isfinite(got)), f"{what}: non-finite output"
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -9 + 2.0 ** -10) * vmax
    off = np.abs(got - ref) / tol
    rel = float(np.linalg.norm(got - ref) / np.linalg.norm(ref))
    assert off.max() <= 1 and rel <= 5e-3, f"{what}: {off.max():.3f} of the bound, rel-F {rel:.2e}"


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
