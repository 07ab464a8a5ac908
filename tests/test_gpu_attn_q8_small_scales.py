"""Attention over an 8-bit cache whose scale bytes are the smallest there are (tolerances: q8_helpers.py).

A score is q . (byte 2^x) scale: keys shifted by 2^60 under a softmax scale of 2^-60 of the one
before give the same scores, and values shifted by 2^60 the outputs times 2^60. The oracle is
given the shifted ones, which bf16 holds.
"""
import numpy as np
import pytest

import workloads as W
from q8_helpers import close, draw, reference, run

pytestmark = pytest.mark.gpu

SHIFT = 60


@pytest.mark.parametrize("low,high", [(1, 2), (1, 7), (6, 8)])
@pytest.mark.parametrize("heads", [(8, 2, 128), (6, 2, 64)], ids=str)
def test_key_scales_of_the_smallest_exponents(cuda_lib, heads, low, high):
    """Chunks (one with history) and a decode row; scores of a few units."""
    hq, hkv, d = heads
    b, (kc, ks, vc, vs) = draw(W.BatchSpec(hist=[200, 0, 600], qlen=[130, 70, 1], num_q_heads=hq, num_kv_heads=hkv,
                                           head_dim=d, page_size=16, seed=2000 + high))
    rng = np.random.default_rng(2001)
    ks = np.where(ks != 255, rng.integers(low, high + 1, ks.shape), 255).astype(np.uint8)
    scale = 2.0 ** (127 - high - 6) / np.sqrt(d)
    scale = float(np.float32(scale))
    got, flags = run(cuda_lib, b, (kc, ks, vc, vs), scale=scale)
    assert flags == 0
    up = np.where(ks != 255, ks + SHIFT, 255).astype(np.uint8)
    ref, vmax = reference(b, (kc, up, vc, vs), scale=float(scale * 2.0 ** -SHIFT))
    close(got, ref, vmax)


@pytest.mark.parametrize("low,high", [(1, 2), (1, 7), (3, 9)])
@pytest.mark.parametrize("heads", [(8, 2, 128), (6, 2, 64)], ids=str)
def test_value_scales_of_the_smallest_exponents(cuda_lib, heads, low, high):
    """Values of 2^-126 to 2^-118 times their bytes: the output is theirs, digit for digit that of larger ones."""
    hq, hkv, d = heads
    b, (kc, ks, vc, vs) = draw(W.BatchSpec(hist=[200, 0, 600], qlen=[130, 70, 1], num_q_heads=hq, num_kv_heads=hkv,
                                           head_dim=d, page_size=16, seed=2100 + high))
    rng = np.random.default_rng(2101)
    vs = np.where(vs != 255, rng.integers(low, high + 1, vs.shape), 255).astype(np.uint8)
    got, flags = run(cuda_lib, b, (kc, ks, vc, vs))
    assert flags == 0
    ref, vmax = reference(b, (kc, ks, vc, np.where(vs != 255, vs + SHIFT, 255).astype(np.uint8)))
    # bf16 outputs under its smallest normal number are off by at most 2^-134
    close(got * 2.0 ** SHIFT, ref, vmax + 2.0 ** (SHIFT - 134 + 8))


@pytest.mark.parametrize("qlen", [1, 64])
def test_long_rows_of_tiny_values(cuda_lib, qlen):
    """The writer's smallest scale, 2^-117, in rows of 20000 keys that count alike: one over the row's sum times
    that scale is no normal fp32 number, the output is."""
    b, (kc, ks, vc, vs) = draw(W.BatchSpec(hist=[20000 - qlen], qlen=[qlen], num_q_heads=32, num_kv_heads=8, head_dim=128,
                                           page_size=64, seed=2200))
    vs = np.where(vs != 255, 10, 255).astype(np.uint8)
    caches = (kc, ks, vc & 0x7F, vs)             # no signs: the output is of the values' size
    got, flags = run(cuda_lib, b, caches, max_kv_splits=1, scale=1e-4)
    assert flags == 0
    at = np.arange(0, qlen, 9)
    ref, vmax = reference(b, caches, scale=1e-4, rows=at)
    close(got[at], ref, vmax)
