"""The warp-wide bounded wait gives one verdict to all lanes where those of the plain wait differ, and the drain of a
ring leaves when its copies have landed or its limit has passed. No copy is in flight in the self-test."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("limit_us", [50, 2000])
def test_one_verdict_for_a_warp(cuda_lib, limit_us):
    out = cuda_lib.cpp_selftest_warp_wait(limit_us * 1000).cpu().tolist()
    assert out[:32] == [0] + [1] * 31            # what the plain wait says: lane 0 gave up, the others did not
    assert out[32:64] == [0] * 32


@pytest.mark.parametrize("limit_us", [50, 2000])
def test_drain(cuda_lib, limit_us):
    out = cuda_lib.cpp_selftest_warp_wait(limit_us * 1000).cpu().tolist()
    landed, us, never, never_us = out[64:]
    assert landed == 1 and limit_us // 2 <= us < 500_000
    assert never == 0 and limit_us <= never_us < 500_000


def test_limit_outside_range_is_refused(cuda_lib):
    out = torch.zeros(68, dtype=torch.int32, device="cuda")
    s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    for bad in (0, 999, 100_000_001):
        assert cuda_lib.load().cpp_selftest_warp_wait(bad, ctypes.c_void_p(out.data_ptr()), s) == -2
    assert cuda_lib.load().cpp_selftest_warp_wait(1000, None, s) == -1
