"""The 8-bit append goes on with blocks of any exponent, those that only another writer leaves among them."""
import numpy as np
import pytest
import torch

from oracle import append as A
from test_gpu_rope_append import bf16, same_bytes, wide

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("P", [8, 16])
@pytest.mark.parametrize("gain", [1e-30, 1.0, 1e30, 3e38])
def test_runs_in_blocks_of_any_exponent(cuda_lib, P, gain):
    """One token into the middle of a block of every scale byte from 0 to 254: the exponent never falls, and where it
    stays the block's other bytes do."""
    d, n = 64, 255
    rng = np.random.default_rng(31)
    kc = torch.from_numpy(rng.integers(0, 127, (n, 2, P, d)).astype(np.uint8)).cuda()
    ks = torch.arange(n, device="cuda").to(torch.uint8).view(n, 1, 1).repeat(1, 2, 1)
    vc, vs = kc.clone(), ks.clone()
    want, wscale = kc.cpu().numpy().copy(), ks.cpu().numpy().copy()
    x = bf16(rng, (n, 2, d)).clamp(-1, 1) * gain
    x = x.to(torch.bfloat16).cuda()
    slots = np.arange(n) * P + 5
    A.append_q8(wide(x), slots, want, wscale)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cuda_lib.cpp_rope_kv_cache_write_q8(None, x, x, None, None, torch.from_numpy(slots).cuda(), kc, vc, ks, vs, None, err)
    for c, s in ((kc, ks), (vc, vs)):
        assert np.array_equal(s.cpu().numpy(), wscale)
        assert same_bytes(c.cpu().numpy(), want)
    assert cuda_lib.cpp_read_device_error(err) == 0
