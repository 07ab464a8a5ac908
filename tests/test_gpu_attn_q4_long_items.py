"""Chunks over so many keys that a CTA's work item takes more than a second: no wait gives up (GPU)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_items_of_more_than_a_second(cuda_lib):
    """Two q heads a CTA, whole units (max_kv_splits 1), 160 of them: the loader of Q waits through a CTA's first item for
    room for its second's. All keys of the history are one page's, over and over, with scores of -1.44 * 64 * 6 * 16 /
    sqrt(128) = -782 (in powers of two) against the chunk's own zero: nothing of theirs is left, and the output is the mean of the
    chunk's values up to the row. Those values are multiples of 1/2 up to 6, so that their sums are exact."""
    P, tokens, heads = 256, 1280, 16
    pages, own = 390625, tokens // P
    keys = pages * P
    gen = torch.Generator("cuda").manual_seed(1)
    q = torch.zeros(tokens, 2 * heads, 128, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 64
    k_codes = torch.zeros(1 + own, heads, P, 64, dtype=torch.uint8, device="cuda")
    k_codes[0, :, :, 0] = 15                                                            # column 0: -6
    k_scale = torch.full((1 + own, heads, P, 8), 19 << 3, dtype=torch.uint8, device="cuda")      # 16
    v_codes = torch.randint(0, 256, (1 + own, heads, P, 64), dtype=torch.uint8, device="cuda", generator=gen)
    v_scale = torch.full((1 + own, heads, P, 8), 15 << 3, dtype=torch.uint8, device="cuda")      # 1
    lens = [torch.tensor([x], dtype=torch.int32, device="cuda") for x in (tokens, keys + tokens)]
    table = torch.zeros(1, pages + own, dtype=torch.int32, device="cuda")
    table[0, pages:] = torch.arange(1, 1 + own)
    ws = torch.empty(cuda_lib.cpp_attn_workspace_bytes(1, tokens, 2 * heads, heads, 128, 1), dtype=torch.uint8, device="cuda")
    out, err = torch.full_like(q, float("nan")), torch.zeros(1, dtype=torch.int32, device="cuda")
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    cuda_lib.cpp_chunked_prefill_attn_q4(q, k_codes, v_codes, k_scale, v_scale, *lens, table, out, ws, err, max_kv_splits=1)
    end.record()
    assert cuda_lib.cpp_read_device_error(err) == 0
    ms = start.elapsed_time(end)
    print(f"{ms:.0f} ms")
    assert ms > 2000, "two items a CTA, each of more than the second that other waits may take"
    value = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    value = torch.cat([value, -value])
    v = torch.stack([value[(v_codes[1:] & 15).long()], value[(v_codes[1:] >> 4).long()]], -1).flatten(-2)
    v = v.transpose(1, 2).reshape(tokens, heads, 128).cumsum(0) / torch.arange(1, tokens + 1, device="cuda")[:, None, None]
    ref = v.repeat_interleave(2, 1)
    # a sum times the reciprocal of the row's count, each rounded once in fp32, and half a bf16 step
    assert bool(((out.double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -22) * ref.abs()).all())
