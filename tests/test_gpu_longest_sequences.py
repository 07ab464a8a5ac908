"""Sequences at the end of what an int counts: refused, whatever the table holds, before any kernel looks a page up."""
import pytest
import torch

pytestmark = pytest.mark.gpu

KINDS = ["bf16", "8 bit", "4 bit"]


def call(cpsa, kind, query_lens, seq_lens, heads=2, P=256, blocks=1 << 23):
    """One call over one page, which every entry of the table names; (the output, filled with 5 before, the flags)."""
    T, B, d = sum(query_lens), len(query_lens), 64
    q = torch.ones(T, heads, d, dtype=torch.bfloat16, device="cuda")
    byte = lambda *s: torch.full(s, 1, dtype=torch.uint8, device="cuda")
    cache = {"bf16": lambda: [torch.ones(1, heads, P, d, dtype=torch.bfloat16, device="cuda")] * 2,
             "8 bit": lambda: [byte(1, heads, P, d)] * 2 + [byte(1, heads, P // 16)] * 2,
             "4 bit": lambda: [byte(1, heads, P, d // 2)] * 2 + [byte(1, heads, P, d // 16)] * 2}[kind]()
    table = torch.zeros(B, blocks, dtype=torch.int32, device="cuda")
    lens = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (query_lens, seq_lens)]
    ws = torch.empty(cpsa.cpp_attn_workspace_bytes(B, T, heads, heads, d, 8), dtype=torch.uint8, device="cuda")
    out, err = torch.full_like(q, 5.0), torch.zeros(1, dtype=torch.int32, device="cuda")
    attend = {"bf16": cpsa.cpp_chunked_prefill_attn, "8 bit": cpsa.cpp_chunked_prefill_attn_q8,
              "4 bit": cpsa.cpp_chunked_prefill_attn_q4}[kind]
    attend(q, *cache, *lens, table, out, ws, err)
    return out, cpsa.cpp_read_device_error(err)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("s", [2 ** 31 - 1, 2 ** 31 - 64, 2 ** 31 - 2 ** 16 + 1])
@pytest.mark.parametrize("lens", [[1], [3], [300], [1, 1], [1, 40], [200, 1, 2, 1, 1], [1] * 40], ids=str)
def test_too_long(cuda_lib, lens, s, kind):
    """The table of 2^23 pages of 256 would hold them. The other requests are short, and served."""
    other = [7 + n for n in lens[1:]]
    out, flags = call(cuda_lib, kind, lens, [s] + other)
    assert flags == cuda_lib.DEV_SEQ_GT_TABLE
    assert bool((out[:lens[0]] == 5.0).all())
    assert not bool((out[lens[0]:] == 5.0).any()) and bool(torch.isfinite(out).all())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("others", [0, 1, 5, 40])
def test_more_tiles_than_an_int_counts(cuda_lib, others, kind):
    """Many query tiles and heads over a long history: each number an int, their product not. Nothing is computed."""
    tokens = 12800 if others == 0 else 1280            # alone: more than a batch that plans itself
    out, flags = call(cuda_lib, kind, [tokens] + [1] * others, [2 ** 30] + [9] * others, heads=64, blocks=1 << 22)
    assert flags == cuda_lib.DEV_PLAN_OVERFLOW
    assert bool((out == 5.0).all())
