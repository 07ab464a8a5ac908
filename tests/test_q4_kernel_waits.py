"""Bounded waits and registers of the 4-bit cache's kernels, read off their sources (CPU), as test_kernel_waits.py and
test_chunk_kernel_roles.py do for the others."""
import re

import pytest

from test_chunk_kernel_roles import holds, role_branches
from test_kernel_waits import function, own_verdicts, source


def test_waits_of_the_decode_kernel():
    text = source("decode_q4.cu")
    assert "mbar_wait" in text and own_verdicts(text) == []
    body = function(text, "\ndecode_q4_kernel")
    assert re.search(r"mbar_drain\(bars->full, g, C::kStages\);\s*return;", body), "the producer leaves its copies behind"


@pytest.mark.parametrize("name,drain", [("q4_load", r"mbar_drain\(q8t->full, half, C::kRawStages\);\s*$"),
                                        ("q4_load_q", r"mbar_drain\(q4t->q_raw, u, C::kQRing\);\s*$")])
def test_waits_of_the_chunk_kernels_loaders(name, drain):
    body = function(source("prefill_tc.cu"), name)
    assert "mbar_wait" in body and own_verdicts(body) == [] and re.search(drain, body)


@pytest.mark.parametrize("nq", [1, 2])
def test_a_group_of_four_warps_moves_registers_in_one_place(nq):
    branches = role_branches()
    where = [next(i for i, (c, _) in enumerate(branches) if holds(c, w, nq)) for w in range(16)]
    text = source("prefill_tc.cu")
    count = {n: int(re.search(rf"void regs_q4_{n}\(\) {{ asm volatile\(\"setmaxnreg\.\w+\.sync\.aligned\.u32 (\d+);", text)[1])
             for n in ("softmax", "others")}
    registers = 0
    for g in range(4):
        group = set(where[4 * g:4 * g + 4])
        assert len(group) == 1
        body = branches[group.pop()][1]
        calls = re.findall(r"regs_q4_(\w+)\(\);", body)
        assert len(calls) == 1, f"warps {4 * g} to {4 * g + 3}: {calls}"
        before = body[:body.index("regs_q4_" + calls[0])]
        assert "warp ==" not in before and "warp !=" not in before
        registers += 128 * count[calls[0]]
    assert registers <= 512 * 128, "more registers than the block starts with: the group that takes them would wait"


def test_ring_of_q_tiles_leaves_the_exponents_alone():
    """Tile u's exponents are read until an item later; they are written again at u + 6, once tile u + 6 - (NQ + 1)'s
    buffer is free: a tile of a later item than u's, whose first MMA comes after all of u's item's (one or two q heads)."""
    text = source("prefill_tc.cu")
    assert re.search(r"int8_t qe\[6\]\[128\];", text) and re.search(r"kQRing = NQ \+ 1;", text)
    for nq in (1, 2):
        for u in range(12):
            assert (u + 6 - (nq + 1)) // nq > u // nq
