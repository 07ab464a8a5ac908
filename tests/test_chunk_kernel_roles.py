"""The 8-bit chunk kernel moves registers between groups of four warps (setmaxnreg), which all four have to do by
one and the same instruction: read off the kernel's source, for one and two q heads a CTA (CPU)."""
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "chunked_prefill_paged_slot_gb300",
                      "csrc", "prefill_tc.cu")


def role_branches():
    """[(condition of warp, body)] of the kernel's chain of roles, at the kernel's own indentation."""
    text = open(SOURCE).read()
    text = text[text.index("\nchunk_attn_kernel("):]
    text = text[text.index("\n    if (Q8 && warp >= C::kLoadWarp"):text.index("\n    // the softmax warps' output stores")]
    parts = re.split(r"\n    (?:\} else )?if (?:constexpr )?\((.*)\) \{\n|\n    \} (else) \{\n", text)[1:]
    return [(parts[i] if parts[i] is not None else "true", parts[i + 2]) for i in range(0, len(parts), 3)]


def holds(condition, warp, nq):
    names = dict(kLoadWarp=8, kConverters=4, kMmaWarp=12, kWriteWarp=10, kQ8LoadWarp=13)
    text = open(SOURCE).read()
    assert re.search(r"kLoadWarp = 8;", text) and re.search(r"kMmaWarp = Q8 \? 12 : 9;", text)
    assert re.search(r"kConverters = 4;", text) and re.search(r"kQ8LoadWarp = 13;", text)
    c = re.sub(r"C::(\w+)", lambda m: str(names[m.group(1)]), condition)
    c = c.replace("&&", " and ").replace("||", " or ").replace("!Q8", " not Q8 ").replace("/", "//").replace("true", "True")
    return eval(c, {"Q8": True, "warp": warp, "NQ": nq})


@pytest.mark.parametrize("nq", [1, 2])
def test_a_group_of_four_warps_moves_registers_in_one_place(nq):
    branches = role_branches()
    assert len(branches) >= 5
    where = [next(i for i, (c, _) in enumerate(branches) if holds(c, w, nq)) for w in range(16)]
    registers = 0
    for g in range(4):
        group = set(where[4 * g:4 * g + 4])
        assert len(group) == 1, f"warps {4 * g} to {4 * g + 3} take the branches {sorted(group)}"
        body = branches[group.pop()][1]
        calls = re.findall(r"regs_(keep|take)_(\d+)\(\);", body)
        assert len(calls) == 1, f"warps {4 * g} to {4 * g + 3}: {calls}"
        # ahead of anything that tells the group's warps apart
        before = body[:body.index("regs_" + "_".join(calls[0]))]
        assert "warp ==" not in before and "warp !=" not in before
        registers += 128 * int(calls[0][1])
    assert registers <= 512 * 128, "more registers than the block starts with: the group that takes them would wait"
