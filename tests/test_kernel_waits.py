"""Bounded waits of the kernels that issue copies, read off their sources (CPU): a warp takes one verdict, since
lanes that part go on to different collectives of the whole warp and may never meet again, and a role that
issues copies leaves only once they have landed."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "chunked_prefill_paged_slot_gb300", "csrc")


def source(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


def own_verdicts(text):
    """Waits and looks at the abort flag whose outcome each lane takes for itself (a wait whose outcome nothing looks
    at is a statement of its own)."""
    text = re.sub(r"^\s*mbar_wait\(.*\);$", "", text, flags=re.M)
    text = re.sub(r"__(?:all|any)_sync\(0xffffffffu, (?:mbar_wait(?:_sleep)?\(|\*abort)", "combined(", text)
    return re.findall(r"\bmbar_wait(?:_sleep)?\(.*|!\*abort\b.*", text)


def function(text, name):
    """The text of a function (from its name to the closing brace in the first column)."""
    at = text.index(name + "(")
    return text[at:text.index("\n}\n", at)]


def test_waits_of_the_8_bit_decode_kernel():
    text = source("decode_q8.cu")
    assert "mbar_wait" in text and own_verdicts(text) == []
    body = function(text, "\ndecode_q8_kernel")
    assert re.search(r"mbar_drain\(bars->full, g, C::kStages\);\s*return;", body), "the producer leaves its copies behind"


@pytest.mark.parametrize("name", ["q8_load", "q8_convert"])
def test_waits_of_the_8_bit_chunk_kernel(name):
    body = function(source("prefill_tc.cu"), name)
    assert "mbar_wait" in body and own_verdicts(body) == []
    if name == "q8_load":
        assert re.search(r"mbar_drain\(q8t->full, half, kQ8Stages\);\s*$", body)


def test_waits_of_the_chunk_kernel():
    text = source("prefill_tc.cu")
    assert "mbar_wait" in text and own_verdicts(text) == []


@pytest.mark.parametrize("name", ["decode_attn_kernel", "decode_group_kernel"])
def test_waits_of_the_bf16_decode_kernels(name):
    """No lane leaves a loop by its own verdict: a producer's stops issuing copies, a consumer's goes on."""
    body = function(source("decode.cu"), "\n" + name)
    waits = [body[m.end():body.index(";", m.end())] for m in re.finditer(r"\bmbar_wait\(", body)]
    assert len(waits) == 3
    for w in waits:
        assert re.search(r"abort\)$|abort\)\)\s*last = g$", w), w
    assert "!*abort" not in body and not re.search(r"\bstop\b", body)
    issues = re.findall(r"if \(lane == 0([^{\n]*)", body[:body.index("return;")])
    assert sum("g < last" in c for c in issues) >= 2, issues


def test_producers_over_the_bf16_cache_wait_for_their_copies():
    decode = source("decode.cu")
    for name in ("\ndecode_attn_kernel", "\ndecode_group_kernel"):
        assert re.search(r"mbar_drain\(bars->full, min\(g, last\), C::kStages\);\s*mbar_drain\(&bars->patch, patch_uses, 1\);"
                         r"\s*\}\s*return;", function(decode, name)), name
    chunk = function(source("prefill_tc.cu"), "\nchunk_attn_kernel")
    assert re.search(r"mbar_drain\(&bars->q_full, q_uses, 1\);\s*mbar_drain\(bars->slot_full, slot_it, C::kSlots\);\s*"
                     r"mbar_drain\(&bars->tail, tail_uses, 1\);\s*\} else if \(warp == C::kWriteWarp\)", chunk)
