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
    """Waits and looks at the abort flag whose outcome each lane takes for itself."""
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
