"""The ring of Q tiles of the 4-bit chunk kernel and their exponents, read off the source (CPU): every role takes its index
from the same two functions, the compiler checks what these have to hold, and a buffer is given up with its item's last
scores."""
import re

from test_kernel_waits import function, source

TEXT = source("prefill_tc.cu")


def test_one_index_function_for_all_roles():
    """Reads and writes of the exponents by q4_exps, of the ring's barriers and buffers by q_ring; no modulus besides."""
    assert len(re.findall(r"%\s*\(?kQRing|%\s*C::kQRing", TEXT)) == 1 and len(re.findall(r"%\s*kQ4Exps", TEXT)) == 1
    assert not re.search(r"%\s*6\b", TEXT)
    q4 = re.findall(r"->qe\[([^\]]*(?:\[[^\]]*\])?[^\]]*)\]", TEXT)
    assert sum(x.startswith("q4_exps(") for x in q4) == 2 and all(x.startswith("q4_exps(") or x.endswith("& 1") for x in q4), q4
    for bars in ("q_raw", "q_full", "q_empty"):
        for index in re.findall(rf"q[48]t->{bars}\[([^\]]*)\]", TEXT):
            assert index in ("b", "s") or index.startswith("C::q_ring("), (bars, index)
    assert len(re.findall(r"uint32_t b = C::q_ring\(\w+\);", TEXT)) == 2


def test_what_the_compiler_checks():
    assert re.search(r"kQ4Exps = sizeof\(Q4Tiles::qe\) / sizeof\(Q4Tiles::qe\[0\]\);", TEXT)
    assert re.search(r"kQ4ExpsKept = \(int\)kQ4Exps - ChunkCfg<128, NQ, true, true>::kQRing >= NQ;", TEXT)
    assert re.search(r"static_assert\(kQ4ExpsKept<1> && kQ4ExpsKept<2>", TEXT)


def test_a_buffer_is_given_up_with_the_last_scores():
    """q_done(head) stands right behind the scores' commit, under the item's only tile or its last one."""
    body = function(TEXT, "\nchunk_attn_kernel")
    calls = [m.start() for m in re.finditer(r"(?<!auto )\bq_done\(\w+\);", body)]
    assert len(calls) == 3
    for at in calls:
        before = re.sub(r"\s+", " ", body[:at])
        assert re.search(r"issue_qk\((\w+), sK\); commit\(&bars->s_full\[\1\]\); if \((n == 1|t \+ 2 == n)\) $", before), before[-120:]
