"""The one wait of the 4-bit chunk kernel that takes as long as its work items, read off its source (CPU): its limit grows
with them. (A unit over 10^8 keys takes longer than the limit of the other waits.)"""
import re

from test_kernel_waits import function, source


def test_limit_of_the_q_loaders_wait():
    body = function(source("prefill_tc.cu"), "q4_load_q")
    wait = re.search(r"mbar_wait_warp\(&q4t->q_empty\[.*?, abort, (\w+)\)", body, re.S)
    assert wait, "the wait for a free buffer takes the limit of short waits"
    assert re.search(rf"uint64_t {wait[1]} = kWaitLimitNs \+ \(uint64_t\)\(ahead\[0\] \+ ahead\[1\]\) \* kWaitTileNs;", body)
    assert "ahead[0] = ahead[1];" in body and "ahead[1] = w.kt1 - w.kt0;" in body


def test_a_tiles_share_of_the_limit():
    """A tile takes 1.8 us; with other loads in its way, some times that."""
    assert int(re.search(r"kWaitTileNs = (\d+);", source("common.cuh"))[1]) >= 8 * 1800
