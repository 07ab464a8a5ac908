"""The plan's kernels, read off their source (CPU): none walks a request's units twice. (Of one large chunk beside
decode rows the second walk, to count the pieces, cost more than the rest of the plan.)"""
import re

import pytest

from test_kernel_waits import function, source


@pytest.mark.parametrize("name", ["plan_small_kernel", "plan_warps_kernel", "plan_kernel"])
def test_units_are_walked_once(name):
    body = function(source("plan.cu"), name)
    assert len(re.findall(r"\brequest_work\(", body)) == 1


def test_the_choice_of_a_kernel_goes_by_what_the_host_knows():
    """Requests and tokens: an estimate of the units says nothing of how they are spread over the requests."""
    body = function(source("plan.cu"), "cudaError_t launch_plan")
    assert "kTileM" not in body and "Hkv" not in body
