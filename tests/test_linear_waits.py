"""Host-only checks, on the sources, of how the tensor-core kernels of linear
attention end when a bounded wait runs out.  (A wait that runs out cannot be
brought about by any call, so nothing here runs a kernel.)

A wait is answered per thread: while a barrier completes, the give-up flag may go
up, and lanes of one warp may then get different answers.  A lane that leaves on
its own answer while others go on to an instruction of the whole warp (tcgen05.ld,
tcgen05.st, a shuffle, a warp barrier) would hold them there for good.  So a
function with such instructions takes its answers by vote.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_deltanet_04_b200", "csrc")
WARP_WIDE = re.compile(r"\btmem_(ld|st|wait)|__syncwarp|__shfl|warp_arrive|\btc_fence_before_sync")


def read(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def functions(source):
    """{name: body} of the __device__ and __global__ functions of a source."""
    out = {}
    for m in re.finditer(r"__(?:device|global)__[^;{=]*?\b(\w+)\s*\([^;{]*\)\s*\{", source):
        depth, at = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(source[at], 0)
            at += 1
        out[m.group(1)] = source[m.end():at - 1]
    return out


def waits(body):
    """Names of the abortable waits that a body calls (one argument is the flag)."""
    return set(re.findall(r"\b(\w*wait)\((?:&bar|&ms->\w+(?:\[[^\]]*(?:\[[^\]]*\])?[^\]]*\])?), [^;]*abort", body))


@pytest.mark.parametrize("name", ["linear_states.cu", "linear_out.cu", "linear_backward.cu"])
def test_whole_warps_take_their_answers_by_vote(name):
    seen = set()
    for fn, body in functions(read(name)).items():
        used = waits(body)
        seen |= used
        if WARP_WIDE.search(body):
            assert used <= {"warp_wait"}, f"{name}: {fn} goes on lane by lane after {used}"
        else:
            assert "warp_wait" not in used, f"{name}: {fn} votes outside a whole warp"
    assert "warp_wait" in seen, seen


def test_the_vote_is_one_of_all_lanes():
    body = functions(read("linear_tc.cuh"))["warp_wait"]
    assert re.search(r"return __all_sync\(0xffffffffu, thread_wait\(bar, parity, abort, err\)\);", body)
