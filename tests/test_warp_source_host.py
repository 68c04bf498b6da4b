"""What the kernels' sources keep to where one lane of a warp acts for all 32.

A lane that leaves its warp in a branch of its own may be compiled to run on by
itself, past waits and tensor-memory loads that are the whole warp's: it then
signals stages that the other 31 lanes have not reached.  Which of the two the
compiler makes of a branch is not visible in a call's results, so this reads the
sources: a branch that one lane takes to copy, to arrive or to commit ends in a warp
barrier (an arrival as a predicated instruction takes no branch).
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "gqa_kv_cache_append_gb300", "csrc")
KERNELS = ["chunk_attn.cu", "chunk_kernel.cuh", "decode_fp8.cu", "decode_tc.cu", "decode_simt.cu",
           "proj_tc.cu"]
ACTS = re.compile(r"\b(mbar_arrive|mbar_arrive_expect_tx|mma_commit|tma_load_[23]d|bulk_load)\(")


def text(name):
    with open(os.path.join(CSRC, name)) as f:
        s = f.read()
    s = re.sub(r"//[^\n]*", "", s)
    return re.sub(r"/\*.*?\*/", "", s, flags=re.S)


def closing(s, at, pair):
    """Index behind the bracket that closes the one at s[at]."""
    depth = 0
    for k in range(at, len(s)):
        depth += (s[k] == pair[0]) - (s[k] == pair[1])
        if depth == 0:
            return k + 1
    raise AssertionError("unbalanced source")


def one_lane_branches(s):
    """(statement, what follows it) of every `if` that a single lane takes."""
    for m in re.finditer(r"\bif\s*(?:constexpr\s*)?\(", s):
        end = closing(s, m.end() - 1, "()")
        cond = s[m.end():end - 1]
        if not re.search(r"\b(lane|ct) == 0\b|\belect_one\(\)|\bleader\b", cond):
            continue
        rest = s[end:].lstrip()
        at = len(s) - len(rest)
        stop = closing(s, at, "{}") if rest[0] == "{" else s.index(";", at) + 1
        yield s[at:stop], s[stop:].lstrip()


@pytest.mark.parametrize("name", KERNELS)
def test_branches_of_one_lane_end_in_a_warp_barrier(name):
    open_ended = [b for b, after in one_lane_branches(text(name))
                  if ACTS.search(b) and not after.startswith("__syncwarp();")]
    assert not open_ended


@pytest.mark.parametrize("name", ["decode_tc.cu", "proj_tc.cu"])
def test_loads_of_tensor_memory_are_the_whole_warps(name):
    # one lane's answer to a bounded wait would split the warp before them
    assert not re.search(r"const bool ok = mbar_wait\(", text(name))


@pytest.mark.parametrize("name", ["chunk_attn.cu", "chunk_kernel.cuh"])
def test_a_warpgroup_splits_its_registers_at_one_instruction(name):
    # all four warps of a warpgroup execute the same setmaxnreg
    s = text(name)
    assert s.count("setmaxnreg.dec") == 1 and s.count("setmaxnreg.inc") == 1
