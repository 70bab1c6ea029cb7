"""Read from the sources (no GPU): the delta kernels reach instructions on tensor memory with whole warps.

`.sync.aligned` instructions (allocation, loads, stores, waits) are undefined for a warp that is not
converged.  Going back from each of them, the line that makes the warp converge (__syncwarp, __all_sync,
or another such instruction) has to come before any branch that may differ between its lanes."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "state_space_model_mamba_gb300", "csrc")
ALIGNED = re.compile(r"\btmem_(alloc|dealloc|ld16x3|ld16x2|ld16|st16|wait_st)\(")
CONVERGED = re.compile(r"__syncwarp\(\)|__all_sync\(")
# names that hold something of a thread's own; the others in conditions are the same for a warp
OWN = re.compile(r"\b(tid|lane|live|row|tok|limit)\b")


def branches(line):
    """Whether a condition on the line may differ between lanes."""
    for m in re.finditer(r"\b(?:if|for|while)(?: constexpr)? \(", line):
        depth, end = 1, m.end()
        while end < len(line) and depth:
            depth += {"(": 1, ")": -1}.get(line[end], 0)
            end += 1
        if OWN.search(line[m.end():end]):
            return True
    return False


def lines(path):
    text = re.sub(r"/\*.*?\*/", lambda m: "\n" * m.group().count("\n"), open(path).read(), flags=re.S)
    return [re.sub(r"//.*", "", x) for x in text.split("\n")]


def unconverged(text):
    found = []
    for n, line in enumerate(text):
        if not ALIGNED.search(line):
            continue
        for back in range(n, -1, -1):
            before = text[back] if back < n else line[:ALIGNED.search(line).start()]
            if CONVERGED.search(before) or (back < n and ALIGNED.search(before)):
                break
            if branches(before) or before.startswith("__global__"):
                found.append((n + 1, line.strip(), back + 1))
                break
    return found


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "delta_*.cu"))), ids=os.path.basename)
def test_tensor_memory_is_reached_by_whole_warps(path):
    assert unconverged(lines(path)) == []


def test_the_check_sees_a_branch_of_one_lane():
    bad = ["    if (tid == 0) {", "        mbar_init(&bar, 1);", "    }", "    if (warp == 0) tmem_alloc(&s, 256);"]
    assert [x[0] for x in unconverged(bad)] == [4]
    assert unconverged(bad[:3] + ["    if (warp == 0) {", "        __syncwarp();", "        tmem_alloc(&s, 256);", "    }"]) == []
