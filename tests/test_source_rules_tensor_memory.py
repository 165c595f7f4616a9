"""Static checks of the kernels that use tensor memory (no GPU)."""
from __future__ import annotations

import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "xlstm_mlstm_cell_b200", "csrc")


def kernels():
    """(file, body) of every kernel that frees tensor memory."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = open(path).read()
        for m in re.finditer(r"^__global__ ", text, flags=re.M):
            body = text[m.start():text.index("\n}\n", m.start())]
            if "tmem_dealloc" in body:
                yield os.path.basename(path), body


def test_tensor_memory_is_freed_after_the_mmas():
    """After a wait that gave up, a kernel frees its tensor memory only once it has waited (bounded) for its MMAs:
    for a barrier that they commit to, or for a fixed time behind the CTA's abort flag."""
    found = 0
    for name, body in kernels():
        end = body[:body.rindex("tmem_dealloc")]
        commits = set(re.findall(r"mma_commit\w*\(&?([\w\[\]]+)", body))
        drains = set(re.findall(r"mbar_wait_drain\(&?([\w\[\]]+)", end))
        waits = re.search(r"if \(\*reinterpret_cast<volatile uint32_t \*>\(abort_flag\)\) \{", end)
        assert waits or commits & drains, "%s: MMAs commit to %s, drained are %s" % (name, sorted(commits), sorted(drains))
        found += 1
    assert found >= 8


def test_mmas_are_ordered_behind_the_waits_before_them():
    """In the delta rule's kernels an MMA that follows a wait for other threads has the fence between the two that
    orders tensor-memory operations behind the wait: those threads may have read the accumulator it writes.
    (The preparation's MMAs wait for a copy alone.)"""
    found = 0
    for name, body in kernels():
        if not name.startswith("gdelta"):
            continue
        for m in re.finditer(r"\bmma_ss\(", body):
            wait = body.rindex("mbar_wait(", 0, m.start())
            if body[wait:].startswith("mbar_wait(&bars[0]"):
                continue
            assert "tc_fence_after" in body[wait:m.start()], "%s: no fence behind %s" % (name, body[wait:].split(";")[0])
            found += 1
    assert found >= 8
