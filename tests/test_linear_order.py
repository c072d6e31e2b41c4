"""The order of the grids of the chunked linear attention, read from its source (no GPU). Where a grid lets the next one start
early (griddepcontrol.launch_dependents), that next one has to execute griddepcontrol.wait, in every block: whatever is launched
behind it waits for its end alone, which must not come before the first grid's. A breach shows on a GPU by chance at most."""
import os
import re

import pytest

from context_scan_gb300 import _build

WAIT = 'asm volatile("griddepcontrol.wait;" ::: "memory");'


def body(file, head):
    """From `head` in the file to the brace that closes its block."""
    text = open(os.path.join(_build.CSRC, file)).read()
    text = re.sub(r"//[^\n]*", "", text)
    at = text.index("{", text.index(head))
    depth, i = 0, at
    while True:
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        i += 1
        if depth == 0:
            return text[at:i]


def test_blocks_without_work_wait():
    # before the one return of the kernel, and before the state warps of a block with work do anything that could end them
    kernel = body("gdn_linear_tc.cu", "tc_kernel(const __grid_constant__")
    leave = body("gdn_linear_tc.cu", "if (!item_of(p, blockIdx.x")
    assert len(re.findall(r"\breturn\b", kernel)) == 1 == len(re.findall(r"\breturn\b", leave))
    assert re.search(r"if \(p\.phase == 2\) " + re.escape(WAIT) + r"\s*return;", leave)


def test_blocks_with_work_wait():
    state = body("gdn_linear_tc.cu", "void state_warps(const Work& w")
    wait = state.index("if (w.p->phase == 2) " + WAIT)
    before = re.sub(r"auto (slot|given) = \[&\]\(.*?\n    \};", "", state[:wait], flags=re.S)
    assert "return" not in before and "wait(B_" not in before


@pytest.mark.parametrize("file,kernel", [("gdn_linear_simt.cu", "simt_kernel(const"), ("gdn_linear.cu", "group_kernel(const"),
                                         ("gdn_qk_norm.cu", "qk_sum_kernel(const")])
def test_others_wait_first(file, kernel):
    text = body(file, kernel)
    assert WAIT in text and ("return" not in text or text.index(WAIT) < text.index("return"))
