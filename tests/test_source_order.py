"""What the text of the kernels has to keep for the stream's order to hold (CPU only).

The kernels around the experts start while the launch ahead still runs and wait for its end
(pdl_wait) before they touch memory.  Plain C++ accesses stay behind that wait, which clobbers
memory; inline assembly does only if it says the same, and a non-coherent load asks for data
that nothing writes while the kernel lives, which an early start cannot promise.
"""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_moe_expert_nf4_b200", "csrc")
FILES = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")))


def _code(path):
    return re.sub(r"//[^\n]*", "", open(path).read())


def _reach(path, seen=None):
    """The file and the headers of this folder that it includes."""
    seen = set() if seen is None else seen
    if path in seen or not os.path.exists(path):
        return seen
    seen.add(path)
    for name in re.findall(r'#include "([^"]+)"', open(path).read()):
        _reach(os.path.join(CSRC, name), seen)
    return seen


EARLY = sorted(set().union(*(_reach(f) for f in FILES if f.endswith(".cu") and "pdl_wait();" in _code(f))))


def _asm(code):
    """(qualifier, body) of every asm statement, by matching its parentheses outside of strings."""
    for m in re.finditer(r"\basm\b\s*(volatile)?\s*\(", code):
        depth, i, text = 1, m.end(), False
        while depth:
            c = code[i]
            if c == '"' and code[i - 1] != "\\":
                text = not text
            elif not text:
                depth += (c == "(") - (c == ")")
            i += 1
        yield m.group(1), code[m.end():i - 1]


def test_kernels_that_start_early_are_found():
    assert {"block_norm.cu", "block_norm.cuh", "ffn.cu", "gemv.cu", "tcgen05.cuh"} <= {os.path.basename(f) for f in EARLY}


@pytest.mark.parametrize("path", EARLY, ids=os.path.basename)
def test_early_kernels_read_memory_in_order(path):
    for qualifier, body in _asm(_code(path)):
        if not re.search(r"\b(ld|st|red|atom|cp|prefetch)\b[\w.:]*global", body):
            continue
        assert ".nc" not in body, body
        assert qualifier == "volatile" and '"memory"' in body, body


def _function(code, name):
    at = re.search(r"\b" + name + r"\([^)]*\)\s*\{", code).end()
    depth, i = 1, at
    while depth:
        depth += (code[i] == "{") - (code[i] == "}")
        i += 1
    return code[at:i - 1]


def test_warps_meet_before_aligned_barriers():
    """barrier.cluster with .aligned wants a warp's lanes together; its callers come from branches of single lanes."""
    body = _function(_code(os.path.join(CSRC, "tcgen05.cuh")), "cluster_sync_all")
    assert ".aligned" in body and 0 <= body.find("__syncwarp()") < body.find("barrier.cluster")


def test_a_warp_leaves_a_wait_together():
    """In the feed-forward kernel whole warps wait and go on to .aligned instructions: the wait's answer is one for
    all lanes.  (A wait by itself answers each lane, and one may run out of time alone.)"""
    code = _code(os.path.join(CSRC, "ffn.cu"))
    assert not re.search(r"\bmbar_wait\(", code) and "mbar_wait_warp(" in code
    assert "__all_sync" in _function(_code(os.path.join(CSRC, "async.cuh")), "mbar_wait_warp")
