"""Kernels launched programmatically may start before the kernel ahead of them
in the stream has ended.  Whoever is launched behind such a kernel waits for
that kernel alone, so the order of the whole stream holds only if every grid
waits for its predecessor before any of its CTAs leaves.  Read from the
sources: a race cannot be shown by running it."""
import os
import re

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "paged_kv_cache_383_b200", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def body(text, kernel):
    """The braces of a __global__ function, from its name on."""
    at = re.search(r"__global__[^{;]*?\b%s\(" % kernel, text).end()
    at = text.index("{", text.index(")", at))
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at:i + 1]


def test_reduce_waits_before_it_leaves():
    """Sequences of one partition leave the reduce nothing to do."""
    code = body(source("decode_common.cuh"), "reduce_kernel")
    assert "return" in code
    assert code.index("pdl_wait") < code.index("return")


@pytest.mark.parametrize("name,kernel", [
    ("append.cu", "append_kernel"), ("cache_ops_q8.cu", "move_blocks_q8_kernel")])
def test_writers_release_their_successors_after_waiting(name, kernel):
    """An attention call behind these reads its lengths before its own wait:
    they must not let it start while a kernel before them (the writer of the
    lengths, say) still runs."""
    code = body(source(name), kernel)
    assert code.index("pdl_wait") < code.index("pdl_trigger")
    head = code[:code.index("pdl_trigger")]
    assert "return" not in head and "if" not in head
