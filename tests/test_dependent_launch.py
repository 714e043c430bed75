"""Kernels that start while the one before them still runs (programmatic dependent launch), from their
sources on the CPU: each waits, whatever its arguments, before anything that touches global memory.
What an earlier kernel wrote is promised to a grid after its own wait only, so a wait of the kernel
in between is not enough."""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "nf4_base_lora_blockwise_b200", "csrc")
WAIT = "pdl_wait();"
# Loads, stores and atomics by the names that the sources give them, and members behind a pointer.
TOUCHES = re.compile(r"\b(load_\w+|load8|ld_\w+|ldg\w*|__ldg|__ldcg|st_\w+|store_\w+|atomic\w+|issue\w*"
                     r"|copy16|tma_load\w*|scalars|token_of)\s*(<[^;()]*>)?\(|\bst->|\ba\.\w+\[")


def _uncommented(text):
    return re.sub(r"//[^\n]*", "", text)


def _body(text, at):
    """The braces that open at or after `at`."""
    start = text.index("{", at)
    depth = 0
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[start + 1:i]
    raise AssertionError("unbalanced braces")


def _kernels():
    found = {}
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = _uncommented(open(path).read())
        for m in re.finditer(r"__global__", text):
            # The name stands before the list of parameters, after the launch bounds.
            head = re.sub(r"__launch_bounds__\([^)]*\)", lambda b: " " * len(b.group()),
                          text[m.end():m.end() + 400])
            name = re.search(r"(\w+)\s*\(", head)
            end, depth = m.end() + name.end(), 1
            while depth:
                depth += {"(": 1, ")": -1}.get(text[end], 0)
                end += 1
            if text[end:].lstrip().startswith(";"):
                continue  # a declaration
            found[name.group(1)] = _body(text, end)
    return found


KERNELS = {k: b for k, b in _kernels().items() if "pdl_wait" in b}


def test_kernels_are_found():
    assert {"adam_step_kernel", "adam_norm_kernel", "rope_kernel", "residual_norm_fwd_kernel",
            "residual_norm_bwd_kernel", "column_sum_kernel", "qlora_gemm_kernel"} <= set(KERNELS)


@pytest.mark.parametrize("name", sorted(KERNELS))
def test_the_wait_comes_first(name):
    body = KERNELS[name]
    before = body[:body.index(WAIT)]
    assert before.count("{") == before.count("}"), "the wait is inside a branch"
    assert not before.strip() or before.rstrip()[-1] in ";}", "the wait is a branch's statement"
    hit = TOUCHES.search(before)
    assert hit is None, hit.group()
    assert body.count(WAIT) == 1
