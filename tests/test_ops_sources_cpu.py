"""Which loads the few-token operators' kernels use (the sources, read as text).

A load through the read-only path (__ldg, or a const __restrict__ pointer of a kernel) is for memory
that nothing writes while the kernel lives. A kernel of a programmatic dependent launch lives from
before the end of the one whose results it reads, and some inputs may be the output's own buffer:
neither may be read that way."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dropless_token_routing_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def early_starting():
    return [n for n in sorted(os.listdir(CSRC)) if n.endswith(".cu") and "pdl_wait()" in source(n)]


def body(text, head):
    """The function that starts at `head`, to the brace that closes it."""
    at = text.index(head)
    start = text.index("{", at)
    depth = 0
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at:i + 1]
    raise AssertionError(head)


def test_the_kernels_that_start_early_are_found():
    assert {"linear.cu", "linear_pair.cu", "linear_stream.cu", "verify.cu"} <= set(early_starting())


@pytest.mark.parametrize("name", early_starting())
def test_no_read_only_loads_in_kernels_that_start_early(name):
    text = source(name)
    assert "__ldg" not in text
    assert not re.search(r"const\s+[\w:]+\s*\*\s*__restrict__", text)


def test_shared_loads_that_early_kernels_use():
    text = source("common.cuh")
    assert "__ldg" not in body(text, "void load8_unaligned")
    # the vectors of eight have both kinds of load
    plain = re.findall(r"void load_plain\([^{]*\{[^}]*\}", text)
    assert len(plain) == 2 and not any("__ldg" in p for p in plain)
    assert not re.search(r"\]\.load\(", body(source("linear.cu"), "linear_dz_kernel"))


def test_few_token_layer_reads_x_plainly():
    """y may be x's buffer."""
    text = source("decode.cu")
    hidden = body(text, "void hidden_rows")
    assert not re.search(r"__ldg\([^;]*\bx \+", hidden)
    assert not re.search(r"__restrict__ x\b", hidden)
