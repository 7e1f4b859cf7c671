"""What the kernels between the layers promise each other that no run can show, read from their sources: no value of global memory is
taken before the wait for the kernels before, and no rule knows the GPU's size."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(__file__), "..", "bit_grouped_expert_top_gb300", "csrc")
FILES = ["norm.cu", "q4_matvec.cu", "rope.cu", "verify.cu"]


def text(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _closing(s, at):
    """Index behind the brace that closes the one at `at`."""
    depth = 0
    for i in range(at, len(s)):
        depth += {"{": 1, "}": -1}.get(s[i], 0)
        if depth == 0:
            return i + 1
    raise AssertionError("unbalanced braces")


def kernels(name):
    """Name and body of each kernel of a file."""
    s = text(name)
    for m in re.finditer(r"__global__ void(?: __launch_bounds__\([^{]*?\))?\s+(\w+)\(const __grid_constant__ \w+ a\)\s*\{", s):
        yield m[1], s[m.end() - 1:_closing(s, m.end() - 1)]


def before_the_wait(body):
    """What runs ahead of the kernel's first pdl_wait(): lambdas that are only defined there are left out, their names are kept."""
    s, names = body[:body.index("pdl_wait();")], []
    while m := re.search(r"auto (\w+) = \[[^\]]*\]\([^)]*\)\s*\{", s):
        names.append((m[1], s[m.end() - 1:_closing(s, m.end() - 1)]))
        s = s[:m.start()] + s[_closing(s, m.end() - 1) + 1:]
    return s, names


READS = re.compile(r"\ba\.(?:w|s|b|x|x_scale|p|q|k|u|r|cu|drafts|positions|table|residual|weight)\s*\[|\*reinterpret_cast|\bcopy<|\bload16\(|ld\.global|__ldg")


@pytest.mark.parametrize("name", FILES)
def test_nothing_is_read_ahead_of_the_wait(name):
    """A kernel before this one may have just written any of the arguments, a matrix too, and the one between may let this one start at
    once: behind the wait alone its stores are there."""
    found = 0
    for kernel, body in kernels(name):
        found += 1
        assert body.count("pdl_wait();") == 1, kernel
        ahead, lambdas = before_the_wait(body)
        assert not READS.search(ahead), (kernel, READS.search(ahead)[0])
        for called, does in lambdas:
            if READS.search(does):
                assert not re.search(rf"\b{called}\(", ahead), f"{kernel}: {called}() ahead of the wait"
    assert found == 1


@pytest.mark.parametrize("name", FILES)
def test_no_rule_has_the_number_of_sms_written_in(name):
    """It is the device's: a part of a GPU, or another one, has fewer."""
    assert not re.search(r"\b152\b", text(name))
