"""Chained launches (programmatic dependent launch), read from the sources: a kernel that may start while the launch
before it still runs waits for that launch itself, with nothing in between that could let a later kernel read ahead.

``griddepcontrol.wait`` is what makes the writes of the launch before visible, and only to the grid that executes it;
``griddepcontrol.launch_dependents`` says when the next grid may start and makes nothing visible. So every kernel waits
first, whatever variant it is, and releases only then: a grid that starts early can rely on nothing but its own wait.
"""
import glob
import os
import re

import pytest

from vision_encoder_varlen_gb300 import _build

SOURCES = sorted(glob.glob(os.path.join(_build.CSRC, "*.cu")))


def code(path):
    """The file's statements, a line each, without comments and blank lines."""
    with open(path) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    return [x.strip() for x in text.splitlines() if x.strip()]


def test_the_calls_are_found():
    assert sum("launch_chained(" in line for f in SOURCES for line in code(f)) >= 10


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_each_kernel_waits_before_it_releases(path):
    lines = code(path)
    waits = [i for i, x in enumerate(lines) if "grid_wait()" in x]
    for i in waits:
        assert lines[i] == "grid_wait();", lines[i]           # not on a condition, not at a kernel's end
        assert lines[i + 1] != "}", lines[i - 1:i + 2]
    for i, x in enumerate(lines):
        if "grid_release()" in x:
            assert x == "grid_release();" and i - 1 in waits, lines[i - 1:i + 1]


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_their_pointers_may_change_under_them(path):
    """A parameter declared __restrict__ lets the compiler load through it before the wait, and through a cache that
    does not see the writes of the launch before."""
    kernels = re.split(r"\b__global__\b", "\n".join(code(path)))[1:]
    for k in kernels:
        signature, body = k.split("\n{\n", 1)
        if "grid_wait();" in body:
            assert "__restrict__" not in signature, signature
