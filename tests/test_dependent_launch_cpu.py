"""Programmatic dependent launches: a kernel that waits for the grid before it (``pdl_wait``) may start while that
grid still writes its inputs, so it must not read them as constant data.  No such kernel takes a
``__restrict__`` pointer or loads through ``__ldg``; kernels launched in plain stream order may."""
import glob
import os
import re

import pytest

from depthwise_convolution_nhwc_gb300 import _build


def closing(text, at, pair):
    """Index behind the bracket that closes the one at `at`."""
    depth = 0
    for i in range(at, len(text)):
        depth += (text[i] == pair[0]) - (text[i] == pair[1])
        if depth == 0:
            return i + 1
    raise ValueError("no closing bracket")


def kernels(source):
    """(name, parameters, body) of every kernel defined in a source text."""
    text = re.sub(r"//[^\n]*", "", source)
    for m in re.finditer(r"__global__\s+void\s+", text):
        at = m.end()
        while True:          # (attributes with arguments of their own come before the name)
            name = re.match(r"\s*(\w+)\s*\(", text[at:])
            start = at + name.end() - 1
            end = closing(text, start, "()")
            if name.group(1) != "__launch_bounds__":
                break
            at = end
        rest = text[end:].lstrip()
        if not rest.startswith("{"):
            continue         # a declaration
        body = text.index("{", end)
        yield name.group(1), text[start:end], text[body:closing(text, body, "{}")]


def test_kernels_are_found():
    src = "__global__ void __launch_bounds__(f(2), 1)\nk(const float* __restrict__ p) { if (p) { g(); } }\n__global__ void d(int);"
    assert list(kernels(src)) == [("k", "(const float* __restrict__ p)", "{ if (p) { g(); } }")]


SOURCES = sorted(glob.glob(os.path.join(_build.CSRC, "*.cu")) + glob.glob(os.path.join(_build.CSRC, "*.cuh")))


def test_dependents_read_nothing_as_constant():
    waiting = 0
    for path in SOURCES:
        with open(path) as f:
            for name, params, body in kernels(f.read()):
                if "pdl_wait()" not in body:
                    continue
                waiting += 1
                where = f"{os.path.basename(path)}: {name}"
                assert "__restrict__" not in params, where
                assert "__ldg(" not in body and ".global.nc" not in body, where
    assert waiting >= 15
