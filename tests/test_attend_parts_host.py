"""How the CTAs that share an item of cache_attend tell of its parts: the kernels' own text
(csrc/qm_attend_parts.h), compiled for the host."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "packed_qmatmul_gb300", "csrc")

SOURCE = r"""
#include "qm_attend_parts.h"
extern "C" int last_part(const int* desc, int c, int runs) { return qm::attend::last_part(desc, c, runs); }
"""


@pytest.fixture(scope="module")
def parts(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("parts")
    (d / "parts.cpp").write_text(SOURCE)
    lib = str(d / "parts.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-I", CSRC, "-o", lib, str(d / "parts.cpp")], check=True)
    return ctypes.CDLL(lib)


def last_part(parts, desc, c):
    return parts.last_part(desc.ctypes.data_as(ctypes.c_void_p), c, len(desc))


def descriptors(items, runs):
    """Of runs whose items [first, last] are split between CTAs."""
    d = np.zeros((runs, 8), np.int32)
    for first, last in items:
        d[first, 1:7] = 1, 7, 1, 256, 200, 90
        d[first + 1: last, 0] = 1
        d[last, 0] = 2
    return d


def test_parts_of_split_items(parts):
    d = descriptors([(0, 1), (1, 4), (6, 9)], 10)
    assert [last_part(parts, d, c) for c in range(10)] == [1, 4, -1, -1, -1, -1, 9, -1, -1, -1]


@pytest.mark.parametrize("gone", range(10))
def test_an_item_with_a_missing_part_is_not_joined(parts, gone):
    """A CTA whose wait gave up publishes no descriptor: no item that it has a part of is joined, the others are."""
    items = [(0, 1), (1, 4), (6, 9)]
    d = descriptors(items, 10)
    d[gone] = 0
    want = [-1] * 10
    for first, last in items:
        if not first <= gone <= last:
            want[first] = last
    assert [last_part(parts, d, c) for c in range(10)] == want


def test_no_descriptor_past_the_last_run_is_looked_at(parts):
    d = descriptors([(2, 5)], 8)
    d[6:] = 2  # not part of the runs below
    d[3:6, 0] = 1
    assert parts.last_part(d.ctypes.data_as(ctypes.c_void_p), 2, 6) == -1
    assert parts.last_part(d.ctypes.data_as(ctypes.c_void_p), 5, 6) == -1
