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
typedef unsigned long long u64;
struct Word {
    u64* p;
    u64 swap(u64 v) const { u64 old = *p; *p = v; return old; }
    void set(u64 v) const { *p = v; }
};
extern "C" {
int last_part(const int* desc, int c, int runs) { return qm::attend::last_part(desc, c, runs); }
u64 swap(u64* flag, u64 v) { return Word{flag}.swap(v); }
void take_back(u64* flag, u64 before, u64 mark) { qm::attend::take_back(Word{flag}, before, mark); }
int item_each(int items, int most, int64_t total, int used, int runs, int cost) { return qm::attend::item_each(items, most, total, used, runs, cost); }
int give_up(u64* flag, u64 mark) { return qm::attend::give_up(Word{flag}, mark); }
}
"""


@pytest.fixture(scope="module")
def parts(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("parts")
    (d / "parts.cpp").write_text(SOURCE)
    lib = str(d / "parts.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-I", CSRC, "-o", lib, str(d / "parts.cpp")], check=True)
    lib = ctypes.CDLL(lib)
    word, flag = ctypes.c_uint64, ctypes.POINTER(ctypes.c_uint64)
    lib.swap.argtypes, lib.swap.restype = [flag, word], word
    lib.take_back.argtypes, lib.take_back.restype = [flag, word, word], None
    lib.give_up.argtypes, lib.give_up.restype = [flag, word], ctypes.c_int
    return lib


def test_an_item_to_each_cta(parts):
    def each(items, most, total, runs=152):
        return bool(parts.item_each(items, most, ctypes.c_int64(total), min(runs, total), runs, 8))

    assert each(152, 9, 152) and not each(153, 9, 153)
    assert each(10, 18, 1520) and not each(10, 19, 1520)
    assert not each(0, 0, 0)  # no sequence has rows: no run to take a share of


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


# ---------------------------------------------------------------- the flags of attend_rows_kernel
MARK = 0x9E3779B97F4A7C15


class Replay:
    """One run of a captured call: a part's CTA and the item's joiner over one flag, each step an exchange or a store."""

    def __init__(self, parts, flag):
        self.parts, self.flag = parts, flag

    def part_is_there(self):
        before = self.parts.swap(ctypes.byref(self.flag), MARK)
        self.parts.take_back(ctypes.byref(self.flag), before, MARK)

    def seen(self):
        return self.flag.value == MARK

    def joined(self):
        self.flag.value = 0

    def gives_up(self):
        return bool(self.parts.give_up(ctypes.byref(self.flag), MARK))


@pytest.mark.parametrize("held", [0, 1, 12345, MARK ^ 2])  # what the workspace held
def test_no_flag_stays_at_its_mark_whatever_ends_a_call(parts, held):
    def replay():
        r = Replay(parts, flag)
        assert not r.seen()  # nothing of an earlier replay is taken for this one's
        return r

    def plain():
        r = replay()
        r.part_is_there()
        assert r.seen()
        r.joined()

    flag = ctypes.c_uint64(held)
    plain()
    for late in (False, True):
        r = replay()
        if late:  # the joiner's wait gave up, then the part came
            assert not r.gives_up()
            assert not r.seen()
            r.part_is_there()
        else:  # it came between the joiner's last look and its giving up
            r.part_is_there()
            assert r.gives_up()
        assert flag.value == 0
        plain()
        plain()
