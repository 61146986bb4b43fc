"""The kernel that the 8-bit product takes for a shape (host arithmetic, CPU only): the shapes that the GPU
tests run reach every kernel that the planner can return, so that a change of its costs cannot take
one of them out of the tests unseen."""

import math
import os
import random
import shutil
import subprocess

import pytest

from w8a8_shapes import AT_LARGEST_PITCH, LARGEST_PITCH, PLANS

SRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "native", "w8a8_plans.cpp")


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    exe = str(tmp_path_factory.mktemp("plans") / "plans")
    subprocess.run([cxx, "-O2", "-std=c++17", "-Wall", "-Werror", "-o", exe, SRC], check=True)

    def ask(queries):
        """(tile, parts, tail, shifted) of each (M, N, K, may_split, byte of a cache line, pitch)."""
        text = "\n".join(" ".join(str(v) for v in q) for q in queries)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.split()
        return [(out[i], int(out[i + 1]), out[i + 2], int(out[i + 3])) for i in range(0, len(out), 4)]

    return ask


def test_listed_shapes_take_the_kernels_they_name(plans):
    got = plans([(M, N, K, 1, 0, K) for M, N, K, *_ in PLANS])
    wrong = [(p, g) for p, g in zip(PLANS, got) if tuple(p[3:]) != g]
    assert not wrong
    got = plans([(M, N, K, 1, 0, LARGEST_PITCH) for M, N, K, *_ in AT_LARGEST_PITCH])
    assert got == [tuple(p[3:]) for p in AT_LARGEST_PITCH]


def _kind(plan):
    tile, parts, tail, off = plan
    return tile, parts > 1, tail, off


def test_no_shape_takes_a_kernel_that_is_not_listed(plans):
    rng = random.Random(11)
    log = lambda lo, hi: int(math.exp(rng.uniform(math.log(lo), math.log(hi))))   # noqa: E731
    shapes = [(log(9, 80000), log(1, 40000), max(16, log(16, 131000) // 16 * 16)) for _ in range(200000)]
    found = {_kind(p) for p in plans([(*s, 1, 0, s[2]) for s in shapes])}
    assert found == {_kind(p[3:]) for p in PLANS}


def test_two_output_alignments_and_unequal_parts_for_each_kernel():
    for kind in {_kind(p[3:]) for p in PLANS}:
        mine = [p for p in PLANS if _kind(p[3:]) == kind]
        assert {p[1] % 8 == 0 for p in mine} == {True, False}
        assert all(p[4] == 1 or (p[2] + 127) // 128 % p[4] for p in mine)


def test_rows_off_the_lines_by_pitch_or_by_start_are_shifted(plans):
    assert [p[3] for p in plans([(300, 2000, 2048, 1, 0, 2048), (300, 2000, 2048, 1, 0, 2064), (300, 2000, 2048, 1, 16, 2048),
                                 (300, 2000, 1024, 1, 16, 1040)])] == [0, 1, 1, 0]
