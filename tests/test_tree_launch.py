"""How a launch of the tree attention picks its slices (csrc/tree_launch.h, host code), with made-up
answers in the device's place."""

import os
import shutil
import subprocess

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "structured_sparse_attention_b200", "csrc")

PROGRAM = r"""
#include <cassert>
#include <cstdio>

#include "tree_launch.h"

using namespace ssa;

int asked;

int main() {
    // clusters of k CTAs on a device of n places
    auto of = [](int n) { return [n](int k) { ++asked; return n / k; }; };
    {
        static ClusterCounts c;
        assert(pick_slices(c, 0, 1, 8, of(148)) == 8 && pick_slices(c, 0, 18, 8, of(148)) == 8);
        assert(pick_slices(c, 0, 19, 8, of(148)) == 7 && pick_slices(c, 0, 75, 8, of(148)) == 1);
        assert(pick_slices(c, 0, 1, 3, of(148)) == 3 && pick_slices(c, 0, 1, 0, of(148)) == 1);
        const int before = asked;  // every number has been asked for by now: never again
        assert(pick_slices(c, 0, 37, 8, of(148)) == 4 && asked == before);
    }
    {  // each device answers for itself
        static ClusterCounts c;
        assert(pick_slices(c, 0, 20, 8, of(160)) == 8);
        assert(pick_slices(c, 1, 20, 8, of(80)) == 4);
        assert(pick_slices(c, 0, 20, 8, of(160)) == 8);
        assert(pick_slices(c, 63, 20, 8, of(40)) == 2 && pick_slices(c, 64, 20, 8, of(160)) == 8);
    }
    {  // no answer: none for this call, asked again by the next
        static ClusterCounts c;
        assert(pick_slices(c, 2, 1, 8, [](int) { return -1; }) == 1);
        assert(pick_slices(c, 2, 1, 8, [](int k) { return k > 4 ? -1 : 148 / k; }) == 4);
        assert(pick_slices(c, 2, 1, 8, of(148)) == 8);
    }
    {  // none at all is an answer
        static ClusterCounts c;
        assert(pick_slices(c, 0, 1, 8, of(0)) == 1);
        const int before = asked;
        assert(pick_slices(c, 0, 1, 8, of(148)) == 1 && asked == before);
    }
    std::puts("ok");
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ is not installed")
def test_pick_slices(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, "-o", str(exe), str(src)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout == "ok\n", out.stderr
