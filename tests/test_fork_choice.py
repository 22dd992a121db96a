"""Which form smla_fork_block_tables takes (CPU: the host's rule, compiled by itself)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "sparse_mla_attention_04_gb300")


@pytest.fixture(scope="module")
def by_one_block(tmp_path_factory):
    from sparse_mla_attention_04_gb300 import build
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    at = tmp_path_factory.mktemp("fork")
    (at / "rule.cpp").write_text("""
#include "smla_step.h"
#include <cstdio>
#include <cstdlib>
int main(int argc, char **argv)
{
    for (int i = 1; i + 2 < argc; i += 3)
        std::printf("%d", (int)smla::fork_by_one_block(std::atoi(argv[i]), std::atoi(argv[i + 1]), std::atoi(argv[i + 2])));
}
""")
    cxx = shutil.which("g++") or "c++"
    subprocess.run([cxx, "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I", os.path.join(PKG, "csrc"), "-I",
                    os.path.join(ROOT, "include"), "-I", cuda, str(at / "rule.cpp"), "-o", str(at / "rule")], check=True)

    def rule(*cases):
        args = [str(x) for c in cases for x in c]
        return [x == "1" for x in subprocess.run([str(at / "rule")] + args, capture_output=True, text=True, check=True).stdout]
    return rule


def test_rows_up_to_the_limits(by_one_block):
    """2^30 old and 2^30 new rows are 2^31 in all: never one block's work."""
    most = 1 << 30
    large = [(most, most, 0), (most, most, 1), (most, most - 1, 1), (most, 0, 1), (0, most, 0), (1, 1, most), (7, 5, 100000000)]
    assert by_one_block(*large) == [False] * len(large)
    assert by_one_block((0, 0, 0), (1, 4, 8), (0, 3, 4), (3, 0, 4), (1, 1, 1)) == [True] * 5


def test_a_row_is_a_unit_however_narrow(by_one_block):
    """One block has 32 warps, a unit of up to 256 entries of one row to each: more units than that go to the phases."""
    for few in ((16, 16, 256), (1, 31, 1), (31, 1, 0), (1, 1, 4096), (1, 4, 600), (3, 5, 700)):
        assert by_one_block(few) == [True], few
    for many in ((16, 17, 1), (16, 16, 257), (256, 256, 2), (1000, 1000, 2), (4000, 4000, 1), (1, 1, 4097), (64, 64, 8)):
        assert by_one_block(many) == [False], many
