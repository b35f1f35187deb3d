"""The choice of a product's kernel, compiled for the host: what it counts
cannot be more than the launch has."""

import shutil
import subprocess

import pytest

from tile_size_decision_gb300 import build

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>

#include "product_choice.h"

// Seven numbers a product (fp8 m n k groups sms pairs); a line of the choice each.
int main(int argc, char** argv) {
    for (int i = 1; i + 6 < argc; i += 7) {
        auto v = [&](int j) { return std::atoll(argv[i + j]); };
        const tiles::Choice c = tiles::choose(v(0) != 0, v(1), v(2), v(3), v(4),
                                              static_cast<int>(v(5)), static_cast<int>(v(6)));
        std::printf("%d %d %d %d\n", c.pair, c.rows, c.cols, c.split);
    }
}
"""


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("needs a C++ compiler")
    d = tmp_path_factory.mktemp("choice")
    (d / "choice.cpp").write_text(PROGRAM)
    exe = str(d / "choice")
    subprocess.run([cxx, "-O1", "-std=c++17", "-I", build.CSRC, "-o", exe, str(d / "choice.cpp")],
                   check=True)

    def run(products, sms=152, pairs=76):
        args = [str(int(v)) for p in products for v in (*p, sms, pairs)]
        out = subprocess.run([exe, *args], check=True, capture_output=True, text=True).stdout
        return [tuple(int(v) for v in line.split()) for line in out.splitlines()]

    return run


@pytest.mark.parametrize("fp8", [0, 1])
def test_groups_that_cannot_have_rows_change_nothing(choose, fp8):
    sizes = [(n, k) for n in (128, 2048, 4096) for k in (256, 2048, 4096)]
    for m in (1, 2, 5, 8, 16):
        same = choose([(fp8, m, n, k, m) for n, k in sizes])
        for groups in (16, 32, 64, 256, 4096):
            if groups >= m:
                assert choose([(fp8, m, n, k, groups) for n, k in sizes]) == same, (m, groups)


@pytest.mark.parametrize("fp8", [0, 1])
def test_one_row_of_many_groups_is_split_like_a_dense_row(choose, fp8):
    # One row tile, 16 blocks of 128 columns, 152 SMs: eight CTAs along K.
    assert choose([(fp8, 1, 2048, 4096, 32)]) == choose([(fp8, 1, 2048, 4096, 0)])
    (pair, rows, _, split), = choose([(fp8, 1, 2048, 4096, 32)])
    assert not pair and rows == 16 and split == 8


def test_the_choice_is_one_the_kernels_have(choose):
    for fp8 in (0, 1):
        ps = [(fp8, m, n, k, g) for m in (1, 17, 300, 5000, 32768) for n in (8, 200, 2048)
              for k in (16, 1024, 4096) for g in (0, 1, 7, 32, 300)]
        for pair, rows, cols, split in choose(ps):
            if pair:
                assert rows == 256 and split == 1 and cols % 32 == 0
                assert 64 <= cols <= 256 if fp8 else cols == 256
            else:
                assert rows in (16, 32, 64) and cols == 128 and split in (1, 2, 4, 8)
