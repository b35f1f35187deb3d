"""The lookup of a row tile among ragged groups, on 32 host threads that stand
for a warp's lanes: the units that name the tiles come in no promised order."""

import shutil
import subprocess

import numpy as np
import pytest

from tile_size_decision_gb300 import build

PROGRAM = r"""
#include <algorithm>
#include <condition_variable>
#include <cstdio>
#include <cstdlib>
#include <mutex>
#include <thread>
#include <vector>

#include "row_tiles.h"

std::mutex mu;
std::condition_variable cv;
int waiting = 0, turn = 0;
int value[32];
thread_local int self;

void meet() {
    std::unique_lock<std::mutex> lock(mu);
    const int mine = turn;
    if (++waiting == 32) {
        waiting = 0;
        ++turn;
        cv.notify_all();
    } else {
        cv.wait(lock, [&] { return turn != mine; });
    }
}

struct Threads {
    static int lane() { return self; }
    static int first(unsigned mask) { return __builtin_ffs(static_cast<int>(mask)) - 1; }
    static int shfl(int v, int src) {
        value[self] = v;
        meet();
        const int r = value[src & 31];
        meet();
        return r;
    }
    static int shfl_up(int v, int d) { return shfl(v, self >= d ? self - d : self); }
    static unsigned ballot(bool p) {
        value[self] = p;
        meet();
        unsigned r = 0;
        for (int i = 0; i < 32; ++i) r |= static_cast<unsigned>(value[i]) << i;
        meet();
        return r;
    }
};

// tile_rows m groups offsets... -- wants...; a line "found group row0 end" each.
int main(int argc, char** argv) {
    const int tile_rows = std::atoi(argv[1]), m = std::atoi(argv[2]), groups = std::atoi(argv[3]);
    std::vector<int> offsets, wants;
    for (int i = 4; i < 5 + groups; ++i) offsets.push_back(std::atoi(argv[i]));
    for (int i = 5 + groups; i < argc; ++i) wants.push_back(std::atoi(argv[i]));
    std::vector<std::thread> lanes;
    for (int l = 0; l < 32; ++l)
        lanes.emplace_back([&, l] {
            self = l;
            tiles::RowTileLookup<Threads> cursor;
            for (int want : wants) {
                tiles::RowTile t{-1, -1, -1};
                const bool found = cursor.seek(offsets.data(), groups, m, tile_rows, want, &t);
                if (l == 0) std::printf("%d %d %d %d\n", found, t.group, t.row0, t.end);
            }
        });
    for (std::thread& t : lanes) t.join();
}
"""


@pytest.fixture(scope="module")
def lookup(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("needs a C++ compiler")
    d = tmp_path_factory.mktemp("row_tiles")
    (d / "lookup.cpp").write_text(PROGRAM)
    exe = str(d / "lookup")
    subprocess.run([cxx, "-O1", "-std=c++17", "-pthread", "-I", build.CSRC, "-o", exe,
                    str(d / "lookup.cpp")], check=True)

    def run(offsets, m, tile_rows, wants):
        args = [exe, tile_rows, m, len(offsets) - 1, *offsets, *wants]
        out = subprocess.run([str(a) for a in args], check=True, capture_output=True, text=True,
                             timeout=60).stdout
        return [tuple(int(v) for v in line.split()) for line in out.splitlines()]

    return run


def all_tiles(offsets, m, tile_rows):
    """(group, row0, end) of every tile, in group order."""
    tiles = []
    off = [min(max(int(o), 0), m) for o in offsets]
    for g, (lo, hi) in enumerate(zip(off, off[1:])):
        tiles += [(g, r, hi) for r in range(lo, hi, tile_rows)]
    return tiles


def ragged(groups, seed, most=40):
    rng = np.random.default_rng(seed)
    sizes = rng.integers(0, most, groups) * (rng.random(groups) < 0.7)
    return np.concatenate([[0], np.cumsum(sizes)])


@pytest.mark.parametrize("groups", [1, 2, 32, 33, 70, 129])
@pytest.mark.parametrize("order", ["ascending", "descending", "shuffled", "back and forth"])
def test_tiles_in_any_order(lookup, groups, order):
    offsets, rows = ragged(groups, groups), 16
    m = int(offsets[-1])
    tiles = all_tiles(offsets, m, rows)
    wants = list(range(len(tiles) + 3))              # a few past the last one
    if order == "descending":
        wants.reverse()
    elif order == "shuffled":
        np.random.default_rng(1).shuffle(wants)
    elif order == "back and forth":
        wants = [w for i in range((len(wants) + 1) // 2) for w in (wants[-1 - i], wants[i])]
    got = lookup(offsets, m, rows, wants)
    assert len(got) == len(wants)
    for want, (found, *tile) in zip(wants, got):
        if want < len(tiles):
            assert found and tuple(tile) == tiles[want], want
        else:
            assert not found, want


def test_offsets_past_the_rows_and_descending_pairs(lookup):
    offsets = [-5, 20, 10, 10, 90, 200]
    tiles = all_tiles(offsets, 64, 16)
    got = lookup(offsets, 64, 16, range(len(tiles) + 1))
    assert [t[1:] for t in got[:-1]] == tiles and not got[-1][0]
