"""The walk of a workgroup that goes on from tile to tile, compiled for the
host: whatever tiles it passes, every tile is met once."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import memory_bound_mxfp4_amd as moe
from test_tile_order import SIZES

CSRC = os.path.join(os.path.dirname(moe.LIB_PATH), "csrc")
SOURCE = """
#include "tile_order.h"
// how often each tile is met by the workgroups of a grid, which pass those that `passed` names
extern "C" void walks(int grid, int tiles_n, int tiles_m, int count, int parts, int band, const char* passed, int* met) {
  for (int b = 0; b < grid; ++b) {
    auto locate = [&](unsigned& block) {  // the next tile that is not passed
      for (;;) {
        const moe::TileAt t = moe::next_tile(block, grid, tiles_n, tiles_m, count, parts, band);
        if (!t.any) return false;
        const int at = (t.tm * tiles_n + t.tn) * parts + t.part;
        ++met[at];
        if (!passed[at]) return true;
      }
    };
    for (unsigned block = b; locate(block);) {
    }
  }
}
"""


@pytest.fixture(scope="module")
def walks(tmp_path_factory):
    where = tmp_path_factory.mktemp("tile_walk")
    src, so = str(where / "walks.cpp"), str(where / "walks.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run(["g++", "-O1", "-fwrapv", "-std=c++17", "-shared", "-fPIC", "-D__host__=", "-D__device__=",
                    "-D__forceinline__=inline", "-I", CSRC, src, "-o", so], check=True)
    lib = ctypes.CDLL(so)

    def run(grid, tiles_n, tiles_m, count, parts, band, passed):
        passed = np.ascontiguousarray(passed, np.int8)
        met = np.zeros(len(passed), np.int32)
        lib.walks(grid, tiles_n, tiles_m, count, parts, band, ctypes.c_void_p(passed.ctypes.data),
                  ctypes.c_void_p(met.ctypes.data))
        return met
    return run


@pytest.mark.parametrize("grid", [8, 16, 256])
@pytest.mark.parametrize("tiles_n,tiles_m,parts,band", SIZES)
def test_a_walk_meets_every_tile_once(walks, tiles_n, tiles_m, parts, band, grid):
    """No tile is passed, all, those at the end (a padded batch's slots without an expert), some, most."""
    rng = np.random.default_rng(tiles_m)
    size = tiles_n * tiles_m * parts
    row = np.arange(size) // (tiles_n * parts)
    for count in sorted({0, 1, tiles_m // 2, tiles_m}):
        for passed in (row < 0, row >= 0, row >= count - count // 9, rng.random(size) < 0.3, rng.random(size) < 0.9):
            met = walks(grid, tiles_n, tiles_m, count, parts, band, passed)
            assert (met == (row < count)).all(), (count, met.max(), np.argwhere(met != (row < count))[:4])
