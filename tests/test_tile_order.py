"""Which tile a workgroup of the 8-bit tile kernel works on, compiled for the
host: every tile once, and no tile outside the map whatever the number of
tiles says (it comes from device memory)."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import memory_bound_mxfp4_amd as moe

CSRC = os.path.join(os.path.dirname(moe.LIB_PATH), "csrc")
SOURCE = """
#include "tile_order.h"
extern "C" void tiles(int blocks, int tiles_n, int tiles_m, int count, int parts, int band, int* out) {
  for (int b = 0; b < blocks; ++b) {
    const moe::TileAt t = moe::tile_at(b, tiles_n, tiles_m, count, parts, band);
    out[4 * b] = t.any;
    out[4 * b + 1] = t.tm;
    out[4 * b + 2] = t.tn;
    out[4 * b + 3] = t.part;
  }
}
"""


@pytest.fixture(scope="module")
def tiles(tmp_path_factory):
    where = tmp_path_factory.mktemp("tile_order")
    src, so = str(where / "tiles.cpp"), str(where / "tiles.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run(["g++", "-O1", "-fwrapv", "-std=c++17", "-shared", "-fPIC", "-D__host__=", "-D__device__=",
                    "-D__forceinline__=inline", "-I", CSRC, src, "-o", so], check=True)
    lib = ctypes.CDLL(so)

    def run(tiles_n, tiles_m, count, parts, band):
        blocks = 8 * ((tiles_n * tiles_m * parts + 7) // 8)
        out = np.zeros((blocks, 4), np.int32)
        lib.tiles(blocks, tiles_n, tiles_m, count, parts, band, ctypes.c_void_p(out.ctypes.data))
        return out[out[:, 0] != 0, 1:]
    return run


SIZES = [(1, 1, 1, 1), (28, 191, 1, 2), (28, 191, 1, 8), (7, 13, 1, 8), (112, 3, 8, 8), (24, 1, 3, 8), (56, 961, 1, 1)]


@pytest.mark.parametrize("tiles_n,tiles_m,parts,band", SIZES)
def test_every_tile_once(tiles, tiles_n, tiles_m, parts, band):
    for count in sorted({0, 1, tiles_m // 2, tiles_m - 1, tiles_m}):
        got = tiles(tiles_n, tiles_m, count, parts, band)
        want = [(m, n, p) for m in range(count) for n in range(tiles_n) for p in range(parts)]
        assert sorted(map(tuple, got.tolist())) == want, count


@pytest.mark.parametrize("tiles_n,tiles_m,parts,band", SIZES)
def test_any_count_stays_in_the_map(tiles, tiles_n, tiles_m, parts, band):
    """An unfilled buffer: the product of a negative count and the columns can wrap to a positive number of tiles."""
    rng = np.random.default_rng(tiles_m)
    counts = [-2 ** 31, -1331422904, -2 ** 30, -1, tiles_m + 1, 2 ** 31 - 1]
    counts += rng.integers(-2 ** 31, 2 ** 31, 60).tolist()
    for count in counts:
        got = tiles(tiles_n, tiles_m, count, parts, band)
        assert ((got >= 0) & (got < [tiles_m, tiles_n, parts])).all(), (count, got.max(0))
        assert len(got) == (0 if count <= 0 else tiles_n * tiles_m * parts if count >= tiles_m else len(got)), count
