// tile_order.h -- the tile that a workgroup of the 8-bit tile kernel works on.
// Integer arithmetic alone; the tests compile it for the host.
// Internal to libmoe_mxfp4.so.
#pragma once

namespace moe {

struct TileAt {
  bool any;          // false: this workgroup has none
  int tm, tn, part;  // tile row, tile column, part of a split K
};

// Workgroups go to the 8 XCDs in turn; each XCD gets one
// contiguous run of tiles, in bands of `band_rows` tile rows walked column by column,
// so that the tiles its CUs work on at a time share rows of x and of the
// matrix in its L2.  A band of 8 in a dense product (both are read again and
// again); in a grouped one about the tile rows of an expert, so that its rows
// stay in L2 while its matrix, which nobody else needs, streams by once.
// tiles_m: the tile rows the grid was sized for; count: those there are, a number
// from device memory that may be anything (a groups buffer that was never filled), so
// it is brought into 0 .. tiles_m before it is multiplied.
__host__ __device__ __forceinline__ TileAt tile_at(unsigned block, int tiles_n, int tiles_m, int count, int parts,
                                                   int band_rows) {
  TileAt o{false, 0, 0, 0};
  if (count < tiles_m) tiles_m = count < 0 ? 0 : count;
  const int tiles = tiles_n * tiles_m, per_xcd = (tiles * parts + 7) / 8;
  int id = (int)(block & 7) * per_xcd + (int)(block >> 3);
  if ((int)(block >> 3) >= per_xcd || id >= tiles * parts) return o;
  o.part = id / tiles;
  id -= o.part * tiles;
  const int band = id / (band_rows * tiles_n), in = id - band * band_rows * tiles_n;
  const int rest = tiles_m - band * band_rows, high = rest < band_rows ? rest : band_rows;
  o.tn = in / high;
  o.tm = band * band_rows + in - o.tn * high;
  o.any = true;
  return o;
}

}  // namespace moe
