// block_order.h -- which tile of a block-scaled product comes when: integer
// arithmetic alone, the same on the host and on the device, in 32 bits wherever
// the device does it.
#pragma once

#ifdef __CUDACC__
#define MOE_BOTH __host__ __device__ __forceinline__
#else
#define MOE_BOTH inline
#endif

namespace moe {

// The most rows of a call: a row's number, a tile's 256 rows further on, fits 31 bits.
constexpr int kMostRows = 2147483647 - 511;
// The longest contraction and the most columns.
constexpr int kMostWidth = 1 << 20;

// The tiles of a group of rows: bands of `group` row tiles (or, raster_n, column tiles), each
// swept along the other side, so that the tiles under way share what L2 holds.
struct TileOrder {
  int raster_n, group;
};
struct TileAt {
  int m, n;  // row tile of the group, column tile
};
// Tile `local` of a group of MT x NT tiles.
MOE_BOTH TileAt tile_at(const TileOrder& o, int MT, int NT, int local) {
  const int wide = o.raster_n ? NT : MT, along = o.raster_n ? MT : NT;
  const int band = local / (o.group * along);
  const int base = band * o.group;
  const int size = o.group < wide - base ? o.group : wide - base;
  const int r = local - band * o.group * along;
  const int u = base + r % size, v = r / size;
  return o.raster_n ? TileAt{v, u} : TileAt{u, v};
}

// The smaller operand of a group stays in L2 where it fits, in one band; otherwise bands of
// sixteen tiles.  a_bytes, b_bytes: a group's rows and its weight; slab_a, slab_b: one row
// tile's and one column tile's share of them; MT, NT: the most tiles of a group.  A band is no
// wider than the tiles there are, so that a band's tiles are no more than a group's and fit 31
// bits as those do.
inline TileOrder tile_order(long long a_bytes, long long b_bytes, long long slab_a,
                            long long slab_b, long long MT, long long NT) {
  constexpr long long kL2ResidentBytes = 48ll << 20;
  TileOrder o = {0, 16};
  long long fit = 16;
  if (a_bytes <= kL2ResidentBytes && a_bytes <= b_bytes) {
    fit = kL2ResidentBytes / slab_a;
  } else if (b_bytes <= kL2ResidentBytes) {
    o.raster_n = 1;
    fit = kL2ResidentBytes / slab_b;
  }
  const long long wide = o.raster_n ? NT : MT;
  if (fit > wide) fit = wide;
  o.group = static_cast<int>(fit < 1 ? 1 : (fit > 4096 ? 4096 : fit));
  return o;
}

}  // namespace moe
