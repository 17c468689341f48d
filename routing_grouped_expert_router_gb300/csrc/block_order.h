// block_order.h -- which kernel, tile and piece of a block-scaled product comes
// when: integer arithmetic alone, the same on the host and on the device, in 32
// bits wherever the device does it.
#pragma once

#ifdef __CUDACC__
#define MOE_BOTH __host__ __device__ __forceinline__
#else
#define MOE_BOTH inline
#endif

namespace moe {

constexpr int kBlock = 128;
inline int blocks_of(int n) { return (n + kBlock - 1) / kBlock; }

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

// Whether a group's rows are so few that gemm_block_few.cu's kernel is the faster one where
// another of these launches comes before it (whose end its first weights need not wait for).
// The feed-forward block in a graph, us, that kernel against the pairs':
//   rows to a group           1          8          16         24         32
//   4096, 14336, 1 group      41 : 79    43 : 74    45 : 71    53 : 72    55 : 71
//   4096, 4096, 1 group       23 : 43    25 : 40    27 : 39    35 : 40    37 : 41
//   2048, 1408, 1 group       16 : 26    17 : 26    18 : 26    23 : 26    24 : 26
//   2048, 1408, 8 groups      24 : 42    25 : 41    28 : 42    39 : 42    40 : 42
//   4096, 2048, 4 groups      30 : 50    30 : 49    37 : 49    59 : 49    60 : 49
//   4096, 14336, 8 groups     283 : 382  289 : 319  294 : 320  316 : 323  318 : 324
//   2048, 1408, 64 groups     122 : 172  126 : 160  137 : 161  165 : 164  172 : 165
// The steps of such a launch are counted in 32 bits.
inline bool few_rows(int rows, int E, int K, int N) {
  return rows <= (E == 1 ? 32 : 16ll * E) && (rows / 16 + E) * (N / 128 + 1ll) * blocks_of(K) < 2147483647ll;
}
// The same for a product by itself, whose weights may be what the launch before writes: the
// rows have to fit its smallest tile (16, twice a group's mean), or the weights' stream to be
// long beside the join.  Products in a graph, us, as above:
//   rows to a group           1          4          8          16         32
//   4096 x 14336, 1 group     16 : 26    16 : 20    16 : 19    17 : 20    19 : 20
//   4096 x 4096, 1 group      10 : 17    10 : 16    12 : 15    13 : 15    19 : 15
//   8192 x 2048, 1 group      13 : 18    12 : 18    15 : 18    18 : 18    28 : 18
//   14336 x 4096, 1 group     17 : 29    17 : 27    18 : 24    20 : 24    26 : 24
//   2048 x 1408, 8 groups     12 : 13    12 : 12    12 : 12    14 : 13    19 : 13
//   4096 x 1024, 8 groups     13 : 18    13 : 18    14 : 18    16 : 18    22 : 18
//   512 x 2048, 64 groups     23 : 23    23 : 23    24 : 24    27 : 24    33 : 26
//   2048 x 640, 64 groups     24 : 29    25 : 29    25 : 29    27 : 30    36 : 30
//   2048 x 1408, 64 groups    40 : 50    41 : 50    43 : 52    46 : 53    55 : 52
//   4096 x 14336, 8 groups    78 : 120   79 : 92    81 : 93    83 : 95    89 : 97
inline bool few_rows_alone(int rows, int E, int K, int N) {
  return few_rows(rows, E, K, N) &&
         (rows <= (E == 1 ? 16 : 8ll * E) || 1ll * E * K * N > 64ll << 20);
}
// Activations to a tile: 16 where they hold twice a group's mean (one group: all rows), or 32,
// which do for all that few_rows lets through.
inline int few_tile_rows(int rows, int E) {
  return (E == 1 ? rows : 2 * ((rows + E - 1) / E)) <= 16 ? 16 : 32;
}

// How all steps, nkb to a tile, are cut into contiguous pieces, one for each block.  Where every
// tile can have the same number of pieces (per > 0) and enough blocks get one, no block has parts
// of two tiles, and its first load comes sooner; otherwise all steps are cut into equal pieces.
// The first `longer` pieces (of each tile, or of all) have a step more than the others' `each`.
// Enough: three quarters of the blocks stream as fast as all; with fewer, 5 ns a step in the
// ratio stay below the 3 us that parts of two tiles cost.  In a graph, us, alike and not: one row
// by 4096 and 14336 (112 tiles of 152) 41 46, 8 experts of 2048 and 1408 (88) 24.6 28.4.
// In 32 bits (see few_rows).
constexpr int kMinSteps = 4;  // pieces of fewer cost more to join than they save
struct Share {
  int nkb, per, each, longer;
  int t, kb, count;  // this block's first tile and step, its steps
  MOE_BOTH int lo(int c) const { return each * c + (c < longer ? c : longer); }
  MOE_BOTH int owner(int s) const {
    const int edge = (each + 1) * longer;
    return s < edge ? s / (each + 1) : longer + (s - edge) / each;
  }
};
// The share of block `me` of `grid`.
MOE_BOTH Share share_of(int tiles, int nkb, int grid, int me) {
  const int steps = tiles * nkb;
  Share share = {nkb, 0, 0, 0, 0, 0, 0};
  if (steps == 0) return share;
  if (tiles <= grid) {
    const int most = nkb / kMinSteps, room = grid / tiles;
    const int per = most < 1 ? 1 : room < most ? room : most, used = tiles * per;
    if ((per + 1) * kMinSteps > nkb ||
        static_cast<long long>(steps) * (3 * grid - 4 * used) <= 2400ll * used) {
      share.per = per;
      share.each = nkb / per;
      share.longer = nkb - share.each * per;
      share.t = me / per;
      const int piece = me - share.t * per;
      share.kb = share.lo(piece);
      share.count = share.t < tiles ? share.each + (piece < share.longer) : 0;
      return share;
    }
  }
  const int most = steps / kMinSteps;
  const int blocks = most < 1 ? 1 : most < grid ? most : grid;
  share.each = steps / blocks;
  share.longer = steps - share.each * blocks;
  // blocks past the pieces: none
  const int lo = me < blocks ? share.lo(me) : steps;
  share.count = (me + 1 < blocks ? share.lo(me + 1) : steps) - lo;
  share.t = lo / nkb;
  share.kb = lo - share.t * nkb;
  return share;
}

}  // namespace moe
