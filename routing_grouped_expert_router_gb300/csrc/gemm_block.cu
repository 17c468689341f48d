// gemm_block.cu -- grouped products of e4m3 codes with a float32 scale for each
// block of 128 (see block.cuh):
//   C[p, n] = sum_b sa[b, p] sb[e, b, n/128] sum_{k in block b} qa[p, k] qb[e, k, n]
// in four forms: the plain product, FC1 with SwiGLU and H's codes, FC2's data
// gradient with the SwiGLU backward and its codes, and FC1's data gradient (two
// products in one sum).
//
// A persistent kernel of CTA pairs (tcgen05.mma.cta_group::2, 256 rows x 256
// columns, 128 deep).  The scales change with every block of the contraction, so
// tensor memory holds one block's sums only: eight warps a CTA take them out,
// times the row's and the column block's scale, and add them to sums in
// registers, 64 x 2 for each of 256 threads, while the tensor cores work on the
// next block in another accumulator.  Roles of a CTA's 384 threads:
//   warps 0, 2  TMA producers of A (128 rows a stage) and B (128 columns a stage)
//   warp 1      tensor memory; in the even CTA the MMA issuer of the pair
//   warp 3      scales: places the tiles and copies each block's 128 row scales and
//               its columns' into a ring of slots, up to SLOTS * GROUP blocks ahead
//               (the way through a busy L2 takes some 2000 cycles, more than two
//               blocks' sums; read by the sum warps themselves, two blocks ahead, the
//               scales held those up for 700 cycles every two blocks)
//   warps 4-11  the sums (warp w: TMEM lanes 32 (w mod 4), columns 64 ((w-4)/4)
//               of each half) and, at a tile's end, its epilogue
// The weight's square blocks let both uses of a weight, as it is (MN-major B)
// and transposed (K-major B), take the same codes.
//
// Where tiles are so few that two pairs or more would go to one, and the contraction is long,
// each pair takes a piece of a tile's contraction; the last to arrive adds the pieces' sums in
// their order (20 to 128 rows by 14336 x 4096: 23 to 29 us, 50 in one piece; see pieces_of).
//
// Measured: 16384 x 4096 x 14336 in eight groups, bf16 out, 716 us after a pause (2.69 PFLOP/s,
// 0.67 of twice the measured bf16 rate); in a row of calls, under the power cap, 786 to 826 us
// (2.3 to 2.4).  After a pause: 666 us without the multiply-adds, 603 without the loads from
// tensor memory too, 516 without operand loads as well.  A block takes some 900 cycles, 512 of
// them the tensor cores'; no unit is busy for more than 62% of them (the tensor pipe), and what
// holds up the others is not known.  One CTA instead of a pair, four accumulators
// of 128 columns (818 us), sixteen sum warps of half the columns (799), a block's first columns
// asked for during the block before (740) and two issuing warps were all slower; packed
// multiply-adds made no difference.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "block.cuh"
#include "block_groups.cuh"
#include "block_quant.cuh"
#include "grouped_gemm.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace moe {

namespace {

enum Form { PLAIN_BF16 = 0, PLAIN_F32 = 1, GATED = 2, GATED_BWD = 3 };

constexpr int kTimeoutCode = 5;   // MOE_ERR_DEVICE_TIMEOUT
constexpr int PM = 256;           // rows of a pair's tile
constexpr int NUM_THREADS = 384;
constexpr int FIRST_SUM_WARP = 4;
constexpr int SUM_WARPS = 8;
constexpr int LOAD_A = 0, ISSUE = 1, LOAD_B = 2, SCALES = 3;  // warps
constexpr int SET_BYTES = 2048;   // 32 rows x 64 bytes: one copy of an epilogue
constexpr int SLOTS = 4;          // groups of blocks whose scales wait for the sums
constexpr int GROUP = 4;          // blocks of a slot
constexpr int kMostPairs = kPartBlocks / 2;  // of the grid: each has room for shared sums

struct Params {
  int E;
  const int32_t* offsets;   // NULL: one group of all rows
  int rows;
  int N;                    // output columns of one weight
  int kblocks;              // blocks of the contraction of one product
  int products;             // 2: the blocks of (a1, b1) follow those of (a0, b0)
  const float* sa[2];       // activations' scales [kblocks, rows]
  const float* sb[2];       // weights' scales [E, ., .]; GATED: W1's and W3's
  int sb_group;             // scales of one group
  int sb_k, sb_n;           // strides of the contraction's and the column's block
  int nblocks;              // column blocks of one weight
  void* out[3];
  uint8_t* codes[2];
  float* scales[2];
  int* status;
  TileOrder order;          // of a group's tiles
  float* part;              // shared tiles' sums
  uint32_t* arrived;        // a byte for each CTA's rows of a shared tile
  int most_pieces;          // of a tile
};

struct Maps {
  CUtensorMap a[2], b[2];
  CUtensorMap o[3];   // outputs, boxes of 64 bytes x 32 rows
  CUtensorMap c[1];   // GATED: H's codes
  CUtensorMap i[2];   // GATED_BWD: A and B
};

// A pair's tile: NH halves of 128 columns, the even CTA loading the first, the odd the
// second (NH = 1: 64 columns each).
template <int FORM>
struct Shape {
  static constexpr int NH = FORM == GATED_BWD ? 1 : 2;
  static constexpr int COLS = 128 * NH;
  static constexpr int OUT_COLS = FORM == GATED ? 128 : COLS;  // output columns of a tile
  static constexpr int B_COLS = COLS / 2;               // B columns a CTA loads
  static constexpr int A_BYTES = 128 * 128;
  static constexpr int STAGE_BYTES = A_BYTES + B_COLS * 128;
  static constexpr int STAGES = NH == 2 ? 4 : 6;
  static constexpr int BUFS = 512 / COLS;               // accumulators in tensor memory
  // Registers of a thread: 168 at launch (3 x 168 x 128 = 64512), then FEW for warps 0-3 and
  // MANY for the others, 504 x 128 again.  What the sums spill costs more than what the
  // others do: 789 against 725 us for the product of 16384 x 4096 x 14336.
  static constexpr int FEW = FORM == GATED_BWD ? 56 : 40, MANY = (504 - FEW) / 2;
  static constexpr int SETS = 4;                        // of a warp
  static constexpr int TOPS = FORM == GATED ? 1 : FORM == GATED_BWD ? 2 : 0;
};

// The scales of up to GROUP blocks, with the place of their tile.
struct alignas(16) Slot {
  float a[128][GROUP];
  float b[2][GROUP];
  int nb, row0, row_end;   // nb < 0: no more tiles
};
template <int FORM>
struct alignas(16) Ctrl {
  using S = Shape<FORM>;
  uint64_t full[S::STAGES], empty[S::STAGES];
  uint64_t tfull[S::BUFS], tempty[S::BUFS];
  uint64_t sfull[SLOTS], sempty[SLOTS];
  uint64_t ab[SUM_WARPS];   // GATED_BWD: A and B in a warp's sets
  uint64_t met;             // the sum warps, once for each tile (TOPS)
  uint64_t join;            // the sum warps, twice for a shared tile
  uint64_t drain;
  uint32_t tmem_base;
  uint32_t last;            // whether this CTA joins the tile
  int off[kMaxGroups + 1];
  int cum[kMaxGroups + 1];       // row tiles before each group
  Slot slots[SLOTS];
  uint16_t tops[S::TOPS ? 2 * S::TOPS * 256 : 1];  // bf16 patterns [tile parity][value][side][row]
};
template <int FORM>
constexpr int smem_bytes() {
  return 1024 + Shape<FORM>::STAGES * Shape<FORM>::STAGE_BYTES +
         SUM_WARPS * Shape<FORM>::SETS * SET_BYTES + static_cast<int>(sizeof(Ctrl<FORM>));
}
static_assert(smem_bytes<PLAIN_BF16>() <= 232448 && smem_bytes<GATED>() <= 232448 &&
                  smem_bytes<GATED_BWD>() <= 232448,
              "over the 227 KiB of shared memory");

struct Tile {
  int e, nb, row0, row_end;
};

// Tile t: groups in order; within one, as p.order has them.
template <int FORM>
__device__ __forceinline__ bool place(const Params& p, const int* off, const int* cum, int t,
                                      Tile& tl) {
  const int NT = (p.N + Shape<FORM>::OUT_COLS - 1) / Shape<FORM>::OUT_COLS;
  if (t >= NT * cum[p.E]) return false;
  int e = 0, hi = p.E - 1;
  while (e < hi) {  // the last group that begins at or before t (it has rows)
    const int mid = (e + hi + 1) >> 1;
    if (NT * cum[mid] <= t)
      e = mid;
    else
      hi = mid - 1;
  }
  const int local = t - NT * cum[e];
  const TileAt at = tile_at(p.order, cum[e + 1] - cum[e], NT, local);
  tl.e = e;
  tl.nb = at.n;
  tl.row0 = off[e] + at.m * PM;
  tl.row_end = off[e + 1];
  return true;
}

// 32 columns of this thread's TMEM lane: asked for here, there after tmem_wait().
__device__ __forceinline__ void tmem_ask32(uint32_t taddr, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
        "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
        "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]),
        "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]),
        "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr));
}
// The wait names the registers that the loads fill, so that nothing reads them before.
__device__ __forceinline__ void tmem_wait(float (&v)[32]) {
  asm volatile(
      "tcgen05.wait::ld.sync.aligned;"
      : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]),
        "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]),
        "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]),
        "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]), "+f"(v[25]),
        "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29])
      :);
  asm volatile("" : "+f"(v[30]), "+f"(v[31]) : : "memory");
}
__device__ __forceinline__ void add_32(const float (&v)[32], float scale, float* sums) {
#pragma unroll
  for (int i = 0; i < 32; ++i) sums[i] = fmaf(v[i], scale, sums[i]);
}
// sigmoid and silu with the fast exponential and quotient: their few ulps are far below the
// bf16 rounding of all that is stored.  Past a = -87.3 the quotient is 0, which loses 88.8 *
// 2^-126 of silu at most.  (Two sigmoids with one reciprocal were slower.)
__device__ __forceinline__ float sigmoid_f(float a) { return __fdividef(1.0f, 1.0f + __expf(-a)); }
__device__ __forceinline__ float silu_f(float a) { return __fdividef(a, 1.0f + __expf(-a)); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ float lo_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_of(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// A warp's sets between its registers and the TMA unit: 32 rows of 64 bytes, 16-byte
// piece j of row i in slot j ^ ((i / 2) mod 4) (64-byte swizzle; no bank conflicts).  Two
// sets go out together.
struct Staging {
  uint4* sets;
  int next = 0;
  // Two sets whose last copies have been read.
  __device__ __forceinline__ uint4* take(int lane) {
    uint4* s = sets + next * (2 * SET_BYTES / 16);
    next ^= 1;
    if (lane == 0) bulk_wait_read_1();
    __syncwarp();
    return s;
  }
};
__device__ __forceinline__ int slot_of(int lane, int j) { return lane * 4 + (j ^ ((lane >> 1) & 3)); }
// Two pieces of 64 bytes (w) of each of a warp's 32 rows to out [., N] (elements of SIZE
// bytes) at (row, col) and right of it: whole rows by TMA, or, where a row is not this
// group's, each lane its own.  PIECES = 1: one piece.
template <int SIZE, int PIECES = 2>
__device__ __forceinline__ void put(Staging& st, const CUtensorMap* map, void* out, int N,
                                    const uint4 (&w)[4 * PIECES], int row, int col, bool row_ok,
                                    bool all_ok, int lane) {
  constexpr int WIDE = 64 / SIZE;
  if (col >= N) return;
  if (all_ok) {
    uint4* set = st.take(lane);
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) set[i * (SET_BYTES / 16) + slot_of(lane, j)] = w[4 * i + j];
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(map, smem_u32(set), col, row - lane);
      if (PIECES == 2 && col + WIDE < N)
        tma_store_2d(map, smem_u32(set + SET_BYTES / 16), col + WIDE, row - lane);
      bulk_commit();
    }
  } else if (row_ok) {
    uint4* d = reinterpret_cast<uint4*>(static_cast<uint8_t*>(out) +
                                        (static_cast<size_t>(row) * N + col) * SIZE);
#pragma unroll
    for (int j = 0; j < 4 * PIECES; ++j)
      if (col + 16 / SIZE * j < N) d[j] = w[j];
  }
}
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                    pack_bf16(f[6], f[7]));
}
// 64 columns of fp32 as bf16.
__device__ __forceinline__ void put_bf16(Staging& st, const CUtensorMap* map, void* out, int N,
                                         const float* f, int row, int col, bool row_ok,
                                         bool all_ok, int lane) {
  uint4 w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack8(f + 8 * i);
  put<2>(st, map, out, N, w, row, col, row_ok, all_ok, lane);
}
__device__ __forceinline__ void put_f32(Staging& st, const CUtensorMap* map, void* out, int N,
                                        const float* f, int row, int col, bool row_ok,
                                        bool all_ok, int lane) {
#pragma unroll
  for (int i = 0; i < 64; i += 32) {
    uint4 w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      w[j] = make_uint4(__float_as_uint(f[i + 4 * j]), __float_as_uint(f[i + 4 * j + 1]),
                        __float_as_uint(f[i + 4 * j + 2]), __float_as_uint(f[i + 4 * j + 3]));
    put<4>(st, map, out, N, w, row, col + i, row_ok, all_ok, lane);
  }
}
// 16 codes of eight bf16 pairs.
__device__ __forceinline__ uint4 codes16(const uint32_t* w, const BlockScale& b) {
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float v[4] = {lo_of(w[2 * i]), hi_of(w[2 * i]), lo_of(w[2 * i + 1]), hi_of(w[2 * i + 1])};
    c[i] = codes4(v, b);
  }
  return make_uint4(c[0], c[1], c[2], c[3]);
}

// An asynchronous copy of four bytes (of zero, where `real` is not set).
__device__ __forceinline__ void copy_4(float* dst, const float* src, bool real) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(real ? 4 : 0)
               : "memory");
}
// Arrives on `bar` once this thread's copies so far are there.
__device__ __forceinline__ void arrive_copied(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// The pair's MMA on descriptors given by their low words; the high word (1024 bytes between
// groups of eight rows, version, 128-byte swizzle) is the same for all.
__device__ __forceinline__ void umma2_e4m3_at(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo,
                                              uint32_t idesc, uint32_t accumulate) {
  constexpr uint32_t HI = (1024u >> 4) | (1u << 14) | (2u << 29);
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 a, {%1, %5};\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(HI)
      : "memory");
}

// A whole warp's wait: true for all lanes or for none.
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity, int* status) {
  bool ok = mbar_try_wait(bar, parity);
  if (__all_sync(0xffffffffu, ok)) return true;
  ok = mbar_wait(bar, parity, status, kTimeoutCode);
  return __all_sync(0xffffffffu, ok);
}

// SMALL: a launch of few tiles, which may begin before the kernel before has ended and whose
// pairs may share a tile's contraction (a kernel of its own: what that keeps in registers costs
// large launches 4%).
template <int FORM, bool B_MN, bool SMALL>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    block_pair_kernel(const __grid_constant__ Params p, const __grid_constant__ Maps maps) {
  using S = Shape<FORM>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* staging = smem + S::STAGES * S::STAGE_BYTES;
  Ctrl<FORM>& c = *reinterpret_cast<Ctrl<FORM>*>(staging + SUM_WARPS * S::SETS * SET_BYTES);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int cid = static_cast<int>(cluster_id_x());
  const int ncl = static_cast<int>(cluster_count_x());

  // ------------------------------------------------------------ set-up
  if (warp == 0 && lane == 0) {
    for (int s = 0; s < S::STAGES; ++s) {
      mbar_init(smem_u32(&c.full[s]), 2);  // the producers of A and of B
      mbar_init(smem_u32(&c.empty[s]), 1);
    }
    for (int b = 0; b < S::BUFS; ++b) {
      mbar_init(smem_u32(&c.tfull[b]), 1);
      mbar_init(smem_u32(&c.tempty[b]), 2 * SUM_WARPS);
    }
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(smem_u32(&c.sfull[i]), 33);  // 32 lanes' copies, and the tile's place
      mbar_init(smem_u32(&c.sempty[i]), SUM_WARPS);
    }
    for (int w = 0; w < SUM_WARPS; ++w) mbar_init(smem_u32(&c.ab[w]), 1);
    mbar_init(smem_u32(&c.met), SUM_WARPS);
    mbar_init(smem_u32(&c.join), SUM_WARPS);
    mbar_init(smem_u32(&c.drain), 1);
    fence_mbar_init();
    tma_prefetch_desc(&maps.a[0]);
    tma_prefetch_desc(&maps.b[0]);
  }
  if (warp == ISSUE) {
    tmem_alloc2(smem_u32(&c.tmem_base), 512);
    tmem_relinquish2();
    tc_fence_before();
  }
  // launched early (launch_with), the set-up so far ran beside the end of the kernel before,
  // which may have written all that is read from here on
  if (SMALL) cudaGridDependencySynchronize();
  if (warp == FIRST_SUM_WARP)
    group_tables(p.offsets, p.E, p.rows, PM, c.off, c.cum, p.status, lane);
  cluster_sync_all();  // both CTAs' barriers exist before any arrival from the other
  tc_fence_after();
  constexpr uint32_t tmem_base = 0;  // all 512 columns are this block's
  // With two pairs or more to a tile, each takes a piece of the contraction: this one's tiles
  // are tile0, tile0 + ncl, .. (with pieces only the first exists), its blocks kb_lo ..
  // kb_lo + nkb - 1.
  const int tiles = ((p.N + S::OUT_COLS - 1) / S::OUT_COLS) * c.cum[p.E];
  int pieces = 1, tile0 = cid, kb_lo = 0, nkb = p.kblocks * p.products;
  if (SMALL && tiles > 0 && 2 * tiles <= ncl) {
    pieces = min(ncl / tiles, p.most_pieces);
    tile0 = cid < tiles * pieces ? cid / pieces : tiles;
    const int piece = cid % pieces;
    kb_lo = nkb * piece / pieces;
    nkb = nkb * (piece + 1) / pieces - kb_lo;
  }
  // Every wait below is bounded: a role whose wait runs out records it and ends, and those
  // that wait for it do the same.
  if (warp < FIRST_SUM_WARP) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::FEW));
    if (warp == LOAD_A || warp == LOAD_B) {
      // ------------------------------------------------------ TMA producers
      const bool is_a = warp == LOAD_A;
      const bool one = elect_one();
      int s = 0, asked = 0;
      uint32_t ph = 1;
      bool ok = true;
      Tile tl;
      for (int t = tile0; ok && place<FORM>(p, c.off, c.cum, t, tl); t += ncl) {
        const int e = __shfl_sync(0xffffffffu, tl.e, 0);
        const int at = __shfl_sync(0xffffffffu,
                                   is_a ? tl.row0 + rank * 128
                                        : (FORM == GATED ? tl.nb * 128
                                                         : tl.nb * S::COLS + rank * S::B_COLS),
                                   0);
        for (int kb = kb_lo; kb < kb_lo + nkb; ++kb) {
          ok = wait_all(smem_u32(&c.empty[s]), ph, p.status);
          if (!ok) break;
          const int which = kb >= p.kblocks ? 1 : 0;
          const int k = (which ? kb - p.kblocks : kb) * kBlock;
          if (one) {
            // the even CTA's barrier counts both CTAs' bytes
            const uint32_t own = smem_u32(&c.full[s]);
            const uint32_t dst = smem_u32(smem + s * S::STAGE_BYTES) + (is_a ? 0 : S::A_BYTES);
            if (rank == 0) {
              mbar_expect_tx(own, 2 * (is_a ? S::A_BYTES : S::STAGE_BYTES - S::A_BYTES));
              if (is_a)
                tma_load_2d(dst, &maps.a[which], k, at, own);
              else
                tma_load_3d(dst, FORM == GATED ? &maps.b[0] : &maps.b[which], B_MN ? at : k,
                            B_MN ? k : at, e, own);
            } else {
              const uint32_t bar = mapa_shared(own, 0);
              if (is_a)
                tma_load_2d_pair(dst, &maps.a[which], k, at, bar);
              else
                tma_load_3d_pair(dst, FORM == GATED ? &maps.b[1] : &maps.b[which], B_MN ? at : k,
                                 B_MN ? k : at, e, bar);
            }
          }
          __syncwarp();
          ++asked;
          if (++s == S::STAGES) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      if (!ok && rank == 0) {
        // the loads already asked for land before the CTA can end
        const int first = asked > S::STAGES ? asked - S::STAGES : 0;
        for (int r = first; r < asked; ++r)
          mbar_wait_cluster(smem_u32(&c.full[r % S::STAGES]), (r / S::STAGES) & 1, p.status,
                            kTimeoutCode);
      }
    } else if (warp == ISSUE) {
      if (rank == 0) {
        // ----------------------------------------------- MMA issuer (even CTA)
        constexpr uint32_t IDESC = idesc_e4m3(PM, S::COLS) | (B_MN ? 1u << 16 : 0u);
        // 32 deep: 32 bytes of a K-major row; 32 rows of 128 bytes of an MN-major tile
        constexpr uint32_t B_STEP = B_MN ? 32 * 128 : 32;
        const uint32_t a_lo = static_cast<uint32_t>(smem_desc(smem_u32(smem), 16, 1024));
        const bool one = elect_one();
        const int all = tile0 < tiles ? ((tiles - tile0 + ncl - 1) / ncl) * nkb : 0;
        int left = __shfl_sync(0xffffffffu, all, 0);
        int s = 0, buf = 0;
        uint32_t ph = 0, bph = 1;
        bool ok = true;
        for (; left > 0; --left) {
          ok = wait_all(smem_u32(&c.full[s]), ph, p.status) &&
               wait_all(smem_u32(&c.tempty[buf]), bph, p.status);
          if (!ok) break;
          tc_fence_after();
          const uint32_t a = a_lo + s * (S::STAGE_BYTES >> 4);
          const uint32_t b = a + (S::A_BYTES >> 4);
          if (one) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma2_e4m3_at(tmem_base + buf * S::COLS, a + (kk * 32 >> 4), b + (kk * B_STEP >> 4),
                            IDESC, kk != 0);
            umma2_commit_mc(smem_u32(&c.tfull[buf]), 0x3);
            umma2_commit_mc(smem_u32(&c.empty[s]), 0x3);
          }
          __syncwarp();
          if (++s == S::STAGES) {
            s = 0;
            ph ^= 1;
          }
          if (++buf == S::BUFS) {
            buf = 0;
            bph ^= 1;
          }
        }
        if (one) {
          umma2_commit(smem_u32(&c.drain));
          mbar_wait(smem_u32(&c.drain), 0, p.status, kTimeoutCode);
        }
        __syncwarp();
      }
    } else if (warp == SCALES) {
      // ------------------------------------------------------------- scales
      int i = 0;
      uint32_t ph = 1;
      bool ok = true;
      Tile tl = {};
      auto give = [&](int nb) {  // what a slot says of its tile, and that it is filled
        if (lane == 0) {
          c.slots[i].nb = nb;
          c.slots[i].row0 = tl.row0;
          c.slots[i].row_end = tl.row_end;
        }
        arrive_copied(smem_u32(&c.sfull[i]));
        if (lane == 0) mbar_arrive(smem_u32(&c.sfull[i]));
        __syncwarp();
        if (++i == SLOTS) {
          i = 0;
          ph ^= 1;
        }
      };
      for (int t = tile0; ok && place<FORM>(p, c.off, c.cum, t, tl); t += ncl) {
        // indexes fit 32 bits: a scale stands for 128 bytes of codes or more
        const int row = tl.row0 + rank * 128 + lane;
        uint32_t base = 0;
        if (lane < S::NH) {
          // past the last column block: its products are zeros
          const int n = FORM == GATED ? tl.nb : min(S::NH * tl.nb + lane, p.nblocks - 1);
          base = static_cast<uint32_t>(tl.e) * p.sb_group + static_cast<uint32_t>(n) * p.sb_n;
        }
        for (int kb0 = 0; kb0 < nkb; kb0 += GROUP) {
          ok = wait_all(smem_u32(&c.sempty[i]), ph, p.status);
          if (!ok) break;
#pragma unroll
          for (int g = 0; g < GROUP; ++g) {
            if (kb0 + g >= nkb) break;
            const int product = kb_lo + kb0 + g >= p.kblocks ? 1 : 0;
            const uint32_t k = kb_lo + kb0 + g - (product ? p.kblocks : 0);
            const float* sa = p.sa[product] + k * static_cast<uint32_t>(p.rows);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const bool real = row + 32 * j < tl.row_end;
              copy_4(&c.slots[i].a[lane + 32 * j][g], sa + (real ? row + 32 * j : 0), real);
            }
            if (lane < S::NH)
              copy_4(&c.slots[i].b[lane][g],
                     p.sb[FORM == GATED ? lane : product] + (base + k * p.sb_k), true);
          }
          give(tl.nb);
        }
      }
      if (ok && wait_all(smem_u32(&c.sempty[i]), ph, p.status)) give(-1);
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::MANY));
    // ------------------------------------------- sums and epilogue (8 warps)
    const int quarter = warp & 3;                    // TMEM lanes this warp may read
    const int side = (warp - FIRST_SUM_WARP) >> 2;   // which 64 columns of each half
    const int trow = quarter * 32 + lane;            // TMEM lane: row of this CTA's 128
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    Staging st;
    st.sets = reinterpret_cast<uint4*>(staging + (warp - FIRST_SUM_WARP) * S::SETS * SET_BYTES);
    int it = 0, i = 0, buf = 0;
    uint32_t iph = 0, bph = 0;
    int asked = 0, had = 0;  // GATED_BWD: loads of A and B into the sets, and those that landed
    bool ok = true;
    for (;; ++it) {
      ok = wait_all(smem_u32(&c.sfull[i]), iph, p.status);
      if (!ok) break;
      const int nb = c.slots[i].nb;
      if (nb < 0) break;
      const int row = c.slots[i].row0 + rank * 128 + trow;
      const bool row_ok = row < c.slots[i].row_end;
      const bool all_ok = __all_sync(0xffffffffu, row_ok);
      const int col0 = nb * S::OUT_COLS + side * 64;
      if constexpr (FORM == GATED_BWD) {
        // this warp's rows and columns of A and B come while the sums run
        if (col0 < p.N) {
          fence_proxy_async_smem();  // the reads of the sets come before the refill
          __syncwarp();
          ++asked;
          if (lane == 0) {
            bulk_wait_read_0();
            const uint32_t bar = smem_u32(&c.ab[warp - FIRST_SUM_WARP]);
            mbar_expect_tx(bar, 4 * SET_BYTES);
#pragma unroll
            for (int j = 0; j < 4; ++j)  // A's 64 columns in sets 0 and 1, B's in 2 and 3
              tma_load_2d(smem_u32(st.sets + j * (SET_BYTES / 16)), &maps.i[j >> 1],
                          col0 + 32 * (j & 1), row - lane, bar);
          }
        }
      }
      float sums[S::NH][64];
#pragma unroll
      for (int h = 0; h < S::NH; ++h)
#pragma unroll
        for (int j = 0; j < 64; ++j) sums[h][j] = 0.f;
      bool ready = false;   // the next accumulator, looked at while the last one was added
#pragma unroll 1
      for (int kb0 = 0; kb0 < nkb; kb0 += GROUP) {
        if (kb0 && !(ok = wait_all(smem_u32(&c.sfull[i]), iph, p.status))) break;
        float scale[S::NH][GROUP];
        {
          const float4 a = *reinterpret_cast<const float4*>(c.slots[i].a[trow]);
#pragma unroll
          for (int h = 0; h < S::NH; ++h) {
            const float4 b = *reinterpret_cast<const float4*>(c.slots[i].b[h]);
            scale[h][0] = a.x * b.x;
            scale[h][1] = a.y * b.y;
            scale[h][2] = a.z * b.z;
            scale[h][3] = a.w * b.w;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&c.sempty[i]));
        if (++i == SLOTS) {
          i = 0;
          iph ^= 1;
        }
#pragma unroll
        for (int g = 0; g < GROUP; ++g) {
          if (kb0 + g >= nkb) break;
          if (!ready && !(ok = wait_all(smem_u32(&c.tfull[buf]), bph, p.status))) break;
          tc_fence_after();
          const uint32_t at = tmem_base + buf * S::COLS + lanes + side * 64;
          const uint32_t done = smem_u32(&c.tempty[buf]);
          if (++buf == S::BUFS) {
            buf = 0;
            bph ^= 1;
          }
          // 32 columns come while those before are added; the accumulator is free as soon as
          // the last have come
          float v[32], w[32];
          tmem_ask32(at, v);
          ready = __all_sync(0xffffffffu, mbar_test_wait(smem_u32(&c.tfull[buf]), bph));
          tmem_wait(v);
          tmem_ask32(at + 32, w);
          add_32(v, scale[0][g], sums[0]);
          tmem_wait(w);
          if constexpr (S::NH == 2) {
            tmem_ask32(at + 128, v);
            add_32(w, scale[0][g], sums[0] + 32);
            tmem_wait(v);
            tmem_ask32(at + 160, w);
            add_32(v, scale[S::NH - 1][g], sums[S::NH - 1]);
            tmem_wait(w);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote(mapa_shared(done, 0));
          add_32(w, scale[S::NH - 1][g], sums[S::NH - 1] + 32);
        }
        if (!ok) break;
      }
      if (!ok) break;
      if (SMALL && pieces > 1) {
        // This piece's sums to its slot; the last of the tile's to arrive adds all in order and
        // goes on to the epilogue.
        constexpr int SLOT = 128 * S::COLS / 4;  // four columns of a row side by side
        float4* slot = reinterpret_cast<float4*>(p.part) + static_cast<size_t>(2 * cid + rank) * SLOT +
                       side * 16 * 128 + trow;
        if (row_ok) {
#pragma unroll
          for (int h = 0; h < S::NH; ++h)
#pragma unroll
            for (int j = 0; j < 16; ++j)
              __stcg(slot + (h * 32 + j) * 128, make_float4(sums[h][4 * j], sums[h][4 * j + 1],
                                                            sums[h][4 * j + 2], sums[h][4 * j + 3]));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&c.join));
        if (!(ok = wait_all(smem_u32(&c.join), 0, p.status))) break;
        if (warp == FIRST_SUM_WARP && lane == 0) {
          fence_gpu();  // what the eight warps wrote before they met
          const int index = 2 * tile0 + rank;
          const uint32_t shift = 8 * (index & 3);
          uint32_t* word = p.arrived + (index >> 2);
          const uint32_t old = (atomicAdd(word, 1u << shift) >> shift) & 0xFFu;
          c.last = old == static_cast<uint32_t>(pieces - 1);
          // every piece is there: the byte is zero again for the next call
          if (c.last) atomicSub(word, static_cast<uint32_t>(pieces) << shift);
          fence_gpu();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&c.join));
        if (!(ok = wait_all(smem_u32(&c.join), 1, p.status))) break;
        if (!c.last) continue;
        if (row_ok) {
          const float4* from = slot - static_cast<size_t>(2 * (cid % pieces)) * SLOT;
#pragma unroll
          for (int h = 0; h < S::NH; ++h)
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float4 v = __ldcg(from + (h * 32 + j) * 128);
              sums[h][4 * j] = v.x;
              sums[h][4 * j + 1] = v.y;
              sums[h][4 * j + 2] = v.z;
              sums[h][4 * j + 3] = v.w;
            }
#pragma unroll 1
          for (int b = 1; b < pieces; ++b) {
            from += 2 * SLOT;
#pragma unroll
            for (int h = 0; h < S::NH; ++h)
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const float4 v = __ldcg(from + (h * 32 + j) * 128);
                sums[h][4 * j] += v.x;
                sums[h][4 * j + 1] += v.y;
                sums[h][4 * j + 2] += v.z;
                sums[h][4 * j + 3] += v.w;
              }
          }
        }
      }
      if constexpr (FORM == PLAIN_BF16) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          put_bf16(st, &maps.o[0], p.out[0], p.N, sums[h], row, col0 + h * 128, row_ok, all_ok, lane);
      } else if constexpr (FORM == PLAIN_F32) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          put_f32(st, &maps.o[0], p.out[0], p.N, sums[h], row, col0 + h * 128, row_ok, all_ok, lane);
      } else if constexpr (FORM == GATED) {
        if (p.out[0]) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
            put_bf16(st, &maps.o[h], p.out[h], p.N, sums[h], row, col0, row_ok, all_ok, lane);
        }
        uint32_t w[32];  // H
        uint32_t top = 0;
        if (col0 < p.N) {
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            w[j] = pack_bf16(silu_f(sums[0][2 * j]) * sums[1][2 * j],
                             silu_f(sums[0][2 * j + 1]) * sums[1][2 * j + 1]);
            top = top_2(top, w[j]);
          }
        }
        top = top_of_2(top);
        uint16_t* tops = c.tops + (it & 1) * 256;
        tops[side * 128 + trow] = static_cast<uint16_t>(top >> 16);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&c.met));
        if (p.out[0]) {
          uint4 h8[8];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            h8[j] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
          put<2>(st, &maps.o[2], p.out[2], p.N, h8, row, col0, row_ok, all_ok, lane);
        }
        if (!(ok = wait_all(smem_u32(&c.met), it & 1, p.status))) break;
        top = max(top, static_cast<uint32_t>(tops[(side ^ 1) * 128 + trow]) << 16);
        if (col0 < p.N) {
          const BlockScale bs = block_scale(top);
          if (row_ok && side == 0) p.scales[0][static_cast<size_t>(nb) * p.rows + row] = bs.s;
          const uint4 q4[4] = {codes16(w, bs), codes16(w + 8, bs), codes16(w + 16, bs), codes16(w + 24, bs)};
          put<1, 1>(st, &maps.c[0], p.codes[0], p.N, q4, row, col0, row_ok, all_ok, lane);
        }
      } else {
        uint32_t top_a = 0, top_b = 0;
        uint4* sa = st.sets;
        uint4* sb = st.sets + 2 * (SET_BYTES / 16);
        if (col0 < p.N) {
          if (!(ok = wait_all(smem_u32(&c.ab[warp - FIRST_SUM_WARP]), had & 1, p.status))) break;
          ++had;
#pragma unroll 1
          for (int i0 = 0; i0 < 4; ++i0) {
#pragma unroll
            for (int i1 = 0; i1 < 2; ++i1) {
              const int j = 2 * i0 + i1;
              const int at = (j >> 2) * (SET_BYTES / 16) + slot_of(lane, j & 3);
              const uint4 ra = sa[at], rb = sb[at];
              const uint32_t wa[4] = {ra.x, ra.y, ra.z, ra.w}, wb[4] = {rb.x, rb.y, rb.z, rb.w};
              uint32_t da[4], db[4];
#pragma unroll
              for (int m = 0; m < 4; ++m) {
                const float* dh = sums[0] + 8 * i1 + 2 * m;
                const float av[2] = {lo_of(wa[m]), hi_of(wa[m])}, bv[2] = {lo_of(wb[m]), hi_of(wb[m])};
                float xa[2], xb[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  const float sg = sigmoid_f(av[k]);
                  const float dhs = dh[k] * sg;
                  xa[k] = dhs * bv[k] * (1.0f + av[k] * (1.0f - sg));
                  xb[k] = dhs * av[k];
                }
                da[m] = pack_bf16(xa[0], xa[1]);
                db[m] = pack_bf16(xb[0], xb[1]);
                top_a = top_2(top_a, da[m]);
                top_b = top_2(top_b, db[m]);
              }
              sa[at] = make_uint4(da[0], da[1], da[2], da[3]);
              sb[at] = make_uint4(db[0], db[1], db[2], db[3]);
            }
            // the next 16 sums move down (unrolled over all 64 columns this loop was slower)
#pragma unroll
            for (int m = 0; m < 48; ++m) sums[0][m] = sums[0][m + 16];
          }
          if (all_ok) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                tma_store_2d(&maps.o[j >> 1], smem_u32(st.sets + j * (SET_BYTES / 16)),
                             col0 + 32 * (j & 1), row - lane);
              bulk_commit();
            }
          }
        }
        top_a = top_of_2(top_a);
        top_b = top_of_2(top_b);
        uint16_t* tops = c.tops + (it & 1) * 512;
        tops[side * 128 + trow] = static_cast<uint16_t>(top_a >> 16);
        tops[256 + side * 128 + trow] = static_cast<uint16_t>(top_b >> 16);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&c.met));
        if (!(ok = wait_all(smem_u32(&c.met), it & 1, p.status))) break;
        top_a = max(top_a, static_cast<uint32_t>(tops[(side ^ 1) * 128 + trow]) << 16);
        top_b = max(top_b, static_cast<uint32_t>(tops[256 + (side ^ 1) * 128 + trow]) << 16);
        if (col0 < p.N && row_ok) {
          const BlockScale ba = block_scale(top_a), bb = block_scale(top_b);
          if (side == 0) {
            p.scales[0][static_cast<size_t>(nb) * p.rows + row] = ba.s;
            p.scales[1][static_cast<size_t>(nb) * p.rows + row] = bb.s;
          }
          const size_t o = static_cast<size_t>(row) * p.N + col0;
#pragma unroll 1
          for (int v = 0; v < 2; ++v) {
            const uint4* set = v ? sb : sa;
            const BlockScale b = v ? bb : ba;
            uint4* d = reinterpret_cast<uint4*>(p.codes[v] + o);
            uint4* keep = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out[v]) + o);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint4* half = set + (j >> 1) * (SET_BYTES / 16);
              const uint4 x = half[slot_of(lane, (2 * j) & 3)], y = half[slot_of(lane, (2 * j + 1) & 3)];
              const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
              d[j] = codes16(w, b);
              if (!all_ok) {
                keep[2 * j] = x;
                keep[2 * j + 1] = y;
              }
            }
          }
        }
      }
    }
    if (had < asked)  // after an abort: loads of A and B still on their way
      mbar_wait(smem_u32(&c.ab[warp - FIRST_SUM_WARP]), had & 1, p.status, kTimeoutCode);
    if (lane == 0) bulk_wait_all();  // staged rows written out before the CTA ends
  }

  // ------------------------------------------------------------ teardown
  __syncthreads();
  cluster_sync_all();  // the pair's MMAs and TMEM reads are finished
  if (warp == ISSUE) {
    tc_fence_after();
    tmem_dealloc2(tmem_base, 512);
  }
}

template <int FORM>
long long column_tiles(const Params& p) {
  return (p.N + Shape<FORM>::OUT_COLS - 1) / Shape<FORM>::OUT_COLS;
}
// The order of a group's tiles; a_row, b_col: bytes of a row of A and of a column of the weight
// (of both, where there are two).
template <int FORM>
void set_order(Params& p, long long a_row, long long b_col) {
  const long long cols = Shape<FORM>::OUT_COLS, rows_each = (p.rows + p.E - 1ll) / p.E;
  p.order = tile_order(rows_each * a_row, p.N * b_col, PM * a_row, cols * b_col,
                       (p.rows + PM - 1) / PM, column_tiles<FORM>(p));
}
template <int FORM>
long long most_tiles(const Params& p) {
  return column_tiles<FORM>(p) * ((p.rows + PM - 1) / PM + p.E);
}
template <int FORM, bool B_MN, bool SMALL>
cudaError_t launch_with(const Params& p, const Maps& m, int num_sms, bool early, cudaStream_t s) {
  auto kern = block_pair_kernel<FORM, B_MN, SMALL>;
  constexpr int smem = smem_bytes<FORM>();
  const cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(NUM_THREADS, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int fit = pairs_that_fit(reinterpret_cast<const void*>(kern), cfg, num_sms);
  if (SMALL && fit > kMostPairs) fit = kMostPairs;
  const long long items = most_tiles<FORM>(p) * (SMALL ? p.most_pieces : 1);
  cfg.gridDim = dim3(2 * static_cast<unsigned>(items < fit ? items : fit), 1, 1);
  if (early) cfg.numAttrs = 2;
  const cudaError_t le = cudaLaunchKernelEx(&cfg, kern, p, m);
  return le == cudaSuccess ? launched() : le;
}
// Which of the two: the small one where pairs may share tiles, and for launches of some 15 us
// (32 blocks in turn) or less in a stream, which then begin before the kernel before has ended.
// Calls in a stream, us, without and with: 1037 x 1104 x 720 12.3 10.9, 100 x 4096 x 4096
// 20.4 17.7, its feed-forward block 44.9 41.6; with 64 blocks in turn 70.7 73.8.  In a graph an
// early launch gains nothing.
template <int FORM, bool B_MN>
cudaError_t launch_pairs(Params& p, const Maps& m, int num_sms, cudaStream_t s) {
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  const cudaError_t e = cudaStreamIsCapturing(s, &capture);
  if (e != cudaSuccess) return e;
  const bool stream = capture == cudaStreamCaptureStatusNone;
  const long long pairs = num_sms > 1 ? num_sms / 2 : 1;
  const long long turns = (most_tiles<FORM>(p) + pairs - 1) / pairs;
  // the fewest tiles that these rows can make; the kernel counts those there are
  const long long least = column_tiles<FORM>(p) * ((p.rows + PM - 1) / PM);
  const bool shared = p.most_pieces > 1 && 2 * least <= pairs;
  // a launch that is small for its early start alone shares no tile, however few there are:
  // in a graph it would not, and the same inputs give the same bits
  if (!shared) p.most_pieces = 1;
  return shared || (stream && turns * p.kblocks * p.products <= 32)
             ? launch_with<FORM, B_MN, true>(p, m, num_sms, stream, s)
             : launch_with<FORM, B_MN, false>(p, m, num_sms, false, s);
}

// Pieces of a tile's contraction of `blocks` blocks, where pairs would idle otherwise.  Blocks
// take 0.45 us each in their turn; a join takes some 4.5 us, and 0.5 to 1.5 for each piece (few
// rows to 128).  Times in us, one group, 20 and 128 rows, in a graph, of 1, 2, 3, 4 pieces:
//   2048 x 4096    11.7 12.5 12.9 13.4    12.6 15.8 16.6 17.7
//   4096 x 4096    18.5 16.0 14.7 15.0    19.2 19.5 18.7 19.8
//   8192 x 2048    30.5 22.0 18.5 17.2    31.4 25.3 22.8 21.7
//   14336 x 4096   50.2 31.9 25.8 23.4    51.3 35.5 30.2 28.7
int pieces_of(int blocks) {
  if (blocks < 32) return 1;
  int n = 3;
  while (10 * (n + 1) * (n + 1) <= 3 * blocks) ++n;
  return n;
}

Params params_of(const BlockRows& r, int K, int N, bool trans, int products = 1) {
  Params p;
  memset(&p, 0, sizeof(p));
  p.E = r.E;
  p.offsets = r.offsets;
  p.rows = r.rows;
  p.status = r.status;
  p.N = N;
  p.kblocks = blocks_of(K);
  p.products = products;
  p.part = r.part;
  p.arrived = reinterpret_cast<uint32_t*>(r.status) + 16;  // bytes 64 .. 223 of the header
  p.most_pieces = pieces_of(p.kblocks * products);
  p.nblocks = blocks_of(N);
  p.sb_group = p.kblocks * p.nblocks;
  p.sb_k = trans ? 1 : p.nblocks;
  p.sb_n = trans ? p.kblocks : 1;
  return p;
}

bool map_rows(CUtensorMap* m, const void* q, int K, int rows) {
  return make_map_kmajor(m, q, K, rows, 128, true);
}
// A weight as it lies: boxes of 128 contiguous codes x box_rows.
bool map_weight(CUtensorMap* m, const void* q, int E, int K, int N, bool trans, int cols) {
  return trans ? make_map_codes(m, q, K, N, E, cols) : make_map_codes(m, q, N, K, E, 128);
}

}  // namespace

cudaError_t block_product(const BlockRows& r, const Coded& a, const Coded& b, int K, int N,
                          bool trans, bool out_f32, void* C, cudaStream_t s, bool ahead) {
  if (r.rows == 0) return cudaSuccess;
  if (ahead ? few_rows(r.rows, r.E, K, N) : few_rows_alone(r.rows, r.E, K, N))
    return few_product(r, a, b, K, N, trans, out_f32, C, s, ahead);
  Params p = params_of(r, K, N, trans);
  p.sa[0] = a.s;
  p.sb[0] = b.s;
  p.out[0] = C;
  Maps m;
  memset(&m, 0, sizeof(m));
  if (!map_rows(&m.a[0], a.q, K, r.rows) || !map_weight(&m.b[0], b.q, r.E, K, N, trans, 128) ||
      !make_map_box(&m.o[0], C, out_f32 ? 4 : 2, N, r.rows))
    return cudaErrorInvalidValue;
  set_order<PLAIN_BF16>(p, K, K);
  if (out_f32)
    return trans ? launch_pairs<PLAIN_F32, false>(p, m, r.num_sms, s)
                 : launch_pairs<PLAIN_F32, true>(p, m, r.num_sms, s);
  return trans ? launch_pairs<PLAIN_BF16, false>(p, m, r.num_sms, s)
               : launch_pairs<PLAIN_BF16, true>(p, m, r.num_sms, s);
}

cudaError_t block_fc1_fwd(const BlockRows& r, const Coded& x, const Coded& w1, const Coded& w3,
                          int h, int f, uint16_t* A, uint16_t* B, uint16_t* H, uint8_t* Hq,
                          float* sh, cudaStream_t s) {
  if (r.rows == 0) return cudaSuccess;
  if (few_rows(r.rows, r.E, h, f)) return few_fc1_fwd(r, x, w1, w3, h, f, A, B, H, Hq, sh, s);
  Params p = params_of(r, h, f, false);
  p.sa[0] = x.s;
  p.sb[0] = w1.s;
  p.sb[1] = w3.s;
  p.out[0] = A;
  p.out[1] = B;
  p.out[2] = H;
  p.codes[0] = Hq;
  p.scales[0] = sh;
  Maps m;
  memset(&m, 0, sizeof(m));
  if (!map_rows(&m.a[0], x.q, h, r.rows) || !map_weight(&m.b[0], w1.q, r.E, h, f, false, 128) ||
      !map_weight(&m.b[1], w3.q, r.E, h, f, false, 128))
    return cudaErrorInvalidValue;
  if (!make_map_box(&m.c[0], Hq, 1, f, r.rows)) return cudaErrorInvalidValue;
  if (A && (!make_map_box(&m.o[0], A, 2, f, r.rows) ||
            !make_map_box(&m.o[1], B, 2, f, r.rows) ||
            !make_map_box(&m.o[2], H, 2, f, r.rows)))
    return cudaErrorInvalidValue;
  set_order<GATED>(p, h, 2ll * h);
  return launch_pairs<GATED, true>(p, m, r.num_sms, s);
}

cudaError_t block_fc2_dgrad(const BlockRows& r, const Coded& dy, const Coded& w2, int h, int f,
                            const uint16_t* A, const uint16_t* B, uint16_t* dA, uint16_t* dB,
                            uint8_t* dAq, float* sda, uint8_t* dBq, float* sdb, cudaStream_t s) {
  if (r.rows == 0) return cudaSuccess;
  Params p = params_of(r, h, f, true);
  p.sa[0] = dy.s;
  p.sb[0] = w2.s;
  p.out[0] = dA;
  p.out[1] = dB;
  p.codes[0] = dAq;
  p.scales[0] = sda;
  p.codes[1] = dBq;
  p.scales[1] = sdb;
  Maps m;
  memset(&m, 0, sizeof(m));
  if (!map_rows(&m.a[0], dy.q, h, r.rows) || !map_weight(&m.b[0], w2.q, r.E, h, f, true, 64) ||
      !make_map_box(&m.o[0], dA, 2, f, r.rows) || !make_map_box(&m.o[1], dB, 2, f, r.rows) ||
      !make_map_box(&m.i[0], A, 2, f, r.rows) || !make_map_box(&m.i[1], B, 2, f, r.rows))
    return cudaErrorInvalidValue;
  set_order<GATED_BWD>(p, h, h);
  return launch_pairs<GATED_BWD, false>(p, m, r.num_sms, s);
}

cudaError_t block_fc1_dgrad(const BlockRows& r, const Coded& da, const Coded& db, const Coded& w1,
                            const Coded& w3, int h, int f, bool out_f32, void* dX,
                            cudaStream_t s) {
  if (r.rows == 0) return cudaSuccess;
  Params p = params_of(r, f, h, true, 2);
  p.sa[0] = da.s;
  p.sa[1] = db.s;
  p.sb[0] = w1.s;
  p.sb[1] = w3.s;
  p.out[0] = dX;
  Maps m;
  memset(&m, 0, sizeof(m));
  if (!map_rows(&m.a[0], da.q, f, r.rows) || !map_rows(&m.a[1], db.q, f, r.rows) ||
      !map_weight(&m.b[0], w1.q, r.E, f, h, true, 128) ||
      !map_weight(&m.b[1], w3.q, r.E, f, h, true, 128) ||
      !make_map_box(&m.o[0], dX, out_f32 ? 4 : 2, h, r.rows))
    return cudaErrorInvalidValue;
  set_order<PLAIN_BF16>(p, 2ll * f, 2ll * f);
  return out_f32 ? launch_pairs<PLAIN_F32, false>(p, m, r.num_sms, s)
                 : launch_pairs<PLAIN_BF16, false>(p, m, r.num_sms, s);
}

}  // namespace moe
