// gemm_block_few.cu -- the block-scaled products of block.cuh for a few rows to a
// group, as a serving step has them: bound by reading each weight once.
//
//   * The product is taken transposed: 128 columns of the weight are the tensor
//     cores' rows (from the weight's own layout, MN-major or K-major), 16 or 32 rows
//     of activations their columns, so that a block of 128 x 128 codes costs one
//     block's MMAs whatever the number of rows.  A step has two such blocks: side by
//     side in one weight (256 bytes in a row of it: with 128 HBM moved 10% less), or the
//     same columns of W1 and W3.
//   * All k-steps of all tiles are cut into contiguous pieces, one for each block of
//     the grid: the same number for every tile, or, where that leaves too many SMs idle,
//     equal ones whatever the tiles' number.  A tile that several blocks share is joined
//     by the last to arrive, in the pieces' order: the same inputs give the same bits.
//   * A ring of some 190 KiB of stages is under way on each SM.
// Measured, in a graph, weights not in L2: one row by 4096 x 14336, 16 us (8.8 at the copy
// bandwidth); 192 rows in 64 groups of 2048 x 1408, 40 us (25.6).  What is left is the start
// (some 3 us to the first weights), the join of shared tiles (2 to 3 us) and SMs that HBM
// serves unevenly.
// Roles of a block's 256 threads: warp 0 loads weights, warp 3 activations, warp 2
// scales, warp 1 issues the MMAs, warps 4-7 take each step's sums out of tensor
// memory, times the scales, into sums in registers (one output column to a thread).
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

enum Form { PLAIN_BF16 = 0, PLAIN_F32 = 1, GATED = 2 };

constexpr int kTimeoutCode = 5;  // MOE_ERR_DEVICE_TIMEOUT
constexpr int MAX_BLOCKS = kPartBlocks;  // of the grid
constexpr int NUM_THREADS = 256;
constexpr int W_BYTES = 128 * 128;
constexpr int SLOTS = 8;         // steps whose scales wait
constexpr int LOAD_W = 0, ISSUE = 1, SCALES = 2, LOAD_X = 3, FIRST_SUM_WARP = 4;

struct Params {
  int E;
  const int32_t* offsets;   // NULL: one group of all rows
  int rows, N, nkb;
  const float* sa;          // [nkb, rows]
  const float* sb[2];
  int sb_group, sb_k, sb_n; // scales of a group; strides of the contraction's and the column's block
  void* out[3];             // GATED: A, B, H (or NULL)
  uint8_t* codes;           // GATED: H's
  float* scales;
  float* part;              // [grid, 2] slots of a shared tile's sums
  uint32_t* arrived;        // a byte for each block of the grid: pieces of its last tile
  int ahead;                // the kernel before (which has waited for all before it) writes
                            // neither the weights nor the offsets
  int* status;
};
struct Maps {
  CUtensorMap x, w[2];
};

template <int FORM, int NT>
struct Shape {
  static constexpr int NB = 2;                       // blocks of weights in a step
  static constexpr int COLS = FORM == GATED ? 128 : 256;  // output columns of a tile
  static constexpr int X_BYTES = NT * 128;
  static constexpr int STAGE_BYTES = NB * W_BYTES + X_BYTES;
  static constexpr int UNIT = NB * NT;               // accumulator columns of a step
  static constexpr int PITCH = (FORM == PLAIN_F32 ? 512 : 256) + 16;  // staging: bytes of a row
  static constexpr int FIT = (232448 - 1024 - NT * PITCH - 3 * 1024) / STAGE_BYTES;
  static constexpr int STAGES = FIT > 12 ? 12 : FIT;
  static constexpr int BUFS = 4;                     // steps whose sums wait in tensor memory
  static constexpr int TMEM = BUFS * UNIT;           // columns (a power of two, 128 or 256)
  static_assert(X_BYTES % 1024 == 0 && TMEM <= 256 && TMEM >= 32 && STAGES >= 2, "does not fit");
};
template <int NT>
struct alignas(16) Slot {
  float a[NT];
  float b[2];
};
template <int FORM, int NT>
struct alignas(16) Ctrl {
  using S = Shape<FORM, NT>;
  uint64_t full[S::STAGES], empty[S::STAGES];
  uint64_t tfull[S::BUFS], tempty[S::BUFS];
  uint64_t sfull[SLOTS], sempty[SLOTS];
  uint64_t met, drain;
  uint32_t tmem_base;
  uint32_t last;            // whether this block joins the tile
  int off[kMaxGroups + 1];
  int cum[kMaxGroups + 1];       // row tiles before each group
  Slot<NT> slots[SLOTS];
};
static_assert(2 * 2 * 32 * 128 <= 128 * 256, "a block's two slots fit its part");
template <int FORM, int NT>
constexpr int smem_bytes() {
  using S = Shape<FORM, NT>;
  return 1024 + S::STAGES * S::STAGE_BYTES + NT * S::PITCH + static_cast<int>(sizeof(Ctrl<FORM, NT>));
}

struct Tile {
  int e, n, row0, row_end;  // group, column tile, rows
};
// Steps of weights that a block asks L2 for before the kernel before has ended.
constexpr int kEarlySteps = 4;

// Tile t: groups in order; in one, column tiles in order; row tiles of a column tile
// side by side, so that they find the weight in L2.
template <int FORM, int NT>
__device__ __forceinline__ Tile place(const Params& p, const int* off, const int* cum, int t) {
  const int tiles_n = (p.N + Shape<FORM, NT>::COLS - 1) / Shape<FORM, NT>::COLS;
  int e = 0, hi = p.E - 1;
  while (e < hi) {
    const int mid = (e + hi + 1) >> 1;
    if (tiles_n * cum[mid] <= t)
      e = mid;
    else
      hi = mid - 1;
  }
  const int local = t - tiles_n * cum[e];
  const int mt = cum[e + 1] - cum[e];
  Tile tl;
  tl.e = e;
  tl.n = local / mt;
  tl.row0 = off[e] + (local - tl.n * mt) * NT;
  tl.row_end = off[e + 1];
  return tl;
}

__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, int* status) {
  bool ok = mbar_try_wait(smem_u32(bar), parity);
  if (__all_sync(0xffffffffu, ok)) return true;
  ok = mbar_wait(smem_u32(bar), parity, status, kTimeoutCode);
  return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ void copy_4(float* dst, const float* src, bool real) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(real ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ float silu_f(float a) { return __fdividef(a, 1.0f + __expf(-a)); }

// NT columns of this thread's TMEM lane.
template <int NT>
__device__ __forceinline__ void tmem_columns(uint32_t taddr, float (&v)[NT]) {
  if constexpr (NT == 16) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
  } else {
    tmem_ld32(taddr, v);
  }
}

template <int FORM, int NT, bool TRANS>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    block_few_kernel(const __grid_constant__ Params p, const __grid_constant__ Maps maps) {
  using S = Shape<FORM, NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* staging = smem + S::STAGES * S::STAGE_BYTES;
  Ctrl<FORM, NT>& c = *reinterpret_cast<Ctrl<FORM, NT>*>(staging + NT * S::PITCH);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < S::STAGES; ++s) {
      mbar_init(smem_u32(&c.full[s]), 2);  // the producers of weights and of activations
      mbar_init(smem_u32(&c.empty[s]), 1);
    }
    for (int b = 0; b < S::BUFS; ++b) {
      mbar_init(smem_u32(&c.tfull[b]), 1);
      mbar_init(smem_u32(&c.tempty[b]), 4);
    }
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(smem_u32(&c.sfull[i]), 32);
      mbar_init(smem_u32(&c.sempty[i]), 4);
    }
    mbar_init(smem_u32(&c.met), 4);
    mbar_init(smem_u32(&c.drain), 1);
    fence_mbar_init();
    tma_prefetch_desc(&maps.x);
    tma_prefetch_desc(&maps.w[0]);
  }
  if (warp == ISSUE) {
    tmem_alloc(smem_u32(&c.tmem_base), S::TMEM);
    tmem_relinquish();
    tc_fence_before();
  }
  if (!p.ahead) {
    // One group: the steps are known before its rows are, and the weights can come to L2 while
    // the kernel before ends (should it write them, L2 has what it wrote).
    if (warp == LOAD_W && p.E == 1) {
      const int row_tiles = (p.rows + NT - 1) / NT;
      const Share guess = share_of((p.N + S::COLS - 1) / S::COLS * row_tiles, p.nkb, gridDim.x, blockIdx.x);
      const int from = guess.t * p.nkb + guess.kb, to = from + min(guess.count, kEarlySteps);
      if (elect_one())
        for (int i = from; i < to; ++i) {
          const int n = i / p.nkb / row_tiles * S::COLS;
          const int k = i % p.nkb * kBlock;
#pragma unroll
          for (int o = 0; o < S::NB; ++o) {
            const int at = n + (FORM == GATED ? 0 : o * 128);
            tma_prefetch_l2_3d(&maps.w[FORM == GATED ? o : 0], TRANS ? k : at, TRANS ? at : k, 0);
          }
        }
      __syncwarp();
    }
    // the kernel before may have written all that is read from here on
    cudaGridDependencySynchronize();
  }
  if (warp == FIRST_SUM_WARP)
    group_tables(p.offsets, p.E, p.rows, NT, c.off, c.cum, p.status, lane);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = c.tmem_base;
  const int nkb = p.nkb;
  const Share share = share_of((p.N + S::COLS - 1) / S::COLS * c.cum[p.E], nkb, gridDim.x, blockIdx.x);
  const int me = static_cast<int>(blockIdx.x);
  const int count = share.count;
  int t = share.t, kb = share.kb;

  // Ahead of the end of the kernel before, the weights stream in; what it writes (the
  // activations, their scales, the slots of shared tiles) waits for it.  The kernel after
  // this one may start once all before this one are done.
  if (p.ahead && warp != LOAD_W && warp != ISSUE) cudaGridDependencySynchronize();
  if (warp == FIRST_SUM_WARP) cudaTriggerProgrammaticLaunchCompletion();

  if (warp == LOAD_W || warp == LOAD_X) {
    // -------------------------------------------------------- TMA producers
    const bool one = elect_one();
    int s = 0, asked = 0;
    uint32_t ph = 1;
    bool ok = true;
    Tile tl = {};
    for (int i = 0; i < count; ++i) {
      if (i == 0 || kb == 0) tl = place<FORM, NT>(p, c.off, c.cum, t);
      ok = wait_all(&c.empty[s], ph, p.status);
      if (!ok) break;
      if (one) {
        const uint32_t bar = smem_u32(&c.full[s]);
        const uint32_t dst = smem_u32(smem + s * S::STAGE_BYTES);
        const int k = kb * kBlock;
        if (warp == LOAD_W) {
          mbar_expect_tx(bar, S::NB * W_BYTES);
#pragma unroll
          for (int o = 0; o < S::NB; ++o) {
            const int n = tl.n * S::COLS + (FORM == GATED ? 0 : o * 128);
            tma_load_3d(dst + o * W_BYTES, &maps.w[FORM == GATED ? o : 0], TRANS ? k : n,
                        TRANS ? n : k, tl.e, bar);
          }
        } else {
          mbar_expect_tx(bar, S::X_BYTES);
          tma_load_2d(dst + S::NB * W_BYTES, &maps.x, k, tl.row0, bar);
        }
      }
      __syncwarp();
      ++asked;
      if (++s == S::STAGES) {
        s = 0;
        ph ^= 1;
      }
      if (++kb == nkb) {
        kb = 0;
        ++t;
      }
    }
    if (!ok) {
      // the loads already asked for land before the block can end
      const int first = asked > S::STAGES ? asked - S::STAGES : 0;
      for (int r = first; r < asked; ++r)
        mbar_wait(smem_u32(&c.full[r % S::STAGES]), (r / S::STAGES) & 1, p.status, kTimeoutCode);
    }
  } else if (warp == ISSUE) {
    // ---------------------------------------------------------- MMA issuer
    constexpr uint32_t IDESC = idesc_e4m3(128, NT) | (TRANS ? 0u : 1u << 15);
    // 32 deep: 32 bytes of a K-major row; 32 rows of 128 bytes of an MN-major tile
    constexpr uint32_t W_STEP = TRANS ? 32 : 32 * 128;
    const bool one = elect_one();
    const uint64_t base = smem_desc(smem_u32(smem), 16, 1024);
    int s = 0, buf = 0;
    uint32_t ph = 0, bph = 1;
    for (int i = 0; i < count; ++i) {
      if (!wait_all(&c.full[s], ph, p.status) || !wait_all(&c.tempty[buf], bph, p.status)) break;
      tc_fence_after();
      const uint64_t w = base + s * (S::STAGE_BYTES >> 4);
      if (one) {
#pragma unroll
        for (int o = 0; o < S::NB; ++o)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_e4m3(tmem_base + buf * S::UNIT + o * NT, w + ((o * W_BYTES + kk * W_STEP) >> 4),
                      w + ((S::NB * W_BYTES + kk * 32) >> 4), IDESC, kk != 0);
        umma_commit(smem_u32(&c.empty[s]));
        umma_commit(smem_u32(&c.tfull[buf]));
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
      umma_commit(smem_u32(&c.drain));
      mbar_wait(smem_u32(&c.drain), 0, p.status, kTimeoutCode);
    }
    __syncwarp();
  } else if (warp == SCALES) {
    // -------------------------------------------------------------- scales
    int i = 0;
    uint32_t ph = 1;
    Tile tl = {};
    for (int n = 0; n < count; ++n) {
      if (n == 0 || kb == 0) tl = place<FORM, NT>(p, c.off, c.cum, t);
      if (!wait_all(&c.sempty[i], ph, p.status)) break;
      // indexes fit 32 bits: a scale stands for 128 bytes of codes or more
#pragma unroll
      for (int j = lane; j < NT; j += 32) {
        const int row = tl.row0 + j;
        const bool real = row < tl.row_end;
        copy_4(&c.slots[i].a[j], p.sa + (static_cast<uint32_t>(kb) * p.rows + (real ? row : 0)), real);
      }
      if (lane < S::NB) {
        // past the last column block: its products are zeros
        const int n = FORM == GATED ? tl.n : min(2 * tl.n + lane, (p.N + 127) / 128 - 1);
        copy_4(&c.slots[i].b[lane],
               p.sb[FORM == GATED ? lane : 0] +
                   (static_cast<uint32_t>(tl.e) * p.sb_group + static_cast<uint32_t>(kb) * p.sb_k +
                    static_cast<uint32_t>(n) * p.sb_n),
               true);
      }
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&c.sfull[i]))
                   : "memory");
      if (++i == SLOTS) {
        i = 0;
        ph ^= 1;
      }
      if (++kb == nkb) {
        kb = 0;
        ++t;
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    // --------------------------------------------- sums and epilogue (4 warps)
    const int tid = threadIdx.x - 32 * FIRST_SUM_WARP;  // TMEM lane: output column of the tile
    const uint32_t lanes = static_cast<uint32_t>(tid & ~31) << 16;
    uint32_t meetings = 0;
    // The four warps: what each wrote before is seen by all after.
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&c.met));
      return wait_all(&c.met, meetings++ & 1, p.status);
    };
    int i = 0, buf = 0;
    uint32_t iph = 0, bph = 0;
    bool ok = true;
    int left = count;
    while (ok && left > 0) {
      const Tile tl = place<FORM, NT>(p, c.off, c.cum, t);
      const int n = min(nkb - kb, left);  // this block's steps of the tile
      // Where the tile is shared: the pieces' blocks, and the first one's slot (the others
      // begin with the tile: slot 0).  Divisions, done while the first weights are on the way.
      int first = 0, last = 0, first_slot = 0;
      if (share.per) {
        first = t * share.per;
        last = first + share.per - 1;
      } else if (n < nkb) {
        const int s0 = t * nkb;
        first = share.owner(s0);
        last = share.owner(s0 + nkb - 1);
        first_slot = share.lo(first) == s0 ? 0 : 1;
      }
      float sums[S::NB][NT];
#pragma unroll
      for (int o = 0; o < S::NB; ++o)
#pragma unroll
        for (int j = 0; j < NT; ++j) sums[o][j] = 0.f;
#pragma unroll 1
      for (int step = 0; step < n; ++step) {
        if (!(ok = wait_all(&c.sfull[i], iph, p.status) && wait_all(&c.tfull[buf], bph, p.status))) break;
        tc_fence_after();
#pragma unroll
        for (int o = 0; o < S::NB; ++o) {
          float v[NT];
          tmem_columns<NT>(tmem_base + buf * S::UNIT + o * NT + lanes, v);
          const float b = c.slots[i].b[o];
#pragma unroll
          for (int j = 0; j < NT; j += 4) {
            const float4 a = *reinterpret_cast<const float4*>(&c.slots[i].a[j]);
            sums[o][j] = fmaf(v[j], a.x * b, sums[o][j]);
            sums[o][j + 1] = fmaf(v[j + 1], a.y * b, sums[o][j + 1]);
            sums[o][j + 2] = fmaf(v[j + 2], a.z * b, sums[o][j + 2]);
            sums[o][j + 3] = fmaf(v[j + 3], a.w * b, sums[o][j + 3]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&c.tempty[buf]));
          mbar_arrive(smem_u32(&c.sempty[i]));
        }
        if (++i == SLOTS) {
          i = 0;
          iph ^= 1;
        }
        if (++buf == S::BUFS) {
          buf = 0;
          bph ^= 1;
        }
      }
      if (!ok) break;
      bool mine = true;  // whether the tile is finished here
      if (n < nkb) {
        // shared: this block's sums to its slot; the last to arrive adds all in order
        constexpr int SLOT = S::NB * NT * 128;
        float* slot = p.part + (2ll * me + (me == first ? first_slot : 0)) * SLOT + tid;
#pragma unroll
        for (int o = 0; o < S::NB; ++o)
#pragma unroll
          for (int j = 0; j < NT; ++j)
            if (tl.row0 + j < tl.row_end) slot[(o * NT + j) * 128] = sums[o][j];
        if (!(ok = meet())) break;
        if (tid == 0) {
          fence_gpu();  // what the four warps wrote before they met
          const uint32_t shift = 8 * (first & 3);
          const uint32_t old = (atomicAdd(p.arrived + (first >> 2), 1u << shift) >> shift) & 0xFFu;
          c.last = old == static_cast<uint32_t>(last - first);
          // every piece is there: the byte is zero again for the next call
          if (c.last) atomicSub(p.arrived + (first >> 2), static_cast<uint32_t>(last - first + 1) << shift);
          fence_gpu();
        }
        if (!(ok = meet())) break;
        mine = c.last != 0;
        if (mine) {
#pragma unroll
          for (int o = 0; o < S::NB; ++o)
#pragma unroll
            for (int j = 0; j < NT; ++j) sums[o][j] = 0.f;
#pragma unroll 2
          for (int b = first; b <= last; ++b) {
            const float* from = p.part + (2ll * b + (b == first ? first_slot : 0)) * SLOT + tid;
#pragma unroll
            for (int o = 0; o < S::NB; ++o)
#pragma unroll
              for (int j = 0; j < NT; ++j)
                if (tl.row0 + j < tl.row_end) sums[o][j] += __ldcg(from + (o * NT + j) * 128);
          }
        }
      }
      if (mine) {
        // A thread's column goes to a staging area, and a warp takes whole rows from there: the
        // loop over rows is one short piece of code (unrolled with the sums in registers it was
        // fetched anew for each tile, 7000 cycles).
        const int rows = min(NT, tl.row_end - tl.row0);
        constexpr int PASSES = FORM == GATED ? 3 : 2;
        for (int pass = FORM == GATED && !p.out[0] ? 2 : 0; ok && pass < PASSES; ++pass) {
          // of a row, four columns to a lane
          const int col = tl.n * S::COLS + (FORM == GATED ? 0 : pass * 128) + 4 * lane;
          const bool col_ok = col < p.N;
          if (FORM != GATED && tl.n * S::COLS + pass * 128 >= p.N) break;
          if (!(ok = meet())) break;  // the area's last rows have been read
          float* f = reinterpret_cast<float*>(staging) + tid;
          __nv_bfloat16* h = reinterpret_cast<__nv_bfloat16*>(staging) + tid;
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const float a = FORM == GATED || pass == 0 ? sums[0][j] : sums[1][j];
            if (FORM == PLAIN_F32)
              f[j * (S::PITCH / 4)] = a;
            else
              h[j * (S::PITCH / 2)] = __float2bfloat16_rn(FORM != GATED || pass == 0 ? a
                                                          : pass == 1 ? sums[1][j]
                                                                      : silu_f(a) * sums[1][j]);
          }
          if (!(ok = meet())) break;
#pragma unroll 1
          for (int j = warp - FIRST_SUM_WARP; j < rows; j += 4) {
            const size_t at = static_cast<size_t>(tl.row0 + j) * p.N + col;
            if constexpr (FORM == PLAIN_F32) {
              if (col_ok)
                *reinterpret_cast<float4*>(static_cast<float*>(p.out[0]) + at) =
                    *reinterpret_cast<const float4*>(staging + j * S::PITCH + 16 * lane);
            } else {
              uint2 w = *reinterpret_cast<const uint2*>(staging + j * S::PITCH + 8 * lane);
              if (!col_ok) w = make_uint2(0, 0);
              void* out = p.out[FORM == GATED ? pass : 0];
              if (out && col_ok) *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) = w;
              if (FORM == GATED && pass == 2) {
                const BlockScale b = block_scale(
                    __reduce_max_sync(0xffffffffu, top_of_pair(top_of_pair(0, w.x), w.y)));
                const float v[4] = {__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u),
                                    __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u)};
                if (col_ok) *reinterpret_cast<uint32_t*>(p.codes + at) = codes4(v, b);
                if (lane == 0) p.scales[static_cast<size_t>(tl.n) * p.rows + tl.row0 + j] = b.s;
              }
            }
          }
        }
      }
      left -= n;
      kb += n;
      if (kb == nkb) {
        kb = 0;
        ++t;
      }
    }
  }

  __syncthreads();
  if (warp == ISSUE) {
    tc_fence_after();
    tmem_dealloc(tmem_base, S::TMEM);
  }
}

template <int FORM, int NT, bool TRANS>
cudaError_t launch(const Params& p, const Maps& m, int num_sms, cudaStream_t s) {
  auto kern = block_few_kernel<FORM, NT, TRANS>;
  constexpr int smem = smem_bytes<FORM, NT>();
  static_assert(smem <= 232448, "over the 227 KiB of shared memory");
  const cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(num_sms < MAX_BLOCKS ? num_sms : MAX_BLOCKS, 1, 1);
  cfg.blockDim = dim3(NUM_THREADS, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  const cudaError_t le = cudaLaunchKernelEx(&cfg, kern, p, m);
  return le == cudaSuccess ? launched() : le;
}
template <int FORM, bool TRANS>
cudaError_t launch(int nt, const Params& p, const Maps& m, int num_sms, cudaStream_t s) {
  return nt == 16 ? launch<FORM, 16, TRANS>(p, m, num_sms, s)
                  : launch<FORM, 32, TRANS>(p, m, num_sms, s);
}

bool fill(Params& p, Maps& m, const BlockRows& r, const Coded& x, int K, int N, bool trans, int nt,
          bool ahead) {
  memset(&p, 0, sizeof(p));
  memset(&m, 0, sizeof(m));
  p.E = r.E;
  p.offsets = r.offsets;
  p.rows = r.rows;
  p.N = N;
  p.nkb = blocks_of(K);
  p.sa = x.s;
  p.sb_group = p.nkb * blocks_of(N);
  p.sb_k = trans ? 1 : blocks_of(N);
  p.sb_n = trans ? p.nkb : 1;
  p.part = r.part;
  p.arrived = reinterpret_cast<uint32_t*>(r.status) + 16;  // bytes 64 .. 223 of the header
  p.status = r.status;
  p.ahead = ahead;
  return make_map_kmajor(&m.x, x.q, K, r.rows, nt, true);
}
bool map_weight(CUtensorMap* m, const void* q, int E, int K, int N, bool trans) {
  return trans ? make_map_codes(m, q, K, N, E, 128) : make_map_codes(m, q, N, K, E, 128);
}

}  // namespace

cudaError_t few_product(const BlockRows& r, const Coded& a, const Coded& b, int K, int N, bool trans,
                        bool out_f32, void* C, cudaStream_t s, bool ahead) {
  Params p;
  Maps m;
  const int nt = few_tile_rows(r.rows, r.E);
  if (!fill(p, m, r, a, K, N, trans, nt, ahead) || !map_weight(&m.w[0], b.q, r.E, K, N, trans))
    return cudaErrorInvalidValue;
  p.sb[0] = b.s;
  p.out[0] = C;
  if (out_f32)
    return trans ? launch<PLAIN_F32, true>(nt, p, m, r.num_sms, s)
                 : launch<PLAIN_F32, false>(nt, p, m, r.num_sms, s);
  return trans ? launch<PLAIN_BF16, true>(nt, p, m, r.num_sms, s)
               : launch<PLAIN_BF16, false>(nt, p, m, r.num_sms, s);
}

cudaError_t few_fc1_fwd(const BlockRows& r, const Coded& x, const Coded& w1, const Coded& w3,
                        int h, int f, uint16_t* A, uint16_t* B, uint16_t* H,
                        uint8_t* Hq, float* sh, cudaStream_t s) {
  Params p;
  Maps m;
  const int nt = few_tile_rows(r.rows, r.E);
  if (!fill(p, m, r, x, h, f, false, nt, true) || !map_weight(&m.w[0], w1.q, r.E, h, f, false) ||
      !map_weight(&m.w[1], w3.q, r.E, h, f, false))
    return cudaErrorInvalidValue;
  p.sb[0] = w1.s;
  p.sb[1] = w3.s;
  p.out[0] = A;
  p.out[1] = B;
  p.out[2] = H;
  p.codes = Hq;
  p.scales = sh;
  return launch<GATED, false>(nt, p, m, r.num_sms, s);
}

}  // namespace moe
