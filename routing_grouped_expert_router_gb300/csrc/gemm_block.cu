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
//   warp 0      TMA producer: 128 rows of A and 128 columns of B a stage
//   warp 1      tensor memory; in the even CTA the MMA issuer of the pair
//   warps 2-3   none: registers are dealt out by groups of four warps
//   warps 4-11  the sums (warp w: TMEM lanes 32 (w mod 4), columns 64 ((w-4)/4)
//               of each half) and, at a tile's end, its epilogue
// The weight's square blocks let both uses of a weight, as it is (MN-major B)
// and transposed (K-major B), take the same codes.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "block.cuh"
#include "block_quant.cuh"
#include "grouped_gemm.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace moe {

namespace {

enum Form { PLAIN_BF16 = 0, PLAIN_F32 = 1, GATED = 2, GATED_BWD = 3 };

constexpr int kTimeoutCode = 5;   // MOE_ERR_DEVICE_TIMEOUT
constexpr int MAX_E = 64;
constexpr int PM = 256;           // rows of a pair's tile
constexpr int NUM_THREADS = 384;
// Registers of a thread: 168 at launch (3 x 168 x 128 = 64512), then 72 for warps 0-3 and
// 216 for the others, 504 x 128 again.
constexpr int FEW_REGS = 72, MANY_REGS = 216;
constexpr int FIRST_SUM_WARP = 4;
constexpr int SUM_WARPS = 8;
constexpr int SET_BYTES = 4096;   // 32 rows x 128 bytes: one copy of an epilogue

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
  int raster_n, group;      // tile order (see place)
};

struct Maps {
  CUtensorMap a[2], b[2];
  CUtensorMap o[3];   // outputs, 128-byte boxes of 32 rows
  CUtensorMap i[2];   // GATED_BWD: A and B
};

template <int FORM>
struct Shape {
  static constexpr int NH = FORM == GATED_BWD ? 1 : 2;  // halves of 128 columns
  static constexpr int COLS = 128 * NH;                 // accumulator columns
  static constexpr int OUT_COLS = FORM == GATED ? 128 : COLS;  // output columns of a tile
  static constexpr int B_COLS = COLS / 2;               // B columns a CTA loads
  static constexpr int A_BYTES = 128 * 128;
  static constexpr int STAGE_BYTES = A_BYTES + B_COLS * 128;
  static constexpr int STAGES = NH == 2 ? 5 : 6;
  static constexpr int BUFS = 512 / COLS;               // accumulators in tensor memory
  static constexpr int TOPS = FORM == GATED ? 1 : FORM == GATED_BWD ? 2 : 0;
};

template <int FORM>
struct alignas(8) Ctrl {
  using S = Shape<FORM>;
  uint64_t full[S::STAGES], empty[S::STAGES];
  uint64_t tfull[S::BUFS], tempty[S::BUFS];
  uint64_t ab[SUM_WARPS];   // GATED_BWD: A and B in a warp's two sets
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  int off[MAX_E + 1];
  int cum[MAX_E + 1];       // row tiles before each group
  uint16_t tops[S::TOPS ? 2 * S::TOPS * 256 : 1];  // bf16 patterns [tile parity][value][warps' half][row]
};
template <int FORM>
constexpr int smem_bytes() {
  return 1024 + Shape<FORM>::STAGES * Shape<FORM>::STAGE_BYTES + SUM_WARPS * 2 * SET_BYTES +
         static_cast<int>(sizeof(Ctrl<FORM>));
}
static_assert(smem_bytes<PLAIN_BF16>() <= 232448 && smem_bytes<GATED>() <= 232448 &&
                  smem_bytes<GATED_BWD>() <= 232448,
              "over the 227 KiB of shared memory");

struct Tile {
  int e, nb, row0, row_end;
};

// Tile t: groups in order; within one, bands of p.group row tiles (or, raster_n,
// column tiles) swept along the other side, so that the tiles under way share
// what L2 holds.
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
  const int MT = cum[e + 1] - cum[e];
  const int wide = p.raster_n ? NT : MT, along = p.raster_n ? MT : NT;
  const int band = local / (p.group * along);
  const int base = band * p.group;
  const int size = min(p.group, wide - base);
  const int r = local - band * p.group * along;
  const int u = base + r % size, v = r / size;
  tl.e = e;
  tl.nb = p.raster_n ? u : v;
  tl.row0 = off[e] + (p.raster_n ? v : u) * PM;
  tl.row_end = off[e + 1];
  return true;
}

// This thread's scales of one block: its row's, and those of the halves' columns.
struct Scales {
  float a, b[2];
};
// Walks the blocks of a CTA's tiles ahead of the sums.
template <int FORM>
struct ScaleWalk {
  const float* a;
  const float* b[2];
  int kb, t;
  bool real, row_ok;
  __device__ __forceinline__ void enter(const Params& p, const int* off, const int* cum,
                                        int row_in_tile) {
    Tile tl;
    real = place<FORM>(p, off, cum, t, tl);
    kb = 0;
    if (!real) return;
    const int row = tl.row0 + row_in_tile;
    row_ok = row < tl.row_end;
    point(p, tl.e, tl.nb, row, 0);
    e_ = tl.e;
    nb_ = tl.nb;
    row_ = row;
  }
  __device__ __forceinline__ void point(const Params& p, int e, int nb, int row, int product) {
    a = p.sa[product] + (row_ok ? row : 0);
    if (FORM == GATED) {
      for (int i = 0; i < 2; ++i)
        b[i] = p.sb[i] + static_cast<size_t>(e) * p.sb_group + static_cast<size_t>(nb) * p.sb_n;
    } else {
#pragma unroll
      for (int i = 0; i < Shape<FORM>::NH; ++i) {
        const int n = min(Shape<FORM>::NH * nb + i, p.nblocks - 1);  // past the last: zeros anyway
        b[i] = p.sb[product] + static_cast<size_t>(e) * p.sb_group + static_cast<size_t>(n) * p.sb_n;
      }
    }
  }
  __device__ __forceinline__ Scales next(const Params& p, const int* off, const int* cum,
                                         int row_in_tile, int step) {
    Scales s = {0.f, {0.f, 0.f}};
    if (!real) return s;
    if (row_ok) s.a = __ldg(a);
#pragma unroll
    for (int i = 0; i < Shape<FORM>::NH; ++i) s.b[i] = __ldg(b[i]);
    ++kb;
    a += p.rows;
#pragma unroll
    for (int i = 0; i < Shape<FORM>::NH; ++i) b[i] += p.sb_k;
    if (kb == p.kblocks && p.products == 2) point(p, e_, nb_, row_, 1);
    if (kb == p.kblocks * p.products) {
      t += step;
      enter(p, off, cum, row_in_tile);
    }
    return s;
  }
  int e_, nb_, row_;
};

__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void split(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
// sums += scale * (32 columns of this thread's TMEM lane)
__device__ __forceinline__ void add_block(uint32_t taddr, float scale, uint64_t* sums) {
  float v[32];
  tmem_ld32(taddr, v);
  const uint64_t s2 = pair_of(scale, scale);
#pragma unroll
  for (int i = 0; i < 16; ++i)
    asm("fma.rn.f32x2 %0, %1, %2, %0;"
        : "+l"(sums[i])
        : "l"(pair_of(v[2 * i], v[2 * i + 1])), "l"(s2));
}

// sigmoid and silu with the fast exponential and quotient: their few ulps are
// far below the bf16 rounding of all that is stored.
__device__ __forceinline__ float sigmoid_f(float a) { return __fdividef(1.0f, 1.0f + __expf(-a)); }
__device__ __forceinline__ float silu_f(float a) { return __fdividef(a, 1.0f + __expf(-a)); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ float lo_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_of(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// A warp's two 4 KiB sets between its registers and the TMA unit: 32 rows of 128
// bytes, 16-byte piece j of row i in slot j ^ (i mod 8) (128-byte swizzle).
struct Staging {
  uint4* sets;
  int used = 0;
  // A set whose last copy has been read.
  __device__ __forceinline__ uint4* take(int lane) {
    uint4* s = sets + (used++ & 1) * (SET_BYTES / 16);
    if (lane == 0) bulk_wait_read_1();
    __syncwarp();
    return s;
  }
};
__device__ __forceinline__ void send(const CUtensorMap* map, uint4* set, int x, int y, int lane) {
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(map, smem_u32(set), x, y);
    bulk_commit();
  }
}
// 64 columns of bf16 (w: 32 pairs) of a warp's 32 rows to out [., N] at (row, col): whole
// rows by TMA, or, where a row is not this group's, each lane its own.
__device__ __forceinline__ void put_bf16(Staging& st, const CUtensorMap* map, void* out, int N,
                                         const uint32_t* w, int row, int col, bool row_ok,
                                         bool all_ok, int lane) {
  if (all_ok) {
    uint4* set = st.take(lane);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      set[lane * 8 + (j ^ (lane & 7))] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
    send(map, set, col, row - lane, lane);
  } else if (row_ok) {
    uint4* d = reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + static_cast<size_t>(row) * N + col);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (col + 8 * j < N) d[j] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
  }
}
__device__ __forceinline__ void put_f32(Staging& st, const CUtensorMap* map, void* out, int N,
                                        const uint64_t* v, int row, int col, bool row_ok,
                                        bool all_ok, int lane) {
  float f[32];
#pragma unroll
  for (int i = 0; i < 16; ++i) split(v[i], f[2 * i], f[2 * i + 1]);
  if (all_ok) {
    float4* set = reinterpret_cast<float4*>(st.take(lane));
#pragma unroll
    for (int j = 0; j < 8; ++j)
      set[lane * 8 + (j ^ (lane & 7))] = make_float4(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
    send(map, reinterpret_cast<uint4*>(set), col, row - lane, lane);
  } else if (row_ok) {
    float4* d = reinterpret_cast<float4*>(static_cast<float*>(out) + static_cast<size_t>(row) * N + col);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (col + 4 * j < N) d[j] = make_float4(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
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

__device__ __forceinline__ void sum_warps_sync() {
  asm volatile("bar.sync 1, 256;" ::: "memory");
}

template <int FORM, bool B_MN>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    block_pair_kernel(const __grid_constant__ Params p, const __grid_constant__ Maps maps) {
  using S = Shape<FORM>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* staging = smem + S::STAGES * S::STAGE_BYTES;
  Ctrl<FORM>& c = *reinterpret_cast<Ctrl<FORM>*>(staging + SUM_WARPS * 2 * SET_BYTES);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int cid = static_cast<int>(cluster_id_x());
  const int ncl = static_cast<int>(cluster_count_x());
  const int nkb = p.kblocks * p.products;

  // ------------------------------------------------------------ set-up
  if (warp == 0 && lane == 0) {
    for (int s = 0; s < S::STAGES; ++s) {
      mbar_init(smem_u32(&c.full[s]), 1);
      mbar_init(smem_u32(&c.empty[s]), 1);
    }
    for (int b = 0; b < S::BUFS; ++b) {
      mbar_init(smem_u32(&c.tfull[b]), 1);
      mbar_init(smem_u32(&c.tempty[b]), 2 * SUM_WARPS);
    }
    for (int w = 0; w < SUM_WARPS; ++w) mbar_init(smem_u32(&c.ab[w]), 1);
    mbar_init(smem_u32(&c.drain), 1);
    c.abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&maps.a[0]);
    tma_prefetch_desc(&maps.b[0]);
  }
  if (warp == 1) {
    tmem_alloc2(smem_u32(&c.tmem_base), 512);
    tmem_relinquish2();
    tc_fence_before();
  }
  if (warp >= FIRST_SUM_WARP) {
    for (int e = threadIdx.x - 32 * FIRST_SUM_WARP; e <= p.E; e += 256)
      c.off[e] = p.offsets ? __ldg(p.offsets + e) : (e ? p.rows : 0);
  }
  __syncthreads();
  if (threadIdx.x == 32 * FIRST_SUM_WARP) {
    // clamped into order, so that every access stays inside its buffer
    bool bad = c.off[0] != 0;
    for (int e = 0; e <= p.E; ++e) {
      const int o = c.off[e], low = e ? c.off[e - 1] : 0;
      const int in = min(max(o, low), p.rows);
      bad = bad || in != o;
      c.off[e] = in;
    }
    if (bad) report_bad_index(p.status);
    c.cum[0] = 0;
    for (int e = 0; e < p.E; ++e) c.cum[e + 1] = c.cum[e] + (c.off[e + 1] - c.off[e] + PM - 1) / PM;
  }
  cluster_sync_all();  // both CTAs' barriers exist before any arrival from the other
  tc_fence_after();
  const uint32_t tmem_base = c.tmem_base;
  volatile int* abort_flag = &c.abort;
  const uint32_t peer_abort = mapa_shared(smem_u32(&c.abort), rank ^ 1u);
  auto give_up = [&]() {
    *abort_flag = 1;
    st_cluster_u32(peer_abort, 1);
  };

  if (warp < FIRST_SUM_WARP) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(FEW_REGS));
  if (warp == 0) {
    // ------------------------------------------------------- TMA producer
    if (lane == 0) {
      int q = 0;
      bool ok = true;
      Tile tl;
      for (int t = cid; ok && place<FORM>(p, c.off, c.cum, t, tl); t += ncl) {
        for (int kb = 0; kb < nkb; ++kb, ++q) {
          const int s = q % S::STAGES;
          const uint32_t ph = (q / S::STAGES) & 1;
          if (*abort_flag || !mbar_wait(smem_u32(&c.empty[s]), ph ^ 1, p.status, kTimeoutCode)) {
            give_up();
            ok = false;
            break;
          }
          // the even CTA's barrier counts both CTAs' bytes
          const uint32_t own = smem_u32(&c.full[s]);
          const uint32_t bar = rank == 0 ? own : mapa_shared(own, 0);
          if (rank == 0) mbar_expect_tx(own, 2 * S::STAGE_BYTES);
          const int which = kb >= p.kblocks ? 1 : 0;
          const int k = (which ? kb - p.kblocks : kb) * kBlock;
          const uint32_t a_dst = smem_u32(smem + s * S::STAGE_BYTES);
          const uint32_t b_dst = a_dst + S::A_BYTES;
          const CUtensorMap* bm = FORM == GATED ? &maps.b[rank] : &maps.b[which];
          const int n = FORM == GATED ? tl.nb * 128 : tl.nb * S::COLS + rank * S::B_COLS;
          if (rank == 0) {
            tma_load_2d(a_dst, &maps.a[which], k, tl.row0, bar);
            tma_load_3d(b_dst, bm, B_MN ? n : k, B_MN ? k : n, tl.e, bar);
          } else {
            tma_load_2d_pair(a_dst, &maps.a[which], k, tl.row0 + 128, bar);
            tma_load_3d_pair(b_dst, bm, B_MN ? n : k, B_MN ? k : n, tl.e, bar);
          }
        }
      }
      if (!ok && rank == 0) {
        // the loads already asked for land before the CTA can end
        const int first = q > S::STAGES ? q - S::STAGES : 0;
        for (int r = first; r < q; ++r)
          mbar_wait_cluster(smem_u32(&c.full[r % S::STAGES]), (r / S::STAGES) & 1, p.status,
                            kTimeoutCode);
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {
      // ----------------------------------------------- MMA issuer (even CTA)
      constexpr uint32_t IDESC = idesc_e4m3(PM, S::COLS) | (B_MN ? 1u << 16 : 0u);
      // 32 deep: 32 bytes of a K-major row; 32 rows of 128 bytes of an MN-major tile
      constexpr uint32_t B_STEP = B_MN ? 32 * 128 : 32;
      int q = 0;
      bool ok = true;
      Tile tl;
      for (int t = cid; ok && place<FORM>(p, c.off, c.cum, t, tl); t += ncl) {
        for (int kb = 0; kb < nkb; ++kb, ++q) {
          const int s = q % S::STAGES;
          const int buf = q % S::BUFS;
          if (*abort_flag ||
              !mbar_wait(smem_u32(&c.tempty[buf]), ((q / S::BUFS) & 1) ^ 1, p.status,
                         kTimeoutCode) ||
              !mbar_wait(smem_u32(&c.full[s]), (q / S::STAGES) & 1, p.status, kTimeoutCode)) {
            give_up();
            ok = false;
            break;
          }
          if (lane == 0) {
            tc_fence_after();
            const uint32_t a_base = smem_u32(smem + s * S::STAGE_BYTES);
            const uint32_t b_base = a_base + S::A_BYTES;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma2_e4m3(tmem_base + buf * S::COLS, smem_desc(a_base + kk * 32, 16, 1024),
                         smem_desc(b_base + kk * B_STEP, 16, 1024), IDESC, kk != 0);
            umma2_commit_mc(smem_u32(&c.empty[s]), 0x3);
            umma2_commit_mc(smem_u32(&c.tfull[buf]), 0x3);
          }
          __syncwarp();
        }
      }
      if (lane == 0) {
        umma2_commit(smem_u32(&c.drain));
        mbar_wait(smem_u32(&c.drain), 0, p.status, kTimeoutCode);
      }
      __syncwarp();
    }
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(MANY_REGS));
    // ------------------------------------------- sums and epilogue (8 warps)
    const int quarter = warp & 3;                 // TMEM lanes this warp may read
    const int side = (warp - FIRST_SUM_WARP) >> 2;             // which 64 columns of each half
    const int trow = quarter * 32 + lane;         // TMEM lane: row of this CTA's 128
    const int row_in_tile = rank * 128 + trow;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    Staging st;
    st.sets = reinterpret_cast<uint4*>(staging + (warp - FIRST_SUM_WARP) * 2 * SET_BYTES);
    int q = 0, it = 0;
    Tile tl;
    ScaleWalk<FORM> walk;
    walk.t = cid;
    walk.enter(p, c.off, c.cum, row_in_tile);
    // two blocks ahead: a load's way to L2 and back
    Scales s0 = walk.next(p, c.off, c.cum, row_in_tile, ncl);
    Scales s1 = walk.next(p, c.off, c.cum, row_in_tile, ncl);
    int asked = 0, had = 0;  // GATED_BWD: loads of A and B into the sets, and those that landed
    bool ok = true;
    // After an abort the forms that meet at a barrier for each tile go on meeting there.
    for (int t = cid; (ok || S::TOPS) && place<FORM>(p, c.off, c.cum, t, tl); t += ncl, ++it) {
      const int row = tl.row0 + row_in_tile;
      const bool row_ok = row < tl.row_end;
      const bool all_ok = __all_sync(0xffffffffu, row_ok);
      const int col0 = tl.nb * S::OUT_COLS + side * 64;
      if constexpr (FORM == GATED_BWD) {
        // this warp's rows and columns of A and B come while the sums run
        if (ok && col0 < p.N) {
          fence_proxy_async_smem();  // the reads of the sets come before the refill
          __syncwarp();
          ++asked;
          if (lane == 0) {
            bulk_wait_read_0();
            mbar_expect_tx(smem_u32(&c.ab[warp - FIRST_SUM_WARP]), 2 * SET_BYTES);
            tma_load_2d(smem_u32(st.sets), &maps.i[0], col0, row - lane, smem_u32(&c.ab[warp - FIRST_SUM_WARP]));
            tma_load_2d(smem_u32(st.sets + SET_BYTES / 16), &maps.i[1], col0, row - lane,
                        smem_u32(&c.ab[warp - FIRST_SUM_WARP]));
          }
        }
      }
      uint64_t sums[S::NH][32];
#pragma unroll
      for (int h = 0; h < S::NH; ++h)
#pragma unroll
        for (int i = 0; i < 32; ++i) sums[h][i] = 0;
#pragma unroll 1
      for (int kb = 0; ok && kb < nkb; ++kb, ++q) {
        const Scales s = s0;
        s0 = s1;
        s1 = walk.next(p, c.off, c.cum, row_in_tile, ncl);
        const int buf = q % S::BUFS;
        const bool got = !*abort_flag &&
                         mbar_wait(smem_u32(&c.tfull[buf]), (q / S::BUFS) & 1, p.status, kTimeoutCode);
        if (!__all_sync(0xffffffffu, got)) {
          give_up();
          ok = false;
          continue;
        }
        tc_fence_after();
        const uint32_t at = tmem_base + buf * S::COLS + lanes + side * 64;
#pragma unroll
        for (int h = 0; h < S::NH; ++h) {
          add_block(at + h * 128, s.a * s.b[h], sums[h]);
          add_block(at + h * 128 + 32, s.a * s.b[h], sums[h] + 16);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(mapa_shared(smem_u32(&c.tempty[buf]), 0));
      }
      if (!ok) {
        if (S::TOPS) sum_warps_sync();
        continue;
      }
      if constexpr (FORM == PLAIN_BF16) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int col = col0 + h * 128;
          if (col >= p.N) continue;
          uint32_t w[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float lo, hi;
            split(sums[h][i], lo, hi);
            w[i] = pack_bf16(lo, hi);
          }
          put_bf16(st, &maps.o[0], p.out[0], p.N, w, row, col, row_ok, all_ok, lane);
        }
      } else if constexpr (FORM == PLAIN_F32) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int col = col0 + h * 128 + i * 32;
            if (col < p.N)
              put_f32(st, &maps.o[0], p.out[0], p.N, sums[h] + 16 * i, row, col, row_ok, all_ok, lane);
          }
      } else if constexpr (FORM == GATED) {
        uint32_t w[32];
        uint32_t top = 0;
        if (col0 < p.N) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float a0, a1, b0, b1;
            split(sums[0][i], a0, a1);
            split(sums[1][i], b0, b1);
            w[i] = pack_bf16(silu_f(a0) * b0, silu_f(a1) * b1);
            top = top_of_pair(top, w[i]);
          }
        }
        uint16_t* tops = c.tops + (it & 1) * 256;
        tops[side * 128 + trow] = static_cast<uint16_t>(top >> 16);
        sum_warps_sync();
        top = max(top, static_cast<uint32_t>(tops[(side ^ 1) * 128 + trow]) << 16);
        if (col0 < p.N) {
          const BlockScale bs = block_scale(top);
          if (row_ok) {
            if (side == 0) p.scales[0][static_cast<size_t>(tl.nb) * p.rows + row] = bs.s;
            uint4* d = reinterpret_cast<uint4*>(p.codes[0] + static_cast<size_t>(row) * p.N + col0);
#pragma unroll
            for (int j = 0; j < 4; ++j) d[j] = codes16(w + 8 * j, bs);
          }
          if (p.out[0]) {
            put_bf16(st, &maps.o[2], p.out[2], p.N, w, row, col0, row_ok, all_ok, lane);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                float lo, hi;
                split(sums[h][i], lo, hi);
                w[i] = pack_bf16(lo, hi);
              }
              put_bf16(st, &maps.o[h], p.out[h], p.N, w, row, col0, row_ok, all_ok, lane);
            }
          }
        }
      } else {
        uint32_t top_a = 0, top_b = 0;
        uint4* sa = st.sets;
        uint4* sb = st.sets + SET_BYTES / 16;
        if (col0 < p.N) {
          const bool got = mbar_wait(smem_u32(&c.ab[warp - FIRST_SUM_WARP]), had & 1, p.status,
                                     kTimeoutCode);
          ++had;
          if (!__all_sync(0xffffffffu, got)) {
            give_up();
            ok = false;
          }
        }
        if (ok && col0 < p.N) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int at = lane * 8 + (j ^ (lane & 7));
            const uint4 ra = sa[at], rb = sb[at];
            const uint32_t wa[4] = {ra.x, ra.y, ra.z, ra.w}, wb[4] = {rb.x, rb.y, rb.z, rb.w};
            uint32_t da[4], db[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float dh[2];
              split(sums[0][4 * j + i], dh[0], dh[1]);
              const float av[2] = {lo_of(wa[i]), hi_of(wa[i])}, bv[2] = {lo_of(wb[i]), hi_of(wb[i])};
              float xa[2], xb[2];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const float sg = sigmoid_f(av[k]);
                xa[k] = dh[k] * bv[k] * sg * (1.0f + av[k] * (1.0f - sg));
                xb[k] = dh[k] * av[k] * sg;
              }
              da[i] = pack_bf16(xa[0], xa[1]);
              db[i] = pack_bf16(xb[0], xb[1]);
              top_a = top_of_pair(top_a, da[i]);
              top_b = top_of_pair(top_b, db[i]);
            }
            sa[at] = make_uint4(da[0], da[1], da[2], da[3]);
            sb[at] = make_uint4(db[0], db[1], db[2], db[3]);
          }
        }
        uint16_t* tops = c.tops + (it & 1) * 512;
        tops[side * 128 + trow] = static_cast<uint16_t>(top_a >> 16);
        tops[256 + side * 128 + trow] = static_cast<uint16_t>(top_b >> 16);
        sum_warps_sync();
        if (!ok) continue;
        top_a = max(top_a, static_cast<uint32_t>(tops[(side ^ 1) * 128 + trow]) << 16);
        top_b = max(top_b, static_cast<uint32_t>(tops[256 + (side ^ 1) * 128 + trow]) << 16);
        if (col0 < p.N) {
          if (all_ok) {
            send(&maps.o[0], sa, col0, row - lane, lane);
            send(&maps.o[1], sb, col0, row - lane, lane);
          }
          if (row_ok) {
            const BlockScale ba = block_scale(top_a), bb = block_scale(top_b);
            if (side == 0) {
              p.scales[0][static_cast<size_t>(tl.nb) * p.rows + row] = ba.s;
              p.scales[1][static_cast<size_t>(tl.nb) * p.rows + row] = bb.s;
            }
            const size_t o = static_cast<size_t>(row) * p.N + col0;
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              const uint4* set = v ? sb : sa;
              const BlockScale& b = v ? bb : ba;
              uint4* d = reinterpret_cast<uint4*>(p.codes[v] + o);
              uint4* keep = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out[v]) + o);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint4 x = set[lane * 8 + ((2 * j) ^ (lane & 7))];
                const uint4 y = set[lane * 8 + ((2 * j + 1) ^ (lane & 7))];
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
    }
    if (had < asked)  // after an abort: loads of A and B still on their way
      mbar_wait(smem_u32(&c.ab[warp - FIRST_SUM_WARP]), had & 1, p.status, kTimeoutCode);
    if (lane == 0) bulk_wait_all();  // staged rows written out before the CTA ends
  }

  // ------------------------------------------------------------ teardown
  __syncthreads();
  cluster_sync_all();  // the pair's MMAs and TMEM reads are finished
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc2(tmem_base, 512);
  }
}

// The smaller operand of a group stays in L2 where it fits, in one band; otherwise
// bands of eight pair tiles.
constexpr long long kL2ResidentBytes = 48ll << 20;
void set_raster(Params& p, long long a_bytes, long long b_bytes, long long slab_a, long long slab_b) {
  auto bands = [](long long slab) {
    const long long g = slab > 0 ? kL2ResidentBytes / slab : 1;
    return static_cast<int>(g < 1 ? 1 : (g > 4096 ? 4096 : g));
  };
  p.raster_n = 0;
  p.group = 16;
  if (a_bytes <= kL2ResidentBytes && a_bytes <= b_bytes) {
    p.group = bands(slab_a);
  } else if (b_bytes <= kL2ResidentBytes) {
    p.raster_n = 1;
    p.group = bands(slab_b);
  }
}

template <int FORM, bool B_MN>
cudaError_t launch_pairs(const Params& p, const Maps& m, int num_sms, cudaStream_t s) {
  auto kern = block_pair_kernel<FORM, B_MN>;
  constexpr int smem = smem_bytes<FORM>();
  const cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(NUM_THREADS, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const long long nt = (p.N + Shape<FORM>::OUT_COLS - 1) / Shape<FORM>::OUT_COLS;
  const long long most = nt * ((p.rows + PM - 1) / PM + p.E);
  const int fit = pairs_that_fit(reinterpret_cast<const void*>(kern), cfg, num_sms);
  cfg.gridDim = dim3(2 * static_cast<unsigned>(most < fit ? most : fit), 1, 1);
  const cudaError_t le = cudaLaunchKernelEx(&cfg, kern, p, m);
  return le == cudaSuccess ? launched() : le;
}

Params params_of(const BlockRows& r, int K, int N, bool trans) {
  Params p;
  memset(&p, 0, sizeof(p));
  p.E = r.E;
  p.offsets = r.offsets;
  p.rows = r.rows;
  p.status = r.status;
  p.N = N;
  p.kblocks = blocks_of(K);
  p.products = 1;
  p.nblocks = blocks_of(N);
  p.sb_group = p.kblocks * p.nblocks;
  p.sb_k = trans ? 1 : p.nblocks;
  p.sb_n = trans ? p.kblocks : 1;
  return p;
}
long long rows_each(const BlockRows& r) { return (r.rows + r.E - 1) / r.E; }

bool map_rows(CUtensorMap* m, const void* q, int K, int rows) {
  return make_map_kmajor(m, q, K, rows, 128, true);
}
// A weight as it lies: boxes of 128 contiguous codes x box_rows.
bool map_weight(CUtensorMap* m, const void* q, int E, int K, int N, bool trans, int cols) {
  return trans ? make_map_codes(m, q, K, N, E, cols) : make_map_codes(m, q, N, K, E, 128);
}

}  // namespace

cudaError_t block_product(const BlockRows& r, const Coded& a, const Coded& b, int K, int N,
                          bool trans, bool out_f32, void* C, cudaStream_t s) {
  if (r.rows == 0) return cudaSuccess;
  Params p = params_of(r, K, N, trans);
  p.sa[0] = a.s;
  p.sb[0] = b.s;
  p.out[0] = C;
  Maps m;
  memset(&m, 0, sizeof(m));
  if (!map_rows(&m.a[0], a.q, K, r.rows) || !map_weight(&m.b[0], b.q, r.E, K, N, trans, 128) ||
      !make_map_box(&m.o[0], C, out_f32, N, r.rows))
    return cudaErrorInvalidValue;
  set_raster(p, rows_each(r) * K, 1ll * K * N, 1ll * PM * K, 256ll * K);
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
  if (A && (!make_map_box(&m.o[0], A, false, f, r.rows) ||
            !make_map_box(&m.o[1], B, false, f, r.rows) ||
            !make_map_box(&m.o[2], H, false, f, r.rows)))
    return cudaErrorInvalidValue;
  set_raster(p, rows_each(r) * h, 2ll * h * f, 1ll * PM * h, 256ll * h);
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
      !make_map_box(&m.o[0], dA, false, f, r.rows) || !make_map_box(&m.o[1], dB, false, f, r.rows) ||
      !make_map_box(&m.i[0], A, false, f, r.rows) || !make_map_box(&m.i[1], B, false, f, r.rows))
    return cudaErrorInvalidValue;
  set_raster(p, rows_each(r) * h, 1ll * h * f, 1ll * PM * h, 128ll * h);
  return launch_pairs<GATED_BWD, false>(p, m, r.num_sms, s);
}

cudaError_t block_fc1_dgrad(const BlockRows& r, const Coded& da, const Coded& db, const Coded& w1,
                            const Coded& w3, int h, int f, bool out_f32, void* dX,
                            cudaStream_t s) {
  if (r.rows == 0) return cudaSuccess;
  Params p = params_of(r, f, h, true);
  p.products = 2;
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
      !make_map_box(&m.o[0], dX, out_f32, h, r.rows))
    return cudaErrorInvalidValue;
  set_raster(p, rows_each(r) * 2 * f, 2ll * f * h, 1ll * PM * 2 * f, 256ll * 2 * f);
  return out_f32 ? launch_pairs<PLAIN_F32, false>(p, m, r.num_sms, s)
                 : launch_pairs<PLAIN_BF16, false>(p, m, r.num_sms, s);
}

}  // namespace moe
