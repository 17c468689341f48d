// decode.cu -- the whole MoE layer for a few tokens in one kernel:
// moe_layer_decode, moe_layer_decode_fp8 and moe_layer_decode_fp8_as_fwd.
//
//   l = x Wg (+ b);  the k largest;  gates = softmax over them
//   H[p] = silu(x W1[e]) * (x W3[e])     for each placed assignment p = (t, e)
//   O[p] = H[p] W2[e];   y[t] = sum_j gates[t,j] O[p(t,j)]
//
// What bounds it: the weights of the chosen experts are read once, and with at
// most 128 tokens they are nearly all the bytes and leave the tensor cores idle
// most of the time (128 tokens x 2 slots over 8 experts: 32 MACs for each
// weight, where a GB300 can do 280 in the time its 2 bytes take to arrive).  So
// the kernel is built as a stream of weights:
//   * one persistent cooperative kernel, one block for each SM, four phases
//     (route, FC1, FC2, combine);
//   * the products are taken transposed, weights as the 128-row operand A of
//     tcgen05.mma and the tokens as its N columns (16 to 128), so that the
//     smallest batch wastes columns of an idle tensor core, not bytes;
//   * 32 KiB weight stages (two 128-column tiles x 64 rows of bf16, 128 of
//     e4m3) flow through a ring of up to 5 stages that TMA fills, about 170 KiB
//     in flight on each SM; nothing but the TMA and MMA units touches them;
//   * each phase's k-steps, over all its tiles in a row, are cut into pieces
//     whatever the tiles' borders: the number of experts hit decides the tiles,
//     and a tile for each block would leave up to half of the SMs idle in the
//     last wave.  Every block starts on a piece of its own; in long phases the
//     last sixth is cut smaller and taken by whoever is free (see Cut).  A tile
//     that two or more pieces share is joined in the pieces' order, by the whole
//     grid: FC1's after a barrier, since SwiGLU needs the whole sums, FC2's when
//     y is combined.  So the result does not depend on timing;
//   * FC2's first stages of weights are loaded before the barriers that make H
//     whole (bringing more of them into L2 meanwhile gained nothing).
// Measured on GB300 (1.9 GHz): 128 tokens, top 2 of 8 experts of 4096 x 14336 in
// 456 us, the weights at 6.2 TB/s over all and 6.7 in FC1 (a kernel of these
// loads and nothing else reads 7.1); 32 tokens, top 6 of 64 experts of 2048 x 1408
// in 179 us (DRAM reads 1.08 GB, the weights hit; tensor pipe 8% busy); one token
// of the same layer in 38 us, of which the weights need 15: the rest is the
// router (5), the first loads (3), four grid barriers (1 each), joins and combine.
// Where an expert has many rows and its tiles few k-steps, FC1's end bounds
// instead, a tile's rows in four warps: 128 tokens, top 8 of 64 experts of
// 512 x 8192, 281 us (weights 238), with 114 rows to the busiest expert 389 (230);
// e4m3, with a row at a time, 400 (119) and 970 or more (115).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "../../include/moe.h"
#include "api_internal.h"
#include "decode.cuh"
#include "grouped_gemm.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

// Warp 0 feeds the ring, warp 1 issues the MMAs, warps 4 to 7 are the epilogue;
// the others help where a phase's work is spread over all threads.
constexpr int kThreads = 512;
constexpr int kHelpers = kThreads - 64;
constexpr int kIdleWarps = kThreads / 32 - 6;  // neither of those roles
constexpr int kWBytes = 32768;     // weights of a stage
constexpr int kMaxStages = 5;
constexpr int kQueue = 4;          // pieces between the producer and the others
constexpr int kMaxRows = kDecodeMaxT * 8;  // placed assignments
constexpr int kMaxE = 64;
constexpr int kMaxPieces = 640, kMaxTiles = 1024;
constexpr int kGroupTok = 8;       // tokens of a router work unit at most
constexpr int kTimeoutCode = MOE_ERR_DEVICE_TIMEOUT;
constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kSmemMax = 232448;

// The workspace's first 256 bytes: the status word, then words that are zero
// between calls (every call leaves them so).
constexpr int kBarWord = 16;    // arrivals at the grid barriers
constexpr int kExitWord = 17;   // blocks that are done
constexpr int kGroupWord = 32;  // router units done for each token group (16)

struct Params {
  int T, h, f, E, k, capacity;
  int n1;                   // T rounded up to 16: FC1's MMA columns
  int ring_bytes;           // shared memory of the ring
  int tok_group, groups, slices, slice_h;  // router work units
  const uint16_t* x;
  const float *Wg, *b;
  int32_t* idx;
  float* gates;
  float* logits;            // [groups, slices, tok_group, E]
  uint16_t* H;              // [T*k, f]; bf16 weights: [2, T*k, f], H's high and low parts
  float* O;                 // [T*k, h]
  float* part;              // FC1 [2 * pieces][T, 2, 128]: sums of shared tiles;
                            // FC2 [pieces][T, 256]: of tiles begun in another piece
  unsigned* claim;          // [2]: pieces taken of FC1's and FC2's later rounds
  uint16_t* y;
  // e4m3
  uint8_t *xq, *Hq;
  float* sx;
  unsigned* amax;           // [T*k]: bits of max |H|
  const float *s1, *s3, *s2;
  int* status;
};

struct Maps {
  CUtensorMap x, w1, w3, h, w2;
};

struct alignas(16) Ctrl {
  uint64_t full[kMaxStages], empty[kMaxStages], tfull[2], tempty[2], hready, drain, rbar;
  uint64_t qfull[kQueue], qempty[kQueue];
  uint32_t tmem_base;
  int abort, flag, go, nact, most;  // most: rows of the busiest expert
  int piece[kQueue];        // the block's pieces in order, -1 at a phase's end
  int off[kMaxE + 1];       // first row of each expert
  int act[kMaxE];           // experts with rows
  int act_of[kMaxE];        // its inverse
  float gate[kMaxRows];     // by assignment
  float sx[kDecodeMaxT];
  int16_t pos[kMaxRows];    // assignment -> row, -1 dropped
  uint8_t exp[kMaxRows];    // assignment -> expert
  uint8_t tok[kMaxRows];    // row -> token
  int joins;
  uint32_t tile[kMaxTiles]; // FC2 tile -> its first piece | further pieces << 16
  union {
    uint16_t hist[kMaxRows / 32][kMaxE];  // dispatch
    // FC1 tiles to join: the piece after the one that begins it | parts << 16;
    // its expert among the active ones << 16 | its number
    uint2 join[kMaxPieces];
  };
};

// One phase's k-steps [0, total) cut into pieces, in up to kRounds rounds of one
// piece for each block.  Piece b of round 0 is block b's; those of the later,
// ever smaller rounds go to whoever comes first.  The SMs do not stream equally
// fast: on GB300 whole groups of 16 to 20 were 10 to 17% behind the others,
// which ones changing with the weights' addresses (16 tokens, 11 of 32 experts:
// 345 us for the fastest SM's share of FC1, 389 us for the slowest's).  Below
// kRoundsFrom k-steps for each block the phase is too short to gain by it.
constexpr int kRounds = 4;
constexpr unsigned kRoundsFrom = 48;
struct Cut {
  unsigned total, blocks, rounds;
  unsigned at[kRounds + 1];  // rounds' borders
  // Later rounds of 8, 5 and 3% of a block's share, but of no fewer than `least`
  // k-steps a piece: every piece of a tile is one more sum to add.  Round 0 is
  // half of all at the least.
  __device__ Cut(unsigned n, unsigned grid, unsigned tile_steps) : total(n) {
    const unsigned share = n / grid, least = max(4u, tile_steps / 8u);
    rounds = share >= max(kRoundsFrom, 2u * (kRounds - 1) * least) ? kRounds : 1;
    blocks = n < grid ? n : grid;
    at[0] = 0;
    at[4] = n;
    at[3] = rounds == 1 ? n : n - grid * max(least, share * 3u / 100u);
    at[2] = rounds == 1 ? n : at[3] - grid * max(least, share * 5u / 100u);
    at[1] = rounds == 1 ? n : at[2] - grid * max(least, share * 8u / 100u);
  }
  __device__ unsigned start(unsigned piece) const {
    const unsigned r = piece / blocks, j = piece - r * blocks;
    unsigned lo = at[0], hi = at[1];
#pragma unroll
    for (int i = 1; i < kRounds; ++i)
      if (r >= i) {
        lo = at[i];
        hi = at[i + 1];
      }
    return lo + j * (hi - lo) / blocks;
  }
  __device__ unsigned end(unsigned piece) const {
    return piece + 1 == rounds * blocks ? total : start(piece + 1);
  }
  __device__ unsigned piece_of(unsigned q) const {
    unsigned r = 0, lo = at[0], hi = at[1];
#pragma unroll
    for (int i = 1; i < kRounds; ++i)
      if (q >= at[i]) {
        r = i;
        lo = at[i];
        hi = at[i + 1];
      }
    return r * blocks + ((q - lo + 1) * blocks - 1) / (hi - lo);
  }
};

__device__ __forceinline__ void fence_proxy_async_all() {
  asm volatile("fence.proxy.async;" ::: "memory");
}

// Waits (with a limit) until *word has reached `target`; what was written before
// the words that took it there is then seen.
__device__ __forceinline__ bool wait_count(const unsigned* word, unsigned target, int* status) {
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    unsigned v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(word) : "memory");
    if (static_cast<int>(v - target) >= 0) break;
    if ((i & 255u) == 0) {
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > kWaitLimitNs) {
        atomicExch(status, kTimeoutCode);
        return false;
      }
    }
  }
  return true;
}

// A barrier over the grid, by one thread of each block between two barriers of
// the block: everything that its threads wrote before is seen by every block
// after.  Release and acquire carry that; full fences made it 0.4 us slower.
// `target` counts all arrivals of the launch so far.
__device__ __forceinline__ bool grid_barrier(unsigned* word, unsigned target, int* status) {
  asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(word) : "memory");
  return wait_count(word, target, status);
}

// A barrier of all warps but 0 and 1.
__device__ __forceinline__ void helper_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kHelpers) : "memory");
}

// Accumulator columns [col, col + 16) of this thread's lane.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
// One column (no wait).
__device__ __forceinline__ void tmem_ld1(uint32_t taddr, uint32_t& r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr) : "memory");
}
__device__ __forceinline__ void tmem_wait8(uint32_t (&a)[8], uint32_t (&b)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(a[0]), "+r"(a[1]), "+r"(a[2]), "+r"(a[3]), "+r"(a[4]), "+r"(a[5]),
                 "+r"(a[6]), "+r"(a[7]), "+r"(b[0]), "+r"(b[1]), "+r"(b[2]), "+r"(b[3]),
                 "+r"(b[4]), "+r"(b[5]), "+r"(b[6]), "+r"(b[7])::"memory");
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// The scale and codes of a quantised row.  moe_layer_decode_fp8's scale is amax
// times the fp32 reciprocal of 448, moe_layer_decode_fp8_as_fwd's is fp8.cu's
// quotient.  They are an ulp apart, but 0.8 to 6% of a bf16 row's values lie
// exactly between two codes, and that ulp chooses.
template <bool QUOT>
__device__ __forceinline__ float scale_of(float amax) {
  if (!(amax > 0.f)) return 1.0f;
  return QUOT ? __fdiv_rn(amax, 448.0f) : __fmul_rn(amax, 1.0f / 448.0f);
}
__device__ __forceinline__ uint32_t quant2(uint32_t w, float s) {
  return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(
      make_float2(__fdiv_rn(bf16_lo(w), s), __fdiv_rn(bf16_hi(w), s)), __NV_SATFINITE, __NV_E4M3));
}
__device__ __forceinline__ uint2 quant8(const uint4& w, float s) {
  return make_uint2(quant2(w.x, s) | quant2(w.y, s) << 16, quant2(w.z, s) | quant2(w.w, s) << 16);
}
__device__ __forceinline__ float amax8(const uint4& w) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = fmaxf(m, fmaxf(fabsf(bf16_lo(u[i])), fabsf(bf16_hi(u[i]))));
  return m;
}

// ------------------------------------------------------------------ route
// A logit as an integer of the same order (-0 as 0, NaN as minus infinity).
__device__ __forceinline__ unsigned order_of(float v) {
  const unsigned u = __float_as_uint(isnan(v) ? -INFINITY : v + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Top-k of one token by a warp: lane l holds the logits of experts l and
// l + 32.  k rounds of a warp maximum (ties to the lower id), then the softmax
// over the chosen.
__device__ void select_topk(const Params& p, int t, float l0, float l1, int lane) {
  // 0 is below every logit: an expert that is taken or does not exist
  unsigned o0 = lane < p.E ? order_of(l0) : 0u, o1 = lane + 32 < p.E ? order_of(l1) : 0u;
  float top = 0.f, mine = 0.f, sum = 0.f;
  int chosen = 0;
  for (int j = 0; j < p.k; ++j) {
    const unsigned best = __reduce_max_sync(kFull, max(o0, o1));
    const unsigned m0 = __ballot_sync(kFull, o0 == best), m1 = __ballot_sync(kFull, o1 == best);
    const int be = m0 ? __ffs(m0) - 1 : 31 + __ffs(m1);
    if (be == lane) o0 = 0;
    if (be == lane + 32) o1 = 0;
    const float lv = __shfl_sync(kFull, be < 32 ? l0 : l1, be & 31);
    if (j == 0) top = lv;
    const float ev = expf(lv - top);
    sum += ev;
    if (lane == j) {
      chosen = be;
      mine = ev;
    }
  }
  if (lane < p.k) {
    p.idx[t * p.k + lane] = chosen;
    p.gates[t * p.k + lane] = mine / sum;
  }
}

// s[0] + s[stride] + ... (n of them): four chains in a fixed order.
__device__ __forceinline__ float add_up(const float* s, int n, int stride) {
  float v[4] = {};
  int i = 0;
#pragma unroll 2
  for (; i + 4 <= n; i += 4)
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] += s[(i + u) * stride];
  for (; i < n; ++i) v[0] += s[i * stride];
  return (v[0] + v[1]) + (v[2] + v[3]);
}

// A router unit is a group of tokens x a slice of h: fp32 partial logits.  All
// that a unit reads is asked for at once (the slice's rows of Wg are one
// contiguous piece); what this phase costs is latency, and loads in the loop's
// order took 14 us for one token and 25 us for 32 where this takes 4 to 5.
// The block that finishes a group's last slice adds the slices in a fixed order and
// chooses the experts of its tokens, one warp for each.
// False, in the whole block, where a wait ran out.
__device__ bool route(const Params& p, Ctrl& c, uint8_t* smem) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  unsigned* words = reinterpret_cast<unsigned*>(p.status);
  const int parts = kThreads / p.E;
  const int e = tid % p.E, part = tid / p.E;
  float* wg = reinterpret_cast<float*>(smem);                          // [nj][E]
  uint8_t* xs = smem + static_cast<size_t>(p.slice_h) * p.E * 4;       // [8][nj] bf16
  float* red = reinterpret_cast<float*>(smem + static_cast<size_t>(p.slice_h) *
                                                  (p.E * 4 + kGroupTok * 2));  // [8][kThreads]
  float* logit = red + kThreads * kGroupTok;                           // [8][kMaxE]
  const uint32_t bar = smem_u32(&c.rbar);
  uint32_t ph = 0;
  for (int unit = blockIdx.x; unit < p.groups * p.slices; unit += gridDim.x) {
    const int g = unit / p.slices, s = unit % p.slices;
    const int t0 = g * p.tok_group, nt = min(p.tok_group, p.T - t0);
    const int j0 = s * p.slice_h, nj = min(p.slice_h, p.h - j0);
    fence_proxy_async_all();
    __syncthreads();
    if (tid == 0) {
      mbar_expect_tx(bar, nj * (p.E * 4 + nt * 2));
      bulk_load(smem_u32(wg), p.Wg + static_cast<size_t>(j0) * p.E, nj * p.E * 4, bar);
      for (int t = 0; t < nt; ++t)
        bulk_load(smem_u32(xs) + t * nj * 2, p.x + static_cast<size_t>(t0 + t) * p.h + j0, nj * 2,
                  bar);
    }
    const bool got = mbar_wait(bar, ph, p.status, kTimeoutCode);
    float acc[kGroupTok] = {};
    if (got && part < parts)
      for (int j = part * 8; j < nj; j += parts * 8) {
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = wg[(j + i) * p.E + e];
#pragma unroll
        for (int t = 0; t < kGroupTok; ++t) {
          if (t >= nt) break;
          const uint4 q = *reinterpret_cast<const uint4*>(xs + (t * nj + j) * 2);
          acc[t] = fmaf(bf16_lo(q.x), w[0], acc[t]);
          acc[t] = fmaf(bf16_hi(q.x), w[1], acc[t]);
          acc[t] = fmaf(bf16_lo(q.y), w[2], acc[t]);
          acc[t] = fmaf(bf16_hi(q.y), w[3], acc[t]);
          acc[t] = fmaf(bf16_lo(q.z), w[4], acc[t]);
          acc[t] = fmaf(bf16_hi(q.z), w[5], acc[t]);
          acc[t] = fmaf(bf16_lo(q.w), w[6], acc[t]);
          acc[t] = fmaf(bf16_hi(q.w), w[7], acc[t]);
        }
      }
#pragma unroll
    for (int t = 0; t < kGroupTok; ++t)
      if (t < nt) red[t * kThreads + tid] = acc[t];
    if (!__syncthreads_and(got)) {  // the loads must land before the block ends
      if (tid == 0) mbar_wait(bar, ph, p.status, kTimeoutCode);
      return false;
    }
    ph ^= 1;
    // [group][slice][token][expert]
    const int pairs = p.tok_group * p.E;  // 512 at most
    float* mine = p.logits + static_cast<size_t>(unit) * pairs;
    for (int i = tid; i < nt * p.E; i += kThreads) {
      const int t = i / p.E;
      mine[i] = add_up(red + t * kThreads + i - t * p.E, parts, p.E);
    }
    __syncthreads();
    if (tid == 0) {
      unsigned n;
      asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;"
                   : "=r"(n)
                   : "l"(words + kGroupWord + g)
                   : "memory");
      c.flag = n + 1 == static_cast<unsigned>(p.slices);
      if (c.flag) words[kGroupWord + g] = 0;
    }
    __syncthreads();
    if (!c.flag) continue;
    // a thread adds up one pair's slices, or every few of them, straight from L2
    const float* all = p.logits + static_cast<size_t>(g) * p.slices * pairs;
    const int adders = kThreads / pairs, pair = tid % pairs;
    float v = 0.f;
    if (tid < adders * pairs)
#pragma unroll 8
      for (int q = tid / pairs; q < p.slices; q += adders)
        v += __ldcg(all + static_cast<size_t>(q) * pairs + pair);
    red[tid] = v;
    __syncthreads();
    if (tid < nt * p.E) {
      const int t = tid / p.E, ee = tid - t * p.E;
      const float sum = add_up(red + tid, adders, pairs);
      logit[t * kMaxE + ee] = p.b ? sum + __ldg(p.b + ee) : sum;
    }
    __syncthreads();
    if (warp < nt)
      select_topk(p, t0 + warp, lane < p.E ? logit[warp * kMaxE + lane] : 0.f,
                  lane + 32 < p.E ? logit[warp * kMaxE + lane + 32] : 0.f, lane);
  }
  return true;
}

// x rows to e4m3, a block for each row, from the last block on: with few tokens
// the router has no unit for it, and it must not hold up the router's.
template <bool QUOT>
__device__ void quant_x(const Params& p, float* red) {
  const int tid = threadIdx.x, n8 = p.h / 8;
  for (int t = gridDim.x - 1 - blockIdx.x; t < p.T; t += gridDim.x) {
    const uint4* row = reinterpret_cast<const uint4*>(p.x + static_cast<size_t>(t) * p.h);
    float m = 0.f;
    for (int c = tid; c < n8; c += kThreads) m = fmaxf(m, amax8(row[c]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    __syncthreads();
    if ((tid & 31) == 0) red[tid >> 5] = m;
    __syncthreads();
    for (int w = 0; w < kThreads / 32; ++w) m = fmaxf(m, red[w]);
    const float s = scale_of<QUOT>(m);
    if (tid == 0) p.sx[t] = s;
    uint2* out = reinterpret_cast<uint2*>(p.xq + static_cast<size_t>(t) * p.h);
    for (int c = tid; c < n8; c += kThreads) out[c] = quant8(row[c], s);
  }
}

// --------------------------------------------------------------- dispatch
// Every block builds the same lists from the chosen experts: the rows of each
// expert in ascending assignment order, at most `capacity` of them (and T: no
// token chooses an expert twice).  The ids come from memory: where the
// workspace's header was not zero they may be what an earlier call left there,
// so one out of range is recorded and not placed, and so is a row past T.
__device__ void dispatch(const Params& p, Ctrl& c, bool f8) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int R = p.T * p.k, chunks = (R + 31) / 32;
  constexpr int kMine = kMaxRows / kThreads;
  int rank[kMine], mine[kMine];  // my assignments' rank within their chunk of 32, expert
  float gate[kMine], sx = 0.f;
#pragma unroll
  for (int n = 0; n < kMine; ++n) {  // all loads at once
    const int a = (warp + n * (kThreads / 32)) * 32 + lane;
    mine[n] = a < R ? __ldcg(p.idx + a) : -1;
    gate[n] = a < R ? __ldcg(p.gates + a) : 0.f;
  }
#pragma unroll
  for (int n = 0; n < kMine; ++n)
    if (static_cast<unsigned>(mine[n]) >= static_cast<unsigned>(p.E)) mine[n] = -1;
  if (f8 && tid < p.T) sx = __ldcg(p.sx + tid);
  for (int i = tid; i < chunks * kMaxE; i += kThreads) c.hist[i / kMaxE][i % kMaxE] = 0;
  if (f8 && tid < p.T) c.sx[tid] = sx;
  __syncthreads();
#pragma unroll
  for (int n = 0; n < kMine; ++n) {
    const int ch = warp + n * (kThreads / 32), a = ch * 32 + lane, e = mine[n];
    if (ch >= chunks) break;
    if (e >= 0) {
      c.gate[a] = gate[n];
      c.exp[a] = static_cast<uint8_t>(e);
    }
    const unsigned same = __match_any_sync(kFull, e);
    rank[n] = __popc(same & ((1u << lane) - 1));
    if (e >= 0 && rank[n] == 0) c.hist[ch][e] = static_cast<uint16_t>(__popc(same));
  }
  __syncthreads();
  if (tid < kMaxE) {  // hist: counts -> assignments of the expert before the chunk
    int n = 0;
    for (int ch = 0; ch < chunks; ++ch) {
      const int v = c.hist[ch][tid];
      c.hist[ch][tid] = static_cast<uint16_t>(n);
      n += v;
    }
    c.act_of[tid] = min(n, p.capacity);
  }
  __syncthreads();
  if (warp == 0) {  // offsets and the list of experts with rows
    const int n0 = c.act_of[lane], n1 = c.act_of[lane + 32];
    int s0 = n0, s1 = n1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u0 = __shfl_up_sync(kFull, s0, o), u1 = __shfl_up_sync(kFull, s1, o);
      if (lane >= o) {
        s0 += u0;
        s1 += u1;
      }
    }
    const int all0 = __shfl_sync(kFull, s0, 31);
    if (lane == 0) c.off[0] = 0;
    c.off[lane + 1] = s0;
    c.off[lane + 33] = all0 + s1;
    const unsigned m0 = __ballot_sync(kFull, n0 > 0), m1 = __ballot_sync(kFull, n1 > 0);
    const unsigned below = (1u << lane) - 1;
    const int i0 = __popc(m0 & below), i1 = __popc(m0) + __popc(m1 & below);
    __syncwarp();
    if (n0 > 0) c.act[i0] = lane;
    if (n1 > 0) c.act[i1] = lane + 32;
    c.act_of[lane] = i0;
    c.act_of[lane + 32] = i1;
    const int most = __reduce_max_sync(kFull, max(n0, n1));
    if (lane == 0) {
      c.nact = __popc(m0) + __popc(m1);
      c.most = most;
    }
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < kMine; ++n) {
    const int ch = warp + n * (kThreads / 32), a = ch * 32 + lane, e = mine[n];
    if (a >= R) break;
    const int r = e < 0 ? p.T : c.hist[ch][e] + rank[n];
    if (r >= p.T) report_bad_index(p.status);
    const bool placed = r < p.capacity;
    const int row = placed ? c.off[e] + r : -1;
    c.pos[a] = static_cast<int16_t>(row);
    if (placed) c.tok[row] = static_cast<uint8_t>(a / p.k);
  }
  __syncthreads();
}

// ------------------------------------------------------------- FC1's ends
__device__ __forceinline__ float4 add4(const float4& a, const float4& b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

// The low parts of two values with the high parts hi (0 where those are not finite).
__device__ __forceinline__ uint32_t low_parts(float a, float b, uint32_t hi) {
  const float ha = bf16_lo(hi), hb = bf16_hi(hi);
  const __nv_bfloat162 v = __floats2bfloat162_rn(fabsf(ha) < INFINITY ? a - ha : 0.f,
                                                 fabsf(hb) < INFINITY ? b - hb : 0.f);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// H of a row's column from its two sums.  With bf16 weights it enters FC2 as two
// bf16 operands, its rounded value and what that leaves: 16 bits, where one
// bf16 made y's error 1.4 times that of y's own rounding (0.0024 against
// 0.0017).  They are more columns of an idle tensor pipe and no more weights.
// n of eight rows side by side: one after another, with the second part's
// stores, 128 skewed tokens over 64 experts of 512 x 8192 took 468 us, so 389.
__device__ __forceinline__ void store_h8(const Params& p, int row, int n, int col,
                                         const uint32_t (&a)[8], const uint32_t (&b)[8]) {
  if (col >= p.f) return;
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = __uint_as_float(a[i]);
    v[i] = x / (1.f + expf(-x)) * __uint_as_float(b[i]);
  }
  uint16_t* at = p.H + static_cast<size_t>(row) * p.f + col;
  uint16_t* low = at + static_cast<size_t>(p.T) * p.k * p.f;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[i], v[i + 1]);
    const uint32_t hi = *reinterpret_cast<const uint32_t*>(&h);
    const uint32_t lo = low_parts(v[i], v[i + 1], hi);
    if (i < n) {
      at[i * p.f] = static_cast<uint16_t>(hi);
      low[i * p.f] = static_cast<uint16_t>(lo);
    }
    if (i + 1 < n) {
      at[(i + 1) * p.f] = static_cast<uint16_t>(hi >> 16);
      low[(i + 1) * p.f] = static_cast<uint16_t>(lo >> 16);
    }
  }
}

// The same of one row with e4m3 weights: H's bf16 value is what its codes are
// made from.
__device__ __forceinline__ void store_h(const Params& p, const Ctrl& c, int row, int col, float a,
                                        float b, float w1, float w3, int lane) {
  float m = 0.f;
  if (col < p.f) {
    const float s = c.sx[c.tok[row]];
    a *= s * w1;
    b *= s * w3;
    const __nv_bfloat16 hv = __float2bfloat16_rn(a / (1.f + expf(-a)) * b);
    p.H[static_cast<size_t>(row) * p.f + col] = *reinterpret_cast<const uint16_t*>(&hv);
    m = fabsf(__bfloat162float(hv));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
  if (lane == 0) atomicMax(p.amax + row, __float_as_uint(m));
}

// H of a row's four columns (f is a multiple of 64: all in range or none).
template <bool F8>
__device__ __forceinline__ void store_h4(const Params& p, const Ctrl& c, int row, int col, float4 a,
                                         float4 b, float4 w1, float4 w3, int lane) {
  float m = 0.f;
  if (col < p.f) {
    if (F8) {
      const float s = c.sx[c.tok[row]];
      a = make_float4(a.x * (s * w1.x), a.y * (s * w1.y), a.z * (s * w1.z), a.w * (s * w1.w));
      b = make_float4(b.x * (s * w3.x), b.y * (s * w3.y), b.z * (s * w3.z), b.w * (s * w3.w));
    }
    const float4 v = make_float4(a.x / (1.f + expf(-a.x)) * b.x, a.y / (1.f + expf(-a.y)) * b.y,
                                 a.z / (1.f + expf(-a.z)) * b.z, a.w / (1.f + expf(-a.w)) * b.w);
    const __nv_bfloat162 xy = __floats2bfloat162_rn(v.x, v.y), zw = __floats2bfloat162_rn(v.z, v.w);
    uint2 out;
    out.x = *reinterpret_cast<const uint32_t*>(&xy);
    out.y = *reinterpret_cast<const uint32_t*>(&zw);
    uint16_t* at = p.H + static_cast<size_t>(row) * p.f + col;
    *reinterpret_cast<uint2*>(at) = out;
    if (!F8)
      *reinterpret_cast<uint2*>(at + static_cast<size_t>(p.T) * p.k * p.f) =
          make_uint2(low_parts(v.x, v.y, out.x), low_parts(v.z, v.w, out.y));
    m = fmaxf(fmaxf(fabsf(bf16_lo(out.x)), fabsf(bf16_hi(out.x))),
              fmaxf(fabsf(bf16_lo(out.y)), fabsf(bf16_hi(out.y))));
  }
  if (F8) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    if (lane == 0) atomicMax(p.amax + row, __float_as_uint(m));
  }
}

// y: 64 columns of a token to a warp, four to a lane, each half of the warp
// with every second sum.  This is latency: lane j of the first 8 looks up slot
// j's row and the pieces that its tile went through (divisions for each slot in
// every thread cost 4 us; the idle warps make a table of them during FC2), then
// eight chains of loads run side by side, LANES of them for each of up to
// 8 / LANES slots, with the slot's row of O and the parts that other pieces left
// of it dealt out to them and the halves in turn.
struct Look {
  int row, n;      // the slot's row; how many further parts
  unsigned at;     // the row's place in the first piece's part
  float gate;
};
__device__ __forceinline__ Look look_of(const Params& p, const Ctrl& c, const Cut& cut,
                                        unsigned tiles, unsigned ksn, int t, int b, int lane) {
  Look l = {-1, 0, 0, 0.f};
  if (lane < p.k) {
    const int a = t * p.k + lane;
    l.row = c.pos[a];
    if (l.row >= 0) {
      l.gate = c.gate[a];
      const int e = c.exp[a];
      const unsigned i = c.act_of[e] * tiles + b / 4;
      unsigned first, n;
      if (i < kMaxTiles) {
        first = c.tile[i] & 0xFFFFu;
        n = c.tile[i] >> 16;
      } else {
        first = cut.piece_of(i * ksn);
        n = cut.piece_of(i * ksn + ksn - 1) - first;
      }
      l.n = n;
      l.at = first * p.T + l.row - c.off[e];
    }
  }
  return l;
}
template <int LANES>
__device__ __forceinline__ void combine(const Params& p, const Look& l, int t, int b, int lane) {
  constexpr int kStep = 2 * LANES;
  const int half = lane >> 4, col = b * 64 + (lane & 15) * 4;
  const size_t stride = static_cast<size_t>(kStep) * p.T * 64;  // float4s
  float4 v[8];
  const float4* src[8];
  int left[8];
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    const int j = w / LANES, u = (w % LANES) * 2 + half;  // u: the first sum of this chain
    const int row = __shfl_sync(kFull, l.row, j), n = __shfl_sync(kFull, l.n, j);
    const unsigned at = __shfl_sync(kFull, l.at, j);
    v[w] = make_float4(0.f, 0.f, 0.f, 0.f);
    left[w] = row >= 0 && n >= u ? (n - u) / kStep + 1 : 0;
    src[w] = reinterpret_cast<const float4*>(p.part) +
             (static_cast<size_t>(at + u * p.T) * 64 + (col & 255) / 4);
    if (u == 0 && row >= 0) {
      v[w] = __ldcg(reinterpret_cast<const float4*>(p.O + static_cast<size_t>(row) * p.h + col));
      src[w] += stride;
      --left[w];
    }
  }
  for (bool any = true; any;) {
    any = false;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      if (left[w] == 0) continue;
      any = true;
      v[w] = add4(v[w], __ldcg(src[w]));
      src[w] += stride;
      --left[w];
    }
  }
  __syncwarp();
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int j = 0; j < 8 / LANES; ++j) {
    float4 o = v[j * LANES];
#pragma unroll
    for (int u = 1; u < LANES; ++u) o = add4(o, v[j * LANES + u]);
    const float g = __shfl_sync(kFull, l.gate, j);
    if (__shfl_sync(kFull, l.row, j) < 0) continue;
    sum.x = fmaf(g, o.x, sum.x);
    sum.y = fmaf(g, o.y, sum.y);
    sum.z = fmaf(g, o.z, sum.z);
    sum.w = fmaf(g, o.w, sum.w);
  }
  sum.x += __shfl_xor_sync(kFull, sum.x, 16);
  sum.y += __shfl_xor_sync(kFull, sum.y, 16);
  sum.z += __shfl_xor_sync(kFull, sum.z, 16);
  sum.w += __shfl_xor_sync(kFull, sum.w, 16);
  if (half) return;
  const __nv_bfloat162 lo = __floats2bfloat162_rn(sum.x, sum.y);
  const __nv_bfloat162 hi = __floats2bfloat162_rn(sum.z, sum.w);
  uint2 out;
  out.x = *reinterpret_cast<const uint32_t*>(&lo);
  out.y = *reinterpret_cast<const uint32_t*>(&hi);
  *reinterpret_cast<uint2*>(p.y + static_cast<size_t>(t) * p.h + col) = out;
}

// Two rows of a tile of FC1 that pieces share: at src, what the piece that began
// it left, then the parts of the pieces after it, in order.
template <bool F8>
__device__ __forceinline__ void join_rows(const Params& p, const Ctrl& c, const float4* src,
                                          unsigned parts, int e, int row, int rows, int col,
                                          int lane) {
  const size_t slot = static_cast<size_t>(p.T) * 64;  // float4s
  const unsigned odd = rows > 1 ? 64 : 0;
  float4 va = __ldcg(src), vb = __ldcg(src + 32);
  float4 ua = __ldcg(src + odd), ub = __ldcg(src + odd + 32);
  src += slot;
#pragma unroll 4
  for (unsigned o = 0; o < parts; ++o, src += 2 * slot) {
    va = add4(va, __ldcg(src));
    vb = add4(vb, __ldcg(src + 32));
    ua = add4(ua, __ldcg(src + odd));
    ub = add4(ub, __ldcg(src + odd + 32));
  }
  float4 w1 = make_float4(0.f, 0.f, 0.f, 0.f), w3 = w1;
  if (F8) {
    w1 = __ldg(reinterpret_cast<const float4*>(p.s1 + static_cast<size_t>(e) * p.f + col));
    w3 = __ldg(reinterpret_cast<const float4*>(p.s3 + static_cast<size_t>(e) * p.f + col));
  }
  store_h4<F8>(p, c, row, col, va, vb, w1, w3, lane);
  if (odd) store_h4<F8>(p, c, row + 1, col, ua, ub, w1, w3, lane);
}

// QUOT: the e4m3 scales of moe_layer_decode_fp8_as_fwd.  A variant of its own: with a
// choice at run time one token took 78.5 us in place of 78.0, 24 tokens 106.4 for 105.5.
template <bool F8, bool QUOT>
__global__ void __launch_bounds__(kThreads, 1)
    decode_kernel(const __grid_constant__ Params p, const __grid_constant__ Maps maps) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  constexpr int kParts = F8 ? 1 : 2;  // FC2's operands of tokens (see store_h)
  Ctrl& c = *reinterpret_cast<Ctrl*>(smem + p.ring_bytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const unsigned G = gridDim.x;
  unsigned* words = reinterpret_cast<unsigned*>(p.status);
  volatile int* abort_flag = &c.abort;

  if (tid == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(smem_u32(&c.full[s]), 1);
      mbar_init(smem_u32(&c.empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&c.tfull[b]), 1);
      mbar_init(smem_u32(&c.tempty[b]), 128);
    }
    mbar_init(smem_u32(&c.hready), 1);
    mbar_init(smem_u32(&c.drain), 1);
    mbar_init(smem_u32(&c.rbar), 1);
    for (int i = 0; i < kQueue; ++i) {
      mbar_init(smem_u32(&c.qfull[i]), 1);
      mbar_init(smem_u32(&c.qempty[i]), 5);  // the MMA warp and four epilogue warps
    }
    c.abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&maps.x);
    tma_prefetch_desc(&maps.w1);
    tma_prefetch_desc(&maps.w3);
    tma_prefetch_desc(&maps.h);
    tma_prefetch_desc(&maps.w2);
    if (blockIdx.x == 0) p.claim[0] = p.claim[1] = 0;
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&c.tmem_base), 512);
    tmem_relinquish();
    tc_fence_before();
  }
  // ------------------------------------------------------------- route
  if (F8)
    for (int i = blockIdx.x * kThreads + tid; i < p.T * p.k; i += G * kThreads) p.amax[i] = 0;
  const bool routed = route(p, c, smem);
  if (F8 && routed) quant_x<QUOT>(p, reinterpret_cast<float*>(smem));
  fence_proxy_async_all();  // xq for TMA; and the ring's memory, used by route above
  __syncthreads();
  // (a block that gave up does not arrive: the others give up here too)
  if (tid == 0 && !(routed && grid_barrier(words + kBarWord, G, p.status))) c.abort = 1;
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem_base;
  if (!c.abort) {
    dispatch(p, c, F8);
    fence_proxy_async_all();

    constexpr int KB = F8 ? 128 : 64;  // contraction indices of a stage
    const unsigned ks1 = p.h / KB, nt1 = (p.f + 127) / 128;
    const unsigned ks2 = p.f / KB, nt2 = (p.h + 255) / 256;
    const Cut cut1(c.nact * nt1 * ks1, G, ks1), cut2(c.nact * nt2 * ks2, G, ks2);
    const unsigned cta = blockIdx.x;
    // A stage holds FC1's n1 rows of x, or all parts of the busiest expert's rows of
    // H: 128 tokens over 8 experts have 4 stages so, where room for both parts of
    // 128 rows would leave 3 (456 and 465 us).
    const uint32_t ring = smem_u32(smem);
    const int stage_bytes = kWBytes + max(p.n1, kParts * ((c.most + 15) / 16 * 16)) * 128;
    const int stages = min(kMaxStages, p.ring_bytes / stage_bytes);

    if (warp == 0) {
      // ---------------------------------------------------- TMA producer
      if (lane == 0) {
        int s = 0;        // next stage
        uint32_t ph = 0;  // its use count's parity
        int filled = 0;
        int published = 0;
        bool ok = true;
        auto claim = [&](unsigned bytes) {
          if (*abort_flag ||
              !mbar_wait(smem_u32(&c.empty[s]), ph ^ 1, p.status, kTimeoutCode)) {
            *abort_flag = 1;
            ok = false;
            return;
          }
          mbar_expect_tx(smem_u32(&c.full[s]), bytes);
          if (filled < stages) ++filled;
        };
        auto next = [&] {
          if (++s == stages) {
            s = 0;
            ph ^= 1;
          }
        };
        auto publish = [&](int piece) {
          const int i = published % kQueue;
          if (!ok || *abort_flag ||
              !mbar_wait(smem_u32(&c.qempty[i]), ((published / kQueue) & 1) ^ 1, p.status,
                         kTimeoutCode)) {
            *abort_flag = 1;
            ok = false;
            return;
          }
          c.piece[i] = piece;
          mbar_arrive(smem_u32(&c.qfull[i]));
          ++published;
        };
        // the block's next piece of a phase, -1 when there is none
        auto more = [&](const Cut& cut, unsigned* taken) {
          if (cut.rounds == 1) return -1;
          const unsigned i = cut.blocks + atomicAdd(taken, 1u);
          return i < cut.rounds * cut.blocks ? static_cast<int>(i) : -1;
        };
        unsigned ks, ai, tile;  // where the weights' loads are
        auto seek = [&](unsigned q, unsigned ksn, unsigned tiles) {
          const unsigned item = q / ksn;
          ks = q - item * ksn;
          ai = item / tiles;
          tile = item - ai * tiles;
        };
        auto step = [&](unsigned ksn, unsigned tiles) {
          if (++ks < ksn) return;
          ks = 0;
          if (++tile < tiles) return;
          tile = 0;
          ++ai;
        };
        int piece = cta < cut1.blocks ? static_cast<int>(cta) : -1;
        for (; ok && piece >= 0; piece = more(cut1, p.claim)) {
          publish(piece);
          const unsigned q1 = cut1.end(piece);
          unsigned q = cut1.start(piece);
          seek(q, ks1, nt1);
          for (; ok && q < q1; ++q) {
            claim(kWBytes + p.n1 * 128);
            if (!ok) break;
            const uint32_t dst = ring + s * stage_bytes, bar = smem_u32(&c.full[s]);
            const int e = c.act[ai], k0 = ks * KB;
            if (F8) {
              tma_load_3d(dst, &maps.w1, k0, tile * 256, e, bar);
            } else {
              tma_load_3d(dst, &maps.w1, 0, e * p.h + k0, tile * 2, bar);
              tma_load_3d(dst + kWBytes / 2, &maps.w3, 0, e * p.h + k0, tile * 2, bar);
            }
            tma_load_2d(dst + kWBytes, &maps.x, k0, 0, bar);
            next();
            step(ks1, nt1);
          }
        }
        publish(-1);
        // FC2.  The first stages' weights are asked for at once; their rows of H
        // follow when every block's are written.
        unsigned hks = 0, hai = 0, htile = 0;  // where the H loads are
        int hs = s;
        auto load_h = [&] {
          const int e = c.act[hai], r0 = c.off[e], n = c.off[e + 1] - r0;
          const int low = (n + 15) / 16 * 16 * 128;  // the low parts follow
          const uint32_t dst = ring + hs * stage_bytes + kWBytes, bar = smem_u32(&c.full[hs]);
          for (int r = 0; r < n; r += 16) {
            tma_load_2d(dst + r * 128, &maps.h, hks * KB, r0 + r, bar);
            if (!F8) tma_load_2d(dst + low + r * 128, &maps.h, hks * KB, p.T * p.k + r0 + r, bar);
          }
          if (++hs == stages) hs = 0;
          if (++hks < ks2) return;
          hks = 0;
          if (++htile < nt2) return;
          htile = 0;
          ++hai;
        };
        unsigned waiting = 0;  // stages whose H is not yet asked for
        bool ready = false;
        piece = cta < cut2.blocks ? static_cast<int>(cta) : -1;
        for (; ok && piece >= 0; piece = more(cut2, p.claim + 1)) {
          publish(piece);
          const unsigned q0 = cut2.start(piece), q1 = cut2.end(piece);
          const unsigned ahead = min(q1 - q0, static_cast<unsigned>(stages));
          seek(q0, ks2, nt2);
          hks = ks;
          hai = ai;
          htile = tile;
          for (unsigned q = q0; ok && q < q1; ++q) {
            const int e = c.act[ai];
            const int rows16 = (c.off[e + 1] - c.off[e] + 15) / 16 * 16;
            claim(kWBytes + kParts * rows16 * 128);
            if (!ok) break;
            const uint32_t dst = ring + s * stage_bytes, bar = smem_u32(&c.full[s]);
            if (F8)
              tma_load_3d(dst, &maps.w2, ks * KB, tile * 256, e, bar);
            else
              tma_load_3d(dst, &maps.w2, 0, e * p.f + ks * KB, tile * 4, bar);
            ++waiting;
            next();
            step(ks2, nt2);
            if (!ready && q + 1 - q0 < ahead) continue;
            if (!ready) {
              if (!mbar_wait(smem_u32(&c.hready), 0, p.status, kTimeoutCode)) {
                *abort_flag = 1;
                ok = false;
              }
              ready = true;
              fence_proxy_async_all();
            }
            // on failure too: the stages' loads must all land before the block ends
            for (; waiting > 0; --waiting) load_h();
          }
        }
        publish(-1);
        if (!ok) {
          for (; waiting > 0; --waiting) load_h();
          for (int i = 0; i < filled; ++i) {
            s = s == 0 ? stages - 1 : s - 1;
            if (s == stages - 1) ph ^= 1;
            mbar_wait(smem_u32(&c.full[s]), ph, p.status, kTimeoutCode);
          }
        }
      }
    } else if (warp == 1) {
      // ------------------------------------------------------ MMA issuer
      int s = 0, it = 0;
      uint32_t ph = 0;
      bool ok = true;
      int popped = 0;
      auto pop = [&] {
        const int i = popped % kQueue;
        if (*abort_flag || !mbar_wait(smem_u32(&c.qfull[i]), (popped / kQueue) & 1, p.status,
                                      kTimeoutCode)) {
          *abort_flag = 1;
          ok = false;
        }
        const int v = c.piece[i];
        __syncwarp();
        ++popped;
        if (lane == 0) mbar_arrive(smem_u32(&c.qempty[i]));
        ok = __all_sync(kFull, ok);
        return ok ? v : -1;
      };
      // All that a k-step needs is worked out by the whole warp, and only the
      // instructions are issued by one thread: the eight MMAs take the
      // descriptors from uniform registers, which code under `lane == 0` has to
      // fill one by one.  That and the look-ups for each step took 0.77 us, more
      // than the 0.7 us in which a step's 32 KiB arrive.
      constexpr uint32_t kA = F8 ? 2 : 128;  // 16-byte units from one MMA's A to the next
      const uint64_t a_ring = smem_desc(0, F8 ? 16 : 8192, 1024) + (ring >> 4);
      const uint64_t b_ring = smem_desc(0, 16, 1024) + ((ring + kWBytes) >> 4);
      const uint32_t stage16 = stage_bytes >> 4;
      auto phase = [&](unsigned q0, unsigned q1, unsigned ksn, unsigned tiles, bool fc1) {
        unsigned item = q0 / ksn;
        for (unsigned q = q0; q < q1; ++item) {
          const unsigned end = min(q1, (item + 1) * ksn);
          int n = p.n1;
          if (!fc1) {
            const int e = c.act[item / tiles];
            n = (c.off[e + 1] - c.off[e] + 15) / 16 * 16;
          }
          const uint32_t idesc = F8 ? idesc_e4m3(128, n) : idesc_bf16(128, n, true, false);
          const int buf = it & 1;
          const uint32_t acc = tmem + buf * 256;
          ok = !*abort_flag && mbar_wait(smem_u32(&c.tempty[buf]), ((it >> 1) & 1) ^ 1, p.status,
                                         kTimeoutCode);
          uint32_t add = 0;
          for (; q < end; ++q) {
            // the whole warp goes on or stops
            ok = __all_sync(kFull, ok && mbar_wait(smem_u32(&c.full[s]), ph, p.status,
                                                   kTimeoutCode));
            if (!ok) {
              *abort_flag = 1;
              return;
            }
            tc_fence_after();
            const uint64_t ad = a_ring + s * stage16, bd = b_ring + s * stage16;
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                  const uint64_t am = ad + kk * kA + m * (kWBytes / 32);
                  if (F8)
                    umma_e4m3(acc + m * 128, am, bd + kk * 2, idesc, kk ? 1u : add);
                  else
                    umma_bf16(acc + m * 128, am, bd + kk * 2, idesc, kk ? 1u : add);
                  if (!F8 && !fc1)
                    umma_bf16(acc + m * 128, am, bd + n * 8 + kk * 2, idesc, 1u);
                }
              }
              umma_commit(smem_u32(&c.empty[s]));
              if (q + 1 == end) umma_commit(smem_u32(&c.tfull[buf]));
            }
            add = 1;
            if (++s == stages) {
              s = 0;
              ph ^= 1;
            }
          }
          ++it;
        }
      };
      for (int i; (i = pop()) >= 0 && ok;) phase(cut1.start(i), cut1.end(i), ks1, nt1, true);
      if (ok)
        for (int i; (i = pop()) >= 0 && ok;) phase(cut2.start(i), cut2.end(i), ks2, nt2, false);
      // every MMA must be done before tensor memory is freed
      if (elect_one()) umma_commit(smem_u32(&c.drain));
      mbar_wait(smem_u32(&c.drain), 0, p.status, kTimeoutCode);
      __syncwarp();
    } else {
      // ------------------------------------------- epilogue and helpers
      const bool epilogue = warp >= 4 && warp < 8;
      const int idle = warp < 4 ? warp - 2 : warp - 6;  // 0 .. kIdleWarps - 1
      const int r = (warp & 3) * 32 + lane;  // my row of the 128-row tiles
      const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
      int it = 0;
      bool ok = true;
      auto filled = [&](int buf) {
        const bool got = !*abort_flag && mbar_wait(smem_u32(&c.tfull[buf]), (it >> 1) & 1,
                                                   p.status, kTimeoutCode);
        if (!__all_sync(kFull, got)) {
          *abort_flag = 1;
          ok = false;
        }
        tc_fence_after();
        return ok;
      };
      int popped = 0;
      unsigned q = 0, q_end = 0;
      int piece = -1;
      auto pop = [&](const Cut& cut) {  // the next piece's range, false at the phase's end
        const int i = popped % kQueue;
        const bool got = !*abort_flag && mbar_wait(smem_u32(&c.qfull[i]), (popped / kQueue) & 1,
                                                   p.status, kTimeoutCode);
        piece = c.piece[i];
        ++popped;
        if (!__all_sync(kFull, got)) {
          *abort_flag = 1;
          ok = false;
          return false;
        }
        if (lane == 0) mbar_arrive(smem_u32(&c.qempty[i]));
        if (piece < 0) return false;
        q = cut.start(piece);
        q_end = cut.end(piece);
        return true;
      };
      // ---- FC1
      while (epilogue && ok && (q < q_end || pop(cut1))) {
        const unsigned item = q / ks1, q_item = item * ks1;
        const unsigned end = min(q_end, q_item + ks1);
        const int buf = it & 1;
        if (!filled(buf)) break;
        const int e = c.act[item / nt1], col = (item % nt1) * 128 + r;
        const int row0 = c.off[e], n = c.off[e + 1] - row0;
        const uint32_t acc = tl + buf * 256;
        const bool whole = q == q_item && end == q_item + ks1;
        float w1 = 0.f, w3 = 0.f;
        if (F8 && col < p.f) {
          w1 = __ldg(p.s1 + static_cast<size_t>(e) * p.f + col);
          w3 = __ldg(p.s3 + static_cast<size_t>(e) * p.f + col);
        }
        // two slots for each piece: a tile begun before it, a tile begun in it
        const size_t slot = static_cast<size_t>(2) * p.T * 128;
        float* mine = p.part + (2 * piece + (q == q_item)) * slot;
        for (int i0 = 0; i0 < n; i0 += 8) {
          uint32_t ra[8], rb[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t t = c.tok[row0 + min(i0 + i, n - 1)];
            tmem_ld1(acc + t, ra[i]);
            tmem_ld1(acc + 128 + t, rb[i]);
          }
          tmem_wait8(ra, rb);
          if (!F8 && whole) {
            store_h8(p, row0 + i0, n - i0, col, ra, rb);
            continue;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (i0 + i >= n) break;
            const float va = __uint_as_float(ra[i]), vb = __uint_as_float(rb[i]);
            if (whole) {
              store_h(p, c, row0 + i0 + i, col, va, vb, w1, w3, lane);
            } else {
              __stcg(mine + (i0 + i) * 256 + r, va);
              __stcg(mine + (i0 + i) * 256 + 128 + r, vb);
            }
          }
        }
        tc_fence_before();
        mbar_arrive(smem_u32(&c.tempty[buf]));
        ++it;
        q = end;
      }
      // The tiles of FC1 that pieces share, listed by an idle warp (in the same
      // order in every block): a tile goes with the first border inside it.
      if (warp == 2) {
        const unsigned pieces = cut1.rounds * cut1.blocks;
        int listed = 0;
        for (unsigned i0 = 0; i0 < pieces; i0 += 32) {
          const unsigned i = i0 + lane;
          unsigned parts = 0, item = 0;
          if (i > 0 && i < pieces) {
            const unsigned begin = cut1.start(i);
            item = begin / ks1;
            if (begin != item * ks1 && cut1.piece_of(item * ks1) == i - 1)
              parts = cut1.piece_of(item * ks1 + ks1 - 1) - i + 1;
          }
          const unsigned some = __ballot_sync(kFull, parts > 0);
          if (parts > 0)
            c.join[listed + __popc(some & ((1u << lane) - 1))] =
                make_uint2(i | parts << 16, (item / nt1) << 16 | item % nt1);
          listed += __popc(some);
        }
        if (lane == 0) c.joins = listed;
      }
      // A grid barrier of these warps.  Whether to go on is one thread's reading,
      // so that all of them do the same even while another warp gives up.
      unsigned arrived = G;
      auto grid_sync = [&] {
        fence_proxy_async_all();
        helper_sync();
        arrived += G;
        if (tid == 64) {
          if (!grid_barrier(words + kBarWord, arrived, p.status)) *abort_flag = 1;
          c.go = !*abort_flag;
        }
        helper_sync();
        return c.go != 0;
      };
      bool go = grid_sync();
      if (go) {  // two rows to a warp, four columns to a lane
        const unsigned pairs = (c.most + 1) / 2, works = c.joins * pairs;
        for (unsigned w = cta + (warp - 2) * G; w < works; w += G * (kHelpers / 32)) {
          const unsigned at = w / pairs, i0 = (w - at * pairs) * 2;
          const uint2 j = c.join[at];
          const unsigned i = j.x & 0xFFFFu, parts = j.x >> 16;
          const int e = c.act[j.y >> 16], row = c.off[e] + i0, rows = c.off[e + 1] - row;
          if (rows > 0)
            join_rows<F8>(p, c,
                          reinterpret_cast<const float4*>(
                              p.part + (2 * i - 1) * (static_cast<size_t>(2) * p.T * 128) +
                              i0 * 256) + lane,
                          parts, e, row, rows, (j.y & 0xFFFFu) * 128 + lane * 4, lane);
        }
      }
      go = grid_sync();
      if (F8 && go) {  // rows of H to e4m3, 8 values at a time over the whole grid
        const int n8 = p.f / 8, all = c.off[kMaxE] * n8;
        for (int i = cta * kHelpers + tid - 64; i < all; i += G * kHelpers) {
          const int row = i / n8;
          const float s = scale_of<QUOT>(__uint_as_float(__ldcg(p.amax + row)));
          const uint4 w = __ldcg(reinterpret_cast<const uint4*>(p.H) + i);
          reinterpret_cast<uint2*>(p.Hq)[i] = quant8(w, s);
        }
        go = grid_sync();
      }
      fence_proxy_async_all();
      if (tid == 64) mbar_arrive(smem_u32(&c.hready));
      ok = ok && go;
      if (!epilogue) {  // for the combine: the pieces that each tile goes through
        const unsigned tiles = min(c.nact * nt2, static_cast<unsigned>(kMaxTiles));
        for (unsigned i = idle * 32 + lane; i < tiles; i += kIdleWarps * 32) {
          const unsigned first = cut2.piece_of(i * ks2);
          c.tile[i] = first | (cut2.piece_of(i * ks2 + ks2 - 1) - first) << 16;
        }
      }
      // ---- FC2: rows of O where this piece begins the tile, else of its part
      q = q_end = 0;
      while (epilogue && ok && (q < q_end || pop(cut2))) {
        const unsigned item = q / ks2, q_item = item * ks2;
        const unsigned end = min(q_end, q_item + ks2);
        const int buf = it & 1;
        if (!filled(buf)) break;
        const int e = c.act[item / nt2], col0 = (item % nt2) * 256;
        const int row0 = c.off[e], n = c.off[e + 1] - row0;
        const bool begun = q == q_item;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const int col = col0 + m * 128 + r;
          float w2 = 1.f;
          if (F8 && col < p.h) w2 = __ldg(p.s2 + static_cast<size_t>(e) * p.h + col);
          float* dst = begun ? p.O + static_cast<size_t>(row0) * p.h + col
                             : p.part + static_cast<size_t>(piece) * p.T * 256 + m * 128 + r;
          const size_t ld = begun ? p.h : 256;
          for (int i0 = 0; i0 < n; i0 += 16) {
            float v[16];
            tmem_ld16(tl + buf * 256 + m * 128 + i0, v);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              if (i0 + i >= n || col >= p.h) break;
              if (F8) v[i] *= scale_of<QUOT>(__uint_as_float(__ldcg(p.amax + row0 + i0 + i))) * w2;
              __stcg(dst + (i0 + i) * ld, v[i]);
            }
          }
        }
        tc_fence_before();
        mbar_arrive(smem_u32(&c.tempty[buf]));
        ++it;
        q = end;
      }
    }
    // ------------------------------------------------------------ combine
    __syncthreads();
    if (tid == 0 && (*abort_flag ||
                     !grid_barrier(words + kBarWord, (F8 ? 5 : 4) * G, p.status)))
      *abort_flag = 1;
    __syncthreads();
    if (!*abort_flag) {
      const int blocks = p.h / 64, tasks = p.T * blocks;
      for (int i = cta + warp * G; i < tasks; i += G * (kThreads / 32)) {
        const int t = i / blocks, b = i - t * blocks;
        const Look look = look_of(p, c, cut2, nt2, ks2, t, b, lane);
        if (p.k <= 2)
          combine<4>(p, look, t, b, lane);
        else if (p.k <= 4)
          combine<2>(p, look, t, b, lane);
        else
          combine<1>(p, look, t, b, lane);
      }
    }
  }
  // ------------------------------------------------------------- teardown
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  // the last block to finish leaves the header's words zero for the next call
  if (tid == 0 && atomicAdd(words + kExitWord, 1u) == G - 1) {
    words[kBarWord] = 0;
    words[kExitWord] = 0;
    for (int g = 0; g < 16; ++g) words[kGroupWord + g] = 0;
    __threadfence();
  }
}

// ------------------------------------------------------------------- host
size_t up256(size_t n) { return (n + 255) / 256 * 256; }

struct Layout {
  size_t logits, idx, gates, H, O, part, claim, xq, sx, Hq, amax, total;
};

struct Plan {
  int n1, ring, smem;
  int tok_group, groups, slices, slice_h;
  size_t pieces;
};

// The most k-steps that a phase can have, with every expert that can be hit.
long long most_steps(const moe_dims& d, bool fp8) {
  const long long kb = fp8 ? 128 : 64;
  const long long e = static_cast<long long>(d.T) * d.k < d.E ? d.T * d.k : d.E;
  const long long t1 = e * ((d.f + 127ll) / 128) * (d.h / kb);
  const long long t2 = e * ((d.h + 255ll) / 256) * (d.f / kb);
  return t1 > t2 ? t1 : t2;
}

// Blocks = SMs.  Router units: token groups x slices of h, about one for each
// block; groups of up to 8 tokens so that 128 tokens make 16 groups, and single
// tokens up to 16.
Plan plan_of(const moe_dims& d, int blocks, bool fp8) {
  Plan p = {};
  p.n1 = (d.T + 15) / 16 * 16;
  p.ring = (kSmemMax - 1024 - static_cast<int>(sizeof(Ctrl))) / 1024 * 1024;
  const int most_ring = kMaxStages * (kWBytes + (fp8 ? 1 : 2) * p.n1 * 128);
  if (p.ring > most_ring) p.ring = most_ring;
  p.smem = 1024 + p.ring + static_cast<int>(sizeof(Ctrl));
  p.tok_group = (d.T + 15) / 16;
  p.groups = (d.T + p.tok_group - 1) / p.tok_group;
  int n = blocks / p.groups;
  if (n < 1) n = 1;
  p.slice_h = ((d.h + n - 1) / n + 7) / 8 * 8;
  if (p.slice_h < 32) p.slice_h = 32;  // a few long slices add up sooner than many short ones
  // a slice of Wg and x, the threads' sums and the logits fit the ring
  const int room = p.ring - (kThreads + kMaxE) * kGroupTok * 4;
  const int most = room / (d.E * 4 + kGroupTok * 2) / 8 * 8;
  if (p.slice_h > most) p.slice_h = most;
  p.slices = (d.h + p.slice_h - 1) / p.slice_h;
  p.pieces = static_cast<size_t>(blocks) *
             (most_steps(d, fp8) >= static_cast<long long>(kRoundsFrom) * blocks ? kRounds : 1);
  return p;
}

Layout layout(const moe_dims& d, bool fp8) {
  const size_t R = static_cast<size_t>(d.T) * d.k, T = d.T, h = d.h, f = d.f;
  const size_t blocks = moe_api::num_sms();
  const Plan plan = d.T > 0 ? plan_of(d, static_cast<int>(blocks), fp8) : Plan{};
  size_t off = 256;
  auto take = [&](size_t n) {
    const size_t o = off;
    off += up256(n);
    return o;
  };
  Layout L = {};
  L.logits = take(static_cast<size_t>(plan.groups) * plan.slices * plan.tok_group * d.E * 4);
  L.idx = take(R * 4);
  L.gates = take(R * 4);
  L.H = take(R * f * (fp8 ? 2 : 4));
  L.O = take(R * h * 4);
  L.part = take(2 * plan.pieces * 2 * T * 128 * 4);
  L.claim = take(8);
  if (fp8) {
    L.xq = take(T * h);
    L.sx = take(T * 4);
    L.Hq = take(R * f);
    L.amax = take(R * 4);
  }
  L.total = off;
  return L;
}

// k-steps times blocks, and times 100, stay below 2^32 (Cut's arithmetic).
bool supported(const moe_dims& d, bool fp8) {
  if (d.T > kDecodeMaxT || d.sar != 0 || (fp8 && (d.h % 128 != 0 || d.f % 128 != 0))) return false;
  // (a k-step is 32 KiB of weights: 14 million of them are 450 GB)
  if (most_steps(d, fp8) >= (1ll << 31) / moe_api::num_sms()) return false;
  if (moe_api::num_sms() * kRounds > kMaxPieces) return false;
  if (d.f > (1 << 22)) return false;  // Ctrl::join's tile numbers
  return static_cast<long long>(d.E) * (d.h > d.f ? d.h : d.f) * 2 < (1ll << 31);
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool ptr_ok(const void* p) { return p && aligned(p, 16); }

template <bool F8, bool QUOT>
cudaError_t launch(const Params& p, const Maps& m, int smem, int blocks, cudaStream_t s) {
  const void* kern = reinterpret_cast<const void*>(decode_kernel<F8, QUOT>);
  const cudaError_t e = set_smem_once(kern, kSmemMax);
  if (e != cudaSuccess) return e;
  void* args[2] = {const_cast<Params*>(&p), const_cast<Maps*>(&m)};
  const cudaError_t l = cudaLaunchCooperativeKernel(kern, dim3(blocks), dim3(kThreads), args,
                                                    static_cast<size_t>(smem), s);
  if (l == cudaSuccess) return launched();
  cudaGetLastError();  // reported here, not by the next launch
  return l;
}

moe_status decode(const moe_dims* dims, const moe_bf16* x, const float* Wg, const float* b,
                  const moe_bf16* W1, const moe_bf16* W3, const moe_bf16* W2, const void* qw,
                  moe_bf16* y, int32_t* topk_idx, float* gates, void* ws, size_t ws_bytes,
                  cudaStream_t stream, bool fp8, bool quotient) {
  const moe_status st = moe_api::check_dims(dims, true);
  if (st != MOE_OK) return st;
  const moe_dims& d = *dims;
  if (!supported(d, fp8)) return MOE_ERR_UNSUPPORTED;
  const bool empty = d.T == 0;
  if ((!empty && (!ptr_ok(x) || !ptr_ok(y))) || !aligned(x, 16) || !aligned(y, 16) ||
      !ptr_ok(Wg) || (d.has_bias && !ptr_ok(b)) || !aligned(topk_idx, 16) || !aligned(gates, 16))
    return MOE_ERR_INVALID_ARG;
  if (fp8 ? (!qw || !aligned(qw, 256)) : (!ptr_ok(W1) || !ptr_ok(W3) || !ptr_ok(W2)))
    return MOE_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, 256)) return MOE_ERR_INVALID_ARG;
  const Layout L = layout(d, fp8);
  if (ws_bytes < L.total) return MOE_ERR_WORKSPACE;
  if (empty) return MOE_OK;
  uint8_t* w = static_cast<uint8_t*>(ws);
  const int blocks = moe_api::num_sms();
  const Plan plan = plan_of(d, blocks, fp8);
  Params p = {};
  p.T = d.T;
  p.h = d.h;
  p.f = d.f;
  p.E = d.E;
  p.k = d.k;
  p.capacity = d.capacity > 0 && d.capacity < d.T ? d.capacity : d.T;
  p.n1 = plan.n1;
  p.ring_bytes = plan.ring;
  p.tok_group = plan.tok_group;
  p.groups = plan.groups;
  p.slices = plan.slices;
  p.slice_h = plan.slice_h;
  p.x = x;
  p.Wg = Wg;
  p.b = d.has_bias ? b : nullptr;
  p.idx = topk_idx ? topk_idx : reinterpret_cast<int32_t*>(w + L.idx);
  p.gates = gates ? gates : reinterpret_cast<float*>(w + L.gates);
  p.logits = reinterpret_cast<float*>(w + L.logits);
  p.H = reinterpret_cast<uint16_t*>(w + L.H);
  p.O = reinterpret_cast<float*>(w + L.O);
  p.part = reinterpret_cast<float*>(w + L.part);
  p.claim = reinterpret_cast<unsigned*>(w + L.claim);
  p.y = y;
  p.status = reinterpret_cast<int*>(ws);
  Maps m;
  memset(&m, 0, sizeof(m));
  const uint64_t R = static_cast<uint64_t>(d.T) * d.k, E = d.E, h = d.h, f = d.f;
  cudaError_t e;
  if (fp8) {
    auto view = [&](const char* name) {
      return moe_fp8_weight_view(dims, const_cast<void*>(qw), name);
    };
    p.xq = w + L.xq;
    p.sx = reinterpret_cast<float*>(w + L.sx);
    p.Hq = w + L.Hq;
    p.amax = reinterpret_cast<unsigned*>(w + L.amax);
    p.s1 = static_cast<const float*>(view("s1"));
    p.s3 = static_cast<const float*>(view("s3"));
    p.s2 = static_cast<const float*>(view("s2"));
    if (!make_map_kmajor(&m.x, p.xq, h, d.T, plan.n1, true) ||
        !make_map_codes(&m.w1, view("W13q"), h, 2 * f, E, 256) ||
        !make_map_kmajor(&m.h, p.Hq, f, R, 16, true) ||
        !make_map_codes(&m.w2, view("W2q"), f, h, E, 256))
      return MOE_ERR_CUDA;
    m.w3 = m.w1;
    e = quotient ? launch<true, true>(p, m, plan.smem, blocks, stream)
                 : launch<true, false>(p, m, plan.smem, blocks, stream);
  } else {
    if (!make_map_kmajor(&m.x, x, h, d.T, plan.n1, false) || !make_map_columns(&m.w1, W1, f, E * h, 2) ||
        !make_map_columns(&m.w3, W3, f, E * h, 2) || !make_map_kmajor(&m.h, p.H, f, 2 * R, 16, false) ||
        !make_map_columns(&m.w2, W2, h, E * f, 4))
      return MOE_ERR_CUDA;
    e = launch<false, false>(p, m, plan.smem, blocks, stream);
  }
  if (e != cudaSuccess || !moe_api::note(stream, "layer_decode")) return MOE_ERR_CUDA;
  return MOE_OK;
}

}  // namespace

size_t decode_workspace_bytes(const moe_dims& d, bool fp8) {
  return supported(d, fp8) ? layout(d, fp8).total : 0;
}

}  // namespace moe

extern "C" {

moe_status moe_layer_decode(const moe_dims* dims, const moe_bf16* x, const float* Wg,
                            const float* b, const moe_bf16* W1, const moe_bf16* W3,
                            const moe_bf16* W2, moe_bf16* y, int32_t* topk_idx, float* gates,
                            void* ws, size_t ws_bytes, moe_stream_t stream) {
  return moe::decode(dims, x, Wg, b, W1, W3, W2, nullptr, y, topk_idx, gates, ws, ws_bytes,
                     reinterpret_cast<cudaStream_t>(stream), false, false);
}

moe_status moe_layer_decode_fp8(const moe_dims* dims, const moe_bf16* x, const float* Wg,
                                const float* b, const void* qw, moe_bf16* y, int32_t* topk_idx,
                                float* gates, void* ws, size_t ws_bytes, moe_stream_t stream) {
  return moe::decode(dims, x, Wg, b, nullptr, nullptr, nullptr, qw, y, topk_idx, gates, ws,
                     ws_bytes, reinterpret_cast<cudaStream_t>(stream), true, false);
}

moe_status moe_layer_decode_fp8_as_fwd(const moe_dims* dims, const moe_bf16* x, const float* Wg,
                                       const float* b, const void* qw, moe_bf16* y,
                                       int32_t* topk_idx, float* gates, void* ws, size_t ws_bytes,
                                       moe_stream_t stream) {
  return moe::decode(dims, x, Wg, b, nullptr, nullptr, nullptr, qw, y, topk_idx, gates, ws,
                     ws_bytes, reinterpret_cast<cudaStream_t>(stream), true, true);
}

}  // extern "C"
