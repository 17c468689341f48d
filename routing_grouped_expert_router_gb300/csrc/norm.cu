// norm.cu -- the norms before and after the MoE block, fused with its gate
// and residual scale: moe_block_norm_fwd and moe_block_norm_bwd.
//
//   z = y / rms(y) * w_post;  r_out = alpha r + beta gate * z;
//   u = r_out / rms(r_out) * w_pre
//
// Both directions are bound by HBM: the forward reads r and y and writes r_out
// and u (8 bytes for each element with a bf16 residual), the backward reads
// r_out, y, du and dr_out and writes dr and dy (12 bytes).  Each row is read
// once.  A row has two sums in a chain, and a block that waits for its loads and
// then for its sums leaves HBM idle (a block for each row: 4.5 TB/s forward), so
// the blocks stay, each with a ring of the next rows in shared memory that bulk
// copies fill, and keep the channel weights in registers: two to four 8-element
// pieces of the row to a thread, the same columns for every row.
// Measured on GB300, bf16, 16384 x 4096: forward 82 us (6.5 TB/s, 0.96 of a copy's
// rate), backward 128 us (rows 120, the column sums the rest); 7 x 6400 fp32
// forward 3.6 us, 1021 x 2056 fp32 backward 12.9.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/moe.h"
#include "api_internal.h"
#include "kernels.cuh"
#include "ptx.cuh"

namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kMaxH = 8192;
constexpr int kMaxThreads = 512;
constexpr int kFwdThreads = 1024;  // of the forward's blocks on an SM
constexpr int kPieces = 2;  // 8-element pieces of a row for each thread

constexpr int kMaxSlots = 4;

struct Args {
  const void* r;        // fwd: r; bwd: r_out (NULL without w_pre)
  const uint16_t* y;
  const float* w_post;
  const float* gate;
  const float* w_pre;
  const uint16_t* du;
  const void* dr_out;
  void* out_r;          // fwd: r_out; bwd: dr
  uint4* out_u;         // fwd: u; bwd: dy
  float* dgate;         // bwd, token gate
  float* partial;       // bwd: column sums of each block
  int* status;
  int T, h;
  int gate_kind;
  int slots, slot_bytes;
  float eps, alpha, beta, inv_h;
};

// Pairs of fp32 values for Blackwell's packed arithmetic: these kernels issue
// about 20 instructions for each element otherwise, which bounded them.
typedef unsigned long long f2;
__device__ __forceinline__ f2 pair(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 split(f2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 both(float v) { return pair(v, v); }
__device__ __forceinline__ float sum2(f2 v) {
  const float2 s = split(v);
  return s.x + s.y;
}

// Eight bf16 values as four pairs, and back.
__device__ __forceinline__ void unpack8(const uint4& q, f2* v) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
__device__ __forceinline__ uint4 pack8(const f2* v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 s = split(v[i]);
    const __nv_bfloat162 p = __floats2bfloat162_rn(s.x, s.y);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight fp32 values, as the residual stream and the channel weights have them.
__device__ __forceinline__ void load8(const float* p, f2* v) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = pair(a.x, a.y);
  v[1] = pair(a.z, a.w);
  v[2] = pair(b.x, b.y);
  v[3] = pair(b.z, b.w);
}
__device__ __forceinline__ void store8(float* p, const f2* v) {
  const float2 a = split(v[0]), b = split(v[1]), c = split(v[2]), d = split(v[3]);
  reinterpret_cast<float4*>(p)[0] = make_float4(a.x, a.y, b.x, b.y);
  reinterpret_cast<float4*>(p)[1] = make_float4(c.x, c.y, d.x, d.y);
}
// Eight values of the residual stream at element offset o.
template <bool F32>
__device__ __forceinline__ void load_res(const void* p, size_t o, f2* v) {
  if (F32)
    load8(static_cast<const float*>(p) + o, v);
  else
    unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + o), v);
}
// Stores eight values in the residual's type and leaves the stored ones in v.
template <bool F32>
__device__ __forceinline__ void store_res(void* p, size_t o, f2* v) {
  if (F32) {
    store8(static_cast<float*>(p) + o, v);
  } else {
    const uint4 q = pack8(v);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + o) = q;
    unpack8(q, v);
  }
}

// Sums over the block, in every thread.  The order is fixed: a butterfly within
// each warp, then the warps in order.  red[..][warp] of the warps that do not
// exist is zero.  `half` alternates so that one barrier for each call is enough.
// Returns whether `ok` held in every thread.
__device__ __forceinline__ float sum_warps(const float* s) {
  const float4* q = reinterpret_cast<const float4*>(s);
  const float4 a = q[0], b = q[1];
  float v = ((a.x + a.y) + (a.z + a.w)) + ((b.x + b.y) + (b.z + b.w));
  if (blockDim.x > 256) {
    const float4 c = q[2], d = q[3];
    v += ((c.x + c.y) + (c.z + c.w)) + ((d.x + d.y) + (d.z + d.w));
  }
  return v;
}
typedef float Red1[2][16];
__device__ __forceinline__ bool block_sum(float& v, Red1& red, int& half, bool ok) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  if ((threadIdx.x & 31) == 0) red[half][threadIdx.x >> 5] = v;
  ok = __syncthreads_and(ok);
  v = sum_warps(red[half]);
  half ^= 1;
  return ok;
}
// The same for R rows at once.
template <int R>
struct RedRows {
  float one[2][R][16], three[2][R][3][16];
};
template <int R>
__device__ __forceinline__ void block_sum(float (&v)[R], RedRows<R>& red, int& half) {
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[r] += __shfl_xor_sync(kFull, v[r], o);
    if ((threadIdx.x & 31) == 0) red.one[half][r][threadIdx.x >> 5] = v[r];
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r) v[r] = sum_warps(red.one[half][r]);
  half ^= 1;
}
// Three sums of each row: each exchange halves what a lane holds, so that 6
// shuffles do instead of 15; lanes 0, 8 and 16 end up with one sum each.
template <int R>
__device__ __forceinline__ bool block_sum3(float (&v)[R][3], RedRows<R>& red, int& half, bool ok) {
  const int lane = threadIdx.x & 31;
  const bool hi = lane & 16, mid = lane & 8;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float x0 = (hi ? v[r][2] : v[r][0]) + __shfl_xor_sync(kFull, hi ? v[r][0] : v[r][2], 16);
    float x1 = (hi ? 0.f : v[r][1]) + __shfl_xor_sync(kFull, hi ? v[r][1] : 0.f, 16);
    x0 = (mid ? x1 : x0) + __shfl_xor_sync(kFull, mid ? x0 : x1, 8);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) x0 += __shfl_xor_sync(kFull, x0, o);
    if ((lane & 7) == 0 && lane < 24) red.three[half][r][lane >> 3][threadIdx.x >> 5] = x0;
  }
  ok = __syncthreads_and(ok);
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < 3; ++i) v[r][i] = sum_warps(red.three[half][r][i]);
  half ^= 1;
  return ok;
}

// 1 / rms of a row from its sum of squares: the fast reciprocal root and one
// Newton step, within about an ulp (0 where the sum overflowed).
__device__ __forceinline__ float inv_rms(float ss, const Args& a) {
  const float x = fmaf(ss, a.inv_h, a.eps), y = rsqrtf(x);
  return x < INFINITY ? fmaf(0.5f * y, fmaf(-x * y, y, 1.f), y) : y;
}

// The block's ring of rows.  Row number n of the block (token blockIdx.x + n *
// gridDim.x) goes through slot n % slots; a slot holds `streams` arrays' rows,
// one after another.
constexpr int kMaxStreams = 4;
struct Ring {
  const uint8_t* src[kMaxStreams];
  uint32_t bytes[kMaxStreams];  // of a row; 0: not read
  uint32_t total;
};
__device__ __forceinline__ void ring_load(const Args& a, const Ring& g, uint64_t* full,
                                          uint8_t* smem, int n) {
  const long long t = blockIdx.x + static_cast<long long>(n) * gridDim.x;
  if (t >= a.T) return;
  const int s = n % a.slots;
  const uint32_t bar = moe::smem_u32(&full[s]);
  uint32_t dst = moe::smem_u32(smem) + s * a.slot_bytes;
  moe::mbar_expect_tx(bar, g.total);
#pragma unroll
  for (int i = 0; i < kMaxStreams; ++i)
    if (g.bytes[i]) {
      moe::bulk_load(dst, g.src[i] + t * g.bytes[i], g.bytes[i], bar);
      dst += g.bytes[i];
    }
}
__device__ __forceinline__ bool ring_wait(const Args& a, uint64_t* full, int n) {
  return moe::mbar_wait(moe::smem_u32(&full[n % a.slots]), (n / a.slots) & 1, a.status,
                        MOE_ERR_DEVICE_TIMEOUT);
}
// After a wait for row n ran out: the rows asked for land before the block ends,
// that one among them.
__device__ __forceinline__ void ring_drain(const Args& a, uint64_t* full, int n) {
  if (threadIdx.x == 0)
    for (int i = 0; i < a.slots; ++i)
      if (blockIdx.x + static_cast<long long>(n + i) * gridDim.x < a.T) ring_wait(a, full, n + i);
}

// These kernels are launched before the stream's work ahead of them has ended,
// which they wait for here: a step of a few rows is shorter than a launch.
// Nothing that another kernel wrote is read, and nothing is written, before.
__device__ __forceinline__ void after_stream() {
  cudaGridDependencySynchronize();
  cudaTriggerProgrammaticLaunchCompletion();
}

// KEEP: a thread keeps its pieces of r and y between the two sums and the slot is
// free after the first; otherwise it reads y again, with registers to spare for
// twice the threads on an SM.  N: pieces of a row to a thread.
constexpr int kKeepThreads = 256;  // of a block with three pieces to a thread
template <bool F32, bool KEEP, int N>
__global__ void __launch_bounds__(N == 3 ? kKeepThreads : kMaxThreads, KEEP && N == 2 ? 1 : 2)
    block_norm_fwd_kernel(const Args a) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[kMaxSlots];
  __shared__ __align__(16) Red1 red;
  int half = 0;
  if (threadIdx.x < 32) red[threadIdx.x >> 4][threadIdx.x & 15] = 0.f;
  Ring g;
  g.src[0] = static_cast<const uint8_t*>(a.r);
  g.src[1] = reinterpret_cast<const uint8_t*>(a.y);
  g.bytes[0] = a.h * (F32 ? 4 : 2);
  g.bytes[1] = a.y ? a.h * 2 : 0;
  g.bytes[2] = g.bytes[3] = 0;
  g.total = g.bytes[0] + g.bytes[1];
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.slots; ++s) moe::mbar_init(moe::smem_u32(&full[s]), 1);
    moe::fence_mbar_init();
  }
  after_stream();
  if (threadIdx.x == 0)
    for (int n = 0; n < a.slots; ++n) ring_load(a, g, full, smem, n);
  // the scale of each of my columns of y, and of u
  f2 wz[N][4], wu[N][4];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = (threadIdx.x + i * blockDim.x) * 8;
    if (c >= a.h) continue;
    f2 w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) wz[i][j] = both(a.beta);
    if (a.gate_kind == MOE_GATE_CHANNEL) {
      load8(a.gate + c, w);
#pragma unroll
      for (int j = 0; j < 4; ++j) wz[i][j] = mul2(wz[i][j], w[j]);
    }
    if (a.w_post) {
      load8(a.w_post + c, w);
#pragma unroll
      for (int j = 0; j < 4; ++j) wz[i][j] = mul2(wz[i][j], w[j]);
    }
    if (a.w_pre) load8(a.w_pre + c, wu[i]);
  }
  __syncthreads();
  int n = 0;
  for (int t = blockIdx.x; t < a.T; ++n) {
    const size_t row = static_cast<size_t>(t) * a.h;
    float s = 1.f;
    if (a.gate_kind == MOE_GATE_TOKEN) s = __ldg(a.gate + t);
    bool ok = ring_wait(a, full, n);
    const uint8_t* slot = smem + (n % a.slots) * a.slot_bytes;
    const uint8_t* sy = slot + g.bytes[0];
    const f2 al = both(a.alpha);
    f2 v[N][4], acc = 0;
    float ss = 0.f;
    if (KEEP) {
      f2 z[N][4];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = (threadIdx.x + i * blockDim.x) * 8;
        if (c >= a.h) continue;
        load_res<F32>(slot, c, v[i]);
        if (!a.y) continue;
        unpack8(*reinterpret_cast<const uint4*>(sy + c * 2), z[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc = fma2(z[i][j], z[i][j], acc);
      }
      // the barrier of this sum also ends the reads of the slot
      ss = sum2(acc);
      ok = block_sum(ss, red, half, ok);
      if (threadIdx.x == 0 && ok) ring_load(a, g, full, smem, n + a.slots);
      if (!ok) break;
      if (a.y) {
        if (a.w_post) s *= inv_rms(ss, a);
        const f2 s2 = both(s);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int c = (threadIdx.x + i * blockDim.x) * 8;
          if (c >= a.h) continue;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            v[i][j] = fma2(mul2(s2, z[i][j]), wz[i][j], mul2(al, v[i][j]));
          store_res<F32>(a.out_r, row + c, v[i]);
        }
      }
      if (a.w_pre) {
        acc = 0;
#pragma unroll
        for (int i = 0; i < N; ++i)
          if ((threadIdx.x + i * blockDim.x) * 8 < a.h)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc = fma2(v[i][j], v[i][j], acc);
        ss = sum2(acc);
        block_sum(ss, red, half, true);
      }
    } else {
      f2 z[4];
      if (a.w_post) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int c = (threadIdx.x + i * blockDim.x) * 8;
          if (c >= a.h) continue;
          unpack8(*reinterpret_cast<const uint4*>(sy + c * 2), z);
#pragma unroll
          for (int j = 0; j < 4; ++j) acc = fma2(z[j], z[j], acc);
        }
        ss = sum2(acc);
        ok = block_sum(ss, red, half, ok);
        s *= inv_rms(ss, a);
      }
      const f2 s2 = both(s);
      acc = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = (threadIdx.x + i * blockDim.x) * 8;
        if (c >= a.h) continue;
        load_res<F32>(slot, c, v[i]);
        if (a.y) {
          unpack8(*reinterpret_cast<const uint4*>(sy + c * 2), z);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            v[i][j] = fma2(mul2(s2, z[j]), wz[i][j], mul2(al, v[i][j]));
          store_res<F32>(a.out_r, row + c, v[i]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) acc = fma2(v[i][j], v[i][j], acc);
      }
      ss = sum2(acc);
      ok = block_sum(ss, red, half, ok);
      if (!ok) break;
      if (threadIdx.x == 0) ring_load(a, g, full, smem, n + a.slots);
    }
    if (a.w_pre) {
      const f2 rv = both(inv_rms(ss, a));
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = (threadIdx.x + i * blockDim.x) * 8;
        if (c >= a.h) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i][j] = mul2(mul2(rv, v[i][j]), wu[i][j]);
        a.out_u[(row + c) >> 3] = pack8(v[i]);
      }
    }
    if (a.T - t <= static_cast<int>(gridDim.x)) return;
    t += gridDim.x;
  }
  if (n > 0 || static_cast<int>(blockIdx.x) < a.T) ring_drain(a, full, n);
}

// The backward of a row, with v = r_out, rv = 1 / rms(v), n = y / rms(y) (n = y
// without w_post), and the row sums S:
//   G  = dr_out + rv (du w_pre - v rv^2 S(du w_pre v) / h)
//   q  = beta gate G;  dy = (q w_post - n S(q w_post n) / h) / rms(y)
// Column sums: P = sum_t du v rv (dw_pre) and Q = sum_t g_t G n, from which
// dw_post = beta gate_c Q and the channel gate's gradient = beta w_post Q, so one
// sum serves both (g_t: the token gate, else 1).  Each block keeps P and Q of its
// rows in registers and writes them once; block_norm_cols_kernel adds the
// blocks in order.
// R rows go through these steps side by side: two where a block is alone on
// its SM (long rows) and a thread may have the registers for it.
// ALL: every optional part is there (the training step's call), so the loops over a
// row's pieces hold no branch on one, and the two pieces overlap (2^25 elements,
// bf16, share of HBM without / with: h 1288 63 / 74%, 4096 80 / 88, 6400 64 / 73).
// N pieces of the row to a thread: three (12 warps on an SM, 168 registers) where
// that holds more columns on an SM than two (16 warps), and in a block of 256
// threads that is alone on its SM three, with two rows side by side, or four.
constexpr int kPairThreads = 384, kThreeThreads = 192, kWideThreads = 256;
template <bool F32, int R, bool ALL, int N>
__global__ void __launch_bounds__(R * N > 3 && N > 2 ? kWideThreads
                                  : R == 2             ? kPairThreads
                                  : N == 3             ? kThreeThreads
                                                       : kMaxThreads,
                                  R == 1 && N == 3 ? 2 : 1)
    block_norm_bwd_kernel(const Args a) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[kMaxSlots];
  __shared__ __align__(16) RedRows<R> red;
  const bool has_y = ALL || a.y, has_dr = ALL || a.dr_out;
  const bool post = ALL || a.w_post, pre = ALL || a.w_pre;
  int half3 = 0, half1 = 0;
  for (int i = threadIdx.x; i < static_cast<int>(sizeof(red) / 4); i += blockDim.x)
    reinterpret_cast<float*>(&red)[i] = 0.f;
  const uint32_t res = a.h * (F32 ? 4 : 2), row16 = a.h * 2;
  Ring g;
  g.src[0] = static_cast<const uint8_t*>(a.r);
  g.src[1] = reinterpret_cast<const uint8_t*>(a.du);
  g.src[2] = reinterpret_cast<const uint8_t*>(a.y);
  g.src[3] = static_cast<const uint8_t*>(a.dr_out);
  g.bytes[0] = a.w_pre ? res : 0;
  g.bytes[1] = a.w_pre ? row16 : 0;
  g.bytes[2] = a.y ? row16 : 0;
  g.bytes[3] = a.dr_out ? res : 0;
  g.total = g.bytes[0] + g.bytes[1] + g.bytes[2] + g.bytes[3];
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.slots; ++s) moe::mbar_init(moe::smem_u32(&full[s]), 1);
    moe::fence_mbar_init();
  }
  after_stream();
  if (threadIdx.x == 0)
    for (int n = 0; n < a.slots; ++n) ring_load(a, g, full, smem, n);
  // w_pre, and the factor of G in dz's product with w_post
  f2 wu[N][4], wz[N][4];
  f2 P[N][4], Q[N][4];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = (threadIdx.x + i * blockDim.x) * 8;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      P[i][j] = Q[i][j] = wu[i][j] = 0;
      wz[i][j] = both(a.beta);
    }
    if (c >= a.h) continue;
    f2 w[4];
    if (a.w_pre) load8(a.w_pre + c, wu[i]);
    if (a.gate_kind == MOE_GATE_CHANNEL) {
      load8(a.gate + c, w);
#pragma unroll
      for (int j = 0; j < 4; ++j) wz[i][j] = mul2(wz[i][j], w[j]);
    }
    if (a.w_post) {
      load8(a.w_post + c, w);
#pragma unroll
      for (int j = 0; j < 4; ++j) wz[i][j] = mul2(wz[i][j], w[j]);
    }
  }
  const float al = a.y ? a.alpha : 1.f;
  const bool token = a.gate_kind == MOE_GATE_TOKEN;
  const uint32_t at_y = g.bytes[0] + g.bytes[1], at_dr = at_y + g.bytes[2];
  __syncthreads();
  int n = 0;
  bool ok = true;
  for (long long t0 = blockIdx.x; t0 < a.T; t0 += static_cast<long long>(R) * gridDim.x, n += R) {
    int t[R];
    bool live[R];
    float gt[R], s3[R][3];
    const uint8_t* sv[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      live[r] = t0 + r * gridDim.x < a.T;
      t[r] = static_cast<int>(live[r] ? t0 + r * gridDim.x : t0);
      gt[r] = token ? __ldg(a.gate + t[r]) : 1.f;
      sv[r] = smem + ((n + r) % a.slots) * a.slot_bytes;
      if (R == 1 || live[r]) ok = ring_wait(a, full, n + r) && ok;
      f2 acc[3] = {0, 0, 0};
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = (threadIdx.x + i * blockDim.x) * 8;
        if (c >= a.h || (R > 1 && !live[r])) continue;
        f2 v[4], d[4];
        if (pre) {
          load_res<F32>(sv[r], c, v);
          unpack8(*reinterpret_cast<const uint4*>(sv[r] + g.bytes[0] + c * 2), d);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            acc[0] = fma2(v[j], v[j], acc[0]);
            acc[1] = fma2(mul2(d[j], wu[i][j]), v[j], acc[1]);
          }
        }
        if (post) {
          unpack8(*reinterpret_cast<const uint4*>(sv[r] + at_y + c * 2), v);
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[2] = fma2(v[j], v[j], acc[2]);
        }
      }
#pragma unroll
      for (int i = 0; i < 3; ++i) s3[r][i] = sum2(acc[i]);
    }
    ok = block_sum3<R>(s3, red, half3, ok);
    if (!ok) break;
    f2 G[R][N][4];
    uint4 y[R][N];
    float s1[R], rys[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float rvs = pre ? inv_rms(s3[r][0], a) : 0.f;
      rys[r] = post ? inv_rms(s3[r][2], a) : 1.f;
      const f2 rv = both(rvs), k1 = both(-s3[r][1] * a.inv_h * rvs * rvs * rvs);
      const f2 al2 = both(al), gy = both(gt[r] * rys[r]);
      const size_t row = static_cast<size_t>(t[r]) * a.h;
      f2 dot = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = (threadIdx.x + i * blockDim.x) * 8;
        if (c >= a.h || (R > 1 && !live[r])) continue;
        f2 v[4], d[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) G[r][i][j] = 0;
        if (has_dr) load_res<F32>(sv[r] + at_dr, c, G[r][i]);
        if (pre) {
          load_res<F32>(sv[r], c, v);
          unpack8(*reinterpret_cast<const uint4*>(sv[r] + g.bytes[0] + c * 2), d);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const f2 dn = mul2(rv, d[j]);
            P[i][j] = fma2(dn, v[j], P[i][j]);
            G[r][i][j] = fma2(dn, wu[i][j], fma2(k1, v[j], G[r][i][j]));
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = mul2(al2, G[r][i][j]);
        store_res<F32>(a.out_r, row + c, v);
        if (!has_y) continue;
        y[r][i] = *reinterpret_cast<const uint4*>(sv[r] + at_y + c * 2);
        unpack8(y[r][i], v);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          Q[i][j] = fma2(mul2(gy, G[r][i][j]), v[j], Q[i][j]);
          G[r][i][j] = mul2(G[r][i][j], wz[i][j]);
          dot = fma2(G[r][i][j], v[j], dot);
        }
      }
      s1[r] = sum2(dot) * rys[r];
    }
    // the projection of dy on y's row, which without the token's gate is also
    // that gate's gradient; the barrier ends the reads of the slots
    block_sum<R>(s1, red, half1);
    if (threadIdx.x == 0)
#pragma unroll
      for (int r = 0; r < R; ++r) ring_load(a, g, full, smem, n + r + a.slots);
    if (!has_y) continue;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (R > 1 && !live[r]) break;
      const size_t row = static_cast<size_t>(t[r]) * a.h;
      const f2 k2 = both(-s1[r] * a.inv_h * rys[r]), gy = both(gt[r] * rys[r]);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = (threadIdx.x + i * blockDim.x) * 8;
        if (c >= a.h) continue;
        f2 v[4];
        unpack8(y[r][i], v);
#pragma unroll
        for (int j = 0; j < 4; ++j)  // (without a norm dy does not depend on y, finite or not)
          v[j] = mul2(gy, post ? fma2(k2, v[j], G[r][i][j]) : G[r][i][j]);
        a.out_u[(row + c) >> 3] = pack8(v);
      }
      if (a.dgate && threadIdx.x == 0) a.dgate[t[r]] = s1[r];
    }
  }
  if (!ok) ring_drain(a, full, n);
  float* part = a.partial + static_cast<size_t>(blockIdx.x) * 2 * a.h;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = (threadIdx.x + i * blockDim.x) * 8;
    if (c >= a.h) continue;
    store8(part + c, P[i]);
    store8(part + a.h + c, Q[i]);
  }
}

// The column gradients from the blocks' sums, a fixed order for each column:
// interleaved chains, then those in order.  COLS columns to a block: 8 where two
// blocks of 8 for each SM hold all, else 16 (1021 x 2056: 13.9 us in all
// with 32 or 16, 12.9 with 8; 16384 x 4096: 128.6 with 32, 128.0 with 16, 131 with 8).
constexpr int kColThreads = 1024;
template <int COLS>
__global__ void __launch_bounds__(kColThreads)
    block_norm_cols_kernel(const float* partial, int nblk, int h, const float* w_post,
                           const float* gate, float beta, float* dw_pre, float* dw_post,
                           float* dgate) {
  constexpr int kChains = kColThreads / COLS;
  after_stream();
  __shared__ float sums[2][kChains][COLS + 1];
  const int g = threadIdx.x / COLS, i = threadIdx.x % COLS;
  const int c = blockIdx.x * COLS + i;
  float p = 0.f, q = 0.f;
  if (c < h) {
#pragma unroll 8
    for (int b = g; b < nblk; b += kChains) {
      p += __ldcg(partial + static_cast<size_t>(b) * 2 * h + c);
      q += __ldcg(partial + static_cast<size_t>(b) * 2 * h + h + c);
    }
  }
  sums[0][g][i] = p;
  sums[1][g][i] = q;
  __syncthreads();
  // a warp for each of the two sums of each column
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (warp >= 2 * COLS) return;
  const int which = warp / COLS, col = blockIdx.x * COLS + warp % COLS;
  float v = 0.f;
#pragma unroll
  for (int n = lane; n < kChains; n += 32) v += sums[which][n][warp % COLS];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  if (lane != 0 || col >= h) return;
  if (which == 0) {
    if (dw_pre) dw_pre[col] = v;
    return;
  }
  v *= beta;
  if (dw_post) dw_post[col] = gate ? gate[col] * v : v;
  if (dgate) dgate[col] = w_post ? w_post[col] * v : v;
}

constexpr size_t kAlign = 256;

int threads_for(int h, int pieces) {
  const int need = (h / 8 + pieces - 1) / pieces;
  return (need + 31) / 32 * 32;
}

// Blocks on an SM, and the rows that each keeps on their way: as many threads
// as the registers allow (a forward thread takes 64 to 128, a backward one 128 to 240: the
// weights and column sums), and at least two slots for each block within the
// shared memory.
struct Plan {
  int threads, blocks, pieces, rows, slots, slot_bytes, smem;  // rows: side by side in a block
  int most_blocks;  // of any call with at most as many rows: grows with T
  bool keep;
};
Plan plan_of(const moe_norm_dims& d, bool bwd) {
  constexpr int kSmem = 216 << 10;
  Plan p;
  p.threads = threads_for(d.h, kPieces);
  p.pieces = kPieces;
  const int res = d.res_f32 ? 4 : 2;
  p.slot_bytes = d.h * (bwd ? 2 * res + 4 : res + 2);
  // Forward: two pieces of a row to a thread, which keeps them, where 512 threads
  // hold enough columns at once that way; else three, up to 6144 columns; else two
  // that are read again (h 6400 bf16, share of HBM over 2^25 elements: kept 73%,
  // read again 82).  Two read again / three kept, bf16: h 768 71 / 80%, 1288 78 /
  // 88, 2056 78 / 87, 3328 84 / 89, 4608 82 / 89, 5120 82 / 89, 6144 80 / 82; fp32:
  // 4352 81 / 87, 5120 80 / 88, 5632 80 / 86.  Two kept, bf16: 2048 89, 4096 88.
  p.keep = kMaxThreads / p.threads * d.h >= (d.res_f32 ? 5700 : 7000);
  if (!bwd && !p.keep && threads_for(d.h, 3) <= kKeepThreads) {
    p.keep = true;
    p.pieces = 3;
    p.threads = threads_for(d.h, 3);
  }
  int per_sm = (bwd || p.keep ? kMaxThreads : kFwdThreads) / p.threads;
  // Backward, bf16 residual: three pieces to a thread where blocks of two hold few
  // columns on an SM and blocks of three more.  Share of HBM over 2^25 elements,
  // two / three: h 768 74 / 81%, 1288 76 / 82, 2056 79 / 87, 2816 78 / 86, 4352 63 /
  // 87, 4608 64 / 85; but 1536 (7680 columns with two) 86 / 82, and of fp32 rows
  // 768 81 / 65, 2816 92 / 79, 4352 85 / 79.
  const int per_sm3 = 2 * kThreeThreads / threads_for(d.h, 3);
  if (bwd && !d.res_f32 && per_sm * d.h < 7000 && per_sm3 > per_sm) {
    p.pieces = 3;
    p.threads = threads_for(d.h, 3);
    per_sm = per_sm3;
  }
  if (per_sm > 16) per_sm = 16;
  // The backward's rows on their way to an SM: 160 KiB at most.  More of them draw
  // less from HBM (fp32, 216 / 160 KiB: h 512 74 / 79%, 1024 78 / 85, 2048 80 / 84,
  // 4096 80 / 89, other sizes the same).
  const int most = bwd ? 160 << 10 : kSmem;
  if (per_sm * 2 * p.slot_bytes > most) per_sm = most / (2 * p.slot_bytes);
  if (per_sm < 1) per_sm = 1;
  // Long bf16 rows, a block to an SM: fewer warps with more pieces each.  Share of
  // HBM with two pieces / 256 threads: h 5120 68 / 74%, 6144 77 / 81, 7168 76 / 79,
  // 8192 81 / 84 (one piece and twice the threads, 5120: 62).
  if (bwd && !d.res_f32 && per_sm == 1) {
    p.threads = kWideThreads;
    p.pieces = d.h <= 24 * kWideThreads ? 3 : 4;
  }
  p.slots = kSmem / (per_sm * p.slot_bytes);
  if (p.slots > kMaxSlots) p.slots = kMaxSlots;
  // Two rows need four slots (one row / two, fp32: h 3584 62 / 83%, 4096 67 / 89).
  p.rows = bwd && per_sm == 1 && p.slots == kMaxSlots && p.threads <= kPairThreads && p.pieces < 4
               ? 2
               : 1;
  // Backward, one row at a time: the row that is worked on and the next.  More of
  // them under way draw less from HBM (2^25 elements, bf16, share with four / two:
  // h 1024 77 / 81%, 1288 70 / 74, 3328 80 / 82, 4096 85 / 88, 8192 83 / 83;
  // 16384 x 4096: 138 us with four, 128 with two).  Rows of four
  // pieces take the three or four that fit: 8192 82 / 84%.
  if (bwd && p.rows == 1 && p.pieces < 4) p.slots = 2;
  p.smem = p.slots * p.slot_bytes;
  const int n = moe_api::num_sms() * per_sm;
  p.most_blocks = p.blocks = d.T < n ? d.T : n;
  // no more blocks than the same number of rounds needs: each leaves its sums
  if (bwd && d.T > 0) {
    const int rounds = (d.T - 1) / (n * p.rows) + 1;
    p.blocks = (d.T - 1) / (rounds * p.rows) + 1;
  }
  return p;
}

template <class... P, class... A>
cudaError_t launch_early(void (*kern)(P...), int blocks, int threads, int smem, cudaStream_t s,
                         A... args) {
  cudaLaunchAttribute early = {};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  if (e == cudaSuccess) return moe::launched();
  cudaGetLastError();  // reported here, not by the next launch
  return e;
}

template <bool F32>
auto fwd_kernel(const Plan& p) {
  if (p.pieces == 3) return block_norm_fwd_kernel<F32, true, 3>;
  if constexpr (!F32)  // fp32 rows that long are always kept
    if (!p.keep) return block_norm_fwd_kernel<F32, false, 2>;
  return block_norm_fwd_kernel<F32, true, 2>;
}

template <bool F32, bool ALL>
auto bwd_kernel(const Plan& p) {
  if constexpr (F32) {
    if (p.rows == 2) return block_norm_bwd_kernel<F32, 2, ALL, 2>;
  } else {
    if (p.rows == 2) return block_norm_bwd_kernel<F32, 2, ALL, 3>;
    if (p.pieces == 3) return block_norm_bwd_kernel<F32, 1, ALL, 3>;
    if (p.pieces == 4) return block_norm_bwd_kernel<F32, 1, ALL, 4>;
  }
  return block_norm_bwd_kernel<F32, 1, ALL, 2>;
}
template <bool F32>
auto bwd_kernel(const Plan& p, bool all) {
  return all ? bwd_kernel<F32, true>(p) : bwd_kernel<F32, false>(p);
}

cudaError_t launch(void (*kern)(Args), Args& a, const Plan& p, cudaStream_t s) {
  const cudaError_t e = moe::set_smem_once(reinterpret_cast<const void*>(kern), 216 << 10);
  if (e != cudaSuccess) return e;
  a.slots = p.slots;
  a.slot_bytes = p.slot_bytes;
  return launch_early(kern, p.blocks, p.threads, p.smem, s, a);
}

moe_status check(const moe_norm_dims* d) {
  if (!d || d->T < 0 || d->h <= 0) return MOE_ERR_INVALID_ARG;
  if (d->res_f32 != 0 && d->res_f32 != 1) return MOE_ERR_INVALID_ARG;
  if (d->gate < MOE_GATE_NONE || d->gate > MOE_GATE_TOKEN) return MOE_ERR_INVALID_ARG;
  if (!(d->eps > 0.f) || !std::isfinite(d->eps) || !std::isfinite(d->alpha) ||
      !std::isfinite(d->beta))
    return MOE_ERR_INVALID_ARG;
  if (d->h % 8 != 0 || d->h > kMaxH) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// present and aligned where wanted, NULL where not
bool is(const void* p, bool wanted) { return wanted ? p && aligned16(p) : p == nullptr; }

Args args_of(const moe_norm_dims& d, const void* r, const moe_bf16* y, const float* w_post,
             const float* gate, const float* w_pre) {
  Args a = {};
  a.r = r;
  a.y = y;
  a.w_post = w_post;
  a.gate_kind = y ? d.gate : MOE_GATE_NONE;
  a.gate = a.gate_kind ? gate : nullptr;
  a.w_pre = w_pre;
  a.T = d.T;
  a.h = d.h;
  a.eps = d.eps;
  a.alpha = d.alpha;
  a.beta = d.beta;
  a.inv_h = 1.0f / static_cast<float>(d.h);
  return a;
}

}  // namespace

extern "C" {

size_t moe_norm_workspace_bytes(const moe_norm_dims* dims) {
  if (check(dims) != MOE_OK) return 0;
  const size_t n =
      static_cast<size_t>(plan_of(*dims, true).most_blocks) * 2 * dims->h * sizeof(float);
  return kAlign + (n + kAlign - 1) / kAlign * kAlign;
}

moe_status moe_block_norm_fwd(const moe_norm_dims* dims, const void* r, const moe_bf16* y,
                              const float* w_post, const float* gate, const float* w_pre,
                              void* r_out, moe_bf16* u, moe_stream_t stream) {
  const moe_status st = check(dims);
  if (st != MOE_OK) return st;
  const moe_norm_dims& d = *dims;
  if (d.T == 0) return MOE_OK;  // empty tensors: which parts are present cannot be told
  if (!y && (w_post || !w_pre)) return MOE_ERR_INVALID_ARG;
  if (!is(r, true) || !aligned16(y) || !aligned16(w_post) || !aligned16(w_pre) ||
      !is(r_out, y != nullptr) || !is(u, w_pre != nullptr))
    return MOE_ERR_INVALID_ARG;
  if (y && d.gate != MOE_GATE_NONE && !is(gate, true)) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  Args a = args_of(d, r, y, w_post, gate, w_pre);
  a.out_r = r_out;
  a.out_u = reinterpret_cast<uint4*>(u);
  a.status = moe::nows_status_word();
  if (!a.status) return moe_api::cuda_error();
  const Plan p = plan_of(d, false);
  const cudaError_t e = launch(d.res_f32 ? fwd_kernel<true>(p) : fwd_kernel<false>(p), a, p, s);
  return e == cudaSuccess && moe_api::note(s, "block_norm_fwd") ? MOE_OK : moe_api::cuda_error();
}

moe_status moe_block_norm_bwd(const moe_norm_dims* dims, const void* r_out, const moe_bf16* y,
                              const float* w_post, const float* gate, const float* w_pre,
                              const moe_bf16* du, const void* dr_out, void* dr, moe_bf16* dy,
                              float* dw_post, float* dgate, float* dw_pre, void* ws,
                              size_t ws_bytes, moe_stream_t stream) {
  const moe_status st = check(dims);
  if (st != MOE_OK) return st;
  const moe_norm_dims& d = *dims;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (d.T == 0) {  // sums over no rows (a token gate's gradient has no elements)
    float* const sums[3] = {dw_post, dw_pre, d.gate == MOE_GATE_CHANNEL ? dgate : nullptr};
    for (float* p : sums) {
      if (!aligned16(p)) return MOE_ERR_INVALID_ARG;
      if (p && cudaMemsetAsync(p, 0, static_cast<size_t>(d.h) * sizeof(float), s) != cudaSuccess)
        return moe_api::cuda_error();
    }
    return MOE_OK;
  }
  const bool post = y != nullptr, gated = post && d.gate != MOE_GATE_NONE;
  if (!post && (w_post || !w_pre)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(y) || !aligned16(w_post) || !aligned16(w_pre) || !aligned16(dr_out) ||
      !aligned16(r_out) || (w_pre && !is(r_out, true)) || !is(du, w_pre != nullptr) ||
      !is(dr, true) || !is(dy, post) || !is(dw_post, w_post != nullptr) ||
      !is(dw_pre, w_pre != nullptr) || !is(dgate, gated) || (gated && !is(gate, true)))
    return MOE_ERR_INVALID_ARG;
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & (kAlign - 1))) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < moe_norm_workspace_bytes(dims)) return MOE_ERR_WORKSPACE;
  Args a = args_of(d, r_out, y, w_post, gate, w_pre);
  a.du = du;
  a.dr_out = dr_out;
  a.out_r = dr;
  a.out_u = reinterpret_cast<uint4*>(dy);
  a.dgate = a.gate_kind == MOE_GATE_TOKEN ? dgate : nullptr;
  a.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kAlign);
  a.status = static_cast<int*>(ws);
  const Plan p = plan_of(d, true);
  const bool all = y && w_post && w_pre && dr_out;
  const cudaError_t e =
      launch(d.res_f32 ? bwd_kernel<true>(p, all) : bwd_kernel<false>(p, all), a, p, s);
  if (e != cudaSuccess || !moe_api::note(s, "block_norm_bwd")) return moe_api::cuda_error();
  const bool channel = a.gate_kind == MOE_GATE_CHANNEL;
  if (dw_pre || dw_post || channel) {
    const int cols = d.h > 16 * moe_api::num_sms() ? 16 : 8;
    if (launch_early(cols == 8 ? block_norm_cols_kernel<8> : block_norm_cols_kernel<16>,
                     (d.h + cols - 1) / cols, kColThreads, 0, s, a.partial, p.blocks, d.h, w_post,
                     channel ? gate : nullptr, d.beta, dw_pre, dw_post,
                     channel ? dgate : nullptr) != cudaSuccess ||
        !moe_api::note(s, "block_norm_cols"))
      return moe_api::cuda_error();
  }
  return MOE_OK;
}

}  // extern "C"
