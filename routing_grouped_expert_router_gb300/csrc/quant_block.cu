// quant_block.cu -- e4m3 codes with a float32 scale for each block of 128: rows
// in 1 x 128 blocks, weights in 128 x 128 blocks.  s = amax / 448 (1 for zeros),
// q = e4m3(v / s); the quotient is the IEEE one (block_quant.cuh).
//
// Both read their input once: a block's values wait in registers for its
// maximum.  HBM bounds them: 3 bytes an element and the scales.  Measured: eight weights of
// 4096 x 14336, 203 us, as fast as a copy; 16384 x 4096 rows, each gathered twice,
// 62 us, 41 at the copy bandwidth with each source row read once (60 with it read twice).
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/moe.h"
#include "api_internal.h"
#include "block.cuh"
#include "block_quant.cuh"
#include "kernels.cuh"

namespace moe {

namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kRowThreads = 128;
constexpr int kRowAhead = 2;  // blocks of a lane under way, 32 bytes of each

__device__ __forceinline__ void codes8(const uint4& w, const BlockScale& b, uint2& out) {
  const float lo[4] = {__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u),
                       __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u)};
  const float hi[4] = {__uint_as_float(w.z << 16), __uint_as_float(w.z & 0xFFFF0000u),
                       __uint_as_float(w.w << 16), __uint_as_float(w.w & 0xFFFF0000u)};
  out = make_uint2(codes4(lo, b), codes4(hi, b));
}
// The larger magnitudes of the low and of the high values, each in its half.
__device__ __forceinline__ uint32_t top8(const uint4& w) {
  return top_2(top_2(top_2(w.x & 0x7FFF7FFFu, w.y), w.z), w.w);
}

// A warp takes a row's blocks four at a time, eight lanes of two 16-byte pieces to a
// block, with kRowAhead such quads under way: sixteen values share the arithmetic of a
// block's scale, which with eight took as many instructions as all else (16384 x 4096
// rows gathered twice: 90 us); with quotients and maxima of one value at a time it was 70.
// blockIdx.y splits a row's quads where there are too few rows to fill the GPU.
__global__ void __launch_bounds__(kRowThreads) quant_rows_block_kernel(
    const uint4* __restrict__ in, const int32_t* __restrict__ idx, int div, long long rows,
    long long src_rows, const int32_t* __restrict__ ends, int n_ends, int n8, int quads,
    int quads_each, uint2* __restrict__ q, float* __restrict__ scale, uint4* __restrict__ copy,
    int* __restrict__ status) {
  // The kernel before may have written what is read here.  The next one may start once all
  // before this one are done: it can read what neither this one nor itself writes.
  cudaGridDependencySynchronize();
  cudaTriggerProgrammaticLaunchCompletion();
  const int lane = threadIdx.x & 31;
  const long long warp0 = (static_cast<long long>(blockIdx.x) * kRowThreads + threadIdx.x) >> 5;
  const long long warps = (static_cast<long long>(gridDim.x) * kRowThreads) >> 5;
  const long long ld = rows;  // of the scales
  long long last = rows;
  if (ends) {
    // the furthest end, as group_tables clamps the groups: offsets out of order leave no row
    // that a product takes without codes
    int top = lane < n_ends ? __ldg(ends + lane) : 0;  // n_ends: at most 65
    if (n_ends > 32 && lane + 32 < n_ends) top = max(top, __ldg(ends + lane + 32));
    if (n_ends > 64) top = max(top, __ldg(ends + 64));
    top = max(top, 0);
    last = min(static_cast<long long>(__reduce_max_sync(kFull, top)), rows);
  }
  const int first_quad = blockIdx.y * quads_each;
  const int end_quad = min(first_quad + quads_each, quads);
  const int c0 = (lane >> 3) * 16 + (lane & 7);  // this lane's first piece of a quad; then + 8
  for (long long p = warp0; p < last; p += warps) {
    long long src = p;
    if (idx) {
      const int32_t a = __ldg(idx + p);
      src = a < 0 ? -1 : a / div;
    }
    const bool bad = src < 0 || src >= src_rows;
    if (bad && lane == 0 && blockIdx.y == 0) report_bad_index(status);
    const uint4* from = in + (bad ? 0 : src) * n8;
    for (int j0 = first_quad; j0 < end_quad; j0 += kRowAhead) {
      uint4 w[kRowAhead][2];
#pragma unroll
      for (int i = 0; i < kRowAhead; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c = (j0 + i) * 64 + c0 + 8 * h;
          w[i][h] = (!bad && j0 + i < end_quad && c < n8) ? __ldg(from + c) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
      for (int i = 0; i < kRowAhead; ++i) {
        if (j0 + i >= end_quad) break;  // the same for the whole warp
        uint32_t top = top_of_2(top_2(top8(w[i][0]), top8(w[i][1])));
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(kFull, top, o));
        const BlockScale b = block_scale(top);
        const int c = (j0 + i) * 64 + c0;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (c + 8 * h < n8) {
            uint2 codes;
            codes8(w[i][h], b, codes);
            // written to be evicted first: the source's rows, read again, stay in L2 longer (64 to 62 us)
            __stcs(q + p * n8 + c + 8 * h, codes);
            if (copy) copy[p * n8 + c + 8 * h] = w[i][h];
          }
        if ((lane & 7) == 0 && c < n8) scale[static_cast<long long>(c >> 4) * ld + p] = b.s;
      }
    }
  }
}

// One 128 x 128 block of one weight to a block of 256 threads: 16 lanes along a
// row's 128 values, 16 rows at a time, eight 16-byte loads a lane under way.
constexpr int kWeightThreads = 256;
__global__ void __launch_bounds__(kWeightThreads) quant_weights_block_kernel(
    const uint4* __restrict__ W, int K, int n8, int kb, int nb, uint2* __restrict__ q,
    float* __restrict__ scale) {
  __shared__ uint32_t tops[kWeightThreads / 32];
  const long long tile = blockIdx.x;
  const int jn = static_cast<int>(tile % nb);
  const long long ek = tile / nb;
  const int jk = static_cast<int>(ek % kb);
  const long long e = ek / kb;
  const int c = jn * 16 + (threadIdx.x & 15);
  const int r0 = jk * kBlock + (threadIdx.x >> 4);
  const long long base = (e * K + r0) * n8 + c;
  uint4 w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    w[i] = (c < n8 && r0 + 16 * i < K) ? __ldg(W + base + 16ll * i * n8) : make_uint4(0, 0, 0, 0);
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = top_2(top, top8(w[i]));
  top = top_of_2(top);
  top = __reduce_max_sync(kFull, top);
  if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kWeightThreads / 32; ++i) top = max(top, tops[i]);
  const BlockScale b = block_scale(top);
  if (threadIdx.x == 0) scale[tile] = b.s;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c < n8 && r0 + 16 * i < K) {
      uint2 codes;
      codes8(w[i], b, codes);
      __stcs(q + base + 16ll * i * n8, codes);
    }
}

}  // namespace

cudaError_t launch_quant_rows_block(const uint16_t* in, const int32_t* idx, int div,
                                    long long rows, long long src_rows, int n, uint8_t* q,
                                    float* scale, int num_sms, cudaStream_t s,
                                    const int32_t* ends, int n_ends, uint16_t* copy,
                                    int* status) {
  if (rows == 0) return cudaSuccess;
  const int quads = (n + 4 * kBlock - 1) / (4 * kBlock);
  const long long row_blocks = (rows + kRowThreads / 32 - 1) / (kRowThreads / 32);
  const long long cap = 16ll * num_sms;
  const int gx = static_cast<int>(row_blocks < cap ? row_blocks : cap);
  // a row's quads over several blocks while the rows alone do not fill the SMs
  int split = static_cast<int>((cap + gx - 1) / gx);
  if (split > quads) split = quads;
  const int each = (quads + split - 1) / split;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(gx, (quads + each - 1) / each, 1);
  cfg.blockDim = dim3(kRowThreads, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(
      &cfg, quant_rows_block_kernel, reinterpret_cast<const uint4*>(in), idx, idx ? div : 1, rows,
      src_rows, ends, n_ends, n / 8, quads, each, reinterpret_cast<uint2*>(q), scale,
      reinterpret_cast<uint4*>(copy), status);
  return e == cudaSuccess ? launched() : e;
}

cudaError_t launch_quant_weights_block(const uint16_t* W, int E, int K, int N, uint8_t* q,
                                       float* scale, cudaStream_t s) {
  const int kb = blocks_of(K), nb = blocks_of(N);
  const long long tiles = static_cast<long long>(E) * kb * nb;
  quant_weights_block_kernel<<<static_cast<unsigned>(tiles), kWeightThreads, 0, s>>>(
      reinterpret_cast<const uint4*>(W), K, N / 8, kb, nb, reinterpret_cast<uint2*>(q), scale);
  return launched();
}

}  // namespace moe

// =================================================================== C ABI
namespace {
bool ptr_ok(const void* p) { return p && reinterpret_cast<uintptr_t>(p) % 16 == 0; }
// The longest side: with a step of the kernels (four blocks of 128) on top it fits 31 bits.
constexpr int32_t kMostSide = 2147483647 - 511;
}  // namespace

extern "C" {

moe_status moe_quantize_rows_fp8_block(const moe_bf16* in, int64_t rows, int32_t n,
                                       const int32_t* idx, int32_t div, int64_t src_rows,
                                       uint8_t* q, float* scale, moe_stream_t stream) {
  if (rows < 0 || src_rows < 0 || n <= 0 || n % 16 != 0 || (idx && div <= 0))
    return MOE_ERR_INVALID_ARG;
  if (n > kMostSide) return MOE_ERR_UNSUPPORTED;
  if (rows > 0 && (!ptr_ok(in) || !ptr_ok(q) || !ptr_ok(scale) || (idx && !ptr_ok(idx))))
    return MOE_ERR_INVALID_ARG;
  if (rows > 0 && !idx && src_rows < rows) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  int* status = moe::nows_status_word();
  if (!status) return moe_api::cuda_error();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (moe::launch_quant_rows_block(in, idx, div, rows, src_rows, n, q, scale, moe_api::num_sms(),
                                   s, nullptr, 0, nullptr, status) != cudaSuccess ||
      !moe_api::note(s, "quant_rows_block"))
    return moe_api::cuda_error();
  return MOE_OK;
}

moe_status moe_quantize_weights_fp8_block(const moe_bf16* W, int32_t E, int32_t K, int32_t N,
                                          uint8_t* q, float* scale, moe_stream_t stream) {
  if (E <= 0 || K <= 0 || N <= 0 || K % 16 != 0 || N % 16 != 0) return MOE_ERR_INVALID_ARG;
  if (K > kMostSide || N > kMostSide ||
      static_cast<double>(E) * moe::blocks_of(K) * moe::blocks_of(N) > 2147483647.0)
    return MOE_ERR_UNSUPPORTED;
  if (!ptr_ok(W) || !ptr_ok(q) || !ptr_ok(scale)) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (moe::launch_quant_weights_block(W, E, K, N, q, scale, s) != cudaSuccess ||
      !moe_api::note(s, "quant_weights_block"))
    return moe_api::cuda_error();
  return MOE_OK;
}

}  // extern "C"
