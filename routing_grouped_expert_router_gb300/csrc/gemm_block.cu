// gemm_block.cu -- grouped products of e4m3 codes with a float32 scale for each
// block of 128 (see block.cuh):
//   C[p, n] = sum_b sa[b, p] sb[e, b, n/128] sum_{k in block b} qa[p, k] qb[e, k, n]
// in four forms: the plain product, FC1 with SwiGLU and H's codes, FC2's data
// gradient with the SwiGLU backward and its codes, and FC1's data gradient (two
// products in one sum).
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "block.cuh"
#include "block_quant.cuh"
#include "kernels.cuh"

namespace moe {

namespace {

enum Form { PLAIN_BF16 = 0, PLAIN_F32 = 1, GATED = 2, GATED_BWD = 3 };

struct SimpleParams {
  BlockRows r;
  const uint8_t* a[2];   // activations' codes (the second: a second product in the same sum)
  const float* sa[2];
  const uint8_t* b[2];   // weights' codes (the second: W3, or that of the second product)
  const float* sb[2];
  int K, N, products;
  int trans;
  void* out[3];
  const uint16_t* in[2];
  uint8_t* codes[2];
  float* scales[2];
};

__device__ __forceinline__ float code_value(uint8_t c) {
  __nv_fp8_e4m3 v;
  v.__x = c;
  return static_cast<float>(v);
}

constexpr int TM = 32, TN = 128, TK = 32;

template <int FORM>
__global__ void __launch_bounds__(256) simple_kernel(SimpleParams p) {
  constexpr int NB = FORM == GATED ? 2 : 1;
  __shared__ float As[TM][TK + 1];
  __shared__ float Bs[NB][TK][TN];
  // this block's group and rows
  int e = 0, row0 = 0, row_end = 0, before = 0;
  bool found = false, bad = false;
  int lo = 0;
  for (int i = 0; i < p.r.E; ++i) {
    const int o0 = p.r.offsets ? p.r.offsets[i] : 0;
    const int o1 = p.r.offsets ? p.r.offsets[i + 1] : p.r.rows;
    if ((i == 0 && o0 != 0) || o1 < o0 || o1 > p.r.rows) bad = true;
    if (i == 0) lo = min(max(o0, 0), p.r.rows);
    const int hi = max(lo, min(max(o1, 0), p.r.rows));
    const int tiles = (hi - lo + TM - 1) / TM;
    if (!found && static_cast<int>(blockIdx.y) < before + tiles) {
      found = true;
      e = i;
      row0 = lo + (blockIdx.y - before) * TM;
      row_end = hi;
    }
    before += tiles;
    lo = hi;
  }
  if (bad && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) report_bad_index(p.r.status);
  if (!found) return;
  const int n0 = blockIdx.x * TN;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int kb = (p.K + 127) / 128, nb = (p.N + 127) / 128;
  float acc[NB][2][8];
#pragma unroll
  for (int o = 0; o < NB; ++o)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[o][i][j] = 0.f;
  for (int prod = 0; prod < p.products; ++prod) {
    const uint8_t* A = p.a[prod];
    const float* sa = p.sa[prod];
    for (int b = 0; b < kb; ++b) {
      float part[NB][2][8];
#pragma unroll
      for (int o = 0; o < NB; ++o)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) part[o][i][j] = 0.f;
      for (int k0 = b * 128; k0 < min(p.K, b * 128 + 128); k0 += TK) {
        __syncthreads();
        for (int i = threadIdx.x; i < TM * TK; i += 256) {
          const int r = row0 + i / TK, k = k0 + i % TK;
          As[i / TK][i % TK] =
              (r < row_end && k < p.K) ? code_value(A[static_cast<size_t>(r) * p.K + k]) : 0.f;
        }
#pragma unroll
        for (int o = 0; o < NB; ++o) {
          const uint8_t* B = p.b[FORM == GATED ? o : prod] + static_cast<size_t>(e) * p.K * p.N;
          for (int i = threadIdx.x; i < TK * TN; i += 256) {
            const int kk = p.trans ? i % TK : i / TN, nn = p.trans ? i / TK : i % TN;
            const int k = k0 + kk, n = n0 + nn;
            Bs[o][kk][nn] = (k < p.K && n < p.N)
                                ? code_value(B[p.trans ? static_cast<size_t>(n) * p.K + k
                                                       : static_cast<size_t>(k) * p.N + n])
                                : 0.f;
          }
        }
        __syncthreads();
        for (int kk = 0; kk < TK; ++kk)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float a = As[ty * 2 + i][kk];
#pragma unroll
            for (int o = 0; o < NB; ++o)
#pragma unroll
              for (int j = 0; j < 8; ++j)
                part[o][i][j] = fmaf(a, Bs[o][kk][tx * 8 + j], part[o][i][j]);
          }
      }
#pragma unroll
      for (int o = 0; o < NB; ++o) {
        const float* sb = p.sb[FORM == GATED ? o : prod] + static_cast<size_t>(e) * kb * nb;
        const float sw = p.trans ? sb[blockIdx.x * kb + b] : sb[b * nb + blockIdx.x];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = row0 + ty * 2 + i;
          const float sc = r < row_end ? sa[static_cast<size_t>(b) * p.r.rows + r] * sw : 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[o][i][j] = fmaf(part[o][i][j], sc, acc[o][i][j]);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = row0 + ty * 2 + i;
    const bool row_ok = r < row_end;
    const size_t at = static_cast<size_t>(r) * p.N + n0 + tx * 8;
    if constexpr (FORM == PLAIN_BF16 || FORM == PLAIN_F32) {
      for (int j = 0; j < 8; ++j)
        if (row_ok && n0 + tx * 8 + j < p.N) {
          if (FORM == PLAIN_F32)
            static_cast<float*>(p.out[0])[at + j] = acc[0][i][j];
          else
            static_cast<__nv_bfloat16*>(p.out[0])[at + j] = __float2bfloat16_rn(acc[0][i][j]);
        }
    } else {
      __nv_bfloat16 v[2][8];
      uint32_t top[2] = {0, 0};
      for (int j = 0; j < 8; ++j) {
        const bool ok = row_ok && n0 + tx * 8 + j < p.N;
        v[0][j] = v[1][j] = __float2bfloat16_rn(0.f);
        if (!ok) continue;
        if constexpr (FORM == GATED) {
          const float a = acc[0][i][j], b = acc[NB - 1][i][j];
          v[0][j] = __float2bfloat16_rn(a / (1.f + expf(-a)) * b);
          if (p.out[0]) {
            static_cast<__nv_bfloat16*>(p.out[0])[at + j] = __float2bfloat16_rn(a);
            static_cast<__nv_bfloat16*>(p.out[1])[at + j] = __float2bfloat16_rn(b);
            static_cast<__nv_bfloat16*>(p.out[2])[at + j] = v[0][j];
          }
        } else {
          const float dh = acc[0][i][j];
          const float a = __uint_as_float(static_cast<uint32_t>(p.in[0][at + j]) << 16);
          const float b = __uint_as_float(static_cast<uint32_t>(p.in[1][at + j]) << 16);
          const float s = 1.f / (1.f + expf(-a));
          v[0][j] = __float2bfloat16_rn(dh * b * s * (1.f + a * (1.f - s)));
          v[1][j] = __float2bfloat16_rn(dh * a * s);
          static_cast<__nv_bfloat16*>(p.out[0])[at + j] = v[0][j];
          static_cast<__nv_bfloat16*>(p.out[1])[at + j] = v[1][j];
        }
        for (int o = 0; o < 2; ++o)
          top[o] = max(top[o], __float_as_uint(__bfloat162float(v[o][j])) & 0x7FFFFFFFu);
      }
      for (int o = 0; o < (FORM == GATED ? 1 : 2); ++o) {
        for (int m = 8; m > 0; m >>= 1)
          top[o] = max(top[o], __shfl_xor_sync(0xFFFFFFFFu, top[o], m));
        const BlockScale bs = block_scale(top[o]);
        if (row_ok && tx == 0)
          p.scales[o][static_cast<size_t>(blockIdx.x) * p.r.rows + r] = bs.s;
        for (int j = 0; j < 8; j += 4) {
          const float f4[4] = {__bfloat162float(v[o][j]), __bfloat162float(v[o][j + 1]),
                               __bfloat162float(v[o][j + 2]), __bfloat162float(v[o][j + 3])};
          if (row_ok && n0 + tx * 8 + j < p.N)
            *reinterpret_cast<uint32_t*>(p.codes[o] + at + j) = codes4(f4, bs);
        }
      }
    }
  }
}

template <int FORM>
cudaError_t run_simple(const SimpleParams& p, cudaStream_t s) {
  if (p.r.rows == 0) return cudaSuccess;
  const dim3 grid((p.N + TN - 1) / TN, (p.r.rows + TM - 1) / TM + p.r.E, 1);
  simple_kernel<FORM><<<grid, 256, 0, s>>>(p);
  return launched();
}

}  // namespace

cudaError_t block_product(const BlockRows& r, const Coded& a, const Coded& b, int K, int N,
                          bool trans, bool out_f32, void* C, cudaStream_t s) {
  SimpleParams p = {};
  p.r = r;
  p.a[0] = a.q;
  p.sa[0] = a.s;
  p.b[0] = b.q;
  p.sb[0] = b.s;
  p.K = K;
  p.N = N;
  p.products = 1;
  p.trans = trans;
  p.out[0] = C;
  return out_f32 ? run_simple<PLAIN_F32>(p, s) : run_simple<PLAIN_BF16>(p, s);
}

cudaError_t block_fc1_fwd(const BlockRows& r, const Coded& x, const Coded& w1, const Coded& w3,
                          int h, int f, uint16_t* A, uint16_t* B, uint16_t* H, uint8_t* Hq,
                          float* sh, cudaStream_t s) {
  SimpleParams p = {};
  p.r = r;
  p.a[0] = x.q;
  p.sa[0] = x.s;
  p.b[0] = w1.q;
  p.sb[0] = w1.s;
  p.b[1] = w3.q;
  p.sb[1] = w3.s;
  p.K = h;
  p.N = f;
  p.products = 1;
  p.out[0] = A;
  p.out[1] = B;
  p.out[2] = H;
  p.codes[0] = Hq;
  p.scales[0] = sh;
  return run_simple<GATED>(p, s);
}

cudaError_t block_fc2_dgrad(const BlockRows& r, const Coded& dy, const Coded& w2, int h, int f,
                            const uint16_t* A, const uint16_t* B, uint16_t* dA, uint16_t* dB,
                            uint8_t* dAq, float* sda, uint8_t* dBq, float* sdb, cudaStream_t s) {
  SimpleParams p = {};
  p.r = r;
  p.a[0] = dy.q;
  p.sa[0] = dy.s;
  p.b[0] = w2.q;
  p.sb[0] = w2.s;
  p.K = h;
  p.N = f;
  p.products = 1;
  p.trans = 1;
  p.in[0] = A;
  p.in[1] = B;
  p.out[0] = dA;
  p.out[1] = dB;
  p.codes[0] = dAq;
  p.scales[0] = sda;
  p.codes[1] = dBq;
  p.scales[1] = sdb;
  return run_simple<GATED_BWD>(p, s);
}

cudaError_t block_fc1_dgrad(const BlockRows& r, const Coded& da, const Coded& db, const Coded& w1,
                            const Coded& w3, int h, int f, bool out_f32, void* dX,
                            cudaStream_t s) {
  SimpleParams p = {};
  p.r = r;
  p.a[0] = da.q;
  p.sa[0] = da.s;
  p.a[1] = db.q;
  p.sa[1] = db.s;
  p.b[0] = w1.q;
  p.sb[0] = w1.s;
  p.b[1] = w3.q;
  p.sb[1] = w3.s;
  p.K = f;
  p.N = h;
  p.products = 2;
  p.trans = 1;
  p.out[0] = dX;
  return out_f32 ? run_simple<PLAIN_F32>(p, s) : run_simple<PLAIN_BF16>(p, s);
}

}  // namespace moe
