// block.cuh -- e4m3 operands with a float32 scale for each block of 128: the
// host-side interface of the quantisers (quant_block.cu) and of the grouped
// products (gemm_block.cu), and the device code that both quantise with.
//
// Activations [R, n]: codes in rows, scales [ceil(n/128), R] (block-major, so
// that a tile's rows read theirs as consecutive floats).  Weights [E, K, N]:
// codes in the weight's own layout, scales [E, ceil(K/128), ceil(N/128)].
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "block_order.h"

namespace moe {

// Rows of `in` (row idx[p] / div, or p) -> codes [rows, n] and block scales
// [ceil(n/128), rows], for p < rows (and, where given, p < the largest of
// ends[0 .. n_ends-1], at most 65: the groups' offsets, or their last alone where they are known
// to be in order).  With copy, the bf16 source rows are also written to copy [rows, n].
// n a multiple of 16.
cudaError_t launch_quant_rows_block(const uint16_t* in, const int32_t* idx, int div,
                                    long long rows, long long src_rows, int n, uint8_t* q,
                                    float* scale, int num_sms, cudaStream_t s,
                                    const int32_t* ends, int n_ends, uint16_t* copy,
                                    int* status);
// Weights [E, K, N] -> codes [E, K, N] and scales [E, ceil(K/128), ceil(N/128)].
cudaError_t launch_quant_weights_block(const uint16_t* W, int E, int K, int N, uint8_t* q,
                                       float* scale, cudaStream_t s);

// The rows of a grouped product: group e's are offsets[e] .. offsets[e+1] - 1
// (all rows where offsets is NULL and E = 1).
struct BlockRows {
  int E;
  const int32_t* offsets;
  int rows;
  int* status;    // device status word, at the start of the workspace's 256-byte header
  int num_sms;
  float* part;    // part_bytes(rows) bytes for the sums of tiles that several blocks share
};
constexpr int kPartBlocks = 160;  // blocks of a grid that have room for a shared tile's sums
inline size_t part_bytes(int rows) {  // 128 x 256 sums for each: the most of either kernel
  return rows ? static_cast<size_t>(kPartBlocks) * 128 * 256 * 4 : 0;
}
// Codes and scales of an activation or a weight.
struct Coded {
  const uint8_t* q;
  const float* s;
};
// C = A B[e] (trans: A B[e]^T, B [E, N, K]); C [rows, N] bf16 or fp32.
// ahead: the launch just before on the stream is one of block_fc1_fwd, so that weights and
// offsets may be read before it ends (few rows).
cudaError_t block_product(const BlockRows& r, const Coded& a, const Coded& b, int K, int N,
                          bool trans, bool out_f32, void* C, cudaStream_t s, bool ahead = false);
// A = X W1, B = X W3, H = silu(A) * B with the codes of bf16(H); A, B, H may be NULL.
// The launch just before on the stream is launch_quant_rows_block's of x.
cudaError_t block_fc1_fwd(const BlockRows& r, const Coded& x, const Coded& w1, const Coded& w3,
                          int h, int f, uint16_t* A, uint16_t* B, uint16_t* H, uint8_t* Hq,
                          float* sh, cudaStream_t s);
// The same for few rows.
cudaError_t few_product(const BlockRows& r, const Coded& a, const Coded& b, int K, int N,
                        bool trans, bool out_f32, void* C, cudaStream_t s, bool ahead);
cudaError_t few_fc1_fwd(const BlockRows& r, const Coded& x, const Coded& w1, const Coded& w3,
                        int h, int f, uint16_t* A, uint16_t* B, uint16_t* H, uint8_t* Hq,
                        float* sh, cudaStream_t s);
// dH = dY W2^T, fused with the SwiGLU backward: dA, dB in bf16 and their codes.
cudaError_t block_fc2_dgrad(const BlockRows& r, const Coded& dy, const Coded& w2, int h, int f,
                            const uint16_t* A, const uint16_t* B, uint16_t* dA, uint16_t* dB,
                            uint8_t* dAq, float* sda, uint8_t* dBq, float* sdb, cudaStream_t s);
// dX = dA W1^T + dB W3^T, bf16 or fp32 [rows, h].
cudaError_t block_fc1_dgrad(const BlockRows& r, const Coded& da, const Coded& db, const Coded& w1,
                            const Coded& w3, int h, int f, bool out_f32, void* dX,
                            cudaStream_t s);

}  // namespace moe
