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

constexpr int kBlock = 128;
inline int blocks_of(int n) { return (n + kBlock - 1) / kBlock; }

// Rows of `in` (row idx[p] / div, or p) -> codes [rows, n] and block scales
// [ceil(n/128), rows], for p < rows (and, where given, p < the largest of
// ends[0 .. n_ends-1]: the groups' offsets, or their last alone where they are known
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
