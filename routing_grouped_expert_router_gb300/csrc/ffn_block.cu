// ffn_block.cu -- entry points of the block-scaled e4m3 product and of the gated
// feed-forward block built from it (include/moe.h): argument checks, the
// workspace's layout and the order of the kernels.  Host code only.
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/moe.h"
#include "api_internal.h"
#include "block.cuh"
#include "grouped_gemm.cuh"
#include "kernels.cuh"

namespace {

constexpr size_t kAlign = 256;

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool ptr_ok(const void* p) { return p && aligned(p, 16); }
// A buffer of `n` elements: may be NULL only when it is empty.
bool buf_ok(const void* p, size_t n) { return n == 0 ? aligned(p, 16) : ptr_ok(p); }

struct Carve {
  size_t off = 0;
  size_t take(size_t bytes) {
    const size_t o = off;
    off += (bytes + kAlign - 1) / kAlign * kAlign;
    return o;
  }
};
template <class T>
T* at(void* base, size_t off) {
  return reinterpret_cast<T*>(static_cast<uint8_t*>(base) + off);
}

// Tiles of one launch are counted in 31 bits.
bool tiles_fit(int rows, int E, int n) {
  return (static_cast<double>(rows) / 16 + E) * (static_cast<double>(n) / 64 + 1) < 2147483647.0;
}

moe_status check_gemm(const moe_gemm_dims* d) {
  if (!d || d->rows < 0 || d->K <= 0 || d->N <= 0 || d->E <= 0) return MOE_ERR_INVALID_ARG;
  if ((d->trans_b | 1) != 1 || (d->out_f32 | 1) != 1) return MOE_ERR_INVALID_ARG;
  if (d->rows > moe::kMostRows || d->E > 64 || d->K % 16 != 0 || d->N % 16 != 0 ||
      d->K > moe::kMostWidth || d->N > moe::kMostWidth || !tiles_fit(d->rows, d->E, d->N))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status check_ffn(const moe_ffn_dims* d) {
  if (!d || d->rows < 0 || d->h <= 0 || d->f <= 0 || d->E <= 0 || (d->dw_bf16 | 1) != 1)
    return MOE_ERR_INVALID_ARG;
  if (d->rows > moe::kMostRows || d->E > 64 || d->h % 64 != 0 || d->f % 64 != 0 ||
      d->h > moe::kMostWidth || d->f > moe::kMostWidth || !tiles_fit(d->rows, d->E, d->h) ||
      !tiles_fit(d->rows, d->E, d->f))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

struct FfnLayout {
  size_t status = 0;
  size_t Xq = 0, sx = 0;                 // the rows' codes (of x, or of dy in the backward)
  size_t Hq = 0, sh = 0;                 // forward
  size_t dA = 0, dB = 0;                 // backward
  size_t dAq = 0, sda = 0, dBq = 0, sdb = 0;
  size_t part = 0;                       // shared tiles' sums
  size_t total = 0;
};
FfnLayout ffn_layout(const moe_ffn_dims& d, bool backward) {
  const size_t R = d.rows, hb = moe::blocks_of(d.h), fb = moe::blocks_of(d.f);
  Carve c;
  FfnLayout L;
  L.status = c.take(kAlign);
  L.Xq = c.take(R * d.h);
  L.sx = c.take(R * hb * 4);
  if (!backward) {
    L.Hq = c.take(R * d.f);
    L.sh = c.take(R * fb * 4);
    L.part = c.take(moe::part_bytes(d.rows));
  } else {
    L.dA = c.take(R * d.f * 2);
    L.dB = c.take(R * d.f * 2);
    L.dAq = c.take(R * d.f);
    L.sda = c.take(R * fb * 4);
    L.dBq = c.take(R * d.f);
    L.sdb = c.take(R * fb * 4);
    L.part = c.take(moe::part_bytes(d.rows));
  }
  L.total = c.off;
  return L;
}

#define BLOCK_RUN(expr, name)                                       \
  do {                                                              \
    if ((expr) != cudaSuccess) return moe_api::cuda_error();        \
    if (!moe_api::note(stream, name)) return moe_api::cuda_error(); \
  } while (0)

}  // namespace

extern "C" {

size_t moe_gemm_workspace_bytes(const moe_gemm_dims* dims) {
  if (check_gemm(dims) != MOE_OK) return 0;
  return kAlign + moe::part_bytes(dims->rows);
}

moe_status moe_gemm_fp8_block(const moe_gemm_dims* dims, const uint8_t* aq, const float* sa,
                              const uint8_t* bq, const float* sb, const int32_t* offsets, void* C,
                              void* ws, size_t ws_bytes, moe_stream_t stream_) {
  const moe_status st = check_gemm(dims);
  if (st != MOE_OK) return st;
  const moe_gemm_dims& d = *dims;
  const size_t R = d.rows;
  if (!buf_ok(aq, R) || !buf_ok(sa, R) || !ptr_ok(bq) || !ptr_ok(sb) || !buf_ok(C, R) ||
      (offsets ? !ptr_ok(offsets) : d.E != 1) || !ws || !aligned(ws, kAlign))
    return MOE_ERR_INVALID_ARG;
  if (ws_bytes < moe_gemm_workspace_bytes(dims)) return MOE_ERR_WORKSPACE;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  const moe::BlockRows r = {d.E, offsets, d.rows, at<int>(ws, 0), moe_api::num_sms(),
                            at<float>(ws, kAlign)};
  BLOCK_RUN(moe::block_product(r, {aq, sa}, {bq, sb}, d.K, d.N, d.trans_b != 0, d.out_f32 != 0, C,
                               stream),
            "block_product");
  return MOE_OK;
}

size_t moe_ffn_workspace_bytes(const moe_ffn_dims* dims, int backward) {
  if (check_ffn(dims) != MOE_OK) return 0;
  return ffn_layout(*dims, backward != 0).total;
}

moe_status moe_gated_ffn_fwd(const moe_ffn_dims* dims, const moe_bf16* x, const int32_t* offsets,
                             const uint8_t* W1q, const float* s1, const uint8_t* W3q,
                             const float* s3, const uint8_t* W2q, const float* s2, moe_bf16* A,
                             moe_bf16* B, moe_bf16* H, moe_bf16* y, void* ws, size_t ws_bytes,
                             moe_stream_t stream_) {
  const moe_status st = check_ffn(dims);
  if (st != MOE_OK) return st;
  const moe_ffn_dims& d = *dims;
  const size_t R = d.rows;
  const bool keep = A || B || H;
  if (!buf_ok(x, R) || (offsets ? !ptr_ok(offsets) : d.E != 1) || !ptr_ok(W1q) || !ptr_ok(s1) ||
      !ptr_ok(W3q) || !ptr_ok(s3) || !ptr_ok(W2q) || !ptr_ok(s2) || !buf_ok(y, R) ||
      (keep && (!buf_ok(A, R) || !buf_ok(B, R) || !buf_ok(H, R))) || !ws || !aligned(ws, kAlign))
    return MOE_ERR_INVALID_ARG;
  const FfnLayout L = ffn_layout(d, false);
  if (ws_bytes < L.total) return MOE_ERR_WORKSPACE;
  if (R == 0) return MOE_OK;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  const moe::BlockRows r = {d.E, offsets, d.rows, at<int>(ws, 0), moe_api::num_sms(),
                            at<float>(ws, L.part)};
  uint8_t *xq = at<uint8_t>(ws, L.Xq), *hq = at<uint8_t>(ws, L.Hq);
  float *sx = at<float>(ws, L.sx), *sh = at<float>(ws, L.sh);
  BLOCK_RUN(moe::launch_quant_rows_block(x, nullptr, 1, d.rows, d.rows, d.h, xq, sx, r.num_sms,
                                         stream, offsets, d.E + 1, nullptr, r.status),
            "quant_rows_block");
  BLOCK_RUN(moe::block_fc1_fwd(r, {xq, sx}, {W1q, s1}, {W3q, s3}, d.h, d.f, A, B, H, hq, sh,
                               stream),
            "block_fc1_fwd");
  BLOCK_RUN(moe::block_product(r, {hq, sh}, {W2q, s2}, d.f, d.h, false, false, y, stream, true),
            "block_fc2_fwd");
  return MOE_OK;
}

moe_status moe_gated_ffn_bwd(const moe_ffn_dims* dims, const moe_bf16* x, const moe_bf16* dy,
                             const int32_t* offsets, const uint8_t* W1q, const float* s1,
                             const uint8_t* W3q, const float* s3, const uint8_t* W2q,
                             const float* s2, const moe_bf16* A, const moe_bf16* B,
                             const moe_bf16* H, moe_bf16* dx, void* dW1, void* dW3, void* dW2,
                             void* ws, size_t ws_bytes, moe_stream_t stream_) {
  const moe_status st = check_ffn(dims);
  if (st != MOE_OK) return st;
  const moe_ffn_dims& d = *dims;
  const size_t R = d.rows;
  const bool wgrads = dW1 || dW3 || dW2;
  if (!buf_ok(x, R) || !buf_ok(dy, R) || (offsets ? !ptr_ok(offsets) : d.E != 1) ||
      !ptr_ok(W1q) || !ptr_ok(s1) || !ptr_ok(W3q) || !ptr_ok(s3) || !ptr_ok(W2q) || !ptr_ok(s2) ||
      !buf_ok(A, R) || !buf_ok(B, R) || !buf_ok(H, R) || !buf_ok(dx, R) ||
      (wgrads && (!ptr_ok(dW1) || !ptr_ok(dW3) || !ptr_ok(dW2))) || !ws || !aligned(ws, kAlign))
    return MOE_ERR_INVALID_ARG;
  const FfnLayout L = ffn_layout(d, true);
  if (ws_bytes < L.total) return MOE_ERR_WORKSPACE;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (R == 0) {
    const size_t bytes = static_cast<size_t>(d.E) * d.h * d.f * (d.dw_bf16 ? 2 : 4);
    if (wgrads)
      for (void* w : {dW1, dW3, dW2})
        BLOCK_RUN(cudaMemsetAsync(w, 0, bytes, stream), "zero_dW");
    return MOE_OK;
  }
  const moe::BlockRows r = {d.E, offsets, d.rows, at<int>(ws, 0), moe_api::num_sms(),
                            at<float>(ws, L.part)};
  uint8_t *dyq = at<uint8_t>(ws, L.Xq), *daq = at<uint8_t>(ws, L.dAq), *dbq = at<uint8_t>(ws, L.dBq);
  float *sdy = at<float>(ws, L.sx), *sda = at<float>(ws, L.sda), *sdb = at<float>(ws, L.sdb);
  uint16_t *da = at<uint16_t>(ws, L.dA), *db = at<uint16_t>(ws, L.dB);
  BLOCK_RUN(moe::launch_quant_rows_block(dy, nullptr, 1, d.rows, d.rows, d.h, dyq, sdy, r.num_sms,
                                         stream, offsets, d.E + 1, nullptr, r.status),
            "quant_rows_block");
  BLOCK_RUN(moe::block_fc2_dgrad(r, {dyq, sdy}, {W2q, s2}, d.h, d.f, A, B, da, db, daq, sda, dbq,
                                 sdb, stream),
            "block_fc2_dgrad");
  BLOCK_RUN(moe::block_fc1_dgrad(r, {daq, sda}, {dbq, sdb}, {W1q, s1}, {W3q, s3}, d.h, d.f, false,
                                 dx, stream),
            "block_fc1_dgrad");
  if (wgrads) {
    moe::GemmProblem g;
    g.E = d.E;
    g.offsets = offsets;
    g.rows = d.rows;
    g.h = d.h;
    g.f = d.f;
    g.status = r.status;
    g.num_sms = r.num_sms;
    BLOCK_RUN(moe::gemm_fc2_wgrad(g, H, dy, dW2, stream, d.dw_bf16 != 0), moe::kGemmNames[4]);
    BLOCK_RUN(moe::gemm_fc1_wgrad(g, x, da, db, dW1, dW3, stream, d.dw_bf16 != 0),
              moe::kGemmNames[5]);
  }
  return MOE_OK;
}

}  // extern "C"
