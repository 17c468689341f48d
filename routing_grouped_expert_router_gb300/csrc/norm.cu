// norm.cu -- the norms before and after the MoE block, fused with its gate
// and residual scale: moe_block_norm_fwd and moe_block_norm_bwd.
//
//   z = y / rms(y) * w_post;  r_out = alpha r + beta gate * z;
//   u = r_out / rms(r_out) * w_pre
//
// Both directions are bound by HBM: the forward reads r and y and writes r_out
// and u (8 bytes for each element with a bf16 residual), the backward reads
// r_out, y, du and dr_out and writes dr and dy (12 bytes).  So a row is read
// once and stays in the registers of one block, two 16-byte pieces for each
// thread, through both of its row sums.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/moe.h"
#include "api_internal.h"
#include "kernels.cuh"

namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kMaxH = 8192;
constexpr int kMaxThreads = 512;
constexpr int kPieces = 2;  // 8-element pieces of a row for each thread

struct Args {
  const void* r;        // fwd: r; bwd: r_out
  const uint4* y;
  const float* w_post;
  const float* gate;
  const float* w_pre;
  const uint4* du;
  const void* dr_out;
  void* out_r;          // fwd: r_out; bwd: dr
  uint4* out_u;         // fwd: u; bwd: dy
  float* dgate;         // bwd, token gate
  float* partial;       // bwd: column sums of each block
  int T, h;
  int gate_kind;
  float eps, alpha, beta, inv_h;
};

__device__ __forceinline__ void unpack8(const uint4& q, float* v) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float* v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight values of the residual stream at element offset o.
template <bool F32>
__device__ __forceinline__ void load_res(const void* p, size_t o, float* v) {
  if (F32) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + o);
    const float4 a = q[0], b = q[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + o), v);
  }
}
// Stores eight values in the residual's type and leaves the stored ones in v.
template <bool F32>
__device__ __forceinline__ void store_res(void* p, size_t o, float* v) {
  if (F32) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + o);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    const uint4 q = pack8(v);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + o) = q;
    unpack8(q, v);
  }
}
__device__ __forceinline__ void load_w(const float* w, int c, float* v) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(w + c));
  const float4 b = __ldg(reinterpret_cast<const float4*>(w + c) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// Sums of N values over the block, in every thread.  The order is fixed:
// butterflies within warps, then the warps in order.  `slot` alternates so
// that one barrier for each call is enough.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float (*red)[N * (kMaxThreads / 32)],
                                          int& slot) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(kFull, v[i], o);
  const int nw = blockDim.x >> 5;
  if (nw == 1) return;
  float* s = red[slot];
  slot ^= 1;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) s[(threadIdx.x >> 5) * N + i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.f;
  for (int w = 0; w < nw; ++w)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += s[w * N + i];
}

// 1 / rms of a row from its sum of squares, correctly rounded: its error would
// shift a whole row, and one for each row costs nothing.
__device__ __forceinline__ float inv_rms(float ss, const Args& a) {
  return __frsqrt_rn(__fdiv_rn(ss, static_cast<float>(a.h)) + a.eps);
}

template <bool F32>
__global__ void __launch_bounds__(kMaxThreads) block_norm_fwd_kernel(const Args a) {
  __shared__ float red[2][kMaxThreads / 32];
  int slot = 0;
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    const size_t row = static_cast<size_t>(t) * a.h;
    float v[kPieces][8], z[kPieces][8];
    float ss[1] = {0.f};
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int c = (threadIdx.x + i * blockDim.x) * 8;
      if (c < a.h) {
        load_res<F32>(a.r, row + c, v[i]);
        if (a.y) unpack8(a.y[(row + c) >> 3], z[i]);
      }
    }
    if (a.y) {
      float ry = 1.f;
      if (a.w_post) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
          if ((threadIdx.x + i * blockDim.x) * 8 < a.h)
#pragma unroll
            for (int j = 0; j < 8; ++j) ss[0] = fmaf(z[i][j], z[i][j], ss[0]);
        block_sum<1>(ss, red, slot);
        ry = inv_rms(ss[0], a);
      }
      float s = a.beta;
      if (a.gate_kind == MOE_GATE_TOKEN) s *= __ldg(a.gate + t);
      ss[0] = 0.f;
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int c = (threadIdx.x + i * blockDim.x) * 8;
        if (c >= a.h) continue;
        float w[8];
        if (a.w_post) {
          load_w(a.w_post, c, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) z[i][j] *= ry * w[j];
        }
        if (a.gate_kind == MOE_GATE_CHANNEL) {
          load_w(a.gate, c, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) z[i][j] *= w[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = fmaf(s, z[i][j], a.alpha * v[i][j]);
        store_res<F32>(a.out_r, row + c, v[i]);
      }
    }
    if (!a.w_pre) continue;
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      if ((threadIdx.x + i * blockDim.x) * 8 < a.h)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss[0] = fmaf(v[i][j], v[i][j], ss[0]);
    block_sum<1>(ss, red, slot);
    const float rv = inv_rms(ss[0], a);
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int c = (threadIdx.x + i * blockDim.x) * 8;
      if (c >= a.h) continue;
      float w[8];
      load_w(a.w_pre, c, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] *= rv * w[j];
      a.out_u[(row + c) >> 3] = pack8(v[i]);
    }
  }
}

// The backward of a row, with v = r_out, rv = 1 / rms(v), n = y / rms(y) (n = y
// without w_post), and the row sums S:
//   G  = dr_out + rv (du w_pre - v rv^2 S(du w_pre v) / h)
//   q  = beta gate G;  dy = (q w_post - n S(q w_post n) / h) / rms(y)
// Column sums: P = sum_t du v rv (dw_pre) and Q = sum_t beta g_t G n, from which
// dw_post = gate_c Q and the channel gate's gradient = w_post Q, so one sum
// serves both (g_t: the token gate, else 1).  Each block keeps P and Q of its
// rows in registers and writes them once; block_norm_cols_kernel adds the
// blocks in order.
template <bool F32>
__global__ void __launch_bounds__(kMaxThreads) block_norm_bwd_kernel(const Args a) {
  __shared__ float red3[2][3 * (kMaxThreads / 32)];
  __shared__ float red1[2][kMaxThreads / 32];
  int slot3 = 0, slot1 = 0;
  float P[kPieces][8], Q[kPieces][8];
#pragma unroll
  for (int i = 0; i < kPieces; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) P[i][j] = Q[i][j] = 0.f;
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    const size_t row = static_cast<size_t>(t) * a.h;
    float v[kPieces][8], g[kPieces][8], n[kPieces][8], du[kPieces][8];
    float s3[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int c = (threadIdx.x + i * blockDim.x) * 8;
      if (c >= a.h) continue;
      if (a.w_pre) {
        load_res<F32>(a.r, row + c, v[i]);
        unpack8(a.du[(row + c) >> 3], du[i]);
      }
      if (a.y) unpack8(a.y[(row + c) >> 3], n[i]);
      if (a.dr_out) {
        load_res<F32>(a.dr_out, row + c, g[i]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) g[i][j] = 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int c = (threadIdx.x + i * blockDim.x) * 8;
      if (c >= a.h) continue;
      float w[8];
      if (a.w_pre) {
        load_w(a.w_pre, c, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          s3[0] = fmaf(v[i][j], v[i][j], s3[0]);
          s3[1] = fmaf(du[i][j] * w[j], v[i][j], s3[1]);
        }
      }
      if (a.w_post)
#pragma unroll
        for (int j = 0; j < 8; ++j) s3[2] = fmaf(n[i][j], n[i][j], s3[2]);
    }
    block_sum<3>(s3, red3, slot3);
    const float rv = inv_rms(s3[0], a);
    const float k1 = s3[1] * a.inv_h * rv * rv * rv;
    const float ry = a.w_post ? inv_rms(s3[2], a) : 1.f;
    const float gt = a.y && a.gate_kind == MOE_GATE_TOKEN ? __ldg(a.gate + t) : 1.f;
    float s1[1] = {0.f};
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int c = (threadIdx.x + i * blockDim.x) * 8;
      if (c >= a.h) continue;
      float w[8], dr[8];
      if (a.w_pre) {
        load_w(a.w_pre, c, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          P[i][j] = fmaf(du[i][j], v[i][j] * rv, P[i][j]);
          g[i][j] += rv * du[i][j] * w[j] - k1 * v[i][j];
        }
      }
      const float al = a.y ? a.alpha : 1.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) dr[j] = al * g[i][j];
      store_res<F32>(a.out_r, row + c, dr);
      if (!a.y) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        n[i][j] *= ry;
        g[i][j] *= a.beta;
        Q[i][j] = fmaf(gt * g[i][j], n[i][j], Q[i][j]);
      }
      if (a.gate_kind == MOE_GATE_CHANNEL) {
        load_w(a.gate, c, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[i][j] *= w[j];
      }
      if (a.w_post) {
        load_w(a.w_post, c, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[i][j] *= w[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) s1[0] = fmaf(g[i][j], n[i][j], s1[0]);
    }
    if (!a.y) continue;
    // the projection of dy on y's row, which without the token's gate is also
    // that gate's gradient
    if (a.w_post || a.gate_kind == MOE_GATE_TOKEN) block_sum<1>(s1, red1, slot1);
    const float k2 = a.w_post ? s1[0] * a.inv_h : 0.f;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int c = (threadIdx.x + i * blockDim.x) * 8;
      if (c >= a.h) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) g[i][j] = gt * ry * (g[i][j] - n[i][j] * k2);
      a.out_u[(row + c) >> 3] = pack8(g[i]);
    }
    if (a.dgate && threadIdx.x == 0) a.dgate[t] = s1[0];
  }
  float* part = a.partial + static_cast<size_t>(blockIdx.x) * 2 * a.h;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int c = (threadIdx.x + i * blockDim.x) * 8;
    if (c >= a.h) continue;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      part[c + j] = P[i][j];
      part[a.h + c + j] = Q[i][j];
    }
  }
}

// The column gradients from the blocks' sums, a fixed order for each column:
// 8 interleaved chains, then those in order.
__global__ void __launch_bounds__(256) block_norm_cols_kernel(const float* partial, int nblk, int h,
                                                              const float* w_post,
                                                              const float* gate, float* dw_pre,
                                                              float* dw_post, float* dgate) {
  __shared__ float sp[8][32], sq[8][32];
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float p = 0.f, q = 0.f;
  if (c < h)
    for (int b = g; b < nblk; b += 8) {
      p += partial[static_cast<size_t>(b) * 2 * h + c];
      q += partial[static_cast<size_t>(b) * 2 * h + h + c];
    }
  sp[g][lane] = p;
  sq[g][lane] = q;
  __syncthreads();
  if (g != 0 || c >= h) return;
  for (int i = 1; i < 8; ++i) {
    p += sp[i][lane];
    q += sq[i][lane];
  }
  if (dw_pre) dw_pre[c] = p;
  if (dw_post) dw_post[c] = gate ? gate[c] * q : q;
  if (dgate) dgate[c] = w_post ? w_post[c] * q : q;
}

constexpr size_t kAlign = 256;

int threads_for(int h) {
  const int need = (h / 8 + kPieces - 1) / kPieces;
  return (need + 31) / 32 * 32;
}

// Blocks of the backward: each keeps column sums, so only as many as run at
// once.
int bwd_blocks(const moe_norm_dims& d) {
  const int per_sm = 1024 / threads_for(d.h) > 8 ? 8 : 1024 / threads_for(d.h);
  const int n = moe_api::num_sms() * per_sm;
  return d.T < n ? d.T : n;
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
  a.y = reinterpret_cast<const uint4*>(y);
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
  const size_t n = static_cast<size_t>(bwd_blocks(*dims)) * 2 * dims->h * sizeof(float);
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
  const int threads = threads_for(d.h);
  if (d.res_f32)
    block_norm_fwd_kernel<true><<<d.T, threads, 0, s>>>(a);
  else
    block_norm_fwd_kernel<false><<<d.T, threads, 0, s>>>(a);
  if (moe::launched() != cudaSuccess || !moe_api::note(s, "block_norm_fwd")) return MOE_ERR_CUDA;
  return MOE_OK;
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
        return MOE_ERR_CUDA;
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
  a.du = reinterpret_cast<const uint4*>(du);
  a.dr_out = dr_out;
  a.out_r = dr;
  a.out_u = reinterpret_cast<uint4*>(dy);
  a.dgate = a.gate_kind == MOE_GATE_TOKEN ? dgate : nullptr;
  a.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kAlign);
  const int threads = threads_for(d.h), blocks = bwd_blocks(d);
  if (d.res_f32)
    block_norm_bwd_kernel<true><<<blocks, threads, 0, s>>>(a);
  else
    block_norm_bwd_kernel<false><<<blocks, threads, 0, s>>>(a);
  if (moe::launched() != cudaSuccess || !moe_api::note(s, "block_norm_bwd")) return MOE_ERR_CUDA;
  const bool channel = a.gate_kind == MOE_GATE_CHANNEL;
  if (dw_pre || dw_post || channel) {
    block_norm_cols_kernel<<<(d.h + 31) / 32, 256, 0, s>>>(a.partial, blocks, d.h, w_post,
                                                           channel ? gate : nullptr, dw_pre,
                                                           dw_post, channel ? dgate : nullptr);
    if (moe::launched() != cudaSuccess || !moe_api::note(s, "block_norm_cols")) return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

}  // extern "C"
