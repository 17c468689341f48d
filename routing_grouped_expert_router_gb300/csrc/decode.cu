// decode.cu -- the whole MoE layer for a few tokens: moe_layer_decode and
// moe_layer_decode_fp8.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "../../include/moe.h"
#include "api_internal.h"
#include "decode.cuh"
#include "kernels.cuh"

namespace moe {
namespace {

constexpr int kTok = 8;  // tokens of an expert summed at once

struct Args {
  int T, h, f, E, k, capacity;
  const int32_t* idx;
  const float* gates;
  // bf16
  const uint16_t* x;
  const uint16_t *W1, *W3, *W2;
  // e4m3
  const uint8_t *xq, *W13q, *W2q, *Hq;
  const float *sx, *sh, *s1, *s3, *s2;
  uint16_t* H;  // [T*k, f]
  float* O;     // [T*k, h]
  uint16_t* y;
};

__device__ __forceinline__ float bf(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
__device__ __forceinline__ float e4(uint8_t v) {
  __nv_fp8_e4m3 q;
  q.__x = v;
  return static_cast<float>(q);
}

// The assignments that expert e keeps, in ascending order, in list; returns
// their number.
__device__ int expert_list(const Args& a, int e, int* list, int* count) {
  if (threadIdx.x == 0) {
    int n = 0;
    for (int i = 0; i < a.T * a.k && n < a.capacity; ++i)
      if (a.idx[i] == e) list[n++] = i;
    *count = n;
  }
  __syncthreads();
  return *count;
}

template <bool F8>
__global__ void decode_fc1_kernel(const Args a) {
  __shared__ int list[kDecodeMaxT], count;
  const int e = blockIdx.y, c = blockIdx.x * blockDim.x + threadIdx.x;
  const int n = expert_list(a, e, list, &count);
  if (c >= a.f) return;
  for (int i0 = 0; i0 < n; i0 += kTok) {
    float sa[kTok] = {}, sb[kTok] = {};
    for (int j = 0; j < a.h; ++j) {
      float w1, w3;
      if (F8) {
        const size_t r = (static_cast<size_t>(e) * 2 * a.f + (c / 128) * 256 + c % 128) * a.h + j;
        w1 = e4(a.W13q[r]);
        w3 = e4(a.W13q[r + static_cast<size_t>(128) * a.h]);
      } else {
        const size_t r = (static_cast<size_t>(e) * a.h + j) * a.f + c;
        w1 = bf(a.W1[r]);
        w3 = bf(a.W3[r]);
      }
#pragma unroll
      for (int i = 0; i < kTok; ++i) {
        const size_t t = list[min(i0 + i, n - 1)] / a.k;
        const float xv = F8 ? e4(a.xq[t * a.h + j]) : bf(a.x[t * a.h + j]);
        sa[i] = fmaf(xv, w1, sa[i]);
        sb[i] = fmaf(xv, w3, sb[i]);
      }
    }
    for (int i = 0; i < kTok && i0 + i < n; ++i) {
      const int p = list[i0 + i];
      float va = sa[i], vb = sb[i];
      if (F8) {
        const float s = a.sx[p / a.k];
        va *= s * a.s1[static_cast<size_t>(e) * a.f + c];
        vb *= s * a.s3[static_cast<size_t>(e) * a.f + c];
      }
      const __nv_bfloat16 hv = __float2bfloat16_rn(va / (1.f + expf(-va)) * vb);
      a.H[static_cast<size_t>(p) * a.f + c] = *reinterpret_cast<const uint16_t*>(&hv);
    }
  }
}

template <bool F8>
__global__ void decode_fc2_kernel(const Args a) {
  __shared__ int list[kDecodeMaxT], count;
  const int e = blockIdx.y, c = blockIdx.x * blockDim.x + threadIdx.x;
  const int n = expert_list(a, e, list, &count);
  if (c >= a.h) return;
  for (int i0 = 0; i0 < n; i0 += kTok) {
    float s[kTok] = {};
    for (int j = 0; j < a.f; ++j) {
      const float w = F8 ? e4(a.W2q[(static_cast<size_t>(e) * a.h + c) * a.f + j])
                         : bf(a.W2[(static_cast<size_t>(e) * a.f + j) * a.h + c]);
#pragma unroll
      for (int i = 0; i < kTok; ++i) {
        const size_t o = static_cast<size_t>(list[min(i0 + i, n - 1)]) * a.f + j;
        s[i] = fmaf(F8 ? e4(a.Hq[o]) : bf(a.H[o]), w, s[i]);
      }
    }
    for (int i = 0; i < kTok && i0 + i < n; ++i) {
      const int p = list[i0 + i];
      float v = s[i];
      if (F8) v *= a.sh[p] * a.s2[static_cast<size_t>(e) * a.h + c];
      a.O[static_cast<size_t>(p) * a.h + c] = v;
    }
  }
}

// y[t] = the gated sum of the token's placed slots, in slot order.
__global__ void decode_combine_kernel(const Args a) {
  const int t = blockIdx.y, c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= a.h) return;
  float s = 0.f;
  for (int j = 0; j < a.k; ++j) {
    const int p = t * a.k + j, e = a.idx[p];
    int before = 0;
    for (int i = 0; i < p; ++i) before += a.idx[i] == e;
    if (before < a.capacity) s = fmaf(a.gates[p], a.O[static_cast<size_t>(p) * a.h + c], s);
  }
  const __nv_bfloat16 v = __float2bfloat16_rn(s);
  a.y[static_cast<size_t>(t) * a.h + c] = *reinterpret_cast<const uint16_t*>(&v);
}

struct Layout {
  size_t logits, idx, gates, H, O, xq, sx, Hq, sh, total;
};
Layout layout(const moe_dims& d, bool fp8) {
  const size_t R = static_cast<size_t>(d.T) * d.k, T = d.T, h = d.h, f = d.f;
  size_t off = 256;
  auto take = [&](size_t n) {
    const size_t o = off;
    off += (n + 255) / 256 * 256;
    return o;
  };
  Layout L = {};
  L.logits = take(router_partial_bytes(d.T, d.h, d.E));
  L.idx = take(R * 4);
  L.gates = take(R * 4);
  L.H = take(R * f * 2);
  L.O = take(R * h * 4);
  if (fp8) {
    L.xq = take(T * h);
    L.sx = take(T * 4);
    L.Hq = take(R * f);
    L.sh = take(R * 4);
  }
  L.total = off;
  return L;
}

bool supported(const moe_dims& d, bool fp8) {
  return d.T <= kDecodeMaxT && d.sar == 0 && (!fp8 || (d.h % 128 == 0 && d.f % 128 == 0));
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool ptr_ok(const void* p) { return p && aligned(p, 16); }

moe_status decode(const moe_dims* dims, const moe_bf16* x, const float* Wg, const float* b,
                  const moe_bf16* W1, const moe_bf16* W3, const moe_bf16* W2, const void* qw,
                  moe_bf16* y, int32_t* topk_idx, float* gates, void* ws, size_t ws_bytes,
                  cudaStream_t stream, bool fp8) {
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
  const int sms = moe_api::num_sms();
  int32_t* idx = topk_idx ? topk_idx : reinterpret_cast<int32_t*>(w + L.idx);
  float* g = gates ? gates : reinterpret_cast<float*>(w + L.gates);
  Args a = {};
  a.T = d.T;
  a.h = d.h;
  a.f = d.f;
  a.E = d.E;
  a.k = d.k;
  a.capacity = d.capacity > 0 ? d.capacity : INT_MAX;
  a.idx = idx;
  a.gates = g;
  a.x = x;
  a.W1 = W1;
  a.W3 = W3;
  a.W2 = W2;
  a.H = reinterpret_cast<uint16_t*>(w + L.H);
  a.O = reinterpret_cast<float*>(w + L.O);
  a.y = y;
  auto run = [&](cudaError_t e, const char* name) {
    return e == cudaSuccess && moe_api::note(stream, name);
  };
  if (!run(launch_router(x, Wg, d.has_bias ? b : nullptr, d.T, d.h, d.E, d.k, idx, g,
                         reinterpret_cast<float*>(w + L.logits), sms, stream),
           "router_topk"))
    return MOE_ERR_CUDA;
  const dim3 g1((d.f + 127) / 128, d.E), g2((d.h + 127) / 128, d.E), g3((d.h + 127) / 128, d.T);
  if (fp8) {
    auto view = [&](const char* name) {
      return moe_fp8_weight_view(dims, const_cast<void*>(qw), name);
    };
    uint8_t* xq = w + L.xq;
    uint8_t* Hq = w + L.Hq;
    float* sx = reinterpret_cast<float*>(w + L.sx);
    float* sh = reinterpret_cast<float*>(w + L.sh);
    a.W13q = static_cast<const uint8_t*>(view("W13q"));
    a.W2q = static_cast<const uint8_t*>(view("W2q"));
    a.s1 = static_cast<const float*>(view("s1"));
    a.s3 = static_cast<const float*>(view("s3"));
    a.s2 = static_cast<const float*>(view("s2"));
    a.xq = xq;
    a.sx = sx;
    a.Hq = Hq;
    a.sh = sh;
    if (!run(launch_quant_rows(x, nullptr, 1, d.T, d.T, d.h, xq, sx, sms, stream), "quant_x"))
      return MOE_ERR_CUDA;
    decode_fc1_kernel<true><<<g1, 128, 0, stream>>>(a);
    if (!run(launched(), "decode_fc1")) return MOE_ERR_CUDA;
    const long long R = static_cast<long long>(d.T) * d.k;
    if (!run(launch_quant_rows(a.H, nullptr, 1, R, R, d.f, Hq, sh, sms, stream), "quant_h"))
      return MOE_ERR_CUDA;
    decode_fc2_kernel<true><<<g2, 128, 0, stream>>>(a);
  } else {
    decode_fc1_kernel<false><<<g1, 128, 0, stream>>>(a);
    if (!run(launched(), "decode_fc1")) return MOE_ERR_CUDA;
    decode_fc2_kernel<false><<<g2, 128, 0, stream>>>(a);
  }
  if (!run(launched(), "decode_fc2")) return MOE_ERR_CUDA;
  decode_combine_kernel<<<g3, 128, 0, stream>>>(a);
  return run(launched(), "decode_combine") ? MOE_OK : MOE_ERR_CUDA;
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
                     reinterpret_cast<cudaStream_t>(stream), false);
}

moe_status moe_layer_decode_fp8(const moe_dims* dims, const moe_bf16* x, const float* Wg,
                                const float* b, const void* qw, moe_bf16* y, int32_t* topk_idx,
                                float* gates, void* ws, size_t ws_bytes, moe_stream_t stream) {
  return moe::decode(dims, x, Wg, b, nullptr, nullptr, nullptr, qw, y, topk_idx, gates, ws,
                     ws_bytes, reinterpret_cast<cudaStream_t>(stream), true);
}

}  // extern "C"
