// block_groups.cuh -- a grouped product's row ranges, made by one warp.
#pragma once
#include <cstdint>

#include "kernels.cuh"

namespace moe {

constexpr int kMaxGroups = 64;

// Orders what this thread wrote, and what it has seen written, before what follows for the
// whole GPU (__threadfence() orders more, and takes longer).
__device__ __forceinline__ void fence_gpu() { asm volatile("fence.acq_rel.gpu;" ::: "memory"); }

// off[0 .. E]: the offsets (all `rows` in one group where `offsets` is NULL), clamped into
// order so that every access that follows stays inside its buffer; one that had to be is
// recorded.  cum[0 .. E]: tiles of `tile` rows before each group.
__device__ __forceinline__ void group_tables(const int32_t* offsets, int E, int rows, int tile,
                                             int* off, int* cum, int* status, int lane) {
  constexpr unsigned kAll = 0xFFFFFFFFu;
  int top = 0;
  bool bad = false;
  for (int base = 0; base <= E; base += 32) {
    const int e = base + lane;
    int o = rows;
    if (e <= E) o = offsets ? __ldg(offsets + e) : (e ? rows : 0);
    int v = max(min(max(o, 0), rows), top);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(kAll, v, d);
      if (lane >= d) v = max(v, u);
    }
    if (e <= E) {
      off[e] = v;
      bad = bad || v != o || (e == 0 && o != 0);
    }
    top = __shfl_sync(kAll, v, 31);
  }
  if (bad) report_bad_index(status);
  __syncwarp();
  int sum = 0;
  for (int base = 0; base < E; base += 32) {
    const int e = base + lane;
    int v = e < E ? (off[e + 1] - off[e] + tile - 1) / tile : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(kAll, v, d);
      if (lane >= d) v += u;
    }
    if (e < E) cum[e + 1] = sum + v;
    sum += __shfl_sync(kAll, v, 31);
  }
  if (lane == 0) cum[0] = 0;
}

}  // namespace moe
