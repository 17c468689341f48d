// decode.cuh -- the whole layer for a few tokens (decode.cu), as api.cu sees it.
#pragma once
#include <cstddef>

#include "../../include/moe.h"

namespace moe {

constexpr int kDecodeMaxT = 128;

// Scratch bytes of moe_layer_decode / moe_layer_decode_fp8 for checked dims;
// 0 where the call would decline them.
size_t decode_workspace_bytes(const moe_dims& d, bool fp8);

}  // namespace moe
