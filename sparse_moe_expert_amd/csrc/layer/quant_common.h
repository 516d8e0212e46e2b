// 4-bit dense weights: formats, their decoding, and the products' arguments.
//
// A weight is e2m1 code * block scale (* global scale).  NVFP4: an e4m3
// scale per 16 weights and one fp32 global scale; MXFP4: a power-of-two
// (e8m0, 2^(byte - 127)) scale per 32 weights.  Codes are packed two per
// byte, element 2i in the low nibble of byte i, rows along the reduction.
#pragma once

#include "row_dot.h"

namespace moe {
namespace {

// weights that share a scale
template <int FMT>
constexpr int kScaleGroup = FMT == MOE_QUANT_NVFP4 ? 16 : 32;

// A 4-bit matrix [N, K]
struct QuantMat {
  const uint8_t* codes;
  const uint8_t* scales;
  const float* g;          // global scale, or null for 1
};

// One block scale as fp32 (exact)
template <int FMT>
__device__ __forceinline__ float block_scale(uint32_t byte) {
  if constexpr (FMT == MOE_QUANT_NVFP4) return __builtin_amdgcn_cvt_f32_fp8((int)byte, 0);
  // 2^-127 is subnormal in fp32
  return byte == 0 ? 5.877471754e-39f : __uint_as_float(byte << 23);
}

__device__ __forceinline__ float bf16_to_f32(uint32_t bits) { return __uint_as_float(bits << 16); }

__device__ __forceinline__ float sigmoid(float v) { return 1.0f / (1.0f + __expf(-v)); }

}  // namespace

// Argument checks shared by the 4-bit products
inline bool quant_format_ok(int f) { return f == MOE_QUANT_NVFP4 || f == MOE_QUANT_MXFP4; }
inline bool quant_dims_ok(int n, int k) { return n >= 1 && k >= 32 && k % 32 == 0; }
inline bool quant_dims_fit(int n, int k) { return n <= (1 << 20) && k <= (1 << 15); }
constexpr int kQuantMaxTokens = 1 << 20;
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace moe
