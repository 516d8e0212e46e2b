// Arguments and outputs of the 8-bit dense layer's kernels.
#pragma once

#include "block_common.h"

#include <type_traits>

namespace moe {

struct LinearArgs {
  const uint8_t* x;
  const float* sx;
  BlockMat w;
  const uint16_t* bias;
  uint16_t* y;
  int T, N, K;
};

// The kernel of few tokens, for the batches that its _ok says
bool linear_few_ok(int T, int N, int K);
moe_status linear_few(const LinearArgs& p, hipStream_t s);

namespace {

// Words of an output row, which starts at any of its elements
typedef uint32_t row_u32x4 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t row_u32x2 __attribute__((ext_vector_type(2), aligned(2)));

// COUNT (a multiple of 4) outputs of a token from n on, from their sums; those
// at or past N are left alone.  The widest stores for every N: the card takes them
// unaligned (T = 3476 4997x128: 27.6 us, 64.8 one element each)
template <int COUNT>
__device__ __forceinline__ void write(const LinearArgs& p, int t, int n, float (&v)[COUNT]) {
  using Words = std::conditional_t<COUNT % 8 == 0, row_u32x4, row_u32x2>;
  constexpr int kWords = COUNT % 8 == 0 ? 4 : 2;
  if (n >= p.N) return;
  const size_t at = (size_t)t * p.N + n;
  const bool all = n + COUNT <= p.N;
  if (p.bias) {                                              // (n is a multiple of COUNT)
#pragma unroll
    for (int i = 0; i < COUNT; i += 4) {
      uint2 b{};
      if (all) {
        b = *reinterpret_cast<const uint2*>(p.bias + n + i);
      } else {
        const uint16_t* const from = p.bias;
        const int last = p.N - 1, at = n + i;
        b.x = from[min(at, last)] | (uint32_t)from[min(at + 1, last)] << 16;
        b.y = from[min(at + 2, last)] | (uint32_t)from[min(at + 3, last)] << 16;
      }
      v[i] += bf16_to_f32(b.x & 0xFFFFu), v[i + 1] += bf16_to_f32(b.x >> 16);
      v[i + 2] += bf16_to_f32(b.y & 0xFFFFu), v[i + 3] += bf16_to_f32(b.y >> 16);
    }
  }
  uint32_t o[COUNT / 2];
#pragma unroll
  for (int i = 0; i < COUNT / 2; ++i) o[i] = to_bf16(v[2 * i]) | to_bf16(v[2 * i + 1]) << 16;
  if (all) {
#pragma unroll
    for (int i = 0; i < COUNT / 2; i += kWords) {
      Words w;
#pragma unroll
      for (int k = 0; k < kWords; ++k) w[k] = o[i + k];
      *reinterpret_cast<Words*>(p.y + at + 2 * i) = w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < COUNT; ++i)
      if (n + i < p.N) p.y[at + i] = (uint16_t)(o[i / 2] >> (i % 2 * 16));
  }
}

}  // namespace
}  // namespace moe
