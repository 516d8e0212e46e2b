// 8-bit products of few tokens: bound by the weight bytes, the smallest calls by
// a launch and three latencies (T = 1 2048x2048 3.4 us).
//
// A workgroup owns RT row tiles of 16 and up to JT token tiles of 16; its eight
// waves take runs of D blocks of the reduction in turn, weights and tokens
// straight from memory in the layout of the products, all of a run's on their way
// at once; their sums meet in LDS.
#pragma once

#include "block_common.h"

namespace moe {
namespace {

constexpr int kFewWaves = 8;
constexpr int kFewThreads = kFewWaves * kWave;

// (through the scalar cache: a uniform value in one register)
template <class V>
__device__ __forceinline__ V scalar_load(const V* at) {
  return *(const __attribute__((address_space(4))) V*)(uintptr_t)at;
}

// The 32 bytes of a lane of the block of a row that starts at byte `row` of the
// resource: those past the row's K values are zero
__device__ __forceinline__ i32x8 load_block(__amdgpu_buffer_rsrc_t r, uint32_t row, int block, int K, int g) {
  const int lo = block * kBlock + g * 16, hi = lo + 64;
  const u32x4 a = __builtin_amdgcn_raw_buffer_load_b128(r, lo < K ? row + (uint32_t)lo : kOutside, 0, 0);
  const u32x4 b = __builtin_amdgcn_raw_buffer_load_b128(r, hi < K ? row + (uint32_t)hi : kOutside, 0, 0);
  return fragment(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b));
}

}  // namespace
}  // namespace moe
