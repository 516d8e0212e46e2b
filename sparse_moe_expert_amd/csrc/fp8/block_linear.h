// Arguments and outputs of the 8-bit dense layer's kernels.
#pragma once

#include "block_common.h"

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

// COUNT (a multiple of 4) outputs of a token from n on, from their sums; those
// at or past N are left alone
template <int COUNT>
__device__ __forceinline__ void write(const LinearArgs& p, int t, int n, float (&v)[COUNT]) {
  if (n >= p.N) return;
  const size_t at = (size_t)t * p.N + n;
  if (p.bias) {
#pragma unroll
    for (int i = 0; i < COUNT; ++i) v[i] += bf16_to_f32(p.bias[min(n + i, p.N - 1)]);
  }
  uint32_t o[COUNT / 2];
#pragma unroll
  for (int i = 0; i < COUNT / 2; ++i) o[i] = to_bf16(v[2 * i]) | to_bf16(v[2 * i + 1]) << 16;
  if (COUNT % 8 == 0 && p.N % 8 == 0 && n + COUNT <= p.N) {
#pragma unroll
    for (int i = 0; i < COUNT / 8; ++i)
      *reinterpret_cast<uint4*>(p.y + at + 8 * i) = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
  } else if (p.N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < COUNT / 4; ++i)
      if (n + 4 * i < p.N) *reinterpret_cast<uint2*>(p.y + at + 4 * i) = make_uint2(o[2 * i], o[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < COUNT; ++i)
      if (n + i < p.N) p.y[at + i] = (uint16_t)(o[i / 2] >> (i % 2 * 16));
  }
}

}  // namespace
}  // namespace moe
