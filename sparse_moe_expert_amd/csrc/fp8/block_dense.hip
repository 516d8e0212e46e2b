// A dense layer in 8 bits: moe_block_linear.
#include "block_common.h"

namespace moe {
namespace {

constexpr int kLinThreads = 256;

struct LinearArgs {
  const uint8_t* x;
  const float* sx;
  BlockMat w;
  const uint16_t* bias;
  uint16_t* y;
  int T, N, K;
};

// A wavefront to 16 rows and 16 tokens, operands straight from memory
__global__ __launch_bounds__(kLinThreads) void linear_kernel(LinearArgs p, int row_groups) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x >> 6;
  const int n0 = ((int)(blockIdx.x % row_groups) * 4 + wave) * 16, t0 = (int)(blockIdx.x / row_groups) * 16;
  if (n0 >= p.N) return;
  const int l16 = lane & 15, g = lane >> 4, kb = blocks_of(p.K);
  const int t = min(t0 + l16, p.T - 1);
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(p.w.q + (size_t)n0 * p.K, (uint32_t)(min(16, p.N - n0) * p.K));
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(p.x + (size_t)t0 * p.K, (uint32_t)(min(16, p.T - t0) * p.K));
  const float* const sw = p.w.s + (size_t)(n0 / kBlock) * kb;
  const float* const sx = p.sx + (size_t)t * kb;
  const uint32_t row = (uint32_t)(l16 * p.K);
  f32x4 acc{};
  for (int b = 0; b < kb; ++b) {
    const int lo = b * kBlock + g * 16, hi = lo + 64;
    const uint32_t a0 = lo < p.K ? row + lo : kOutside, a1 = hi < p.K ? row + hi : kOutside;
    const f32x4 d = block_product(load_fragment(rw, a0, a1), load_fragment(rx, a0, a1));
    const float s = sx[b] * sw[b];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = fmaf(d[i], s, acc[i]);
  }
  if (t0 + l16 >= p.T) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = n0 + g * 4 + i;
    if (n >= p.N) continue;
    const float v = p.bias ? acc[i] + bf16_to_f32(p.bias[n]) : acc[i];
    p.y[(size_t)t * p.N + n] = (uint16_t)to_bf16(v);
  }
}

inline bool linear_dims_ok(int N, int K) { return N >= 1 && K >= 16 && K % 16 == 0; }
inline bool linear_dims_fit(int N, int K) { return N <= (1 << 20) && K <= kBlockMaxK; }

}  // namespace
}  // namespace moe

extern "C" size_t moe_block_linear_workspace_size(int T, int N, int K) {
  using namespace moe;
  (void)T, (void)N, (void)K;
  return 0;
}

extern "C" moe_status moe_block_linear(const uint8_t* x, const float* x_scale, const uint8_t* w, const float* w_scale,
                                       const uint16_t* bias, int T, int N, int K, void* workspace,
                                       size_t workspace_bytes, uint16_t* y, void* stream) {
  using namespace moe;
  if (T < 0 || !linear_dims_ok(N, K)) return MOE_ERR_INVALID_SHAPE;
  if (!linear_dims_fit(N, K) || T > kBlockMaxTokens) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!x || !x_scale || !w || !w_scale || !y) return MOE_ERR_NULL_POINTER;
  const void* const all[] = {x, x_scale, w, w_scale, bias, y};
  for (const void* a : all)
    if (!aligned16(a)) return MOE_ERR_MISALIGNED;
  const size_t need = moe_block_linear_workspace_size(T, N, K);
  if (need > 0 && !workspace) return MOE_ERR_NULL_POINTER;
  if (need > 0 && !aligned16(workspace)) return MOE_ERR_MISALIGNED;
  if (workspace_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  const LinearArgs p{x, x_scale, {w, w_scale}, bias, y, T, N, K};
  const int row_groups = (N + 63) / 64;
  const unsigned grid = (unsigned)row_groups * (unsigned)((T + 15) / 16);       // at most 2^14 * 2^16
  linear_kernel<<<grid, kLinThreads, 0, static_cast<hipStream_t>(stream)>>>(p, row_groups);
  return launch_status();
}
