// Dense products with 4-bit weights: moe_quant_linear and
// moe_quant_shared_expert.
//
//   linear   y[t,n] = bf16( g * sum_k x[t,k] W[n,k] + bias[n] )
//   shared   h[t,r] = bf16( SiLU(Wg[r] . x_t) * (Wu[r] . x_t) )
//            y[t,c] = bf16( add[t,c] + sigmoid(x_t . v) * (Wd[c] . h_t) )
#include "quant_common.h"

namespace moe {
namespace {

// Per token sigmoid(x_t . v), one wavefront a token.
__global__ __launch_bounds__(kWave) void token_gate_kernel(const uint16_t* __restrict__ x,
                                                           const uint16_t* __restrict__ v, int H,
                                                           float* __restrict__ gate) {
  const int t = blockIdx.x, lane = threadIdx.x;
  float acc = 0.0f;
  for (int k = lane; k < H; k += kWave) acc = fmaf(bf16_to_f32(x[(size_t)t * H + k]), bf16_to_f32(v[k]), acc);
  acc = group_sum(acc, kWave);
  if (lane == 0) gate[t] = sigmoid(acc);
}

struct DenseArgs {
  const uint16_t* x;
  QuantMat a, b;            // b: the second matrix of gate/up
  const uint16_t* bias;     // [N] or null
  const float* gate;        // [T] or null
  const uint16_t* add;      // [T, N] or null
  uint16_t* y;
  int T, N, K;
};

constexpr int kRowTokens = 16;

// One wavefront per weight row and 16 tokens.
template <int FMT, bool GU>
__global__ __launch_bounds__(kWave) void dense_row_kernel(DenseArgs p) {
  const int n = blockIdx.x, t0 = blockIdx.y * kRowTokens, lane = threadIdx.x;
  float acc[GU ? 2 : 1][kRowTokens] = {};
  constexpr int G = kScaleGroup<FMT>;
  for (int c = lane; c < p.K / 8; c += kWave) {       // 8 weights, one scale
#pragma unroll
    for (int m = 0; m < (GU ? 2 : 1); ++m) {
      const QuantMat& w = m ? p.b : p.a;
      const uint32_t codes = reinterpret_cast<const uint32_t*>(w.codes + (size_t)n * (p.K / 2))[c];
      const float s = block_scale<FMT>(w.scales[(size_t)n * (p.K / G) + c * 8 / G]);
      const uint32_t wv[4] = {__builtin_bit_cast(uint32_t, fp4x2_to_bf16x2<0>(codes)),
                              __builtin_bit_cast(uint32_t, fp4x2_to_bf16x2<1>(codes)),
                              __builtin_bit_cast(uint32_t, fp4x2_to_bf16x2<2>(codes)),
                              __builtin_bit_cast(uint32_t, fp4x2_to_bf16x2<3>(codes))};
      for (int t = 0; t < kRowTokens; ++t) {
        if (t0 + t >= p.T) break;
        const uint4 xv = reinterpret_cast<const uint4*>(p.x + (size_t)(t0 + t) * p.K)[c];
        const uint32_t xs[4] = {xv.x, xv.y, xv.z, xv.w};
        float d = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) d = __builtin_amdgcn_fdot2_f32_bf16(as_bf16x2(wv[i]), as_bf16x2(xs[i]), d, false);
        acc[m][t] = fmaf(d, s, acc[m][t]);
      }
    }
  }
  const float ga = p.a.g ? *p.a.g : 1.0f, gb = GU && p.b.g ? *p.b.g : 1.0f;
#pragma unroll
  for (int t = 0; t < kRowTokens; ++t) {
    const float a = group_sum(acc[0][t], kWave) * ga;
    const float b = GU ? group_sum(acc[GU ? 1 : 0][t], kWave) * gb : 0.0f;
    if (lane != 0 || t0 + t >= p.T) continue;
    const size_t at = (size_t)(t0 + t) * p.N + n;
    float v = GU ? silu(a) * b : a;
    if (p.bias) v += bf16_to_f32(p.bias[n]);
    if (p.gate) v *= p.gate[t0 + t];
    if (p.add) v += bf16_to_f32(p.add[at]);
    p.y[at] = (uint16_t)f32_to_bf16_rne(v);
  }
}

template <bool GU>
moe_status launch_dense(int format, const DenseArgs& p, hipStream_t s) {
  const dim3 grid((unsigned)p.N, (unsigned)((p.T + kRowTokens - 1) / kRowTokens));
  if (format == MOE_QUANT_NVFP4) dense_row_kernel<MOE_QUANT_NVFP4, GU><<<grid, kWave, 0, s>>>(p);
  else dense_row_kernel<MOE_QUANT_MXFP4, GU><<<grid, kWave, 0, s>>>(p);
  return launch_status();
}

inline size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

}  // namespace
}  // namespace moe

extern "C" moe_status moe_quant_linear(int format, const uint16_t* x, const uint8_t* codes, const uint8_t* scales,
                                       const float* g_scale, const uint16_t* bias, int T, int N, int K, uint16_t* y,
                                       void* stream) {
  using namespace moe;
  if (!quant_format_ok(format) || T < 0 || !quant_dims_ok(N, K)) return MOE_ERR_INVALID_SHAPE;
  if (!quant_dims_fit(N, K) || T > kQuantMaxTokens) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!x || !codes || !scales || !y || (format == MOE_QUANT_NVFP4 && !g_scale)) return MOE_ERR_NULL_POINTER;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(scales) || !aligned16(y) || (bias && !aligned16(bias)) ||
      !aligned4(g_scale))
    return MOE_ERR_MISALIGNED;
  const DenseArgs p{x, {codes, scales, g_scale}, {}, bias, nullptr, nullptr, y, T, N, K};
  return launch_dense<false>(format, p, static_cast<hipStream_t>(stream));
}

extern "C" size_t moe_quant_shared_expert_workspace_size(int T, int H, int Is) {
  (void)H;
  if (T <= 0 || Is <= 0) return 0;
  return moe::align256((size_t)T * (size_t)Is * 2) + moe::align256((size_t)T * 4);
}

extern "C" moe_status moe_quant_shared_expert(int format, const uint16_t* x, const uint8_t* gate_codes,
                                              const uint8_t* gate_scales, const float* gate_g,
                                              const uint8_t* up_codes, const uint8_t* up_scales, const float* up_g,
                                              const uint8_t* down_codes, const uint8_t* down_scales,
                                              const float* down_g, const uint16_t* token_gate, const uint16_t* add,
                                              int T, int H, int Is, void* workspace, size_t workspace_bytes,
                                              uint16_t* y, void* stream) {
  using namespace moe;
  if (!quant_format_ok(format) || T < 0 || !quant_dims_ok(H, Is) || !quant_dims_ok(Is, H)) return MOE_ERR_INVALID_SHAPE;
  if (H > (1 << 15) || Is > (1 << 15) || T > kQuantMaxTokens) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  const void* need[] = {x, gate_codes, gate_scales, up_codes, up_scales, down_codes, down_scales, workspace, y};
  for (const void* q : need)
    if (!q) return MOE_ERR_NULL_POINTER;
  if (format == MOE_QUANT_NVFP4 && (!gate_g || !up_g || !down_g)) return MOE_ERR_NULL_POINTER;
  for (const void* q : need)
    if (!aligned16(q)) return MOE_ERR_MISALIGNED;
  if (!aligned16(token_gate) || !aligned16(add) || !aligned4(gate_g) || !aligned4(up_g) || !aligned4(down_g))
    return MOE_ERR_MISALIGNED;
  if (workspace_bytes < moe_quant_shared_expert_workspace_size(T, H, Is)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  uint16_t* const h = static_cast<uint16_t*>(workspace);
  float* const gate = token_gate ? reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) +
                                                            align256((size_t)T * (size_t)Is * 2)) : nullptr;
  if (gate) {
    token_gate_kernel<<<(unsigned)T, kWave, 0, s>>>(x, token_gate, H, gate);
    if (launch_status() != MOE_OK) return MOE_ERR_HIP;
  }
  const DenseArgs up{x, {gate_codes, gate_scales, gate_g}, {up_codes, up_scales, up_g}, nullptr, nullptr, nullptr,
                     h, T, Is, H};
  if (launch_dense<true>(format, up, s) != MOE_OK) return MOE_ERR_HIP;
  const DenseArgs down{h, {down_codes, down_scales, down_g}, {}, nullptr, gate, add, y, T, H, Is};
  return launch_dense<false>(format, down, s);
}
