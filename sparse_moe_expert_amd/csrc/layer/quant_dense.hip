// Dense products with 4-bit weights: moe_quant_linear and
// moe_quant_shared_expert.
//
//   linear   y[t,n] = bf16( g * sum_k x[t,k] W[n,k] + bias[n] )
//   shared   h[t,r] = bf16( SiLU(Wg[r] . x_t) * (Wu[r] . x_t) )
//            y[t,c] = bf16( add[t,c] + sigmoid(x_t . v) * (Wd[c] . h_t) )
#include "quant_common.h"

namespace moe {
namespace {

moe_status quant_product(int format, bool gate_up, const DenseArgs& p, hipStream_t s) {
  return quant_few_ok(p) ? quant_few(format, gate_up, p, s) : quant_stream(format, gate_up, p, s);
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
  const DenseArgs p{x, {codes, scales, g_scale}, {}, bias, nullptr, nullptr, y, T, N, K, nullptr, nullptr};
  return quant_product(format, false, p, static_cast<hipStream_t>(stream));
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
  const DenseArgs up{x, {gate_codes, gate_scales, gate_g}, {up_codes, up_scales, up_g}, nullptr, nullptr, nullptr,
                     h, T, Is, H, token_gate, gate};
  const moe_status st = quant_product(format, true, up, s);
  if (st != MOE_OK) return st;
  const DenseArgs down{h, {down_codes, down_scales, down_g}, {}, nullptr, gate, add, y, T, H, Is, nullptr, nullptr};
  return quant_product(format, false, down, s);
}
