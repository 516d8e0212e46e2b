// Dense products with 4-bit weights: moe_quant_linear and
// moe_quant_shared_expert.
//
//   linear   y[t,n] = bf16( g * sum_k x[t,k] W[n,k] + bias[n] )
//   shared   h[t,r] = bf16( SiLU(Wg[r] . x_t) * (Wu[r] . x_t) )
//            y[t,c] = bf16( add[t,c] + sigmoid(x_t . v) * (Wd[c] . h_t) )
//
// h is rounded to bf16, as in moe_shared_expert and moe_expert_ffn: the matrix
// instructions take it so, and its remainder would be a second down product (26
// of the 106 us of T = 4096 2048x2048 at the rate of a large one); fp16 has three
// bits more, but not the range of h nor of MXFP4's weights.  Against fp64
// a shared expert's outputs are off by 2.1e-3 to 2.3e-3 of their size, 1.6e-3 to
// 1.7e-3 of which a bf16 output alone is.
#include "quant_common.h"

namespace moe {
namespace {

size_t product_workspace(bool gate_up, int T, int N, int K) {
  if (quant_few_ok(gate_up, T, N, K) || quant_tile_ok(gate_up, T, N)) return 0;
  return quant_split_workspace(gate_up, T, N, K);
}

// `workspace`: product_workspace bytes
moe_status quant_product(int format, bool gate_up, const DenseArgs& p, void* workspace, hipStream_t s) {
  if (quant_few_ok(gate_up, p.T, p.N, p.K)) return quant_few(format, gate_up, p, s);
  if (quant_tile_ok(gate_up, p.T, p.N)) return quant_tile(format, gate_up, p, s);
  return quant_split(format, gate_up, p, workspace, s);
}

inline size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

}  // namespace
}  // namespace moe

extern "C" size_t moe_quant_linear_workspace_size(int T, int N, int K) {
  using namespace moe;
  if (T <= 0 || T > kQuantMaxTokens || !quant_dims_ok(N, K) || !quant_dims_fit(N, K)) return 0;
  return align256(product_workspace(false, T, N, K));
}

extern "C" moe_status moe_quant_linear(int format, const uint16_t* x, const uint8_t* codes, const uint8_t* scales,
                                       const float* g_scale, const uint16_t* bias, int T, int N, int K,
                                       void* workspace, size_t workspace_bytes, uint16_t* y, void* stream) {
  using namespace moe;
  if (!quant_format_ok(format) || T < 0 || !quant_dims_ok(N, K)) return MOE_ERR_INVALID_SHAPE;
  if (!quant_dims_fit(N, K) || T > kQuantMaxTokens) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!x || !codes || !scales || !y || (format == MOE_QUANT_NVFP4 && !g_scale)) return MOE_ERR_NULL_POINTER;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(scales) || !aligned16(y) || (bias && !aligned16(bias)) ||
      !aligned4(g_scale))
    return MOE_ERR_MISALIGNED;
  const size_t need = moe_quant_linear_workspace_size(T, N, K);
  if (need > 0 && !workspace) return MOE_ERR_NULL_POINTER;
  if (need > 0 && !aligned16(workspace)) return MOE_ERR_MISALIGNED;
  if (workspace_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  const DenseArgs p{x, {codes, scales, g_scale}, {}, bias, nullptr, nullptr, y, T, N, K, nullptr, nullptr};
  return quant_product(format, false, p, workspace, static_cast<hipStream_t>(stream));
}

extern "C" size_t moe_quant_shared_expert_workspace_size(int T, int H, int Is) {
  using namespace moe;
  if (T <= 0 || T > kQuantMaxTokens || !quant_dims_ok(H, Is) || !quant_dims_ok(Is, H) || H > kQuantMaxK || Is > kQuantMaxK)
    return 0;
  // h, the token gates, and the parts' sums of whichever product needs more
  const size_t up = product_workspace(true, T, Is, H), down = product_workspace(false, T, H, Is);
  return align256((size_t)T * (size_t)Is * 2) + align256((size_t)T * 4) + align256(up > down ? up : down);
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
  if (H > kQuantMaxK || Is > kQuantMaxK || T > kQuantMaxTokens) return MOE_ERR_UNSUPPORTED;
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
  uint8_t* const at_gate = static_cast<uint8_t*>(workspace) + align256((size_t)T * (size_t)Is * 2);
  uint8_t* const at_sums = at_gate + align256((size_t)T * 4);
  uint16_t* const h = static_cast<uint16_t*>(workspace);
  float* const gate = token_gate ? reinterpret_cast<float*>(at_gate) : nullptr;
  const DenseArgs up{x, {gate_codes, gate_scales, gate_g}, {up_codes, up_scales, up_g}, nullptr, nullptr, nullptr,
                     h, T, Is, H, token_gate, gate};
  const moe_status st = quant_product(format, true, up, at_sums, s);
  if (st != MOE_OK) return st;
  const DenseArgs down{h, {down_codes, down_scales, down_g}, {}, nullptr, gate, add, y, T, H, Is, nullptr, nullptr};
  return quant_product(format, false, down, at_sums, s);
}
