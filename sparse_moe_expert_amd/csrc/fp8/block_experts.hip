// The routed experts in 8 bits: moe_block_expert_ffn.
//
//   h_r = SiLU(Wg_e x_t) * (Wu_e x_t) in fp32, then in 8 bits by blocks of 128
//   o_r = Wd_e h_r
//   y_t = bf16( sum_j w[t,j] o_(t,j) ), in slot order
#include "block_common.h"

namespace moe {
namespace {

constexpr int kFfnThreads = 256;

struct FfnArgs {
  const uint8_t* x;
  const float* sx;
  BlockMat gate, up, down;
  const float* topk_w;
  const int32_t* count;
  const int32_t* offset;
  const int32_t* active;
  const int32_t* n_active;
  const int32_t* src;
  const int32_t* pos;
  uint16_t* y;
  int T, H, I, E, k;
  float* h;                // [R, I], by bucket position, as are those below
  uint8_t* hq;             // [R, I]
  float* hs;               // [R, blocks of I]
  float* o;                // [R, H]
};

// 16 rows of `w` times 16 token columns
__device__ __forceinline__ f32x4 tile_product(const BlockMat& w, int e, int n0, int N, int K, const uint8_t* xrow,
                                              const float* sx, int lane) {
  const int l16 = lane & 15, g = lane >> 4, kb = blocks_of(K);
  const __amdgpu_buffer_rsrc_t rw =
      make_rsrc(w.q + ((size_t)e * N + n0) * (size_t)K, (uint32_t)(min(16, N - n0) * K));
  const float* const sw = w.s + ((size_t)e * blocks_of(N) + n0 / kBlock) * (size_t)kb;
  f32x4 acc{};
  for (int b = 0; b < kb; ++b) {
    const int lo = b * kBlock + g * 16, hi = lo + 64;
    const uint32_t row = (uint32_t)(l16 * K);
    const i32x8 a = load_fragment(rw, lo < K ? row + lo : kOutside, hi < K ? row + hi : kOutside);
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const i32x8 x = fragment(lo < K ? *reinterpret_cast<const uint4*>(xrow + lo) : zero,
                             hi < K ? *reinterpret_cast<const uint4*>(xrow + hi) : zero);
    const f32x4 d = block_product(a, x);
    const float s = sx[b] * sw[b];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = fmaf(d[i], s, acc[i]);
  }
  return acc;
}

// grid (active experts, rows / 64): a wavefront to 16 rows, all of the expert's routes
template <bool GU>
__global__ __launch_bounds__(kFfnThreads) void experts_kernel(FfnArgs p) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x >> 6;
  if ((int)blockIdx.x >= *p.n_active) return;
  const int e = p.active[blockIdx.x], first = p.offset[e], count = p.count[e];
  const int N = GU ? p.I : p.H, K = GU ? p.H : p.I;
  const int n0 = ((int)blockIdx.y * 4 + wave) * 16;
  if (n0 >= N) return;
  for (int c = 0; c < count; c += 16) {
    const int r = first + min(c + (lane & 15), count - 1);
    const size_t row = GU ? (size_t)(p.src[r] / p.k) : (size_t)r;
    const uint8_t* const x = (GU ? p.x : p.hq) + row * K;
    const float* const sx = (GU ? p.sx : p.hs) + row * blocks_of(K);
    f32x4 v = tile_product(GU ? p.gate : p.down, e, n0, N, K, x, sx, lane);
    if constexpr (GU) {
      const f32x4 u = tile_product(p.up, e, n0, N, K, x, sx, lane);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = silu(v[i]) * u[i];
    }
    if (c + (lane & 15) >= count) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = n0 + (lane >> 4) * 4 + i;
      if (n < N) (GU ? p.h : p.o)[(size_t)r * N + n] = v[i];
    }
  }
}

// h in 8 bits: 16 lanes to a block
__global__ __launch_bounds__(kFfnThreads) void quantize_h_kernel(FfnArgs p, size_t blocks) {
  const int ib = blocks_of(p.I);
  const size_t block = (size_t)blockIdx.x * (kFfnThreads / 16) + (threadIdx.x >> 4);
  if (block >= blocks) return;
  const size_t r = block / (size_t)ib;
  const int at = (int)(block - r * (size_t)ib) * kBlock + (threadIdx.x & 15) * 8;
  float v[8] = {};
  if (at < p.I)
    for (int i = 0; i < 8; ++i) v[i] = p.h[r * p.I + at + i];
  uint32_t m = 0;
  for (int i = 0; i < 8; ++i) m = max(m, finite_bits(v[i]));
  const float s = block_scale(__uint_as_float(max16(m)));
  const float inv = 1.0f / s;
  if (at >= p.I) return;
  *reinterpret_cast<uint2*>(p.hq + r * p.I + at) =
      make_uint2(encode4(v[0], v[1], v[2], v[3], inv), encode4(v[4], v[5], v[6], v[7], inv));
  if ((threadIdx.x & 15) == 0) p.hs[block] = s;
}

__global__ __launch_bounds__(kFfnThreads) void combine_kernel(FfnArgs p) {
  const size_t at = (size_t)blockIdx.x * kFfnThreads + threadIdx.x;
  const size_t t = at / (size_t)p.H;
  if (t >= (size_t)p.T) return;
  const int n = (int)(at - t * (size_t)p.H);
  float sum = 0.0f;
  for (int j = 0; j < p.k; ++j) {
    const size_t route = t * p.k + j;
    sum = fmaf(p.topk_w[route], p.o[(size_t)p.pos[route] * p.H + n], sum);
  }
  p.y[at] = (uint16_t)to_bf16(sum);
}

inline bool ffn_dims_ok(int T, int H, int I, int E, int k) {
  return T >= 0 && H >= 16 && H % 16 == 0 && I >= 16 && I % 16 == 0 && E >= 1 && k >= 1 && k <= E;
}
inline bool ffn_dims_fit(int T, int H, int I, int E, int k) {
  return E <= 1024 && k <= 32 && H <= kBlockMaxK && I <= kBlockMaxK && (size_t)T * (size_t)k <= (1u << 24) &&
         (size_t)T * (size_t)H < (1u << 31);
}

}  // namespace
}  // namespace moe

extern "C" size_t moe_block_expert_ffn_workspace_size(int T, int H, int I, int E, int k) {
  using namespace moe;
  if (T <= 0 || !ffn_dims_ok(T, H, I, E, k) || !ffn_dims_fit(T, H, I, E, k)) return 0;
  const size_t R = (size_t)T * (size_t)k;
  return align256(R * I * 4) + align256(R * I) + align256(R * blocks_of(I) * 4) + align256(R * H * 4);
}

extern "C" moe_status moe_block_expert_ffn(const uint8_t* x, const float* x_scale, const uint8_t* w_gate,
                                           const float* s_gate, const uint8_t* w_up, const float* s_up,
                                           const uint8_t* w_down, const float* s_down, const float* topk_w,
                                           const int32_t* expert_count, const int32_t* expert_offset,
                                           const int32_t* active_experts, const int32_t* n_active,
                                           const int32_t* route_src, const int32_t* route_pos, int T, int H, int I,
                                           int E, int k, void* workspace, size_t workspace_bytes, uint16_t* y,
                                           void* stream) {
  using namespace moe;
  if (!ffn_dims_ok(T, H, I, E, k)) return MOE_ERR_INVALID_SHAPE;
  if (!ffn_dims_fit(T, H, I, E, k)) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  const void* const all[] = {x,      x_scale,      w_gate,        s_gate,         w_up,     s_up,      w_down,    s_down,
                             topk_w, expert_count, expert_offset, active_experts, n_active, route_src, route_pos, workspace, y};
  for (const void* a : all)
    if (!a) return MOE_ERR_NULL_POINTER;
  for (const void* a : all)
    if (!aligned16(a)) return MOE_ERR_MISALIGNED;
  if (workspace_bytes < moe_block_expert_ffn_workspace_size(T, H, I, E, k)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  const size_t R = (size_t)T * (size_t)k;
  uint8_t* at = static_cast<uint8_t*>(workspace);
  auto take = [&](size_t n) { uint8_t* const b = at; at += align256(n); return b; };
  FfnArgs p{x, x_scale, {w_gate, s_gate}, {w_up, s_up}, {w_down, s_down}, topk_w, expert_count, expert_offset,
            active_experts, n_active, route_src, route_pos, y, T, H, I, E, k, nullptr, nullptr, nullptr, nullptr};
  p.h = reinterpret_cast<float*>(take(R * I * 4));
  p.hq = take(R * I);
  p.hs = reinterpret_cast<float*>(take(R * blocks_of(I) * 4));
  p.o = reinterpret_cast<float*>(take(R * H * 4));
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const unsigned experts = (unsigned)(R < (size_t)E ? R : (size_t)E);
  experts_kernel<true><<<dim3(experts, (unsigned)(I + 63) / 64), kFfnThreads, 0, s>>>(p);
  const size_t blocks = R * blocks_of(I);
  quantize_h_kernel<<<(unsigned)((blocks + kFfnThreads / 16 - 1) / (kFfnThreads / 16)), kFfnThreads, 0, s>>>(p, blocks);
  experts_kernel<false><<<dim3(experts, (unsigned)(H + 63) / 64), kFfnThreads, 0, s>>>(p);
  combine_kernel<<<(unsigned)(((size_t)T * H + kFfnThreads - 1) / kFfnThreads), kFfnThreads, 0, s>>>(p);
  return launch_status();
}
