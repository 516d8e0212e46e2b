// The routed experts in 8 bits: moe_block_expert_ffn.
//
//   h_r = SiLU(Wg_e x_t) * (Wu_e x_t) in fp32, then in 8 bits by blocks of 128
//   o_r = Wd_e h_r
//   y_t = bf16( sum_j w[t,j] o_(t,j) ), in slot order
#include "block_tile.h"

namespace moe {
namespace {

constexpr int kFfnThreads = 256;
constexpr int kPlanThreads = 1024;

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
  // by bucket position
  uint8_t* hq;             // [R, I]
  float* hs;               // [R, blocks of I]
  float* o;                // [R, H]
  int4* items;             // {expert, first position, routes, 0}; null: each chosen expert is one item
  int* n_items;
};

// An expert's routes in pieces of up to `tt`, experts in order
__global__ __launch_bounds__(kPlanThreads) void plan_kernel(FfnArgs p, int tt) {
  __shared__ int s_sum[kPlanThreads / kWave];
  const int e = threadIdx.x, lane = e & (kWave - 1), wave = e >> 6;
  const int count = e < p.E ? p.count[e] : 0, first = e < p.E ? p.offset[e] : 0;
  const int pieces = (count + tt - 1) / tt;
  int sum = pieces;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int v = __shfl_up(sum, d, kWave);
    if (lane >= d) sum += v;
  }
  if (lane == kWave - 1) s_sum[wave] = sum;
  __syncthreads();
  int at = sum - pieces;
  for (int w = 0; w < wave; ++w) at += s_sum[w];
  for (int i = 0; i < pieces; ++i) p.items[at + i] = make_int4(e, first + i * tt, min(tt, count - i * tt), 0);
  if (e == kPlanThreads - 1) *p.n_items = at + pieces;
}

// The workgroup's item and row tile: the items go round the XCDs, an item's row
// tiles stay on one, whose L2 then holds its tokens.  False: none.
__device__ __forceinline__ bool item_of(const FfnArgs& p, int row_tiles, int4& item, int& tile) {
  const int i = (int)blockIdx.x / kXcds / row_tiles * kXcds + (int)blockIdx.x % kXcds;
  tile = (int)blockIdx.x / kXcds % row_tiles;
  if (p.items) {
    if (i >= *p.n_items) return false;
    item = p.items[i];
  } else {
    if (i >= *p.n_active) return false;
    item.x = p.active[i];
    item.y = p.offset[item.x];
    item.z = p.count[item.x];
  }
  return true;
}

// h of 128 rows of an item's routes, in 8 bits: the rows are one block, whose
// largest value goes from wave to wave through LDS
template <int TT>
__global__ __launch_bounds__(kTileThreads, 2) void gate_up_kernel(FfnArgs p, int row_tiles) {
  using T = Tile<TT, true>;
  MOE_TILE_STAGES(T)
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wave / T::WT, wt = wave % T::WT;
  int4 item;
  int tile;
  if (!item_of(p, row_tiles, item, tile)) return;
  const int e = item.x, first = item.y, toks = item.z;
  const int n0 = tile * kBlock, rows = min(kBlock, p.I - n0), kb = blocks_of(p.H), ib = blocks_of(p.I);
  T tl;
  const size_t at = ((size_t)e * p.I + n0) * (size_t)p.H, at_s = ((size_t)e * ib + tile) * (size_t)kb;
  tl.weights(p.gate.q + at, p.up.q + at, rows, p.H, wave, lane);
  auto token = [&](int r) { return (uint32_t)(p.src[first + min(r, toks - 1)] / p.k); };
  tl.rx = make_rsrc(p.x, (uint32_t)p.T * (uint32_t)p.H);
  tl.tokens(wave, lane, [&](int r) { return token(r) * (uint32_t)p.H; });
  tl.scales(p.sx, (uint32_t)p.T * (uint32_t)kb * 4u, p.gate.s + at_s, p.up.s + at_s, kb, wave, lane,
            [&](int r) { return token(r) * (uint32_t)kb * 4u; });
  const int live = (toks - wt * T::JT * 16 + 15) / 16;
  tl.template run<false>(stage_at, wave, wr, wt, lane, 0, kb, p.H, live);

  constexpr int HT = T::MT / 2;
  const int g = lane >> 4;
  uint32_t* const s_max = reinterpret_cast<uint32_t*>(s_0);            // [WR][TT]
  __syncthreads();
#pragma unroll
  for (int j = 0; j < T::JT; ++j) {
    uint32_t top = 0;
#pragma unroll
    for (int m = 0; m < HT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float h = silu(tl.acc[m][j][i]) * tl.acc[m + HT][j][i];
        tl.acc[m][j][i] = h;
        top = max(top, finite_bits(h));
      }
    top = max(top, (uint32_t)__shfl_xor((int)top, 16, kWave));
    top = max(top, (uint32_t)__shfl_xor((int)top, 32, kWave));
    if (g == 0) s_max[wr * TT + (wt * T::JT + j) * 16 + lane] = top;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < T::JT; ++j) {
    const int r = (wt * T::JT + j) * 16 + (lane & 15);
    if (r >= toks) continue;
    uint32_t top = 0;
#pragma unroll
    for (int w = 0; w < T::WR; ++w) top = max(top, s_max[w * TT + r]);
    const float s = block_scale(__uint_as_float(top)), inv = 1.0f / s;
    const size_t row = (size_t)(first + r);
    if (wr == 0 && g == 0) p.hs[row * ib + tile] = s;
#pragma unroll
    for (int m = 0; m < HT; ++m) {
      const int n = n0 + T::row_of(wr, m) + g * 4;
      const f32x4 v = tl.acc[m][j];
      if (n < p.I) *reinterpret_cast<uint32_t*>(p.hq + row * p.I + n) = encode4(v[0], v[1], v[2], v[3], inv);
    }
  }
}

// o of 256 rows of an item's routes
template <int TT>
__global__ __launch_bounds__(kTileThreads, 2) void down_kernel(FfnArgs p, int row_tiles) {
  using T = Tile<TT, false>;
  MOE_TILE_STAGES(T)
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wave / T::WT, wt = wave % T::WT;
  int4 item;
  int tile;
  if (!item_of(p, row_tiles, item, tile)) return;
  const int e = item.x, first = item.y, toks = item.z;
  const int n0 = tile * kTileRows, rows = min(kTileRows, p.H - n0), kb = blocks_of(p.I);
  T tl;
  const uint8_t* const w = p.down.q + ((size_t)e * p.H + n0) * (size_t)p.I;
  tl.weights(w, w, rows, p.I, wave, lane);
  tl.rx = make_rsrc(p.hq + (size_t)first * p.I, (uint32_t)toks * (uint32_t)p.I);
  tl.tokens(wave, lane, [&](int r) { return (uint32_t)min(r, toks - 1) * (uint32_t)p.I; });
  const float* const sw = p.down.s + ((size_t)e * blocks_of(p.H) + n0 / kBlock) * (size_t)kb;
  tl.scales(p.hs + (size_t)first * kb, (uint32_t)toks * (uint32_t)kb * 4u, sw, rows > kBlock ? sw + kb : sw, kb, wave, lane,
            [&](int r) { return (uint32_t)min(r, toks - 1) * (uint32_t)kb * 4u; });
  const int live = (toks - wt * T::JT * 16 + 15) / 16;
  tl.template run<false>(stage_at, wave, wr, wt, lane, 0, kb, p.I, live);
#pragma unroll
  for (int j = 0; j < T::JT; ++j) {
    const int r = (wt * T::JT + j) * 16 + (lane & 15);
    if (r >= toks) continue;
#pragma unroll
    for (int m = 0; m < T::MT; ++m) {
      const int n = n0 + T::row_of(wr, m) + (lane >> 4) * 4;
      if (n < p.H) *reinterpret_cast<f32x4*>(p.o + (size_t)(first + r) * p.H + n) = tl.acc[m][j];
    }
  }
}

// A thread to four outputs of a token
__global__ __launch_bounds__(kFfnThreads) void combine_kernel(FfnArgs p) {
  const size_t i = (size_t)blockIdx.x * kFfnThreads + threadIdx.x;
  const int quads = p.H / 4;
  const int t = (int)(i / (size_t)quads), n = (int)(i - (size_t)t * quads) * 4;
  if (t >= p.T) return;
  float v[4] = {};
  for (int j = 0; j < p.k; ++j) {
    const size_t route = (size_t)t * p.k + j;
    const f32x4 o = *reinterpret_cast<const f32x4*>(p.o + (size_t)p.pos[route] * p.H + n);
    const float w = p.topk_w[route];
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = fmaf(w, o[c], v[c]);
  }
  *reinterpret_cast<uint2*>(p.y + (size_t)t * p.H + n) =
      make_uint2(to_bf16(v[0]) | to_bf16(v[1]) << 16, to_bf16(v[2]) | to_bf16(v[3]) << 16);
}

// Tokens of a tile; up to that many the experts themselves are the items
int tile_tokens(int T) { return T <= 16 ? 16 : T <= 32 ? 32 : T <= 64 ? 64 : 128; }
// Most items that R routes can make
int most_items(size_t R, int E, int tt) {
  const size_t experts = R < (size_t)E ? R : (size_t)E;
  return (int)(experts + R / (size_t)tt);
}

template <int TT>
void launch_products(const FfnArgs& p, int items, hipStream_t s) {
  const unsigned groups = (unsigned)(items + kXcds - 1) / kXcds * kXcds;
  const int up = blocks_of(p.I), down = (p.H + kTileRows - 1) / kTileRows;
  gate_up_kernel<TT><<<groups * up, kTileThreads, 0, s>>>(p, up);
  down_kernel<TT><<<groups * down, kTileThreads, 0, s>>>(p, down);
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
  const int tt = tile_tokens(T);
  return align256(R * I) + align256(R * blocks_of(I) * 4) + align256(R * H * 4) +
         (T > tt ? align256((size_t)most_items(R, E, tt) * sizeof(int4)) + 256 : 0);
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
            active_experts, n_active, route_src, route_pos, y, T, H, I, E, k, nullptr, nullptr, nullptr, nullptr, nullptr};
  p.hq = take(R * I);
  p.hs = reinterpret_cast<float*>(take(R * blocks_of(I) * 4));
  p.o = reinterpret_cast<float*>(take(R * H * 4));
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const int tt = tile_tokens(T);
  int items = (int)(R < (size_t)E ? R : (size_t)E);
  if (T > tt) {
    items = most_items(R, E, tt);
    p.items = reinterpret_cast<int4*>(take((size_t)items * sizeof(int4)));
    p.n_items = reinterpret_cast<int*>(take(4));
    plan_kernel<<<1, kPlanThreads, 0, s>>>(p, tt);
  }
  switch (tt) {
    case 16: launch_products<16>(p, items, s); break;
    case 32: launch_products<32>(p, items, s); break;
    case 64: launch_products<64>(p, items, s); break;
    default: launch_products<128>(p, items, s);
  }
  combine_kernel<<<(unsigned)(((size_t)T * (H / 4) + kFfnThreads - 1) / kFfnThreads), kFfnThreads, 0, s>>>(p);
  return launch_status();
}
