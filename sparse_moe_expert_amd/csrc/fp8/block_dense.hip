// A dense layer in 8 bits: moe_block_linear.
#include "block_tile.h"

namespace moe {
namespace {

struct LinearArgs {
  const uint8_t* x;
  const float* sx;
  BlockMat w;
  const uint16_t* bias;
  uint16_t* y;
  int T, N, K;
};

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

// Tiles of 256 rows by TT tokens; with more than one part of the reduction
// (`splits`) fp32 sums go to [part][T][Np], Np rows of whole tiles.
template <int TT>
__global__ __launch_bounds__(kTileThreads, 2) void linear_tile_kernel(LinearArgs p, int row_tiles, int token_tiles, int splits,
                                                                      float* __restrict__ sums) {
  using T = Tile<TT, false>;
  MOE_TILE_STAGES(T)
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wave % T::WR, wt = wave / T::WR;
  const int tiles = row_tiles * token_tiles, per = (tiles + kXcds - 1) / kXcds;
  const int part = (int)blockIdx.x / (per * kXcds), at = (int)blockIdx.x % (per * kXcds);
  const int tile = at % kXcds * per + at / kXcds;
  if (tile >= tiles) return;
  // groups of four token tiles, row tile by row tile
  const int group = tile / (4 * row_tiles), in = tile % (4 * row_tiles), width = min(4, token_tiles - group * 4);
  const int n0 = in / width * kTileRows, t0 = (group * 4 + in % width) * TT;
  const int rows = min(kTileRows, p.N - n0), toks = min(TT, p.T - t0), kb = blocks_of(p.K);
  const int first = (int)((long long)kb * part / splits), steps = (int)((long long)kb * (part + 1) / splits) - first;

  T tl;
  const uint8_t* const w = p.w.q + (size_t)n0 * p.K;
  tl.weights(w, w, rows, p.K, wave, lane);
  tl.rx = make_rsrc(p.x + (size_t)t0 * p.K, (uint32_t)toks * (uint32_t)p.K);
  tl.tokens(wave, lane, [&](int r) { return r < toks ? (uint32_t)r * (uint32_t)p.K : kOutside; });
  const float* const sw = p.w.s + (size_t)(n0 / kBlock) * kb;
  tl.token_scales(p.sx + (size_t)t0 * kb, (uint32_t)toks * (uint32_t)kb * 4u, 4, wave, lane,
                  [&](int r) { return (uint32_t)min(r, toks - 1) * (uint32_t)kb * 4u; });
  tl.weight_scales(sw, rows > kBlock ? sw + kb : sw, kb, wave);
  tl.template run<true, true, 0>(stage_at, wave, wr, wt, lane, first, steps, 1, p.K, [](int) {}, [&](int) MOE_INLINE {
#pragma unroll
    for (int j = 0; j < T::JT; ++j) {
      const int r = (wt * T::JT + j) * 16 + (lane & 15);
      if (r >= toks) continue;
#pragma unroll
      for (int m = 0; m < T::MT; m += T::Q) {
        const int n = n0 + T::group_of(wr, m) + (lane >> 4) * (4 * T::Q);
        if (splits > 1) {
          const size_t np = (size_t)row_tiles * kTileRows;
          float* const to = sums + ((size_t)part * p.T + t0 + r) * np + n;
#pragma unroll
          for (int q = 0; q < T::Q; ++q) *reinterpret_cast<f32x4*>(to + 4 * q) = tl.acc[m + q][j];
        } else {
          float v[4 * T::Q];
#pragma unroll
          for (int i = 0; i < 4 * T::Q; ++i) v[i] = tl.acc[m + i / 4][j][i % 4];
          write(p, t0 + r, n, v);
        }
      }
    }
  }, [](int) { return true; });
}

// The parts' sums, in order, to outputs: a thread to four of a token
__global__ __launch_bounds__(256) void linear_join_kernel(LinearArgs p, int np, int splits, const float* __restrict__ sums) {
  const int quads = (p.N + 3) / 4;
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  const int t = (int)(i / (size_t)quads), n = (int)(i - (size_t)t * quads) * 4;
  if (t >= p.T) return;
  float v[4] = {};
  for (int s = 0; s < splits; ++s) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(sums + ((size_t)s * p.T + t) * (size_t)np + n);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] += a[k];
  }
  write(p, t, n, v);
}

struct Plan {
  int tt, row_tiles, token_tiles, splits;
  size_t sums() const { return splits > 1 ? (size_t)splits * row_tiles * kTileRows * 4 : 0; }      // a token
};

Plan plan_of(int T, int N, int K) {
  Plan pl;
  pl.row_tiles = (N + kTileRows - 1) / kTileRows;
  pl.tt = T <= 16 ? 16 : T <= 32 ? 32 : T <= 64 ? 64 : T <= 128 ? 128 : 256;
  if (pl.tt == 256 && (long long)pl.row_tiles * ((T + 255) / 256) < 160) pl.tt = 128;
  pl.token_tiles = (T + pl.tt - 1) / pl.tt;
  const int tiles = pl.row_tiles * pl.token_tiles, kb = blocks_of(K);
  pl.splits = tiles >= 128 ? 1 : 256 / tiles;
  if (pl.splits > kb) pl.splits = kb;
  if (pl.splits > 16) pl.splits = 16;
  while (pl.splits > 1 && pl.sums() * T > MOE_BLOCK_SUMS_BYTES) --pl.splits;
  return pl;
}

template <int TT>
void launch_tiles(const LinearArgs& p, const Plan& pl, float* sums, hipStream_t s) {
  const int tiles = pl.row_tiles * pl.token_tiles;
  const unsigned grid = (unsigned)((tiles + kXcds - 1) / kXcds * kXcds) * (unsigned)pl.splits;
  linear_tile_kernel<TT><<<grid, kTileThreads, 0, s>>>(p, pl.row_tiles, pl.token_tiles, pl.splits, sums);
}

inline bool linear_dims_ok(int N, int K) { return N >= 1 && K >= 16 && K % 16 == 0; }
inline bool linear_dims_fit(int N, int K) { return N <= (1 << 20) && K <= kBlockMaxK; }

}  // namespace
}  // namespace moe

extern "C" size_t moe_block_linear_workspace_size(int T, int N, int K) {
  using namespace moe;
  if (T <= 0 || T > kBlockMaxTokens || !linear_dims_ok(N, K) || !linear_dims_fit(N, K)) return 0;
  return align256(plan_of(T, N, K).sums() * T);
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
  const Plan pl = plan_of(T, N, K);
  float* const sums = static_cast<float*>(workspace);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  switch (pl.tt) {
    case 16: launch_tiles<16>(p, pl, sums, s); break;
    case 32: launch_tiles<32>(p, pl, sums, s); break;
    case 64: launch_tiles<64>(p, pl, sums, s); break;
    case 128: launch_tiles<128>(p, pl, sums, s); break;
    default: launch_tiles<256>(p, pl, sums, s);
  }
  if (pl.splits > 1) {
    const size_t quads = (size_t)T * ((N + 3) / 4);
    linear_join_kernel<<<(unsigned)((quads + 255) / 256), 256, 0, s>>>(p, pl.row_tiles * kTileRows, pl.splits, sums);
  }
  return launch_status();
}
