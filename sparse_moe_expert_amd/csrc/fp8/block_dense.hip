// A dense layer in 8 bits: moe_block_linear.
//
// Few tokens are bound by the weight bytes (block_few.hip), more of them by the
// products, of which each is worth its loads only in tiles of many rows and
// tokens; where such tiles are too few for the chip, smaller ones take more loads
// in less time.  (T = 32 9999x4096 13.5 us, 3.1 TB/s, with the weights from HBM, 9.8
// with one weight read again and again, from the Infinity Cache; T = 333 2560x5200
// 18.8 and 17.9; 4096^3 66.4 and 63.6, 2070 and 2160 TFLOP/s.)
#include "block_linear.h"
#include "block_tile.h"

namespace moe {
namespace {

// Tiles of ROWS rows by TT tokens; with more than one part of the reduction
// (`splits`) fp32 sums go to [part][T][Np], Np rows of whole tiles.
template <int TT, int ROWS, int U>
__global__ __launch_bounds__(kTileThreads, 2) void linear_tile_kernel(LinearArgs p, int row_tiles, int token_tiles, int splits,
                                                                      float* __restrict__ sums) {
  using T = Tile<TT, false, ROWS, U>;
  MOE_TILE_STAGES(T)
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wave % T::WR, wt = wave / T::WR;
  const int tiles = row_tiles * token_tiles, per = (tiles + kXcds - 1) / kXcds;
  const int part = (int)blockIdx.x / (per * kXcds), at = (int)blockIdx.x % (per * kXcds);
  const int tile = at % kXcds * per + at / kXcds;
  if (tile >= tiles) return;
  // groups of four token tiles, row tile by row tile
  const int group = tile / (4 * row_tiles), in = tile % (4 * row_tiles), width = min(4, token_tiles - group * 4);
  const int n0 = in / width * ROWS, t0 = (group * 4 + in % width) * TT;
  const int rows = min(ROWS, p.N - n0), toks = min(TT, p.T - t0), kb = blocks_of(p.K);
  const int all = (kb + U - 1) / U, first = (int)((long long)all * part / splits);
  const int steps = (int)((long long)all * (part + 1) / splits) - first;

  T tl;
  const uint8_t* const w = p.w.q + (size_t)n0 * p.K;
  tl.weights(w, w, rows, p.K, wave, lane);
  tl.rx = make_rsrc(p.x + (size_t)t0 * p.K, (uint32_t)toks * (uint32_t)p.K);
  tl.tokens(p.K, wave, lane);
  const float* const sw = p.w.s + (size_t)(n0 / kBlock) * kb;
  tl.token_scales(p.sx + (size_t)t0 * kb, (uint32_t)toks * (uint32_t)kb * 4u, 4, wave, lane,
                  [&](int r) { return (uint32_t)min(r, toks - 1) * (uint32_t)kb * 4u; });
  tl.weight_scales(sw, rows > kBlock ? sw + kb : sw, kb, wave);
  tl.template run<true, true, 0>(stage_at, wave, wr, wt, lane, first, steps, 1, p.K, [](int) {}, [&](int) MOE_INLINE {
#pragma unroll
    for (int j = 0; j < T::JT; ++j) {
      const int r = T::token_tile(wt, j) * 16 + (lane & 15);
      if (r >= toks) continue;
#pragma unroll
      for (int m = 0; m < T::MT; m += T::Q) {
        const int n = n0 + T::group_of(wr, m) + (lane >> 4) * (4 * T::Q);
        if (splits > 1) {
          const size_t np = (size_t)row_tiles * ROWS;
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
  }, [](int) { return T::JT; });
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

// (the size of a workspace does not go by the device that asks)
constexpr int kComputeUnits = 256;

// A kernel of tiles: its tokens, rows, blocks a step; about what a workgroup's
// start and end take and a block of its reduction, in ns, measured with up to 256
// tiles on one weight.  A block's bytes over its time are 39 to 57 KB a us for every
// kind: it goes by what a compute unit brings into its LDS.  (Weights from HBM, rows
// x tokens: T = 333 2560x5200 18.6 us with 64x64 tiles, 22.2 with 128x64 in two parts;
// T = 500 2048x2048 8.7, 10.7 with 128x64, 15.3 with 128x128; T = 1000 4096x4096
// 30.5 with 128x128, 37.1 with 128x64, 41.7 with 256x128; T = 2000 2560x2560 27.8
// with 256x128, 36.9 with 128x128.)
struct Kind {
  int tt, rows, unit;
  float start_ns, block_ns;
};
constexpr Kind kKinds[] = {{256, 256, 1, 9000.0f, 1650.0f}, {128, 256, 1, 5500.0f, 1080.0f}, {128, 128, 1, 3400.0f, 670.0f},
                           {64, 128, 1, 2400.0f, 430.0f},   {64, 64, 2, 1900.0f, 330.0f},    {32, 64, 2, 1500.0f, 210.0f}};

struct Plan {
  int kind, row_tiles, token_tiles, splits;
  size_t sums() const { return splits > 1 ? (size_t)splits * row_tiles * kKinds[kind].rows * 4 : 0; }       // a token
};

// The kind and number of parts that should take least: rounds of workgroups, one
// on a compute unit, and where there are parts (few tiles, a long reduction) their
// sums written and joined.
Plan plan_of(int T, int N, int K) {
  Plan best{};
  float least = 0.0f;
  const int kb = blocks_of(K), units = kComputeUnits;
  for (int kind = 0; kind < (int)(sizeof(kKinds) / sizeof(kKinds[0])); ++kind) {
    const Kind& c = kKinds[kind];
    Plan pl{kind, (N + c.rows - 1) / c.rows, (T + c.tt - 1) / c.tt, 1};
    const long long tiles = (long long)pl.row_tiles * pl.token_tiles;
    const int steps = (kb + c.unit - 1) / c.unit;
    for (pl.splits = 1; pl.splits <= 16 && pl.splits <= steps; ++pl.splits) {
      if (pl.splits > 1 && (tiles * pl.splits > units || pl.sums() * T > MOE_BLOCK_SUMS_BYTES)) break;
      const long long rounds = (tiles * pl.splits + units - 1) / units;
      float ns = (float)rounds * (c.start_ns + (float)((steps + pl.splits - 1) / pl.splits * c.unit) * c.block_ns);
      if (pl.splits > 1) ns += 4000.0f + (float)(pl.sums() * T) / 3000.0f;
      if (least == 0.0f || ns < least) least = ns, best = pl;
    }
  }
  return best;
}

template <int KIND>
void launch_tiles(const LinearArgs& p, const Plan& pl, float* sums, hipStream_t s) {
  constexpr Kind c = kKinds[KIND];
  const int tiles = pl.row_tiles * pl.token_tiles;
  const unsigned grid = (unsigned)((tiles + kXcds - 1) / kXcds * kXcds) * (unsigned)pl.splits;
  linear_tile_kernel<c.tt, c.rows, c.unit><<<grid, kTileThreads, 0, s>>>(p, pl.row_tiles, pl.token_tiles, pl.splits, sums);
}

inline bool linear_dims_ok(int N, int K) { return N >= 1 && K >= 16 && K % 16 == 0; }
inline bool linear_dims_fit(int N, int K) { return N <= (1 << 20) && K <= kBlockMaxK; }

}  // namespace
}  // namespace moe

extern "C" size_t moe_block_linear_workspace_size(int T, int N, int K) {
  using namespace moe;
  if (T <= 0 || T > kBlockMaxTokens || !linear_dims_ok(N, K) || !linear_dims_fit(N, K) || linear_few_ok(T, N, K)) return 0;
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
  if (linear_few_ok(T, N, K)) return linear_few(p, static_cast<hipStream_t>(stream));
  const Plan pl = plan_of(T, N, K);
  float* const sums = static_cast<float*>(workspace);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  switch (pl.kind) {
    case 0: launch_tiles<0>(p, pl, sums, s); break;
    case 1: launch_tiles<1>(p, pl, sums, s); break;
    case 2: launch_tiles<2>(p, pl, sums, s); break;
    case 3: launch_tiles<3>(p, pl, sums, s); break;
    case 4: launch_tiles<4>(p, pl, sums, s); break;
    default: launch_tiles<5>(p, pl, sums, s);
  }
  if (pl.splits > 1) {
    const size_t quads = (size_t)T * ((N + 3) / 4);
    linear_join_kernel<<<(unsigned)((quads + 255) / 256), 256, 0, s>>>(p, pl.row_tiles * kKinds[pl.kind].rows, pl.splits, sums);
  }
  return launch_status();
}
