// The routed experts in 8 bits: moe_block_expert_ffn.
//
//   h_r = SiLU(Wg_e x_t) * (Wu_e x_t) in fp32, then in 8 bits by blocks of 128
//   o_r = Wd_e h_r
//   y_t = bf16( sum_j w[t,j] o_(t,j) ), in slot order
//
// Routes are grouped by expert, so that an expert's weights are read once for all
// of its routes in a tile: bound by the weight bytes while an expert has few
// routes (T = 100 2560x640 of 512 experts: 2.2 GB in 413 to 418 us, 5.2 to 5.3
// TB/s; T = 4096 2048x512 of 512: 432 to 436, of which the sums written and read are
// 70), by the products of tiles that are not full else (T = 2000 4096x2048 of 16: 184
// to 189, 1070 to 1090 TFLOP/s).
//
// h in 8 bits is what makes the second product one of 8 bits.  Where h lies next
// to the middle between two codes, what an 8-bit product cuts (block_common.h) can
// turn its code over: a token's y is off by 1.8e-3 of its size in the median (1.7e-3
// is its rounding to bf16), 4e-3 to 8e-3 in one of 100, 1.1e-2 to 1.4e-2 in the worst
// of 4096.  Up to 128 tokens the first products are made in bf16 and cut nothing:
// 1.7e-3, and 1.9e-3 in the worst, where the rounding of fp32 sums turned a code over.
#include "block_few.h"
#include "block_tile.h"

namespace moe {
namespace {

constexpr int kFfnThreads = 256;
constexpr int kPlanThreads = 1024;

// Up to so many tokens there is no plan: the chosen experts are the items
constexpr int kUnplanned = 128;

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
  float* xs;               // [blocks of H, R] the tokens' scales; null: taken from sx
  uint8_t* hq;             // [R, I]
  float* hs;               // [blocks of I, R]
  uint16_t* o;             // [R, H] fp16, over
  float* os;               // [R, blocks of H] powers of two
  int4* items;             // {expert, first position, routes, 0}; null: a chosen expert is one item
  int* n_items;
};

// Sum over the lanes up to this one
__device__ __forceinline__ int wave_scan(int v) {
  auto from = [&](auto ctrl, auto rows) {
    return __builtin_amdgcn_update_dpp(0, v, decltype(ctrl)::value, decltype(rows)::value, 0xF, false);
  };
  using std::integral_constant;
  v += from(integral_constant<int, 0x111>{}, integral_constant<int, 0xF>{});       // within rows of 16: from 1, 2, 4, 8 lanes below
  v += from(integral_constant<int, 0x112>{}, integral_constant<int, 0xF>{});
  v += from(integral_constant<int, 0x114>{}, integral_constant<int, 0xF>{});
  v += from(integral_constant<int, 0x118>{}, integral_constant<int, 0xF>{});
  v += from(integral_constant<int, 0x142>{}, integral_constant<int, 0xA>{});       // row 0's last to row 1, 2's to 3
  v += from(integral_constant<int, 0x143>{}, integral_constant<int, 0xC>{});       // lane 31 to rows 2 and 3
  return v;
}

// An item for each piece of an expert's routes, experts in order.  Pieces hold up
// to `size` routes, between half a tile and a whole one, chosen so that the
// workgroups' longest run of gate/up tiles takes the least loads: `size` token
// rows and 256 weight rows a step.  (T = 2000 4096x2048 of 16 experts: gate/up
// 127 us with whole tiles, 123 so, down 76 and 71.  The products follow a piece's
// size in steps only: of a tile of 256 tokens the waves of two of the SIMDs hold the
// first and the third 64, so that from 129 tokens on they make all of theirs.)
//
// The other workgroups copy the tokens' scales to bucket positions, a block of H
// together: of [T, blocks] the tiles would fetch a cache line for each four
// bytes (T = 4096 2048x512 of 512 experts: gate/up 257 us, and 231 so).
constexpr int kScaleRows = 64;               // positions a workgroup

template <int TT>
__global__ __launch_bounds__(kPlanThreads) void plan_kernel(FfnArgs p, int row_tiles, int groups) {
  if (blockIdx.x > 0) {
    const int R = p.T * p.k, kb = blocks_of(p.H), r = ((int)blockIdx.x - 1) * kScaleRows + (int)threadIdx.x % kScaleRows;
    if (r >= R) return;
    const float* const from = p.sx + (size_t)(p.src[r] / p.k) * kb;
    for (int b = (int)threadIdx.x / kScaleRows; b < kb; b += kPlanThreads / kScaleRows) p.xs[(size_t)b * R + r] = from[b];
    return;
  }
  // whole token tiles, so that no piece is empty
  constexpr int kSizes = TT / 32 + 1, kWaves = kPlanThreads / kWave;
  __shared__ int s_sum[kSizes][kWaves];
  __shared__ int s_before[kWaves];
  const int e = threadIdx.x, lane = e & (kWave - 1), wave = e >> 6;
  const int count = e < p.E ? p.count[e] : 0, first = e < p.E ? p.offset[e] : 0;
  for_each<kSizes>([&](auto c) MOE_INLINE {
    constexpr int C = decltype(c)::value, kSize = TT / 2 + 16 * C;
    const int sum = wave_scan((count + kSize - 1) / kSize);
    if (lane == kWave - 1) s_sum[C][wave] = sum;
  });
  __syncthreads();
  int items = 0;
  const int mine = min(lane, kSizes - 1);                    // a lane to a size
  for (int w = 0; w < kWaves; ++w) items += s_sum[mine][w];
  const long long cost = (((long long)items * row_tiles + groups - 1) / groups) * (kTileRows + TT / 2 + 16 * mine);
  int size = TT;
  long long best = __shfl(cost, kSizes - 1, kWave);
  for (int c = kSizes - 2; c >= 0; --c) {
    const long long other = __shfl(cost, c, kWave);
    if (other < best) best = other, size = TT / 2 + 16 * c;
  }
  const int pieces = (count + size - 1) / size;
  const int sum = wave_scan(pieces);
  if (lane == kWave - 1) s_before[wave] = sum;
  __syncthreads();
  int at = sum - pieces;
  for (int w = 0; w < wave; ++w) at += s_before[w];
  // even pieces, of whole token tiles
  const int even = pieces > 0 ? ((count + pieces - 1) / pieces + 15) & ~15 : 0;
  for (int i = 0; i < pieces; ++i) p.items[at + i] = make_int4(e, first + i * even, min(even, count - i * even), 0);
  if (e == kPlanThreads - 1) *p.n_items = at + pieces;
}

// Up to TT routes of an expert, from a bucket position on
struct Item {
  int expert, first, toks;
};
// (through the scalar cache: vector loads would wait for the loads in flight)
template <int TT>
__device__ __forceinline__ Item item_at(const FfnArgs& p, int i, int pass, int& longest) {
  if (TT > kUnplanned || p.items) {
    const i32x4 v = scalar_load(reinterpret_cast<const i32x4*>(p.items) + i);
    return {v[0], v[1], v[2]};
  }
  const int e = scalar_load(p.active + i), count = scalar_load(p.count + e), from = pass * TT;
  longest = max(longest, count);
  const int rest = min(count - from, TT);
  return {e, scalar_load(p.offset + e) + (rest > 0 ? from : 0), max(rest, 0)};
}

// Without a plan a chosen expert is an item, of up to T routes, unless a token
// names an expert twice: what is past TT routes of an expert then takes the
// workgroup another pass over its tiles.  Between two: the loads of the last,
// out of range, have been written, and nobody reads its stages any more.
__device__ __forceinline__ void next_pass() {
  wait_loads<0>();
  wait_lds();
  barrier();
}

// A workgroup's tiles: a run of those of all items, an item's row tiles one
// after another, so that its loads' addresses seldom change, and those of an XCD
// next to each other: workgroups that read the same tokens, and pieces of an
// expert's routes that read the same weights, share an L2.
struct Run {
  int first, tiles;
};
__device__ __forceinline__ Run run_of(const FfnArgs& p, int row_tiles) {
  const long long all = (long long)scalar_load(p.items ? p.n_items : p.n_active) * row_tiles;
  const int groups = (int)gridDim.x / kXcds, at = (int)blockIdx.x % kXcds * groups + (int)blockIdx.x / kXcds;
  const int first = (int)(all * at / (int)gridDim.x);
  return {first, (int)(all * (at + 1) / (int)gridDim.x) - first};
}

// h of 128 rows of an item's routes, in 8 bits: the rows are one block, whose
// largest value goes from wave to wave through LDS.  WIDE: products in bf16, which
// lose no bit; without a plan, where the weights' bytes mostly take longer (weights
// from HBM: T = 4 2048x512 of 512 experts 38.2 us, 37.8 in 8 bits, T = 1 23.6 and
// 21.4, T = 100 2560x640 418 and 414; of 3 experts T = 120 4096x2048 80.6 and 60.8; but
// T = 4096 2048x512 of 512 477 and 432).
template <int TT, bool WIDE>
__global__ __launch_bounds__(kTileThreads, 2) void gate_up_kernel(FfnArgs p, int row_tiles) {
  using T = Tile<TT, true, kTileRows, 1, WIDE>;
  MOE_TILE_STAGES(T)
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wave % T::WR, wt = wave / T::WR;
  __shared__ uint32_t s_max[T::WR * TT];
  const Run run = run_of(p, row_tiles);
  if (run.tiles == 0) return;
  const int kb = blocks_of(p.H), ib = blocks_of(p.I);
  T tl;
  tl.rx = make_rsrc(p.x, (uint32_t)p.T * (uint32_t)p.H);
  int pass = 0, longest = 0;                                 // an expert's routes, of those that were items
  int loaded = -1;                                           // the item that the loads' addresses are of
  Item item_in;
  auto begin = [&](int i) MOE_INLINE {
    const int at = run.first + i, number = at / row_tiles, tile = at - number * row_tiles;
    if (number != loaded) {
      loaded = number;
      item_in = item_at<TT>(p, number, pass, longest);
      auto token = [&](int r) MOE_INLINE { return (uint32_t)(p.src[item_in.first + max(min(r, item_in.toks - 1), 0)] / p.k); };
      tl.gathered_tokens(wave, lane, [&](int r) MOE_INLINE {
        const uint32_t at = token(r) * (uint32_t)p.H;
        return r < item_in.toks ? at : kOutside;
      });
      if (p.xs)
        tl.token_scales(p.xs + item_in.first, (uint32_t)item_in.toks * 4u, (size_t)p.T * p.k * 4, wave, lane,
                        [](int r) { return (uint32_t)r * 4u; });
      else
        tl.token_scales(p.sx, (uint32_t)p.T * (uint32_t)kb * 4u, 4, wave, lane,
                        [&](int r) { return token(r) * (uint32_t)kb * 4u; });
    }
    const int n0 = tile * kBlock;
    const size_t row = (size_t)item_in.expert * p.I + n0, scale = ((size_t)item_in.expert * ib + tile) * (size_t)kb;
    tl.weights(p.gate.q + row * p.H, p.up.q + row * p.H, min(kBlock, p.I - n0), p.H, wave, lane);
    tl.weight_scales(p.gate.s + scale, p.up.s + scale, kb, wave);
  };
  // The item whose sums are made.  When a tile's last step is done, the next one's
  // first kLead are issued: with more steps than that a tile, the loads are still at
  // it, and its item is theirs.
  Item item;
  int done;
  auto live = [&](int i) MOE_INLINE {
    const int number = (run.first + i) / row_tiles;
    if (number != done) {
      done = number;
      item = kb > T::kLead ? item_in : item_at<TT>(p, number, pass, longest);
    }
    return T::tiles_of(wt, item.toks);
  };
  auto end = [&](int i) MOE_INLINE {
    const int tile = (run.first + i) % row_tiles, n0 = tile * kBlock, first = item.first, toks = item.toks;
    constexpr int HT = T::HT, Q = T::Q;
    int l = lane;
    asm volatile("" : "+v"(l));                              // (addresses are made here, and not kept through the loop)
    const int g = l >> 4, n = n0 + T::group_of(wr, 0) + g * (4 * Q);
#pragma unroll
    for (int j = 0; j < T::JT; ++j) {
      float h[4 * HT];
#pragma unroll
      for (int i = 0; i < 4 * HT; ++i) {
        const float a = tl.acc[i / 4][j][i % 4];
        h[i] = a * __builtin_amdgcn_rcpf(1.0f + __expf(-a)) * tl.acc[i / 4 + HT][j][i % 4];
        tl.acc[i / 4][j][i % 4] = h[i];
      }
      uint32_t top = n < p.I ? largest(h) : 0u;              // (rows past I are not its)
      top = max(top, (uint32_t)__shfl_xor((int)top, 16, kWave));
      top = max(top, (uint32_t)__shfl_xor((int)top, 32, kWave));
      if (g == 0) s_max[wr * TT + T::token_tile(wt, j) * 16 + l] = top;
    }
    wait_lds();
    barrier();
    // every lane stores, those past the item's routes or I out of range
    const __amdgpu_buffer_rsrc_t to_q = make_rsrc(p.hq + (size_t)first * p.I, (uint32_t)toks * (uint32_t)p.I);
    const __amdgpu_buffer_rsrc_t to_s = make_rsrc(p.hs + (size_t)tile * p.T * p.k + first, (uint32_t)toks * 4u);
#pragma unroll
    for (int j = 0; j < T::JT; ++j) {
      const int r = T::token_tile(wt, j) * 16 + (l & 15);
      uint32_t top = 0;
#pragma unroll
      for (int w = 0; w < T::WR; ++w) top = max(top, s_max[w * TT + r]);
      const float s = block_scale(__uint_as_float(top));
      const float lift = lift_of(s);
      const Divisor d{s * lift, 1.0f / (s * lift)};
      __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(s), to_s,
                                            wr == 0 && g == 0 ? (uint32_t)r * 4u : kOutside, 0, 0);
      uint32_t c[Q];
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const f32x4 v = tl.acc[q][j] * lift;
        c[q] = encode4(v[0], v[1], v[2], v[3], d);
      }
      static_assert(HT == Q, "a lane's values of a token are neighbours");
      const uint32_t at = n < p.I && r < toks ? (uint32_t)r * (uint32_t)p.I + (uint32_t)n : kOutside;      // (I is a multiple of 16)
      if constexpr (Q == 4) __builtin_amdgcn_raw_buffer_store_b128(u32x4{c[0], c[1], c[2], c[3]}, to_q, at, 0, 0);
      else if constexpr (Q == 2) __builtin_amdgcn_raw_buffer_store_b64(u32x2{c[0], c[1]}, to_q, at, 0, 0);
      else __builtin_amdgcn_raw_buffer_store_b32(c[0], to_q, at, 0, 0);
    }
  };
  for (;; ++pass, next_pass()) {
    loaded = -1;
    begin(0);
    item = item_in, done = loaded;
    tl.template run<false, false, 2 * T::JT>(stage_at, wave, wr, wt, lane, 0, kb, run.tiles, p.H, begin, end, live);
    if (TT > kUnplanned || longest <= (pass + 1) * TT) break;
  }
}

// o of 256 rows of an item's routes
template <int TT>
__global__ __launch_bounds__(kTileThreads, 2) void down_kernel(FfnArgs p, int row_tiles) {
  using T = Tile<TT, false>;
  MOE_TILE_STAGES(T)
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wave % T::WR, wt = wave / T::WR;
  __shared__ uint32_t s_max[T::WR * TT];
  const Run run = run_of(p, row_tiles);
  if (run.tiles == 0) return;
  const int kb = blocks_of(p.I), hb = blocks_of(p.H);
  T tl;
  int pass = 0, longest = 0;                                 // an expert's routes, of those that were items
  int loaded = -1;                                           // the item that the loads' addresses are of
  Item item_in;
  auto begin = [&](int i) MOE_INLINE {
    const int at = run.first + i, number = at / row_tiles, n0 = (at - number * row_tiles) * kTileRows;
    if (number != loaded) {
      loaded = number;
      item_in = item_at<TT>(p, number, pass, longest);
      tl.rx = make_rsrc(p.hq + (size_t)item_in.first * p.I, (uint32_t)item_in.toks * (uint32_t)p.I);
      tl.tokens(p.I, wave, lane);
      tl.token_scales(p.hs + item_in.first, (uint32_t)item_in.toks * 4u, (size_t)p.T * p.k * 4, wave, lane,
                      [](int r) { return (uint32_t)r * 4u; });
    }
    const int rows = min(kTileRows, p.H - n0);
    const uint8_t* const w = p.down.q + ((size_t)item_in.expert * p.H + n0) * (size_t)p.I;
    tl.weights(w, w, rows, p.I, wave, lane);
    const float* const sw = p.down.s + ((size_t)item_in.expert * hb + n0 / kBlock) * (size_t)kb;
    tl.weight_scales(sw, rows > kBlock ? sw + kb : sw, kb, wave);
  };
  // The item whose sums are made.  When a tile's last step is done, the next one's
  // first kLead are issued: with more steps than that a tile, the loads are still at
  // it, and its item is theirs.
  Item item;
  int done;
  auto live = [&](int i) MOE_INLINE {
    const int number = (run.first + i) / row_tiles;
    if (number != done) {
      done = number;
      item = kb > T::kLead ? item_in : item_at<TT>(p, number, pass, longest);
    }
    return T::tiles_of(wt, item.toks);
  };
  auto end = [&](int i) MOE_INLINE {
    const int n0 = (run.first + i) % row_tiles * kTileRows, first = item.first, toks = item.toks;
    // Each route's 128 outputs over the power of two that puts the largest
    // between 2^14 and 2^15: fp16 then keeps 11 bits of every output down to 2^-28
    // of it, and loses it below 2^-40.  o in fp32 would be twice the bytes: of T =
    // 4096 2048x512 of 512 experts 168 MB more, written and read again.
    int l = lane;
    asm volatile("" : "+v"(l));                              // (addresses are made here, and not kept through the loop)
    const int g = l >> 4;
#pragma unroll
    for (int j = 0; j < T::JT; ++j) {
      float v[4 * T::MT];
#pragma unroll
      for (int i = 0; i < 4 * T::MT; ++i) v[i] = tl.acc[i / 4][j][i % 4];
#pragma unroll
      for (int m = 0; m < T::MT; m += T::Q) {                // (rows past H are not its)
        if (n0 + T::group_of(wr, m) + g * (4 * T::Q) < p.H) continue;
#pragma unroll
        for (int i = 0; i < 4 * T::Q; ++i) v[4 * m + i] = 0.0f;
      }
      uint32_t top = largest(v);
      top = max(top, (uint32_t)__shfl_xor((int)top, 16, kWave));
      top = max(top, (uint32_t)__shfl_xor((int)top, 32, kWave));
      if (g == 0) s_max[wr * TT + T::token_tile(wt, j) * 16 + l] = top;
    }
    wait_lds();
    barrier();
    constexpr int kShare = T::WR / 2;                        // waves of a block of rows
    const int block = n0 / kBlock + wr / kShare;
    // every lane stores, those past the item's routes or H out of range
    const __amdgpu_buffer_rsrc_t to_o = make_rsrc(p.o + (size_t)first * p.H, (uint32_t)toks * (uint32_t)p.H * 2u);
    const __amdgpu_buffer_rsrc_t to_s = make_rsrc(p.os + (size_t)first * hb, (uint32_t)toks * (uint32_t)hb * 4u);
#pragma unroll
    for (int j = 0; j < T::JT; ++j) {
      const int r = T::token_tile(wt, j) * 16 + (l & 15);
      uint32_t top = 0;
#pragma unroll
      for (int w = 0; w < kShare; ++w) top = max(top, s_max[(wr / kShare * kShare + w) * TT + r]);
      const uint32_t ex = max(top >> 23, 15u);
      const float inv = __uint_as_float((268u - ex) << 23);
      const bool whose = wr % kShare == 0 && g == 0 && r < toks && block < hb;
      __builtin_amdgcn_raw_buffer_store_b32((ex - 14u) << 23, to_s, whose ? (uint32_t)(r * hb + block) * 4u : kOutside, 0, 0);
#pragma unroll
      for (int m = 0; m < T::MT; m += T::Q) {
        const int n = n0 + T::group_of(wr, m) + g * (4 * T::Q);
        uint32_t c[2 * T::Q];
#pragma unroll
        for (int q = 0; q < T::Q; ++q) {
          const f32x4 v = tl.acc[m + q][j];
          c[2 * q] = f32_to_f16_bits(v[0] * inv) | f32_to_f16_bits(v[1] * inv) << 16;
          c[2 * q + 1] = f32_to_f16_bits(v[2] * inv) | f32_to_f16_bits(v[3] * inv) << 16;
        }
        const uint32_t at = n < p.H && r < toks ? ((uint32_t)r * (uint32_t)p.H + (uint32_t)n) * 2u : kOutside;       // (H is a multiple of 16)
#pragma unroll
        for (int q = 0; q < T::Q / 2; ++q)
          __builtin_amdgcn_raw_buffer_store_b128(u32x4{c[4 * q], c[4 * q + 1], c[4 * q + 2], c[4 * q + 3]}, to_o, at + 16 * q, 0, 0);
      }
    }
  };
  for (;; ++pass, next_pass()) {
    loaded = -1;
    begin(0);
    item = item_in, done = loaded;
    tl.template run<false, false, (1 + T::MT / 2) * T::JT>(stage_at, wave, wr, wt, lane, 0, kb, run.tiles, p.I, begin, end, live);
    if (TT > kUnplanned || longest <= (pass + 1) * TT) break;
  }
}

// A thread to eight outputs of a token
__global__ __launch_bounds__(kFfnThreads) void combine_kernel(FfnArgs p) {
  const size_t i = (size_t)blockIdx.x * kFfnThreads + threadIdx.x;
  const int pieces = p.H / 8, hb = blocks_of(p.H);
  const int t = (int)(i / (size_t)pieces), n = (int)(i - (size_t)t * pieces) * 8;
  if (t >= p.T) return;
  float v[8] = {};
  const int32_t* const pos = p.pos + (size_t)t * p.k;
  const float* const weight = p.topk_w + (size_t)t * p.k;
  constexpr int kAhead = 4;                                  // routes whose loads are in flight together
  for (int j0 = 0; j0 < p.k; j0 += kAhead) {
    uint4 o[kAhead];
    float w[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int j = min(j0 + a, p.k - 1);
      const size_t row = (size_t)pos[j];
      o[a] = *reinterpret_cast<const uint4*>(p.o + row * p.H + n);
      w[a] = weight[j] * p.os[row * hb + n / kBlock];
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      if (j0 + a >= p.k) break;
      const uint32_t u[4] = {o[a].x, o[a].y, o[a].z, o[a].w};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        v[2 * c] = fmaf(w[a], f16_bits_to_f32(u[c] & 0xFFFFu), v[2 * c]);
        v[2 * c + 1] = fmaf(w[a], f16_bits_to_f32(u[c] >> 16), v[2 * c + 1]);
      }
    }
  }
  *reinterpret_cast<uint4*>(p.y + (size_t)t * p.H + n) =
      make_uint4(to_bf16(v[0]) | to_bf16(v[1]) << 16, to_bf16(v[2]) | to_bf16(v[3]) << 16,
                 to_bf16(v[4]) | to_bf16(v[5]) << 16, to_bf16(v[6]) | to_bf16(v[7]) << 16);
}

// Few routes: ROWS outputs of every token.  A wave takes the chosen experts in
// turn, all of an expert's reduction at once; the routes' sums meet in LDS, where
// a token's are added in slot order.  Bound by the weight bytes, and at one
// workgroup a compute unit by how many of those read: 8 rows, half a product's,
// where that many workgroups all run at once (weights in the Infinity Cache: T = 4
// 2048x512 of 512 experts, 40 chosen, 11.9 us, 15.6 with 16 rows; 2048x1024 of 64
// 10.2 and 12.6; but 2304x512 of 256 18.7 and 13.4).  In a launch of its own the sum
// took 5 us more.
constexpr int kDownWaves = 16;
constexpr int kDownGroups = 256;             // workgroups that run at once, one on a compute unit
constexpr int kDownThreads = kDownWaves * kWave;
constexpr int kDownRoutes = 512;             // most, of up to 16 tokens

template <int ROWS>
__global__ __launch_bounds__(kDownThreads, 4) void down_combine_kernel(FfnArgs p) {
  __shared__ float s_o[kDownRoutes][ROWS + 1], s_weight[kDownRoutes];
  __shared__ int s_expert[kDownRoutes][3], s_pos[kDownRoutes];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4, n0 = (int)blockIdx.x * ROWS;
  const int R = p.T * p.k, kb = blocks_of(p.I), hb = blocks_of(p.H);
  // all that the weights' addresses and the sums go by, once
  for (int i = tid; i < R; i += kDownThreads) {
    const int a = min(i, p.E - 1), active = *p.n_active, e = p.active[a];
    const float weight = p.topk_w[i];
    const int pos = p.pos[i];
    if (a < active) s_expert[a][0] = e, s_expert[a][1] = p.offset[e], s_expert[a][2] = p.count[e];
    s_weight[i] = weight, s_pos[i] = pos;
  }
  __syncthreads();
  const int active = scalar_load(p.n_active);
  for (int a = wave; a < active; a += kDownWaves) {
    const int e = __builtin_amdgcn_readfirstlane(s_expert[a][0]), first = __builtin_amdgcn_readfirstlane(s_expert[a][1]);
    const int count = __builtin_amdgcn_readfirstlane(s_expert[a][2]);
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(p.down.q + ((size_t)e * p.H + n0) * (size_t)p.I, (uint32_t)(ROWS * p.I));
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(p.hq, (uint32_t)R * (uint32_t)p.I);
    const float* const sw = p.down.s + ((size_t)e * hb + n0 / kBlock) * (size_t)kb;
    for (int c0 = 0; c0 < count; c0 += 16) {                 // (more than 16 where a token names an expert twice)
      const int r = first + min(c0 + l16, count - 1);
      f32x4 sum{};
      constexpr int kAhead = 4;                              // blocks whose loads are in flight together
      for (int b0 = 0; b0 < kb; b0 += kAhead) {
        i32x8 w[kAhead], x[kAhead];
        float s[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          w[i] = load_block(rw, (uint32_t)(l16 * p.I), b0 + i, p.I, g);
          x[i] = load_block(rx, (uint32_t)(r * p.I), b0 + i, p.I, g);
          const int b = min(b0 + i, kb - 1);
          s[i] = p.hs[(size_t)b * R + r] * scalar_load(sw + b);
        }
        __builtin_amdgcn_sched_barrier(0);                   // (all loads first)
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          if (b0 + i >= kb) break;
          const f32x4 d = block_product(w[i], x[i]);
#pragma unroll
          for (int c = 0; c < 4; ++c) sum[c] = fmaf(d[c], s[i], sum[c]);
        }
      }
      if (c0 + l16 < count && g * 4 < ROWS) {
#pragma unroll
        for (int c = 0; c < 4; ++c) s_o[r][g * 4 + c] = sum[c];
      }
    }
  }
  __syncthreads();
  for (int i = tid; i < p.T * ROWS; i += kDownThreads) {
    const int t = i / ROWS, n = i % ROWS;
    float v = 0.0f;
    for (int j = 0; j < p.k; ++j) v = fmaf(s_weight[t * p.k + j], s_o[s_pos[t * p.k + j]][n], v);
    p.y[(size_t)t * p.H + n0 + n] = (uint16_t)to_bf16(v);
  }
}

// Tokens of a tile.  Beyond 128 by an expert's routes on average: wide tiles need
// fewer weight loads, narrow ones waste less (2048x512: 125 routes 72.8 us with 256,
// 91.9 with 128, 80 routes 458 and 429; 4096x2048: 125 routes 126 and 140, 75
// routes 121 and 116).
int tile_tokens(int T, int E, int k) {
  if (T <= kUnplanned) return T <= 16 ? 16 : T <= 32 ? 32 : T <= 64 ? 64 : 128;
  return (long long)T * k >= 100ll * E ? 256 : 128;
}
// Most items that R routes can make, in pieces of half a tile or more
int most_items(size_t R, int E, int tt) {
  const size_t experts = R < (size_t)E ? R : (size_t)E;
  return (int)(experts + 2 * R / (size_t)tt);
}

template <int TT>
void launch_products(const FfnArgs& p, int items, hipStream_t s) {
  const int up = blocks_of(p.I), down = (p.H + kTileRows - 1) / kTileRows;
  const int most = (device_cu_count() + kXcds - 1) / kXcds * kXcds;    // a workgroup takes a compute unit's LDS
  auto grid = [&](int row_tiles) {
    const long long tiles = ((long long)items * row_tiles + kXcds - 1) / kXcds * kXcds;
    return (unsigned)(tiles < most ? tiles : most);
  };
  if constexpr (TT <= kUnplanned)
    if (!p.items) gate_up_kernel<TT, true><<<grid(up), kTileThreads, 0, s>>>(p, up);
  if constexpr (TT >= kUnplanned)
    if (p.items) gate_up_kernel<TT, false><<<grid(up), kTileThreads, 0, s>>>(p, up);
  if constexpr (TT == 16) {
    if (p.H / 8 <= kDownGroups) down_combine_kernel<8><<<(unsigned)p.H / 8, kDownThreads, 0, s>>>(p);
    else down_combine_kernel<16><<<(unsigned)p.H / 16, kDownThreads, 0, s>>>(p);
  } else {
    down_kernel<TT><<<grid(down), kTileThreads, 0, s>>>(p, down);
    combine_kernel<<<(unsigned)(((size_t)p.T * (p.H / 8) + kFfnThreads - 1) / kFfnThreads), kFfnThreads, 0, s>>>(p);
  }
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
  return align256(R * I) + align256(R * blocks_of(I) * 4) + align256(R * H * 2) + align256(R * blocks_of(H) * 4) +
         (T > kUnplanned ? align256((size_t)most_items(R, E, 128) * sizeof(int4)) + 256 + align256(R * blocks_of(H) * 4) : 0);
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
            active_experts, n_active, route_src, route_pos, y, T, H, I, E, k, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr};
  p.hq = take(R * I);
  p.hs = reinterpret_cast<float*>(take(R * blocks_of(I) * 4));
  p.o = reinterpret_cast<uint16_t*>(take(R * H * 2));
  p.os = reinterpret_cast<float*>(take(R * blocks_of(H) * 4));
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const int tt = tile_tokens(T, E, k);
  int items = (int)(R < (size_t)E ? R : (size_t)E);
  if (T > kUnplanned) {
    items = most_items(R, E, tt);
    p.items = reinterpret_cast<int4*>(take((size_t)items * sizeof(int4)));
    p.n_items = reinterpret_cast<int*>(take(4));
    p.xs = reinterpret_cast<float*>(take(R * blocks_of(H) * 4));
    const unsigned grid = 1 + (unsigned)((R + kScaleRows - 1) / kScaleRows);
    if (tt == 128) plan_kernel<128><<<grid, kPlanThreads, 0, s>>>(p, blocks_of(I), device_cu_count());
    else plan_kernel<256><<<grid, kPlanThreads, 0, s>>>(p, blocks_of(I), device_cu_count());
  }
  switch (tt) {
    case 16: launch_products<16>(p, items, s); break;
    case 32: launch_products<32>(p, items, s); break;
    case 64: launch_products<64>(p, items, s); break;
    case 128: launch_products<128>(p, items, s); break;
    default: launch_products<256>(p, items, s);
  }
  return launch_status();
}
