// The products of a tile: ROWS weight rows (of a gate/up pair 128 of each) by TT
// tokens, by a workgroup of eight waves.
//
// Tokens, weights and scales go straight to LDS (buffer_load ... lds), U blocks
// of 128 of the reduction a step, in a ring of NS stages.  A row's step is 128
// bytes, its 16-byte chunks permuted so that the reads of 16 lanes, one chunk of
// the 16 rows of a product, hit all banks.  The rows of Q products are
// interleaved by fours, so that a lane's sums of them are 4Q neighbouring outputs
// of a token.  The waves stand WR x WT over the tile; a wave holds
// the step's fragments of its JT token tiles and goes through its MT row tiles,
// each product followed, three products later, by the four multiply-adds that
// scale it onto the sums: the matrix pipe and the vector pipe then work side by
// side.
//
// What bounds it: of 4096^3 a step of 256 x 256 takes 1.2 us with its loads left
// out, 1.0 with its products left out, and 1.7 whole.  The 72 loads of a step and
// the waves' reads of the products' operands share the path into LDS, and one
// workgroup fills a compute unit's LDS, so that nothing else runs meanwhile.
#pragma once

#include "block_common.h"

#include <type_traits>

// of a lambda: its captures stay in registers
#define MOE_INLINE __attribute__((always_inline))

namespace moe {
namespace {

constexpr int kTileThreads = 512;
constexpr int kTileRows = 256;
constexpr int kXcds = 8;

__device__ __forceinline__ void fence() { asm volatile("" ::: "memory"); }

// s_waitcnt vmcnt(N), as the compiler's own, which then does not wait for what
// came before once more
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N < 64, "six bits");
  fence();
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0F70);
  fence();
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// Workgroup barrier without the fence of __syncthreads(), which would wait for
// every load in flight
__device__ __forceinline__ void barrier() {
  fence();
  __builtin_amdgcn_s_barrier();
  fence();
}

// f(integral_constant 0 .. N-1), unrolled
template <int N, int I = 0, class F>
__device__ __forceinline__ void for_each(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    for_each<N, I + 1>(f);
  }
}

// A stage: the weights of a step with all its scales, and the tokens
struct Stage {
  uint8_t* w;
  uint8_t* x;
};

// ROWS: weight rows of the tile (256 of a pair, 128 of each matrix); U: blocks of
// the reduction a step; WIDE: products in bf16
template <int TT, bool PAIR, int ROWS = kTileRows, int U = 1, bool WIDE = false>
struct Tile {
  static constexpr int WR = TT == ROWS ? 2 : TT == 16 ? 8 : 4, WT = 8 / WR;
  static constexpr int MT = ROWS / WR / 16, JT = TT / WT / 16;        // row tiles, token tiles a wave
  static constexpr int HT = PAIR ? MT / 2 : MT, Q = HT < 4 ? HT : 4;       // row tiles of one matrix, interleaved ones
  static constexpr int kWeightBytes = U * ROWS * kBlock, kTokenBytes = U * TT * kBlock;
  static constexpr int kScaleGroups = (TT + 63) / 64 + 2;                  // 64 of the tokens' scales each, and the weights'
  static constexpr int kScaledBytes = kWeightBytes + U * kScaleGroups * 256;         // the weights and all scales
  static constexpr int kFit = 160 * 1024 / (kScaledBytes + kTokenBytes), NS = kFit < 4 ? kFit : 4, kLead = NS - 1;
  static constexpr int WL = U * ROWS / 64, XL = U * TT < 64 ? 1 : U * TT / 64;       // a wave's loads of 1 KB a step
  static constexpr int kLoads = WL + 1 + XL;
  static constexpr uint32_t kStep = U * kBlock, kNoStep = kOutside / kStep;          // a step's bytes of a row; one past all
  static_assert(NS >= 2 && (kLead - 1) * kLoads < 48, "two stages or more, and stores behind the loads");
  static_assert(U * kScaleGroups <= 8 && (ROWS == kTileRows || !PAIR), "one load of scales a wave");

  __amdgpu_buffer_rsrc_t rw, rx;             // the wave's weight rows, the tokens
  const float* s_from;                       // the wave's scales
  uint32_t s_bytes, s_blocks;                // s_blocks: a row's
  size_t s_stride;
  uint32_t w_off[WL], s_off;
  uint32_t x_off[PAIR ? XL : 1], x_row;      // of a pair's tokens, gathered; else of the first piece's, 64 rows apart
  uint32_t token_at, scale_at;               // where a wave's first token piece and its scales go
  uint32_t scale_block;                           // the block of the step that its scales are of
  f32x4 acc[MT][JT];

  // Row of the tile (of a pair: in the 128 of either matrix, the second's from
  // 128 on) where the interleaved tiles that row tile m is one of start
  static __device__ __forceinline__ int group_of(int wr, int m) {
    if constexpr (PAIR) return (m < HT ? 0 : 128) + (wr * HT + m % HT / Q * Q) * 16;
    return (wr * MT + m / Q * Q) * 16;
  }
  // Row of the product's row l16 of row tile m; D's register i, lane group g: row
  // group_of + g * 4Q + m % Q * 4 + i
  static __device__ __forceinline__ int row_of(int wr, int m, int l16) {
    return group_of(wr, m) + (l16 >> 2) * (4 * Q) + m % Q * 4 + (l16 & 3);
  }
  // What a row's chunks are permuted by (XOR): different for the 16 rows of a
  // product, but for pairs of neighbours, which lie in different halves of the banks
  static __device__ __forceinline__ int mix(int r) { return ((r >> 1) & 1) | (r / (4 * Q) & 3) << 1; }
  static __device__ __forceinline__ int token_mix(int r) { return (r >> 1) & 7; }

  // The wave's pieces, of 8 rows of a block each: the step's blocks one after another
  static __device__ __forceinline__ int weight_piece(int i, int wave) { return wave * WL + i; }
  static __device__ __forceinline__ int token_piece(int i, int wave) { return U * TT < 64 ? wave % (U * TT / 8) : i * 8 + wave; }

  // `first`, `second`: a pair's matrices from the tile's first row on, of which
  // there are `rows` (those past them are out of range); else the first alone.
  __device__ __forceinline__ void weights(const uint8_t* first, const uint8_t* second, int rows, int K, int wave, int lane) {
    const bool other = PAIR && wave >= 4;
    rw = make_rsrc(other ? second : first, (uint32_t)rows * (uint32_t)K);
#pragma unroll
    for (int i = 0; i < WL; ++i) {
      const int q = weight_piece(i, wave), r = q % (ROWS / 8) * 8 + (lane >> 3), c = (lane & 7) ^ mix(r);
      w_off[i] = (uint32_t)(PAIR ? r & 127 : r) * (uint32_t)K + (uint32_t)(q / (ROWS / 8) * kBlock + c * 16);
    }
  }
  // A pair's token row r: f(r) is its offset
  template <class F>
  __device__ __forceinline__ void gathered_tokens(int wave, int lane, F&& f) {
#pragma unroll
    for (int i = 0; i < XL; ++i) {
      const int q = token_piece(i, wave), r = q % (TT / 8) * 8 + (lane >> 3), c = (lane & 7) ^ token_mix(r);
      x_off[i] = f(r) + (uint32_t)(c * 16);
    }
    token_at = token_piece(0, wave) * 1024u;
  }
  // Else rows of K bytes, from the start of rx on, which ends behind the last
  __device__ __forceinline__ void tokens(int K, int wave, int lane) {
    const int q = token_piece(0, wave), r = q % (TT / 8) * 8 + (lane >> 3), c = (lane & 7) ^ token_mix(r);
    x_off[0] = (uint32_t)r * (uint32_t)K + (uint32_t)(q / (TT / 8) * kBlock + c * 16);
    x_row = U > 1 ? kBlock : 64u * (uint32_t)K;              // (U > 1: a wave's pieces are of the same rows)
    static_assert(U == 1 || XL == 1 || (U == 2 && TT == 64), "");
    token_at = q * 1024u;
  }

  // A wave's 64 scales of a step: of tokens, at `first` + step * stride bytes, f(r)
  // the offset of row r's; else one of the weights', of the first matrix or rows,
  // or of the second.
  template <class F>
  __device__ __forceinline__ void token_scales(const float* first, uint32_t bytes, size_t stride, int wave, int lane, F&& f) {
    const int id = wave % (U * kScaleGroups), group = id % kScaleGroups;
    scale_block = (uint32_t)(id / kScaleGroups);
    scale_at = kWeightBytes + id * 256u;
    s_off = 0;
    if (group < kScaleGroups - 2) {
      s_from = first, s_bytes = bytes, s_stride = stride;
      s_off = f(min(group * 64 + lane, TT - 1));
    }
  }
  __device__ __forceinline__ void weight_scales(const float* first, const float* second, int kb, int wave) {
    const int group = wave % (U * kScaleGroups) % kScaleGroups;
    s_blocks = (uint32_t)kb;
    if (group >= kScaleGroups - 2)
      s_from = group == kScaleGroups - 2 ? first : second, s_bytes = (uint32_t)kb * 4u, s_stride = 4;
  }

  __device__ __forceinline__ void issue(const Stage& stage, int wave, uint32_t step) {
    // (kNoStep added to a missing row's kOutside would be an offset in range again)
    const __amdgpu_buffer_rsrc_t tokens = PAIR && step >= kNoStep ? make_rsrc(nullptr, 0) : rx;
#pragma unroll
    for (int i = 0; i < XL; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(tokens, stage.x + token_at + i * 8192, 16,
                                               (PAIR ? x_off[PAIR ? i : 0] : x_off[0] + (uint32_t)i * x_row) + step * kStep, 0, 0, 0);
    fence();
#pragma unroll
    for (int i = 0; i < WL; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, stage.w + weight_piece(i, wave) * 1024, 16, w_off[i] + step * kStep, 0, 0, 0);
    // (U > 1: a row's last step may have no second block)
    const uint32_t block = step * U + scale_block;
    const bool none = U > 1 ? block >= s_blocks : step >= kNoStep;
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(reinterpret_cast<const uint8_t*>(s_from) + (none ? 0 : block * s_stride), s_bytes);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, stage.w + scale_at, 4, none ? kOutside : s_off, 0, 0, 0);
    fence();
  }

  // What follows a row's last value, `rest` from the step's first, is not its:
  // zero, in the pieces that this wave loaded
  __device__ __forceinline__ void clear_tail(const Stage& stage, int wave, int lane, int rest) {
    auto clear = [&](uint8_t* piece, int block, int by) {
      if (((lane & 7) ^ by) * 16 >= rest - block * kBlock) *reinterpret_cast<uint4*>(piece + lane * 16) = make_uint4(0, 0, 0, 0);
    };
#pragma unroll
    for (int i = 0; i < WL; ++i) {
      const int q = weight_piece(i, wave);
      clear(stage.w + q * 1024, q / (ROWS / 8), mix(q % (ROWS / 8) * 8 + (lane >> 3)));
    }
#pragma unroll
    for (int i = 0; i < XL; ++i) {
      const int q = token_piece(i, wave);
      clear(stage.x + token_at + i * 8192, q / (TT / 8), token_mix(q % (TT / 8) * 8 + (lane >> 3)));
    }
  }

  static __device__ __forceinline__ i32x8 read(const uint8_t* rows, int r, int x, int g) {
    const uint8_t* const row = rows + r * kBlock;
    return fragment(*reinterpret_cast<const i32x4*>(row + ((g ^ x) << 4)),
                    *reinterpret_cast<const i32x4*>(row + (((g + 4) ^ x) << 4)));
  }

  // A wave's token tile j, of the tile's 16-token tiles: two runs of kHalf, the
  // second from the tile's middle on, so that in a tile that is not full some waves
  // of each SIMD make half the products (T = 4096 2048x512 of 512 experts: down 161
  // us, 174 with one run each; not for 256 tokens, whose products in both forms leave
  // too few registers: 8192 tokens of the same 617 us, 602 with one run).
  static constexpr int kHalf = TT <= 128 && JT > 1 ? JT / 2 : JT;
  static __device__ __forceinline__ int token_tile(int wt, int j) { return j / kHalf * (kHalf * WT) + wt * kHalf + j % kHalf; }
  // Of a wave's, those up to the end of the last run with any of `toks` tokens
  static __device__ __forceinline__ int tiles_of(int wt, int toks) {
    const int at = wt * kHalf * 16;
    return kHalf < JT && toks > at + kHalf * WT * 16 ? JT : toks > at ? kHalf : 0;
  }

  // The products of block u of a step and the wave's first J token tiles
  template <int J>
  __device__ __forceinline__ void products(const Stage& stage, int u, int wr, int wt, int lane) {
    const int l16 = lane & 15, g = lane >> 4;
    const uint8_t* const weights = stage.w + u * (ROWS * kBlock);
    const uint8_t* const tokens = stage.x + u * (TT * kBlock);
    const float* const scales = reinterpret_cast<const float*>(stage.w + kWeightBytes + u * kScaleGroups * 256);
    const float* const sw = scales + (kScaleGroups - 2) * 64;
    const float s0 = PAIR || wr * MT < 8 ? sw[0] : sw[64], s1 = PAIR ? sw[64] : s0;
    i32x8 b[J], a[2];
    float s[2][J];
    const int by = (l16 >> 1 & 1) | (l16 >> 2) << 1;         // mix(row_of(...))
    a[0] = read(weights, row_of(wr, 0, l16), by, g);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int r = token_tile(wt, j) * 16 + l16;
      b[j] = read(tokens, r, token_mix(r), g);
      s[0][j] = scales[r];
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
      if constexpr (PAIR) s[1][j] = s[0][j] * s1;
      s[0][j] *= s0;
    }
    // (4096^3: 67.8 us with 3, 72.1 with 2, 75.4 with 1)
    constexpr int kDelay = 3, kAll = MT * J;
    Wide wide_a, wide_b[WIDE ? J : 1];
    if constexpr (WIDE) {
#pragma unroll
      for (int j = 0; j < J; ++j) wide_b[j] = widen(b[j]);
    }
    f32x4 d[kDelay + 1];
    for_each<kAll + kDelay>([&](auto n_c) MOE_INLINE {
      constexpr int n = decltype(n_c)::value, q = n - kDelay;
      if constexpr (n < kAll) {
        if constexpr (n % J == 0 && n / J + 1 < MT) a[(n / J + 1) % 2] = read(weights, row_of(wr, n / J + 1, l16), by, g);
        if constexpr (WIDE && n % J == 0) wide_a = widen(a[n / J % 2]);
        if constexpr (WIDE) d[n % (kDelay + 1)] = block_product(wide_a, wide_b[n % J]);
        else d[n % (kDelay + 1)] = block_product(a[n / J % 2], b[n % J]);
      }
      if constexpr (q >= 0) {
        const float scale = s[PAIR && q / J >= HT][q % J];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[q / J][q % J][i] = fmaf(d[q % (kDelay + 1)][i], scale, acc[q / J][q % J][i]);
        asm volatile("" : "+v"(acc[q / J][q % J]));         // here, and not where the sums are used next
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  }

  __device__ __forceinline__ void clear_sums() {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < JT; ++j) acc[m][j] = f32x4{};
  }

  // `tiles` tiles of `steps` steps each, from step `first` of the reduction on,
  // as one stream: while a tile's last steps are multiplied the next one's first
  // are on their way.  begin(i) sets the loads to tile i (0 is set before);
  // end(i) finishes tile i's sums; live(i): this wave's tiles_of its tokens (ALL: not
  // asked).  ONE: one tile only; else end(i) stores STORES times, whatever the tile,
  // and the next step need not wait for that.
  template <bool ALL, bool ONE, int STORES, class At, class Begin, class End, class Live>
  __device__ __forceinline__ void run(At&& stage_at, int wave, int wr, int wt, int lane, int first, int steps, int tiles, int K,
                                      Begin&& begin, End&& end, Live&& live) {
    int in = 0, tile_in = 0;                                 // the next loads' step and tile
    // past the last tile they are issued out of range: they read nothing
    auto load = [&](const Stage& stage) MOE_INLINE {
      issue(stage, wave, tile_in < tiles ? (uint32_t)(first + in) : kNoStep);
      ++in;
      if (ONE) {
        if (in == steps) tile_in = 1;
      } else if (in == steps) {
        in = 0;
        if (++tile_in < tiles) begin(tile_in);
      }
    };
    for_each<kLead>([&](auto s) MOE_INLINE { load(stage_at(s)); });
    clear_sums();
    int out = 0, tile_out = 0;
    int here = ALL ? JT : live(0);
    auto body = [&](auto stage_c) MOE_INLINE {
      constexpr int S = decltype(stage_c)::value;
      const Stage stage = stage_at(stage_c);
      // this wave's loads of the step have landed (loads and stores end in order)
      if (!ONE && out == 0 && tile_out > 0) wait_loads<(kLead - 1) * kLoads + STORES>();
      else wait_loads<(kLead - 1) * kLoads>();
      const int rest = K - (first + out) * (int)kStep;
      if (rest < (int)kStep) clear_tail(stage, wave, lane, rest);
      wait_lds();                                            // and its reads of the step before returned
      barrier();
      // (before the products: spread between them, 4096^3 takes 66.5 us and not 65.0)
      load(stage_at(std::integral_constant<int, (S + kLead) % NS>{}));
      for_each<ALL || kHalf == JT ? 1 : 2>([&](auto half) MOE_INLINE {
        constexpr int J = decltype(half)::value ? kHalf : JT;
        if (!ALL && (here == 0 || (kHalf < JT && (here <= kHalf) != (J < JT)))) return;
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (u == 0 || rest > u * kBlock) products<J>(stage, u, wr, wt, lane);
      });
      ++out;
      if (!ONE && out == steps) {
        out = 0;
        end(tile_out);
        if (++tile_out < tiles) {
          clear_sums();
          if constexpr (!ALL) here = live(tile_out);
        }
      }
    };
    int left = tiles * steps;
    for (; left >= NS; left -= NS) for_each<NS>([&](auto i) MOE_INLINE { body(i); });
    for_each<NS - 1>([&](auto i) MOE_INLINE {
      if (decltype(i)::value < left) body(i);
    });
    wait_loads<0>();                                         // the loads past the last step have landed
    if (ONE) end(0);
  }
};

// The stages' memory, one array each, so that reads of one are seen not to
// alias the loads in flight to the others; and stage_at of Tile::run
#define MOE_TILE_STAGES(TILE)                                                          \
  __shared__ __align__(16) uint8_t s_w0[TILE::kScaledBytes];                           \
  __shared__ __align__(16) uint8_t s_w1[TILE::kScaledBytes];                           \
  __shared__ __align__(16) uint8_t s_w2[TILE::NS > 2 ? TILE::kScaledBytes : 16];       \
  __shared__ __align__(16) uint8_t s_w3[TILE::NS > 3 ? TILE::kScaledBytes : 16];       \
  __shared__ __align__(16) uint8_t s_x0[TILE::kTokenBytes];                            \
  __shared__ __align__(16) uint8_t s_x1[TILE::kTokenBytes];                            \
  __shared__ __align__(16) uint8_t s_x2[TILE::NS > 2 ? TILE::kTokenBytes : 16];        \
  __shared__ __align__(16) uint8_t s_x3[TILE::NS > 3 ? TILE::kTokenBytes : 16];        \
  auto stage_at = [&](auto i) -> Stage {                                               \
    constexpr int I = decltype(i)::value;                                              \
    if constexpr (I == 0) return {s_w0, s_x0};                                         \
    else if constexpr (I == 1) return {s_w1, s_x1};                                    \
    else if constexpr (I == 2) return {s_w2, s_x2};                                    \
    else return {s_w3, s_x3};                                                          \
  };

}  // namespace
}  // namespace moe
