// The products of a tile: 256 weight rows (of a gate/up pair 128 of each) by TT
// tokens, by a workgroup of eight waves.
//
// Tokens, weights and scales go straight to LDS (buffer_load ... lds), a block
// of 128 of the reduction a step, in a ring of NS stages.  A row's step is 128
// bytes, chunk c of 16 at c ^ ((r >> 1) & 7): the reads of 16 lanes, one chunk of
// 16 rows, hit all banks.  The waves stand WR x WT over the tile; a wave holds
// the step's fragments of its JT token tiles and goes through its MT row tiles,
// each product followed, three products later, by the four multiply-adds that
// scale it onto the sums: the matrix pipe and the vector pipe then work side by
// side.
#pragma once

#include "block_common.h"

#include <type_traits>

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

template <int TT, bool PAIR>
struct Tile {
  static constexpr int WR = TT == 256 ? 2 : TT == 16 ? 8 : 4, WT = 8 / WR;
  static constexpr int MT = kTileRows / WR / 16, JT = TT / WT / 16;        // row tiles, token tiles a wave
  static constexpr int kWeightBytes = kTileRows * kBlock, kTokenBytes = TT * kBlock;
  static constexpr int kScaleGroups = (TT + 63) / 64 + 2;                  // 64 of the tokens' scales each, and the weights'
  static constexpr int kStageBytes = kWeightBytes + kTokenBytes + kScaleGroups * 256;
  static constexpr int kFit = 160 * 1024 / kStageBytes, NS = kFit < 4 ? kFit : 4, kLead = NS - 1;
  static constexpr int XL = TT < 64 ? 1 : TT / 64;                         // a wave's token loads a step
  static constexpr int kLoads = 4 + XL + 1;
  static_assert(NS >= 2 && (kLead - 1) * kLoads < 64, "two stages or more");

  __amdgpu_buffer_rsrc_t rw, rx, rs;         // the wave's weight rows, the tokens, the wave's scales
  uint32_t w_off[4], x_off[XL], s_off;
  uint32_t token_at, scale_at;               // where a wave's first token piece and its scales go in a stage
  f32x4 acc[MT][JT];

  // Row of the tile where a wave's row tile m starts (of a pair: in the 128 of
  // either matrix, the second's from 128 on)
  static __device__ __forceinline__ int row_of(int wr, int m) {
    if constexpr (PAIR) return (m < MT / 2 ? 0 : 128) + wr * (MT / 2 * 16) + m % (MT / 2) * 16;
    return (wr * MT + m) * 16;
  }

  // The wave's loads.  Weight piece i: 8 rows from (wave * 4 + i) * 8 on.
  // `first`, `second`: a pair's matrices from the tile's first row on, of which
  // there are `rows` (those past them repeat the last); else the first alone.
  __device__ __forceinline__ void weights(const uint8_t* first, const uint8_t* second, int rows, int K, int wave, int lane) {
    const bool other = PAIR && wave >= 4;
    rw = make_rsrc(other ? second : first, (uint32_t)rows * (uint32_t)K);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = (wave * 4 + i) * 8 + (lane >> 3), c = (lane & 7) ^ ((r >> 1) & 7);
      const int in = PAIR ? r & 127 : r;
      w_off[i] = (uint32_t)min(in, rows - 1) * (uint32_t)K + (uint32_t)c * 16u;
    }
  }
  // Token row r's place in the tile's token loads: f(r) is its offset
  template <class F>
  __device__ __forceinline__ void tokens(int wave, int lane, F&& f) {
#pragma unroll
    for (int i = 0; i < XL; ++i) {
      const int piece = TT < 64 ? wave % (TT / 8) : i * 8 + wave;          // 8 rows each
      const int r = piece * 8 + (lane >> 3), c = (lane & 7) ^ ((r >> 1) & 7);
      x_off[i] = f(r) + (uint32_t)c * 16u;
    }
    token_at = kWeightBytes + (TT < 64 ? wave % (TT / 8) : wave) * 1024u;
  }

  // A wave's 64 scales: of tokens, f(r) the offset of row r's in sx; else one of
  // the weights', of the first matrix or rows, or of the second
  template <class F>
  __device__ __forceinline__ void scales(const float* sx, uint32_t bytes, const float* first, const float* second, int kb,
                                         int wave, int lane, F&& f) {
    const int group = wave % kScaleGroups;
    scale_at = kWeightBytes + kTokenBytes + group * 256u;
    if (group < kScaleGroups - 2) {
      rs = make_rsrc(sx, bytes);
      s_off = f(min(group * 64 + lane, TT - 1));
    } else {
      rs = make_rsrc(group == kScaleGroups - 2 ? first : second, (uint32_t)kb * 4u);
      s_off = 0;
    }
  }

  __device__ __forceinline__ void issue(uint8_t* stage, int wave, uint32_t step) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, stage + (wave * 4 + i) * 1024, 16, w_off[i] + step * kBlock, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < XL; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, stage + token_at + i * 8192, 16, x_off[i] + step * kBlock, 0, 0, 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, stage + scale_at, 4, s_off + step * 4u, 0, 0, 0);
  }

  // What follows a row's last value in its last step is not its: zero, in the
  // pieces that this wave loaded (chunks from `from` on)
  __device__ __forceinline__ void clear_tail(uint8_t* stage, int wave, int lane, int from) {
    auto clear = [&](uint32_t at, int r) {
      if (((lane & 7) ^ ((r >> 1) & 7)) >= from) *reinterpret_cast<uint4*>(stage + at + lane * 16) = make_uint4(0, 0, 0, 0);
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) clear((wave * 4 + i) * 1024, (wave * 4 + i) * 8 + (lane >> 3));
#pragma unroll
    for (int i = 0; i < XL; ++i) clear(token_at + i * 8192, (TT < 64 ? wave % (TT / 8) : i * 8 + wave) * 8 + (lane >> 3));
  }

  static __device__ __forceinline__ i32x8 read(const uint8_t* rows, int r, int g) {
    const uint8_t* const row = rows + r * kBlock;
    const int x = (r >> 1) & 7;
    return fragment(*reinterpret_cast<const i32x4*>(row + ((g ^ x) << 4)),
                    *reinterpret_cast<const i32x4*>(row + (((g + 4) ^ x) << 4)));
  }

  // One step's products of the first JL token tiles
  template <int JL>
  __device__ __forceinline__ void products(const uint8_t* stage, int wr, int wt, int lane) {
    const int l16 = lane & 15, g = lane >> 4;
    const float* const scales = reinterpret_cast<const float*>(stage + kWeightBytes + kTokenBytes);
    const float* const sw = scales + (kScaleGroups - 2) * 64;
    const float s0 = PAIR || wr * MT < 8 ? sw[0] : sw[64], s1 = PAIR ? sw[64] : s0;
    i32x8 b[JL], a[2];
    float s[2][JL];
    a[0] = read(stage, row_of(wr, 0) + l16, g);
#pragma unroll
    for (int j = 0; j < JL; ++j) {
      const int r = (wt * JT + j) * 16 + l16;
      b[j] = read(stage + kWeightBytes, r, g);
      s[0][j] = scales[r];
    }
#pragma unroll
    for (int j = 0; j < JL; ++j) {
      if constexpr (PAIR) s[1][j] = s[0][j] * s1;
      s[0][j] *= s0;
    }
    constexpr int kDelay = 3, kAll = MT * JL;
    f32x4 d[kDelay + 1];
    for_each<kAll + kDelay>([&](auto n_c) {
      constexpr int n = decltype(n_c)::value, q = n - kDelay;
      if constexpr (n < kAll) {
        if constexpr (n % JL == 0 && n / JL + 1 < MT) a[(n / JL + 1) % 2] = read(stage, row_of(wr, n / JL + 1) + l16, g);
        d[n % (kDelay + 1)] = block_product(a[n / JL % 2], b[n % JL]);
      }
      if constexpr (q >= 0) {
        const float scale = s[PAIR && q / JL >= MT / 2][q % JL];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[q / JL][q % JL][i] = fmaf(d[q % (kDelay + 1)][i], scale, acc[q / JL][q % JL][i]);
        asm volatile("" : "+v"(acc[q / JL][q % JL]));         // here, and not where the sums are used next
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  }
  // Of those below `live`, or of all
  template <bool ALL>
  __device__ __forceinline__ void step(const uint8_t* stage, int wr, int wt, int lane, int live) {
    if constexpr (ALL) {
      products<JT>(stage, wr, wt, lane);
    } else {
      for_each<JT>([&](auto j) {
        constexpr int JL = decltype(j)::value + 1;
        if (live == JL || (JL == JT && live > JT)) products<JL>(stage, wr, wt, lane);
      });
    }
  }

  // All steps first .. first + steps; stages: NS arrays, so that reads of one
  // are seen not to alias the loads in flight to the others
  template <bool ALL, class Stage>
  __device__ __forceinline__ void run(Stage&& stage_at, int wave, int wr, int wt, int lane, int first, int steps, int K, int live) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < JT; ++j) acc[m][j] = f32x4{};
    // a step past the last is issued out of range: it reads nothing
    auto at = [&](int s) { return s < steps ? (uint32_t)(first + s) : kOutside / kBlock; };
    for_each<kLead>([&](auto s) {
      issue(stage_at(s), wave, at(decltype(s)::value));
      fence();
    });
    auto body = [&](auto stage_c, int s) {
      constexpr int S = decltype(stage_c)::value;
      uint8_t* const stage = stage_at(stage_c);
      wait_loads<(kLead - 1) * kLoads>();                    // this wave's loads of step s have landed
      const int rest = K - (first + s) * kBlock;
      if (rest < kBlock) clear_tail(stage, wave, lane, rest / 16);
      wait_lds();                                            // and its reads of step s-1 returned
      barrier();
      issue(stage_at(std::integral_constant<int, (S + kLead) % NS>{}), wave, at(s + kLead));
      fence();
      step<ALL>(stage, wr, wt, lane, live);
    };
    int s0 = 0;
    for (; s0 + NS <= steps; s0 += NS)
      for_each<NS>([&](auto i) { body(i, s0 + decltype(i)::value); });
    for_each<NS - 1>([&](auto i) {
      if (s0 + decltype(i)::value < steps) body(i, s0 + decltype(i)::value);
    });
    wait_loads<0>();                                         // the loads past the last step have landed
  }
};

// The stages' memory, and stage_at of Tile::run
#define MOE_TILE_STAGES(TILE)                                                          \
  __shared__ __align__(16) uint8_t s_0[TILE::kStageBytes];                             \
  __shared__ __align__(16) uint8_t s_1[TILE::kStageBytes];                             \
  __shared__ __align__(16) uint8_t s_2[TILE::NS > 2 ? TILE::kStageBytes : 16];         \
  __shared__ __align__(16) uint8_t s_3[TILE::NS > 3 ? TILE::kStageBytes : 16];         \
  auto stage_at = [&](auto i) -> uint8_t* {                                            \
    constexpr int I = decltype(i)::value;                                              \
    if constexpr (I == 0) return s_0;                                                  \
    else if constexpr (I == 1) return s_1;                                             \
    else if constexpr (I == 2) return s_2;                                             \
    else return s_3;                                                                   \
  };

}  // namespace
}  // namespace moe
