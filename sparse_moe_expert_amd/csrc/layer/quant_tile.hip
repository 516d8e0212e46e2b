// 4-bit products of many tokens: bound by the matrix cores.
//
// A workgroup of four waves owns 128 tokens and 256 weight rows (128 rows of
// both matrices of a gate/up pair); a wave owns 64 of the rows (32 of each
// matrix) and all of the tokens, so that every weight is decoded once a
// workgroup and every token fragment read from LDS feeds two products.
// v_mfma_f32_32x32x16_bf16, weights as A: lane l holds row l%32, reduction
// indices 8*(l/32)..+8; tokens as B: column l%32, the same indices; D
// register r is row 8*(r/4) + 4*(l/32) + r%4, column l%32.  The reduction
// index is permuted alike in both: in a step of 64 the lane half h covers
// 32h .. 32h+32, so that a lane's codes of a step are one 16-byte load.
//
// What it waits for is L1: every compute unit fetches a 128-byte line for each
// row's codes and scales of a step, and with two workgroups there those are
// out again before the next step asks for the rest of the line.  So a row's
// codes of two steps are loaded together, and its scales of four: 4096^3
// (NVFP4) 140 us loaded step by step, 128 with both by twos, 121 so (118 to 127
// from card to card, MXFP4 112 to 119); more do not fit the registers.  A bf16
// library product of the size takes 106 us (of which 35 us power: it takes 67 us
// on zeros).
//
// Tokens go straight to a ring of four LDS stages (16-byte chunk c of token
// row r at c ^ ((r >> 1) & 7): the reads of 16 lanes hit all banks), codes and
// scales to rings of registers, issued two steps ahead.  With two stages
// more than steps in flight one barrier a step is enough: the stage that step
// s fills was read in step s-2, and a wave passes step s-1's barrier only when
// every wave's reads of s-2 have returned.
//
// Workgroups are dealt round robin to the 8 XCDs; each XCD takes consecutive
// tiles, the row tiles of one token tile after another, so that its L2 holds
// the tokens that its workgroups share.
#include "quant_common.h"

#include <type_traits>

namespace moe {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kTileThreads = 256;
constexpr int kTileTokens = 128;
constexpr int kTileK = 64;
constexpr int kStages = 4, kLead = 2;
constexpr int kStageBytes = kTileTokens * kTileK * 2;        // 16 KB
constexpr int kXcds = 8;

// A row's scales of four steps are loaded at once, from the dword they start
// in.  WIDE: they always start at a multiple of four bytes; else they are
// shifted into place (2048x4096x2592: 52.1 us, 56.7 loaded step by step; 2560:
// 48.3).
template <int FMT, bool GU, bool WIDE>
struct RowTile {
  static constexpr int kCodeLoads = 4, kTokenLoads = 4;      // of two steps, of one
  __amdgpu_buffer_rsrc_t rc[GU ? 2 : 1], rs[GU ? 2 : 1], rx;
  uint32_t c_off[2], s_off[2], x_off[4];
  uint32_t shift[2];                                         // bytes into the first dword
  uint4 wc[kStages][2];
  uint4 wide[2][2];                                          // scales of this ring, of the next

  // Codes of the steps a and b = a + 1, of stages S and S + 1: their lines are
  // fetched once for both
  template <int S>
  __device__ __forceinline__ void issue_weights(uint32_t a, uint32_t b) {
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const int r = GU ? m : 0;
      wc[S][m] = to_uint4(__builtin_amdgcn_raw_buffer_load_b128(rc[r], c_off[m] + a * 32u, 0, 0));
      wc[S + 1][m] = to_uint4(__builtin_amdgcn_raw_buffer_load_b128(rc[r], c_off[m] + b * 32u, 0, 0));
    }
  }
  // The scales of four steps (past the last one too: a shifted row ends in the
  // dword after them)
  template <int W>
  __device__ __forceinline__ void issue_scales(uint32_t step) {
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const int r = GU ? m : 0;
      if constexpr (FMT == MOE_QUANT_NVFP4) {
        wide[W][m] = to_uint4(__builtin_amdgcn_raw_buffer_load_b128(rs[r], s_off[m] + step * 4u, 0, 0));
      } else {
        const auto v = __builtin_amdgcn_raw_buffer_load_b64(rs[r], s_off[m] + step * 2u, 0, 0);
        wide[W][m].x = v[0], wide[W][m].y = v[1];
      }
    }
  }
  __device__ __forceinline__ void issue_tokens(uint8_t* stage, int wave, uint32_t step) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, stage + (i * 4 + wave) * 1024, 16, x_off[i] + step * 128u, 0, 0, 0);
  }

  // Row tile m, group i (8 weights) of the step in `stage`: codes and scale (of
  // the lane's half of the step)
  __device__ __forceinline__ uint32_t word(int stage, int m, int i) const {
    const uint4 c = wc[stage][m];
    return i == 0 ? c.x : i == 1 ? c.y : i == 2 ? c.z : c.w;
  }
  __device__ __forceinline__ float scale(int S, bool next, int m, int i, int half) const {
    constexpr bool kNv = FMT == MOE_QUANT_NVFP4;
    const uint4 w = wide[next][m];
    const uint32_t after = wide[1][m].x;                     // (next: stage 0 only, which needs none)
    const int at = kNv ? S : S / 2;                          // the step's dword
    uint32_t sb = at == 0 ? w.x : at == 1 ? w.y : at == 2 ? w.z : w.w;
    if constexpr (!WIDE)
      sb = __builtin_amdgcn_alignbyte(at == (kNv ? 3 : 1) ? after : at == 0 ? w.y : at == 1 ? w.z : w.w, sb, shift[m]);
    if constexpr (kNv) {
      sb >>= half * 16;
      return i < 2 ? __builtin_amdgcn_cvt_f32_fp8((int)sb, 0) : __builtin_amdgcn_cvt_f32_fp8((int)sb, 1);
    } else {
      return __uint_as_float((sb >> (S % 2 * 16 + half * 8) & 0xFFu) << 23);
    }
  }
};

template <int FMT, bool GU, bool WIDE>
__global__ __launch_bounds__(kTileThreads, 2) void quant_tile_kernel(DenseArgs p, int row_tiles, int tiles) {
  using Tile = RowTile<FMT, GU, WIDE>;
  constexpr int kRows = GU ? 128 : 256;
  // one array per stage, so that reads of one stage are seen not to alias the
  // loads in flight to the others
  __shared__ __align__(16) uint8_t s_0[kStageBytes];
  __shared__ __align__(16) uint8_t s_1[kStageBytes];
  __shared__ __align__(16) uint8_t s_2[kStageBytes];
  __shared__ __align__(16) uint8_t s_3[kStageBytes];
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int per = (tiles + kXcds - 1) / kXcds;
  if (GU && (int)blockIdx.x >= per * kXcds) {                // token gates, one wave a token
    const int t = ((int)blockIdx.x - per * kXcds) * 4 + wave;
    if (t < p.T) token_gate_row(p, t, lane);
    return;
  }
  const int tile = (int)(blockIdx.x % kXcds) * per + (int)(blockIdx.x / kXcds);
  if (tile >= tiles) return;
  const int n0 = (tile % row_tiles) * kRows, t0 = (tile / row_tiles) * kTileTokens;
  const int l32 = lane & 31, half = lane >> 5;
  const int rows = min(kRows, p.N - n0), toks = min(kTileTokens, p.T - t0);

  const float ga = global_scale(p.a), gb = GU ? global_scale(p.b) : 1.0f;       // (early: not when they are needed)
  Tile tl;
  const uint32_t code_row = (uint32_t)p.K / 2, scale_row = (uint32_t)(p.K / kScaleGroup<FMT>);
#pragma unroll
  for (int m = 0; m < (GU ? 2 : 1); ++m) {
    const QuantMat& w = m ? p.b : p.a;
    tl.rc[m] = make_rsrc(w.codes + (size_t)n0 * code_row, (uint32_t)rows * code_row);
    tl.rs[m] = make_rsrc(w.scales + (size_t)n0 * scale_row, ((uint32_t)rows * scale_row + 3u) & ~3u);
  }
  tl.rx = make_rsrc(p.x + (size_t)t0 * p.K, (uint32_t)toks * (uint32_t)p.K * 2u);
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const uint32_t row = (uint32_t)((GU ? 0 : m * 128) + wave * 32 + l32);
    tl.c_off[m] = row * code_row + (uint32_t)half * 16u;
    tl.s_off[m] = row * scale_row & ~3u;
    tl.shift[m] = row * scale_row & 3u;
  }
  // piece i of a wave: 8 token rows of 128 bytes; rows past the last token repeat it
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = (i * 4 + wave) * 8 + (lane >> 3), c = (lane & 7) ^ ((row >> 1) & 7);
    tl.x_off[i] = (uint32_t)min(row, toks - 1) * (uint32_t)p.K * 2u + (uint32_t)c * 16u;
  }
  const int steps = (p.K + kTileK - 1) / kTileK;
  f32x16 acc[2][4];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[m][j] = f32x16{};

  // a step past the last one is issued out of range: it reads nothing
  auto at = [&](int s) { return s < steps ? (uint32_t)s : kOutside / 128u; };
  // The half of step s that a lane takes its scales of.  Where K ends with half a
  // step the second half's tokens are zero, but its scale bytes may lie behind
  // the matrix, and zero times a NaN would count: it takes the first half's.
  auto scale_half = [&](int s) { return WIDE || p.K - s * kTileK >= kTileK ? half : 0; };
  tl.template issue_scales<0>(0);
  tl.template issue_weights<0>(at(0), at(1));
  fence();
  tl.issue_tokens(s_0, wave, at(0));
  fence();
  tl.issue_tokens(s_1, wave, at(1));
  fence();
  bf16x8 af[2];                                              // the next products' weights
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const uint32_t c = tl.word(0, m, 0);
    const float s = tl.scale(0, false, m, 0, scale_half(0));
    af[m] = __builtin_bit_cast(bf16x8, make_uint4(fp4x2_scaled<FMT, 0>(c, s), fp4x2_scaled<FMT, 1>(c, s),
                                                  fp4x2_scaled<FMT, 2>(c, s), fp4x2_scaled<FMT, 3>(c, s)));
  }
  auto body = [&](auto stage_c, int s) {
    constexpr int S = decltype(stage_c)::value, F = (S + kLead) % kStages;
    constexpr int kScalesAt = WIDE ? 2 : 0;                  // shifted ones are needed a step earlier
    if constexpr (S % 2 == 0) {
      if constexpr (S == kScalesAt) tl.template issue_scales<1>((uint32_t)(s - S) + kStages);
      tl.template issue_weights<F>(at(s + kLead), at(s + kLead + 1));
      fence();
    }
    tl.issue_tokens(F == 0 ? s_0 : F == 1 ? s_1 : F == 2 ? s_2 : s_3, wave, at(s + kLead));
    // this wave's tokens of step s are here; since then two steps' tokens,
    // the codes of a pair of steps, and scales where they were issued
    wait_vm<kLead * Tile::kTokenLoads + Tile::kCodeLoads + (S / 2 == kScalesAt / 2 ? 2 : 0)>();
    uint8_t* const stage = S == 0 ? s_0 : S == 1 ? s_1 : S == 2 ? s_2 : s_3;
    if (p.K - s * kTileK < kTileK) {                         // half a step: what follows a token's row is not its
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = (i * 4 + wave) * 8 + (lane >> 3);
        if (((lane & 7) ^ ((row >> 1) & 7)) >= 4)
          *reinterpret_cast<uint4*>(stage + (i * 4 + wave) * 1024 + lane * 16) = make_uint4(0, 0, 0, 0);
      }
    }
    wait_lds();                                              // and its reads of step s-1 have returned
    barrier();
    __builtin_amdgcn_sched_barrier(0);
    const int half_here = scale_half(s), half_next = scale_half(s + 1);
    // Four groups of eight products, of all four token tiles also where the
    // last ones are past T (branches around them would keep the products of a
    // tile apart).  Under a group's products the next group's weights are
    // decoded and its tokens read.
    bf16x8 b[2][4];
    auto read = [&](int i, int j) {
      const int row = j * 32 + l32;
      b[i & 1][j] = *reinterpret_cast<const bf16x8*>(stage + row * 128 + (((half * 4 + i) ^ ((row >> 1) & 7)) << 4));
    };
#pragma unroll
    for (int j = 0; j < 4; ++j) read(0, j);
    for_each<4>([&](auto i_c) {
      constexpr int i = decltype(i_c)::value;
      uint32_t next[2][4];
      for_each<8>([&](auto n_c) {
        constexpr int n = decltype(n_c)::value, j = n / 2, m = n % 2, D = n % 4, W = n / 4;
        if constexpr (i < 3 && m == 0) read(i + 1, j);
        acc[m][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(af[m], b[i & 1][j], acc[m][j], 0, 0, 0);
        const float sc = tl.scale(i < 3 ? S : (S + 1) % kStages, i == 3 && S == 3, W, (i + 1) % 4, i < 3 ? half_here : half_next);
        next[W][D] = fp4x2_scaled<FMT, D>(tl.word(i < 3 ? S : (S + 1) % kStages, W, (i + 1) % 4), sc);
        asm volatile("" : "+v"(next[W][D]));
        __builtin_amdgcn_sched_barrier(0);
      });
#pragma unroll
      for (int m = 0; m < 2; ++m) af[m] = __builtin_bit_cast(bf16x8, make_uint4(next[m][0], next[m][1], next[m][2], next[m][3]));
    });
  };
  int s0 = 0;
  for (; s0 + kStages <= steps; s0 += kStages) {
    body(std::integral_constant<int, 0>{}, s0);
    body(std::integral_constant<int, 1>{}, s0 + 1);
    body(std::integral_constant<int, 2>{}, s0 + 2);
    body(std::integral_constant<int, 3>{}, s0 + 3);
#pragma unroll
    for (int m = 0; m < 2; ++m) tl.wide[0][m] = tl.wide[1][m];
  }
  if (s0 < steps) body(std::integral_constant<int, 0>{}, s0);
  if (s0 + 1 < steps) body(std::integral_constant<int, 1>{}, s0 + 1);
  if (s0 + 2 < steps) body(std::integral_constant<int, 2>{}, s0 + 2);
  wait_vm<0>();                                              // the loads past the last step have landed

  // Sums to LDS as fp32, then whole 16-byte pieces of output rows.  One array
  // takes 32 tokens x 128 rows, chunk c of four rows of token t at c ^ (t & 15).
  constexpr int kRound = GU ? 4 : 2;                         // token tiles a round
#pragma unroll
  for (int j0 = 0; j0 < 4; j0 += kRound) {
    if (j0 * 32 >= toks) break;
    __syncthreads();
#pragma unroll
    for (int jj = 0; jj < kRound; ++jj) {
      const int j = j0 + jj;
#pragma unroll
      for (int m = 0; m < (GU ? 1 : 2); ++m) {
        const int a = GU ? jj : jj * 2 + m;
        uint8_t* const out = (a == 0 ? s_0 : a == 1 ? s_1 : a == 2 ? s_2 : s_3) + l32 * 512;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          f32x4 v;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[i] = acc[m][j][r * 4 + i];
            if constexpr (GU) {
              v[i] = silu(v[i] * ga) * (acc[1][j][r * 4 + i] * gb);
            }
          }
          const int c = wave * 8 + r * 2 + half;
          *reinterpret_cast<f32x4*>(out + ((c ^ (l32 & 15)) << 4)) = v;
        }
      }
    }
    __syncthreads();
    auto array = [&](int tok, int row) -> const uint8_t* {
      const int a = GU ? tok >> 5 : (tok >> 5) * 2 + (row >> 7);
      return (a == 0 ? s_0 : a == 1 ? s_1 : a == 2 ? s_2 : s_3) + (tok & 31) * 512;
    };
    const int here = min(toks - j0 * 32, kRound * 32);
    if (!GU && p.N % 8 != 0) {
      // Output rows that do not start at 16 bytes (never a pair's): pieces of eight that do,
      // which begin up to seven rows before the tile, the outer ones one by
      // one.  2048x4095x4096: 79.5 us, 92 with all outputs one by one (N = 4096: 71);
      // with a bias, read one by one, 88 (69).
      constexpr int kPieces = kRows / 8 + 1;
      for (int i = tid; i < here * kPieces; i += kTileThreads) {
        const int tok = i / kPieces, t = t0 + j0 * 32 + tok;
        const size_t at = (size_t)t * p.N + n0;
        const int r0 = i % kPieces * 8 - (int)(at & 7);
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int row = min(max(r0 + k, 0), kRows - 1);
          v[k] = *reinterpret_cast<const float*>(array(tok, row) + ((((row & 127) >> 2) ^ (tok & 15)) << 4) + (row & 3) * 4);
        }
        const float gate = p.gate ? p.gate[t] : 1.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int row = min(max(r0 + k, 0), rows - 1);
          if (p.bias) v[k] = v[k] * ga + bf16_to_f32(p.bias[n0 + row]);
          else v[k] *= ga;
          v[k] *= gate;
          if (p.add) v[k] += bf16_to_f32(p.add[at + row]);
        }
        uint32_t o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = f32_to_bf16_rne(v[k]);
        if (r0 >= 0 && r0 + 8 <= rows) {
          *reinterpret_cast<uint4*>(p.y + at + r0) =
              make_uint4(o[0] | o[1] << 16, o[2] | o[3] << 16, o[4] | o[5] << 16, o[6] | o[7] << 16);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (r0 + k >= 0 && r0 + k < rows) p.y[at + r0 + k] = (uint16_t)o[k];
        }
      }
      continue;
    }
    const int pieces = here * (kRows / 8);
    for (int i = tid; i < pieces; i += kTileThreads) {
      const int tok = i / (kRows / 8), piece = i % (kRows / 8);        // a token's eight rows
      const int n = n0 + piece * 8, t = t0 + j0 * 32 + tok;
      if (n >= p.N) continue;
      const int c = (piece & 15) * 2;
      const uint8_t* const in = array(tok, piece * 8);
      const f32x4 lo = *reinterpret_cast<const f32x4*>(in + ((c ^ (tok & 15)) << 4));
      const f32x4 hi = *reinterpret_cast<const f32x4*>(in + (((c + 1) ^ (tok & 15)) << 4));
      write8<GU>(p, t, n, lo, hi, ga);
    }
  }
}

template <int FMT, bool GU, bool WIDE>
moe_status launch(const DenseArgs& p, hipStream_t s) {
  constexpr int kRows = GU ? 128 : 256;
  const int row_tiles = (p.N + kRows - 1) / kRows;
  const int tiles = row_tiles * ((p.T + kTileTokens - 1) / kTileTokens);      // at most 2^26 (N and T up to 2^20)
  const int grid = (tiles + kXcds - 1) / kXcds * kXcds + (GU && p.token_gate ? (p.T + 3) / 4 : 0);
  quant_tile_kernel<FMT, GU, WIDE><<<(unsigned)grid, kTileThreads, 0, s>>>(p, row_tiles, tiles);
  return launch_status();
}

}  // namespace

// Fewer tiles than this leave too many compute units idle, and the split
// kernel's smaller ones take less.  4096x4096, 128 tiles: 61.4 us and 47.2
// split; 160 tiles: 61.7 and 65.1; 240 tiles: 66.3 and 87.1.
constexpr long long kEnoughTiles = 160;

bool quant_tile_ok(bool gate_up, int T, int N) {
  const int rows = gate_up ? 128 : 256;
  return T > 64 && (long long)((N + rows - 1) / rows) * ((T + kTileTokens - 1) / kTileTokens) >= kEnoughTiles;
}

moe_status quant_tile(int format, bool gate_up, const DenseArgs& p, hipStream_t s) {
  if (format == MOE_QUANT_NVFP4) {
    if (p.K % 64 == 0) return gate_up ? launch<MOE_QUANT_NVFP4, true, true>(p, s) : launch<MOE_QUANT_NVFP4, false, true>(p, s);
    return gate_up ? launch<MOE_QUANT_NVFP4, true, false>(p, s) : launch<MOE_QUANT_NVFP4, false, false>(p, s);
  }
  if (p.K % 128 == 0) return gate_up ? launch<MOE_QUANT_MXFP4, true, true>(p, s) : launch<MOE_QUANT_MXFP4, false, true>(p, s);
  return gate_up ? launch<MOE_QUANT_MXFP4, true, false>(p, s) : launch<MOE_QUANT_MXFP4, false, false>(p, s);
}

}  // namespace moe
