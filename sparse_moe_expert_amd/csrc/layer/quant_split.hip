// 4-bit products of batches whose tiles are too few for the chip: 64 or 128
// weight rows by 16, 32 or 64 tokens, the reduction split over workgroups
// where the tiles alone do not fill it.
//
// Tokens, codes and scales all go straight to LDS (buffer_load ... lds), steps
// of 256 or 512 of the reduction, in a ring of as many stages as LDS holds: a
// row's code bytes of a step are whole cache lines, each taken by 8 lanes of
// one load.  (Loaded to registers, in the layout of the matrix tiles, each load
// touches 16 bytes of 64 rows' lines, and the scales 2 bytes of them: the
// lines that a compute unit's L1 then fetches again and again were 4 times the
// bytes used, and set the time.)
//
// Eight waves: with RG = rows / 32, wave w takes 32 rows (w % RG) and the
// 8/RG-th part w / RG of each step, so that every weight is decoded once.  Of a
// gate/up pair the first half of the rows is the first matrix's.
// v_mfma_f32_32x32x16_bf16, weights as A: lane l holds row l%32, reduction
// indices 8*(l/32)..+8; tokens as B: column l%32, the same indices; D
// register r is row 8*(r/4) + 4*(l/32) + r%4, column l%32.  The reduction
// index is permuted alike in both: the lane halves take the halves of a wave's
// part, and a lane's codes of it are one or two 16-byte chunks.
//
// LDS: a token's step is its 16-byte chunks, c at c ^ (t & 15); a row's codes
// 128 bytes, chunk c at c ^ ((r >> 1) & 7), or 256, c at c ^ (r & 15): the reads
// of 16 lanes hit all banks.
//
// With more than one part (`splits`) the workgroups leave fp32 sums in the
// workspace, [part][matrix][T][Np] (Np: N rounded up to whole tiles), and
// quant_join_kernel adds them in order and finishes the outputs.
//
// Bound by the steps, each a barrier with one workgroup a compute unit, more
// than by bytes: T = 32 9999x4096 11 to 12 us, most of it 8 steps on 157 of the
// 256 compute units (the weights, 23 MB, take 4.8 us at the rate of a copy);
// splitting each tile in two takes a unit's time off and adds the join's.
// MXFP4, T = 32: 9999x4096 10.5 us, 10240x2560 8 to 9 (14 MB, 3.0 us).
#include "quant_common.h"

#include <type_traits>

namespace moe {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kSplitWaves = 8;
constexpr int kSplitThreads = kSplitWaves * kWave;
constexpr uint32_t kSplitLds = 160 * 1024;
constexpr int kMaxSplits = 16;

// Reduction indices of a step, and the multiple of them that a part of the
// reduction starts at.  NVFP4, whose weights take twice MXFP4's instructions,
// has fewer barriers with longer steps, three stages of which LDS holds for up
// to 32 tokens: T = 32 9999x4096, measured in turn, 512: 13.2 us, 256: 15.0; MXFP4,
// T = 32 10240x2560, with less of its loads in flight: 11.0 and 9.8.
constexpr int split_unit(int rows, int tokens) { return rows == 64 && tokens <= 32 ? 512 : 256; }
constexpr int split_step(int format, int rows, int tokens) {
  return format == MOE_QUANT_NVFP4 ? split_unit(rows, tokens) : 256;
}

// WIDE: the scales of a row's step start at a multiple of four bytes and go
// to LDS with the rest; else every lane loads its own, two bytes at a time
// (NVFP4) or one.
template <int FMT, bool GU, int ROWS, int TOK, bool WIDE>
struct SplitTile {
  static constexpr int SK = split_step(FMT, ROWS, TOK);
  static constexpr int kTokenBytes = TOK * SK * 2, kCodeBytes = ROWS * SK / 2;
  static constexpr int kScaleBytes = WIDE ? kSplitThreads * 4 : 0;
  static constexpr int kStageBytes = kTokenBytes + kCodeBytes + kScaleBytes;
  static constexpr int kFit = kSplitLds / kStageBytes, kStages = kFit < 6 ? kFit : 6;
  static constexpr int RG = ROWS / 32, KP = kSplitWaves / RG, U = SK / 64 / KP;      // row groups, parts of a step, chunks a lane
  static constexpr int XL = kTokenBytes / 1024 / kSplitWaves, CL = kCodeBytes / 1024 / kSplitWaves;
  static constexpr int kLoads = XL + CL + (WIDE ? 1 : U);    // a step's, per wave
  __amdgpu_buffer_rsrc_t rc, rs, rx;                         // the wave's matrix, the tokens
  uint32_t c_off[CL], s_off, x_off[XL];
  uint16_t ws[kStages][U];

  template <int S>
  __device__ __forceinline__ void issue(uint8_t* stage, int wave, uint32_t step) {
#pragma unroll
    for (int i = 0; i < XL; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, stage + (i * kSplitWaves + wave) * 1024, 16, x_off[i] + step * (SK * 2u), 0, 0, 0);
    // wave w loads the codes of ROWS/8 rows from w * ROWS/8 on, of one matrix only
#pragma unroll
    for (int i = 0; i < CL; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rc, stage + kTokenBytes + (wave * CL + i) * 1024, 16, c_off[i] + step * (SK / 2u), 0, 0, 0);
    constexpr uint32_t kStep = SK / kScaleGroup<FMT>;        // scale bytes of a row's step
    if constexpr (WIDE) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, stage + kTokenBytes + kCodeBytes + wave * 256, 4, s_off + step * kStep, 0, 0, 0);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if constexpr (FMT == MOE_QUANT_NVFP4) ws[S][u] = __builtin_amdgcn_raw_buffer_load_b16(rs, s_off + step * kStep + u * 2u, 0, 0);
        else ws[S][u] = __builtin_amdgcn_raw_buffer_load_b8(rs, s_off + step * kStep + u, 0, 0);
      }
    }
  }
};

template <int FMT, bool GU, int ROWS, int TOK, bool WIDE>
__global__ __launch_bounds__(kSplitThreads, 2) void quant_split_kernel(DenseArgs p, int row_tiles, int tiles, int splits,
                                                                       float* __restrict__ sums) {
  using Tile = SplitTile<FMT, GU, ROWS, TOK, WIDE>;
  constexpr int NS = Tile::kStages, RG = Tile::RG, KP = Tile::KP, U = Tile::U, SK = Tile::SK;
  constexpr int kChunks = SK / 8, kCodeChunks = SK / 32;     // 16-byte pieces of a token's, of a row's step
  constexpr int JT = TOK < 32 ? 1 : TOK / 32, kRows = GU ? ROWS / 2 : ROWS;
  static_assert(NS >= 3 && JT * 16384 <= Tile::kStageBytes, "three stages or more; the waves' sums fit the first ones");
  // one array per stage, so that reads of one stage are seen not to alias the
  // loads in flight to the others
  __shared__ __align__(16) uint8_t s_0[Tile::kStageBytes];
  __shared__ __align__(16) uint8_t s_1[Tile::kStageBytes];
  __shared__ __align__(16) uint8_t s_2[Tile::kStageBytes];
  __shared__ __align__(16) uint8_t s_3[NS > 3 ? Tile::kStageBytes : 16];
  __shared__ __align__(16) uint8_t s_4[NS > 4 ? Tile::kStageBytes : 16];
  __shared__ __align__(16) uint8_t s_5[NS > 5 ? Tile::kStageBytes : 16];
  auto stage_at = [&](auto g) -> uint8_t* {
    constexpr int G = decltype(g)::value % NS;
    if constexpr (G == 0) return s_0;
    else if constexpr (G == 1) return s_1;
    else if constexpr (G == 2) return s_2;
    else if constexpr (G == 3) return s_3;
    else if constexpr (G == 4) return s_4;
    else return s_5;
  };
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  if (GU && (int)blockIdx.x >= tiles * splits) {             // token gates, one wave a token
    const int t = ((int)blockIdx.x - tiles * splits) * kSplitWaves + wave;
    if (t < p.T) token_gate_row(p, t, lane);
    return;
  }
  const int split = (int)blockIdx.x / tiles, tile = (int)blockIdx.x % tiles;
  const int n0 = (tile % row_tiles) * kRows, t0 = (tile / row_tiles) * TOK;
  const int l32 = lane & 31, half = lane >> 5, rg = wave % RG, kp = wave / RG;
  const int rows = min(kRows, p.N - n0), toks = min(TOK, p.T - t0);

  // LDS places: chunk c of row r's codes at c ^ code_swizzle(r)
  auto code_swizzle = [](int r) { return SK == 256 ? (r >> 1) & 7 : r & 15; };
  auto token_row = [&](int i) { return (i * kSplitWaves + wave) * (kWave / kChunks) + lane / kChunks; };
  const float ga = global_scale(p.a), gb = GU ? global_scale(p.b) : 1.0f;       // (early: not when they are needed)
  Tile tl;
  const uint32_t code_row = (uint32_t)p.K / 2, scale_row = (uint32_t)(p.K / kScaleGroup<FMT>);
  // loads: ROWS/8 rows a wave, the second half of the waves the second matrix of a pair
  const QuantMat wc = GU && wave >= 4 ? p.b : p.a;
  tl.rc = make_rsrc(wc.codes + (size_t)n0 * code_row, (uint32_t)rows * code_row);
  tl.rx = make_rsrc(p.x + (size_t)t0 * p.K, (uint32_t)toks * (uint32_t)p.K * 2u);
#pragma unroll
  for (int i = 0; i < Tile::CL; ++i) {
    const int r = (wave * Tile::CL + i) * (kWave / kCodeChunks) + lane / kCodeChunks, c = lane % kCodeChunks ^ code_swizzle(r);
    tl.c_off[i] = (uint32_t)(r % kRows) * code_row + (uint32_t)c * 16u;
  }
#pragma unroll
  for (int i = 0; i < Tile::XL; ++i) {
    const int r = token_row(i), c = lane % kChunks ^ (r & 15);
    tl.x_off[i] = (uint32_t)min(r, toks - 1) * (uint32_t)p.K * 2u + (uint32_t)c * 16u;     // past the last token: it again
  }
  if constexpr (WIDE) {
    // dword w*64 + l of the stage's scales: row by row
    constexpr int kPer = SK / kScaleGroup<FMT> / 4;
    const int r = tid / kPer;
    const QuantMat ws = GU && wave * kWave / kPer >= kRows ? p.b : p.a;   // a wave's rows are of one matrix
    tl.rs = make_rsrc(ws.scales + (size_t)n0 * scale_row, (uint32_t)rows * scale_row);
    tl.s_off = r < ROWS ? (uint32_t)(r % kRows) * scale_row + (uint32_t)(tid % kPer) * 4u : kOutside;
  } else {
    const QuantMat ws = GU && rg >= RG / 2 ? p.b : p.a;
    tl.rs = make_rsrc(ws.scales + (size_t)n0 * scale_row, (uint32_t)rows * scale_row);
    tl.s_off = (uint32_t)((rg * 32 + l32) % kRows) * scale_row + (uint32_t)((kp * 2 + half) * U) * (FMT == MOE_QUANT_NVFP4 ? 2u : 1u);
  }
  constexpr int kUnit = split_unit(ROWS, TOK), kPer = kUnit / SK;      // steps of a unit
  const int units = (p.K + kUnit - 1) / kUnit, each = units / splits, more = units % splits;
  const int first = (split * each + min(split, more)) * kPer;
  const int S = min((each + (split < more ? 1 : 0)) * kPer, (p.K + SK - 1) / SK - first);
  f32x16 acc[JT];
#pragma unroll
  for (int j = 0; j < JT; ++j) acc[j] = f32x16{};

  // a step past this part's last is issued out of range: it reads nothing
  auto at = [&](int s) { return s < S ? (uint32_t)(first + s) : kOutside / 1024u; };
#define MOE_ISSUE(J)                                                                          \
  if constexpr (J < NS - 1) {                                                                 \
    tl.template issue<J>(stage_at(std::integral_constant<int, J>{}), wave, at(J));            \
    fence();                                                                                  \
  }
  MOE_ISSUE(0) MOE_ISSUE(1) MOE_ISSUE(2) MOE_ISSUE(3) MOE_ISSUE(4)
#undef MOE_ISSUE
  auto body = [&](auto stage_c, int s) {
    constexpr int G = decltype(stage_c)::value, F = (G + NS - 1) % NS;
    wait_vm<(NS - 2) * Tile::kLoads>();                      // this wave's part of step s is here
    uint8_t* const stage = stage_at(stage_c);
    const int left = p.K - (first + s) * SK;
    if (left < SK) {                                    // what follows a token's row is not its
#pragma unroll
      for (int i = 0; i < Tile::XL; ++i) {
        if ((lane % kChunks ^ (token_row(i) & 15)) * 8 >= left)
          *reinterpret_cast<uint4*>(stage + (i * kSplitWaves + wave) * 1024 + lane * 16) = make_uint4(0, 0, 0, 0);
      }
    }
    wait_lds();                                              // and its reads of step s-1 have returned
    barrier();                                               // so the stage of step s-1 may be filled again
    tl.template issue<F>(stage_at(std::integral_constant<int, F>{}), wave, at(s + NS - 1));
    const int r = rg * 32 + l32;
    uint32_t sb[U];
    if constexpr (WIDE) {
      const uint8_t* const sr = stage + Tile::kTokenBytes + Tile::kCodeBytes;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = (kp * 2 + half) * U + u;
        if constexpr (FMT == MOE_QUANT_NVFP4) sb[u] = *reinterpret_cast<const uint16_t*>(sr + r * (SK / 16) + c * 2);
        else sb[u] = sr[r * (SK / 32) + c];
      }
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) sb[u] = tl.ws[G][u];
    }
    bf16x8 af[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = ((kp * 2 + half) * U + u) ^ code_swizzle(r);
      dequant32<FMT>(*reinterpret_cast<const uint4*>(stage + Tile::kTokenBytes + r * (SK / 2) + c * 16), sb[u], af[u]);
    }
#pragma unroll
    for (int i = 0; i < 4 * U; ++i)
#pragma unroll
      for (int j = 0; j < JT; ++j) {
        const int t = TOK < 32 ? l32 & (TOK - 1) : j * 32 + l32;
        const bf16x8 b = *reinterpret_cast<const bf16x8*>(stage + t * (SK * 2) + ((((kp * 2 + half) * 4 * U + i) ^ (t & 15)) << 4));
        acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(af[i / 4][i % 4], b, acc[j], 0, 0, 0);
      }
  };
  // whole rings in the loop (one pattern of loads in flight at the back edge), then the rest
  int s0 = 0;
#define MOE_STEP(J) \
  if constexpr (J < NS) body(std::integral_constant<int, J>{}, s0 + J);
#define MOE_REST(J)           \
  if constexpr (J < NS - 1) { \
    if (s0 + J < S) body(std::integral_constant<int, J>{}, s0 + J); \
  }
  for (; s0 + NS <= S; s0 += NS) {
    MOE_STEP(0) MOE_STEP(1) MOE_STEP(2) MOE_STEP(3) MOE_STEP(4) MOE_STEP(5)
  }
  MOE_REST(0) MOE_REST(1) MOE_REST(2) MOE_REST(3) MOE_REST(4)
#undef MOE_STEP
#undef MOE_REST
  wait_vm<0>();                                              // the loads past the last step have landed
  __syncthreads();

  // The waves' sums to LDS (tiles 0..3 in stage 0, 4..7 in stage 1, the
  // others in stage 2): pieces of four rows, register group g of lane l at slot g*64 + (l ^ x), x from
  // the rows, so that a token's pieces lie in different banks
  auto area = [&](int w, int j) {
    const int i = w * JT + j;
    return reinterpret_cast<f32x4*>(i < 4 ? s_0 : i < 8 ? s_1 : s_2) + (i < 4 ? i : i < 8 ? i - 4 : i - 8) * 256;
  };
#pragma unroll
  for (int j = 0; j < JT; ++j) {
    f32x4* const out = area(wave, j);
#pragma unroll
    for (int g = 0; g < 4; ++g)
      out[g * 64 + (lane ^ ((rg * 8 + g * 2 + half) & 15))] =
          f32x4{acc[j][g * 4], acc[j][g * 4 + 1], acc[j][g * 4 + 2], acc[j][g * 4 + 3]};
  }
  __syncthreads();
  const int np = row_tiles * kRows;
  for (int i = tid; i < toks * (kRows / 4); i += kSplitThreads) {
    const int tok = i / (kRows / 4), piece = i % (kRows / 4);          // a token's four rows
    const int w = piece >> 3, g = (piece >> 1) & 3, h = piece & 1, j = tok >> 5, l = h * 32 + (tok & 31);
    auto sum = [&](int v) {
      const int at_l = g * 64 + (l ^ ((v * 8 + g * 2 + h) & 15));
      f32x4 x = area(v, j)[at_l];
#pragma unroll
      for (int k = 1; k < KP; ++k) x += area(v + k * RG, j)[at_l];
      return x;
    };
    const f32x4 a = sum(w), b = GU ? sum(w + RG / 2) : a;
    const int t = t0 + tok, n = n0 + piece * 4;
    if (splits == 1) {
      write4<GU>(p, t, n, a, b, ga, gb);
    } else {
      *reinterpret_cast<f32x4*>(sums + ((size_t)(split * (GU ? 2 : 1)) * p.T + t) * np + n) = a;
      if constexpr (GU) *reinterpret_cast<f32x4*>(sums + ((size_t)(split * 2 + 1) * p.T + t) * np + n) = b;
    }
  }
}

// y[t, 4 rows] from the parts' sums, in the order of the parts
template <bool GU>
__global__ __launch_bounds__(256) void quant_join_kernel(DenseArgs p, int np, int splits, const float* __restrict__ sums) {
  constexpr int NA = GU ? 2 : 1;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const int per = np / 4, t = (int)(i / per), n = (int)(i % per) * 4;
  if (t >= p.T || n >= p.N) return;
  const float ga = global_scale(p.a), gb = GU ? global_scale(p.b) : 1.0f;
  const float* const at = sums + (size_t)t * np + n;
  const size_t part = (size_t)p.T * np;
  f32x4 v[NA] = {};
  constexpr int kTogether = 8;                               // parts in flight: one round trip for all of them
  for (int s0 = 0; s0 < splits; s0 += kTogether) {
    f32x4 q[kTogether][NA];
#pragma unroll
    for (int s = 0; s < kTogether; ++s)
#pragma unroll
      for (int m = 0; m < NA; ++m)
        q[s][m] = *reinterpret_cast<const f32x4*>(at + (min(s0 + s, splits - 1) * NA + m) * part);
#pragma unroll
    for (int s = 0; s < kTogether; ++s)
      if (s0 + s < splits)
#pragma unroll
        for (int m = 0; m < NA; ++m) v[m] += q[s][m];
  }
  write4<GU>(p, t, n, v[0], v[NA - 1], ga, gb);
}

constexpr int kUnits = 256;                                  // workgroups at once: one a compute unit (LDS)
// More parts than one only where all their workgroups run at once: each leaves
// at most 128 rows' sums of 64 tokens.
static_assert(kUnits * 128ull * 64 * sizeof(float) <= MOE_QUANT_SUMS_BYTES, "what moe.h says of the workspace");

struct SplitPlan {
  int tokens, rows, row_tiles, tiles, splits, np;
  float us;
};

// Rows of a tile and parts of the reduction, by the time they should take: one
// workgroup a compute unit (LDS), `rounds` of them, their units at the time
// measured for a unit, and for more than one part the join (its launch, and
// its sums written and read).  T = 64 10240x2560: 13.1 us as 64 rows in one
// part, 17.4 as 128 rows in three; T = 100, where 64 rows take two rounds:
// 20.9 against 17.4 as 128 rows in one part.
SplitPlan plan(bool gate_up, int T, int N, int K) {
  constexpr float kStep64[] = {1.1f, 0.9f}, kStep128[] = {1.2f, 1.4f};       // us a unit, up to 32 and 64 tokens
  constexpr float kJoin = 3.5f, kJoinBytes = 5e6f;                            // us, and bytes a us
  SplitPlan best{};
  const int tokens = T <= 16 ? 16 : T <= 32 ? 32 : 64;
  for (int rows = 64; rows <= (tokens == 16 ? 64 : 128); rows += 64) {
    const int own = gate_up ? rows / 2 : rows, row_tiles = (N + own - 1) / own;
    const int tiles = row_tiles * ((T + tokens - 1) / tokens), unit = split_unit(rows, tokens), units = (K + unit - 1) / unit;
    for (int splits = 1; splits <= kMaxSplits && splits <= units; ++splits) {
      if (splits > 1 && (long long)tiles * splits > kUnits) break;
      const int rounds = (tiles * splits + kUnits - 1) / kUnits;
      float us = (float)rounds * (float)((units + splits - 1) / splits) * (rows == 64 ? kStep64 : kStep128)[tokens > 32];
      if (splits > 1) us += kJoin + 8.0f * splits * (gate_up ? 2 : 1) * (float)T * (float)(row_tiles * own) / kJoinBytes;
      if (best.splits == 0 || us < best.us) best = {tokens, rows, row_tiles, tiles, splits, row_tiles * own, us};
    }
  }
  return best;
}

template <int FMT, bool GU, int ROWS, int TOK, bool WIDE>
moe_status launch(const DenseArgs& p, const SplitPlan& q, void* workspace, hipStream_t s) {
  float* const sums = static_cast<float*>(workspace);
  const int grid = q.tiles * q.splits + (GU && p.token_gate ? (p.T + kSplitWaves - 1) / kSplitWaves : 0);
  quant_split_kernel<FMT, GU, ROWS, TOK, WIDE>
      <<<(unsigned)grid, kSplitThreads, 0, s>>>(p, q.row_tiles, q.tiles, q.splits, sums);
  const moe_status st = launch_status();
  if (st != MOE_OK || q.splits == 1) return st;
  const long long work = (long long)p.T * (q.np / 4);
  quant_join_kernel<GU><<<(unsigned)((work + 255) / 256), 256, 0, s>>>(p, q.np, q.splits, sums);
  return launch_status();
}

template <int FMT, bool GU>
moe_status dispatch(const DenseArgs& p, void* workspace, hipStream_t s) {
  const SplitPlan q = plan(GU, p.T, p.N, p.K);
  const bool wide = (p.K / kScaleGroup<FMT>) % 4 == 0;
#define MOE_SPLIT(ROWS, TOK) \
  return wide ? launch<FMT, GU, ROWS, TOK, true>(p, q, workspace, s) : launch<FMT, GU, ROWS, TOK, false>(p, q, workspace, s)
  if (q.tokens == 16) MOE_SPLIT(64, 16);
  if (q.rows == 64) {
    if (q.tokens == 32) MOE_SPLIT(64, 32);
    MOE_SPLIT(64, 64);
  }
  if (q.tokens == 32) MOE_SPLIT(128, 32);
  MOE_SPLIT(128, 64);
#undef MOE_SPLIT
}

}  // namespace

size_t quant_split_workspace(bool gate_up, int T, int N, int K) {
  const SplitPlan q = plan(gate_up, T, N, K);
  return q.splits == 1 ? 0 : (size_t)q.splits * (gate_up ? 2 : 1) * (size_t)T * (size_t)q.np * 4;
}

float quant_split_us(bool gate_up, int T, int N, int K) { return plan(gate_up, T, N, K).us; }

moe_status quant_split(int format, bool gate_up, const DenseArgs& p, void* workspace, hipStream_t s) {
  if (format == MOE_QUANT_NVFP4)
    return gate_up ? dispatch<MOE_QUANT_NVFP4, true>(p, workspace, s) : dispatch<MOE_QUANT_NVFP4, false>(p, workspace, s);
  return gate_up ? dispatch<MOE_QUANT_MXFP4, true>(p, workspace, s) : dispatch<MOE_QUANT_MXFP4, false>(p, workspace, s);
}

}  // namespace moe
