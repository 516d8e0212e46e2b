// 4-bit products of batches whose tiles are too few for the chip: 128 weight
// rows by 16, 32 or 64 tokens, the reduction split over workgroups.
//
// Tokens, codes and scales all go straight to LDS (buffer_load ... lds),
// steps of 256 of the reduction, two steps ahead in a ring of three stages:
// a row's 128 code bytes of a step are one cache line, which 8 lanes of one
// load take whole.  (Loaded to registers, in the layout of the matrix tiles,
// each load touches 16 bytes of 64 rows' lines, and the scales 2 bytes of
// them: the lines that a compute unit's L1 then fetches again and again were
// 4 times the bytes used, and set the time.)
//
// Eight waves: wave w takes 32 rows (w % 4) and half of each step (w / 4),
// so that every weight is decoded once.  Of a gate/up pair a workgroup has 64
// rows each, waves with w % 4 >= 2 the second matrix's.
// v_mfma_f32_32x32x16_bf16, weights as A: lane l holds row l%32, reduction
// indices 8*(l/32)..+8; tokens as B: column l%32, the same indices; D
// register r is row 8*(r/4) + 4*(l/32) + r%4, column l%32.  The reduction
// index is permuted alike in both: of a wave's 128 the lane half h covers
// 64h .. 64h+64.
//
// LDS: a token's step is 512 bytes, its 16-byte chunk c at c ^ (t & 15); a
// row's codes 128 bytes, chunk c at c ^ ((r >> 1) & 7): the reads of 16 lanes
// hit all banks.
//
// With more than one part (`splits`) the workgroups leave fp32 sums in the
// workspace, [part][matrix][T][Np] (Np: N rounded up to whole tiles), and
// quant_join_kernel adds them in order and finishes the outputs.
#include "quant_common.h"

#include <type_traits>

namespace moe {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kSplitWaves = 8;
constexpr int kSplitThreads = kSplitWaves * kWave;
constexpr int kSplitRows = 128;                              // of one matrix, or 64 of each of two
constexpr int kSplitK = 256;
constexpr int kStages = 3;
constexpr int kMaxSplits = 16;

// WIDE: the scales of a row's step start at a multiple of four bytes and go
// to LDS with the rest; else every lane loads its own, two bytes at a time
// (NVFP4) or one.
template <int FMT, bool GU, int TOK, bool WIDE>
struct SplitTile {
  static constexpr int kTokenBytes = TOK * kSplitK * 2, kCodeBytes = kSplitRows * kSplitK / 2;
  static constexpr int kScaleBytes = WIDE ? kSplitThreads * 4 : 0;
  static constexpr int kStageBytes = kTokenBytes + kCodeBytes + kScaleBytes;
  static constexpr int XL = kTokenBytes / 1024 / kSplitWaves, CL = kCodeBytes / 1024 / kSplitWaves;
  static constexpr int kLoads = XL + CL + (WIDE ? 1 : 2);    // a step's, per wave
  __amdgpu_buffer_rsrc_t rc, rs, rx;                         // the wave's matrix, the tokens
  uint32_t c_off[CL], s_off, x_off[XL];
  uint16_t ws[kStages][2];

  template <int S>
  __device__ __forceinline__ void issue(uint8_t* stage, int wave, uint32_t step) {
#pragma unroll
    for (int i = 0; i < XL; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, stage + (i * kSplitWaves + wave) * 1024, 16, x_off[i] + step * 512u, 0, 0, 0);
    // wave w loads the codes of rows 16w .. 16w+16, and of one matrix only
#pragma unroll
    for (int i = 0; i < CL; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rc, stage + kTokenBytes + (wave * CL + i) * 1024, 16, c_off[i] + step * 128u, 0, 0, 0);
    constexpr uint32_t kStep = FMT == MOE_QUANT_NVFP4 ? 16 : 8;       // scale bytes of a row's step
    if constexpr (WIDE) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, stage + kTokenBytes + kCodeBytes + wave * 256, 4, s_off + step * kStep, 0, 0, 0);
    } else {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if constexpr (FMT == MOE_QUANT_NVFP4) ws[S][u] = __builtin_amdgcn_raw_buffer_load_b16(rs, s_off + step * kStep + u * 2u, 0, 0);
        else ws[S][u] = __builtin_amdgcn_raw_buffer_load_b8(rs, s_off + step * kStep + u, 0, 0);
      }
    }
  }
};

template <int FMT, bool GU, int TOK, bool WIDE>
__global__ __launch_bounds__(kSplitThreads, TOK > 16 ? 2 : 4) void quant_split_kernel(DenseArgs p, int row_tiles, int tiles,
                                                                                   int splits, float* __restrict__ sums) {
  using Tile = SplitTile<FMT, GU, TOK, WIDE>;
  constexpr int JT = TOK < 32 ? 1 : TOK / 32, kRows = GU ? kSplitRows / 2 : kSplitRows;
  static_assert(JT * 16384 <= Tile::kStageBytes, "the waves' sums fit the ring");
  // one array per stage, so that reads of one stage are seen not to alias the
  // loads in flight to the others
  __shared__ __align__(16) uint8_t s_0[Tile::kStageBytes];
  __shared__ __align__(16) uint8_t s_1[Tile::kStageBytes];
  __shared__ __align__(16) uint8_t s_2[Tile::kStageBytes];
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  if ((int)blockIdx.x >= tiles * splits) {                   // token gates, one wave a token
    const int t = ((int)blockIdx.x - tiles * splits) * kSplitWaves + wave;
    if (t < p.T) token_gate_row(p, t, lane);
    return;
  }
  const int split = (int)blockIdx.x / tiles, tile = (int)blockIdx.x % tiles;
  const int n0 = (tile % row_tiles) * kRows, t0 = (tile / row_tiles) * TOK;
  const int l32 = lane & 31, half = lane >> 5, rg = wave & 3, kh = wave >> 2;
  const int rows = min(kRows, p.N - n0), toks = min(TOK, p.T - t0);

  Tile tl;
  const uint32_t code_row = (uint32_t)p.K / 2, scale_row = (uint32_t)(p.K / kScaleGroup<FMT>);
  // loads: 16 rows a wave, the second half of the waves the second matrix of a pair
  const QuantMat wc = GU && wave >= 4 ? p.b : p.a;
  tl.rc = make_rsrc(wc.codes + (size_t)n0 * code_row, (uint32_t)rows * code_row);
  tl.rx = make_rsrc(p.x + (size_t)t0 * p.K, (uint32_t)toks * (uint32_t)p.K * 2u);
#pragma unroll
  for (int i = 0; i < Tile::CL; ++i) {
    const int r = (wave * Tile::CL + i) * 8 + (lane >> 3), c = (lane & 7) ^ ((r >> 1) & 7);
    tl.c_off[i] = (uint32_t)(GU ? r & 63 : r) * code_row + (uint32_t)c * 16u;
  }
#pragma unroll
  for (int i = 0; i < Tile::XL; ++i) {
    const int r = (i * kSplitWaves + wave) * 2 + half, c = l32 ^ (r & 15);
    tl.x_off[i] = (uint32_t)min(r, toks - 1) * (uint32_t)p.K * 2u + (uint32_t)c * 16u;     // past the last token: it again
  }
  if constexpr (WIDE) {
    // dword w*64 + l of the stage's scales: row by row, 4 (NVFP4) or 2 (MXFP4) a row
    constexpr int kPer = FMT == MOE_QUANT_NVFP4 ? 4 : 2;
    const int r = tid / kPer;
    const QuantMat ws = GU && wave * kWave / kPer >= 64 ? p.b : p.a;   // a wave's rows are of one matrix
    tl.rs = make_rsrc(ws.scales + (size_t)n0 * scale_row, (uint32_t)rows * scale_row);
    tl.s_off = r < kSplitRows ? (uint32_t)(GU ? r & 63 : r) * scale_row + (uint32_t)(tid % kPer) * 4u : kOutside;
  } else {
    const QuantMat ws = GU && rg >= 2 ? p.b : p.a;
    tl.rs = make_rsrc(ws.scales + (size_t)n0 * scale_row, (uint32_t)rows * scale_row);
    tl.s_off = (uint32_t)((GU ? rg & 1 : rg) * 32 + l32) * scale_row +
               (uint32_t)(kh * 2 + half) * (FMT == MOE_QUANT_NVFP4 ? 4u : 2u);
  }
  const int all = (p.K + kSplitK - 1) / kSplitK, each = all / splits, more = all % splits;
  const int first = split * each + min(split, more), S = each + (split < more ? 1 : 0);
  f32x16 acc[JT];
#pragma unroll
  for (int j = 0; j < JT; ++j) acc[j] = f32x16{};

  // a step past this part's last is issued out of range: it reads nothing
  auto at = [&](int s) { return s < S ? (uint32_t)(first + s) : kOutside / 1024u; };
  tl.template issue<0>(s_0, wave, at(0));
  fence();
  tl.template issue<1>(s_1, wave, at(1));
  fence();
  auto body = [&](auto stage_c, int s) {
    constexpr int G = decltype(stage_c)::value, F = (G + 2) % kStages;
    wait_vm<Tile::kLoads>();                                 // this wave's part of step s is here
    uint8_t* const stage = G == 0 ? s_0 : G == 1 ? s_1 : s_2;
    const int left = p.K - (first + s) * kSplitK;
    if (left < kSplitK) {                                    // what follows a token's row is not its
#pragma unroll
      for (int i = 0; i < Tile::XL; ++i) {
        const int r = (i * kSplitWaves + wave) * 2 + half;
        if ((l32 ^ (r & 15)) * 8 >= left)
          *reinterpret_cast<uint4*>(stage + (i * kSplitWaves + wave) * 1024 + lane * 16) = make_uint4(0, 0, 0, 0);
      }
    }
    wait_lds();                                              // and its reads of step s-1 have returned
    barrier();                                               // so the stage of step s-1 may be filled again
    tl.template issue<F>(F == 0 ? s_0 : F == 1 ? s_1 : s_2, wave, at(s + 2));
    const int r = rg * 32 + l32;
    uint32_t sb[2];
    if constexpr (WIDE) {
      const uint8_t* const sr = stage + Tile::kTokenBytes + Tile::kCodeBytes;
      if constexpr (FMT == MOE_QUANT_NVFP4) {
        const uint32_t v = *reinterpret_cast<const uint32_t*>(sr + r * 16 + (kh * 2 + half) * 4);
        sb[0] = v, sb[1] = v >> 16;
      } else {
        const uint32_t v = *reinterpret_cast<const uint16_t*>(sr + r * 8 + (kh * 2 + half) * 2);
        sb[0] = v & 0xFFu, sb[1] = v >> 8;
      }
    } else {
      sb[0] = tl.ws[G][0], sb[1] = tl.ws[G][1];
    }
    bf16x8 af[2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int c = (kh * 4 + half * 2 + u) ^ ((r >> 1) & 7);
      dequant32<FMT>(*reinterpret_cast<const uint4*>(stage + Tile::kTokenBytes + r * 128 + c * 16), sb[u], af[u]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < JT; ++j) {
        const int t = TOK < 32 ? l32 & (TOK - 1) : j * 32 + l32;
        const bf16x8 b = *reinterpret_cast<const bf16x8*>(stage + t * 512 + (((kh * 16 + half * 8 + i) ^ (t & 15)) << 4));
        acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(af[i / 4][i % 4], b, acc[j], 0, 0, 0);
      }
  };
  int s0 = 0;
  for (; s0 + kStages <= S; s0 += kStages) {
    body(std::integral_constant<int, 0>{}, s0);
    body(std::integral_constant<int, 1>{}, s0 + 1);
    body(std::integral_constant<int, 2>{}, s0 + 2);
  }
  if (s0 < S) body(std::integral_constant<int, 0>{}, s0);
  if (s0 + 1 < S) body(std::integral_constant<int, 1>{}, s0 + 1);
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
      return area(v, j)[at_l] + area(v + 4, j)[at_l];
    };
    const f32x4 a = sum(w), b = GU ? sum(w + 2) : a;
    const int t = t0 + tok, n = n0 + piece * 4;
    if (splits == 1) {
      write4<GU>(p, t, n, a, b);
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
  write4<GU>(p, t, n, v[0], v[NA - 1]);
}

// Workgroups wanted: one for each of the 256 compute units
constexpr int kWanted = 256;

struct SplitPlan {
  int tokens, row_tiles, tiles, splits, np;
};

SplitPlan plan(bool gate_up, int T, int N, int K) {
  SplitPlan q;
  const int rows = gate_up ? kSplitRows / 2 : kSplitRows;
  q.tokens = T <= 16 ? 16 : T <= 32 ? 32 : 64;
  q.row_tiles = (N + rows - 1) / rows;
  q.np = q.row_tiles * rows;
  q.tiles = q.row_tiles * ((T + q.tokens - 1) / q.tokens);
  const int steps = (K + kSplitK - 1) / kSplitK;
  const int most = steps < kMaxSplits ? steps : kMaxSplits, want = kWanted / q.tiles;
  q.splits = want < 1 ? 1 : want < most ? want : most;
  return q;
}

template <int FMT, bool GU, int TOK, bool WIDE>
moe_status launch(const DenseArgs& p, const SplitPlan& q, void* workspace, hipStream_t s) {
  float* const sums = static_cast<float*>(workspace);
  const int grid = q.tiles * q.splits + (p.token_gate ? (p.T + kSplitWaves - 1) / kSplitWaves : 0);
  quant_split_kernel<FMT, GU, TOK, WIDE><<<(unsigned)grid, kSplitThreads, 0, s>>>(p, q.row_tiles, q.tiles, q.splits, sums);
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
#define MOE_SPLIT(TOK) \
  return wide ? launch<FMT, GU, TOK, true>(p, q, workspace, s) : launch<FMT, GU, TOK, false>(p, q, workspace, s)
  if (q.tokens == 16) MOE_SPLIT(16);
  if (q.tokens == 32) MOE_SPLIT(32);
  MOE_SPLIT(64);
#undef MOE_SPLIT
}

}  // namespace

size_t quant_split_workspace(bool gate_up, int T, int N, int K) {
  const SplitPlan q = plan(gate_up, T, N, K);
  return q.splits == 1 ? 0 : (size_t)q.splits * (gate_up ? 2 : 1) * (size_t)T * (size_t)q.np * 4;
}

moe_status quant_split(int format, bool gate_up, const DenseArgs& p, void* workspace, hipStream_t s) {
  if (format == MOE_QUANT_NVFP4)
    return gate_up ? dispatch<MOE_QUANT_NVFP4, true>(p, workspace, s) : dispatch<MOE_QUANT_NVFP4, false>(p, workspace, s);
  return gate_up ? dispatch<MOE_QUANT_MXFP4, true>(p, workspace, s) : dispatch<MOE_QUANT_MXFP4, false>(p, workspace, s);
}

}  // namespace moe
