// 4-bit products of few tokens: bound by the weight bytes, which are streamed
// once.
//
// A workgroup owns 16 * R weight rows (of one matrix, or the same rows of a
// gate/up pair) and up to TT tokens.  Its waves split the reduction and join
// at the end through LDS in a fixed order: with few rows there are still
// enough waves to keep the memory busy, and no wave waits for another while
// it streams.  The weights are the A operand of v_mfma_f32_16x16x32_bf16, the
// tokens the B operand (columns past the last token repeat it; their sums
// are dropped), so one token costs what sixteen cost and no sum crosses
// lanes.
//
// Lane layout: A lane l holds row l%16, reduction indices 8*(l/16)..+8; B
// lane l column l%16, the same indices; D register r of lane l is row
// 4*(l/16) + r, column l%16.  The reduction index is permuted alike in A and
// B: in a step of 128 the lane quarter q = l/16 covers 32q .. 32q+32, and
// instruction i of the step takes 8 of them, so a lane's codes of a step are
// one 16-byte load, with the two e4m3 scales (one e8m0) of that block.
//
// The tokens' step goes straight to LDS (buffer_load ... lds), into a region
// of the wave's own: 256 bytes a token, 16-byte chunk c of token t at
// c ^ (t % 16), so that the fragment reads of 16 tokens hit all banks.  Codes
// and scales go to a register ring.  A step's loads are issued NS-1 steps
// ahead; past a wave's last step they are issued out of range (which
// returns zeros and reads nothing), so that every iteration has the same
// loads in flight.
#include "quant_common.h"

#include <type_traits>

namespace moe {
namespace {

template <int FMT, bool GU, int R, int TT, int WAVES, int NS>
struct StreamTile {
  static constexpr int NA = (GU ? 2 : 1) * R;                // A operands: R row tiles of each matrix
  static constexpr int NT = TT < 16 ? 1 : TT / 16;
  static constexpr int XL = TT * 256 / 1024;                 // token loads per step
  static constexpr int kLoads = 2 * NA + XL;
  static constexpr int kWaveBytes = TT * 256;
  __amdgpu_buffer_rsrc_t rc[GU ? 2 : 1], rs[GU ? 2 : 1], rx;
  uint32_t c_off[R], s_off[R], x_off[XL];
  uint4 wc[NS][NA];
  uint16_t ws[NS][NA];                                       // 16 bits until used: a widening would wait for its load

  template <int S>
  __device__ __forceinline__ void issue(uint8_t* stage, uint32_t step) {
#pragma unroll
    for (int j = 0; j < XL; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, stage + j * 1024, 16, x_off[j] + step * 256u, 0, 0, 0);
#pragma unroll
    for (int a = 0; a < NA; ++a) {
      const int m = a / R, r = a % R;
      if constexpr (FMT == MOE_QUANT_NVFP4)
        ws[S][a] = __builtin_amdgcn_raw_buffer_load_b16(rs[m], s_off[r] + step * 8u, 0, 0);
      else
        ws[S][a] = __builtin_amdgcn_raw_buffer_load_b8(rs[m], s_off[r] + step * 4u, 0, 0);
      wc[S][a] = to_uint4(__builtin_amdgcn_raw_buffer_load_b128(rc[m], c_off[r] + step * 64u, 0, kStreamAux));
    }
  }
};

template <int FMT, bool GU, int R, int TT, int WAVES, int NS>
__global__ __launch_bounds__(WAVES * kWave) void quant_stream_kernel(DenseArgs p, int row_tiles, int tiles) {
  using Tile = StreamTile<FMT, GU, R, TT, WAVES, NS>;
  constexpr int NA = Tile::NA, NT = Tile::NT, D = NS - 1;
  // one array per stage, so that reads of one stage are seen not to alias the
  // loads in flight to the others
  __shared__ __align__(16) uint8_t s_x0[WAVES * Tile::kWaveBytes];
  __shared__ __align__(16) uint8_t s_x1[WAVES * Tile::kWaveBytes];
  __shared__ __align__(16) uint8_t s_x2[NS > 2 ? WAVES * Tile::kWaveBytes : 16];
  __shared__ __align__(16) uint8_t s_x3[NS > 3 ? WAVES * Tile::kWaveBytes : 16];
  static_assert(NS >= 2 && NS <= 4, "stages");
  constexpr int kRedBytes = WAVES * NA * NT * 1024;          // the waves' sums
  constexpr bool kRedApart = kRedBytes > WAVES * Tile::kWaveBytes;
  __shared__ __align__(16) uint8_t s_red[kRedApart ? kRedBytes : 16];

  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if ((int)blockIdx.x >= tiles) {                            // token gates, one wave a token
    const int t = ((int)blockIdx.x - tiles) * WAVES + wave;
    if (t < p.T) token_gate_row(p, t, lane);
    return;
  }
  const int l16 = lane & 15, q = lane >> 4;
  const int n0 = ((int)blockIdx.x % row_tiles) * 16 * R, t0 = ((int)blockIdx.x / row_tiles) * TT;
  const int rows = min(16 * R, p.N - n0), toks = min(TT, p.T - t0);

  Tile tl;
  const uint32_t code_row = (uint32_t)p.K / 2, scale_row = (uint32_t)(p.K / kScaleGroup<FMT>);
#pragma unroll
  for (int m = 0; m < (GU ? 2 : 1); ++m) {
    const QuantMat& w = m ? p.b : p.a;
    tl.rc[m] = make_rsrc(w.codes + (size_t)n0 * code_row, (uint32_t)rows * code_row);
    tl.rs[m] = make_rsrc(w.scales + (size_t)n0 * scale_row, (uint32_t)rows * scale_row);
  }
  tl.rx = make_rsrc(p.x + (size_t)t0 * p.K, (uint32_t)toks * (uint32_t)p.K * 2u);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    tl.c_off[r] = (uint32_t)(r * 16 + l16) * code_row + (uint32_t)q * 16u;
    tl.s_off[r] = (uint32_t)(r * 16 + l16) * scale_row + (uint32_t)q * (FMT == MOE_QUANT_NVFP4 ? 2u : 1u);
  }
#pragma unroll
  for (int j = 0; j < Tile::XL; ++j) {
    const int row = j * 4 + q, c = l16 ^ (row & 15);         // lane l: token row l/16 of four, chunk position l%16
    tl.x_off[j] = (uint32_t)min(row, toks - 1) * (uint32_t)p.K * 2u + (uint32_t)c * 16u;
  }
  // this wave's steps of 128: the first `more` waves have one step more
  const int steps = (p.K + 127) / 128, each = steps / WAVES, more = steps % WAVES;
  const int first = wave * each + min(wave, more), S = each + (wave < more ? 1 : 0);
  uint8_t* const my[4] = {s_x0 + wave * Tile::kWaveBytes, s_x1 + wave * Tile::kWaveBytes,
                          s_x2 + (NS > 2 ? wave * Tile::kWaveBytes : 0), s_x3 + (NS > 3 ? wave * Tile::kWaveBytes : 0)};

  f32x4 acc[NA][NT];
#pragma unroll
  for (int a = 0; a < NA; ++a)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[a][t] = f32x4{};

  // a step past the last one reads nothing
  auto at = [&](int s) { return s < S ? (uint32_t)(first + s) : kOutside / 256u; };
  tl.template issue<0>(my[0], at(0));
  fence();
  if constexpr (D > 1) {
    tl.template issue<1>(my[1], at(1));
    fence();
  }
  if constexpr (D > 2) {
    tl.template issue<2>(my[2], at(2));
    fence();
  }
  auto body = [&](auto stage_c, int s) {
    constexpr int G = decltype(stage_c)::value;
    wait_lds();                                              // this wave's reads of the stage refilled now
    tl.template issue<(G + D) % NS>(my[(G + D) % NS], at(s + D));
    wait_vm<D * Tile::kLoads>();                             // step s is here
    bf16x8 af[NA][4];
#pragma unroll
    for (int a = 0; a < NA; ++a) dequant32<FMT>(tl.wc[G][a], tl.ws[G][a], af[a]);
    uint8_t* const xs = (G == 0 ? s_x0 : G == 1 ? s_x1 : G == 2 ? s_x2 : s_x3) + wave * Tile::kWaveBytes;
    const int left = p.K - (first + s) * 128;
    if (left < 128) {                                        // what follows a token's row is not its
#pragma unroll
      for (int j = 0; j < Tile::XL; ++j)
        if ((l16 ^ ((j * 4 + q) & 15)) * 8 >= left) *reinterpret_cast<uint4*>(xs + j * 1024 + lane * 16) = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int row = TT < 16 ? min(l16, TT - 1) : t * 16 + l16;
      const uint8_t* const xr = xs + row * 256;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bf16x8 b = *reinterpret_cast<const bf16x8*>(xr + (((q * 4 + i) ^ (row & 15)) << 4));
#pragma unroll
        for (int a = 0; a < NA; ++a) acc[a][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(af[a][i], b, acc[a][t], 0, 0, 0);
      }
    }
  };
  int s0 = 0;
  for (; s0 + NS <= S; s0 += NS) {
    body(std::integral_constant<int, 0>{}, s0);
    body(std::integral_constant<int, 1>{}, s0 + 1);
    if constexpr (NS > 2) body(std::integral_constant<int, 2>{}, s0 + 2);
    if constexpr (NS > 3) body(std::integral_constant<int, 3>{}, s0 + 3);
  }
  if (s0 < S) body(std::integral_constant<int, 0>{}, s0);
  if constexpr (NS > 2)
    if (s0 + 1 < S) body(std::integral_constant<int, 1>{}, s0 + 1);
  if constexpr (NS > 3)
    if (s0 + 2 < S) body(std::integral_constant<int, 2>{}, s0 + 2);
  wait_vm<0>();                                              // the loads past the last step have landed
  __syncthreads();

  f32x4* const red = reinterpret_cast<f32x4*>(kRedApart ? s_red : s_x0);
#pragma unroll
  for (int a = 0; a < NA; ++a)
#pragma unroll
    for (int t = 0; t < NT; ++t) red[((wave * NA + a) * NT + t) * kWave + lane] = acc[a][t];
  __syncthreads();
  for (int i = threadIdx.x; i < R * NT * kWave; i += WAVES * kWave) {
    const int r = i / (NT * kWave), rest = i % (NT * kWave);  // row tile; token tile and lane
    const int t = t0 + (rest >> 6) * 16 + (rest & 15), n = n0 + r * 16 + ((rest >> 4) & 3) * 4;
    if ((rest >> 6) * 16 + (rest & 15) >= toks) continue;
    f32x4 va = red[r * NT * kWave + rest], vb = GU ? red[(R + r) * NT * kWave + rest] : f32x4{};
#pragma unroll
    for (int w = 1; w < WAVES; ++w) {
      va += red[(w * NA + r) * NT * kWave + rest];
      if constexpr (GU) vb += red[(w * NA + R + r) * NT * kWave + rest];
    }
    write4<GU>(p, t, n, va, vb);
  }
}

template <int FMT, bool GU, int R, int TT, int WAVES, int NS>
moe_status launch(const DenseArgs& p, hipStream_t s) {
  const int row_tiles = (p.N + 16 * R - 1) / (16 * R);
  const int tiles = row_tiles * ((p.T + TT - 1) / TT);       // at most 2^29 (N and T up to 2^20)
  const int grid = tiles + (p.token_gate ? (p.T + WAVES - 1) / WAVES : 0);
  quant_stream_kernel<FMT, GU, R, TT, WAVES, NS><<<(unsigned)grid, WAVES * kWave, 0, s>>>(p, row_tiles, tiles);
  return launch_status();
}

template <int FMT, bool GU>
moe_status dispatch(const DenseArgs& p, hipStream_t s) {
  if (p.T <= 16) return launch<FMT, GU, 1, 16, 4, 3>(p, s);
  if (p.T <= 32) return launch<FMT, GU, 2, 32, 4, 2>(p, s);
  return launch<FMT, GU, 2, 64, 4, 2>(p, s);
}

}  // namespace

moe_status quant_stream(int format, bool gate_up, const DenseArgs& p, hipStream_t s) {
  if (format == MOE_QUANT_NVFP4)
    return gate_up ? dispatch<MOE_QUANT_NVFP4, true>(p, s) : dispatch<MOE_QUANT_NVFP4, false>(p, s);
  return gate_up ? dispatch<MOE_QUANT_MXFP4, true>(p, s) : dispatch<MOE_QUANT_MXFP4, false>(p, s);
}

}  // namespace moe
