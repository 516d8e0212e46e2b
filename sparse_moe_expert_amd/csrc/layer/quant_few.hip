// 4-bit products of one to four tokens: bound by the weight bytes and, close
// behind, by the instructions that decode them.
//
// v_mfma_f32_4x4x4_16b_bf16 computes 16 independent 4 x 4 blocks: block b
// takes 4 tokens (A), 4 weight rows (B) and a part of the reduction of its
// own.  A lane's weights of a step are one 16-byte load, row l%4 and the 32
// reduction indices 32*(l/4)..: a wavefront reads 256 contiguous bytes of
// each of four rows, and eight instructions of 4 indices use them up.  For
// NVFP4 the codes enter unscaled (one conversion for two weights): the four
// instructions of a 16-weight scale block start from zero, and their results
// (a lane's: the tokens' of its own row) are scaled as they are added to the
// sums.  Decoding costs about half an instruction a weight instead of 2 for
// scaled weights, as the 16 x 16 tiles need them, and at four tokens a
// quarter of a dot product's.  MXFP4 scales are powers of two and part of the
// conversion.
//
// A wavefront owns four rows (of a matrix, or of each of a gate/up pair) and
// all of the reduction, with P steps of 512 in flight: no sum leaves the
// wavefront, and nothing but the tokens, staged in LDS once for the
// workgroup's wavefronts, is waited for together.  The four rows' scales are
// contiguous and come to LDS as whole lines (a step's 32-byte pieces of the
// rows would be as many requests as the codes).
//
// Tokens in LDS: a kilobyte for a token's step, its 16-byte chunk c at c ^ t
// for token t, so that the reads of 16 lanes hit all banks.
#include "quant_common.h"

#include <type_traits>

namespace moe {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kStepK = 512;
constexpr int kFewWaves = 8;                                 // at most, per workgroup

template <int B>
__device__ __forceinline__ uint32_t fp4x2_bits(uint32_t word, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, scale, B));
}

__device__ __forceinline__ f32x4 mfma4(uint32_t a0, uint32_t a1, uint32_t b0, uint32_t b1, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(__builtin_bit_cast(s16x4, make_uint2(a0, a1)),
                                                __builtin_bit_cast(s16x4, make_uint2(b0, b1)), c, 0, 0, 0);
}

// 16 weights (8 code bytes) of the lane's row against 16 values of its token
__device__ __forceinline__ f32x4 block16(uint32_t c0, uint32_t c1, const uint4 x0, const uint4 x1, float scale, f32x4 d) {
  d = mfma4(x0.x, x0.y, fp4x2_bits<0>(c0, scale), fp4x2_bits<1>(c0, scale), d);
  d = mfma4(x0.z, x0.w, fp4x2_bits<2>(c0, scale), fp4x2_bits<3>(c0, scale), d);
  d = mfma4(x1.x, x1.y, fp4x2_bits<0>(c1, scale), fp4x2_bits<1>(c1, scale), d);
  return mfma4(x1.z, x1.w, fp4x2_bits<2>(c1, scale), fp4x2_bits<3>(c1, scale), d);
}

// LDS bytes of the scales of four rows: whole kilobytes, as they are loaded
__host__ __device__ constexpr uint32_t scale_bytes(uint32_t scale_row) { return (4 * scale_row + 1023u) & ~1023u; }

// TT: tokens whose sums are kept (T or more)
template <int FMT, bool GU, int TT, int P>
__global__ __launch_bounds__(kFewWaves * kWave, 4) void quant_few_kernel(DenseArgs p, int tiles) {
  constexpr int Q = GU ? 2 : 1;                              // row quads: of the matrix, or of gate and up
  extern __shared__ __align__(16) uint8_t s_mem[];           // tokens, then the waves' scales
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = (int)blockDim.x / kWave;
  if ((int)blockIdx.x >= tiles) {                            // token gates, one wave a token
    const int t = ((int)blockIdx.x - tiles) * waves + wave;
    if (t < p.T) token_gate_row(p, t, lane);
    return;
  }
  const int l4 = lane & 3, b = lane >> 2;
  const int n0 = ((int)blockIdx.x * waves + wave) * 4;       // past N: every load is out of range
  const int rows = max(min(4, p.N - n0), 0);
  const int S = (p.K + kStepK - 1) / kStepK;
  const uint32_t code_row = (uint32_t)p.K / 2, scale_row = (uint32_t)(p.K / kScaleGroup<FMT>);
  const uint32_t scale_pad = scale_bytes(scale_row);
  uint8_t* const s_scale = s_mem + p.T * S * 1024 + wave * Q * scale_pad;

  // tokens: piece (t, s), a kilobyte each
  const auto rx = make_rsrc(p.x, (uint32_t)p.T * (uint32_t)p.K * 2u);
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    if (t >= p.T) break;
    for (int s = wave; s < S; s += waves)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, s_mem + (t * S + s) * 1024, 16,
                                               (uint32_t)t * (uint32_t)p.K * 2u + (uint32_t)s * 1024u +
                                                   (uint32_t)(lane ^ t) * 16u, 0, 0, 0);
  }
  __amdgpu_buffer_rsrc_t rc[Q];
#pragma unroll
  for (int m = 0; m < Q; ++m) {
    const QuantMat& w = m ? p.b : p.a;
    rc[m] = make_rsrc(w.codes + (size_t)n0 * code_row, (uint32_t)rows * code_row);
    // (the range is checked a dword at a time; the last one may hold bytes
    // past the end, in the same aligned dword as bytes before it)
    const auto rs = make_rsrc(w.scales + (size_t)n0 * scale_row, ((uint32_t)rows * scale_row + 3u) & ~3u);
    for (uint32_t c = 0; c < scale_pad; c += 1024)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, s_scale + m * scale_pad + c, 16, c + (uint32_t)lane * 16u, 0, 0, 0);
  }
  const uint32_t c_off = (uint32_t)l4 * code_row + (uint32_t)b * 16u;
  uint4 wc[P][Q];
  // a step past the last one is issued out of range: it reads nothing
  auto issue = [&](auto j_c, int s) {
    constexpr int J = decltype(j_c)::value;
    const uint32_t at = c_off + (s < S ? (uint32_t)s * 256u : kOutside);
#pragma unroll
    for (int m = 0; m < Q; ++m) wc[J][m] = to_uint4(__builtin_amdgcn_raw_buffer_load_b128(rc[m], at, 0, kStreamAux));
  };
  fence();
  for_each<P>([&](auto j) {
    issue(j, decltype(j)::value);
    fence();                                                 // in this order: the waits count on it
  });
  wait_loads<P * Q>();                                       // tokens and scales are here, the codes may not be
  const int left = p.K - (S - 1) * kStepK;
  if (left < kStepK && (S - 1) % waves == wave) {            // what follows a token's row is not its
    for (int t = 0; t < p.T; ++t)
      if ((lane ^ t) * 8 >= left) *reinterpret_cast<uint4*>(s_mem + (t * S + S - 1) * 1024 + lane * 16) = make_uint4(0, 0, 0, 0);
    wait_lds();
  }
  barrier();

  f32x4 acc[Q];
#pragma unroll
  for (int m = 0; m < Q; ++m) acc[m] = f32x4{};
  // tokens past the last one repeat it; their sums are dropped
  const int trow = min(l4, p.T - 1);
  const uint8_t* const xr = s_mem + trow * S * 1024;
  uint32_t x_at[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) x_at[i] = (uint32_t)((b * 4 + i) ^ trow) * 16u;
  // zeros that the compiler does not know for constants: it would write them
  // anew before every chain of products
  f32x4 zero{};
  asm volatile("" : "+v"(zero));
  constexpr uint32_t kPer = FMT == MOE_QUANT_NVFP4 ? 2 : 1;  // scale bytes of a lane's step

  // a step's tokens and scales are read from LDS a step ahead
  uint4 xv[2][4];
  uint32_t sv[2][Q];
  auto read = [&](auto j_c, int s) {
    constexpr int J = decltype(j_c)::value & 1;
    s = min(s, S - 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) xv[J][i] = *reinterpret_cast<const uint4*>(xr + s * 1024 + x_at[i]);
    // the scales of the lane's row and block (past the row its last: times zero)
    const uint8_t* const sr = s_scale + min((uint32_t)(s * 16 + b) * kPer, scale_row - kPer) + l4 * scale_row;
#pragma unroll
    for (int m = 0; m < Q; ++m) {
      if constexpr (FMT == MOE_QUANT_NVFP4) sv[J][m] = *reinterpret_cast<const uint16_t*>(sr + m * scale_pad);
      else sv[J][m] = sr[m * scale_pad];
    }
  };
  auto body = [&](auto j_c, int s) {
    constexpr int J = decltype(j_c)::value, X = J & 1;
    read(std::integral_constant<int, J + 1>{}, s + 1);
#pragma unroll
    for (int m = 0; m < Q; ++m) {
      const uint4 c = wc[J][m];
      if constexpr (FMT == MOE_QUANT_NVFP4) {
        const float s0 = __builtin_amdgcn_cvt_f32_fp8((int)sv[X][m], 0), s1 = __builtin_amdgcn_cvt_f32_fp8((int)sv[X][m], 1);
        const f32x4 d0 = block16(c.x, c.y, xv[X][0], xv[X][1], 1.0f, zero);
        const f32x4 d1 = block16(c.z, c.w, xv[X][2], xv[X][3], 1.0f, zero);
#pragma unroll
        for (int t = 0; t < TT; ++t) acc[m][t] = fmaf(d1[t], s1, fmaf(d0[t], s0, acc[m][t]));
      } else {
        const float s0 = __uint_as_float(sv[X][m] << 23);
        acc[m] = block16(c.x, c.y, xv[X][0], xv[X][1], s0, acc[m]);
        acc[m] = block16(c.z, c.w, xv[X][2], xv[X][3], s0, acc[m]);
      }
    }
  };
  // the loads are issued past the last step too, so that every way through
  // the loop has as many in flight and the waits stay loose
  static_assert(P % 2 == 0, "LDS reads alternate");
  read(std::integral_constant<int, 0>{}, 0);
  for (int s = 0; s < S; s += P) {
    for_each<P>([&](auto j) {
      constexpr int J = decltype(j)::value;
      if (s + J < S) body(j, s + J);
      issue(j, s + J + P);
      fence();
    });
  }

  // the sums of the 16 blocks, in every lane of its row
#pragma unroll
  for (int m = 0; m < Q; ++m)
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      float v = acc[m][t];
      v = dpp_add<0x124>(v);                                 // row_ror:4
      v = dpp_add<0x128>(v);                                 // row_ror:8
      const auto h = __builtin_amdgcn_permlane16_swap(fbits(v), fbits(v), false, false);
      v = bitsf(h[0]) + bitsf(h[1]);
      const auto g = __builtin_amdgcn_permlane32_swap(fbits(v), fbits(v), false, false);
      acc[m][t] = bitsf(g[0]) + bitsf(g[1]);
    }
  // lane 4t + r writes token t of row r
  if (lane < 4 * p.T && l4 < rows) {
    float v[Q];
#pragma unroll
    for (int m = 0; m < Q; ++m) {
      v[m] = acc[m][0];
#pragma unroll
      for (int t = 1; t < TT; ++t) v[m] = b == t ? acc[m][t] : v[m];
    }
    write1<GU>(p, b, n0 + l4, v[0], v[Q - 1]);
  }
}

// LDS bytes of a workgroup: the tokens, and its waves' scales
uint32_t lds_bytes(int format, bool gate_up, int T, int K, int waves) {
  const uint32_t S = (uint32_t)(K + kStepK - 1) / kStepK;
  return (uint32_t)T * S * 1024u +
         (uint32_t)waves * (gate_up ? 2 : 1) * scale_bytes((uint32_t)(K / (format == MOE_QUANT_NVFP4 ? 16 : 32)));
}

template <int FMT, bool GU, int TT, int P>
moe_status launch(const DenseArgs& p, hipStream_t s) {
  const int waves = 4;
  const int tiles = (p.N + 4 * waves - 1) / (4 * waves);
  const int grid = tiles + (p.token_gate ? (p.T + waves - 1) / waves : 0);
  quant_few_kernel<FMT, GU, TT, P><<<(unsigned)grid, waves * kWave, lds_bytes(FMT, GU, p.T, p.K, waves), s>>>(p, tiles);
  return launch_status();
}

template <int FMT, bool GU, int TT>
moe_status dispatch_steps(const DenseArgs& p, hipStream_t s) {
  if (p.K <= 2 * kStepK) return launch<FMT, GU, TT, 2>(p, s);
  if (p.K <= 4 * kStepK || GU) return launch<FMT, GU, TT, 4>(p, s);
  return launch<FMT, GU, TT, 8>(p, s);
}

template <int FMT, bool GU>
moe_status dispatch(const DenseArgs& p, hipStream_t s) {
  if (p.T == 1) return dispatch_steps<FMT, GU, 1>(p, s);
  if (p.T == 2) return dispatch_steps<FMT, GU, 2>(p, s);
  return dispatch_steps<FMT, GU, 4>(p, s);
}

}  // namespace

bool quant_few_ok(int T, int K) { return T <= 4 && lds_bytes(MOE_QUANT_NVFP4, true, T, K, 4) <= 128 * 1024; }

moe_status quant_few(int format, bool gate_up, const DenseArgs& p, hipStream_t s) {
  if (format == MOE_QUANT_NVFP4)
    return gate_up ? dispatch<MOE_QUANT_NVFP4, true>(p, s) : dispatch<MOE_QUANT_NVFP4, false>(p, s);
  return gate_up ? dispatch<MOE_QUANT_MXFP4, true>(p, s) : dispatch<MOE_QUANT_MXFP4, false>(p, s);
}

}  // namespace moe
