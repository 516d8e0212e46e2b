// 4-bit products of one to sixteen tokens: bound by the weight bytes and, close
// behind, by the instructions that decode them.
//
// v_mfma_f32_4x4x4_16b_bf16 computes 16 independent 4 x 4 blocks: block b
// takes 4 tokens (A), 4 weight rows (B) and a part of the reduction of its
// own.  A lane's weights of a step are one 16-byte load, row l%4 and the 32
// reduction indices 32*(l/4)..: a wavefront reads 256 contiguous bytes of
// each of four rows, and eight instructions of 4 indices use them up.  For
// NVFP4 the codes enter without their scales (one conversion for two weights): the four
// instructions of a 16-weight scale block start from zero, and their results
// (a lane's: the tokens' of its own row) are scaled as they are added to the
// sums.  Decoding costs about half an instruction a weight instead of 2 for
// scaled weights, as the 16 x 16 tiles need them, and at four tokens a
// quarter of a dot product's.  MXFP4 scales are powers of two and part of the
// conversion.
//
// A wavefront owns four rows of a matrix and all of the reduction, with P
// steps of 512 in flight: no sum leaves the wavefront (but for a gate/up
// pair, whose second half of the waves hands its sums to the first), and
// nothing but the tokens, staged in LDS once for the workgroup's wavefronts,
// is waited for together.  The four rows' scales are contiguous and come to
// LDS as whole lines (a step's 32-byte pieces of the rows would be as many
// requests as the codes).
//
// Tokens in LDS: a kilobyte for a token's step, its 16-byte chunk c at c ^ t
// for token t, so that the reads of 16 lanes hit all banks.  Batches of more
// than 16 tokens are workgroups of 8 or 16 each, while the weights are so small
// that reading them again costs less than joining a split reduction.
//
// T = 1 4096x12288 shared expert (MXFP4, 80 MB): 16.6 to 16.8 us, 4.8 TB/s, as a
// large copy; T = 1 9999x4096 7.0 us (23 MB); T = 4 10240x2560 (MXFP4, 14 MB) 6.0 to
// 6.4 us, T = 1 2048x2048 3.2 us, of which 2.5 a launch.
#include "quant_common.h"

#include <type_traits>

namespace moe {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kStepK = 512;
constexpr int kFewTokens = 16;                               // at most, per workgroup
constexpr int kFewWaves = 16;                                // at most, per workgroup
// NVFP4 codes enter as 2^-7 of their value, exactly, and the sums leave by 2^7
// of theirs: 16 codes of 6 against the largest tokens would pass fp32's range
// before their scale, 2^-9 at least, is applied.
constexpr float kCodeUnit = 1.0f / 128;

template <int B>
__device__ __forceinline__ uint32_t fp4x2_bits(uint32_t word, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, scale, B));
}

__device__ __forceinline__ f32x4 mfma4(uint32_t a0, uint32_t a1, uint32_t b0, uint32_t b1, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(__builtin_bit_cast(s16x4, make_uint2(a0, a1)),
                                                __builtin_bit_cast(s16x4, make_uint2(b0, b1)), c, 0, 0, 0);
}

// 16 weights of the lane's row against 16 values of its token
__device__ __forceinline__ f32x4 block16(const uint32_t (&w)[8], const uint4 x0, const uint4 x1, f32x4 d) {
  d = mfma4(x0.x, x0.y, w[0], w[1], d);
  d = mfma4(x0.z, x0.w, w[2], w[3], d);
  d = mfma4(x1.x, x1.y, w[4], w[5], d);
  return mfma4(x1.z, x1.w, w[6], w[7], d);
}

// 16 weights (8 code bytes) as bf16, times a power of two
__device__ __forceinline__ void decode16(uint32_t c0, uint32_t c1, float scale, uint32_t (&w)[8]) {
  w[0] = fp4x2_bits<0>(c0, scale), w[1] = fp4x2_bits<1>(c0, scale);
  w[2] = fp4x2_bits<2>(c0, scale), w[3] = fp4x2_bits<3>(c0, scale);
  w[4] = fp4x2_bits<0>(c1, scale), w[5] = fp4x2_bits<1>(c1, scale);
  w[6] = fp4x2_bits<2>(c1, scale), w[7] = fp4x2_bits<3>(c1, scale);
}

// LDS bytes of the scales of four rows: whole kilobytes, as they are loaded
__host__ __device__ constexpr uint32_t scale_bytes(uint32_t scale_row) { return (4 * scale_row + 1023u) & ~1023u; }

// TT: tokens whose sums are kept (T or more)
template <int FMT, bool GU, int TT, int P>
__global__ __launch_bounds__(kFewWaves * kWave, 4) void quant_few_kernel(DenseArgs p, int row_tiles, int tiles) {
  constexpr int TG = TT < 4 ? 1 : TT / 4, TR = TT < 4 ? TT : 4;      // groups of tokens, and those of a group
  extern __shared__ __align__(16) uint8_t s_mem[];           // tokens, then the waves' scales
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = (int)blockDim.x / kWave;
  if (GU && (int)blockIdx.x >= tiles) {                      // token gates, one wave a token
    const int t = ((int)blockIdx.x - tiles) * waves + wave;
    if (t < p.T) token_gate_row(p, t, lane);
    return;
  }
  const int l4 = lane & 3, b = lane >> 2;
  const int quads = GU ? waves / 2 : waves, quad = GU && wave >= quads ? wave - quads : wave;
  const bool second = GU && wave >= quads;                   // of a pair's matrices
  const int n0 = ((int)blockIdx.x % row_tiles * quads + quad) * 4;     // past N: every load is out of range
  const int t0 = (int)blockIdx.x / row_tiles * TT, T = min(p.T - t0, TT);
  const int rows = max(min(4, p.N - n0), 0);
  const int S = (p.K + kStepK - 1) / kStepK;
  const uint32_t code_row = (uint32_t)p.K / 2, scale_row = (uint32_t)(p.K / kScaleGroup<FMT>);
  const uint32_t scale_pad = scale_bytes(scale_row);
  uint8_t* const s_scale = s_mem + T * S * 1024 + wave * scale_pad;

  // tokens: piece (t, s), a kilobyte each
  const auto rx = make_rsrc(p.x + (size_t)t0 * p.K, (uint32_t)T * (uint32_t)p.K * 2u);
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    if (t >= T) break;
    for (int s = wave; s < S; s += waves)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, s_mem + (t * S + s) * 1024, 16,
                                               (uint32_t)t * (uint32_t)p.K * 2u + (uint32_t)s * 1024u +
                                                   (uint32_t)(lane ^ t) * 16u, 0, 0, 0);
  }
  const QuantMat w = second ? p.b : p.a;
  const auto rc = make_rsrc(w.codes + (size_t)n0 * code_row, (uint32_t)rows * code_row);
  // (the range is checked a dword at a time; the last one may hold bytes
  // past the end, in the same aligned dword as bytes before it)
  const auto rs = make_rsrc(w.scales + (size_t)n0 * scale_row, ((uint32_t)rows * scale_row + 3u) & ~3u);
  for (uint32_t c = 0; c < scale_pad; c += 1024)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, s_scale + c, 16, c + (uint32_t)lane * 16u, 0, 0, 0);
  const uint32_t c_off = (uint32_t)l4 * code_row + (uint32_t)b * 16u;
  uint4 wc[P];
  // a step past the last one is issued out of range: it reads nothing
  auto issue = [&](auto j_c, int s) {
    constexpr int J = decltype(j_c)::value;
    const uint32_t at = c_off + (s < S ? (uint32_t)s * 256u : kOutside);
    wc[J] = to_uint4(__builtin_amdgcn_raw_buffer_load_b128(rc, at, 0, kStreamAux));
  };
  fence();
  for_each<P>([&](auto j) {
    issue(j, decltype(j)::value);
    fence();                                                 // in this order: the waits count on it
  });
  wait_loads<P>();                                       // tokens and scales are here, the codes may not be
  const int left = p.K - (S - 1) * kStepK;
  if (left < kStepK && (S - 1) % waves == wave) {            // what follows a token's row is not its
    for (int t = 0; t < T; ++t)
      if ((lane ^ t) * 8 >= left) *reinterpret_cast<uint4*>(s_mem + (t * S + S - 1) * 1024 + lane * 16) = make_uint4(0, 0, 0, 0);
    wait_lds();
  }
  barrier();

  f32x4 acc[TG];
#pragma unroll
  for (int g = 0; g < TG; ++g) acc[g] = f32x4{};
  // group g: token 4g + l%4; those past the last one repeat it, their sums are dropped
  constexpr uint32_t kPer = FMT == MOE_QUANT_NVFP4 ? 2 : 1;  // scale bytes of a lane's step
  // zeros that the compiler does not know for constants: it would write them
  // anew before every chain of products
  f32x4 zero{};
  asm volatile("" : "+v"(zero));
  uint4 xv[2][4];
  uint32_t sv[2];
  // a group's tokens are read from LDS a group ahead, a step's scales a step ahead
  auto read_tokens = [&](auto i_c, int s, int g) {
    constexpr int I = decltype(i_c)::value & 1;
    const int t = min(g * 4 + l4, T - 1);
    const uint8_t* const xr = s_mem + (t * S + min(s, S - 1)) * 1024;
#pragma unroll
    for (int i = 0; i < 4; ++i) xv[I][i] = *reinterpret_cast<const uint4*>(xr + (((b * 4 + i) ^ t) << 4));
  };
  auto read_scales = [&](auto j_c, int s) {
    constexpr int J = decltype(j_c)::value & 1;
    // the scales of the lane's row and block (past the row its last: times zero)
    const uint8_t* const sr = s_scale + min((uint32_t)(s * 16 + b) * kPer, scale_row - kPer) + l4 * scale_row;
    if constexpr (FMT == MOE_QUANT_NVFP4) sv[J] = *reinterpret_cast<const uint16_t*>(sr);
    else sv[J] = *sr;
  };
  auto body = [&](auto j_c, int s) {
    constexpr int J = decltype(j_c)::value;
    read_scales(std::integral_constant<int, J + 1>{}, s + 1);
    const uint4 c = wc[J];
    const uint32_t sb = sv[J & 1];
    float s0 = 1.0f, s1 = 1.0f;
    uint32_t w0[8], w1[8];
    if constexpr (FMT == MOE_QUANT_NVFP4) {
      s0 = __builtin_amdgcn_cvt_f32_fp8((int)sb, 0), s1 = __builtin_amdgcn_cvt_f32_fp8((int)sb, 1);
      decode16(c.x, c.y, kCodeUnit, w0);
      decode16(c.z, c.w, kCodeUnit, w1);
    } else {
      decode16(c.x, c.y, __uint_as_float(sb << 23), w0);
      decode16(c.z, c.w, __uint_as_float(sb << 23), w1);
    }
    for_each<TG>([&](auto g_c) {
      constexpr int g = decltype(g_c)::value, X = (J * TG + g) & 1;
      read_tokens(std::integral_constant<int, X + 1>{}, g + 1 < TG ? s : s + 1, (g + 1) % TG);
      if constexpr (FMT == MOE_QUANT_NVFP4) {
        const f32x4 d0 = block16(w0, xv[X][0], xv[X][1], zero), d1 = block16(w1, xv[X][2], xv[X][3], zero);
#pragma unroll
        for (int t = 0; t < TR; ++t) acc[g][t] = fmaf(d1[t], s1, fmaf(d0[t], s0, acc[g][t]));
      } else {
        acc[g] = block16(w0, xv[X][0], xv[X][1], acc[g]);
        acc[g] = block16(w1, xv[X][2], xv[X][3], acc[g]);
      }
    });
  };
  // the loads are issued past the last step too, so that every way through
  // the loop has as many in flight and the waits stay loose
  static_assert(P % 2 == 0, "LDS reads alternate");
  read_scales(std::integral_constant<int, 0>{}, 0);
  read_tokens(std::integral_constant<int, 0>{}, 0, 0);
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
  for (int g = 0; g < TG; ++g)
#pragma unroll
    for (int t = 0; t < TR; ++t) {
      float v = acc[g][t];
      v = dpp_add<0x124>(v);                                 // row_ror:4
      v = dpp_add<0x128>(v);                                 // row_ror:8
      const auto h = __builtin_amdgcn_permlane16_swap(fbits(v), fbits(v), false, false);
      v = bitsf(h[0]) + bitsf(h[1]);
      const auto q = __builtin_amdgcn_permlane32_swap(fbits(v), fbits(v), false, false);
      acc[g][t] = bitsf(q[0]) + bitsf(q[1]);
    }
  // lane 4t + r has token t of row r
  float v = acc[0][0], u = 0.0f;
#pragma unroll
  for (int t = 1; t < TT; ++t) v = b == t ? acc[t / 4][t % 4] : v;
  if constexpr (FMT == MOE_QUANT_NVFP4) v *= 1.0f / kCodeUnit;
  if constexpr (GU) {
    // the scales' place is free once every wave is done with its own
    __syncthreads();
    float* const hand = reinterpret_cast<float*>(s_mem + T * S * 1024) + quad * kWave + lane;
    if (second) *hand = v;
    __syncthreads();
    if (second) return;
    u = *hand;
  }
  if (b < T && l4 < rows) write1<GU>(p, t0 + b, n0 + l4, v, u);
}

// LDS bytes of a workgroup: the tokens, and its waves' scales
uint32_t lds_bytes(int group, int tokens, int K, int waves) {
  const uint32_t S = (uint32_t)(K + kStepK - 1) / kStepK;
  return (uint32_t)tokens * S * 1024u + (uint32_t)waves * scale_bytes((uint32_t)(K / group));
}

constexpr uint32_t kFewLds = 160 * 1024;

struct FewPlan {
  int tokens, waves;         // of a workgroup
  long long bytes;           // tokens and weights that the workgroups load
};

// Waves of a workgroup.  While the tokens take little LDS several workgroups
// share a compute unit, and small ones are best (T = 1 9999x4096: 7.3 us with
// 4 waves, 7.8 with 8 or 10).  Else more waves share one copy of the tokens,
// fewer spread over the 256 compute units more evenly (`bytes`: of the fullest
// of them, times 256).
FewPlan plan(bool gate_up, int tokens, int T, int N, int K) {
  const bool small = tokens * K * 2 <= 48 * 1024;
  FewPlan best{tokens, 0, 0};
  for (int w = 4; w <= (small ? 4 : kFewWaves); w += 2) {
    if (lds_bytes(16, tokens, K, w) > kFewLds) break;
    const int rows = gate_up ? 2 * w : 4 * w;
    long long wgs = (long long)((N + rows - 1) / rows) * ((T + tokens - 1) / tokens);
    if (!small) wgs = (wgs + 255) / 256 * 256;
    const long long bytes = wgs * (tokens * K * 2ll + w * 4ll * K * 9 / 16);
    if (!best.waves || bytes < best.bytes) best = {tokens, w, bytes};
  }
  return best;
}

// Above 8 tokens: tiles of 8 while they load little (T = 16 shared expert
// 2048x512: 7.9 us against 9.1 with 16 tokens a workgroup; T = 24 2560x640:
// 4.5 against 5.2; but T = 100 2048x2048, 83 MB: 11.3 against 9.3), else of 16.
constexpr long long kEightBytes = 40 * 1000 * 1000;

FewPlan plan(bool gate_up, int T, int N, int K) {
  if (T <= 8) return plan(gate_up, T, T, N, K);
  const FewPlan eight = plan(gate_up, 8, T, N, K);
  return eight.waves && eight.bytes <= kEightBytes ? eight : plan(gate_up, T < kFewTokens ? T : kFewTokens, T, N, K);
}

template <int FMT, bool GU, int TT, int P>
moe_status launch(const DenseArgs& p, const FewPlan& q, hipStream_t s) {
  const int waves = q.waves, rows = GU ? 2 * waves : 4 * waves;
  const int row_tiles = (p.N + rows - 1) / rows, tiles = row_tiles * ((p.T + TT - 1) / TT);
  const int grid = tiles + (GU && p.token_gate ? (p.T + waves - 1) / waves : 0);
  const uint32_t lds = lds_bytes(kScaleGroup<FMT>, q.tokens, p.K, waves);
  quant_few_kernel<FMT, GU, TT, P><<<(unsigned)grid, waves * kWave, lds, s>>>(p, row_tiles, tiles);
  return launch_status();
}

template <int FMT, bool GU, int TT>
moe_status dispatch_steps(const DenseArgs& p, const FewPlan& q, hipStream_t s) {
  // steps in flight: no more than there are, and than 128 registers hold
  if (p.K <= 2 * kStepK) return launch<FMT, GU, TT, 2>(p, q, s);
  if (p.K <= 4 * kStepK || TT > 8) return launch<FMT, GU, TT, 4>(p, q, s);
  return launch<FMT, GU, TT, (TT > 8 ? 4 : 8)>(p, q, s);
}

template <int FMT, bool GU>
moe_status dispatch(const DenseArgs& p, hipStream_t s) {
  const FewPlan q = plan(GU, p.T, p.N, p.K);
  if (q.tokens == 1) return dispatch_steps<FMT, GU, 1>(p, q, s);
  if (q.tokens == 2) return dispatch_steps<FMT, GU, 2>(p, q, s);
  if (q.tokens <= 4) return dispatch_steps<FMT, GU, 4>(p, q, s);
  if (q.tokens <= 8) return dispatch_steps<FMT, GU, 8>(p, q, s);
  return dispatch_steps<FMT, GU, 16>(p, q, s);
}

}  // namespace

// Above 16 tokens: while loading each token tile's copy of the weights and each
// row tile's of the tokens (mostly from L2) at kFewRate takes less than the
// split kernel should, which is kSplitMore (of a pair kSplitPairMore) slower to
// begin.
// 4096x4096, T = 32 (52 MB): 9.7 us against 10.5; T = 64 (70 MB): 14.6 against
// 12.4; 2048x2048, T = 64 (17 MB): 6.6 against 9.3; 8192x1024, T = 64 (86 MB):
// 12.1 against 7.2; 2560x640, T = 100 (33 MB): 8.3 against 6.5; shared expert
// 2048x4096, T = 32 (its pair 36 MB): 18.6 against 16.2; 4096x1024, T = 17 (36 MB): 12.0 against
// 14.9.  Past kFewBytes it
// never was the faster one.
// Whole shared experts, NVFP4, their pair by this kernel and by the split one:
// 2048x512 T = 64 9.4 and 12.5, T = 100 12.1 and 14.5, T = 150 14.6 and 15.1; 2560x640
// T = 64 14.2 and 16.5, T = 100 15.7 both (MXFP4 14.7 and 15.1); 4096x1024 T = 32 12.9
// and 14.4; 2048x2048 T = 32 11.9 and 12.0.  A pair's estimate is too low for its
// largest batches, the last before the rule changes over: 2560x640 T = 150 19.6 and
// 16.5, 2048x512 T = 200 17.3 and 15.4.
constexpr float kFewRate = 7e6f, kSplitMore = 1.0f, kSplitPairMore = 0.65f;      // bytes a us, us
constexpr long long kFewBytes = 60 * 1000 * 1000;

bool quant_few_ok(bool gate_up, int T, int N, int K) {
  const FewPlan q = plan(gate_up, T, N, K);
  if (!q.waves || T <= kFewTokens) return q.waves > 0;
  return q.bytes <= kFewBytes && (float)q.bytes <= kFewRate * (quant_split_us(gate_up, T, N, K) + (gate_up ? kSplitPairMore : kSplitMore));
}

moe_status quant_few(int format, bool gate_up, const DenseArgs& p, hipStream_t s) {
  if (format == MOE_QUANT_NVFP4)
    return gate_up ? dispatch<MOE_QUANT_NVFP4, true>(p, s) : dispatch<MOE_QUANT_NVFP4, false>(p, s);
  return gate_up ? dispatch<MOE_QUANT_MXFP4, true>(p, s) : dispatch<MOE_QUANT_MXFP4, false>(p, s);
}

}  // namespace moe
