// 4-bit dense weights: formats, their decoding, and the products' arguments.
//
// A weight is e2m1 code * block scale (* global scale).  NVFP4: an e4m3
// scale per 16 weights and one fp32 global scale; MXFP4: a power-of-two
// (e8m0, 2^(byte - 127)) scale per 32 weights.  Codes are packed two per
// byte, element 2i in the low nibble of byte i, rows along the reduction.
#pragma once

#include "row_dot.h"

#include <type_traits>

namespace moe {

// A 4-bit matrix [N, K]
struct QuantMat {
  const uint8_t* codes;
  const uint8_t* scales;
  const float* g;          // global scale, or null for 1
};

// y[t,n] = bf16( add[t,n] + gate[t] * (x_t . a_n + bias[n]) ), or for a
// gate/up pair y[t,n] = bf16( SiLU(x_t . a_n) * (x_t . b_n) ); a null bias,
// gate or add leaves its term out.  With `token_gate` a pair's launch also fills
// gate_out[t] = sigmoid(x_t . token_gate).
struct DenseArgs {
  const uint16_t* x;
  QuantMat a, b;
  const uint16_t* bias;
  const float* gate;
  const uint16_t* add;
  uint16_t* y;
  int T, N, K;
  const uint16_t* token_gate;
  float* gate_out;
};

// The products' kernels; `gate_up`: the pair a, b.  Arguments already checked.
// quant_few and quant_tile take what their _ok says, quant_split anything
// (with a workspace of quant_split_workspace bytes, in about quant_split_us
// beyond a launch).
size_t quant_split_workspace(bool gate_up, int T, int N, int K);
float quant_split_us(bool gate_up, int T, int N, int K);
moe_status quant_split(int format, bool gate_up, const DenseArgs& p, void* workspace, hipStream_t s);
bool quant_tile_ok(bool gate_up, int T, int N);
moe_status quant_tile(int format, bool gate_up, const DenseArgs& p, hipStream_t s);
bool quant_few_ok(bool gate_up, int T, int N, int K);
moe_status quant_few(int format, bool gate_up, const DenseArgs& p, hipStream_t s);

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// weights that share a scale
template <int FMT>
constexpr int kScaleGroup = FMT == MOE_QUANT_NVFP4 ? 16 : 32;

// Two e2m1 codes (byte B of `word`) times `scale`, as two bf16.  Exact: e2m1
// has 2 significant bits and e4m3 has 4, a bf16 holds 8.  The conversion's
// own scale operand takes powers of two only, which MXFP4's scales are.
template <int FMT, int B>
__device__ __forceinline__ uint32_t fp4x2_scaled(uint32_t word, float scale) {
  if constexpr (FMT == MOE_QUANT_MXFP4) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, scale, B));
  } else {
    const f32x2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, 1.0f, B);
    const bf16x2 r = {(__bf16)(v.x * scale), (__bf16)(v.y * scale)};
    return __builtin_bit_cast(uint32_t, r);
  }
}

// 8 weights (a dword of codes) -> a fragment.  sb: the scale bytes of their 32
// (two e4m3, or one e8m0); `second`: of the second 16.
template <int FMT>
__device__ __forceinline__ bf16x8 dequant8(uint32_t c, uint32_t sb, bool second) {
  float s;
  if constexpr (FMT == MOE_QUANT_NVFP4)
    s = second ? __builtin_amdgcn_cvt_f32_fp8((int)sb, 1) : __builtin_amdgcn_cvt_f32_fp8((int)sb, 0);
  else
    s = __uint_as_float(sb << 23);
  return __builtin_bit_cast(bf16x8, make_uint4(fp4x2_scaled<FMT, 0>(c, s), fp4x2_scaled<FMT, 1>(c, s),
                                               fp4x2_scaled<FMT, 2>(c, s), fp4x2_scaled<FMT, 3>(c, s)));
}

// 32 weights (16 code bytes and their scale bytes) -> four fragments
template <int FMT>
__device__ __forceinline__ void dequant32(const uint4 codes, uint32_t sb, bf16x8 (&fr)[4]) {
  const uint32_t c[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) fr[i] = dequant8<FMT>(c[i], sb, i >= 2);
}

__device__ __forceinline__ float bf16_to_f32(uint32_t bits) { return __uint_as_float(bits << 16); }

__device__ __forceinline__ float sigmoid(float v) { return 1.0f / (1.0f + __expf(-v)); }

// sigmoid(x_t . token_gate) of token t, by one wavefront
__device__ __forceinline__ void token_gate_row(const DenseArgs& p, int t, int lane) {
  float acc = 0.0f;
  const uint4* const xr = reinterpret_cast<const uint4*>(p.x + (size_t)t * p.K);
  const uint4* const vr = reinterpret_cast<const uint4*>(p.token_gate);
  for (int c = lane; c < p.K / 8; c += kWave) {
    const uint4 a = xr[c], b = vr[c];
    acc = __builtin_amdgcn_fdot2_f32_bf16(as_bf16x2(a.x), as_bf16x2(b.x), acc, false);
    acc = __builtin_amdgcn_fdot2_f32_bf16(as_bf16x2(a.y), as_bf16x2(b.y), acc, false);
    acc = __builtin_amdgcn_fdot2_f32_bf16(as_bf16x2(a.z), as_bf16x2(b.z), acc, false);
    acc = __builtin_amdgcn_fdot2_f32_bf16(as_bf16x2(a.w), as_bf16x2(b.w), acc, false);
  }
  acc = group_sum(acc, kWave);
  if (lane == 0) p.gate_out[t] = sigmoid(acc);
}

// One output from its sum (and for a gate/up pair the other's)
template <bool GU>
__device__ __forceinline__ void write1(const DenseArgs& p, int t, int n, float a, float b) {
  const size_t at = (size_t)t * p.N + n;
  a = p.a.g ? a * *p.a.g : a;
  if constexpr (GU) {
    b = p.b.g ? b * *p.b.g : b;
    a = silu(a) * b;
  } else {
    if (p.bias) a += bf16_to_f32(p.bias[n]);
    if (p.gate) a *= p.gate[t];
    if (p.add) a += bf16_to_f32(p.add[at]);
  }
  p.y[at] = (uint16_t)f32_to_bf16_rne(a);
}

// A matrix's global scale
__device__ __forceinline__ float global_scale(const QuantMat& w) { return w.g ? *w.g : 1.0f; }

// y[t, n .. n+3] from sums and the global scales; rows at or past N are left
// alone.  All loads come before the
// first store: the compiler moves none across it (T = 32 9999x4096: 12.6 us, 13.1
// output by output).
template <bool GU>
__device__ __forceinline__ void write4(const DenseArgs& p, int t, int n, f32x4 a, f32x4 b, float ga, float gb) {
  if (n >= p.N) return;
  const size_t at = (size_t)t * p.N;
  const float gate = !GU && p.gate ? p.gate[t] : 1.0f;
  uint32_t v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int c = min(n + j, p.N - 1);
    float o = a[j] * ga;
    if constexpr (GU) {
      o = silu(o) * (b[j] * gb);
    } else {
      if (p.bias) o += bf16_to_f32(p.bias[c]);
      o *= gate;
      if (p.add) o += bf16_to_f32(p.add[at + c]);
    }
    v[j] = f32_to_bf16_rne(o);
  }
  if (GU || p.N % 4 == 0) {                    // 8-byte aligned, and whole fours (a pair's N is a multiple of 32)
    *reinterpret_cast<uint2*>(p.y + at + n) = make_uint2(v[0] | (v[1] << 16), v[2] | (v[3] << 16));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (n + j < p.N) p.y[at + n + j] = (uint16_t)v[j];
  }
}

// y[t, n .. n+7] from sums (of a gate/up pair: from its outputs), N a
// multiple of 8, n < N
template <bool GU>
__device__ __forceinline__ void write8(const DenseArgs& p, int t, int n, f32x4 lo, f32x4 hi, float g) {
  float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  const size_t at = (size_t)t * p.N + n;
  if constexpr (!GU) {
    const float gate = p.gate ? p.gate[t] : 1.0f;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const uint4 bias = p.bias ? *reinterpret_cast<const uint4*>(p.bias + n) : zero;
    const uint4 add = p.add ? *reinterpret_cast<const uint4*>(p.add + at) : zero;
    const uint32_t b[4] = {bias.x, bias.y, bias.z, bias.w}, d[4] = {add.x, add.y, add.z, add.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int sh = i % 2 * 16;
      if (p.bias) v[i] = v[i] * g + bf16_to_f32(b[i / 2] >> sh & 0xFFFFu);
      else v[i] *= g;
      v[i] *= gate;
      if (p.add) v[i] += bf16_to_f32(d[i / 2] >> sh & 0xFFFFu);
    }
  }
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = f32_to_bf16_rne(v[2 * i]) | (f32_to_bf16_rne(v[2 * i + 1]) << 16);
  *reinterpret_cast<uint4*>(p.y + at) = make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void fence() { asm volatile("" ::: "memory"); }

template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// s_waitcnt vmcnt(N), and as the compiler's own, which then does not wait
// for what came before once more
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N < 64, "six bits");
  fence();
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0F70);
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

// Workgroup barrier without the fence of __syncthreads(), which would wait
// for every load in flight.
__device__ __forceinline__ void barrier() {
  fence();
  __builtin_amdgcn_s_barrier();
  fence();
}

// A buffer offset beyond every resource of these kernels
constexpr uint32_t kOutside = 0x60000000u;

__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

}  // namespace

// Argument checks shared by the 4-bit products
inline bool quant_format_ok(int f) { return f == MOE_QUANT_NVFP4 || f == MOE_QUANT_MXFP4; }
inline bool quant_dims_ok(int n, int k) { return n >= 1 && k >= 32 && k % 32 == 0; }
constexpr int kQuantMaxK = 1 << 15;
inline bool quant_dims_fit(int n, int k) { return n <= (1 << 20) && k <= kQuantMaxK; }
constexpr int kQuantMaxTokens = 1 << 20;
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace moe
