// Tokens in 8 bits: moe_norm_quantize and moe_block_quantize.
//
//   r = round(x + residual)                  (the residual's type)
//   y = r / sqrt(mean(r^2) + eps) * (weight + offset)
//   s_b = max(amax_b |y| / 448, 2^-126),  q = e4m3(y / s_b)   for each 128 of y
//
// Bound by memory: a row is read once, kept in registers as fp32, and written
// once in each form.  A thread holds 8 neighbouring values, so that 16 lanes, a
// row of the cross-lane network, hold a block of 128.  The sum of squares is
// fp64: squares of large values leave fp32, and with the row in registers it
// costs less than the loads it runs beside.  (T = 4096 2560, an fp32 residual:
// 25.5 us, 5.4 TB/s; T = 8192 4096 encoded: 18.6 us, 5.5 TB/s.  A large copy
// reaches 5.2.)
#include "block_common.h"

namespace moe {
namespace {

constexpr int kNormThreads = 256;

struct NormArgs {
  const uint16_t* x;
  const void* residual;
  const uint16_t* weight;
  void* residual_out;
  uint16_t* y;
  uint8_t* q;
  float* scale;
  float offset, eps;
  int T, H;
};

__device__ __forceinline__ void unpack8(const uint4 u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_to_f32(w[i] & 0xFFFFu);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(to_bf16(v[0]) | to_bf16(v[1]) << 16, to_bf16(v[2]) | to_bf16(v[3]) << 16,
                    to_bf16(v[4]) | to_bf16(v[5]) << 16, to_bf16(v[6]) | to_bf16(v[7]) << 16);
}

// Eight values of a block that 16 lanes hold (those past the row: zero) to
// codes at q and, from its first lane, the scale
__device__ __forceinline__ void encode8(float (&v)[8], bool here, uint8_t* q, float* scale) {
  const float s = block_scale(__uint_as_float(max16(largest(v))));
  if (!here) return;
  float lifted = s;
  if (__builtin_expect(__any(s < 0x1p-90f), 0)) {
    const float lift = lift_of(s);
    lifted = s * lift;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= lift;
  }
  const Divisor d{lifted, 1.0f / lifted};
  *reinterpret_cast<uint2*>(q) = make_uint2(encode4(v[0], v[1], v[2], v[3], d), encode4(v[4], v[5], v[6], v[7], d));
  if ((threadIdx.x & 15) == 0) *scale = s;
}

// STREAM: 0 no residual, 1 bf16, 2 fp32.  CPT: pieces of 8 values a thread.
template <int STREAM, int CPT>
__global__ __launch_bounds__(kNormThreads) void norm_kernel(NormArgs p) {
  __shared__ double s_sum[kNormThreads / kWave];
  const int t = blockIdx.x, tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid >> 6;
  const size_t row = (size_t)t * p.H;
  float r[CPT][8];
  double sum = 0.0;
#pragma unroll
  for (int c = 0; c < CPT; ++c) {
    const int at = (c * kNormThreads + tid) * 8;
    if (at < p.H) {
      unpack8(*reinterpret_cast<const uint4*>(p.x + row + at), r[c]);
      if constexpr (STREAM == 1) {
        float b[8];
        unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.residual) + row + at), b);
#pragma unroll
        for (int i = 0; i < 8; ++i) r[c][i] += b[i];
        const uint4 w = pack8(r[c]);
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.residual_out) + row + at) = w;
        unpack8(w, r[c]);
      } else if constexpr (STREAM == 2) {
        const float4* const b = reinterpret_cast<const float4*>(static_cast<const float*>(p.residual) + row + at);
        const float4 lo = b[0], hi = b[1];
        const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) r[c][i] += v[i];
        float4* const o = reinterpret_cast<float4*>(static_cast<float*>(p.residual_out) + row + at);
        o[0] = make_float4(r[c][0], r[c][1], r[c][2], r[c][3]);
        o[1] = make_float4(r[c][4], r[c][5], r[c][6], r[c][7]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) r[c][i] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fma((double)r[c][i], (double)r[c][i], sum);
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off, kWave);
  if (lane == 0) s_sum[wave] = sum;
  __syncthreads();
  sum = 0.0;
#pragma unroll
  for (int w = 0; w < kNormThreads / kWave; ++w) sum += s_sum[w];
  const float inv = (float)(1.0 / sqrt(sum / p.H + (double)p.eps));
  const int kb = blocks_of(p.H);
#pragma unroll
  for (int c = 0; c < CPT; ++c) {
    const int at = (c * kNormThreads + tid) * 8;
    const bool here = at < p.H;
    if (here) {
      float w[8];
      unpack8(*reinterpret_cast<const uint4*>(p.weight + at), w);
#pragma unroll
      for (int i = 0; i < 8; ++i) r[c][i] = r[c][i] * inv * (w[i] + p.offset);
      if (p.y) *reinterpret_cast<uint4*>(p.y + row + at) = pack8(r[c]);
    }
    encode8(r[c], here, p.q + row + at, p.scale + (size_t)t * kb + at / kBlock);
  }
}

// A thread to 8 values, 16 neighbouring threads to a block.  The largest batch has
// 2^32 threads, which no row of workgroups can have: two rows of them then.
constexpr size_t kGroupsRow = 1 << 23;

__global__ __launch_bounds__(kNormThreads) void quantize_kernel(const uint16_t* __restrict__ x, uint8_t* __restrict__ q,
                                                                float* __restrict__ scale, int K, int kb, size_t blocks) {
  const size_t block = (blockIdx.y * kGroupsRow + blockIdx.x) * (kNormThreads / 16) + (threadIdx.x >> 4);
  if (block >= blocks) return;               // all 16 lanes of a block alike
  const size_t t = block / (size_t)kb;
  const int at = (int)(block - t * (size_t)kb) * kBlock + (threadIdx.x & 15) * 8;
  float v[8] = {};
  const bool here = at < K;
  if (here) unpack8(*reinterpret_cast<const uint4*>(x + t * (size_t)K + at), v);
  encode8(v, here, q + t * (size_t)K + at, scale + block);
}

template <int STREAM>
moe_status launch_norm(const NormArgs& p, hipStream_t s) {
  const int chunks = (p.H / 8 + kNormThreads - 1) / kNormThreads;
  const unsigned grid = (unsigned)p.T;
  if (chunks <= 1) norm_kernel<STREAM, 1><<<grid, kNormThreads, 0, s>>>(p);
  else if (chunks <= 2) norm_kernel<STREAM, 2><<<grid, kNormThreads, 0, s>>>(p);
  else if (chunks <= 4) norm_kernel<STREAM, 4><<<grid, kNormThreads, 0, s>>>(p);
  else if (chunks <= 8) norm_kernel<STREAM, 8><<<grid, kNormThreads, 0, s>>>(p);
  else norm_kernel<STREAM, 16><<<grid, kNormThreads, 0, s>>>(p);
  return launch_status();
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_norm_quantize(const uint16_t* x, const void* residual, int residual_type,
                                        const uint16_t* weight, float weight_offset, float eps, int T, int H,
                                        void* residual_out, uint16_t* y, uint8_t* q, float* scale, void* stream) {
  using namespace moe;
  if (T < 0 || H < 16 || H % 16 != 0 || (residual_type != MOE_DTYPE_F32 && residual_type != MOE_DTYPE_BF16) ||
      !(eps >= 1e-30f && eps <= 3e38f) || !(weight_offset >= -3e38f && weight_offset <= 3e38f))
    return MOE_ERR_INVALID_SHAPE;
  if (H > kBlockMaxK || T > kBlockMaxTokens) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!x || !weight || !q || !scale || (residual == nullptr) != (residual_out == nullptr)) return MOE_ERR_NULL_POINTER;
  const void* const all[] = {x, residual, weight, residual_out, y, q, scale};
  for (const void* a : all)
    if (!aligned16(a)) return MOE_ERR_MISALIGNED;
  const NormArgs p{x, residual, weight, residual_out, y, q, scale, weight_offset, eps, T, H};
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (!residual) return launch_norm<0>(p, s);
  return residual_type == MOE_DTYPE_BF16 ? launch_norm<1>(p, s) : launch_norm<2>(p, s);
}

extern "C" moe_status moe_block_quantize(const uint16_t* x, int T, int K, uint8_t* q, float* scale, void* stream) {
  using namespace moe;
  if (T < 0 || K < 16 || K % 16 != 0) return MOE_ERR_INVALID_SHAPE;
  if (K > kBlockMaxK || T > kBlockMaxTokens) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!x || !q || !scale) return MOE_ERR_NULL_POINTER;
  if (!aligned16(x) || !aligned16(q) || !aligned16(scale)) return MOE_ERR_MISALIGNED;
  const int kb = blocks_of(K);
  const size_t blocks = (size_t)T * (size_t)kb;              // at most 2^28
  const size_t groups = (blocks + kNormThreads / 16 - 1) / (kNormThreads / 16);
  const dim3 grid((unsigned)(groups < kGroupsRow ? groups : kGroupsRow), (unsigned)((groups + kGroupsRow - 1) / kGroupsRow));
  quantize_kernel<<<grid, kNormThreads, 0, static_cast<hipStream_t>(stream)>>>(x, q, scale, K, kb, blocks);
  return launch_status();
}
