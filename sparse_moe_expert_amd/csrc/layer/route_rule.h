// Grouped routing of one token by one wavefront.
//
// Selection in two steps.  The scores are first computed in fp32, and the
// experts (and groups) ordered by them; an order is taken where every gap that
// decides it is wider than twice the bound on the fp32 error, or separates
// experts of the same logit and bias (which tie exactly, and go by their ids).
// Else the token is ordered again by scores in fp64, as the rule defines them:
// a few tokens in a hundred with spread logits.  An fp32 score takes about 6
// instructions, an fp64 one 60, and 512 experts of them would set the time.
//
// The error bound, u = 2^-24.  Sigmoid: e^-z is off by (1.5 |z| + 2) u of
// itself (product and hardware exponential), the sum and the reciprocal by 3 u;
// s (1 - s) |z| <= 0.224, so s is off by less than 4 u.  Softmax: e^(z - max)
// by (2.5 |d| + 2) u with p |d| <= 0.37, so p by less than 3 u of its own, and
// every p of the token by the same factor of at most 45 u through the sum
// (sum of p |d| <= ln 1024, 22 additions).  The bias adds u |c|.
//
// Lanes: the 64 lanes are shared out over the groups (rounded up to a power of
// two), and a group's experts over its lanes, V at most to a lane, ids
// ascending with lane and place.
#pragma once

#include "select.h"

namespace moe {
namespace {

struct RouteRule {
  int T, E, k;
  int groups, kept, group_top;
  bool renormalise, softmax, bf16;
  float scale;
  int lanes, per_lane;       // of a group; a lane's experts (the last lanes may have fewer)
};

// Lanes of a group: 64 shared out over the groups, rounded up to a power of
// two; each lane holds at most kMaxPerLane of its group's experts.
constexpr int kMaxPerLane = 16;
inline int group_lanes(int groups) {
  int l = kWave;
  while (l > 1 && l * groups > kWave) l >>= 1;
  return l;
}

// A logit or bias at or below this, or NaN, masks its expert: -inf and the
// lowest finite value of fp32 and of bf16 (-3.39e38) alike.
constexpr float kLowest = -3.3e38f;
constexpr float kInf = __builtin_huge_valf();
constexpr float kLog2e = 1.4426950408889634f;

// Logit e of a row, masked ones as -inf, +inf as the largest float (so that a
// softmax over it is defined: such experts share all of the weight).
__device__ __forceinline__ float mask_logit(float z) { return z > kLowest ? fminf(z, 3.402823466e+38f) : -kInf; }

__device__ __forceinline__ float load_logit(const void* __restrict__ p, bool bf16, size_t i) {
  return mask_logit(bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16)
                         : static_cast<const float*>(p)[i]);
}

template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, ((uint64_t)dpp_u32<CTRL>((uint32_t)(u >> 32)) << 32) | dpp_u32<CTRL>((uint32_t)u));
}

// Sum over the wavefront: lane 0's, in every lane (the lanes add in different
// orders, and equal logits must give equal scores)
__device__ __forceinline__ double wave_sum_f64(double v) {
  v += dpp_f64<0xB1>(v);                       // quad_perm [1,0,3,2]
  v += dpp_f64<0x4E>(v);                       // quad_perm [2,3,0,1]
  v += dpp_f64<0x124>(v);                      // row_ror:4
  v += dpp_f64<0x128>(v);                      // row_ror:8
  v += __shfl_xor(v, 16, kWave);
  v += __shfl_xor(v, 32, kWave);
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(u >> 32)), lo = __builtin_amdgcn_readfirstlane((uint32_t)u);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

__device__ __forceinline__ float wave_max_f32(float v) { return from_ordered(wave_max_u32(ordered_bits(v))); }

// The keys of a lane, largest first (bitonic network; V a power of two)
template <int V>
__device__ __forceinline__ void sort_keys(uint64_t (&K)[V]) {
#pragma unroll
  for (int size = 2; size <= V; size <<= 1)
#pragma unroll
    for (int stride = size >> 1; stride > 0; stride >>= 1)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int j = i ^ stride;
        if (j > i) {
          const bool desc = (i & size) == 0;
          const uint64_t a = K[i], b = K[j];
          // one comparison an exchange: a mask the compiler does not see
          // through, and bitwise selects
          uint32_t m = (desc ? (b > a) : (a > b)) ? 0xFFFFFFFFu : 0u;
          asm("" : "+v"(m));
          const uint64_t m64 = ((uint64_t)m << 32) | m;
          K[i] = (b & m64) | (a & ~m64);
          K[j] = (a & m64) | (b & ~m64);
        }
      }
}

// Largest and second largest over a group's lanes, in every one of them
template <class F>
__device__ __forceinline__ void group_best(int lanes, F& a, F& b) {
  for (int o = 1; o < lanes; o <<= 1) {
    const F x = __shfl_xor(a, o, kWave), y = __shfl_xor(b, o, kWave);
    b = fmax(fmin(a, x), fmax(b, y));
    a = fmax(a, x);
  }
}

// A group's value from its two best; -inf where it has none
template <class F>
__device__ __forceinline__ F group_value(int top, F a, F b) {
  return top == 2 && b > -(F)kInf ? a + b : a;
}

// Whether the lane's group is among the `kept` of largest value `v`, lower
// groups first among equals
template <class F>
__device__ __forceinline__ bool group_kept(const RouteRule& r, int group, F v) {
  int before = 0;
  for (int g = 0; g < r.groups; ++g) {
    const F o = __shfl(v, g * r.lanes, kWave);
    before += o > v || (o == v && g < group);
  }
  return before < r.kept;
}

// The k chosen experts of token t by scores in fp64: slot j's in lane j.  Not
// inlined, and reads its logits again: the usual way keeps its registers.
template <int V>
__device__ __noinline__ int select_exact(RouteRule r, const void* logits, const float* bias, int t, float top, int lane,
                                         int group, int e0, int count) {
  const double kMasked = -__builtin_huge_val();
  double c[V];
  double sum = 0.0;
  float z[V], b[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    z[i] = i < count ? load_logit(logits, r.bf16, (size_t)t * r.E + e0 + i) : -kInf;
    b[i] = i < count && bias ? bias[e0 + i] : 0.0f;
    b[i] = b[i] > kLowest ? b[i] : -kInf;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    c[i] = 0.0;
    if (i < count && z[i] > -kInf) c[i] = r.softmax ? exp((double)z[i] - (double)top) : 1.0 / (1.0 + exp(-(double)z[i]));
    sum += c[i];
  }
  const double total = r.softmax ? wave_sum_f64(sum) : 1.0;
#pragma unroll
  for (int i = 0; i < V; ++i)
    c[i] = i < count && z[i] > -kInf && b[i] > -kInf ? c[i] / total + (double)b[i] : kMasked;
  double x = kMasked, y = kMasked;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    y = fmax(y, fmin(x, c[i]));
    x = fmax(x, c[i]);
  }
  group_best(r.lanes, x, y);
  const bool kept = group_kept(r, group, group_value(r.group_top, x, y));
  // the masked experts of the kept groups follow their others
  constexpr double kLast = -1e300, kTaken = -1e306;
#pragma unroll
  for (int i = 0; i < V; ++i) c[i] = kept && group < r.groups && i < count ? fmax(c[i], kLast) : kTaken;
  int mine = 0;
  for (int j = 0; j < r.k; ++j) {
    double best = kMasked;
    int at = 0;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (c[i] > best) {
        best = c[i];
        at = i;
      }
    int e = best > kTaken ? e0 + at : 1 << 20;
    for (int o = 1; o < kWave; o <<= 1) {
      const double ob = __shfl_xor(best, o, kWave);
      const int oe = __shfl_xor(e, o, kWave);
      if (ob > best || (ob == best && oe < e)) {
        best = ob;
        e = oe;
      }
    }
    if (lane == j) mine = e;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (e == e0 + i && i < count) c[i] = kTaken;
  }
  return mine;
}

// Token t: slot j's expert and weight in lane j.
template <int V>
__device__ __forceinline__ void select_grouped(const RouteRule& r, const void* __restrict__ logits,
                                               const float* __restrict__ bias, int t, int lane, int& my_e, float& my_w) {
  const int size = r.E / r.groups, group = lane / r.lanes, at = lane % r.lanes * r.per_lane;
  const int e0 = group * size + at;
  const int count = group < r.groups ? max(min(r.per_lane, size - at), 0) : 0;
  const size_t row = (size_t)t * r.E;
  float z[V], b[V];
#pragma unroll
  for (int i = 0; i < V; ++i) z[i] = -kInf, b[i] = 0.0f;
  bool wide = false;
  if constexpr (V >= 4) wide = r.per_lane == V && size % 4 == 0 && r.E % 4 == 0;       // every count is a multiple of 4
  if (wide) {
    if constexpr (V >= 4) {
#pragma unroll
      for (int i = 0; i < V; i += 4)
        if (i < count) {
          float4 v;
          if (r.bf16) {
            const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(logits) + row + e0 + i);
            v = make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                            __uint_as_float(u.y & 0xFFFF0000u));
          } else {
            v = *reinterpret_cast<const float4*>(static_cast<const float*>(logits) + row + e0 + i);
          }
          z[i] = v.x, z[i + 1] = v.y, z[i + 2] = v.z, z[i + 3] = v.w;
          if (bias) {
            const float4 w = *reinterpret_cast<const float4*>(bias + e0 + i);
            b[i] = w.x, b[i + 1] = w.y, b[i + 2] = w.z, b[i + 3] = w.w;
          }
        }
#pragma unroll
      for (int i = 0; i < V; ++i) z[i] = mask_logit(z[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < count) {
        z[i] = load_logit(logits, r.bf16, row + e0 + i);
        if (bias) b[i] = bias[e0 + i];
      }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) b[i] = b[i] > kLowest ? b[i] : -kInf;

  // fp32 scores
  float top = 0.0f, unit = 1.0f, s[V];
  if (r.softmax) {
    float m = -kInf;
#pragma unroll
    for (int i = 0; i < V; ++i) m = fmaxf(m, z[i]);
    top = wave_max_f32(m);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      s[i] = z[i] > -kInf ? __builtin_amdgcn_exp2f((z[i] - top) * kLog2e) : 0.0f;
      sum += s[i];
    }
    unit = __builtin_amdgcn_rcpf(wave_sum_f32(sum));         // the largest score; inf where all are masked
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] *= unit;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-z[i] * kLog2e));
  }
  // twice the bounds above, of values up to |c|
  const float tol0 = r.softmax ? 2.8e-6f * unit + 4e-7f : 5e-7f;
  auto tol = [&](float c) { return tol0 + 1.5e-7f * fabsf(c); };

  // keys: choice value, then the lower id; 1 for masked, 0 for absent experts
  uint64_t K[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const bool live = z[i] > -kInf && b[i] > -kInf;
    const uint32_t hi = i < count ? (live ? ordered_bits(s[i] + b[i]) : 1u) : 0u;
    K[i] = ((uint64_t)hi << 32) | (i < count ? kIdMask - (uint32_t)(e0 + i) : 0u);
  }
  sort_keys(K);
  auto value = [](uint64_t key) { return (uint32_t)(key >> 32) > 1u ? from_ordered((uint32_t)(key >> 32)) : -kInf; };

  bool doubt = false;                                        // wave-uniform
  if (r.kept < r.groups) {
    float x = value(K[0]), y = V > 1 ? value(K[V > 1 ? 1 : 0]) : -kInf;
    group_best(r.lanes, x, y);
    const float v = group_value(r.group_top, x, y);
    const bool in = group_kept(r, group, v);
    const bool real = group < r.groups;
    const float low = -wave_max_f32(real && in ? -v : -kInf), high = wave_max_f32(real && !in ? v : -kInf);
    // (groups with no expert left tie exactly)
    const float most = wave_max_f32(fmaxf(x > -kInf ? fabsf(x) : 0.0f, y > -kInf ? fabsf(y) : 0.0f));
    doubt = high > -kInf && !(low - high > 2.0f * tol(most) + 3e-7f * most);
    if (!in)
#pragma unroll
      for (int i = 0; i < V; ++i) K[i] = 0;
  }
  uint32_t my_key = 0;
  my_e = 0;
  for (int j = 0; j <= r.k; ++j) {                           // and the first that is not chosen
    uint32_t best;
    const int e = select_round<V>(K, lane, &best);
    if (lane == j) my_key = best, my_e = e;
  }
  // lane j: slot j against the next
  my_e = lane < r.k ? my_e : 0;
  float mz = load_logit(logits, r.bf16, row + my_e), mb = bias ? bias[my_e] : 0.0f;
  {
    const uint32_t next = __shfl_down(my_key, 1, kWave);
    const float nz = __shfl_down(mz, 1, kWave), nb = __shfl_down(mb, 1, kWave);
    const float c = from_ordered(my_key);
    const bool same = lane < r.k - 1 && mz == nz && mb == nb;
    const bool near = lane < r.k && next > 1u && !same && !(c - from_ordered(next) > tol(c));
    doubt = doubt || __any(near);
  }
  if (doubt) {
    my_e = select_exact<V>(r, logits, bias, t, top, lane, group, e0, count);
    my_e = lane < r.k ? my_e : 0;
    mz = load_logit(logits, r.bf16, row + my_e), mb = bias ? bias[my_e] : 0.0f;
  }

  // weights in fp64
  const bool live = lane < r.k && mz > -kInf && mb > kLowest;
  double w = 0.0;
  if (live) w = r.softmax ? exp((double)mz - (double)top) : 1.0 / (1.0 + exp(-(double)mz));
  double total = 1.0;
  if (r.renormalise) {
    total = wave_sum_f64(w);
  } else if (r.softmax) {
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (z[i] > -kInf) sum += exp((double)z[i] - (double)top);
    total = wave_sum_f64(sum);
  }
  w = total > 0.0 ? w / total : 0.0;
  my_w = (float)(w * (double)r.scale);
}

}  // namespace
}  // namespace moe
