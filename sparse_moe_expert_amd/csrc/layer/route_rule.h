// Grouped routing of one token by one wavefront.
//
// Selection in two steps.  The scores are first computed in fp32, and the
// experts (and groups) ordered by them; an order is taken where every gap that
// decides it is wider than twice the bound on the fp32 error, or separates
// experts of the same logit and bias (which tie exactly, and go by their ids).
// Else the first k and a few more, one to a lane, are ordered by scores in
// fp64, as the rule defines them; and where those few do not reach past the
// doubt, all experts are.  Groups in doubt are settled first, by all scores in
// fp64 (4096 tokens of 512 experts with such a token among them: 22 us; 30 where
// it then took the experts by those too).  A few tokens in a hundred with
// spread logits take the second way, hardly any the last.  An fp32 score takes
// about 6 instructions, an fp64 one 60, and 512 experts of them would set the
// time.
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
  bool renormalise, softmax;
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

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* __restrict__ p, size_t i) {
  if constexpr (BF16) return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
  else return static_cast<const float*>(p)[i];
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

__device__ __forceinline__ float read_lane(float v, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}
__device__ __forceinline__ double read_lane(double v, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(u >> 32), lane), lo = __builtin_amdgcn_readlane((uint32_t)u, lane);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

template <int CTRL>
__device__ __forceinline__ float dpp_move(float v) {
  return __builtin_bit_cast(float, dpp_u32<CTRL>(__builtin_bit_cast(uint32_t, v)));
}
template <int CTRL>
__device__ __forceinline__ double dpp_move(double v) { return dpp_f64<CTRL>(v); }

// Largest and second largest over a group's lanes (a power of two of them), in
// every one of them.  Once the lanes of a half agree, a mirrored lane is as
// good as the one opposite.
template <class F>
__device__ __forceinline__ void group_best(int lanes, F& a, F& b) {
  auto merge = [&](F x, F y) {
    b = fmax(fmin(a, x), fmax(b, y));
    a = fmax(a, x);
  };
  if (lanes > 1) merge(dpp_move<0xB1>(a), dpp_move<0xB1>(b));          // quad_perm [1,0,3,2]
  if (lanes > 2) merge(dpp_move<0x4E>(a), dpp_move<0x4E>(b));          // quad_perm [2,3,0,1]
  if (lanes > 4) merge(dpp_move<0x141>(a), dpp_move<0x141>(b));        // row_half_mirror
  if (lanes > 8) merge(dpp_move<0x140>(a), dpp_move<0x140>(b));        // row_mirror
  if (lanes > 16) merge(__shfl_xor(a, 16, kWave), __shfl_xor(b, 16, kWave));
  if (lanes > 32) merge(__shfl_xor(a, 32, kWave), __shfl_xor(b, 32, kWave));
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
    const F o = read_lane(v, g * r.lanes);
    before += o > v || (o == v && g < group);
  }
  return before < r.kept;
}

// The choice values of a lane's experts in fp64 (masked ones -inf), and whether
// its group is kept by them.  Reads its logits again: the usual way keeps its
// registers.
template <int V, bool BF16>
__device__ __forceinline__ bool kept_exact(const RouteRule& r, const void* logits, const float* bias, int t, float top,
                                           int group, int e0, int count, double (&c)[V]) {
  const double kMasked = -__builtin_huge_val();
  double sum = 0.0;
  float z[V], b[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    z[i] = i < count ? mask_logit(load_logit<BF16>(logits, (size_t)t * r.E + e0 + i)) : -kInf;
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
  return group_kept(r, group, group_value(r.group_top, x, y));
}

// The k chosen experts of token t by scores in fp64: slot j's in lane j
template <int V, bool BF16>
__device__ __forceinline__ int select_exact(const RouteRule& r, const void* logits, const float* bias, int t, float top, int lane,
                                            int group, int e0, int count) {
  const double kMasked = -__builtin_huge_val();
  double c[V];
  const bool kept = kept_exact<V, BF16>(r, logits, bias, t, top, group, e0, count, c);
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

// Token t: slot j's expert and weight in lane j.  s_row: 2E floats of LDS, the
// wavefront's own.
template <int V, bool BF16>
__device__ __forceinline__ void select_grouped(const RouteRule& r, const void* __restrict__ logits,
                                               const float* __restrict__ bias, int t, int lane, float* s_row, int& my_e,
                                               float& my_w) {
  const int size = r.E / r.groups, group = lane / r.lanes, at = lane % r.lanes * r.per_lane;
  const int e0 = group * size + at;
  const int count = group < r.groups ? max(min(r.per_lane, size - at), 0) : 0;
  const size_t row = (size_t)t * r.E;
  float z[V], b[V];
  bool wide = false;
  if constexpr (V >= 4) wide = r.per_lane == V && size % 4 == 0;        // every count and row start a multiple of 4
  if (wide) {
    if constexpr (V >= 4) {
#pragma unroll
      for (int i = 0; i < V; i += 4) {                       // (past the lane's experts: any four, not used)
        const int e = min(e0 + i, r.E - 4);
        if constexpr (BF16) {
          const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(logits) + row + e);
          z[i] = __uint_as_float(u.x << 16), z[i + 1] = __uint_as_float(u.x & 0xFFFF0000u);
          z[i + 2] = __uint_as_float(u.y << 16), z[i + 3] = __uint_as_float(u.y & 0xFFFF0000u);
        } else {
          const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(logits) + row + e);
          z[i] = v.x, z[i + 1] = v.y, z[i + 2] = v.z, z[i + 3] = v.w;
        }
        const float4 w = bias ? *reinterpret_cast<const float4*>(bias + e) : make_float4(0, 0, 0, 0);
        b[i] = w.x, b[i + 1] = w.y, b[i + 2] = w.z, b[i + 3] = w.w;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = min(e0 + i, r.E - 1);
      z[i] = load_logit<BF16>(logits, row + e);
      b[i] = bias ? bias[e] : 0.0f;
    }
  }
  float* const s_z = s_row;
  float* const s_b = s_row + r.E;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    z[i] = i < count ? mask_logit(z[i]) : -kInf;
    b[i] = b[i] > kLowest ? b[i] : -kInf;
    if (i < count) s_z[e0 + i] = z[i], s_b[e0 + i] = b[i];
  }

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

  if (r.kept < r.groups) {
    float x = value(K[0]), y = V > 1 ? value(K[V > 1 ? 1 : 0]) : -kInf;
    group_best(r.lanes, x, y);
    const float v = group_value(r.group_top, x, y);
    bool in = group_kept(r, group, v);
    const bool real = group < r.groups;
    const float low = -wave_max_f32(real && in ? -v : -kInf), high = wave_max_f32(real && !in ? v : -kInf);
    // (groups with no expert left tie exactly; the sum of two finite values beyond
    // half the largest float is infinite here and not in fp64)
    const bool outside = x > -kInf && x < kInf && !(fabsf(v) < kInf);
    const float most = wave_max_f32(fmaxf(x > -kInf ? fabsf(x) : 0.0f, y > -kInf ? fabsf(y) : 0.0f));
    if (__any(outside) || (high > -kInf && !(low - high > 2.0f * tol(most) + 3e-7f * most))) {
      double exact[V];
      in = kept_exact<V, BF16>(r, logits, bias, t, top, group, e0, count, exact);
    }
    if (!in)
#pragma unroll
      for (int i = 0; i < V; ++i) K[i] = 0;
  }
  uint32_t my_key = 0;
  int n = 0;                                                 // slots filled: k, and two to five more
  my_e = 0;
  for (; n < r.k + 2; n += 4) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t best;
      const int e = select_round<V>(K, lane, &best);
      if (lane == n + j) my_key = best, my_e = e;
    }
  }
  my_e = my_key > 0u ? my_e : 0;                             // (no expert left)
  float mz = s_z[my_e], mb = s_b[my_e];
  // lane j: slot j against the next
  bool doubt;                                                // wave-uniform
  const float c = from_ordered(my_key);
  {
    const uint32_t next = __shfl_down(my_key, 1, kWave);
    const float nz = __shfl_down(mz, 1, kWave), nb = __shfl_down(mb, 1, kWave);
    const bool same = lane < r.k - 1 && mz == nz && mb == nb;
    const bool near = lane < r.k && next > 1u && !same && !(c - from_ordered(next) > tol(c));
    doubt = __any(near);
  }
  const bool need_total = r.softmax && (doubt || !r.renormalise);
  double total = 1.0;
  if (need_total) {
    double sum = 0.0;
#pragma unroll 1
    for (int i = 0; i < count; ++i) {
      const float x = s_z[e0 + i];
      if (x > -kInf) sum += exp((double)x - (double)top);
    }
    total = wave_sum_f64(sum);
  }
  auto score = [&](float x) {
    if (!(x > -kInf)) return 0.0;
    return r.softmax ? exp((double)x - (double)top) : 1.0 / (1.0 + exp(-(double)x));
  };
  double w = score(mz);
  if (doubt) {
    const float cut = read_lane(c, r.k - 1), last = read_lane(c, n - 1);
    const bool past = __builtin_amdgcn_readlane(my_key, n - 1) <= 1u || cut - last > tol(cut);
    if (past) {
      // masked ones after all others, lanes without an expert last
      const bool live = my_key > 1u;
      double v = live ? w / total + (double)mb : my_key == 1u ? -1e300 : -1e306;
      const int id = my_key > 0u ? my_e : r.E + lane;
      int rank = 0;
      for (int i = 0; i < n; ++i) {
        const double o = read_lane(v, i);
        rank += o > v || (o == v && __builtin_amdgcn_readlane(id, i) < id);
      }
      const int to = (lane < n ? rank : lane) * 4;
      my_e = __builtin_amdgcn_ds_permute(to, my_e);
      my_e = lane < r.k ? my_e : 0;
    } else {
      my_e = select_exact<V, BF16>(r, logits, bias, t, top, lane, group, e0, count);
      my_e = lane < r.k ? my_e : 0;
    }
    mz = s_z[my_e], mb = s_b[my_e];
    w = score(mz);
  }

  // weights in fp64
  w = lane < r.k && mb > -kInf ? w : 0.0;
  if (r.renormalise) total = wave_sum_f64(w);
  w = total > 0.0 ? w / total : 0.0;
  my_w = (float)(w * (double)r.scale);
}

}  // namespace
}  // namespace moe
