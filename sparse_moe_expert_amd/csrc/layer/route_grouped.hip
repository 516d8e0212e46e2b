// Grouped routing: moe_route_grouped and moe_route_grouped_bucket.
//
// Per token, with z the logits and b the balance bias,
//   s_e = sigmoid(z_e)  or  exp(z_e - max z) / sum_i exp(z_i - max z),
//   c_e = s_e + b_e                        (the selection's value; not the weight's)
//   G_g = sum of the group_top largest c of group g (its unmasked experts),
//   the groups_kept groups of largest G, in them the k experts of largest c,
//   w_j = scale * s_j  (/ sum_i s_i over the chosen, where renormalised).
// Equal values go to the lower id, of groups and of experts.  The choice is
// that of scores and choice values in 64 bits (sums s + b of different experts
// often agree to 32 bits, and which expert is taken would hang on the last bit
// of an exponential); route_rule.h has how fp32 decides most of it.
//
// Bound by latency: one token of 256 experts takes 6 us, of which 2.5 are the
// launch, to read a kilobyte; 4096 tokens of 512 experts 20 to 21 us (the bytes
// take 1.8 at the rate of a copy), of which a tracer gives the selection 14 to 15
// and the buckets 8: a sort of each lane's experts and k + 2 rounds over the
// wavefront a token, also of experts whose group is dropped, and 40 workgroups
// that each count all 40960 routes.
//
// A few tokens: one workgroup selects (a wavefront a token) and buckets; a
// larger batch selects over the chip, then buckets in a workgroup for each
// 1024 routes, which counts all routes' experts itself (all of them, and those
// before its own: no hand-off between workgroups).  From 2^17 routes that
// counting would take longer than counting once, in the place of an output
// that is not written yet.
#include "moe_common.h"
#include "route_rule.h"
#include "row_dot.h"

#include <type_traits>

namespace moe {
namespace {

constexpr int kRouteWaves = 4;                 // tokens of a selecting workgroup
// One workgroup, with its waves four to a SIMD, while they have little to do:
// T = 16, E = 256: 9.4 us, 9.6 by two launches; E = 512: 12.4 and 10.6; T = 8,
// E = 512: 8.7 and 10.5.
constexpr int kSmallTokens = 16, kSmallScores = 12 * 512;
constexpr int kBkThreads = 1024, kBkWaves = kBkThreads / kWave;
constexpr int kMaxExperts = 1024;

struct BucketOut {
  int32_t* count;
  int32_t* offset;
  int32_t* active;
  int32_t* n_active;
  int32_t* src;
  int32_t* pos;
};

template <int V, bool BF16>
__global__ __launch_bounds__(kRouteWaves* kWave) void route_grouped_kernel(RouteRule r, const void* __restrict__ logits,
                                                                           const float* __restrict__ bias,
                                                                           int32_t* __restrict__ topk_idx,
                                                                           float* __restrict__ topk_w) {
  extern __shared__ __align__(16) float s_rows[];            // 2E a wave
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = (int)blockIdx.x * kRouteWaves + wave;
  if (t >= r.T) return;
  int e;
  float w;
  select_grouped<V, BF16>(r, logits, bias, t, lane, s_rows + wave * 2 * r.E, e, w);
  if (lane < r.k) {
    topk_idx[(size_t)t * r.k + lane] = e;
    topk_w[(size_t)t * r.k + lane] = w;
  }
}

// Offsets and the active list from the counts s_cnt[E] in LDS, which become the
// offsets; `write`: to global memory too.  s_wave: a pair a wave.
__device__ __forceinline__ void offsets_block(int* s_cnt, int2* s_wave, int E, int threads, bool write, const BucketOut& o) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x >> 6, waves = threads / kWave;
  const int per = (E + threads - 1) / threads, e0 = (int)threadIdx.x * per;
  int routes = 0, actives = 0;
  for (int e = e0; e < min(e0 + per, E); ++e) {
    routes += s_cnt[e];
    actives += s_cnt[e] > 0;
  }
  int off = wave_inclusive_scan(routes), apos = wave_inclusive_scan(actives);
  if (lane == kWave - 1) s_wave[wave] = make_int2(off, apos);
  off -= routes;
  apos -= actives;
  __syncthreads();
  int all = 0, all_active = 0;
#pragma unroll
  for (int w = 0; w < kBkWaves; ++w) {                       // (all read at once; absent waves' are not used)
    const int2 x = s_wave[w];
    off += w < wave ? x.x : 0;
    apos += w < wave ? x.y : 0;
    all += w < waves ? x.x : 0;
    all_active += w < waves ? x.y : 0;
  }
  for (int e = e0; e < min(e0 + per, E); ++e) {
    const int c = s_cnt[e];
    s_cnt[e] = off;
    if (write) {
      o.count[e] = c;
      o.offset[e] = off;
      if (c > 0) o.active[apos] = e;
      if (e >= all_active) o.active[e] = -1;
    }
    off += c;
    apos += c > 0;
  }
  if (write && threadIdx.x == 0) {
    o.offset[E] = all;
    *o.n_active = all_active;
  }
  __syncthreads();
}

// Lanes of the wave with the same expert as this one
__device__ __forceinline__ uint64_t same_expert(int e, bool valid) {
  uint64_t same = __ballot(valid);
#pragma unroll
  for (int b = 0; b < 10; ++b) {                             // ids are below 1024
    const bool bit = (e >> b) & 1;
    const uint64_t have = __ballot(bit);
    same &= bit ? have : ~have;
  }
  return same;
}

// Positions of the routes r0 .. r0 + threads: the base of the expert (its
// offset, and its routes before r0), and its routes before this one in the
// workgroup.  s_wcnt: a row of E bytes a wave that has routes, zero.
template <int WAVES>
__device__ __forceinline__ void place_block(const int* s_base, uint8_t (*s_wcnt)[kMaxExperts], int r, bool valid, int e,
                                            const BucketOut& o) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x >> 6;
  const uint64_t same = same_expert(e, valid);
  int rank = __popcll(same & ((1ull << lane) - 1ull));
  if (valid && rank == 0) s_wcnt[wave][e] = (uint8_t)__popcll(same);
  __syncthreads();
  if (valid) {
#pragma unroll
    for (int w = 0; w < WAVES; ++w) rank += w < wave ? s_wcnt[w][e] : 0;
    const int pos = s_base[e] + rank;
    o.src[pos] = r;
    o.pos[r] = pos;
  }
}

// `bytes` a multiple of 16, as is p
__device__ __forceinline__ void clear(void* p, int bytes, int threads) {
  for (int i = threadIdx.x; i < bytes / 16; i += threads) static_cast<int4*>(p)[i] = make_int4(0, 0, 0, 0);
}

// Selection and buckets of up to 16 tokens; a workgroup of max(T, T*k/64) waves
template <int V, bool BF16>
__global__ __launch_bounds__(kBkThreads) void route_bucket_grouped_kernel(RouteRule r, const void* __restrict__ logits,
                                                                          const float* __restrict__ bias,
                                                                          int32_t* __restrict__ topk_idx,
                                                                          float* __restrict__ topk_w, BucketOut o) {
  extern __shared__ __align__(16) float s_rows[];            // 2E a token
  __shared__ __align__(16) int s_cnt[kMaxExperts];
  __shared__ int s_ids[kSmallTokens * 32];
  __shared__ int2 s_wave[kBkWaves];
  __shared__ __align__(16) uint8_t s_wcnt[kSmallTokens * 32 / kWave][kMaxExperts];      // of the waves that have routes
  const int tid = threadIdx.x, lane = tid & (kWave - 1), threads = (int)blockDim.x;
  const int t = __builtin_amdgcn_readfirstlane(tid >> 6), R = r.T * r.k;
  clear(s_cnt, sizeof(s_cnt), threads);
  clear(s_wcnt, sizeof(s_wcnt), threads);
  if (t < r.T) {
    int e;
    float w;
    select_grouped<V, BF16>(r, logits, bias, t, lane, s_rows + t * 2 * r.E, e, w);
    if (lane < r.k) {
      topk_idx[t * r.k + lane] = e;
      topk_w[t * r.k + lane] = w;
      s_ids[t * r.k + lane] = e;
    }
  }
  __syncthreads();
  const bool valid = tid < R;
  const int e = valid ? s_ids[tid] : 0;
  if (valid) atomicAdd(&s_cnt[e], 1);                        // integer counts: order-free
  __syncthreads();
  offsets_block(s_cnt, s_wave, r.E, threads, true, o);
  place_block<kSmallTokens * 32 / kWave>(s_cnt, s_wcnt, tid, valid, e, o);
}

struct ChunkShared {
  __align__(16) int after[kMaxExperts];                                    // routes from 1024c on
  __align__(16) int before[kMaxExperts];
  int2 wave[kBkWaves];
  __align__(16) uint8_t wcnt[kBkWaves][kMaxExperts];
};

// Workgroup c: routes 1024c .. 1024c + 1024.  All routes are counted, those
// before them apart: these are what earlier workgroups place.
__global__ __launch_bounds__(kBkThreads) void bucket_chunk_kernel(const int32_t* __restrict__ ids, int R, int E, BucketOut o) {
  __shared__ ChunkShared sh;
  const int tid = threadIdx.x, mine = (int)blockIdx.x * kBkThreads;
  // routes past the last read as 0 and are not counted
  const auto all_ids = make_rsrc(ids, (uint32_t)R * 4u);
  const int r = mine + tid;
  const bool valid = r < R;
  const int my_e = (int)__builtin_amdgcn_raw_buffer_load_b32(all_ids, (uint32_t)r * 4u, 0, 0);
  clear(sh.after, sizeof(sh.after), kBkThreads);
  clear(sh.before, sizeof(sh.before), kBkThreads);
  clear(sh.wcnt, sizeof(sh.wcnt), kBkThreads);
  __syncthreads();
  constexpr int kLoads = 8;                                  // four routes each, in flight
  for (int r0 = 0; r0 < R; r0 += kLoads * 4 * kBkThreads) {
    u32x4 v[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads; ++u)
      v[u] = __builtin_amdgcn_raw_buffer_load_b128(all_ids, (uint32_t)(r0 + (u * kBkThreads + tid) * 4) * 4u, 0, 0);
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int at = r0 + (u * kBkThreads + tid) * 4;        // (a multiple of four, as is `mine`)
      int* const cnt = at < mine ? sh.before : sh.after;
      if (at + 4 <= R) {
#pragma unroll
        for (int i = 0; i < 4; ++i) atomicAdd(&cnt[v[u][i]], 1);
      } else {
        for (int i = 0; i < R - at; ++i) atomicAdd(&cnt[v[u][i]], 1);
      }
    }
  }
  __syncthreads();
  if (tid < E) sh.after[tid] += sh.before[tid];
  __syncthreads();
  offsets_block(sh.after, sh.wave, E, kBkThreads, blockIdx.x == 0, o);
  if (tid < E) sh.before[tid] += sh.after[tid];
  // (place_block's own barrier is before its reads of `before`)
  place_block<kBkWaves>(sh.before, sh.wcnt, r, valid, my_e, o);
}

// Many routes, in chunks of 2048: counts[c][e] of every chunk, their prefixes
// over the chunks, route_src, and its inverse.  The counts lie where route_pos
// goes (R >= C * E from 2048 routes on), which only the last kernel writes.
constexpr int kChunk = 2 * kBkThreads;

__global__ __launch_bounds__(kBkThreads) void count_kernel(const int32_t* __restrict__ ids, int R, int E,
                                                           int32_t* __restrict__ counts) {
  __shared__ int s_cnt[kMaxExperts];
  const int tid = threadIdx.x;
  s_cnt[tid] = 0;
  __syncthreads();
  for (int u = 0; u < 2; ++u) {
    const int r = (int)blockIdx.x * kChunk + u * kBkThreads + tid;
    if (r < R) atomicAdd(&s_cnt[ids[r]], 1);
  }
  __syncthreads();
  if (tid < E) counts[(size_t)blockIdx.x * E + tid] = s_cnt[tid];
}

__global__ __launch_bounds__(kBkThreads) void prefix_kernel(int32_t* __restrict__ counts, int C, int E, BucketOut o) {
  __shared__ int s_cnt[kMaxExperts];
  __shared__ int2 s_wave[kBkWaves];
  const int e = threadIdx.x;
  constexpr int kTogether = 16;                              // counts in flight
  int run = 0;
  if (e < E) {
    for (int c0 = 0; c0 < C; c0 += kTogether) {
      int v[kTogether];
#pragma unroll
      for (int j = 0; j < kTogether; ++j) v[j] = c0 + j < C ? counts[(size_t)(c0 + j) * E + e] : 0;
#pragma unroll
      for (int j = 0; j < kTogether; ++j) {
        if (c0 + j < C) counts[(size_t)(c0 + j) * E + e] = run;
        run += v[j];
      }
    }
    s_cnt[e] = run;
  }
  __syncthreads();
  offsets_block(s_cnt, s_wave, E, kBkThreads, true, o);
}

__global__ __launch_bounds__(kBkThreads) void scatter_kernel(const int32_t* __restrict__ ids, int R, int E,
                                                             const int32_t* __restrict__ counts, BucketOut o) {
  __shared__ int s_base[kMaxExperts];
  __shared__ __align__(16) uint8_t s_wcnt[kBkWaves][kMaxExperts];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid >> 6;
  if (tid < E) s_base[tid] = o.offset[tid] + counts[(size_t)blockIdx.x * E + tid];
  for (int u = 0; u < 2; ++u) {
    clear(s_wcnt, sizeof(s_wcnt), kBkThreads);
    const int r = (int)blockIdx.x * kChunk + u * kBkThreads + tid;
    const bool valid = r < R;
    const int e = valid ? ids[r] : 0;
    const uint64_t same = same_expert(e, valid);
    const int rank = __popcll(same & ((1ull << lane) - 1ull));
    __syncthreads();
    if (valid && rank == 0) s_wcnt[wave][e] = (uint8_t)__popcll(same);
    __syncthreads();
    int pos = 0;
    if (valid) {
      pos = s_base[e] + rank;
#pragma unroll
      for (int w = 0; w < kBkWaves; ++w) pos += w < wave ? s_wcnt[w][e] : 0;
      o.src[pos] = r;
    }
    __syncthreads();
    if (valid && rank == 0) atomicAdd(&s_base[e], __popcll(same));
    __syncthreads();
  }
}

__global__ __launch_bounds__(256) void invert_kernel(const int32_t* __restrict__ src, int R, int32_t* __restrict__ pos) {
  const int p = (int)blockIdx.x * 256 + threadIdx.x;
  if (p < R) pos[src[p]] = p;
}

// With the selection, E = 256, k = 8, counted by every workgroup and counted
// once (four launches): 65536 routes 22.9 and 26.9 us, 131072 40.8 and 39.6,
// 240000 64.5 and 57.4 (the bytes 7; by a tracer the selection 40 to 44, the four
// launches 24: each passes over the routes in little more than a launch's
// time, the prefix over 118 chunks is one workgroup's 8.6).
constexpr int kChunkRoutes = (1 << 17) - 1;

moe_status bucket(const int32_t* ids, int R, int E, const BucketOut& o, hipStream_t s) {
  if (R <= kChunkRoutes) {
    bucket_chunk_kernel<<<(unsigned)((R + kBkThreads - 1) / kBkThreads), kBkThreads, 0, s>>>(ids, R, E, o);
    return launch_status();
  }
  const int C = (R + kChunk - 1) / kChunk;
  int32_t* const counts = o.pos;
  count_kernel<<<(unsigned)C, kBkThreads, 0, s>>>(ids, R, E, counts);
  prefix_kernel<<<1, kBkThreads, 0, s>>>(counts, C, E, o);
  scatter_kernel<<<(unsigned)C, kBkThreads, 0, s>>>(ids, R, E, counts, o);
  invert_kernel<<<(unsigned)((R + 255) / 256), 256, 0, s>>>(o.src, R, o.pos);
  return launch_status();
}

RouteRule make_rule(int T, int E, int k, int score, int groups, int groups_kept, int group_top,
                    int renormalise, float scale) {
  const int lanes = group_lanes(groups), size = E / groups;
  return RouteRule{T, E, k, groups, groups_kept, group_top, renormalise != 0, score == MOE_SCORE_SOFTMAX,
                   scale, lanes, (size + lanes - 1) / lanes};
}

// f(experts of a lane, rounded up to a power of two, and whether logits are bf16, as integral constants)
template <bool BF16, class F>
void with_experts(const RouteRule& r, F&& f) {
  const std::integral_constant<bool, BF16> bf16;
  if (r.per_lane <= 1) f(std::integral_constant<int, 1>{}, bf16);
  else if (r.per_lane <= 2) f(std::integral_constant<int, 2>{}, bf16);
  else if (r.per_lane <= 4) f(std::integral_constant<int, 4>{}, bf16);
  else if (r.per_lane <= 8) f(std::integral_constant<int, 8>{}, bf16);
  else f(std::integral_constant<int, 16>{}, bf16);
}
template <class F>
void with_kernel(int logits_type, const RouteRule& r, F&& f) {
  if (logits_type == MOE_DTYPE_BF16) with_experts<true>(r, f);
  else with_experts<false>(r, f);
}

moe_status select(int logits_type, const RouteRule& r, const void* logits, const float* bias, int32_t* topk_idx,
                  float* topk_w, hipStream_t s) {
  with_kernel(logits_type, r, [&](auto v, auto bf16) {
    route_grouped_kernel<decltype(v)::value, decltype(bf16)::value>
        <<<(unsigned)((r.T + kRouteWaves - 1) / kRouteWaves), kRouteWaves * kWave, kRouteWaves * 8u * r.E, s>>>(
            r, logits, bias, topk_idx, topk_w);
  });
  return launch_status();
}

moe_status check_grouped(const void* logits, int logits_type, const float* bias, int T, int E, int k, int score,
                         int groups, int groups_kept, int group_top, float scale, const int32_t* topk_idx,
                         const float* topk_w) {
  if (T < 0 || E < 1 || k < 1 || k > E || groups < 1 || groups_kept < 1 || groups_kept > groups || E % groups != 0 ||
      (long long)groups_kept * (E / groups) < k || (group_top != 1 && group_top != 2) ||
      (logits_type != MOE_DTYPE_F32 && logits_type != MOE_DTYPE_BF16) ||
      (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) || !(scale - scale == 0.0f))
    return MOE_ERR_INVALID_SHAPE;
  if (E > 1024 || k > 32 || groups > kWave || (long long)T * k > (1ll << 24)) return MOE_ERR_UNSUPPORTED;
  if ((E / groups + group_lanes(groups) - 1) / group_lanes(groups) > kMaxPerLane) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!logits || !topk_idx || !topk_w) return MOE_ERR_NULL_POINTER;
  if (!aligned16(logits) || !aligned16(topk_idx) || !aligned16(topk_w) || (bias && !aligned16(bias)))
    return MOE_ERR_MISALIGNED;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_route_grouped(const void* logits, int logits_type, const float* bias, int T, int E, int k,
                                        int score, int groups, int groups_kept, int group_top, int renormalise,
                                        float scale, int32_t* topk_idx, float* topk_w, void* stream) {
  using namespace moe;
  const moe_status st = check_grouped(logits, logits_type, bias, T, E, k, score, groups, groups_kept, group_top, scale,
                                      topk_idx, topk_w);
  if (st != MOE_OK || T == 0) return st;
  return select(logits_type, make_rule(T, E, k, score, groups, groups_kept, group_top, renormalise, scale), logits, bias,
                topk_idx, topk_w, static_cast<hipStream_t>(stream));
}

extern "C" moe_status moe_route_grouped_bucket(const void* logits, int logits_type, const float* bias, int T, int E,
                                               int k, int score, int groups, int groups_kept, int group_top,
                                               int renormalise, float scale, int32_t* topk_idx, float* topk_w,
                                               int32_t* expert_count, int32_t* expert_offset, int32_t* active_experts,
                                               int32_t* n_active, int32_t* route_src, int32_t* route_pos,
                                               void* stream) {
  using namespace moe;
  moe_status st = check_grouped(logits, logits_type, bias, T, E, k, score, groups, groups_kept, group_top, scale,
                                topk_idx, topk_w);
  if (st != MOE_OK || T == 0) return st;
  int32_t* const outs[] = {expert_count, expert_offset, active_experts, n_active, route_src, route_pos};
  for (const int32_t* o : outs)
    if (!o) return MOE_ERR_NULL_POINTER;
  for (const int32_t* o : outs)
    if (!aligned16(o)) return MOE_ERR_MISALIGNED;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const RouteRule r = make_rule(T, E, k, score, groups, groups_kept, group_top, renormalise, scale);
  const BucketOut o{expert_count, expert_offset, active_experts, n_active, route_src, route_pos};
  if (T <= kSmallTokens && T * E <= kSmallScores) {
    const int routes = (T * k + kWave - 1) / kWave, waves = T > routes ? T : routes;
    with_kernel(logits_type, r, [&](auto v, auto bf16) {
      route_bucket_grouped_kernel<decltype(v)::value, decltype(bf16)::value>
          <<<1, (waves < 4 ? 4 : waves) * kWave, T * 8u * E, s>>>(r, logits, bias, topk_idx, topk_w, o);
    });
    return launch_status();
  }
  st = select(logits_type, r, logits, bias, topk_idx, topk_w, s);
  return st == MOE_OK ? bucket(topk_idx, T * k, E, o, s) : st;
}
