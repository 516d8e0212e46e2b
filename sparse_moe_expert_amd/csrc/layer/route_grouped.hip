// Grouped routing: moe_route_grouped and moe_route_grouped_bucket.
//
// Per token, with z the logits and b the balance bias,
//   s_e = sigmoid(z_e)  or  exp(z_e - max z) / sum_i exp(z_i - max z),
//   c_e = s_e + b_e                        (the selection's value; not the weight's)
//   G_g = sum of the group_top largest c of group g (its unmasked experts),
//   the groups_kept groups of largest G, in them the k experts of largest c,
//   w_j = scale * s_j  (/ sum_i s_i over the chosen, where renormalised).
// Equal values go to the lower id, of groups and of experts.  Scores and
// choice values are held in 64 bits: sums s + b of different experts often
// agree to 32 bits, and which expert is taken would hang on the last bit of an
// exponential.
#include "moe_common.h"
#include "bucket_block.h"
#include "route_rule.h"

namespace moe {
namespace {

// One token per wavefront: scores in LDS, k rounds of arg-max over them.
__global__ __launch_bounds__(kWave) void route_grouped_kernel(RouteRule r, const void* __restrict__ logits,
                                                              const float* __restrict__ bias,
                                                              int32_t* __restrict__ topk_idx,
                                                              float* __restrict__ topk_w) {
  __shared__ double s_score[1024];
  __shared__ double s_choice[1024];
  __shared__ double s_group[64];
  __shared__ int s_kept[64];
  const int lane = threadIdx.x, t = blockIdx.x;
  const double kMasked = -__builtin_huge_val();
  double top = kMasked;
  for (int e = lane; e < r.E; e += kWave) {
    const double z = load_logit(logits, r.bf16, (size_t)t * r.E + e);
    s_score[e] = z;
    top = fmax(top, z);
  }
  for (int o = 32; o > 0; o >>= 1) top = fmax(top, __shfl_xor(top, o, kWave));
  double sum = 0.0;
  if (r.softmax) {
    for (int e = lane; e < r.E; e += kWave) {
      const double z = s_score[e];
      if (z > kMasked) sum += exp(z - top);
    }
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, kWave);
  }
  for (int e = lane; e < r.E; e += kWave) {
    const double z = s_score[e];
    double s = 0.0;
    if (z > kMasked) s = r.softmax ? exp(z - top) / sum : 1.0 / (1.0 + exp(-z));
    const float b = bias ? bias[e] : 0.0f;
    s_score[e] = s;
    s_choice[e] = z > kMasked && b > kLowest ? s + (double)b : kMasked;
  }
  __syncthreads();
  const int size = r.E / r.groups;
  if (lane < r.groups) {
    double a = kMasked, c = kMasked;
    for (int i = 0; i < size; ++i) {
      const double v = s_choice[lane * size + i];
      if (v > a) { c = a; a = v; } else if (v > c) { c = v; }
    }
    s_group[lane] = r.group_top == 2 && c > kMasked ? a + c : a;
  }
  __syncthreads();
  if (lane < r.groups) {
    int before = 0;
    for (int g = 0; g < r.groups; ++g)
      before += s_group[g] > s_group[lane] || (s_group[g] == s_group[lane] && g < lane);
    s_kept[lane] = before < r.kept;
  }
  __syncthreads();
  // the masked experts of the kept groups follow its others, lowest id first
  constexpr double kLast = -1e300, kTaken = -1e306;
  for (int e = lane; e < r.E; e += kWave)
    s_choice[e] = s_kept[e / size] ? fmax(s_choice[e], kLast) : kTaken;
  double total = 0.0, my_s = 0.0;
  int my_e = 0;
  for (int j = 0; j < r.k; ++j) {
    double best = -__builtin_huge_val();
    int be = 1 << 20;
    for (int e = lane; e < r.E; e += kWave)
      if (s_choice[e] > best) { best = s_choice[e]; be = e; }
    for (int o = 32; o > 0; o >>= 1) {
      const double v = __shfl_xor(best, o, kWave);
      const int ve = __shfl_xor(be, o, kWave);
      if (v > best || (v == best && ve < be)) { best = v; be = ve; }
    }
    const double s = best > kLast ? s_score[be] : 0.0;
    total += s;
    if (lane == j) { my_s = s; my_e = be; }
    if (lane == (be & (kWave - 1))) s_choice[be] = kTaken;
  }
  if (lane < r.k) {
    double w = my_s;
    if (r.renormalise) w = total > 0.0 ? w / total : 0.0;
    topk_idx[(size_t)t * r.k + lane] = my_e;
    topk_w[(size_t)t * r.k + lane] = (float)(w * (double)r.scale);
  }
}

__global__ __launch_bounds__(kBucketThreads) void bucket_grouped_kernel(
    const int32_t* __restrict__ topk_idx, int R, int E, int32_t* __restrict__ expert_count,
    int32_t* __restrict__ expert_offset, int32_t* __restrict__ active_experts, int32_t* __restrict__ n_active,
    int32_t* __restrict__ route_src, int32_t* __restrict__ route_pos) {
  __shared__ BucketShared sh;
  bucket_block(topk_idx, R, E, sh, expert_count, expert_offset, active_experts, n_active, route_src, route_pos,
               WorkLists{});
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
  const RouteRule r{T, E, k, groups, groups_kept, group_top, renormalise != 0, score == MOE_SCORE_SOFTMAX,
                    logits_type == MOE_DTYPE_BF16, scale};
  route_grouped_kernel<<<T, kWave, 0, static_cast<hipStream_t>(stream)>>>(r, logits, bias, topk_idx, topk_w);
  return launch_status();
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
  st = moe_route_grouped(logits, logits_type, bias, T, E, k, score, groups, groups_kept, group_top, renormalise, scale,
                         topk_idx, topk_w, stream);
  if (st != MOE_OK) return st;
  bucket_grouped_kernel<<<1, kBucketThreads, 0, static_cast<hipStream_t>(stream)>>>(
      topk_idx, T * k, E, expert_count, expert_offset, active_experts, n_active, route_src, route_pos);
  return launch_status();
}
