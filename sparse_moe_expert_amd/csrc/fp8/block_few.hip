// The dense layer of few tokens.
#include "block_few.h"

#include "block_linear.h"

namespace moe {
namespace {

template <int RT, int JT, int D>
__global__ __launch_bounds__(kFewThreads, 2) void linear_few_kernel(LinearArgs p) {
  __shared__ f32x4 s_sum[kFewWaves][RT * JT][kWave];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4, n0 = (int)blockIdx.x * (16 * RT), kb = blocks_of(p.K);
  const int rows = min(16 * RT, p.N - n0);
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(p.w.q + (size_t)n0 * p.K, (uint32_t)rows * (uint32_t)p.K);
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(p.x, (uint32_t)p.T * (uint32_t)p.K);
  const float* const sw = p.w.s + (size_t)(n0 / kBlock) * kb;          // (16 RT rows lie in one block of them)
  f32x4 sum[RT][JT] = {};
  for (int b0 = wave * D; b0 < kb; b0 += kFewWaves * D) {
    i32x8 w[D][RT], x[D][JT];
    float s[D][JT];
    // rows and tokens past the last one repeat it, blocks past the last are zero
#pragma unroll
    for (int i = 0; i < D; ++i)
#pragma unroll
      for (int m = 0; m < RT; ++m) w[i][m] = load_block(rw, (uint32_t)(min(m * 16 + l16, rows - 1) * p.K), b0 + i, p.K, g);
#pragma unroll
    for (int i = 0; i < D; ++i) {
      const int b = min(b0 + i, kb - 1);
      const float scale = scalar_load(sw + b);
      const bool in = b0 + i < kb;
#pragma unroll
      for (int j = 0; j < JT; ++j) {
        const int t = min(j * 16 + l16, p.T - 1);
        x[i][j] = load_block(rx, (uint32_t)(t * p.K), b0 + i, p.K, g);
        s[i][j] = in ? p.sx[(size_t)t * kb + b] * scale : 0.0f;      // (the last one's may be no number)
      }
    }
    __builtin_amdgcn_sched_barrier(0);                       // (all loads first)
#pragma unroll
    for (int i = 0; i < D; ++i)
#pragma unroll
      for (int m = 0; m < RT; ++m)
#pragma unroll
        for (int j = 0; j < JT; ++j) {
          const f32x4 d = block_product(w[i][m], x[i][j]);
#pragma unroll
          for (int c = 0; c < 4; ++c) sum[m][j][c] = fmaf(d[c], s[i][j], sum[m][j][c]);
        }
  }
#pragma unroll
  for (int m = 0; m < RT; ++m)
#pragma unroll
    for (int j = 0; j < JT; ++j) s_sum[wave][m * JT + j][lane] = sum[m][j];
  __syncthreads();
  for (int q = wave; q < RT * JT; q += kFewWaves) {
    float v[4] = {};
    for (int w = 0; w < kFewWaves; ++w) {
      const f32x4 a = s_sum[w][q][lane];
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] += a[c];
    }
    const int t = q % JT * 16 + l16;
    if (t < p.T) write(p, t, n0 + q / JT * 16 + g * 4, v);
  }
}

// Many rows: 64 a workgroup, whose tokens are then read by a quarter as many
// (T = 16 9999x4096 14.0 us, 17.4 with 16 rows; T = 1 12.0 and 14.3); else as many
// workgroups as there are (T = 32 4096x4096 10.8 us, 16.0 with 64 rows), the
// reduction's blocks spread over the waves.  (Weights from HBM, as in a decode loop
// over layers; so are the figures below.)
template <int JT>
void launch(const LinearArgs& p, hipStream_t s) {
  const int kb = blocks_of(p.K);
  const unsigned grid = (unsigned)(p.N + 15) / 16;
  if (p.N >= 8192) linear_few_kernel<4, JT, 2><<<(grid + 3) / 4, kFewThreads, 0, s>>>(p);
  else if (kb > 2 * kFewWaves) linear_few_kernel<1, JT, 4><<<grid, kFewThreads, 0, s>>>(p);
  else if (kb > kFewWaves) linear_few_kernel<1, JT, 2><<<grid, kFewThreads, 0, s>>>(p);
  else linear_few_kernel<1, JT, 1><<<grid, kFewThreads, 0, s>>>(p);
}

}  // namespace

// Beyond 16 tokens, small weights only: T = 32 2048x2048 6.3 us, 7.4 in tiles of 64
// rows; 4096x4096 10.8 and 10.6; 9999x4096 16.7 and 13.5.  (Up to 16 tokens tiles have
// not been fitted: 9999x4096 takes 12.0 us here and 11.1 in tiles for one token, 14.0
// and 11.9 for 16.)
bool linear_few_ok(int T, int N, int K) { return T <= 16 || (T <= 32 && (long long)N * K <= 1 << 23); }

moe_status linear_few(const LinearArgs& p, hipStream_t s) {
  if (p.T <= 16) launch<1>(p, s);
  else launch<2>(p, s);
  return launch_status();
}

}  // namespace moe
