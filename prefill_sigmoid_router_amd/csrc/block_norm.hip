// The norm after a block, the block's gate and scale, the residual, and the norm before the
// next block, in one pass over the rows:
//   u   = N_post(y), or y
//   z   = residual_scale * residual + block_scale * gate * u
//   out = N_pre(z), or z
//   RMS:   N(v) = v * (mean v^2 + eps)^-1/2 * (offset + w) + b
//   LAYER: N(v) = (v - mean v) * (mean (v - mean v)^2 + eps)^-1/2 * (offset + w) + b
// Everything between the loads and the two stores is fp32 in registers (out comes from the
// unrounded z).  The mean of squared distances is taken around each wave's own mean and moved
// to the row's (Chan's pairwise formula: n_w (mean_w - mean)^2 more), so a row whose mean is
// far above its spread loses no more than the mean's own fp32 roundings, and a LAYER norm costs one
// barrier as an RMS norm does.
// Bound by memory where there are many rows: 8192 x 7168, bf16, RMS twice and a gate per channel (470
// MB) takes 91 to 97 us, 4.8 to 5.1 TB/s, where a large copy reaches 4.9; with a gate value for every
// token and channel 113 (5.2).  Gates of the tokens and biases are loaded for each row, behind the next
// row's values, which a wave then waits for: token gate and biases 103 us (4.6 TB/s), LAYER norms twice
// with biases 109 (4.3), those and a full gate 141 (4.2).  One row of 7168 takes 4.4 us: a launch, a
// load and two reductions.
#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "launchers.h"
#include "wave_ops.h"

namespace moe {

namespace {

constexpr int kMaxWaves = 16;

template <bool F32>
struct Raw;   // 8 values as they lie in memory
template <>
struct Raw<false> {
  u32x4 a;
  __device__ void load(const void* p, size_t i) { a = ld16(static_cast<const uint16_t*>(p) + i); }
  __device__ void zero() { a = u32x4{0, 0, 0, 0}; }
  __device__ float get(int j) const { return j & 1 ? bf16hi(a[j >> 1]) : bf16lo(a[j >> 1]); }
};
template <>
struct Raw<true> {
  u32x4 a, b;
  __device__ void load(const void* p, size_t i) {
    a = ld16(static_cast<const float*>(p) + i);
    b = ld16(static_cast<const float*>(p) + i + 4);
  }
  __device__ void zero() { a = b = u32x4{0, 0, 0, 0}; }
  __device__ float get(int j) const { return __uint_as_float(j < 4 ? a[j] : b[j - 4]); }
};

__device__ __forceinline__ void store_bf16(uint16_t* p, const float (&v)[8]) {
  u32x4 u;
#pragma unroll
  for (int q = 0; q < 4; ++q) u[q] = cvt_bf16x2(v[2 * q], v[2 * q + 1]);
  st16(p, u);
}
__device__ __forceinline__ void store_f32(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// Mean (LAYER; else 0) and the mean of squared distances from it, of a row of H values held 8 NC
// to a thread.  ONE: a wave holds the row.  red: [kMaxWaves] pairs, not in use by a reduction
// that waves may still read.
template <int NC, bool ONE>
__device__ __forceinline__ float2 row_moments(const float (&v)[NC][8], const bool (&in)[NC],
                                              bool layer, int H, int wave, int waves, int lane,
                                              float2* red) {
  float mean_w = 0.0f, n_w = 0.0f;
  if (layer) {
    float sum = 0.0f, n = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i)
      if (in[i]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += v[i][j];
        n += 8.0f;
      }
    n_w = wave_sum_f32(n);
    mean_w = n_w > 0.0f ? wave_sum_f32(sum) / n_w : 0.0f;
  }
  float sq = 0.0f;
#pragma unroll
  for (int i = 0; i < NC; ++i)
    if (in[i]) {
#pragma unroll
      for (int j = 0; j < 8; ++j) sq += (v[i][j] - mean_w) * (v[i][j] - mean_w);
    }
  sq = wave_sum_f32(sq);
  const float inv = 1.0f / (float)H;
  if (ONE) return make_float2(mean_w, sq * inv);
  // each wave's values in order, n_w from the wave's place: chunks wave * 64 + threads * i on
  if (lane == 0) {
    red[wave] = make_float2(mean_w, sq);
    if (layer) reinterpret_cast<float*>(red + kMaxWaves)[wave] = n_w;
  }
  __syncthreads();
  float mean = 0.0f, total = 0.0f;
  if (layer) {
    for (int w = 0; w < waves; ++w)
      mean += red[w].x * reinterpret_cast<const float*>(red + kMaxWaves)[w];
    mean *= inv;
    for (int w = 0; w < waves; ++w) {
      const float d = red[w].x - mean;
      total += red[w].y + reinterpret_cast<const float*>(red + kMaxWaves)[w] * (d * d);
    }
  } else {
    for (int w = 0; w < waves; ++w) total += red[w].y;
  }
  return make_float2(mean, total * inv);
}

// A thread holds chunks (8 values) lane + threads * i of its row, i < NC, and walks rows; the next
// row's values are in flight while a row is reduced.  What belongs to the channels is read once:
//   p = (offset + post_w) * channel gate * block_scale,  q = offset + pre_w
// ONE: a wave per row (no barriers), else a workgroup per row.
template <int NC, bool YF32, bool RF32, bool ONE>
__global__ __launch_bounds__(ONE ? 256 : NC == 1 ? 1024 : 512) void block_norm_kernel(BlockNormArgs a) {
  __shared__ float2 red[2][kMaxWaves + kMaxWaves / 2];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int waves = blockDim.x >> 6;
  const int tid = ONE ? lane : threadIdx.x, threads = ONE ? kWave : blockDim.x;
  const int stride = ONE ? gridDim.x * waves : gridDim.x;
  const int chunks = a.H >> 3;
  int row = ONE ? blockIdx.x * waves + wave : blockIdx.x;
  if (row >= a.M) return;
  bool in[NC];
  int at[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = tid + threads * i;
    in[i] = c < chunks;
    at[i] = 8 * c;
  }
  Raw<YF32> y[NC];
  Raw<RF32> r[NC];
  auto fetch = [&](int t) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if (a.y && in[i]) y[i].load(a.y, (size_t)t * a.y_ld + at[i]);
      if (a.residual && in[i]) r[i].load(a.residual, (size_t)t * a.residual_ld + at[i]);
    }
  };
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    y[i].zero();
    r[i].zero();
  }
  fetch(row);
  const bool token_gate = a.gate && a.gate_cols == 1;
  const bool full_gate = a.gate && a.gate_cols > 1 && a.gate_ld != 0;
  const bool channel_gate = a.gate && a.gate_cols > 1 && a.gate_ld == 0;
  float p[NC][8], q[NC][8];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    Raw<false> wp, wg, wq;
    wp.zero();
    wg.zero();
    wq.zero();
    if (a.post_w && in[i]) wp.load(a.post_w, at[i]);
    if (channel_gate && in[i]) wg.load(a.gate, at[i]);
    if (a.pre_w && in[i]) wq.load(a.pre_w, at[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      p[i][j] = a.post != kNormNone && a.post_w ? a.weight_offset + wp.get(j) : 1.0f;
      if (channel_gate) p[i][j] *= wg.get(j);
      p[i][j] *= a.block_scale;
      q[i][j] = a.pre_w ? a.weight_offset + wq.get(j) : 1.0f;
    }
  }
  for (;;) {
    float v[NC][8], w[NC][8];   // y, later z; residual
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[i][j] = y[i].get(j);
        w[i][j] = r[i].get(j) * a.residual_scale;
      }
    const int next = row + stride;
    if (next < a.M) fetch(next);
    const float tg = token_gate ? bf16_to_f32(a.gate[(size_t)row * a.gate_ld]) : 1.0f;
    float f = 1.0f;
    if (a.post != kNormNone) {
      const float2 m = row_moments<NC, ONE>(v, in, a.post == kNormLayer, a.H, wave, waves, lane, red[0]);
      f = 1.0f / sqrtf(m.y + a.eps);
      if (a.post == kNormLayer) {
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][j] -= m.x;
      }
    }
    f *= tg;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if (!in[i]) continue;
      if (full_gate) {
        Raw<false> g;
        g.load(a.gate, (size_t)row * a.gate_ld + at[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] *= g.get(j);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = fmaf(v[i][j] * f, p[i][j], w[i][j]);
      if (a.post != kNormNone && a.post_b) {   // + b gate block_scale
        Raw<false> b, g;
        b.load(a.post_b, at[i]);
        g.zero();
        if (full_gate || channel_gate) g.load(a.gate, (full_gate ? (size_t)row * a.gate_ld : 0) + at[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v[i][j] = fmaf(b.get(j) * (full_gate || channel_gate ? g.get(j) : tg), a.block_scale, v[i][j]);
      }
      if (a.z_out) {
        const size_t o = (size_t)row * a.z_ld + at[i];
        if (RF32) store_f32(static_cast<float*>(a.z_out) + o, v[i]);
        else store_bf16(static_cast<uint16_t*>(a.z_out) + o, v[i]);
      }
    }
    if (a.out) {
      f = 1.0f;
      if (a.pre != kNormNone) {
        const float2 m = row_moments<NC, ONE>(v, in, a.pre == kNormLayer, a.H, wave, waves, lane, red[1]);
        f = 1.0f / sqrtf(m.y + a.eps);
        if (a.pre == kNormLayer) {
#pragma unroll
          for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] -= m.x;
        }
      }
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        if (!in[i]) continue;
        if (a.pre != kNormNone) {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * f * q[i][j];
          if (a.pre_b) {
            Raw<false> b;
            b.load(a.pre_b, at[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] += b.get(j);
          }
        }
        store_bf16(a.out + (size_t)row * a.out_ld + at[i], v[i]);
      }
    }
    if (next >= a.M) return;
    row = next;
    if (!ONE) __syncthreads();   // the next row's reductions reuse red
  }
}

}  // namespace

hipError_t launch_block_norm(const BlockNormArgs& a, hipStream_t s) {
  const int chunks = a.H >> 3;
  int dev = 0, cus = 0;
  hipError_t err = hipGetDevice(&dev);
  if (err == hipSuccess) err = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
  if (err != hipSuccess) return err;
  auto go = [&](auto nc, auto one, int per_cu) {
    constexpr int NC = decltype(nc)::value;
    constexpr bool ONE = decltype(one)::value;
    const int threads = ONE ? 256 : (chunks + NC * kWave - 1) / (NC * kWave) * kWave;
    const int rows = ONE ? threads / kWave : 1;
    const unsigned grid = (unsigned)std::min((a.M + rows - 1) / rows, cus * per_cu);
    auto kernel = a.y_f32 ? (a.residual_f32 ? block_norm_kernel<NC, true, true, ONE>
                                            : block_norm_kernel<NC, true, false, ONE>)
                          : (a.residual_f32 ? block_norm_kernel<NC, false, true, ONE>
                                            : block_norm_kernel<NC, false, false, ONE>);
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(threads), 0, s, a);
    return hipGetLastError();
  };
  using std::integral_constant;
  const std::true_type wave{};
  const std::false_type group{};
  // Measured with RMS twice and a channel gate, us.  A wave per row, no barriers, where it holds the
  // row: H = 512, M = 8192 9.4 (a workgroup per row 11.5); H = 1024, M = 8192 13.1 (15.8).
  if (chunks <= kWave) return go(integral_constant<int, 1>{}, wave, 8);
  // Long rows, two workgroups a CU: H = 16384, M = 1024 31.4 (four 40.6), M = 8192 203 (200).
  if (chunks > 1024) return go(integral_constant<int, 4>{}, group, 2);
  // One or two rows a CU, as many threads as it takes: H = 2048, M = 256 3.7 (two chunks a thread
  // 4.3); H = 7168, M = 8 4.5 (4.8).
  if (a.M <= 2 * cus) return go(integral_constant<int, 1>{}, group, 2);
  // Many rows, two chunks a thread, 16 waves a CU twice over: H = 2048, M = 8192 24.5 (one chunk
  // 31.0); H = 7168, M = 1024 15.9 (16.9), M = 8192 93.0 (91.4; a workgroup for each row that reads
  // what belongs to the channels anew 190).
  if (chunks <= 2 * kWave) return go(integral_constant<int, 2>{}, wave, 4);
  return go(integral_constant<int, 2>{}, group, 32 / ((chunks + 127) / 128));
}

}  // namespace moe
