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
// far above its spread loses nothing, and a LAYER norm costs one barrier as an RMS norm does.
#include <type_traits>

#include "device_common.h"
#include "launchers.h"

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
  for (int q = 0; q < 4; ++q) u[q] = pack_bf16x2(v[2 * q], v[2 * q + 1]);
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
    n_w = wave_sum(n);
    mean_w = n_w > 0.0f ? wave_sum(sum) / n_w : 0.0f;
  }
  float sq = 0.0f;
#pragma unroll
  for (int i = 0; i < NC; ++i)
    if (in[i]) {
#pragma unroll
      for (int j = 0; j < 8; ++j) sq += (v[i][j] - mean_w) * (v[i][j] - mean_w);
    }
  sq = wave_sum(sq);
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

// A thread holds chunks (8 values) lane + threads * i of its row, i < NC.  ONE: a wave per row,
// else a workgroup per row.
template <int NC, bool YF32, bool RF32, bool ONE>
__global__ __launch_bounds__(1024) void block_norm_kernel(BlockNormArgs p) {
  __shared__ float2 red[2][kMaxWaves + kMaxWaves / 2];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int waves = blockDim.x >> 6;
  const int tid = ONE ? lane : threadIdx.x, threads = ONE ? kWave : blockDim.x;
  const int row0 = ONE ? blockIdx.x * waves + wave : blockIdx.x;
  const int stride = ONE ? gridDim.x * waves : gridDim.x;
  const int chunks = p.H >> 3;
  bool in[NC];
  int at[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = tid + threads * i;
    in[i] = c < chunks;
    at[i] = 8 * (in[i] ? c : 0);
  }
  for (int row = row0; row < p.M; row += stride) {
    Raw<YF32> y[NC];
    Raw<RF32> r[NC];
    Raw<false> g[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      y[i].zero();
      r[i].zero();
      if (in[i]) {
        if (p.y) y[i].load(p.y, (size_t)row * p.y_ld + at[i]);
        if (p.residual) r[i].load(p.residual, (size_t)row * p.residual_ld + at[i]);
        if (p.gate && p.gate_cols > 1) g[i].load(p.gate, (size_t)row * p.gate_ld + at[i]);
      }
    }
    const float token_gate =
        p.gate && p.gate_cols == 1 ? bf16_to_f32(p.gate[(size_t)row * p.gate_ld]) : 1.0f;
    float v[NC][8];
    auto normalize = [&](int kind, const uint16_t* w, const uint16_t* b, float2* slot) {
      const float2 m = row_moments<NC, ONE>(v, in, kind == kNormLayer, p.H, wave, waves, lane, slot);
      const float f = 1.0f / sqrtf(m.y + p.eps);
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        if (!in[i]) continue;
        Raw<false> wv, bv;
        if (w) wv.load(w, at[i]);
        if (b) bv.load(b, at[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[i][j] = (v[i][j] - m.x) * f;
          if (w) v[i][j] *= p.weight_offset + wv.get(j);
          if (b) v[i][j] += bv.get(j);
        }
      }
    };
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = y[i].get(j);
    if (p.post != kNormNone) normalize(p.post, p.post_w, p.post_b, red[0]);
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float u = v[i][j] * p.block_scale;
        if (p.gate) u *= p.gate_cols > 1 ? g[i].get(j) : token_gate;
        v[i][j] = r[i].get(j) * p.residual_scale + u;
      }
    if (p.z_out) {
#pragma unroll
      for (int i = 0; i < NC; ++i)
        if (in[i]) {
          const size_t o = (size_t)row * p.z_ld + at[i];
          if (RF32) store_f32(static_cast<float*>(p.z_out) + o, v[i]);
          else store_bf16(static_cast<uint16_t*>(p.z_out) + o, v[i]);
        }
    }
    if (p.pre != kNormNone) normalize(p.pre, p.pre_w, p.pre_b, red[1]);
    if (p.out) {
#pragma unroll
      for (int i = 0; i < NC; ++i)
        if (in[i]) store_bf16(p.out + (size_t)row * p.out_ld + at[i], v[i]);
    }
    if (!ONE) __syncthreads();   // the next row's reductions reuse red
  }
}

}  // namespace

hipError_t launch_block_norm(const BlockNormArgs& a, hipStream_t s) {
  const int chunks = a.H >> 3;
  auto go = [&](auto nc, auto one) {
    constexpr int NC = decltype(nc)::value;
    constexpr bool ONE = decltype(one)::value;
    const int threads = ONE ? 256 : (chunks + NC * kWave - 1) / (NC * kWave) * kWave;
    const int rows = ONE ? threads / kWave : 1;
    const unsigned grid = (unsigned)((a.M + rows - 1) / rows < (1 << 16) ? (a.M + rows - 1) / rows : 1 << 16);
    if (a.y_f32 && a.residual_f32)
      hipLaunchKernelGGL((block_norm_kernel<NC, true, true, ONE>), dim3(grid), dim3(threads), 0, s, a);
    else if (a.y_f32)
      hipLaunchKernelGGL((block_norm_kernel<NC, true, false, ONE>), dim3(grid), dim3(threads), 0, s, a);
    else if (a.residual_f32)
      hipLaunchKernelGGL((block_norm_kernel<NC, false, true, ONE>), dim3(grid), dim3(threads), 0, s, a);
    else
      hipLaunchKernelGGL((block_norm_kernel<NC, false, false, ONE>), dim3(grid), dim3(threads), 0, s, a);
    return hipGetLastError();
  };
  if (chunks <= kWave) return go(std::integral_constant<int, 1>{}, std::true_type{});
  if (chunks <= 1024) return go(std::integral_constant<int, 1>{}, std::false_type{});
  return go(std::integral_constant<int, 2>{}, std::false_type{});
}

}  // namespace moe
