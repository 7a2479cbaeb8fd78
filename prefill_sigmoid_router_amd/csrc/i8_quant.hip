// int8 rows: each row gets the scale a / 127, a its largest magnitude, and the codes
// rint(127 v / a) (nearest, ties to even); a row of zeros gets scale 0 and codes 0, a row
// that holds a NaN or an infinity a scale that is not finite and codes 0, so that products
// with it are not finite either.
//
// bf16 inputs have 8-bit significands, so 127 v is exact in fp32 and 127 v / a, if it is not
// exactly half way between two integers, is at least 2^(j - 17) from half way (j its
// binade), while one correctly rounded fp32 division is off by at most 2^(j - 24): the codes
// are those of exact arithmetic.
#include "device_common.h"
#include "launchers.h"

namespace moe {

namespace {

constexpr int kQThreads = 256;

__device__ __forceinline__ uint32_t max_bits(uint32_t m, u32x4 v) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    m = max(m, v[j] & 0x7fffu);
    m = max(m, (v[j] >> 16) & 0x7fffu);
  }
  return m;
}

// 127 and a, both by 2^-8 where 127 a may pass the largest number (values that this makes
// subnormal have code 0 either way).
struct Quotient {
  float k, a;
};
__device__ __forceinline__ Quotient quotient_of(float a) {
  return a >= 0x1p120f ? Quotient{127.0f * 0x1p-8f, a * 0x1p-8f} : Quotient{127.0f, a};
}
__device__ __forceinline__ uint32_t code_of(float v, Quotient q) {
  return (uint32_t)(int)rintf((q.k * v) / q.a) & 0xffu;
}

__device__ __forceinline__ uint2 codes8(u32x4 v, Quotient a) {
  uint2 c;
  c.x = code_of(bf16lo(v[0]), a) | code_of(bf16hi(v[0]), a) << 8 | code_of(bf16lo(v[1]), a) << 16 |
        code_of(bf16hi(v[1]), a) << 24;
  c.y = code_of(bf16lo(v[2]), a) | code_of(bf16hi(v[2]), a) << 8 | code_of(bf16lo(v[3]), a) << 16 |
        code_of(bf16hi(v[3]), a) << 24;
  return c;
}

// Rows of LANES threads each (a wave or the workgroup); KEEP chunks of 8 values per thread
// stay in registers between the maximum and the codes, later ones are read again.
template <int LANES, int KEEP>
__global__ __launch_bounds__(kQThreads) void i8_rows_kernel(const uint16_t* __restrict__ v,
                                                            int64_t row0, int64_t rows, int K,
                                                            int8_t* __restrict__ codes,
                                                            float* __restrict__ scales) {
  __shared__ uint32_t part[kQThreads / kWave];
  const int lane = threadIdx.x % LANES;
  const int64_t row = row0 + (int64_t)blockIdx.x * (kQThreads / LANES) + threadIdx.x / LANES;
  const bool on = row < rows;   // uniform over a row's threads
  const uint16_t* src = v + row * K;
  const int nchunk = K >> 3;
  u32x4 keep[KEEP];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < KEEP; ++i) {
    const int ch = lane + LANES * i;
    keep[i] = on && ch < nchunk ? ld16(src + (size_t)ch * 8) : u32x4{0, 0, 0, 0};
  }
#pragma unroll
  for (int i = 0; i < KEEP; ++i) m = max_bits(m, keep[i]);
  if (on)
    for (int ch = lane + LANES * KEEP; ch < nchunk; ch += LANES)
      m = max_bits(m, ld16(src + (size_t)ch * 8));
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off, kWave));
  if (LANES > kWave) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kQThreads / kWave; ++w) m = max(m, part[w]);
  }
  if (!on) return;
  const float top = __uint_as_float(m << 16);
  if (lane == 0) scales[row] = top / 127.0f;
  const bool zero = m == 0 || m >= 0x7f80u;
  const Quotient q = quotient_of(top);
  int8_t* dst = codes + row * K;
#pragma unroll
  for (int i = 0; i < KEEP; ++i) {
    const int ch = lane + LANES * i;
    if (ch < nchunk)
      *reinterpret_cast<uint2*>(dst + (size_t)ch * 8) = zero ? uint2{0u, 0u} : codes8(keep[i], q);
  }
  for (int ch = lane + LANES * KEEP; ch < nchunk; ch += LANES)
    *reinterpret_cast<uint2*>(dst + (size_t)ch * 8) =
        zero ? uint2{0u, 0u} : codes8(ld16(src + (size_t)ch * 8), q);
}

// Rows of a plan (one wave each) from the act of the up GEMM.  Rows that hold no real entry
// are skipped.  127 v and the quotient round once each in fp32, which moves a code by one only
// where 127 v / a lies within 127 * 2^-23 of a border.
__global__ __launch_bounds__(kQThreads) void i8_act_kernel(
    const float* __restrict__ act, int64_t rows, int I, const int32_t* __restrict__ plan,
    const int32_t* __restrict__ num_padded, int n_ids, int8_t* __restrict__ codes,
    float* __restrict__ scales) {
  constexpr int KEEP = 4;       // 8-value chunks per lane kept in registers (I <= 2048)
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * (kQThreads / kWave) + (threadIdx.x >> 6);
  if (row >= *num_padded || (uint32_t)plan[row] >= (uint32_t)n_ids) return;
  const int nchunk = I >> 3;
  struct Chunk {
    u32x4 lo, hi;
  };
  auto load = [&](int ch) {
    const float* v = act + ((ch >> 4) * rows + row) * 128 + (ch & 15) * 8;
    return Chunk{ld16(v), ld16(v + 4)};
  };
  auto largest = [](uint32_t m, const Chunk& v) {   // magnitudes' bits order as they do
#pragma unroll
    for (int j = 0; j < 4; ++j) m = max(m, max(v.lo[j] & 0x7fffffffu, v.hi[j] & 0x7fffffffu));
    return m;
  };
  Chunk keep[KEEP];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < KEEP; ++i) {
    const int ch = lane + kWave * i;
    keep[i] = ch < nchunk ? load(ch) : Chunk{u32x4{0, 0, 0, 0}, u32x4{0, 0, 0, 0}};
  }
#pragma unroll
  for (int i = 0; i < KEEP; ++i) m = largest(m, keep[i]);
  for (int ch = lane + kWave * KEEP; ch < nchunk; ch += kWave) m = largest(m, load(ch));
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off, kWave));
  const float top = __uint_as_float(m);
  const bool bad = m >= 0x7f800000u;   // an infinity or a NaN
  if (lane == 0) scales[row] = bad ? __uint_as_float(0x7fc00000u) : top / 127.0f;
  const bool zero = bad || m == 0;
  const Quotient q = quotient_of(top);
  auto put = [&](int ch, const Chunk& v) {
    uint2 c = {0u, 0u};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      c.x |= code_of(__uint_as_float(v.lo[j]), q) << (8 * j);
      c.y |= code_of(__uint_as_float(v.hi[j]), q) << (8 * j);
    }
    *reinterpret_cast<uint2*>(codes + row * I + (size_t)ch * 8) = zero ? uint2{0u, 0u} : c;
  };
#pragma unroll
  for (int i = 0; i < KEEP; ++i)
    if (lane + kWave * i < nchunk) put(lane + kWave * i, keep[i]);
  for (int ch = lane + kWave * KEEP; ch < nchunk; ch += kWave) put(ch, load(ch));
}

}  // namespace

hipError_t launch_i8_act(const float* act, int64_t rows, int I, const int32_t* plan,
                         const int32_t* num_padded, int n_ids, int8_t* codes, float* scales,
                         hipStream_t s) {
  const dim3 grid((unsigned)((rows + 3) / 4));
  hipLaunchKernelGGL(i8_act_kernel, grid, dim3(kQThreads), 0, s, act, rows, I, plan,
                     num_padded, n_ids, codes, scales);
  return hipGetLastError();
}

hipError_t launch_i8_rows(const uint16_t* v, int64_t rows, int K, int8_t* codes,
                          float* scales, hipStream_t s) {
  // a wave per row up to 2048 values (4 chunks a lane), a workgroup per longer row
  const bool wave_rows = K <= 2048;
  const int per = wave_rows ? kQThreads / kWave : 1;
  const int64_t most = (int64_t)per << 23;   // rows of one launch: 2^31 threads
  for (int64_t r0 = 0; r0 < rows; r0 += most) {
    const int64_t n = rows - r0 < most ? rows - r0 : most;
    const dim3 grid((unsigned)((n + per - 1) / per));
    if (wave_rows)
      hipLaunchKernelGGL((i8_rows_kernel<kWave, 4>), grid, dim3(kQThreads), 0, s, v, r0, rows, K,
                         codes, scales);
    else
      hipLaunchKernelGGL((i8_rows_kernel<kQThreads, 4>), grid, dim3(kQThreads), 0, s, v, r0, rows,
                         K, codes, scales);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace moe
