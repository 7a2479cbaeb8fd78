// Reductions of a wave, and pieces of the routers' selections.
#pragma once

#include <math.h>

#include "device_common.h"

namespace moe {

// Largest v of the wave, in every lane (a scalar): DPP shifts inside rows of 16 lanes, then
// row broadcasts; lanes without a source contribute 0.
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
#define MOE_DPP_MAX(ctrl, rows) \
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, rows, 0xf, false))
  MOE_DPP_MAX(0x111, 0xf);  // row_shr 1, 2, 4, 8
  MOE_DPP_MAX(0x112, 0xf);
  MOE_DPP_MAX(0x114, 0xf);
  MOE_DPP_MAX(0x118, 0xf);
  MOE_DPP_MAX(0x142, 0xa);  // row_bcast 15 into rows 1 and 3
  MOE_DPP_MAX(0x143, 0xc);  // row_bcast 31 into rows 2 and 3
#undef MOE_DPP_MAX
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// The same for floats: largest and sum.
#define MOE_DPP_F32(v, old, ctrl, rows)                                                       \
  __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp((int)__float_as_uint(old),            \
                                                        (int)__float_as_uint(v), ctrl, rows, \
                                                        0xf, false))
__device__ __forceinline__ float scan_max_f32(float v) {
  v = fmaxf(v, MOE_DPP_F32(v, -INFINITY, 0x111, 0xf));
  v = fmaxf(v, MOE_DPP_F32(v, -INFINITY, 0x112, 0xf));
  v = fmaxf(v, MOE_DPP_F32(v, -INFINITY, 0x114, 0xf));
  v = fmaxf(v, MOE_DPP_F32(v, -INFINITY, 0x118, 0xf));
  v = fmaxf(v, MOE_DPP_F32(v, -INFINITY, 0x142, 0xa));
  v = fmaxf(v, MOE_DPP_F32(v, -INFINITY, 0x143, 0xc));
  return v;   // largest of the lanes up to this one
}
__device__ __forceinline__ float lane63(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}
__device__ __forceinline__ float wave_max_f32(float v) { return lane63(scan_max_f32(v)); }
__device__ __forceinline__ float wave_sum_f32(float v) {
  v += MOE_DPP_F32(v, 0.0f, 0x111, 0xf);
  v += MOE_DPP_F32(v, 0.0f, 0x112, 0xf);
  v += MOE_DPP_F32(v, 0.0f, 0x114, 0xf);
  v += MOE_DPP_F32(v, 0.0f, 0x118, 0xf);
  v += MOE_DPP_F32(v, 0.0f, 0x142, 0xa);
  v += MOE_DPP_F32(v, 0.0f, 0x143, 0xc);
  return lane63(v);
}
#undef MOE_DPP_F32

// Sum of a wave's doubles, in every lane, in a fixed order: DPP moves of both halves.
__device__ __forceinline__ double wave_sum_f64(double v) {
#define MOE_DPP_ADD(ctrl, rows)                                                              \
  {                                                                                          \
    const uint64_t b = (uint64_t)__double_as_longlong(v);                                    \
    const int lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, ctrl, rows, 0xf, false); \
    const int hi = __builtin_amdgcn_update_dpp(0, (int)(b >> 32), ctrl, rows, 0xf, false);   \
    v += __longlong_as_double((long long)((uint64_t)(uint32_t)hi << 32 | (uint32_t)lo));     \
  }
  MOE_DPP_ADD(0x111, 0xf)
  MOE_DPP_ADD(0x112, 0xf)
  MOE_DPP_ADD(0x114, 0xf)
  MOE_DPP_ADD(0x118, 0xf)
  MOE_DPP_ADD(0x142, 0xa)
  MOE_DPP_ADD(0x143, 0xc)
#undef MOE_DPP_ADD
  const uint64_t b = (uint64_t)__double_as_longlong(v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, 63);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), 63);
  return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}

__device__ __forceinline__ double wave_max_f64(double v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v = fmax(v, __shfl_xor(v, off, kWave));
  return v;
}

// LDS written by some lanes of a wave is read by others of the same wave: LDS operations of
// a wave complete in order, so only the compiler has to keep theirs.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Unsigned integers that order as the numbers do (v not a NaN; -0 counts as +0).  Keys of
// finite numbers and of infinities are above kKeyUnscored.
constexpr uint64_t kKeyTaken = 0, kKeyOutside = 0, kKeyUnscored = 1;
__device__ __forceinline__ uint64_t order_key(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
  return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

// The wave's largest (key, lowest id): id = lane + 64 slot.  Most rounds end after the
// upper 32 bits; equal upper halves compare the lower ones, equal keys the ids.
__device__ __forceinline__ int wave_best(uint64_t key, int slot, int lane) {
  const uint32_t hi = (uint32_t)(key >> 32);
  uint64_t who = __ballot(hi == wave_max_u32(hi));
  if (who & (who - 1)) {
    const bool in = (who >> lane) & 1;
    const uint32_t lo = in ? (uint32_t)key : 0u;
    who &= __ballot(lo == wave_max_u32(lo));
    if (who & (who - 1)) {
      const uint32_t rev = ((who >> lane) & 1) ? 0xFFFFu - (uint32_t)(lane + 64 * slot) : 0u;
      who = __ballot(rev == wave_max_u32(rev));
    }
  }
  return __ffsll((unsigned long long)who) - 1;
}

}  // namespace moe
