// Router with expert groups: sigmoid or softmax scores, a bias that is added for the
// selection only, the best groups, top-k inside them, weights from the unbiased scores.
//
//   l[e]  = x . Wr[e] (fp64 sums), or the caller's logits
//   s[e]  = 1 / (1 + exp(-l[e]))  or  exp(l[e]) / sum exp(l)
//   c[e]  = s[e] + b[e]
//   G[g]  = sum of the group_top (1 or 2) largest c of group g; the topk_group largest
//           groups stay, ties to the lower group
//   picks = the top_k largest c of the groups that stay, ties to the lower id (without a
//           bias the logits are compared: they have the scores' order, also where scores
//           round to the same number)
//   w     = s[pick] (/ sum over the picks) * scale
//
// An expert whose logit is -inf or not a number (or whose c is) has no score: weight 0, it
// adds nothing to its group, it is picked only after every scored expert of the groups that
// stay, in id order; a group without a scored expert comes after all others.  top_k never
// exceeds the experts of the groups that stay, so the picks are always distinct experts.
#include "device_common.h"
#include "launchers.h"

namespace moe {

namespace {

constexpr int kSelWaves = 4;   // tokens per workgroup: one wave each, no barriers

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

// One wave per token; lane l owns experts l, l + 64, ... (SL of them).
template <int SL, typename T>
__global__ __launch_bounds__(kSelWaves* kWave) void select_groups_kernel(
    const T* __restrict__ logits, int64_t ld, const float* __restrict__ bias, int M, int E,
    int top_k, GroupRule rule, int32_t* __restrict__ ids, float* __restrict__ weights) {
  extern __shared__ double sel_lds[];   // per wave: c of E experts, then the picks' scores
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * kSelWaves + wave;
  if (t >= M) return;
  double* s_c = sel_lds + (size_t)wave * (E + top_k);
  double* s_pick = s_c + E;

  double l[SL], score[SL], c[SL];
  bool live[SL];
#pragma unroll
  for (int s = 0; s < SL; ++s) {
    const int e = lane + kWave * s;
    l[s] = e < E ? (double)logits[t * ld + e] : -INFINITY;
    live[s] = l[s] > -INFINITY;
    if (!live[s]) l[s] = -INFINITY;
  }
  if (rule.softmax) {
    double top = -INFINITY, total = 0.0;
#pragma unroll
    for (int s = 0; s < SL; ++s) top = fmax(top, l[s]);
    top = wave_max_f64(top);
    if (top == INFINITY) top = 1.7976931348623157e308;   // +inf counts as the largest number
#pragma unroll
    for (int s = 0; s < SL; ++s) {
      score[s] = live[s] ? exp(fmin(l[s], 1.7976931348623157e308) - top) : 0.0;
      total += score[s];
    }
    total = wave_sum(total);
#pragma unroll
    for (int s = 0; s < SL; ++s) score[s] = live[s] ? score[s] / total : 0.0;
  } else {
#pragma unroll
    for (int s = 0; s < SL; ++s) score[s] = live[s] ? 1.0 / (1.0 + exp(-l[s])) : 0.0;
  }
#pragma unroll
  for (int s = 0; s < SL; ++s) {
    const int e = lane + kWave * s;
    c[s] = score[s];
    if (bias && e < E) c[s] += (double)bias[e];
    live[s] = live[s] && c[s] > -INFINITY;
    if (!live[s]) {
      c[s] = -INFINITY;
      score[s] = 0.0;
    }
  }

  uint64_t stay = ~0ull;   // bit g: group g stays
  if (rule.n_group > 1) {
#pragma unroll
    for (int s = 0; s < SL; ++s)
      if (lane + kWave * s < E) s_c[lane + kWave * s] = c[s];
    wave_lds_fence();
    // span lanes (a power of two) read a group's experts and join their two best; lane
    // g span ends up with group g
    int span = 1;
    while (span * 2 * rule.n_group <= kWave) span *= 2;
    const int g = lane / span, sub = lane % span;
    double b1 = -INFINITY, b2 = -INFINITY;
    if (g < rule.n_group)
      for (int j = sub; j < rule.per; j += span) {
        const double v = s_c[g * rule.per + j];
        b2 = fmax(b2, fmin(b1, v));
        b1 = fmax(b1, v);
      }
    for (int off = 1; off < span; off <<= 1) {
      const double o1 = __shfl_xor(b1, off, kWave), o2 = __shfl_xor(b2, off, kWave);
      b2 = fmax(fmin(b1, o1), fmax(b2, o2));
      b1 = fmax(b1, o1);
    }
    double total = b1;
    if (rule.group_top == 2 && b2 > -INFINITY) total += b2;
    if (g >= rule.n_group) total = -INFINITY;
    int rank = 0;
    for (int j = 0; j < rule.n_group; ++j) {
      const double o = __shfl(total, j * span, kWave);
      rank += (o > total || (o == total && j < g)) ? 1 : 0;
    }
    const uint64_t kept = __ballot(g < rule.n_group && sub == 0 && rank < rule.topk_group);
    stay = 0;
    for (int j = 0; j < rule.n_group; ++j) stay |= ((kept >> (j * span)) & 1) << j;
  }

  uint64_t key[SL];
#pragma unroll
  for (int s = 0; s < SL; ++s) {
    const int e = lane + kWave * s;
    key[s] = kKeyOutside;
    if (e < E && ((stay >> (e / rule.per)) & 1))
      key[s] = live[s] ? order_key(bias ? c[s] : l[s]) : kKeyUnscored;
  }
  for (int r = 0; r < top_k; ++r) {
    uint64_t best = key[0];
    int slot = 0;
#pragma unroll
    for (int s = 1; s < SL; ++s)
      if (key[s] > best) {
        best = key[s];
        slot = s;
      }
    if (lane == wave_best(best, slot, lane)) {
      double sc = score[0];
#pragma unroll
      for (int s = 0; s < SL; ++s)
        if (s == slot) {
          sc = score[s];
          key[s] = kKeyTaken;
        }
      ids[t * top_k + r] = lane + kWave * slot;
      s_pick[r] = sc;
    }
  }
  wave_lds_fence();
  double factor = (double)rule.scale;
  if (rule.renorm) {
    double total = 0.0;
    for (int r = lane; r < top_k; r += kWave) total += s_pick[r];
    total = wave_sum(total);
    factor = total > 0.0 ? factor / total : 0.0;
  }
  for (int r = lane; r < top_k; r += kWave) weights[t * top_k + r] = (float)(s_pick[r] * factor);
}

template <typename T>
hipError_t launch_select(const T* logits, int64_t ld, const float* bias, int M, int E, int top_k,
                         const GroupRule& rule, int32_t* ids, float* w, hipStream_t s) {
  const size_t lds = (size_t)kSelWaves * (E + top_k) * sizeof(double);
  constexpr int kMost = 1 << 24;   // tokens of one launch: 2^30 threads
  for (int t0 = 0; t0 < M; t0 += kMost) {
    const int n = M - t0 < kMost ? M - t0 : kMost;
    const dim3 grid((unsigned)((n + kSelWaves - 1) / kSelWaves));
    const T* lt = logits + t0 * ld;
    int32_t* it = ids + (size_t)t0 * top_k;
    float* wt = w + (size_t)t0 * top_k;
#define MOE_SELECT(SL)                                                                         \
  hipLaunchKernelGGL((select_groups_kernel<SL, T>), grid, dim3(kSelWaves* kWave), lds, s, lt, ld, \
                     bias, n, E, top_k, rule, it, wt)
    if (E <= 64) MOE_SELECT(1);
    else if (E <= 128) MOE_SELECT(2);
    else if (E <= 256) MOE_SELECT(4);
    else if (E <= 512) MOE_SELECT(8);
    else MOE_SELECT(16);
#undef MOE_SELECT
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    if (M - t0 <= kMost) break;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_route_logits(const float* logits, int64_t ld, const float* bias, int M, int E,
                               int top_k, const GroupRule& rule, int32_t* ids, float* w,
                               hipStream_t s) {
  return launch_select<float>(logits, ld, bias, M, E, top_k, rule, ids, w, s);
}

hipError_t launch_route_groups(const uint16_t* x, const uint16_t* wr, const float* bias, int M,
                               int H, int E, int top_k, const GroupRule& rule, int32_t* ids,
                               float* w, void* scratch, hipStream_t s) {
  double* keys = static_cast<double*>(scratch);
  const hipError_t err = launch_router_keys(x, wr, M, H, E, keys, s);
  if (err != hipSuccess) return err;
  return launch_select<double>(keys, E, bias, M, E, top_k, rule, ids, w, s);
}

}  // namespace moe
