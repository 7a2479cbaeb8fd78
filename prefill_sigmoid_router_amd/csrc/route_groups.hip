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
#include <type_traits>

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

// Logits of a token: fp64 keys, the caller's fp32 logits, or fp32 MFMA partial logits with
// their |x| . |w| sums (router_logits_mfma_kernel), which bound their error.
struct KeySource {
  const double* keys;
  int64_t ld;
  __device__ void get(int64_t t, int e, double& l, double& d) const {
    l = keys[t * ld + e];
    d = 0.0;
  }
};
struct LogitSource {
  const float* logits;
  int64_t ld;
  __device__ void get(int64_t t, int e, double& l, double& d) const {
    l = (double)logits[t * ld + e];
    d = 0.0;
  }
};
struct BoundedSource {
  const float *logits, *absdot;
  const uint16_t *x, *wr;
  int parts, M, H;
  double rel;   // error of a partial logit over its |x| . |w| sum
  int64_t ld;
  __device__ void get(int64_t t, int e, double& l, double& d) const {
    double a = 0.0;
    l = 0.0;
    for (int p = 0; p < parts; ++p) {
      l += (double)logits[((int64_t)p * M + t) * ld + e];
      a += (double)absdot[((int64_t)p * M + t) * ld + e];
    }
    d = a * rel + fabs(l) * 0x1p-50 + (double)H * 0x1p-126 + 1e-300;
  }
};

// fp64 dot products of row t of x with rows e0 and e1 of the router weight, by one wave; the
// same order for every expert, so that equal rows give equal sums.
__device__ __forceinline__ void exact_logits(const BoundedSource& q, int64_t t, int e0, int e1,
                                             int lane, double& l0, double& l1) {
  const uint16_t* xr = q.x + t * q.H;
  const uint16_t* w0 = q.wr + (size_t)e0 * q.H;
  const uint16_t* w1 = q.wr + (size_t)e1 * q.H;
  double a0 = 0.0, a1 = 0.0;
  for (int c = lane; c < (q.H >> 3); c += kWave) {
    const u32x4 xv = ld16(xr + (size_t)c * 8), v0 = ld16(w0 + (size_t)c * 8), v1 = ld16(w1 + (size_t)c * 8);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const double lo = bf16lo(xv[j]), hi = bf16hi(xv[j]);
      a0 = fma(lo, (double)bf16lo(v0[j]), a0);
      a0 = fma(hi, (double)bf16hi(v0[j]), a0);
      a1 = fma(lo, (double)bf16lo(v1[j]), a1);
      a1 = fma(hi, (double)bf16hi(v1[j]), a1);
    }
  }
  l0 = wave_sum(a0);
  l1 = wave_sum(a1);
}

// LDS of a wave: c of E experts (and its bound), the picks' scores (values, bounds) and ids.
__host__ __device__ constexpr int select_lds_doubles(bool bounds, int E, int top_k) {
  return bounds ? 2 * E + 3 * top_k + (top_k + 1) / 2 : E + top_k + (top_k + 1) / 2;
}

// One wave per token; lane l owns experts l, l + 64, ... (SL of them).
//
// With bounded logits |l - exact| <= d, every value that a choice compares carries a bound of
// its own (sigmoid: s (1 - s) (e^d - 1) <= 1.2 d s (1 - s) for d <= 1/4; softmax without its
// common divisor: 1.2 d e^l), and a choice stands if no bound can turn it.  Where one can,
// the experts that it hangs on get their exact logits and the token is done again; choices
// between exact values are exact, so this ends.  At M=2048, E=256 about one token in five
// comes to two or three exact logits (recomputing every candidate's: seventeen for each).
template <int SL, typename SRC>
__global__ __launch_bounds__(kSelWaves* kWave) void select_groups_kernel(
    SRC src, const float* __restrict__ bias, int M, int E, int top_k, GroupRule rule,
    int32_t* __restrict__ ids, float* __restrict__ weights) {
  constexpr bool BOUNDS = std::is_same<SRC, BoundedSource>::value;
  extern __shared__ double sel_lds[];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * kSelWaves + wave;
  if (t >= M) return;
  double* s_c = sel_lds + (size_t)wave * select_lds_doubles(BOUNDS, E, top_k);
  double* s_d = s_c + E;                                   // BOUNDS
  double* s_pick = s_c + (BOUNDS ? 2 : 1) * E;
  double* s_pv = s_pick + top_k;                           // BOUNDS: the picks' values
  double* s_pd = s_pv + top_k;                             // BOUNDS: and their bounds
  int* s_id = reinterpret_cast<int*>(s_pick + (BOUNDS ? 3 : 1) * top_k);   // and the picks

  double l[SL], d[SL];
  uint32_t redo = 0;   // bit s: this lane's expert in slot s gets its exact logit
#pragma unroll
  for (int s = 0; s < SL; ++s) {
    const int e = lane + kWave * s;
    l[s] = -INFINITY;
    d[s] = 0.0;
    if (e < E) src.get(t, e, l[s], d[s]);
    if (BOUNDS && !(d[s] <= 0.25)) redo |= 1u << s;        // too wide, or not a number
  }

  for (;;) {
    if constexpr (BOUNDS) {
#pragma unroll
      for (int s = 0; s < SL; ++s) {
        uint64_t todo = __ballot((redo >> s) & 1);
        while (todo) {
          const int a = __ffsll((unsigned long long)todo) - 1;
          todo &= todo - 1;
          const int b = todo ? __ffsll((unsigned long long)todo) - 1 : a;
          todo &= todo ? todo - 1 : 0;
          double la, lb;
          exact_logits(src, t, a + kWave * s, b + kWave * s, lane, la, lb);
          if (lane == a || lane == b) {
            l[s] = lane == a ? la : lb;
            d[s] = 0.0;
          }
        }
      }
      redo = 0;
    }
    // scores (softmax with bounds: without the divisor, which is applied at the end)
    double score[SL], c[SL], dc[SL], divisor = 1.0;
    bool live[SL];
#pragma unroll
    for (int s = 0; s < SL; ++s) live[s] = l[s] > -INFINITY;
    if (rule.softmax) {
      double top = -INFINITY;
#pragma unroll
      for (int s = 0; s < SL; ++s)
        if (live[s]) top = fmax(top, l[s]);
      top = fmin(wave_max_f64(top), 1.7976931348623157e308);   // +inf counts as the largest number
      double total = 0.0;
#pragma unroll
      for (int s = 0; s < SL; ++s) {
        score[s] = live[s] ? exp(fmin(l[s], 1.7976931348623157e308) - top) : 0.0;
        total += score[s];
        dc[s] = 1.2 * d[s] * score[s];
      }
      divisor = wave_sum(total);
      if (!BOUNDS) {
#pragma unroll
        for (int s = 0; s < SL; ++s) score[s] = live[s] ? score[s] / divisor : 0.0;
        divisor = 1.0;
      }
    } else {
#pragma unroll
      for (int s = 0; s < SL; ++s) {
        const double ex = exp(-l[s]);
        score[s] = live[s] ? 1.0 / (1.0 + ex) : 0.0;
        dc[s] = d[s] > 0.0 ? 1.2 * d[s] * score[s] * fmin(1.0, ex * score[s]) + 1e-14 : 0.0;
      }
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
        dc[s] = 0.0;
      }
    }

    uint64_t stay = ~0ull;   // bit g: group g stays
    if (rule.n_group > 1) {
#pragma unroll
      for (int s = 0; s < SL; ++s)
        if (lane + kWave * s < E) {
          s_c[lane + kWave * s] = c[s];
          if (BOUNDS) s_d[lane + kWave * s] = dc[s];
        }
      wave_lds_fence();
      // span lanes (a power of two) read a group's experts and join their two best; lane
      // g span ends up with group g
      int span = 1;
      while (span * 2 * rule.n_group <= kWave) span *= 2;
      const int g = lane / span, sub = lane % span;
      const bool mine = g < rule.n_group;
      double b1 = -INFINITY, b2 = -INFINITY;   // best two c
      double h1 = -INFINITY, h2 = -INFINITY;   // best two c + dc
      double w1 = -INFINITY, w2 = -INFINITY;   // best two c - dc
      auto join = [](double& p1, double& p2, double o1, double o2) {
        p2 = fmax(fmin(p1, o1), fmax(p2, o2));
        p1 = fmax(p1, o1);
      };
      if (mine)
        for (int j = sub; j < rule.per; j += span) {
          const double v = s_c[g * rule.per + j];
          join(b1, b2, v, -INFINITY);
          if (BOUNDS) {
            const double dv = s_d[g * rule.per + j];
            join(h1, h2, v + dv, -INFINITY);
            join(w1, w2, v - dv, -INFINITY);
          }
        }
      for (int off = 1; off < span; off <<= 1) {
        join(b1, b2, __shfl_xor(b1, off, kWave), __shfl_xor(b2, off, kWave));
        if (BOUNDS) {
          join(h1, h2, __shfl_xor(h1, off, kWave), __shfl_xor(h2, off, kWave));
          join(w1, w2, __shfl_xor(w1, off, kWave), __shfl_xor(w2, off, kWave));
        }
      }
      const bool two = rule.group_top == 2;
      const double total = two && b2 > -INFINITY ? b1 + b2 : b1;
      int rank = 0;
      for (int j = 0; j < rule.n_group; ++j) {
        const double o = __shfl(total, j * span, kWave);
        rank += (o > total || (o == total && j < g)) ? 1 : 0;
      }
      const bool keep = mine && rank < rule.topk_group;
      const uint64_t kept = __ballot(keep && sub == 0);
      stay = 0;
      for (int j = 0; j < rule.n_group; ++j) stay |= ((kept >> (j * span)) & 1) << j;
      if (BOUNDS && rule.topk_group < rule.n_group) {
        const double top = two && h2 > -INFINITY ? h1 + h2 : h1;
        const double low = two && w2 > -INFINITY ? w1 + w2 : w1;
        const double least = -wave_max_f64(keep ? -low : -INFINITY);
        const double most = wave_max_f64(mine && !keep ? top : -INFINITY);
        if (!(least > most)) {   // a group's place is open: exact logits of what makes it
          const bool open = mine && (keep ? low <= most : top >= least);
          wave_lds_fence();      // s_c, s_d were read
          if (sub == 0 && mine) s_c[g] = open ? (two ? w2 : w1) : INFINITY;
          wave_lds_fence();
#pragma unroll
          for (int s = 0; s < SL; ++s) {
            const int e = lane + kWave * s;
            if (e < E && d[s] > 0.0 && live[s] && c[s] + dc[s] >= s_c[e / rule.per]) redo |= 1u << s;
          }
          wave_lds_fence();
          if (__any(redo != 0)) continue;
        }
      }
    }

    uint64_t key[SL];
    double v[SL], dv[SL];   // what orders the picks, and its bound
#pragma unroll
    for (int s = 0; s < SL; ++s) {
      const int e = lane + kWave * s;
      v[s] = bias ? c[s] : l[s];
      dv[s] = bias ? dc[s] : d[s];
      key[s] = kKeyOutside;
      if (e < E && ((stay >> (e / rule.per)) & 1)) key[s] = live[s] ? order_key(v[s]) : kKeyUnscored;
    }
    uint32_t inside = 0, taken = 0;
#pragma unroll
    for (int s = 0; s < SL; ++s) inside |= (uint32_t)(key[s] > kKeyUnscored) << s;
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
        double sc = score[0], pv = v[0], pd = dv[0];
#pragma unroll
        for (int s = 0; s < SL; ++s)
          if (s == slot) {
            sc = score[s];
            pv = v[s];
            pd = dv[s];
            key[s] = kKeyTaken;
            taken |= 1u << s;
          }
        s_id[r] = lane + kWave * slot;
        s_pick[r] = sc;
        if (BOUNDS) {
          s_pv[r] = best > kKeyUnscored ? pv : -INFINITY;
          s_pd[r] = best > kKeyUnscored ? pd : 0.0;
        }
      }
    }
    wave_lds_fence();
    if constexpr (BOUNDS) {
      // what is left: the largest value that bounded logits can reach, the largest exact one
      double reach = -INFINITY, exact = -INFINITY;
#pragma unroll
      for (int s = 0; s < SL; ++s)
        if ((inside & ~taken) >> s & 1) {
          if (d[s] > 0.0) reach = fmax(reach, v[s] + dv[s]);
          else exact = fmax(exact, v[s]);
        }
      reach = wave_max_f64(reach);
      exact = wave_max_f64(exact);
      // pick r stands if it is above all behind it (or exact, and so are those it is not above)
      double low = INFINITY, high = -INFINITY;   // hull of the picks that do not stand
      for (int r = lane; r < top_k; r += kWave) {
        const double pv = s_pv[r], pd = s_pd[r];
        double hb = reach, eb = exact;
        for (int j = r + 1; j < top_k; ++j) {
          if (s_pd[j] > 0.0) hb = fmax(hb, s_pv[j] + s_pd[j]);
          else eb = fmax(eb, s_pv[j]);
        }
        if (pv > -INFINITY && (pv - pd <= hb || (pd > 0.0 && pv - pd <= eb))) {
          low = fmin(low, pv - pd);
          high = fmax(high, pv + pd);
        }
      }
      low = -wave_max_f64(-low);
      high = wave_max_f64(high);
      if (low <= high) {
#pragma unroll
        for (int s = 0; s < SL; ++s)
          if ((inside >> s & 1) && d[s] > 0.0 && v[s] + dv[s] >= low && v[s] - dv[s] <= high)
            redo |= 1u << s;
        wave_lds_fence();
        if (__any(redo != 0)) continue;
      }
    }
    double factor = (double)rule.scale / divisor;
    if (rule.renorm) {
      double total = 0.0;
      for (int r = lane; r < top_k; r += kWave) total += s_pick[r];
      total = wave_sum(total);
      factor = total > 0.0 ? (double)rule.scale / total : 0.0;
    }
    for (int r = lane; r < top_k; r += kWave) {
      ids[t * top_k + r] = s_id[r];
      weights[t * top_k + r] = s_pick[r] > 0.0 ? (float)(s_pick[r] * factor) : 0.0f;
    }
    return;
  }
}

template <int SL, typename SRC>
hipError_t launch_select_sl(const SRC& src, const float* bias, int M, int E, int top_k,
                            const GroupRule& rule, int32_t* ids, float* w, hipStream_t s) {
  constexpr bool BOUNDS = std::is_same<SRC, BoundedSource>::value;
  const size_t lds = (size_t)kSelWaves * select_lds_doubles(BOUNDS, E, top_k) * sizeof(double);
  const dim3 grid((unsigned)((M + kSelWaves - 1) / kSelWaves));
  hipLaunchKernelGGL((select_groups_kernel<SL, SRC>), grid, dim3(kSelWaves* kWave), lds, s, src, bias,
                     M, E, top_k, rule, ids, w);
  return hipGetLastError();
}

template <typename SRC>
hipError_t launch_select(const SRC& src, const float* bias, int M, int E, int top_k,
                         const GroupRule& rule, int32_t* ids, float* w, hipStream_t s) {
  if (E <= 64) return launch_select_sl<1>(src, bias, M, E, top_k, rule, ids, w, s);
  if (E <= 128) return launch_select_sl<2>(src, bias, M, E, top_k, rule, ids, w, s);
  if (E <= 256) return launch_select_sl<4>(src, bias, M, E, top_k, rule, ids, w, s);
  if (E <= 512) return launch_select_sl<8>(src, bias, M, E, top_k, rule, ids, w, s);
  if constexpr (!std::is_same<SRC, BoundedSource>::value)
    return launch_select_sl<16>(src, bias, M, E, top_k, rule, ids, w, s);
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_route_logits(const float* logits, int64_t ld, const float* bias, int M, int E,
                               int top_k, const GroupRule& rule, int32_t* ids, float* w,
                               hipStream_t s) {
  return launch_select(LogitSource{logits, ld}, bias, M, E, top_k, rule, ids, w, s);
}

// From this many tokens on bounded fp32 MFMA logits replace fp64 ones for every (token,
// expert).  Not for softmax scores with a bias, whose choices hang on the divisor and so on
// every expert's exact logit, for more experts than 512 (registers), or where a pick of
// nearly all experts leaves most choices open.
constexpr int kBoundedMinTokens = 256, kBoundedMaxExperts = 512;

hipError_t launch_route_groups(const uint16_t* x, const uint16_t* wr, const float* bias, int M,
                               int H, int E, int top_k, const GroupRule& rule, int32_t* ids,
                               float* w, void* scratch, hipStream_t s) {
  if (M >= kBoundedMinTokens && E <= kBoundedMaxExperts && top_k <= 64 && !(rule.softmax && bias)) {
    int parts = 0, nround = 0;
    float* logits = static_cast<float*>(scratch);
    float* absdot = nullptr;
    const hipError_t err = launch_router_logits(x, wr, M, H, E, logits, &absdot, &parts, &nround, s);
    if (err != hipSuccess) return err;
    const double rel = (double)nround * 0x1p-23 * (1.0 + 0x1p-9);
    return launch_select(BoundedSource{logits, absdot, x, wr, parts, M, H, rel, E}, bias, M, E,
                         top_k, rule, ids, w, s);
  }
  double* keys = static_cast<double*>(scratch);
  const hipError_t err = launch_router_keys(x, wr, M, H, E, keys, s);
  if (err != hipSuccess) return err;
  return launch_select(KeySource{keys, E}, bias, M, E, top_k, rule, ids, w, s);
}

}  // namespace moe
