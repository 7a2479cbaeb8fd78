// The whole routed-MoE layer for a few tokens in two kernels.
//
// few_logits_kernel: l[t, e] = x[t] . Wr[e] (+ bias[e]) in fp64, a workgroup per expert; others
// mark the values that the second kernel hands over as not there yet.
//
// few_layer_kernel: everything else, as one queue of work items that persistent workgroups draw
// from by a ticket: all up items, then all down items, then one item per token that joins its
// picks.  Every workgroup first selects the experts of all tokens for itself (a wave per token)
// and lists the touched experts with their rows; that costs less than a hand-over would.
//   up    act[i, c] = silu(x . W13[e, c]) * (x . W13[e, I + c]) for 32 columns of an expert (URG = 2: 64)
//   down  y[i, h] = act[i] . W2[e, h] for 64 of its rows (DRG = 2: 128)
//   join  z = sum_j w_j y[t k + j] + residual, out = z * (mean z^2 + eps)^-1/2 * norm_w
// At a few tokens an expert has few rows, so the layer is a stream of its weights (M=8, H=7168,
// I=2048, k=16: 8 to 9 GB) and the arithmetic is small: no LDS ring and no MFMA tile, but dot
// products straight from the load registers.  A load is 8 weight rows x one 128-byte line,
// nontemporal; a wave keeps 16 to 24 KiB of them in flight and runs on by itself, without a
// barrier, to the end of its rows: M=8 1.24 to 1.38 ms for the 92 to 101 experts that it touches
// (6.2 to 6.6 TB/s; a plain read reaches 7.1), M=1 222 us (6.4).  Small layers are a chain of
// latencies and too few items for the CUs: H=2048, I=1408, 4 of 60 experts, one token 26.5 us, of which
// 10 are its bytes.  The tokens' rows (x in bf16, act in fp32) lie in LDS.  act and y stay in fp32 at all
// times, so the layer rounds only its outputs.
//
// An expert's weights are read once for each group of up to 8 of its rows (fewer where the LDS does not
// hold 8: from H > 8192 or I > 4096 on), so several tokens per expert cost more than the bytes: 16
// tokens, 8 of 16 experts, H=7168, I=2048 read 2.0 GB for 1.4 (380 us, where 199 would do), 2 of 8,
// H=4096, I=14336 6.3 for 2.8 (953 us and 397).
//
// Hand-overs: act and y are written and read past the XCDs' L2s (agent-scope accesses) and carry
// their own flag: a word that has not been written holds kNotThere, a NaN that no result is stored
// as, and whoever needs it loads again until it has gone.  (With a counter that is raised once the
// stores have arrived a hand-over took three trips to memory more, 3 us.)  An item only waits for
// items of lower tickets, tickets are handed out in order, and a workgroup holds at most the item
// that it works on and the next one: the unfinished item with the lowest ticket is always being
// worked on and never waits, so every wait ends, however many workgroups run at once and whatever
// else runs on the GPU.  A wave's polls in a call are bounded all the same, so that calls that share a
// workspace at the same time end too (with results that mean nothing, NaN among them).  They are
// counted and not timed: a clock runs on while the queue is suspended, and a wait that it ends may have
// had its producer suspended with it.
#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "launchers.h"
#include "wave_ops.h"

namespace moe {

namespace {

constexpr int kThreads = 512, kWaves = kThreads / kWave;
constexpr int kUnit = 64;             // K values of a load: 8 lanes x 8
constexpr int kStage = 128 * 1024;    // LDS for the tokens' rows
constexpr int kGroupRows = 8;         // rows of an expert that an item takes, at most

constexpr uint32_t kNotThere = 0xffffffffu;
// Polls of a wave in a call, a sleep of 512 cycles and a trip past the L2s each: seconds of the wave's
// own time, where no call takes one.
constexpr int kPolls = 1 << 22;

// Two products of bf16 pairs added to c.
__device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float c) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, a), __builtin_bit_cast(bf16x2, b),
                                         c, false);
}

// A result for another workgroup.
__device__ __forceinline__ void hand_over(float* p, float v) {
  const uint32_t b = __float_as_uint(v);
  __hip_atomic_store(reinterpret_cast<uint32_t*>(p), b == kNotThere ? 0x7fc00000u : b, __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}

#ifdef __HIP_DEVICE_COMPILE__   // the host pass knows no buffer descriptors
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const float* base) {
  const uint64_t b = (uint64_t)base;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)b);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)(b >> 32));
  return __builtin_amdgcn_make_buffer_rsrc((void*)((uint64_t)hi << 32 | lo), 0, -1, 0x00020000);
}
// N times 4 values that other workgroups hand over, at byte offsets off[]; -1: none (zeros).  All
// are asked for at once, and those with a word that is not there again, as long as the wave has polls
// left.
constexpr int kAgentScope = 16;   // cache policy bit SC1
template <int N>
__device__ __forceinline__ void take(__amdgpu_buffer_rsrc_t from, const int (&off)[N], f32x4 (&v)[N],
                                     int& polls) {
  u32x4 w[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    w[i] = u32x4{0, 0, 0, 0};
    if (off[i] >= 0) w[i] = __builtin_amdgcn_raw_buffer_load_b128(from, off[i], 0, kAgentScope);
  }
  auto missing = [](u32x4 a) {
    return a[0] == kNotThere || a[1] == kNotThere || a[2] == kNotThere || a[3] == kNotThere;
  };
  bool some = false;
#pragma unroll
  for (int i = 0; i < N; ++i) some |= missing(w[i]);
  if (__any(some)) {
    do {
      __builtin_amdgcn_s_sleep(8);
      some = false;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (missing(w[i])) w[i] = __builtin_amdgcn_raw_buffer_load_b128(from, off[i], 0, kAgentScope);
        some |= missing(w[i]);
      }
    } while (__any(some) && --polls > 0);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __builtin_bit_cast(f32x4, w[i]);
}
#endif

// LDS writes are visible behind it; loads stay in flight.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Sum over the 8 lanes that hold a row's parts, in each of them.
__device__ __forceinline__ float sum8(float v) {
#define MOE_DPP_SUM(ctrl) \
  v += __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), ctrl, 0xf, 0xf, false))
  MOE_DPP_SUM(0xB1);   // quad_perm 1, 0, 3, 2
  MOE_DPP_SUM(0x4E);   // quad_perm 2, 3, 0, 1
  MOE_DPP_SUM(0x141);  // row_half_mirror
#undef MOE_DPP_SUM
  return v;
}

// MT tokens against one expert's gate row per workgroup: chunk c of 8 values goes to thread
// c mod 256, the threads' sums meet in a fixed order, so equal rows of Wr give equal logits.  The
// workgroups behind the experts' set act and y to kNotThere, the first one the ticket to 0.
constexpr int kFill = 256 * 64;   // bytes of a workgroup's
template <int MT>
__global__ __launch_bounds__(256) void few_logits_kernel(FewArgs p) {
  __shared__ double part[4][MT];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, e = blockIdx.x;
  if (e >= p.E) {
    const int64_t bytes = (int64_t)p.M * p.top_k * (p.I + p.H) * (int64_t)sizeof(float);   // act, then y
    const int64_t first = (int64_t)(e - p.E) * kFill;
#pragma unroll
    for (int i = 0; i < kFill / 4096; ++i) {
      const int64_t at = first + i * 4096 + tid * 16;
      if (at < bytes) st16(reinterpret_cast<char*>(p.act) + at, u32x4{kNotThere, kNotThere, kNotThere, kNotThere});
    }
    return;
  }
  if (e == 0 && tid == 0) *p.ticket = 0;
  const uint16_t* w = p.router_w + (size_t)e * p.H;
  double acc[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) acc[t] = 0.0;
  const int chunks = p.H >> 3;
  constexpr int PRE = MT <= 4 ? 4 : 2;
  for (int c0 = tid; c0 < chunks; c0 += 256 * PRE) {
    u32x4 wv[PRE], xv[PRE][MT];
#pragma unroll
    for (int q = 0; q < PRE; ++q) {
      const int c = c0 + 256 * q;
      const bool in = c < chunks;
      wv[q] = in ? ld16(w + (size_t)c * 8) : u32x4{0, 0, 0, 0};
#pragma unroll
      for (int t = 0; t < MT; ++t)
        xv[q][t] = in && t < p.M ? ld16(p.x + (size_t)t * p.H + (size_t)c * 8) : u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int q = 0; q < PRE; ++q)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const double lo = bf16lo(wv[q][j]), hi = bf16hi(wv[q][j]);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          acc[t] = fma((double)bf16lo(xv[q][t][j]), lo, acc[t]);
          acc[t] = fma((double)bf16hi(xv[q][t][j]), hi, acc[t]);
        }
      }
  }
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const double s = wave_sum_f64(acc[t]);
    if (lane == 0) part[wave][t] = s;
  }
  __syncthreads();
  if (tid < MT && tid < p.M) {
    double l = ((part[0][tid] + part[1][tid]) + part[2][tid]) + part[3][tid];
    if (p.router_bias) l += (double)p.router_bias[e];
    p.keys[(size_t)tid * p.E + e] = l;
  }
}

// Logits and scores of lane l's experts l, l + 64, ... (SL of them); live: has a score.  `all`: scores
// of every expert, else only what a softmax's sum takes (top and total; sigmoid: nothing).
template <int SL>
__device__ __forceinline__ void load_logits(const FewArgs& p, int t, int lane, double (&l)[SL],
                                            bool (&live)[SL]) {
#pragma unroll
  for (int s = 0; s < SL; ++s) {
    const int e = lane + kWave * s;
    l[s] = e < p.E ? p.keys[(size_t)t * p.E + e] : -INFINITY;
    live[s] = l[s] > -INFINITY;   // (false for NaN)
    l[s] = live[s] ? fmin(l[s], 1.7976931348623157e308) : -INFINITY;
  }
}
struct Softmax {   // of a token: score = exp(l - top) / total
  double top, total;
};
template <int SL>
__device__ __forceinline__ Softmax softmax_of(const double (&l)[SL], const bool (&live)[SL]) {
  Softmax m{-INFINITY, 0.0};
#pragma unroll
  for (int s = 0; s < SL; ++s) m.top = fmax(m.top, l[s]);
  m.top = wave_max_f64(m.top);
#pragma unroll
  for (int s = 0; s < SL; ++s) {
    m.total += live[s] ? exp(l[s] - m.top) : 0.0;
    if (SL > 4) __builtin_amdgcn_sched_barrier(0);   // (16 at once do not fit the registers)
  }
  m.total = wave_sum_f64(m.total);
  return m;
}

// The picks of a token by a wave: ids[0 .. k) in LDS.  s_c: E doubles of LDS.  Scores are computed
// only if the choice hangs on them; the weights come later, beside the weights' stream.
template <int SL>
__device__ __forceinline__ void select_token(const FewArgs& p, int t, int lane, double* s_c, int* s_id) {
  const int E = p.E, k = p.top_k;
  const GroupRule& rule = p.rule;
  double c[SL];   // what orders the picks
  bool live[SL];
  load_logits(p, t, lane, c, live);
  uint64_t stay = ~0ull;   // bit g: group g stays
  if (p.select_bias || rule.topk_group < rule.n_group) {
    double l[SL];
#pragma unroll
    for (int s = 0; s < SL; ++s) l[s] = c[s];
    Softmax m{0.0, 1.0};
    if (rule.softmax) m = softmax_of(l, live);
#pragma unroll
    for (int s = 0; s < SL; ++s) {
      const double e = exp(rule.softmax ? l[s] - m.top : -l[s]);
      const int at = lane + kWave * s;
      c[s] = live[s] ? (rule.softmax ? e / m.total : 1.0 / (1.0 + e)) : -INFINITY;
      if (p.select_bias && at < E) c[s] += (double)p.select_bias[at];
      live[s] = live[s] && c[s] > -INFINITY;
      if (!live[s]) c[s] = -INFINITY;
      if (SL > 4) __builtin_amdgcn_sched_barrier(0);
    }
    if (rule.topk_group < rule.n_group) {
#pragma unroll
      for (int s = 0; s < SL; ++s)
        if (lane + kWave * s < E) s_c[lane + kWave * s] = c[s];
      wave_lds_fence();
      // span lanes (a power of two) read a group's experts and join their two best
      int span = 1;
      while (span * 2 * rule.n_group <= kWave) span *= 2;
      const int g = lane / span, sub = lane % span;
      const bool mine = g < rule.n_group;
      double b1 = -INFINITY, b2 = -INFINITY;
      if (mine)
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
      const double total = rule.group_top == 2 && b2 > -INFINITY ? b1 + b2 : b1;
      int rank = 0;
      for (int j = 0; j < rule.n_group; ++j) {
        const double o = __shfl(total, j * span, kWave);
        rank += (o > total || (o == total && j < g)) ? 1 : 0;
      }
      const uint64_t kept = __ballot(mine && sub == 0 && rank < rule.topk_group);
      stay = 0;
      for (int j = 0; j < rule.n_group; ++j) stay |= ((kept >> (j * span)) & 1) << j;
    }
    if (!p.select_bias) {   // without a bias the logits have the scores' order, also where scores tie
#pragma unroll
      for (int s = 0; s < SL; ++s) c[s] = l[s];
    }
  }
  uint64_t key[SL];
#pragma unroll
  for (int s = 0; s < SL; ++s) {
    const int e = lane + kWave * s;
    key[s] = kKeyOutside;
    if (e < E && ((stay >> (e * rule.per_magic >> 20)) & 1)) key[s] = live[s] ? order_key(c[s]) : kKeyUnscored;
  }
  // The k largest: a threshold with k values (rounded to fp32, which keeps their order) at or above
  // it, by bisection; then each one's rank among them.  Where none turns up in a fp32's bits
  // (values that round to the same, or fewer than k scored): pick by pick.
  if (k <= kWave) {
    float v[SL], low = INFINITY, high = -INFINITY;
#pragma unroll
    for (int s = 0; s < SL; ++s) {
      v[s] = key[s] > kKeyUnscored ? (float)c[s] : -INFINITY;
      if (v[s] > -INFINITY) low = fminf(low, v[s]);
      high = fmaxf(high, v[s]);
    }
    low = -wave_max_f32(-low);
    high = wave_max_f32(high);
    float least = low;
    int count = 0;
#pragma unroll 1
    for (int step = 0; step < 32; ++step) {   // (the first one asks whether all of them are k)
      count = 0;
#pragma unroll
      for (int s = 0; s < SL; ++s) count += __popcll(__ballot(v[s] >= least));
      if (count == k) break;
      if (count > k) low = least;
      else high = least;
      least = low + 0.5f * (high - low);
    }
    if (count == k) {
      uint64_t* const s_key = reinterpret_cast<uint64_t*>(s_c);   // k <= E keys
      int at = 0;
#pragma unroll
      for (int s = 0; s < SL; ++s) {
        const uint64_t who = __ballot(v[s] >= least);
        if (v[s] >= least) {
          const int r = at + __popcll(who & ((1ull << lane) - 1));
          s_key[r] = key[s];
          s_id[r] = lane + kWave * s;
        }
        at += __popcll(who);
      }
      wave_lds_fence();
      const uint64_t mine = s_key[min(lane, k - 1)];
      const int expert = s_id[min(lane, k - 1)];
      const uint32_t lo = (uint32_t)mine, hi = (uint32_t)(mine >> 32);
      int rank = 0;
      for (int r = 0; r < k; ++r) {
        const uint64_t o = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)hi, r) << 32 |
                           (uint32_t)__builtin_amdgcn_readlane((int)lo, r);
        const int id = __builtin_amdgcn_readlane(expert, r);
        rank += o > mine || (o == mine && id < expert) ? 1 : 0;
      }
      wave_lds_fence();
      if (lane < k) s_id[rank] = expert;
      return;
    }
  }
  for (int r = 0; r < k; ++r) {
    uint64_t best = key[0];
    int slot = 0;
#pragma unroll
    for (int s = 1; s < SL; ++s)
      if (key[s] > best) {
        best = key[s];
        slot = s;
      }
    if (lane == wave_best(best, slot, lane)) {
#pragma unroll
      for (int s = 0; s < SL; ++s)
        if (s == slot) key[s] = kKeyTaken;
      s_id[r] = lane + kWave * slot;
    }
  }
}

// The weights of a token's picks by a wave: w[0 .. k) in LDS.  s_c: k doubles of LDS.
template <int SL>
__device__ __forceinline__ void weigh_token(const FewArgs& p, int t, int lane, const int* s_id, double* s_c,
                                            float* s_w) {
  const GroupRule& rule = p.rule;
  Softmax m{0.0, 1.0};
  if (rule.softmax) {
    double l[SL];
    bool live[SL];
    load_logits(p, t, lane, l, live);
    m = softmax_of(l, live);
  }
  double picked = 0.0;   // sum of this lane's picks' scores
  for (int r = lane; r < p.top_k; r += kWave) {
    const int e = s_id[r];
    const double l = fmin(p.keys[(size_t)t * p.E + e], 1.7976931348623157e308);
    const double bias = p.select_bias ? (double)p.select_bias[e] : 0.0;
    double score = 0.0;
    if (l > -INFINITY) {   // (false for NaN)
      score = rule.softmax ? exp(l - m.top) / m.total : 1.0 / (1.0 + exp(-l));
      if (!(score + bias > -INFINITY)) score = 0.0;
    }
    s_c[r] = score;
    picked += score;
  }
  const double divisor = rule.renorm ? wave_sum(picked) : 1.0;
  for (int r = lane; r < p.top_k; r += kWave)
    s_w[r] = s_c[r] > 0.0 ? (float)(s_c[r] / divisor * (double)rule.scale) : 0.0f;
  wave_lds_fence();
}

// Dot products of a wave's 8 RG weight rows (lane: row lane / 8 of each group of 8, part lane % 8
// of a unit) with TT rows in LDS (stride ld values, zeros behind K up to a whole unit): sums over
// the lane's parts.  F32: the LDS rows are fp32 (act), else bf16 (x), whose products with bf16 are
// exact.  UB units are in flight.
template <int RG, int TT, bool F32>
struct Stream {
  static constexpr int UB = RG == 1 ? 16 : F32 ? 8 : 12;
  const uint16_t* row[RG];
  u32x4 w[UB][RG];
  int K, part;

  __device__ void load(int b, int u) {
#pragma unroll
    for (int g = 0; g < RG; ++g)
      w[b][g] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(row[g] + (size_t)u * kUnit));
  }
  __device__ void load_tail(int b, int u) {   // unit u, if there is one, zeros behind K
#pragma unroll
    for (int g = 0; g < RG; ++g) {
      w[b][g] = u32x4{0, 0, 0, 0};
      if (u * kUnit + 8 * part < K)
        w[b][g] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(row[g] + (size_t)u * kUnit));
    }
  }
  __device__ void begin() {
#pragma unroll
    for (int b = 0; b < UB; ++b) load_tail(b, b);
  }
  __device__ void use(int b, int u, const unsigned char* lds, int ld, float (&acc)[RG][TT]) const {
    if constexpr (F32) {
      const float* x = reinterpret_cast<const float*>(lds) + u * kUnit + 8 * part;
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const f32x4 a = *reinterpret_cast<const f32x4*>(x + (size_t)t * ld);
        const f32x4 c = *reinterpret_cast<const f32x4*>(x + (size_t)t * ld + 4);
#pragma unroll
        for (int g = 0; g < RG; ++g) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            acc[g][t] = fmaf(bf16lo(w[b][g][q]), q < 2 ? a[2 * q] : c[2 * q - 4], acc[g][t]);
            acc[g][t] = fmaf(bf16hi(w[b][g][q]), q < 2 ? a[2 * q + 1] : c[2 * q - 3], acc[g][t]);
          }
        }
      }
    } else {
      const uint16_t* x = reinterpret_cast<const uint16_t*>(lds) + u * kUnit + 8 * part;
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const u32x4 a = ld16(x + (size_t)t * ld);
#pragma unroll
        for (int g = 0; g < RG; ++g)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            acc[g][t] = dot2(w[b][g][q], a[q], acc[g][t]);
      }
    }
  }
  __device__ void run(const unsigned char* lds, int ld, float (&acc)[RG][TT]) {
    const int units = (K + kUnit - 1) / kUnit, whole = K / kUnit;
    int u = 0;
    for (; u + 2 * UB <= whole; u += UB) {
#pragma unroll
      for (int b = 0; b < UB; ++b) {
        use(b, u + b, lds, ld, acc);
        load(b, u + UB + b);
      }
    }
    for (; u < units; u += UB) {
#pragma unroll
      for (int b = 0; b < UB; ++b) {
        if (u + b < units) use(b, u + b, lds, ld, acc);
        if (u + UB + b < units) load_tail(b, u + UB + b);
      }
    }
  }
};

struct FewShared {
  unsigned char stage[kStage];
  int ids[kFewMaxPicks];
  float w[kFewMaxPicks];      // of a join item's token
  uint32_t mask[1024];        // tokens that picked an expert
  int first[1024];            // its first row group
  int rows[kFewMaxPicks];     // flat indices t k + j, row group by row group
  int gexp[kFewMaxPicks], gfirst[kFewMaxPicks], gcount[kFewMaxPicks];   // row groups
  int scan[kWaves];
  int ticket;
  float sum[kWaves];
};

// The thread's index, computed with here: what hangs on it is not moved in front of the items' loop,
// where what all kinds of items need would take 2 us before the first one.
__device__ __forceinline__ int thread_here() {
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  return tid;
}

template <int RG, int TT>
__device__ __forceinline__ void up_item(const FewArgs& p, FewShared& s, int u, int tile) {
  const int tid = thread_here(), wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int r = lane >> 3, part = lane & 7;
  const int e = s.gexp[u], first = s.gfirst[u], count = s.gcount[u];
  const int c0 = tile * 32 * RG + wave * 4 * RG;
  Stream<RG, TT, false> st;
  st.K = p.H;
  st.part = part;
#pragma unroll
  for (int g = 0; g < RG; ++g) {
    const int half = RG / 2;
    const bool up = RG == 1 ? r >= 4 : g >= half;
    const int c = RG == 1 ? c0 + (r & 3) : c0 + 8 * (up ? g - half : g) + r;
    const size_t row = (size_t)e * 2 * p.I + (up ? p.I : 0) + min(c, p.I - 1);
    st.row[g] = p.w13 + row * p.H + 8 * part;
  }
  st.begin();
  // the rows' tokens, zeros behind H
  const int ld = (p.H + kUnit - 1) / kUnit * kUnit, per = ld / 8;
  for (int i = tid; i < count * per; i += kThreads) {
    const int t = i / per, c = i % per * 8;
    const u32x4 v = c < p.H ? ld16(p.x + (size_t)(s.rows[first + t] / p.top_k) * p.H + c) : u32x4{0, 0, 0, 0};
    st16(s.stage + ((size_t)t * ld + c) * 2, v);
  }
  lds_barrier();
  float acc[RG][TT];
#pragma unroll
  for (int g = 0; g < RG; ++g)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[g][t] = 0.0f;
  st.run(s.stage, ld, acc);
  // lane (r, t) stores the columns r of row t
  const int i = s.rows[first + min(part, count - 1)];
#pragma unroll
  for (int g = 0; g < (RG + 1) / 2; ++g) {
    float gate = 0.0f, up = 0.0f;
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const float a = sum8(acc[g][t]);
      const float b = RG == 1 ? __shfl_xor(a, 32, kWave) : sum8(acc[RG == 1 ? 0 : g + RG / 2][t]);
      if (part == t) {
        gate = a;
        up = b;
      }
    }
    const int c = RG == 1 ? c0 + r : c0 + 8 * g + r;
    if (part < count && c < p.I && (RG > 1 || r < 4))
      hand_over(p.act + (size_t)i * p.I + c, gate / (1.0f + expf(-gate)) * up);
  }
}

template <int RG, int TT>
__device__ __forceinline__ void down_item(const FewArgs& p, FewShared& s, int u, int tile, int& polls) {
  const int tid = thread_here(), wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int r = lane >> 3, part = lane & 7;
  const int e = s.gexp[u], first = s.gfirst[u], count = s.gcount[u];
  const int h0 = tile * 64 * RG + wave * 8 * RG;
  Stream<RG, TT, true> st;
  st.K = p.I;
  st.part = part;
#pragma unroll
  for (int g = 0; g < RG; ++g)
    st.row[g] = p.w2 + ((size_t)e * p.H + min(h0 + 8 * g + r, p.H - 1)) * p.I + 8 * part;
  st.begin();   // in flight during the wait
  const int ld = (p.I + kUnit - 1) / kUnit * kUnit, per = ld / 4;
#ifdef __HIP_DEVICE_COMPILE__
  const __amdgpu_buffer_rsrc_t act = buffer_of(p.act);
  for (int i0 = tid; i0 < count * per; i0 += 2 * kThreads) {
    int off[2];
    f32x4 v[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int i = i0 + q * kThreads, t = i / per, c = i % per * 4;
      off[q] = i < count * per && c < p.I ? (s.rows[first + t] * p.I + c) * 4 : -1;
    }
    take(act, off, v, polls);
#pragma unroll
    for (int q = 0; q < 2; ++q)
      if (i0 + q * kThreads < count * per)
        *reinterpret_cast<f32x4*>(s.stage + (size_t)(i0 + q * kThreads) * 16) = v[q];
  }
#endif
  lds_barrier();
  float acc[RG][TT];
#pragma unroll
  for (int g = 0; g < RG; ++g)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[g][t] = 0.0f;
  st.run(s.stage, ld, acc);
  const int i = s.rows[first + min(part, count - 1)];
#pragma unroll
  for (int g = 0; g < RG; ++g) {
    float v = 0.0f;
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const float a = sum8(acc[g][t]);
      if (part == t) v = a;
    }
    const int h = h0 + 8 * g + r;
    if (part < count && h < p.H) hand_over(p.y + (size_t)i * p.H + h, v);
  }
}

__device__ __forceinline__ void join_item(const FewArgs& p, FewShared& s, int t, int& polls) {
  const int tid = thread_here(), wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int k = p.top_k;
  if (wave == 0) {
    double* c = reinterpret_cast<double*>(s.stage);
    const int* ids = s.ids + t * k;
    if (p.E <= 64) weigh_token<1>(p, t, lane, ids, c, s.w);
    else if (p.E <= 256) weigh_token<4>(p, t, lane, ids, c, s.w);
    else if (p.E <= 512) weigh_token<8>(p, t, lane, ids, c, s.w);
    else weigh_token<16>(p, t, lane, ids, c, s.w);
    if (p.w_out)
      for (int j = lane; j < k; j += kWave) p.w_out[t * k + j] = s.w[j];
  }
  lds_barrier();
  float* const z = reinterpret_cast<float*>(s.stage);   // each thread's own values
  float sq = 0.0f;
#ifdef __HIP_DEVICE_COMPILE__
  const __amdgpu_buffer_rsrc_t y = buffer_of(p.y + (size_t)t * k * p.H);
  constexpr int B = 8, C = 2;   // picks and 4-value chunks in flight
  for (int h0 = 4 * tid; h0 < p.H; h0 += C * 4 * kThreads) {
    f32x4 m[C];
#pragma unroll
    for (int c = 0; c < C; ++c) m[c] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < k; j0 += B) {
      int off[B * C];
      f32x4 v[B * C];
#pragma unroll
      for (int j = 0; j < B; ++j)
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const int h = h0 + c * 4 * kThreads;
          off[j * C + c] = j0 + j < k && h < p.H ? ((j0 + j) * p.H + h) * 4 : -1;
        }
      take(y, off, v, polls);
#pragma unroll
      for (int j = 0; j < B; ++j) {
        if (j0 + j >= k) break;
        const float w = s.w[j0 + j];
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int q = 0; q < 4; ++q) m[c][q] = fmaf(w, v[j * C + c][q], m[c][q]);
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int h = h0 + c * 4 * kThreads;
      if (h >= p.H) break;
      if (p.residual) {
        const uint2 r = *reinterpret_cast<const uint2*>(p.residual + (size_t)t * p.H + h);
        m[c] += f32x4{bf16lo(r.x), bf16hi(r.x), bf16lo(r.y), bf16hi(r.y)};
      }
      if (p.residual_out)
        *reinterpret_cast<uint2*>(p.residual_out + (size_t)t * p.H + h) =
            make_uint2(cvt_bf16x2(m[c][0], m[c][1]), cvt_bf16x2(m[c][2], m[c][3]));
      *reinterpret_cast<f32x4*>(z + h) = m[c];
      sq += m[c][0] * m[c][0] + m[c][1] * m[c][1] + m[c][2] * m[c][2] + m[c][3] * m[c][3];
    }
  }
#endif
  if (!p.out) return;
  sq = wave_sum_f32(sq);
  if (lane == 0) s.sum[wave] = sq;
  lds_barrier();
  float total = 0.0f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) total += s.sum[w];
  const float f = 1.0f / sqrtf(total / (float)p.H + p.eps);
  for (int h = 4 * tid; h < p.H; h += 4 * kThreads) {
    const f32x4 v = *reinterpret_cast<const f32x4*>(z + h);
    const uint2 g = *reinterpret_cast<const uint2*>(p.norm_w + h);
    *reinterpret_cast<uint2*>(p.out + (size_t)t * p.H + h) =
        make_uint2(cvt_bf16x2(v[0] * f * bf16lo(g.x), v[1] * f * bf16hi(g.x)),
                   cvt_bf16x2(v[2] * f * bf16lo(g.y), v[3] * f * bf16hi(g.y)));
  }
}

template <int URG, int DRG>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2, 2))) void few_layer_kernel(
    FewArgs p) {
  __shared__ __align__(16) FewShared s;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int n = p.M * p.top_k, E = p.E;
  // One lane draws the tickets, of the wave with the fewest tokens to select for: the atomics of all
  // workgroups on one word take 2 us at the start.  The address is per lane for the compiler, which
  // else adds for the whole wave and waits for the sum at once.
  const bool draws = tid == kThreads - kWave;
  int apart = 0, next = 0;
  asm volatile("" : "+v"(apart));
  if (draws)
    next = __hip_atomic_fetch_add(p.ticket + apart, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  for (int e = tid; e < E; e += kThreads) s.mask[e] = 0;
  lds_barrier();
  for (int t = wave; t < p.M; t += kWaves) {
    const int lane = thread_here() & 63;
    double* c = reinterpret_cast<double*>(s.stage) + (size_t)wave * E;
    int* ids = s.ids + t * p.top_k;
    if (E <= 64) select_token<1>(p, t, lane, c, ids);
    else if (E <= 256) select_token<4>(p, t, lane, c, ids);
    else if (E <= 512) select_token<8>(p, t, lane, c, ids);
    else select_token<16>(p, t, lane, c, ids);
    wave_lds_fence();
    for (int j = lane; j < p.top_k; j += kWave) atomicOr(&s.mask[ids[j]], 1u << t);
    wave_lds_fence();   // c is the next token's
  }
  lds_barrier();
  // Row groups: the first token (in order) that picked an expert opens its groups, thread i for
  // the flat index i.  Sums of rows, and of groups in the upper half.
  const int e = tid < n ? s.ids[tid] : 0, t = tid / p.top_k;
  const uint32_t mask = tid < n ? s.mask[e] : 0;
  const bool opens = tid < n && (mask & ((1u << t) - 1)) == 0;
  const int count = opens ? __popc(mask) : 0, mine = (count + p.group_rows - 1) / p.group_rows;
  int scan = count + (mine << 16);
  const int sum = scan;
#define MOE_DPP_SCAN(ctrl, rows) scan += __builtin_amdgcn_update_dpp(0, scan, ctrl, rows, 0xf, false)
  MOE_DPP_SCAN(0x111, 0xf);   // row_shr 1, 2, 4, 8
  MOE_DPP_SCAN(0x112, 0xf);
  MOE_DPP_SCAN(0x114, 0xf);
  MOE_DPP_SCAN(0x118, 0xf);
  MOE_DPP_SCAN(0x142, 0xa);   // row_bcast 15 into rows 1 and 3
  MOE_DPP_SCAN(0x143, 0xc);   // row_bcast 31 into rows 2 and 3
#undef MOE_DPP_SCAN
  if (lane == kWave - 1) s.scan[wave] = scan;
  if (draws) s.ticket = next;
  lds_barrier();
  int before = scan - sum, all = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const int o = s.scan[w];
    before += w < wave ? o : 0;
    all += o;
  }
  if (opens) {
    s.first[e] = before & 0xffff;
    for (int q = 0; q < mine; ++q) {
      const int g = (before >> 16) + q;
      s.gexp[g] = e;
      s.gfirst[g] = (before & 0xffff) + q * p.group_rows;
      s.gcount[g] = min(p.group_rows, count - q * p.group_rows);
    }
  }
  lds_barrier();
  if (tid < n) {
    s.rows[s.first[e] + __popc(mask & ((1u << t) - 1))] = tid;
    if (blockIdx.x == 0 && p.ids_out) p.ids_out[tid] = e;
  }
  lds_barrier();
  const int groups = all >> 16;
  const int ups = groups * p.up_tiles, downs = groups * p.down_tiles;
  int polls = kPolls;
  for (;;) {
    const int item = s.ticket;
    lds_barrier();   // read by all, and the stage is free
    if (item >= ups + downs + p.M) break;
    if (draws)
      next = __hip_atomic_fetch_add(p.ticket + apart, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (item < ups) {
      const int u = item / p.up_tiles, tile = item % p.up_tiles, c = s.gcount[u];
      if (c <= 1) up_item<URG, 1>(p, s, u, tile);
      else if (c <= 2) up_item<URG, 2>(p, s, u, tile);
      else if (c <= 4) up_item<URG, 4>(p, s, u, tile);
      else up_item<URG, 8>(p, s, u, tile);
    } else if (item < ups + downs) {
      const int d = item - ups, u = d / p.down_tiles, tile = d % p.down_tiles, c = s.gcount[u];
      if (c <= 1) down_item<DRG, 1>(p, s, u, tile, polls);
      else if (c <= 2) down_item<DRG, 2>(p, s, u, tile, polls);
      else if (c <= 4) down_item<DRG, 4>(p, s, u, tile, polls);
      else down_item<DRG, 8>(p, s, u, tile, polls);
    } else {
      join_item(p, s, item - ups - downs, polls);
    }
    if (draws) s.ticket = next;
    lds_barrier();
  }
}

inline size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Rows of a group: as many as the stage holds of both kinds, a power of two.  I up to kMaxI (a larger
// row's bytes need not fit an int).
constexpr int kMaxI = kStage / (int)sizeof(float);
int group_rows(int H, int I) {
  const int row = std::max((H + kUnit - 1) / kUnit * kUnit * 2, (I + kUnit - 1) / kUnit * kUnit * 4);
  int g = kGroupRows;
  while (g > 0 && g * row > kStage) g /= 2;
  return g;
}

}  // namespace

bool few_sizes_ok(int H, int I) { return I <= kMaxI && group_rows(H, I) > 0; }

size_t few_scratch_bytes(int M, int H, int E, int I, int top_k) {
  return up256((size_t)M * E * sizeof(double)) + up256(sizeof(int)) +
         up256((size_t)M * top_k * (I + H) * sizeof(float));
}

hipError_t launch_few_layer(FewArgs a, void* scratch, hipStream_t s) {
  char* ws = static_cast<char*>(scratch);
  a.keys = reinterpret_cast<double*>(ws);
  ws += up256((size_t)a.M * a.E * sizeof(double));
  a.ticket = reinterpret_cast<int*>(ws);
  ws += up256(sizeof(int));
  const size_t picks = (size_t)a.M * a.top_k;
  a.act = reinterpret_cast<float*>(ws);
  a.y = a.act + picks * a.I;   // (I is a multiple of 16)
  a.group_rows = group_rows(a.H, a.I);
  const size_t fills = (picks * (a.I + a.H) * sizeof(float) + kFill - 1) / kFill;
  const dim3 experts((unsigned)(a.E + fills)), t256(256);
  if (a.M == 1) hipLaunchKernelGGL((few_logits_kernel<1>), experts, t256, 0, s, a);
  else if (a.M == 2) hipLaunchKernelGGL((few_logits_kernel<2>), experts, t256, 0, s, a);
  else if (a.M <= 4) hipLaunchKernelGGL((few_logits_kernel<4>), experts, t256, 0, s, a);
  else if (a.M <= 8) hipLaunchKernelGGL((few_logits_kernel<8>), experts, t256, 0, s, a);
  else hipLaunchKernelGGL((few_logits_kernel<16>), experts, t256, 0, s, a);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  int dev = 0, cus = 0;
  err = hipGetDevice(&dev);
  if (err == hipSuccess) err = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
  if (err != hipSuccess) return err;
  // Two groups of 8 rows per wave where an expert has several rows (4 picks per expert on average) and
  // every CU still gets an item: each read of a token's values from LDS then serves both.  16 tokens,
  // 8 of 16 experts, H = 7168, I = 2048: 351 us (to 380 from box to box), one group 410; 2 of 4 experts,
  // H = I = 4096: 136 and 150.  With few rows per expert small items spread better: 3 tokens, 6 of 64 experts, H = 4096,
  // I = 1536: 105 us, two groups 114; one token, 4 of 60, H = 2048, I = 1408: 26.6 and 33.4.  (Four
  // groups were never faster.)
  const long groups = std::min((long)a.M * a.top_k, (long)a.E);
  const bool shared = (long)a.M * a.top_k >= 4L * a.E;
  auto up = [&](int rg) { return (a.I + 32 * rg - 1) / (32 * rg); };
  auto down = [&](int rg) { return (a.H + 64 * rg - 1) / (64 * rg); };
  const int urg = shared && groups * up(2) >= cus ? 2 : 1;
  const int drg = shared && groups * down(2) >= cus ? 2 : 1;
  a.up_tiles = up(urg);
  a.down_tiles = down(drg);
  const long most = (long)a.M * a.top_k * std::max(a.up_tiles, a.down_tiles);
  const dim3 grid((unsigned)std::min<long>(cus, std::max<long>(most, a.M))), t(kThreads);
  auto kernel = urg == 2 ? (drg == 2 ? few_layer_kernel<2, 2> : few_layer_kernel<2, 1>)
                         : (drg == 2 ? few_layer_kernel<1, 2> : few_layer_kernel<1, 1>);
  hipLaunchKernelGGL(kernel, grid, t, 0, s, a);
  return hipGetLastError();
}

}  // namespace moe
