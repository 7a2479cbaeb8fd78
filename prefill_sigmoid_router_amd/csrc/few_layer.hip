// The whole routed-MoE layer for a few tokens in two kernels.
//
// few_logits_kernel: l[t, e] = x[t] . Wr[e] (+ bias[e]) in fp64, a workgroup per expert.  It also
// clears the counters that the second kernel works with.
//
// few_layer_kernel: everything else, as one queue of work items that persistent workgroups draw
// from by a ticket: all up items, then all down items, then one item per token that joins its
// picks.  Every workgroup first selects the experts of all tokens for itself (a wave per token)
// and lists the touched experts with their rows; that costs less than a hand-over would.
//   up    act[i, c] = silu(x . W13[e, c]) * (x . W13[e, I + c]) for 32 RG columns of an expert
//   down  y[i, h] = act[i] . W2[e, h] for 64 RG of its rows
//   join  z = sum_j w_j y[t k + j] + residual, out = z * (mean z^2 + eps)^-1/2 * norm_w
// At a few tokens an expert has few rows, so the layer is a stream of its weights (M=8, H=7168,
// I=2048, k=16: 9 GB) and the arithmetic is small: no LDS ring and no MFMA tile, but dot
// products straight from the load registers.  A load is 8 weight rows x one 128-byte line,
// nontemporal; a wave keeps 32 KiB of them in flight and runs on by itself, without a barrier,
// to the end of its rows.  The tokens' rows (x in bf16, act in fp32) lie in LDS.  act and y stay
// in fp32 at all times, so the layer rounds only its outputs.
//
// Hand-overs: act and y are written and read past the XCDs' L2s (agent-scope accesses); a
// workgroup's stores have arrived (vmcnt 0 in every wave, barrier) before one thread raises the
// item's counter; whoever needs them waits for the counter and loads afterwards.  A waiting item
// only waits for items of lower tickets, tickets are handed out in order, and a workgroup holds
// at most the item that it works on and the next one: the unfinished item with the lowest ticket
// is always being worked on and never waits, so every wait ends, however many workgroups run at
// once and whatever else runs on the GPU.  A wait is bounded all the same, so that calls that
// share a workspace at the same time end too (with results that mean nothing).
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

// Counters, cleared by few_logits_kernel.
constexpr int kTicket = 0, kDownDone = 1, kUpDone = 2;
constexpr int kCounters = kUpDone + kFewMaxPicks;

// Two products of bf16 pairs added to c.
__device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float c) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, a), __builtin_bit_cast(bf16x2, b),
                                         c, false);
}

template <typename T>
__device__ __forceinline__ void store_agent(T* p, T v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename T>
__device__ __forceinline__ T load_agent(const T* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ float2 load_agent2(const float* p) {   // 8-byte aligned
  const uint64_t v = load_agent(reinterpret_cast<const uint64_t*>(p));
  return make_float2(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32)));
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
// c mod 256, the threads' sums meet in a fixed order, so equal rows of Wr give equal logits.
template <int MT>
__global__ __launch_bounds__(256) void few_logits_kernel(FewArgs p) {
  __shared__ double part[4][MT];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, e = blockIdx.x;
  if (e == 0)
    for (int i = tid; i < kCounters; i += 256) p.sync[i] = 0;
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

// The picks of a token by a wave, lane l owning experts l, l + 64, ... (SL of them): ids[0 .. k)
// in LDS, then weights.  s_c: E doubles of LDS.
template <int SL>
__device__ __forceinline__ void select_token(const FewArgs& p, int t, int lane, double* s_c,
                                             int* s_id, float* s_w) {
  const int E = p.E, k = p.top_k;
  const GroupRule& rule = p.rule;
  double l[SL], c[SL], score[SL];
  bool live[SL];
#pragma unroll
  for (int s = 0; s < SL; ++s) {
    const int e = lane + kWave * s;
    l[s] = e < E ? p.keys[(size_t)t * E + e] : -INFINITY;
    live[s] = l[s] > -INFINITY;   // (false for NaN)
    if (!live[s]) l[s] = -INFINITY;
  }
  if (rule.softmax) {
    double top = -INFINITY, total = 0.0;
#pragma unroll
    for (int s = 0; s < SL; ++s) top = fmax(top, l[s]);
    top = fmin(wave_max_f64(top), 1.7976931348623157e308);
#pragma unroll
    for (int s = 0; s < SL; ++s) {
      score[s] = live[s] ? exp(fmin(l[s], 1.7976931348623157e308) - top) : 0.0;
      total += score[s];
    }
    total = wave_sum_f64(total);
#pragma unroll
    for (int s = 0; s < SL; ++s) score[s] = live[s] ? score[s] / total : 0.0;
  } else {
#pragma unroll
    for (int s = 0; s < SL; ++s) score[s] = live[s] ? 1.0 / (1.0 + exp(-l[s])) : 0.0;
  }
#pragma unroll
  for (int s = 0; s < SL; ++s) {
    const int e = lane + kWave * s;
    c[s] = live[s] ? score[s] : -INFINITY;
    if (p.select_bias && e < E) c[s] += (double)p.select_bias[e];
    live[s] = live[s] && c[s] > -INFINITY;
    if (!live[s]) {
      c[s] = -INFINITY;
      score[s] = 0.0;
    }
  }
  uint64_t stay = ~0ull;   // bit g: group g stays
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
  uint64_t key[SL];
#pragma unroll
  for (int s = 0; s < SL; ++s) {
    const int e = lane + kWave * s;
    key[s] = kKeyOutside;
    if (e < E && ((stay >> (e / rule.per)) & 1))
      key[s] = live[s] ? order_key(p.select_bias ? c[s] : l[s]) : kKeyUnscored;
  }
  double picked = 0.0;   // sum of this lane's picks' scores
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
      double sc = score[0];
#pragma unroll
      for (int s = 0; s < SL; ++s)
        if (s == slot) {
          sc = score[s];
          key[s] = kKeyTaken;
        }
      s_id[r] = lane + kWave * slot;
      s_c[r] = sc;   // (k <= E, and the group sums are done)
    }
  }
  wave_lds_fence();
  double divisor = 1.0;
  if (rule.renorm) {
    for (int r = lane; r < k; r += kWave) picked += s_c[r];
    divisor = wave_sum(picked);
  }
  for (int r = lane; r < k; r += kWave)
    s_w[r] = s_c[r] > 0.0 ? (float)(s_c[r] / divisor * (double)rule.scale) : 0.0f;
}

// Dot products of a wave's 8 RG weight rows (lane: row lane / 8 of each group of 8, part lane % 8
// of a unit) with TT rows in LDS (stride ld values, zeros behind K up to a whole unit): sums over
// the lane's parts.  F32: the LDS rows are fp32 (act), else bf16 (x), whose products with bf16 are
// exact.  UB units are in flight.
template <int RG, int TT, bool F32>
struct Stream {
  static constexpr int UB = RG == 4 ? 6 : RG == 2 ? 12 : 16;
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
  float w[kFewMaxPicks];
  uint32_t mask[1024];        // tokens that picked an expert
  int first[1024];            // where its rows begin
  int rows[kFewMaxPicks];     // flat indices t k + j, expert by expert
  int gexp[kFewMaxPicks], gfirst[kFewMaxPicks], gcount[kFewMaxPicks];   // row groups
  int scan[kWaves];
  int groups, ticket;
  float sum[kWaves];
};

// Thread 0 waits until *p reaches n, for at most two seconds; then everyone goes on.
__device__ __forceinline__ void wait_counter(const int* p, int n) {
  if (threadIdx.x == 0) {
    const uint64_t end = __builtin_amdgcn_s_memrealtime() + 200000000ull;   // of 100 MHz
    while (load_agent(p) < n && __builtin_amdgcn_s_memrealtime() < end) __builtin_amdgcn_s_sleep(1);
  }
  __syncthreads();
}
// Raises *p once every store of the workgroup has arrived.
__device__ __forceinline__ void raise_counter(int* p) {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (threadIdx.x == 0) __hip_atomic_fetch_add(p, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

template <int RG, int TT>
__device__ __forceinline__ void up_item(const FewArgs& p, FewShared& s, int u, int tile) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
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
  for (int i = threadIdx.x; i < count * per; i += kThreads) {
    const int t = i / per, c = i % per * 8;
    const u32x4 v = c < p.H ? ld16(p.x + (size_t)(s.rows[first + t] / p.top_k) * p.H + c) : u32x4{0, 0, 0, 0};
    st16(s.stage + ((size_t)t * ld + c) * 2, v);
  }
  __syncthreads();
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
      store_agent(p.act + (size_t)i * p.I + c, gate / (1.0f + expf(-gate)) * up);
  }
  raise_counter(p.sync + kUpDone + u);
}

template <int RG, int TT>
__device__ __forceinline__ void down_item(const FewArgs& p, FewShared& s, int u, int tile) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
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
  wait_counter(p.sync + kUpDone + u, p.up_tiles);
  const int ld = (p.I + kUnit - 1) / kUnit * kUnit, per = ld / 2;
  for (int i = threadIdx.x; i < count * per; i += kThreads) {
    const int t = i / per, c = i % per * 2;
    const float2 v = c < p.I ? load_agent2(p.act + (size_t)s.rows[first + t] * p.I + c) : make_float2(0.0f, 0.0f);
    *reinterpret_cast<float2*>(s.stage + ((size_t)t * ld + c) * 4) = v;
  }
  __syncthreads();
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
    if (part < count && h < p.H) store_agent(p.y + (size_t)i * p.H + h, v);
  }
  raise_counter(p.sync + kDownDone);
}

__device__ __forceinline__ void join_item(const FewArgs& p, FewShared& s, int t, int downs) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, k = p.top_k;
  wait_counter(p.sync + kDownDone, downs);
  float* z = reinterpret_cast<float*>(s.stage);
  float sq = 0.0f;
  constexpr int B = 16;   // picks' values in flight
  for (int h = 2 * threadIdx.x; h < p.H; h += 2 * kThreads) {
    const float* y = p.y + (size_t)t * k * p.H + h;
    float a = 0.0f, b = 0.0f;
    for (int j0 = 0; j0 < k; j0 += B) {
      float2 v[B];
#pragma unroll
      for (int j = 0; j < B; ++j) v[j] = load_agent2(y + (size_t)min(j0 + j, k - 1) * p.H);
#pragma unroll
      for (int j = 0; j < B; ++j) {
        const float w = j0 + j < k ? s.w[t * k + j0 + j] : 0.0f;
        if (j0 + j < k) {
          a = fmaf(w, v[j].x, a);
          b = fmaf(w, v[j].y, b);
        }
      }
    }
    if (p.residual) {
      const uint32_t r = *reinterpret_cast<const uint32_t*>(p.residual + (size_t)t * p.H + h);
      a += bf16lo(r);
      b += bf16hi(r);
    }
    if (p.residual_out)
      *reinterpret_cast<uint32_t*>(p.residual_out + (size_t)t * p.H + h) = cvt_bf16x2(a, b);
    *reinterpret_cast<float2*>(z + h) = make_float2(a, b);   // read by this thread only
    sq += a * a + b * b;
  }
  if (!p.out) return;
  sq = wave_sum_f32(sq);
  if (lane == 0) s.sum[wave] = sq;
  __syncthreads();
  float total = 0.0f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) total += s.sum[w];
  const float f = 1.0f / sqrtf(total / (float)p.H + p.eps);
  for (int h = 2 * threadIdx.x; h < p.H; h += 2 * kThreads) {
    const float2 v = *reinterpret_cast<const float2*>(z + h);
    const uint32_t g = *reinterpret_cast<const uint32_t*>(p.norm_w + h);
    *reinterpret_cast<uint32_t*>(p.out + (size_t)t * p.H + h) =
        cvt_bf16x2(v.x * f * bf16lo(g), v.y * f * bf16hi(g));
  }
}

template <int RG>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2, 2))) void few_layer_kernel(
    FewArgs p) {
  __shared__ __align__(16) FewShared s;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int n = p.M * p.top_k, E = p.E;
  int next = 0;
  if (tid == 0)
    next = __hip_atomic_fetch_add(p.sync + kTicket, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  for (int e = tid; e < E; e += kThreads) s.mask[e] = 0;
  __syncthreads();
  for (int t = wave; t < p.M; t += kWaves) {
    double* c = reinterpret_cast<double*>(s.stage) + (size_t)wave * E;
    int* ids = s.ids + t * p.top_k;
    float* w = s.w + t * p.top_k;
    if (E <= 64) select_token<1>(p, t, lane, c, ids, w);
    else if (E <= 256) select_token<4>(p, t, lane, c, ids, w);
    else select_token<16>(p, t, lane, c, ids, w);
    wave_lds_fence();
    for (int j = lane; j < p.top_k; j += kWave) atomicOr(&s.mask[ids[j]], 1u << t);
    wave_lds_fence();   // c is the next token's
  }
  __syncthreads();
  // rows and row groups of the touched experts: thread i owns experts 2 i and 2 i + 1
  int sum = 0;   // rows, and groups in the upper half
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int e = 2 * tid + q, c = e < E ? __popc(s.mask[e]) : 0;
    sum += c + ((c + p.group_rows - 1) / p.group_rows << 16);
  }
  int scan = sum;
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) {
    const int o = __shfl_up(scan, off, kWave);
    if (lane >= off) scan += o;
  }
  if (lane == kWave - 1) s.scan[wave] = scan;
  __syncthreads();
  int before = scan - sum, all = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const int o = s.scan[w];
    before += w < wave ? o : 0;
    all += o;
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int e = 2 * tid + q, c = e < E ? __popc(s.mask[e]) : 0;
    if (c == 0) continue;
    s.first[e] = before & 0xffff;
    for (int r = 0; r < c; r += p.group_rows) {
      const int g = (before >> 16) + r / p.group_rows;
      s.gexp[g] = e;
      s.gfirst[g] = (before & 0xffff) + r;
      s.gcount[g] = min(p.group_rows, c - r);
    }
    before += c + ((c + p.group_rows - 1) / p.group_rows << 16);
  }
  const int groups = all >> 16;
  if (tid == 0) s.ticket = next;
  __syncthreads();
  for (int i = tid; i < n; i += kThreads) {
    const int e = s.ids[i], t = i / p.top_k;
    s.rows[s.first[e] + __popc(s.mask[e] & ((1u << t) - 1))] = i;
    if (blockIdx.x == 0) {
      if (p.ids_out) p.ids_out[i] = e;
      if (p.w_out) p.w_out[i] = s.w[i];
    }
  }
  __syncthreads();
  const int ups = groups * p.up_tiles, downs = groups * p.down_tiles;
  for (;;) {
    const int item = s.ticket;
    __syncthreads();   // read by all, and the stage is free
    if (item >= ups + downs + p.M) break;
    if (tid == 0)
      next = __hip_atomic_fetch_add(p.sync + kTicket, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (item < ups) {
      const int u = item / p.up_tiles, tile = item % p.up_tiles, c = s.gcount[u];
      if (c <= 1) up_item<RG, 1>(p, s, u, tile);
      else if (c <= 2) up_item<RG, 2>(p, s, u, tile);
      else if (c <= 4) up_item<RG, 4>(p, s, u, tile);
      else up_item<RG, 8>(p, s, u, tile);
    } else if (item < ups + downs) {
      const int d = item - ups, u = d / p.down_tiles, tile = d % p.down_tiles, c = s.gcount[u];
      if (c <= 1) down_item<RG, 1>(p, s, u, tile);
      else if (c <= 2) down_item<RG, 2>(p, s, u, tile);
      else if (c <= 4) down_item<RG, 4>(p, s, u, tile);
      else down_item<RG, 8>(p, s, u, tile);
    } else {
      join_item(p, s, item - ups - downs, downs);
    }
    if (tid == 0) s.ticket = next;
    __syncthreads();
  }
}

inline size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Rows of a group: as many as the stage holds of both kinds, a power of two.
int group_rows(int H, int I) {
  const int row = std::max((H + kUnit - 1) / kUnit * kUnit * 2, (I + kUnit - 1) / kUnit * kUnit * 4);
  int g = kGroupRows;
  while (g > 0 && g * row > kStage) g /= 2;
  return g;
}

}  // namespace

bool few_sizes_ok(int H, int I) { return group_rows(H, I) > 0; }

size_t few_scratch_bytes(int M, int H, int E, int I, int top_k) {
  return up256((size_t)M * E * sizeof(double)) + up256(kCounters * sizeof(int)) +
         up256((size_t)M * top_k * I * sizeof(float)) + up256((size_t)M * top_k * H * sizeof(float));
}

hipError_t launch_few_layer(FewArgs a, void* scratch, hipStream_t s) {
  char* ws = static_cast<char*>(scratch);
  a.keys = reinterpret_cast<double*>(ws);
  ws += up256((size_t)a.M * a.E * sizeof(double));
  a.sync = reinterpret_cast<int*>(ws);
  ws += up256(kCounters * sizeof(int));
  a.act = reinterpret_cast<float*>(ws);
  ws += up256((size_t)a.M * a.top_k * a.I * sizeof(float));
  a.y = reinterpret_cast<float*>(ws);
  a.group_rows = group_rows(a.H, a.I);
  const dim3 experts((unsigned)a.E), t256(256);
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
  // the widest items that leave every CU some
  const long groups = std::min((long)a.M * a.top_k, (long)a.E);
  auto tiles = [&](int rg) { return (long)((a.I + 32 * rg - 1) / (32 * rg)); };
  const int rg = groups * tiles(4) >= cus ? 4 : groups * tiles(2) >= cus ? 2 : 1;
  a.up_tiles = (int)tiles(rg);
  a.down_tiles = (a.H + 64 * rg - 1) / (64 * rg);
  const long most = (long)a.M * a.top_k * std::max(a.up_tiles, a.down_tiles);
  const dim3 grid((unsigned)std::min<long>(cus, std::max<long>(most, a.M))), t(kThreads);
  if (rg == 4) hipLaunchKernelGGL((few_layer_kernel<4>), grid, t, 0, s, a);
  else if (rg == 2) hipLaunchKernelGGL((few_layer_kernel<2>), grid, t, 0, s, a);
  else hipLaunchKernelGGL((few_layer_kernel<1>), grid, t, 0, s, a);
  return hipGetLastError();
}

}  // namespace moe
