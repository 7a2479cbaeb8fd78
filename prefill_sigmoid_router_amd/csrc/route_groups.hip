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
#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "launchers.h"
#include "tiled_common.h"
#include "wave_ops.h"

namespace moe {

namespace {

constexpr int kSelWaves = 4;   // tokens per workgroup: one wave each, no barriers

// fp32 logits with a bound, for many tokens.
//
// bf16 products are exact in fp32, so only the sums round: a product passes at most 31
// roundings inside its 32-wide MFMA, one for each of the 8 MFMAs of a 256-wide piece of K,
// whose sum then goes to fp64, and one more when a part's logit is stored in fp32: 40
// roundings of at most 2^-23 of A = sum |x| |w| over the part (2^-24, doubled in case the
// hardware truncates).  A comes from the same fragments with the sign bits cleared; its own
// roundings are within 2^-10 of it; the largest A of four neighbouring experts is kept for all
// of them (a few per cent more, a quarter of the writes).  (One running fp32 sum over the part: 88 to 144 roundings
// and three times as many choices that the bound leaves open.)
//
// 64 tokens x 64 experts x one part of K per workgroup, 2 x 2 waves of 32 x 32; 64-wide chunks
// (one 128-byte line per row) by direct copies into a 4-stage LDS ring, two workgroups per
// CU.  The expert tiles of a token tile run on one XCD and share its rows through the L2.
// M=2048, E=256, H=7168: 23 us, 5 of them launch, first copies and stores, the rest 28 steps of
// 0.65 us in which fragment reads, products and copies of four waves take turns (tiles of
// 128 x 128 with 8 waves: 23 us too, and twice the partial sums for the selection to read).
constexpr int kBlTile = 64, kBlStages = 4, kBlRounds = 40;

__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2))) void bounded_logits_kernel(
    const uint16_t* __restrict__ x, const uint16_t* __restrict__ wr, int M, int H, int E, int parts,
    int kpart, int per_xcd, float* __restrict__ logits, float* __restrict__ absdot,
    int* __restrict__ count) {
  constexpr int STAGE = 2 * kBlTile * 128, PPW = 4;
  __shared__ __align__(16) unsigned char lds[kBlStages * STAGE];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int li = lane & 15, lg = lane >> 4, rr = lane >> 3;
  const int etiles = (E + kBlTile - 1) / kBlTile, ttiles = (M + kBlTile - 1) / kBlTile;
  if (count && blockIdx.x == 0 && threadIdx.x == 0) *count = 0;   // of the selection that follows
  const int slot = blockIdx.x / kXcds, item = (blockIdx.x % kXcds) * per_xcd + slot;
  if (slot >= per_xcd || item >= etiles * ttiles * parts) return;
  const int e0 = item % etiles * kBlTile;
  const int part = item / etiles % parts, t0 = item / (etiles * parts) * kBlTile;
  const int kbeg = min(H, part * kpart), klen = min(H, kbeg + kpart) - kbeg;

  // LDS rows 0 .. 63 tokens, 64 .. 127 experts; slot q of row r holds part q ^ (r / 2) % 8.
  // Rows past the last repeat it and are never stored.
  const uint16_t* src[PPW];
  int koff[PPW];
#pragma unroll
  for (int i = 0; i < PPW; ++i) {
    const int r = (wave * PPW + i) * 8 + rr;
    koff[i] = 8 * ((lane & 7) ^ ((r >> 1) & 7));
    src[i] = (r < kBlTile ? x + (size_t)min(t0 + r, M - 1) * H
                          : wr + (size_t)min(e0 + r - kBlTile, E - 1) * H) + kbeg + koff[i];
  }
  const int nch = (klen + 63) / 64, ndma = klen / 64;
  auto issue = [&](int c) {
    unsigned char* base = lds + (c % kBlStages) * STAGE + wave * PPW * 1024;
    if (c < ndma) {
#pragma unroll
      for (int i = 0; i < PPW; ++i)
        __builtin_amdgcn_global_load_lds((global_void*)(src[i] + c * 64),
                                         (lds_void*)(base + i * 1024), 16, 0, 0);
    } else {
#pragma unroll
      for (int i = 0; i < PPW; ++i)
        *reinterpret_cast<u32x4*>(base + i * 1024 + lane * 16) =
            c * 64 + koff[i] < klen ? ld16(src[i] + c * 64) : u32x4{0, 0, 0, 0};
    }
  };
  const int trow = 32 * (wave & 1), erow = kBlTile + 32 * (wave >> 1);
  auto frag = [&](int c, int row, int ks) {
    return *reinterpret_cast<const u32x4*>(lds + (c % kBlStages) * STAGE + (row + li) * 128 +
                                           (((lg + 4 * ks) ^ (li >> 1)) * 16));
  };
  const u32x4 mag = u32x4{0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu};
  f32x4 acc[2][2], aab[2][2];   // [expert tile][token tile]
  double sum[2][2][4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      acc[i][j] = aab[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int q = 0; q < 4; ++q) sum[i][j][q] = 0.0;
    }
  auto flush = [&] {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int q = 0; q < 4; ++q) sum[i][j][q] += (double)acc[i][j][q];
        acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
  };
  auto step = [&](int c) {
    const int after = c < ndma ? min(kBlStages - 2, ndma - 1 - c) : 0;
    if (after >= 2) wait_vmcnt<2 * PPW>();
    else if (after == 1) wait_vmcnt<PPW>();
    else wait_vmcnt<0>();
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (c + kBlStages - 1 < nch) issue(c + kBlStages - 1);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      u32x4 xf[2], wf[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        xf[j] = frag(c, trow + 16 * j, ks);
        wf[j] = frag(c, erow + 16 * j, ks);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          acc[i][j] = mfma16x16x32(wf[i], xf[j], acc[i][j]);
          aab[i][j] = mfma16x16x32(wf[i] & mag, xf[j] & mag, aab[i][j]);
        }
    }
  };
#pragma unroll
  for (int c = 0; c < kBlStages - 1; ++c)
    if (c < nch) issue(c);
  int c = 0;
  for (; c + 4 <= nch; c += 4) {   // 256 values of K
#pragma unroll
    for (int k = 0; k < 4; ++k) step(c + k);
    flush();
  }
  for (; c < nch; ++c) step(c);
  flush();
  // lane (li, lg): token li of a tile, experts 4 lg .. 4 lg + 3
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int t = t0 + trow + 16 * j + li;
    if (t >= M) continue;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = e0 + (erow - kBlTile) + 16 * i + 4 * lg;
      if (e >= E) continue;
      const size_t row = (size_t)part * M + t;
      float* l = logits + row * E + e;
      const f32x4 a = aab[i][j];   // (rows past the last expert repeat it)
      absdot[row * ((E + 3) / 4) + e / 4] = fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3]));
      if (E % 4 == 0) {
        *reinterpret_cast<float4*>(l) = make_float4((float)sum[i][j][0], (float)sum[i][j][1],
                                                    (float)sum[i][j][2], (float)sum[i][j][3]);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (e + q < E) l[q] = (float)sum[i][j][q];
      }
    }
  }
}

// Logits of a token: fp64 keys, the caller's fp32 logits, or fp32 MFMA partial logits with
// their |x| . |w| sums (bounded_logits_kernel), which bound their error.  -inf past the last.
struct SameRows {   // row t of the source is token t
  __device__ int64_t rows(int M) const { return M; }
  __device__ int64_t token(int64_t row) const { return row; }
};
struct KeySource : SameRows {
  const double* keys;
  int64_t ld;
  template <int SL>
  __device__ void get(int64_t t, int E, int lane, double (&l)[SL], double (&d)[SL]) const {
#pragma unroll
    for (int s = 0; s < SL; ++s) {
      l[s] = lane + kWave * s < E ? keys[t * ld + lane + kWave * s] : -INFINITY;
      d[s] = 0.0;
    }
  }
};
// Tokens for which every expert's exact logit is needed, in any order: *count of them were
// asked for, the first `room` have a row.
struct TokenList {
  int *count, *tokens;
  int room;
};
struct ListSource {   // exact logits of listed tokens
  const double* keys;
  int64_t ld;
  TokenList list;
  __device__ int64_t rows(int) const { return min(*list.count, list.room); }
  __device__ int64_t token(int64_t row) const { return list.tokens[row]; }
  template <int SL>
  __device__ void get(int64_t row, int E, int lane, double (&l)[SL], double (&d)[SL]) const {
    KeySource{{}, keys, ld}.get<SL>(row, E, lane, l, d);
  }
};
struct LogitSource : SameRows {
  const float* logits;
  int64_t ld;
  template <int SL>
  __device__ void get(int64_t t, int E, int lane, double (&l)[SL], double (&d)[SL]) const {
#pragma unroll
    for (int s = 0; s < SL; ++s) {
      l[s] = lane + kWave * s < E ? (double)logits[t * ld + lane + kWave * s] : -INFINITY;
      d[s] = 0.0;
    }
  }
};
struct BoundedSource : SameRows {
  const float *logits, *absdot;
  const uint16_t *x, *wr;
  int parts, M, H;
  double rel;   // error of a partial logit over its |x| . |w| sum
  TokenList list;   // softmax with a bias only
  template <int SL>
  __device__ void get(int64_t t, int E, int lane, double (&l)[SL], double (&d)[SL]) const {
    constexpr int B = SL > 4 ? 2 : 4;   // parts in flight
#pragma unroll
    for (int s = 0; s < SL; ++s) l[s] = d[s] = 0.0;
    for (int p0 = 0; p0 < parts; p0 += B) {
      float v[B][SL], a[B][SL];
#pragma unroll
      for (int p = 0; p < B; ++p) {
        const int64_t row = (int64_t)min(p0 + p, parts - 1) * M + t;
#pragma unroll
        for (int s = 0; s < SL; ++s) {
          const int e = min(lane + kWave * s, E - 1);
          v[p][s] = logits[row * E + e];
          a[p][s] = absdot[row * ((E + 3) / 4) + e / 4];
        }
      }
#pragma unroll
      for (int p = 0; p < B; ++p) {
        if (p0 + p >= parts) break;
#pragma unroll
        for (int s = 0; s < SL; ++s) {
          l[s] += (double)v[p][s];
          d[s] += (double)a[p][s];
        }
      }
    }
#pragma unroll
    for (int s = 0; s < SL; ++s) {
      // (subnormal products may be flushed: H times the smallest normal number)
      const bool in = lane + kWave * s < E;
      l[s] = in ? l[s] : -INFINITY;
      d[s] = in ? d[s] * rel + (double)H * 0x1p-126 : 0.0;
    }
  }
};

// An expert that may be among the picks: one per lane.
struct Candidate {
  int id;
  double l, d;       // logit and its bound
  double b;          // bias
  uint32_t lo, hi;   // ends of the fp32 interval of what orders the picks, as order32 keys
};

// Exact logits that the workgroup's waves ask for: fp64 dot products in quarters of the row,
// added in order, so that equal rows of the router weight give equal sums.  Each wave leaves up
// to kAsk experts a round, worked off two at a time (most tokens that ask have two): each pair
// by all waves, a quarter each, or, where there are many, by one.
constexpr int kAsk = 32;
struct ExactQueue {
  int expert[kSelWaves][kAsk];   // -1: none
  alignas(16) int asked[kSelWaves];
  double part[kSelWaves][kAsk][kSelWaves];
};

// A quarter of N dot products of row t of x, B chunks of 8 values a lane in flight per row
// (4: H = 7168 in one batch).
template <int N, int B>
__device__ __forceinline__ void quarter_dots(const BoundedSource& q, int64_t t, const int* experts,
                                             int quarter, int lane, double (&sum)[N]) {
  const uint16_t* xr = q.x + t * q.H;
  const uint16_t* w[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    w[i] = q.wr + (size_t)max(experts[i], 0) * q.H;
    sum[i] = 0.0;
  }
  const int n = q.H >> 3, beg = n * quarter / kSelWaves, end = n * (quarter + 1) / kSelWaves;
  for (int c0 = beg + lane; c0 < end; c0 += kWave * B) {
    u32x4 xv[B], v[N][B];
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int c = c0 + kWave * b;
      const bool in = c < end;
      xv[b] = in ? ld16(xr + (size_t)c * 8) : u32x4{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < N; ++i) v[i][b] = in ? ld16(w[i] + (size_t)c * 8) : u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int b = 0; b < B; ++b)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const double lo = bf16lo(xv[b][j]), hi = bf16hi(xv[b][j]);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          sum[i] = fma(lo, (double)bf16lo(v[i][b][j]), sum[i]);
          sum[i] = fma(hi, (double)bf16hi(v[i][b][j]), sum[i]);
        }
      }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) sum[i] = wave_sum_f64(sum[i]);
}

// All waves of the workgroup, together: computes what `redo` (bit s: this lane's expert in
// slot s) and `ask` (this lane's candidate) ask for as far as the queue goes and clears those.
// False if no wave asked.
template <int SL>
__device__ __forceinline__ bool exact_round(const BoundedSource& q, ExactQueue& queue, int64_t t0,
                                            int64_t M, int wave, int lane, uint32_t& redo,
                                            double (&l)[SL], double (&d)[SL], bool& ask,
                                            Candidate& mine) {
  if (lane < kAsk) queue.expert[wave][lane] = -1;
  wave_lds_fence();
  int asked = 0;
  int at[SL + 1];   // this lane's place in the queue for slot s, and for its candidate
#pragma unroll
  for (int s = 0; s <= SL; ++s) {
    const bool wants = s < SL ? (redo >> s) & 1 : ask;
    const uint64_t who = __ballot(wants);
    const int place = asked + __builtin_amdgcn_mbcnt_hi((uint32_t)(who >> 32),
                                                        __builtin_amdgcn_mbcnt_lo((uint32_t)who, 0));
    at[s] = wants && place < kAsk ? place : -1;
    if (at[s] >= 0) queue.expert[wave][place] = s < SL ? lane + kWave * s : mine.id;
    asked += __popcll(who);
  }
  if (lane == 0) queue.asked[wave] = min(asked, kAsk);
  if (!__syncthreads_or(asked)) return false;
  const int4 n4 = *reinterpret_cast<const int4*>(queue.asked);
  const int n[kSelWaves] = {
      __builtin_amdgcn_readfirstlane(n4.x), __builtin_amdgcn_readfirstlane(n4.y),
      __builtin_amdgcn_readfirstlane(n4.z), __builtin_amdgcn_readfirstlane(n4.w)};
  // each pair over the waves, or a pair per wave
  const bool split = n[0] + n[1] + n[2] + n[3] < 4 * kSelWaves;
  int pair = 0;
#pragma unroll 1
  for (int w = 0; w < kSelWaves; ++w) {
    const int64_t t = min(t0 + w, M - 1);
    const int asks = w == 0 ? n[0] : w == 1 ? n[1] : w == 2 ? n[2] : n[3];
    for (int i = 0; i < asks; i += 2, ++pair) {
      if (!split && pair % kSelWaves != wave) continue;
      for (int quarter = split ? wave : 0; quarter < (split ? wave + 1 : kSelWaves); ++quarter) {
        double sum[2];
        quarter_dots<2, (SL > 4 ? 2 : 4)>(q, t, &queue.expert[w][i], quarter, lane, sum);
        if (lane == 0) {
#pragma unroll
          for (int j = 0; j < 2; ++j) queue.part[w][i + j][quarter] = sum[j];
        }
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int s = 0; s <= SL; ++s)
    if (at[s] >= 0) {
      const double* part = queue.part[wave][at[s]];
      const double got = ((part[0] + part[1]) + part[2]) + part[3];
      if (s < SL) {
        l[s] = got;
        d[s] = 0.0;
        redo &= ~(1u << s);
      } else {
        mine.l = got;
        mine.d = 0.0;
        ask = false;
      }
    }
  return true;
}
static_assert(kSelWaves == 4 && kAsk % 2 == 0, "the sums and pairs above");

// Selection of a token by fp32 values with bounds, in two steps: groups and candidates
// (collect_fast), order and weights (rank_fast).  kDone: no bound can turn a choice.  kRedo:
// `redo` or `ask` mark the experts whose exact logits can settle it.  kAll: every one is needed
// (a softmax's divisor decides).  kOpen: the fp64 code below decides.  Each value's bound covers its logit's (|l - exact| <= d, and l's rounding
// to fp32) and the fp32 arithmetic: __expf of z is within (|z| + 4) 2^-22 of itself,
// reciprocals and products within a few 2^-24.
//
// Top-k without rounds: the k-th largest of the 64 lanes' largest values is a lower limit of
// the k-th largest of all; what can reach it (k and a few) is collected, one per lane, and
// ranked by counting the intervals above each, or, where intervals meet, the fp64 values.  (A
// round of a k-step selection costs 500 cycles: M=8192, E=384, k=8 22 us.)
enum Fast { kDone, kRedo, kAll, kOpen };

// Bounded logits also make the weights: where a bound could move one by more than this part of
// itself, the exact logit does.  (Sums of many bf16 products are a thousand times closer than
// their bounds, so that weights are within 2e-7 at H=7168; only large terms that cancel reach
// this.)
constexpr double kWeightBound = 0x1p-9;

__device__ __forceinline__ uint32_t order32(float f) {   // orders as the numbers do
  const uint32_t bits = __float_as_uint(f + 0.0f);
  return (int)bits < 0 ? ~bits : bits | 0x80000000u;
}

template <int SL>
__device__ __forceinline__ Fast collect_fast(const double (&l)[SL], const double (&d)[SL],
                                             const float (&b)[SL], bool bounded, bool bias, int E,
                                             int top_k, const GroupRule& rule, float* s_v,
                                             float* s_d, uint32_t* s_key, int* s_id, int lane,
                                             uint32_t& redo, float& top, int& found,
                                             Candidate& mine) {
  constexpr float u = 0x1p-22f;
  float v[SL], dv[SL];
  uint32_t live = 0;
  bool odd = false;   // a logit or bound that fp32 does not hold
#pragma unroll
  for (int s = 0; s < SL; ++s) {
    v[s] = (float)l[s];
    dv[s] = (float)d[s] * 1.001f + fabsf(v[s]) * u;
    const bool has = l[s] > -INFINITY;
    live |= (uint32_t)has << s;
    // (given logits may mask experts; bounded ones that are not finite may be due to fp32)
    odd |= (has || (bounded && lane + kWave * s < E)) && !(fabsf(v[s]) < 1e30f && dv[s] <= 0.25f);
    if (!has) v[s] = dv[s] = 0.0f;
  }
  if (__any(odd)) return kOpen;
  float c[SL], dc[SL];
  // scores only where something but the picks' weights needs them
  const bool by_group = rule.n_group > 1 && rule.topk_group < rule.n_group;
  top = -INFINITY;
  if (rule.softmax) {
#pragma unroll
    for (int s = 0; s < SL; ++s)
      if (live >> s & 1) top = fmaxf(top, v[s]);
    top = wave_max_f32(top);
  }
  if (bias || by_group) {
    if (rule.softmax) {
      float total = 0.0f;
#pragma unroll
      for (int s = 0; s < SL; ++s) {
        const float z = v[s] - top;
        c[s] = live >> s & 1 ? __expf(z) : 0.0f;
        // (below the smallest normal number, 87.3 under the top, __expf gives 0)
        dc[s] = c[s] * (dv[s] + 0.6f * dv[s] * dv[s] + (4.0f - z) * u) + 0x1p-125f;
        total += c[s];
      }
      if (bias) {
        float off = 0.0f;
#pragma unroll
        for (int s = 0; s < SL; ++s) off += dc[s];
        total = wave_sum_f32(total);
        const float inv = total > 0.0f ? __builtin_amdgcn_rcpf(total) : 0.0f;
        off = bounded ? wave_sum_f32(off) * inv * 1.001f : 0.0f;   // the divisor's, of itself
        off += 2.0f * off * off;
#pragma unroll
        for (int s = 0; s < SL; ++s) {
          c[s] *= inv;
          dc[s] = dc[s] * inv + c[s] * (off + 80.0f * u);
        }
      }
    } else {
#pragma unroll
      for (int s = 0; s < SL; ++s) {
        const float ex = __expf(-fmaxf(v[s], -80.0f));
        const float sc = __builtin_amdgcn_rcpf(1.0f + ex);
        c[s] = live >> s & 1 ? sc : 0.0f;
        const float grow = dv[s] + 0.6f * dv[s] * dv[s] + (fabsf(v[s]) + 4.0f) * u;
        dc[s] = c[s] * (fminf(1.0f, ex * sc) * grow + 2.0f * u);
        if (v[s] < -79.0f) dc[s] += 1e-34f;
      }
    }
    if (bias) {
#pragma unroll
      for (int s = 0; s < SL; ++s) {
        c[s] += b[s];
        dc[s] += fabsf(c[s]) * u + 1e-37f;
        if ((live >> s & 1) && !(fabsf(c[s]) < 1e30f)) odd = true;
      }
      if (__any(odd)) return kOpen;
    }
  }
  uint64_t stay = ~0ull;
  auto group_of = [&](int e) { return (int)((uint32_t)e * rule.per_magic >> 20); };
  if (by_group) {
#pragma unroll
    for (int s = 0; s < SL; ++s) {
      const int e = lane + kWave * s;
      if (e < E) {
        s_v[e] = live >> s & 1 ? c[s] : -INFINITY;
        s_d[e] = live >> s & 1 ? dc[s] : 0.0f;
      }
    }
    wave_lds_fence();
    // span lanes (a power of two) join a group's two best values, upper and lower ends
    int span = 1, log = 0;
    while (span * 2 * rule.n_group <= kWave) {
      span *= 2;
      ++log;
    }
    const int g = lane >> log, sub = lane & (span - 1);
    float h1 = -INFINITY, h2 = -INFINITY, w1 = -INFINITY, w2 = -INFINITY;
    auto join = [](float& p1, float& p2, float o1, float o2) {
      p2 = fmaxf(fminf(p1, o1), fmaxf(p2, o2));
      p1 = fmaxf(p1, o1);
    };
    if (g < rule.n_group)
      for (int j0 = sub; j0 < rule.per; j0 += 4 * span) {
        float x[4], dx[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = g * rule.per + min(j0 + i * span, rule.per - 1);
          x[i] = j0 + i * span < rule.per ? s_v[j] : -INFINITY;
          dx[i] = s_d[j];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          join(h1, h2, x[i] + dx[i], -INFINITY);
          join(w1, w2, x[i] - dx[i], -INFINITY);
        }
      }
    for (int off = 1; off < span; off <<= 1) {
      join(h1, h2, __shfl_xor(h1, off, kWave), __shfl_xor(h2, off, kWave));
      join(w1, w2, __shfl_xor(w1, off, kWave), __shfl_xor(w2, off, kWave));
    }
    const bool two = rule.group_top == 2;
    // (outwards by the sums' rounding)
    float most = two && h2 > -INFINITY ? h1 + h2 : h1, least = two && w2 > -INFINITY ? w1 + w2 : w1;
    if (most > -INFINITY) most += fabsf(most) * u;
    if (least > -INFINITY) least -= fabsf(least) * u;
    float* const s_most = reinterpret_cast<float*>(s_key);   // 64 each
    float* const s_least = reinterpret_cast<float*>(s_id);
    s_most[lane] = s_least[lane] = -INFINITY;
    wave_lds_fence();
    if (sub == 0 && g < rule.n_group) {
      s_most[g] = most;
      s_least[g] = least;
    }
    wave_lds_fence();
    // a group stays if fewer than topk_group others can reach it; the rest must be out of reach
    const bool group = lane < rule.n_group;
    const float my_least = s_least[lane], my_most = s_most[lane];
    int ahead = 0, open = -1;   // groups certainly above this one, those (without it) that may be
    for (int j = 0; j < rule.n_group; j += 4) {
      const float4 m = *reinterpret_cast<const float4*>(s_most + j);
      const float4 n = *reinterpret_cast<const float4*>(s_least + j);
      ahead += (n.x > my_most) + (n.y > my_most) + (n.z > my_most) + (n.w > my_most);
      open += (m.x >= my_least) + (m.y >= my_least) + (m.z >= my_least) + (m.w >= my_least);
    }
    const bool in = group && open < rule.topk_group, out = group && ahead >= rule.topk_group;
    if (__any(group && !in && !out)) {
      // what can make an open group's score: values that reach its group_top-th lower end
      wave_lds_fence();
      if (sub == 0 && g < rule.n_group) s_v[g] = two ? w2 : w1;
      if (group) s_d[lane] = !in && !out ? 1.0f : 0.0f;
      wave_lds_fence();
#pragma unroll
      for (int s = 0; s < SL; ++s) {
        const int e = lane + kWave * s;
        if (e < E && (live >> s & 1) && d[s] > 0.0) {
          const int ge = group_of(e);
          if (s_d[ge] != 0.0f && c[s] + dc[s] >= s_v[ge]) redo |= 1u << s;
        }
      }
      if (__any(redo != 0)) return kRedo;
      bool inexact = false;
#pragma unroll
      for (int s = 0; s < SL; ++s) inexact |= d[s] > 0.0;
      return rule.softmax && bias && __any(inexact) ? kAll : kOpen;
    }
    stay = __ballot(in);
    wave_lds_fence();
  }
  if (bias) {
#pragma unroll
    for (int s = 0; s < SL; ++s) {
      v[s] = c[s];
      dv[s] = dc[s];
    }
  }
  // limit: the largest lower end that at least top_k lanes reach with one of their values
  uint32_t inside = 0, largest = 0;
#pragma unroll
  for (int s = 0; s < SL; ++s) {
    const bool is = (live >> s & 1) && (!by_group || (stay >> group_of(lane + kWave * s) & 1));
    inside |= (uint32_t)is << s;
    if (is) largest = max(largest, order32(v[s] - dv[s]));
  }
  s_key[lane] = largest;
  wave_lds_fence();
  int reached = 0;
#pragma unroll
  for (int j = 0; j < kWave; j += 4) {
    const uint4 o = *reinterpret_cast<const uint4*>(s_key + j);
    reached += (o.x >= largest) + (o.y >= largest) + (o.z >= largest) + (o.w >= largest);
  }
  const uint32_t limit = wave_max_u32(reached >= top_k ? largest : 0u);
  wave_lds_fence();
  // candidates: what can reach the limit, one per lane, in slot and lane order
  double* s_l = reinterpret_cast<double*>(s_v);   // s_v and s_d are free: 64 of each
  double* s_b = s_l + kWave;
  float* s_bias = reinterpret_cast<float*>(s_b + kWave);
  uint32_t* s_hi = reinterpret_cast<uint32_t*>(s_bias + kWave);
  found = 0;
#pragma unroll
  for (int s = 0; s < SL; ++s) {
    const uint32_t hi = order32(v[s] + dv[s]);
    const bool is = (inside >> s & 1) && hi >= limit;
    const uint64_t who = __ballot(is);
    const int at = found + __builtin_amdgcn_mbcnt_hi((uint32_t)(who >> 32),
                                                     __builtin_amdgcn_mbcnt_lo((uint32_t)who, 0));
    found += __popcll(who);
    if (is && at < kWave) {
      s_id[at] = lane + kWave * s;
      s_l[at] = l[s];
      s_b[at] = d[s];
      s_bias[at] = b[s];
      s_key[at] = order32(v[s] - dv[s]);
      s_hi[at] = hi;
    }
  }
  if (found < top_k || found > kWave) return kOpen;   // too few scored experts, or many alike
  wave_lds_fence();
  const bool cand = lane < found;
  mine.id = cand ? s_id[lane] : 0;
  mine.l = cand ? s_l[lane] : 0.0;
  mine.d = cand ? s_b[lane] : 0.0;
  mine.b = cand ? (double)s_bias[lane] : 0.0;
  mine.lo = cand ? s_key[lane] : 0u;
  mine.hi = cand ? s_hi[lane] : 0u;
  wave_lds_fence();
  return kDone;
}

// again: after exact logits came in, which the fp32 intervals do not hold
template <int SL, bool BOUNDS>
__device__ __forceinline__ Fast rank_fast(const double (&l)[SL], const double (&d)[SL],
                                          const Candidate& mine, bool again, bool bias, int64_t t,
                                          int E, int top_k, const GroupRule& rule, float top,
                                          int found, double* s_val, uint32_t* s_key, int lane,
                                          uint32_t& redo, bool& ask, int32_t* ids,
                                          float* weights) {
  const bool cand = lane < found;
  const double ex = exp(rule.softmax ? mine.l - (double)top : -mine.l);
  const double score = rule.softmax ? ex : 1.0 / (1.0 + ex);
  int rank = 0, reach = -1;   // candidates certainly above this one, those (without it) that may be
  for (int j = 0; j < found; ++j) {
    rank += (uint32_t)__builtin_amdgcn_readlane((int)mine.lo, j) > mine.hi ? 1 : 0;
    reach += (uint32_t)__builtin_amdgcn_readlane((int)mine.hi, j) >= mine.lo ? 1 : 0;
  }
  if (__any(cand && (again || (rank != reach && rank < top_k)))) {
    // the same in fp64, by values with the bounds that their logits' leave; a softmax's divisor
    // moves two values by the difference of their scores
    const bool shared = rule.softmax && bias;
    double z = 1.0, dz = 0.0;
    if (shared) {
      double total = 0.0, off = 0.0;
#pragma unroll
      for (int s = 0; s < SL; ++s)
        if (l[s] > -INFINITY) {
          const double e = exp(l[s] - (double)top);
          total += e;
          off += e * (d[s] + 0.6 * d[s] * d[s]);
        }
      z = wave_sum_f64(total);
      if (BOUNDS) dz = wave_sum_f64(off) / z;
      dz += 2.0 * dz * dz;   // 1 / (1 - dz) - 1 for dz < 0.4
    }
    double* s_bound = s_val + kWave;
    double* s_part = s_bound + kWave;
    const double part = score / z;
    double my_v = cand ? mine.l : -INFINITY, my_d = mine.d;
    if (bias && cand) {
      my_v = part + mine.b;
      const double grow = my_d + 0.6 * my_d * my_d;
      if (my_d > 0.0) my_d = grow * part * (rule.softmax ? 1.0 : fmin(1.0, ex * score)) + 1e-14;
    }
    s_val[lane] = my_v;
    s_bound[lane] = my_d;
    s_part[lane] = part;
    wave_lds_fence();
    rank = 0;
    bool close = false;   // another candidate that the bounds cannot tell from this one
    for (int j0 = 0; j0 < found; j0 += 4) {   // (places past the last hold -inf and 0)
      double o[4], tol[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[i] = s_val[j0 + i];
        tol[i] = my_d + s_bound[j0 + i];
        if (shared) tol[i] += dz * fabs(s_part[j0 + i] - part);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        rank += (o[i] > my_v || (o[i] == my_v && j0 + i < lane)) ? 1 : 0;
        close |= j0 + i != lane && fabs(o[i] - my_v) <= tol[i] && tol[i] > 0.0;
      }
    }
    if (__any(cand && close)) {   // it matters if one of the two is picked
      s_key[lane] = (uint32_t)rank;
      wave_lds_fence();
      bool matters = false;
#pragma unroll 4
      for (int j = 0; j < found; ++j) {
        double tol = my_d + s_bound[j];
        if (shared) tol += dz * fabs(s_part[j] - part);
        matters |= j != lane && fabs(s_val[j] - my_v) <= tol && tol > 0.0 &&
                   (rank < top_k || (int)s_key[j] < top_k);
      }
      wave_lds_fence();
      if (__any(cand && matters)) {
        ask = cand && matters && my_d > 0.0;
        return __any(ask) ? kRedo : kAll;   // (only the divisor leaves it open)
      }
    }
  }
  const bool picked = cand && rank < top_k;
  if (BOUNDS) {
    ask = picked && mine.d * (rule.softmax ? 1.0 : ex * score) > kWeightBound;
    if (__any(ask)) return kRedo;
  }
  double divisor = 1.0;
  if (rule.renorm) {
    divisor = wave_sum_f64(picked ? score : 0.0);
  } else if (rule.softmax) {
    double total = 0.0, off = 0.0;
#pragma unroll
    for (int s = 0; s < SL; ++s)
      if (l[s] > -INFINITY) {
        const double e = exp(l[s] - (double)top);
        total += e;
        off += e * d[s];
      }
    divisor = wave_sum_f64(total);
    if (BOUNDS && wave_sum_f64(off) > kWeightBound * divisor) {   // the divisor's own terms
#pragma unroll
      for (int s = 0; s < SL; ++s)
        if (l[s] > -INFINITY && exp(l[s] - (double)top) * d[s] * E > kWeightBound * divisor)
          redo |= 1u << s;
      if (__any(redo != 0)) return kRedo;
    }
  }
  if (picked) {   // (1 / divisor may be past the largest number where score / divisor is not)
    ids[t * top_k + rank] = mine.id;
    weights[t * top_k + rank] = divisor > 0.0 ? (float)(score / divisor * (double)rule.scale) : 0.0f;
  }
  return kDone;
}

// Doubles of an array with a place for each expert: 192 at least in all (64 candidates' three).
__host__ __device__ constexpr int select_lds_experts(bool bounds, int E) {
  const int even = (E + 1) / 2 * 2, least = bounds ? 96 : 192;
  return even > least ? even : least;
}

// LDS of a wave, in doubles: c of E experts (and its bound), the picks' scores (values, bounds)
// and ids (room for 64), 64 keys; a multiple of 16 bytes, as are the parts before the ids.
__host__ __device__ constexpr int select_lds_doubles(bool bounds, int E, int top_k) {
  const int even_E = select_lds_experts(bounds, E), even_k = (top_k + 1) / 2 * 2;
  const int ids = ((top_k > 64 ? top_k : 64) + 3) / 4 * 2;
  return (bounds ? 2 * even_E + 3 * even_k : even_E + even_k) + ids + 32;
}

// The same in fp64: kDone, or (with bounds) kRedo.
//
// With bounded logits |l - exact| <= d, every value that a choice compares carries a bound of
// its own (sigmoid: s (1 - s) (e^d - 1) <= 1.2 d s (1 - s) for d <= 1/4; softmax without its
// common divisor: 1.2 d e^l), and a choice stands if no bound can turn it.  Where one can,
// the experts that it hangs on are asked for; choices between exact values are exact, so this
// ends.  (Softmax with a bias: the kernel asks for every logit first.)
template <int SL, bool BOUNDS>
__device__ __forceinline__ Fast select_fp64(const double (&l)[SL], const double (&d)[SL],
                                            const float* bias, int64_t t, int E, int top_k,
                                            const GroupRule& rule, double* s_c, double* s_d,
                                            double* s_pick, double* s_pv, double* s_pd, int* s_id,
                                            int lane, uint32_t& redo, int32_t* ids,
                                            float* weights) {
  // scores (softmax with bounds and no bias: without the divisor, which is applied at the end)
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
    divisor = wave_sum_f64(total);
    if (!BOUNDS || bias) {
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
        if (__any(redo != 0)) return kRedo;
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
      if (__any(redo != 0)) return kRedo;
    }
  }
  if (BOUNDS) {   // as in rank_fast; a softmax's divisor too
    const bool all = rule.softmax && !rule.renorm;
#pragma unroll
    for (int s = 0; s < SL; ++s) {
      const double part = d[s] * (rule.softmax ? 1.0 : 1.0 - score[s]);
      if ((taken >> s & 1) && score[s] > 0.0 && part > kWeightBound) redo |= 1u << s;
      if (all && live[s] && score[s] * d[s] * E > kWeightBound * divisor) redo |= 1u << s;
    }
    wave_lds_fence();
    if (__any(redo != 0)) return kRedo;
  }
  if (rule.renorm) {
    double total = 0.0;
    for (int r = lane; r < top_k; r += kWave) total += s_pick[r];
    divisor = wave_sum(total);
  }
  for (int r = lane; r < top_k; r += kWave) {
    ids[t * top_k + r] = s_id[r];
    weights[t * top_k + r] =
        s_pick[r] > 0.0 ? (float)(s_pick[r] / divisor * (double)rule.scale) : 0.0f;
  }
  return kDone;
}

// One wave per token; lane l owns experts l, l + 64, ... (SL of them).  At M=2048, E=256, k=16
// one token in nine asks for exact logits, mostly two.  Bound by latencies, not by work: one
// wave takes 6 us from start to end (M=8: 5.9 us), and what asks a second time as long again and
// the dot products (M=2048: 25 us).
template <int SL, typename SRC>
__global__ __launch_bounds__(kSelWaves* kWave, 2) void select_groups_kernel(
    SRC src, const float* __restrict__ bias, int M, int E, int top_k, GroupRule rule,
    int32_t* __restrict__ ids, float* __restrict__ weights) {
  constexpr bool BOUNDS = std::is_same<SRC, BoundedSource>::value;
  extern __shared__ __align__(16) double sel_lds[];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int64_t t0 = (int64_t)blockIdx.x * kSelWaves, row = t0 + wave;
  const bool on = row < src.rows(M);
  if (!BOUNDS && !on) return;
  const int64_t t = on ? src.token(row) : row;
  double* s_c = sel_lds + (size_t)wave * select_lds_doubles(BOUNDS, E, top_k);
  const int even_E = select_lds_experts(BOUNDS, E), even_k = (top_k + 1) / 2 * 2;
  double* s_d = s_c + even_E;                              // BOUNDS
  double* s_pick = s_c + (BOUNDS ? 2 : 1) * even_E;
  double* s_pv = s_pick + even_k;                          // BOUNDS: the picks' values
  double* s_pd = s_pv + even_k;                            // BOUNDS: and their bounds
  int* s_id = reinterpret_cast<int*>(s_pick + (BOUNDS ? 3 : 1) * even_k);   // and the picks
  uint32_t* s_key = reinterpret_cast<uint32_t*>(s_id + (max(top_k, kWave) + 3) / 4 * 4);

  float b[SL];
  double l[SL], d[SL];
  src.template get<SL>(min(row, (int64_t)M - 1), E, lane, l, d);
#pragma unroll
  for (int s = 0; s < SL; ++s) {
    const int e = lane + kWave * s;
    b[s] = bias && e < E ? bias[e] : 0.0f;
  }
  uint32_t redo = 0;   // bit s: this lane's expert in slot s gets its exact logit
  if (BOUNDS && on) {
#pragma unroll
    for (int s = 0; s < SL; ++s)
      if (!(d[s] <= 0.25)) redo |= 1u << s;   // too wide, or not a number
  }
  enum { kCollect, kRank, kSlow } stage = top_k <= kWave ? kCollect : kSlow;
  bool ask = false, again = false;   // this lane's candidate gets its exact logit; some did
  float top = 0.0f;
  int found = 0;
  Candidate mine{};
  auto select = [&]() -> Fast {
    Fast got = kOpen;
    if (stage == kCollect) {
      got = collect_fast<SL>(l, d, b, BOUNDS, bias != nullptr, E, top_k, rule,
                             reinterpret_cast<float*>(s_c), reinterpret_cast<float*>(s_c) + E, s_key,
                             s_id, lane, redo, top, found, mine);
      if (got == kRedo) return got;
      if (got != kAll) stage = got == kDone ? kRank : kSlow;
    }
    if (stage == kRank) {
      got = rank_fast<SL, BOUNDS>(l, d, mine, again, bias != nullptr, t, E, top_k, rule, top, found,
                                  s_c, s_key, lane, redo, ask, ids, weights);
      again = true;
      if (__any(redo != 0) || got == kAll) {
        stage = kCollect;
        again = false;
      }
      if (got != kAll) return got;
    }
    if constexpr (BOUNDS) {
      bool inexact = false;
#pragma unroll
      for (int s = 0; s < SL; ++s) inexact |= d[s] > 0.0;
      if (got == kAll || (rule.softmax && bias && __any(inexact))) {
        // a kernel of its own does it for listed tokens; the workgroup where the list is full
        if (src.list.room > 0) {
          int at = 0;
          if (lane == 0) at = atomicAdd(src.list.count, 1);
          at = __builtin_amdgcn_readfirstlane(at);
          if (at < src.list.room) {
            if (lane == 0) src.list.tokens[at] = (int)t;
            return kDone;
          }
        }
#pragma unroll
        for (int s = 0; s < SL; ++s) redo |= (uint32_t)(d[s] > 0.0) << s;
        if (__any(redo != 0)) return kRedo;
      }
    }
    wave_lds_fence();
    return select_fp64<SL, BOUNDS>(l, d, bias, t, E, top_k, rule, s_c, s_d, s_pick, s_pv, s_pd, s_id,
                                   lane, redo, ids, weights);
  };
  if constexpr (BOUNDS) {
    __shared__ ExactQueue queue;
    bool done = !on;
    for (;;) {
      if (!done && !__any(redo != 0 || ask)) done = select() == kDone;
      if (!exact_round<SL>(src, queue, t0, M, wave, lane, redo, l, d, ask, mine)) break;
    }
  } else {
    select();
  }
}

// Exact logits of listed tokens, with the sums of exact_round: 8 experts of a token per
// workgroup at a time, two per wave.  Softmax scores with a bias: 3 to 5 tokens in 100 have two
// experts whose order hangs on the divisor, and so on every logit (one workgroup takes 460 us
// for one token's at E=512, H=7168).
__global__ __launch_bounds__(kSelWaves* kWave, 2) void exact_rows_kernel(BoundedSource src, int E,
                                                                          double* __restrict__ keys) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int groups = (E + 2 * kSelWaves - 1) / (2 * kSelWaves);
  const int64_t items = (int64_t)min(*src.list.count, src.list.room) * groups;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int64_t row = item / groups;
    const int e = (int)(item % groups) * 2 * kSelWaves + 2 * wave;
    if (e >= E) continue;
    const int64_t t = src.list.tokens[row];
    const int pair[2] = {e, min(e + 1, E - 1)};
    double part[2][kSelWaves];
#pragma unroll
    for (int quarter = 0; quarter < kSelWaves; ++quarter) {
      double sum[2];
      quarter_dots<2, 4>(src, t, pair, quarter, lane, sum);
      part[0][quarter] = sum[0];
      part[1][quarter] = sum[1];
    }
    if (lane < 2 && e + lane < E) {
      const double(&p)[kSelWaves] = part[0];
      const double(&q)[kSelWaves] = part[1];
      keys[row * E + e + lane] = lane == 0 ? ((p[0] + p[1]) + p[2]) + p[3]
                                           : ((q[0] + q[1]) + q[2]) + q[3];
    }
  }
}

template <int SL, typename SRC>
hipError_t launch_select_sl(const SRC& src, const float* bias, int M, int E, int top_k,
                            const GroupRule& rule, int32_t* ids, float* w, hipStream_t s) {
  constexpr bool BOUNDS = std::is_same<SRC, BoundedSource>::value;
  const size_t lds = (size_t)kSelWaves * select_lds_doubles(BOUNDS, E, top_k) * sizeof(double);
  const dim3 grid((unsigned)((M + kSelWaves - 1) / kSelWaves));   // M: rows of the source at most
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
  if constexpr (std::is_same<SRC, KeySource>::value || std::is_same<SRC, LogitSource>::value)
    return launch_select_sl<16>(src, bias, M, E, top_k, rule, ids, w, s);
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_route_logits(const float* logits, int64_t ld, const float* bias, int M, int E,
                               int top_k, const GroupRule& rule, int32_t* ids, float* w,
                               hipStream_t s) {
  return launch_select(LogitSource{{}, logits, ld}, bias, M, E, top_k, rule, ids, w, s);
}

namespace {

// K in parts (of whole 256-wide pieces) so that about 512 workgroups run; more than 8 cost the
// selection more than they save (M=333, E=160, H=4096: 4, 8, 16 parts 28, 26, 29 us in all).
constexpr int kBlMaxParts = 8, kBlWorkgroups = 512;
int bounded_parts(int64_t M, int E) {
  const int64_t tiles = (int64_t)((E + kBlTile - 1) / kBlTile) * ((M + kBlTile - 1) / kBlTile);
  return (int)std::min<int64_t>(kBlMaxParts, (kBlWorkgroups + tiles - 1) / tiles);
}

}  // namespace

// fp64 keys, or the parts' fp32 logits and |x| |w| sums: M times bounded_parts is at most
// M + 512 * 64 / (tiles of 64 experts), which grows with M, so that a workspace for some
// number of tokens does for fewer.
size_t route_groups_scratch_bytes(int M, int E) {
  const size_t etiles = (E + kBlTile - 1) / kBlTile;
  const size_t rows = std::min((size_t)M * kBlMaxParts, (size_t)M + kBlWorkgroups * kBlTile / etiles);
  return rows * E * 2 * sizeof(float);
}

// From this many logits on bounded fp32 MFMA sums replace fp64 ones for every (token, expert).
// Measured at H=7168, bounded against fp64, us: E=256 M=64 25 / 22, M=128 29 / 32, M=255 31 /
// 54; E=512 M=64 41 / 35, M=128 41 / 57; E=64 M=255 21 / 19.  Softmax scores with a bias, with
// the listed tokens' two launches: E=512 M=255 66 / 94, M=128 58 / 52, M=4096, k=8 154 / 1,322
// (k=16 205).  Not for few experts (a tile of 64 stays mostly empty), more than 512 (the selection
// spills 66 registers a lane from 257 on, and 16 slots a lane would spill twice as many), or a pick
// of nearly all, which leaves most choices open.
constexpr int kBoundedMinLogits = 40000, kBoundedMinExperts = 32, kBoundedMaxExperts = 512;

hipError_t launch_route_groups(const uint16_t* x, const uint16_t* wr, const float* bias, int M,
                               int H, int E, int top_k, const GroupRule& rule, int32_t* ids,
                               float* w, void* scratch, hipStream_t s) {
  const bool divisor = rule.softmax && bias;   // choices hang on every expert's logit
  if ((int64_t)M * E >= (divisor ? 2 : 1) * kBoundedMinLogits && E >= kBoundedMinExperts &&
      E <= kBoundedMaxExperts && top_k <= 64) {
    const int64_t tiles = (int64_t)((E + kBlTile - 1) / kBlTile) * ((M + kBlTile - 1) / kBlTile);
    const int pieces = (H + 255) / 256;
    int parts = std::min(bounded_parts(M, E), pieces);
    const int kpart = (pieces + parts - 1) / parts * 256;
    parts = (H + kpart - 1) / kpart;
    const int per_xcd = (int)((tiles * parts + kXcds - 1) / kXcds);
    float* logits = static_cast<float*>(scratch);
    float* absdot = logits + (size_t)parts * M * E;
    // behind them (8 bytes for a value are there, about 5 used): exact logits of one token in
    // eight, their list and its length
    const size_t used = ((size_t)parts * M * (E + (E + 3) / 4) * sizeof(float) + 7) / 8 * 8;
    double* keys = reinterpret_cast<double*>(static_cast<char*>(scratch) + used);
    TokenList list{nullptr, nullptr, 0};
    if (divisor) {
      const size_t left = route_groups_scratch_bytes(M, E) - used - sizeof(int);
      list.room = (int)std::min((size_t)M / 8, left / ((size_t)E * sizeof(double) + sizeof(int)));
      list.tokens = reinterpret_cast<int*>(keys + (size_t)list.room * E);
      list.count = list.tokens + list.room;
    }
    hipLaunchKernelGGL(bounded_logits_kernel, dim3((unsigned)per_xcd * kXcds), dim3(256), 0, s, x,
                       wr, M, H, E, parts, kpart, per_xcd, logits, absdot, list.count);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    const double rel = kBlRounds * 0x1p-23 * (1.0 + 0x1p-9);
    const BoundedSource src{{}, logits, absdot, x, wr, parts, M, H, rel, list};
    err = launch_select(src, bias, M, E, top_k, rule, ids, w, s);
    if (err != hipSuccess || !divisor) return err;
    hipLaunchKernelGGL(exact_rows_kernel, dim3(1024), dim3(kSelWaves* kWave), 0, s, src, E, keys);
    err = hipGetLastError();
    if (err != hipSuccess) return err;
    return launch_select(ListSource{keys, E, list}, bias, list.room, E, top_k, rule, ids, w, s);
  }
  double* keys = static_cast<double*>(scratch);
  constexpr int kMost = 1 << 17;   // tokens of one launch (its grid has them in y)
  for (int t0 = 0; t0 < M; t0 += kMost) {
    const hipError_t err = launch_router_keys(x + (size_t)t0 * H, wr, std::min(kMost, M - t0), H, E,
                                              keys + (size_t)t0 * E, s);
    if (err != hipSuccess) return err;
  }
  return launch_select(KeySource{{}, keys, E}, bias, M, E, top_k, rule, ids, w, s);
}

}  // namespace moe
