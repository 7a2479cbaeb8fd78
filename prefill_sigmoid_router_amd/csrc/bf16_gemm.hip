// bf16 matrix products with an epilogue:
//   h = x . w^T (fp32 sums) + bias;  v = act(h), or act(h[n]) * h[N + n] (GATED: w has 2 N rows,
//   gate rows first);  out = v + residual
//
// Sums, bias, activation and residual are fp32; the result is rounded once, to the type of out.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "launchers.h"
#include "tiled_common.h"

namespace moe {

namespace {

constexpr int kKC = 64;   // K values per chunk: one 128-byte line per row

// __expf is exp2 of a rounded product: within about (1.5 |z| + 2) 2^-24 of itself; the reciprocal
// within 2^-23.
__device__ __forceinline__ float sigmoid_fast(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}

template <int N>
__device__ __forceinline__ void activate(int act, float (&v)[N]) {
  switch (act) {   // the same for every lane
    case kActRelu:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = v[i] < 0.0f ? 0.0f : v[i];   // (NaN stays)
      break;
    case kActSilu:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] *= sigmoid_fast(v[i]);
      break;
    case kActGelu:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = 0.5f * v[i] * erfcf(-0.70710678f * v[i]);
      break;
    case kActGeluTanh:   // 1/2 (1 + tanh u) = sigmoid(2 u)
#pragma unroll
      for (int i = 0; i < N; ++i)
        v[i] *= sigmoid_fast(1.5957691f * fmaf(0.044715f * v[i] * v[i], v[i], v[i]));
      break;
    default: break;
  }
}

// N consecutive bf16 or fp32 values from element i on (16-byte aligned).
template <int N>
__device__ __forceinline__ void load_values(const void* p, bool f32, size_t i, float (&v)[N]) {
  if (f32) {
#pragma unroll
    for (int q = 0; q < N; q += 4) {
      const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i + q);
      v[q] = a.x;
      v[q + 1] = a.y;
      v[q + 2] = a.z;
      v[q + 3] = a.w;
    }
  } else {
#pragma unroll
    for (int q = 0; q < N; q += 8) {
      const u32x4 a = ld16(static_cast<const uint16_t*>(p) + i + q);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[q + 2 * j] = bf16lo(a[j]);
        v[q + 2 * j + 1] = bf16hi(a[j]);
      }
    }
  }
}
template <int N>
__device__ __forceinline__ void store_values(void* p, bool f32, size_t i, const float (&v)[N]) {
  if (f32) {
#pragma unroll
    for (int q = 0; q < N; q += 4)
      *reinterpret_cast<float4*>(static_cast<float*>(p) + i + q) =
          make_float4(v[q], v[q + 1], v[q + 2], v[q + 3]);
  } else {
#pragma unroll
    for (int q = 0; q < N; q += 8) {
      u32x4 a;
#pragma unroll
      for (int j = 0; j < 4; ++j) a[j] = pack_bf16x2(v[q + 2 * j], v[q + 2 * j + 1]);
      st16(static_cast<uint16_t*>(p) + i + q, a);
    }
  }
}
__device__ __forceinline__ float load_value(const void* p, bool f32, size_t i) {
  return f32 ? static_cast<const float*>(p)[i] : bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
}
__device__ __forceinline__ void store_value(void* p, bool f32, size_t i, float v) {
  if (f32) static_cast<float*>(p)[i] = v;
  else static_cast<uint16_t*>(p)[i] = (uint16_t)f32_to_bf16_rne(v);
}

// One result: sums h (gate) and u (up rows, GATED) of token m, column n.
template <bool GATED>
__device__ __forceinline__ void finish_one(const GemmArgs& p, int m, int n, float h, float u) {
  if (p.bias) {
    h += bf16_to_f32(p.bias[n]);
    if (GATED) u += bf16_to_f32(p.bias[p.N + n]);
  }
  float v[1] = {h};
  activate(p.act, v);
  if (GATED) v[0] *= u;
  if (p.residual) v[0] += load_value(p.residual, p.residual_f32, (size_t)m * p.residual_ld + n);
  store_value(p.out, p.out_f32, (size_t)m * p.out_ld + n, v[0]);
}

// C results of token m, columns n .. n + C - 1 (n a multiple of 8).
template <bool GATED, int C>
__device__ __forceinline__ void finish(const GemmArgs& p, int m, int n, float (&h)[C], float (&u)[C]) {
  if (!p.wide || n + C > p.N) {
#pragma unroll 1
    for (int i = 0; i < C && n + i < p.N; ++i) {
      float a = h[0], b = u[0];   // (no indexed registers)
#pragma unroll
      for (int q = 1; q < C; ++q) {
        a = q == i ? h[q] : a;
        b = q == i ? u[q] : b;
      }
      finish_one<GATED>(p, m, n + i, a, b);
    }
    return;
  }
  float t[C];
  if (p.bias) {
    load_values(p.bias, false, n, t);
#pragma unroll
    for (int i = 0; i < C; ++i) h[i] += t[i];
    if (GATED) {
      load_values(p.bias, false, (size_t)p.N + n, t);
#pragma unroll
      for (int i = 0; i < C; ++i) u[i] += t[i];
    }
  }
  activate(p.act, h);
  if (GATED) {
#pragma unroll
    for (int i = 0; i < C; ++i) h[i] *= u[i];
  }
  if (p.residual) {
    load_values(p.residual, p.residual_f32, (size_t)m * p.residual_ld + n, t);
#pragma unroll
    for (int i = 0; i < C; ++i) h[i] += t[i];
  }
  store_values(p.out, p.out_f32, (size_t)m * p.out_ld + n, h);
}

// LDS rows are one 128-byte line of a chunk each; 16-byte slot q of row r holds the part
// q ^ f(r) of the line, with f chosen so that the 16 rows of a fragment read (which also differ
// in r % 2) meet no bank twice.  Token fragments are 16 consecutive rows.  Weight fragment j of a
// wave's rows holds rows SPAN (i / 4) + 4 j + i % 4, i = 0 .. 15, SPAN = 8 (GATED) or 16: a lane's
// results of all the fragments then are SPAN consecutive columns.
__device__ __forceinline__ int token_swizzle(int r) { return (r >> 1) & 7; }
template <int SPAN>
__device__ __forceinline__ int weight_swizzle(int r) {
  return ((r >> 1) & 1) | ((r / SPAN) & 3) << 1;
}

// Tiles of BM tokens x 64 WN weight rows (GATED: 32 WN gate and as many up rows), K in chunks
// of 64.  Both operands are copied global -> LDS in 1 KiB pieces of 8 rows x one line.  A ring of
// S stages keeps S - 1 chunks in flight; each wave waits for its own copies and a bare barrier
// publishes them.  Only a partial last chunk goes through registers (zero-filled).
template <int BM, int WN, int WM>
struct RingCfg {
  static constexpr int WT = 4 * WN;              // weight row tiles of 16
  static constexpr int MT = BM / 16;             // token row tiles
  static constexpr int MTW = MT / WM;            // token row tiles per wave
  static constexpr int PIECES = (WT + MT) * 2;   // 1 KiB copies per chunk
  static constexpr int PPW = PIECES / (WN * WM);
  static_assert(PIECES % (WN * WM) == 0, "copies must split evenly over the waves");
  static_assert(MT % WM == 0, "token tiles must split evenly over the waves");
};

template <int PPW, int A>
__device__ __forceinline__ void wait_after(int after) {
  if constexpr (A <= 0) {
    wait_vmcnt<0>();
  } else {
    if (after >= A) wait_vmcnt<A * PPW>();
    else wait_after<PPW, A - 1>(after);
  }
}

template <int BM, int WN, int WM, int S, bool GATED>
__global__ __launch_bounds__(64 * WN * WM) void ring_kernel(GemmArgs p) {
  using C = RingCfg<BM, WN, WM>;
  static_assert((S - 2) * C::PPW <= 63, "the copies in flight must fit the vmcnt counter");
  static_assert(S * C::PIECES * 1024 <= 160 * 1024, "the ring must fit the LDS");
  __shared__ __align__(16) unsigned char lds[S * C::PIECES * 1024];
  constexpr int SPAN = GATED ? 8 : 16, COLS = GATED ? 32 * WN : 64 * WN;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int li = lane & 15, lg = lane >> 4;
  const int wn = wave % WN, wm = wave / WN;
  const int K = p.K;
  TiledWalk walk((p.M + BM - 1) / BM, (p.N + COLS - 1) / COLS);
  int ntile, ti;
  while (walk.next(ntile, ti)) {
    const int start = ti * BM, nlive = min(BM, p.M - start), col0 = ntile * COLS;
    const int mt_active = (nlive + 15) >> 4;
    // piece f of a chunk: LDS rows 8f .. 8f + 7 (weight rows first); lane l copies slot l % 8
    // of row 8f + l / 8.  Rows past the last repeat it; their results are never stored.
    const uint16_t* src[C::PPW];
    int koff[C::PPW];
#pragma unroll
    for (int i = 0; i < C::PPW; ++i) {
      const int lr = 8 * (wave * C::PPW + i) + (lane >> 3);
      if (lr < 64 * WN) {
        koff[i] = 8 * ((lane & 7) ^ weight_swizzle<SPAN>(lr));
        const bool up = GATED && lr >= 32 * WN;
        const int col = min(col0 + (up ? lr - 32 * WN : lr), p.N - 1);
        src[i] = p.w + (size_t)(up ? p.N + col : col) * K + koff[i];
      } else {
        const int r = lr - 64 * WN;
        koff[i] = 8 * ((lane & 7) ^ token_swizzle(r));
        src[i] = p.x + (size_t)(start + min(r, nlive - 1)) * p.x_ld + koff[i];
      }
    }
    const int nch = (K + kKC - 1) / kKC, ndma = K / kKC;   // chunks, whole ones
    auto issue = [&](int c) {
      unsigned char* base = lds + (size_t)(c % S) * C::PIECES * 1024 + wave * C::PPW * 1024;
      if (c < ndma) {
#pragma unroll
        for (int i = 0; i < C::PPW; ++i)
          __builtin_amdgcn_global_load_lds((global_void*)(src[i] + (size_t)c * kKC),
                                           (lds_void*)(base + i * 1024), 16, 0, 0);
      } else {
#pragma unroll
        for (int i = 0; i < C::PPW; ++i)
          *reinterpret_cast<u32x4*>(base + i * 1024 + lane * 16) =
              c * kKC + koff[i] < K ? ld16(src[i] + (size_t)c * kKC) : u32x4{0, 0, 0, 0};
      }
    };
    const int wrow = (GATED ? 32 : 64) * wn + SPAN * (li >> 2) + (li & 3);
    const int wslot = weight_swizzle<SPAN>(wrow), tslot = token_swizzle(li);
    auto frag = [&](int c, int row, int slot) -> u32x4 {
      return *reinterpret_cast<const u32x4*>(lds + (size_t)(c % S) * C::PIECES * 1024 + row * 128 +
                                             slot * 16);
    };
    f32x4 acc[4][C::MTW];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int s = 0; s < C::MTW; ++s) acc[j][s] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int my_active = mt_active - wm * C::MTW;
#pragma unroll
    for (int q = 0; q < S - 1; ++q)
      if (q < nch) issue(q);
    for (int c = 0; c < nch; ++c) {
      // this wave's whole chunks issued after c (the tail chunk's loads are complete when
      // they are stored)
      wait_after<C::PPW, S - 2>(c < ndma ? min(S - 2, ndma - 1 - c) : 0);
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      if (c + S - 1 < nch) issue(c + S - 1);
      if (my_active > 0) {
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          u32x4 wa[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            wa[j] = frag(c, GATED ? wrow + 4 * (j & 1) + (j >> 1) * 32 * WN : wrow + 4 * j,
                         (lg + 4 * ks) ^ wslot);
#pragma unroll
          for (int s = 0; s < C::MTW; ++s) {
            if (s < my_active) {
              const u32x4 xb = frag(c, 64 * WN + 16 * (wm * C::MTW + s) + li, (lg + 4 * ks) ^ tslot);
#pragma unroll
              for (int j = 0; j < 4; ++j) acc[j][s] = mfma16x16x32(wa[j], xb, acc[j][s]);
            }
          }
        }
      }
    }
    // lane (li, lg) holds token row li of each token tile and SPAN columns from n0 on
    const int n0 = col0 + (GATED ? 32 : 64) * wn + SPAN * lg;
#pragma unroll
    for (int s = 0; s < C::MTW; ++s) {
      const int r = 16 * (wm * C::MTW + s) + li;
      if (s >= my_active || r >= nlive || n0 >= p.N) continue;
      float h[SPAN], u[SPAN];
#pragma unroll
      for (int q = 0; q < SPAN; ++q) {
        h[q] = acc[q >> 2][s][q & 3];
        u[q] = GATED ? acc[2 + (q >> 2 & 1)][s][q & 3] : 0.0f;
      }
      finish<GATED>(p, start + r, n0, h, u);
    }
    __syncthreads();   // the next item's first copies reuse the ring
  }
}

template <int BM, int WN, int WM, int S, bool GATED>
hipError_t launch_ring(const GemmArgs& a, hipStream_t s) {
  const int cols = GATED ? 32 * WN : 64 * WN;
  const long items = (long)((a.M + BM - 1) / BM) * ((a.N + cols - 1) / cols);
  const long grid = walk_grid(items, S * RingCfg<BM, WN, WM>::PIECES * 1024);
  hipLaunchKernelGGL((ring_kernel<BM, WN, WM, S, GATED>), dim3((unsigned)grid), dim3(64 * WN * WM), 0,
                     s, a);
  return hipGetLastError();
}

// Few tokens: 16 weight rows (GATED: 8 gate and 8 up rows) x 16 MT tokens per workgroup, the
// 64-wide units of K dealt over its 8 waves, whose sums meet in LDS in a fixed order.  Fragments
// come straight from memory (a weight row's line is read by one wave), BATCH units at a time in
// flight.
template <int MT, bool GATED>
__global__ __launch_bounds__(512) void skinny_kernel(GemmArgs p, int n_ntiles, int mblocks, int per_xcd) {
  constexpr int WAVES = 8, BATCH = MT == 1 ? 4 : MT == 2 ? 2 : 1, COLS = GATED ? 8 : 16;
  __shared__ float part[WAVES][MT][4][kWave];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int li = lane & 15, lg = lane >> 4;
  // the token blocks of a weight tile run on one XCD
  const int slot = blockIdx.x / kXcds, item = (blockIdx.x % kXcds) * per_xcd + slot;
  if (slot >= per_xcd || item >= n_ntiles * mblocks) return;
  const int n0 = item / mblocks * COLS, m0 = item % mblocks * (16 * MT);
  const int K = p.K, units = (K + kKC - 1) / kKC, whole = K / kKC;
  const int col = min(n0 + (GATED ? li & 7 : li), p.N - 1);
  const uint16_t* wrow = p.w + (size_t)(GATED && li >= 8 ? p.N + col : col) * K + 8 * lg;
  const uint16_t* trow[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) trow[t] = p.x + (size_t)min(m0 + 16 * t + li, p.M - 1) * p.x_ld + 8 * lg;
  f32x4 acc[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int u0 = wave; u0 < units; u0 += WAVES * BATCH) {
    u32x4 w[BATCH][2], x[BATCH][MT][2];
#pragma unroll
    for (int b = 0; b < BATCH; ++b) {
      const int u = u0 + WAVES * b;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // behind column K zeros meet zeros
        const bool in = u < whole || (u < units && u * kKC + 32 * h + 8 * lg < K);
        const size_t off = (size_t)u * kKC + 32 * h;
        w[b][h] = in ? ld16(wrow + off) : u32x4{0, 0, 0, 0};
#pragma unroll
        for (int t = 0; t < MT; ++t) x[b][t][h] = in ? ld16(trow[t] + off) : u32x4{0, 0, 0, 0};
      }
    }
#pragma unroll
    for (int b = 0; b < BATCH; ++b)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[t] = mfma16x16x32(w[b][h], x[b][t][h], acc[t]);
  }
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int q = 0; q < 4; ++q) part[wave][t][q][lane] = acc[t][q];
  __syncthreads();
  // thread -> token r, column c: weight row c is result c % 4 of lane 16 (c / 4) + r % 16 of
  // token tile r / 16
  for (int i = threadIdx.x; i < COLS * 16 * MT; i += 64 * WAVES) {
    const int r = i / COLS, c = i % COLS;
    if (m0 + r >= p.M || n0 + c >= p.N) continue;
    float h = 0.0f, u = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      h += part[w][r >> 4][c & 3][16 * (c >> 2) + (r & 15)];
      if (GATED) u += part[w][r >> 4][c & 3][16 * ((c + 8) >> 2) + (r & 15)];
    }
    finish_one<GATED>(p, m0 + r, n0 + c, h, u);
  }
}

template <int MT, bool GATED>
hipError_t launch_skinny(const GemmArgs& a, hipStream_t s) {
  const int n_ntiles = (a.N + (GATED ? 7 : 15)) / (GATED ? 8 : 16);
  const int mblocks = (a.M + 16 * MT - 1) / (16 * MT);
  const int64_t per_xcd = ((int64_t)n_ntiles * mblocks + kXcds - 1) / kXcds;
  hipLaunchKernelGGL((skinny_kernel<MT, GATED>), dim3((unsigned)(per_xcd * kXcds)), dim3(512), 0, s, a,
                     n_ntiles, mblocks, (int)per_xcd);
  return hipGetLastError();
}

template <bool GATED>
hipError_t launch_sized(const GemmArgs& a, hipStream_t s) {
  if (a.M <= 16) return launch_skinny<1, GATED>(a, s);
  if (a.M <= 32) return launch_skinny<2, GATED>(a, s);
  if (a.M <= 512) return launch_ring<64, 1, 4, 4, GATED>(a, s);
  return launch_ring<128, 4, 2, 3, GATED>(a, s);
}

}  // namespace

hipError_t launch_bf16_matmul(const GemmArgs& a, hipStream_t s) {
  return a.gated ? launch_sized<true>(a, s) : launch_sized<false>(a, s);
}

}  // namespace moe
