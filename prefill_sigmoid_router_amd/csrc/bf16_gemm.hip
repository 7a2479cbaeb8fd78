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
// within 2^-23.  Where it would be subnormal (z < -87) it may be 0.
__device__ __forceinline__ float sigmoid_fast(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}

// h Phi(h).  With t = 1 / (1 + |h| / 8^1/2), erfc(|h| / 2^1/2) = t 2^(P(t) - h^2 log2(e) / 2); P is a
// Chebyshev fit over t in [1/8, 1] of log2(erfc(z) e^(z^2) / t), z = 2 / t - 2, good to 2^-23.  With
// the exponent's roundings the result is within (1.25 h^2 + 14) 2^-24 of itself (erfcf of the device
// library takes four times the instructions).
__device__ __forceinline__ float gelu_exact(float h) {
  const float t = __builtin_amdgcn_rcpf(fmaf(fabsf(h), 0.35355339f, 1.0f));
  float s = 0.2387803f;
  s = fmaf(s, t, -1.1418399f);
  s = fmaf(s, t, 2.0388212f);
  s = fmaf(s, t, -1.4883672f);
  s = fmaf(s, t, 0.27622172f);
  s = fmaf(s, t, -0.20144565f);
  s = fmaf(s, t, 0.117095776f);
  s = fmaf(s, t, 0.54421836f);
  s = fmaf(s, t, 1.4422425f);
  s = fmaf(s, t, -1.825727f);
  const float e = t * __builtin_amdgcn_exp2f(fmaf(h * h, -0.72134752f, s));
  return h < 0.0f ? 0.5f * h * e : h * fmaf(e, -0.5f, 1.0f);
}

template <int R, int C>
__device__ __forceinline__ void activate(int act, float (&v)[R][C]) {
  auto each = [&](auto f) {
#pragma unroll
    for (int k = 0; k < R; ++k)
#pragma unroll
      for (int q = 0; q < C; ++q) v[k][q] = f(v[k][q]);
  };
  switch (act) {   // the same for every lane
    case kActRelu: each([](float z) { return z < 0.0f ? 0.0f : z; }); break;   // (NaN stays)
    case kActSilu: each([](float z) { return z * sigmoid_fast(z); }); break;
    case kActGelu: each([](float z) { return gelu_exact(z); }); break;
    case kActGeluTanh:   // 1/2 (1 + tanh u) = sigmoid(2 u)
      each([](float z) { return z * sigmoid_fast(1.5957691f * fmaf(0.044715f * z * z, z, z)); });
      break;
    default: break;
  }
}

__device__ __forceinline__ float load_value(const void* p, bool f32, size_t i) {
  return f32 ? static_cast<const float*>(p)[i] : bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
}
__device__ __forceinline__ void store_value(void* p, bool f32, size_t i, float v) {
  if (f32) static_cast<float*>(p)[i] = v;
  else static_cast<uint16_t*>(p)[i] = (uint16_t)f32_to_bf16_rne(v);
}

// C values of a row from column n on (a multiple of 8) go 16 bytes at a time, or one by one.
template <int C>
__device__ __forceinline__ bool wide_at(const GemmArgs& p, int n) {
  return p.wide && n + C <= p.N;
}

// C values of bias for the columns n ..; gated: those of the up rows, `from` = N values on.
template <int C>
__device__ __forceinline__ void load_bias(const GemmArgs& p, int n, int from, float (&b)[C]) {
#pragma unroll
  for (int q = 0; q < C; ++q) b[q] = 0.0f;
  if (!p.bias) return;
  const uint16_t* src = p.bias + from + n;
  if (wide_at<C>(p, n)) {
#pragma unroll
    for (int q = 0; q < C; q += 8) {
      const u32x4 a = ld16(src + q);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        b[q + 2 * j] = bf16lo(a[j]);
        b[q + 2 * j + 1] = bf16hi(a[j]);
      }
    }
  } else {
#pragma unroll
    for (int q = 0; q < C; ++q)
      if (n + q < p.N) b[q] = bf16_to_f32(src[q]);
  }
}

// C values of the residual's row m, as they come: in flight until they are needed.
template <int C>
struct Residual {
  uint32_t r[C];
  __device__ __forceinline__ void load(const GemmArgs& p, int m, int n) {
    const size_t i = (size_t)m * p.residual_ld + n;
    if (wide_at<C>(p, n)) {
      const char* src = static_cast<const char*>(p.residual) + i * (p.residual_f32 ? 4 : 2);
#pragma unroll
      for (int q = 0; q < C / 4; ++q)
        if (q < C / 8 || p.residual_f32) {
          const u32x4 a = ld16(src + 16 * q);
#pragma unroll
          for (int j = 0; j < 4; ++j) r[4 * q + j] = a[j];
        }
    } else {
#pragma unroll
      for (int q = 0; q < C; ++q)
        r[q] = n + q < p.N ? __float_as_uint(load_value(p.residual, p.residual_f32, i + q)) : 0u;
    }
  }
  __device__ __forceinline__ void add(const GemmArgs& p, int n, float (&v)[C]) const {
    if (wide_at<C>(p, n) && !p.residual_f32) {
#pragma unroll
      for (int q = 0; q < C; q += 2) {
        v[q] += bf16lo(r[q / 2]);
        v[q + 1] += bf16hi(r[q / 2]);
      }
    } else {
#pragma unroll
      for (int q = 0; q < C; ++q) v[q] += __uint_as_float(r[q]);
    }
  }
};

// C results each of R tokens m (those from p.M on are left out), columns n ..: sums h (of the gate
// rows) and u (of the up rows, GATED), and what is added to them.  before_stores issues loads for
// later: issued behind the stores they would wait for them.
template <bool GATED, int R, int C, class F>
__device__ __forceinline__ void finish(const GemmArgs& p, const int (&m)[R], int n, float (&h)[R][C],
                                       float (&u)[R][C], const float (&bh)[C], const float (&bu)[C],
                                       const Residual<C> (&res)[R], F before_stores) {
  if (p.bias) {
#pragma unroll
    for (int k = 0; k < R; ++k)
#pragma unroll
      for (int q = 0; q < C; ++q) {
        h[k][q] += bh[q];
        if (GATED) u[k][q] += bu[q];
      }
  }
  activate(p.act, h);
  if (GATED) {
#pragma unroll
    for (int k = 0; k < R; ++k)
#pragma unroll
      for (int q = 0; q < C; ++q) h[k][q] *= u[k][q];
  }
  if (p.residual) {
#pragma unroll
    for (int k = 0; k < R; ++k) res[k].add(p, n, h[k]);
  }
  before_stores();
  if (wide_at<C>(p, n)) {
#pragma unroll
    for (int k = 0; k < R; ++k) {
      if (m[k] >= p.M) continue;
      const size_t o = (size_t)m[k] * p.out_ld + n;
      if (p.out_f32) {
#pragma unroll
        for (int q = 0; q < C; q += 4)
          *reinterpret_cast<float4*>(static_cast<float*>(p.out) + o + q) =
              make_float4(h[k][q], h[k][q + 1], h[k][q + 2], h[k][q + 3]);
      } else {
#pragma unroll
        for (int q = 0; q < C; q += 8) {
          u32x4 a;
#pragma unroll
          for (int j = 0; j < 4; ++j) a[j] = cvt_bf16x2(h[k][q + 2 * j], h[k][q + 2 * j + 1]);
          st16(static_cast<uint16_t*>(p.out) + o + q, a);
        }
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < R; ++k) {
      if (m[k] >= p.M) continue;
      const size_t o = (size_t)m[k] * p.out_ld + n;
#pragma unroll
      for (int q = 0; q < C; ++q)
        if (n + q < p.N) store_value(p.out, p.out_f32, o + q, h[k][q]);
    }
  }
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
// S stages keeps S chunks in flight; each wave waits for its own copies and a bare barrier
// publishes them.  Only a partial last chunk goes through registers (zero-filled).  A chunk's
// fragments are read while the one before is multiplied (without that a chunk of a 64 x 64 tile took
// 0.40 us, most of it LDS latency).
// SPLIT: an item is a tile and one of p.splits parts of K, whose fp32 sums go to p.partial
// [splits][M][p.partial_ld] (GATED: the up rows' columns behind the gate rows'), where join_kernel
// adds them in order.
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

template <int BM, int WN, int WM, int S, bool GATED, bool SPLIT>
__global__ __launch_bounds__(64 * WN * WM) void ring_kernel(GemmArgs p) {
  using C = RingCfg<BM, WN, WM>;
  static_assert((S - 1) * C::PPW <= 63, "the copies in flight must fit the vmcnt counter");
  static_assert(S * C::PIECES * 1024 <= 160 * 1024, "the ring must fit the LDS");
  __shared__ __align__(16) unsigned char lds[S * C::PIECES * 1024];
  constexpr int SPAN = GATED ? 8 : 16, COLS = GATED ? 32 * WN : 64 * WN;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int li = lane & 15, lg = lane >> 4;
  const int wn = wave % WN, wm = wave / WN;
  const int K = p.K;
  const int all = (K + kKC - 1) / kKC, ndma = K / kKC;   // chunks, whole ones
  const int ntiles = (p.N + COLS - 1) / COLS;
  TiledWalk walk((p.M + BM - 1) / BM, SPLIT ? ntiles * p.splits : ntiles);
  int ntile, ti;
  while (walk.next(ntile, ti)) {
    const int split = SPLIT ? ntile % p.splits : 0;
    if (SPLIT) ntile /= p.splits;
    const int first = SPLIT ? (int)((int64_t)all * split / p.splits) : 0;
    const int nch = SPLIT ? (int)((int64_t)all * (split + 1) / p.splits) : all;
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
        src[i] = p.w + (size_t)(up ? p.N + col : col) * K + koff[i] + (size_t)first * kKC;
      } else {
        const int r = lr - 64 * WN;
        koff[i] = 8 * ((lane & 7) ^ token_swizzle(r));
        src[i] = p.x + (size_t)(start + min(r, nlive - 1)) * p.x_ld + koff[i] + (size_t)first * kKC;
      }
    }
    constexpr int STAGE = C::PIECES * 1024;
    int put = 0, get = 0;   // stages that the next copy fills, that the next chunk is read from
    auto copy = [&] {   // the next chunk, a whole one
      unsigned char* base = lds + put * STAGE + wave * C::PPW * 1024;
      put = put == S - 1 ? 0 : put + 1;
#pragma unroll
      for (int i = 0; i < C::PPW; ++i) {
        __builtin_amdgcn_global_load_lds((global_void*)src[i], (lds_void*)(base + i * 1024), 16, 0, 0);
        src[i] += kKC;
      }
    };
    auto issue = [&](int c) {   // the next chunk, c
      if (c < ndma) {
        copy();
        return;
      }
      unsigned char* base = lds + put * STAGE + wave * C::PPW * 1024;
      put = put == S - 1 ? 0 : put + 1;
#pragma unroll
      for (int i = 0; i < C::PPW; ++i)
        *reinterpret_cast<u32x4*>(base + i * 1024 + lane * 16) =
            c * kKC + koff[i] < K ? ld16(src[i]) : u32x4{0, 0, 0, 0};
    };
    const int my_active = mt_active - wm * C::MTW;
    const int wrow = (GATED ? 32 : 64) * wn + SPAN * (li >> 2) + (li & 3);
    const int waddr = wrow * 128 + 16 * (lg ^ weight_swizzle<SPAN>(wrow));
    const int taddr = (64 * WN + 16 * C::MTW * wm + li) * 128 + 16 * (lg ^ token_swizzle(li));
    u32x4 wa[2][2][4], xb[2][2][C::MTW];   // fragments of even and odd chunks, both halves of K
    auto read = [&](int set) {   // of the next chunk
      const unsigned char* base = lds + get * STAGE;
      get = get == S - 1 ? 0 : get + 1;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {   // half ks: slot lg + 4 ks, that is byte 64 ks flipped
#pragma unroll
        for (int j = 0; j < 4; ++j)
          wa[set][ks][j] = *reinterpret_cast<const u32x4*>(
              base + (waddr ^ 64 * ks) + 512 * (GATED ? j & 1 : j) + (GATED ? (j >> 1) * 32 * WN * 128 : 0));
#pragma unroll
        for (int s = 0; s < C::MTW; ++s)
          xb[set][ks][s] = *reinterpret_cast<const u32x4*>(base + (taddr ^ 64 * ks) + 2048 * s);
      }
    };
    f32x4 acc[4][C::MTW];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int s = 0; s < C::MTW; ++s) acc[j][s] = f32x4{0.f, 0.f, 0.f, 0.f};
    // Chunk c has landed, and chunk c - 1 has been read: this wave's whole chunks issued after c
    // may be in flight (the tail chunk's loads are complete when they are stored).
    auto landed = [&](int c, int after) {
      wait_after<C::PPW, S - 1>(c < ndma ? min(after, min(ndma, nch) - 1 - c) : 0);
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    };
#pragma unroll
    for (int q = 0; q < S; ++q)
      if (first + q < nch) issue(first + q);
    landed(first, S - 1);
    read(0);
    // Chunk c is multiplied while the next one's fragments are read and chunk c + S is copied into
    // the stage that c has left.  ON: those exist and are whole.
    auto step = [&](int c, auto parity, auto on) {
      constexpr int set = decltype(parity)::value;
      constexpr bool ON = decltype(on)::value;
      if (ON) {
        wait_vmcnt<(S - 2) * C::PPW>();
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        copy();
        read(set ^ 1);
      } else if (c + 1 < nch) {
        landed(c + 1, S - 2);
        if (c + S < nch) issue(c + S);
        read(set ^ 1);
      }
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int s = 0; s < C::MTW; ++s)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[j][s] = mfma16x16x32(wa[set][ks][j], xb[set][ks][s], acc[j][s]);
    };
    const std::integral_constant<int, 0> even{};
    const std::integral_constant<int, 1> odd{};
    int c = first;
#pragma unroll 1
    for (; c + 1 + S < min(nch, ndma); c += 2) {
      step(c, even, std::true_type{});
      step(c + 1, odd, std::true_type{});
    }
#pragma unroll 1
    for (; c < nch; c += 2) {
      step(c, even, std::false_type{});
      if (c + 1 < nch) step(c + 1, odd, std::false_type{});
    }
    // lane (li, lg) holds token row li of each token tile and SPAN columns from n0 on
    const int n0 = col0 + (GATED ? 32 : 64) * wn + SPAN * lg;
    if constexpr (SPLIT) {
#pragma unroll
      for (int s = 0; s < C::MTW; ++s) {
        const int r = 16 * (wm * C::MTW + s) + li;
        if (r >= nlive || n0 >= p.N) continue;
        float* dst = p.partial + ((size_t)split * p.M + start + r) * p.partial_ld + n0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float* at = !GATED ? dst + 4 * j : dst + (j >> 1) * (p.partial_ld / 2) + 4 * (j & 1);
          *reinterpret_cast<f32x4*>(at) = acc[j][s];   // (rows are whole numbers of tiles' columns)
        }
      }
    } else if (n0 < p.N && my_active > 0) {
      float bh[SPAN], bu[SPAN];
      load_bias(p, n0, 0, bh);
      if (GATED) load_bias(p, n0, p.N, bu);
      Residual<SPAN> res[C::MTW];
      if (p.residual) {
#pragma unroll
        for (int s = 0; s < C::MTW; ++s)
          res[s].load(p, start + min(16 * (wm * C::MTW + s) + li, nlive - 1), n0);
      }
      float h[C::MTW][SPAN], u[C::MTW][SPAN];
      int m[C::MTW];
#pragma unroll
      for (int s = 0; s < C::MTW; ++s) {
        const int r = 16 * (wm * C::MTW + s) + li;
        m[s] = r < nlive ? start + r : p.M;
#pragma unroll
        for (int q = 0; q < SPAN; ++q) {
          h[s][q] = acc[q >> 2][s][q & 3];
          u[s][q] = GATED ? acc[2 + (q >> 2 & 1)][s][q & 3] : 0.0f;
        }
      }
      finish<GATED>(p, m, n0, h, u, bh, bu, res, [] {});
    }
    __syncthreads();   // the next item's first copies reuse the ring
  }
}

// Sums of the parts of K, in order, and the epilogue: 8 columns of a token per thread.
template <bool GATED>
__global__ __launch_bounds__(256) void join_kernel(GemmArgs p) {
  const int groups = (p.N + 7) / 8;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)p.M * groups) return;
  const int m[1] = {(int)(i / groups)}, n = (int)(i % groups) * 8;
  float h[1][8], u[1][8], bh[8], bu[8];
  Residual<8> res[1];
  if (p.residual) res[0].load(p, m[0], n);
  load_bias(p, n, 0, bh);
  if (GATED) load_bias(p, n, p.N, bu);
#pragma unroll
  for (int q = 0; q < 8; ++q) h[0][q] = u[0][q] = 0.0f;
#pragma unroll 8
  for (int s = 0; s < p.splits; ++s) {
    const float* src = p.partial + ((size_t)s * p.M + m[0]) * p.partial_ld + n;
#pragma unroll
    for (int q = 0; q < 8; q += 4) {
      const f32x4 a = *reinterpret_cast<const f32x4*>(src + q);
      f32x4 b = f32x4{0.f, 0.f, 0.f, 0.f};
      if (GATED) b = *reinterpret_cast<const f32x4*>(src + p.partial_ld / 2 + q);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        h[0][q + e] += a[e];
        u[0][q + e] += b[e];
      }
    }
  }
  finish<GATED>(p, m, n, h, u, bh, bu, res, [] {});
}

template <int BM, int WN, int WM, int S, bool GATED>
hipError_t launch_ring(const GemmArgs& a, hipStream_t s) {
  const int cols = GATED ? 32 * WN : 64 * WN;
  const long items = (long)((a.M + BM - 1) / BM) * ((a.N + cols - 1) / cols);
  const long grid = walk_grid(items, S * RingCfg<BM, WN, WM>::PIECES * 1024);
  hipLaunchKernelGGL((ring_kernel<BM, WN, WM, S, GATED, false>), dim3((unsigned)grid), dim3(64 * WN * WM),
                     0, s, a);
  return hipGetLastError();
}

// 64 x 64 tiles with K in parts.
constexpr int kSplitLd = 64;   // rows of partial sums are a multiple of a tile's columns
int partial_ld(int N, bool gated) {
  const int cols = gated ? kSplitLd / 2 : kSplitLd;
  return (N + cols - 1) / cols * kSplitLd;
}
template <bool GATED>
hipError_t launch_split(GemmArgs a, int splits, float* partial, hipStream_t s) {
  const int cols = GATED ? 32 : 64;
  a.splits = splits;
  a.partial = partial;
  a.partial_ld = partial_ld(a.N, GATED);
  const long items = (long)((a.M + 63) / 64) * ((a.N + cols - 1) / cols) * splits;
  const long grid = walk_grid(items, 4 * RingCfg<64, 1, 4>::PIECES * 1024);
  hipLaunchKernelGGL((ring_kernel<64, 1, 4, 4, GATED, true>), dim3((unsigned)grid), dim3(256), 0, s, a);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const int64_t threads = (int64_t)a.M * ((a.N + 7) / 8);
  hipLaunchKernelGGL((join_kernel<GATED>), dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, s, a);
  return hipGetLastError();
}

// Few tokens: 16 weight rows (GATED: 8 gate and 8 up rows) x 8 XP tokens per workgroup, the
// 64-wide units of K dealt over its 8 waves, whose sums meet in LDS in a fixed order.  A wave copies
// its units global -> LDS in 1 KiB pieces of 8 rows x one line, two at a time in flight (three to six
// were no faster: the LDS then holds fewer workgroups), and waits for nobody else's.  Bound by the
// weights: M = 8, N = 4096, K = 7168 10.8 us (5.4 TB/s), M = 32 11.9.  (Fragments straight from
// memory, each lane its row's 16 bytes, took 13.5 and 21.4: 64 lines to look up per load.)
template <int XP, bool GATED>
__global__ __launch_bounds__(512) void skinny_kernel(GemmArgs p, int n_ntiles, int mblocks, int per_xcd) {
  constexpr int WAVES = 8, AHEAD = 2, COLS = GATED ? 8 : 16, MT = (XP + 1) / 2, PIECES = 2 + XP;
  constexpr int UNIT = PIECES * 1024;
  static_assert(WAVES * AHEAD * UNIT <= 160 * 1024, "the units in flight must fit the LDS");
  static_assert(AHEAD * UNIT >= MT * 1024, "the sums take the units' place");
  __shared__ __align__(16) unsigned char lds[WAVES * AHEAD * UNIT];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int li = lane & 15, lg = lane >> 4;
  // the token blocks of a weight tile run on one XCD
  const int slot = blockIdx.x / kXcds, item = (blockIdx.x % kXcds) * per_xcd + slot;
  if (slot >= per_xcd || item >= n_ntiles * mblocks) return;
  const int n0 = item / mblocks * COLS, m0 = item % mblocks * (8 * XP);
  const int K = p.K, units = (K + kKC - 1) / kKC, whole = K / kKC;
  // piece f: rows 8f .. 8f + 7 (weight rows first); lane l copies slot l % 8 of row l / 8.  Rows past
  // the last repeat it; their results are not stored.
  const uint16_t* src[PIECES];
  int koff[2];   // of pieces with an even and an odd number
#pragma unroll
  for (int f = 0; f < 2; ++f) koff[f] = 8 * ((lane & 7) ^ token_swizzle(8 * f + (lane >> 3)));
#pragma unroll
  for (int f = 0; f < PIECES; ++f) {
    const int r = 8 * f + (lane >> 3);
    if (f < 2) {
      const bool up = GATED && f == 1;
      const int col = min(n0 + (up ? r - 8 : r), p.N - 1);
      src[f] = p.w + (size_t)(up ? p.N + col : col) * K;
    } else {
      src[f] = p.x + (size_t)min(m0 + r - 16, p.M - 1) * p.x_ld;
    }
    src[f] += koff[f & 1] + wave * kKC;
  }
  unsigned char* const ring = lds + wave * AHEAD * UNIT;
  const int mine = (units - wave + WAVES - 1) / WAVES;         // units wave, wave + WAVES, ...
  const int mine_whole = (whole - wave + WAVES - 1) / WAVES;   // (0 or 1 fewer)
  int put = 0, get = 0;
  auto copy = [&] {   // the next unit, a whole one
    unsigned char* base = ring + put * UNIT;
    put = put == AHEAD - 1 ? 0 : put + 1;
#pragma unroll
    for (int f = 0; f < PIECES; ++f) {
      __builtin_amdgcn_global_load_lds((global_void*)src[f], (lds_void*)(base + f * 1024), 16, 0, 0);
      src[f] += WAVES * kKC;
    }
  };
  auto issue = [&](int i) {   // this wave's unit i
    if (i < mine_whole) {
      copy();
      return;
    }
    unsigned char* base = ring + put * UNIT;
    put = put == AHEAD - 1 ? 0 : put + 1;
#pragma unroll
    for (int f = 0; f < PIECES; ++f)
      *reinterpret_cast<u32x4*>(base + f * 1024 + lane * 16) =
          whole * kKC + koff[f & 1] < K ? ld16(src[f]) : u32x4{0, 0, 0, 0};
  };
  const int row = XP == 1 ? li & 7 : li;
  const int waddr = li * 128 + 16 * (lg ^ token_swizzle(li));
  const int xaddr = 2048 + row * 128 + 16 * (lg ^ token_swizzle(row));
  f32x4 acc[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  u32x4 w[2], x[2][MT];
  auto read = [&] {
    const unsigned char* base = ring + get * UNIT;
    get = get == AHEAD - 1 ? 0 : get + 1;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      w[h] = *reinterpret_cast<const u32x4*>(base + (waddr ^ 64 * h));
#pragma unroll
      for (int t = 0; t < MT; ++t) x[h][t] = *reinterpret_cast<const u32x4*>(base + (xaddr ^ 64 * h) + 2048 * t);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the slot can be filled again
  };
  auto multiply = [&] {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[t] = mfma16x16x32(w[h], x[h][t], acc[t]);
  };
#pragma unroll
  for (int q = 0; q < AHEAD; ++q)
    if (q < mine) issue(q);
  int i = 0;
  for (; i + AHEAD < mine_whole; ++i) {
    wait_vmcnt<(AHEAD - 1) * PIECES>();
    read();
    copy();
    multiply();
  }
  for (; i < mine; ++i) {   // (a partial unit's loads are complete when they are stored)
    wait_after<PIECES, AHEAD - 1>(i < mine_whole ? min(AHEAD, mine_whole - i) - 1 : 0);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    read();
    if (i + AHEAD < mine) issue(i + AHEAD);
    multiply();
  }
  __syncthreads();
  auto part = reinterpret_cast<float(*)[MT][4][kWave]>(lds);
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int q = 0; q < 4; ++q) part[wave][t][q][lane] = acc[t][q];
  __syncthreads();
  // thread -> token r, column c, with the residual in flight beside the sums: weight row c is
  // result c % 4 of lane 16 (c / 4) + r % 16 of token tile r / 16
  for (int i = threadIdx.x; i < COLS * 8 * XP; i += 64 * WAVES) {
    const int r = i / COLS, c = i % COLS;
    if (m0 + r >= p.M || n0 + c >= p.N) continue;
    const int n = n0 + c;
    const float bh = p.bias ? bf16_to_f32(p.bias[n]) : 0.0f;
    const float bu = GATED && p.bias ? bf16_to_f32(p.bias[p.N + n]) : 0.0f;
    const float res =
        p.residual ? load_value(p.residual, p.residual_f32, (size_t)(m0 + r) * p.residual_ld + n) : 0.0f;
    float h[1][1] = {{0.0f}}, u = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      h[0][0] += part[w][r >> 4][c & 3][16 * (c >> 2) + (r & 15)];
      if (GATED) u += part[w][r >> 4][c & 3][16 * ((c + 8) >> 2) + (r & 15)];
    }
    h[0][0] += bh;
    activate(p.act, h);
    if (GATED) h[0][0] *= u + bu;
    if (p.residual) h[0][0] += res;
    store_value(p.out, p.out_f32, (size_t)(m0 + r) * p.out_ld + n, h[0][0]);
  }
}

template <int XP, bool GATED>
hipError_t launch_skinny(const GemmArgs& a, hipStream_t s) {
  const int n_ntiles = (a.N + (GATED ? 7 : 15)) / (GATED ? 8 : 16);
  const int mblocks = (a.M + 8 * XP - 1) / (8 * XP);
  const int64_t per_xcd = ((int64_t)n_ntiles * mblocks + kXcds - 1) / kXcds;
  hipLaunchKernelGGL((skinny_kernel<XP, GATED>), dim3((unsigned)(per_xcd * kXcds)), dim3(512), 0, s, a,
                     n_ntiles, mblocks, (int)per_xcd);
  return hipGetLastError();
}

// Many tokens: 256 tokens x 256 weight rows (GATED: 128 gate and 128 up rows) per workgroup of 4
// waves, a wave 128 x 128 on v_mfma_f32_32x32x16_bf16, whose 256 sums a lane fill the
// accumulation registers: fragment reads then take half of the LDS's rate (8 waves of 64 x 128:
// three quarters, and with the copies' writes all of it).
//
// 8192 x 2 x 2048 x 7168, gated: 379 us (1.27 PFLOP/s; a library product of the same sizes without
// the epilogue 309), MFMAs busy 62 % of the time at 1.9 GHz.  That is from some 100 calls in a row on;
// the first 40 after a pause, while the clock settles, take 390 to 530 (the library's 310 to 520).
// K in chunks of 64, a panel of 256 weight rows and one of 256 token rows each, in a ring of five
// LDS slots of 32 KiB: two of the present chunk, two of the next, one more.  A chunk is 4 steps of
// 16 values; a step's 16 MFMAs run on one of two sets of fragment registers while the next step's
// fragments are read into the other.  Before the last step of chunk c every wave has read all of it
// and its copies of chunk c + 1 have landed: one barrier, which frees two slots, for the tokens of
// chunk c + 2 (copied in that step and the next) and the weights of chunk c + 3 (in the two steps
// after).  So every step copies 16 KiB: with two stages of both and all 64 copies of the waves in
// one step they wait for the address unit (M = N = 4096, K = 7168: 222 us, in two steps 206, without
// copies 167).  The stream of chunks runs on into the workgroup's next item; results go through
// the two slots that an item's last chunk frees.
//
// LDS rows as above.  Fragment row r of the weights is row 16 (r / 4 % 2) + 4 (r / 8) + r % 4 of
// its 32, so that a lane's 16 sums of a fragment are 16 consecutive columns.
#ifdef __HIP_DEVICE_COMPILE__   // the host pass knows no buffer descriptors
// Buffer descriptor of raw bytes from a wave-uniform pointer on, without a bound.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const uint16_t* base) {
  const uint64_t b = (uint64_t)base;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)b);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)(b >> 32));
  return __builtin_amdgcn_make_buffer_rsrc((void*)((uint64_t)hi << 32 | lo), 0, -1, 0x00020000);
}
#endif

constexpr int kBig = 256, kBigSlot = kBig * 128, kBigSlots = 5;
constexpr int kBigMinChunks = 2;
constexpr int64_t kBigMaxLd = 1 << 23;   // 64 rows within 32-bit byte offsets

typedef __attribute__((ext_vector_type(16))) float f32x16;
__device__ __forceinline__ f32x16 mfma32x32x16(u32x4 a, u32x4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(a), as_bf16x8(b), c, 0, 0, 0);
}

// This workgroup's items: each XCD has a contiguous share of them, in which 32 in a row (what an
// XCD's CUs work on at once) are 4 column tiles x 8 token tiles: 12 panels for its L2 to hold,
// where 32 token tiles of one column tile are 33.
struct BlockWalk {
  int mtiles, ntiles, items, per_xcd, first, slot, stride;
  __device__ BlockWalk(int mt, int nt)
      : mtiles(mt), ntiles(nt), items(mt * nt), per_xcd((items + kXcds - 1) / kXcds),
        first((blockIdx.x % kXcds) * per_xcd), slot(blockIdx.x / kXcds), stride(gridDim.x / kXcds) {}
  __device__ bool next(int& mtile, int& ntile) {
    const int item = first + slot;
    if (slot >= per_xcd || item >= items) return false;
    slot += stride;
    const int group = item / (4 * mtiles), in = item % (4 * mtiles);
    const int width = min(4, ntiles - 4 * group);
    mtile = in / width;
    ntile = 4 * group + in % width;
    return true;
  }
};

template <bool GATED, bool RAGGED>
__device__ __forceinline__ void big_products(const GemmArgs& p, unsigned char* lds) {
#ifdef __HIP_DEVICE_COMPILE__
  constexpr int COLS = GATED ? kBig / 2 : kBig;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wn = wave & 1, wm = wave >> 1, r = lane & 31, h = lane >> 5, rr = lane >> 3;
  const int K = p.K, nch = (K + kKC - 1) / kKC, whole = K / kKC;
  // fragment addresses of step 0; step s: ^ 32 s
  const int wperm = 16 * (r >> 2 & 1) + 4 * (r >> 3) + (r & 3);
  const int wswz = (wperm >> 1 & 3) | (wperm >> 4) << 2;
  const int waddr = (GATED ? 64 : 128) * wn * 128 + wperm * 128 + 16 * (h ^ wswz);
  const int taddr = (128 * wm + r) * 128 + 16 * (h ^ (r >> 1 & 7));
  f32x16 acc[4][4];
  u32x4 wa[2][4], tb[2][4];   // fragments of even and odd steps
  auto slot_at = [&](int slot) { return lds + (slot < kBigSlots ? slot : slot - kBigSlots) * kBigSlot; };
  auto read = [&](int slot, int s) {   // the weights' slot; the tokens' is the next
    const unsigned char *wbase = slot_at(slot), *tbase = slot_at(slot + 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      wa[s & 1][i] = *reinterpret_cast<const u32x4*>(
          wbase + (waddr ^ (32 * s)) + (GATED ? (i & 1) * 4096 + (i >> 1) * 16384 : i * 4096));
      tb[s & 1][i] = *reinterpret_cast<const u32x4*>(tbase + (taddr ^ (32 * s)) + i * 4096);
    }
  };
  auto multiply = [&](int s) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = mfma32x32x16(wa[s & 1][i], tb[s & 1][j], acc[i][j]);
  };
  // A wave copies weight rows 64 wave .. and token rows 64 wave .., 8 pieces of 8 rows each; lane l
  // slot l % 8 of row l / 8.  Rows past the last repeat it.
  __amdgpu_buffer_rsrc_t wsrc, tsrc;
  uint32_t woff[8], toff[8];
  auto wpart = [&](int i) { return (lane & 7) ^ ((rr >> 1 & 3) | (i >> 1 & 1) << 2); };
  auto tpart = [&](int i) { return (lane & 7) ^ ((8 * i + rr) >> 1 & 7); };
  auto sources = [&](int m0, int n0) {
    int rr = lane >> 3;   // (computed here, not held through the item's loop)
    asm volatile("" : "+v"(rr));
    const int wfirst = min(n0 + 64 * (GATED ? wave & 1 : wave), p.N - 1);
    const int tfirst = min(m0 + 64 * wave, p.M - 1);
    wsrc = buffer_of(p.w + ((size_t)(GATED && wave >= 2 ? p.N : 0) + wfirst) * K);
    tsrc = buffer_of(p.x + (size_t)tfirst * p.x_ld);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      woff[i] = 2 * (uint32_t)min(8 * i + rr, p.N - 1 - wfirst) * (uint32_t)K + 16 * wpart(i);
      toff[i] = 2 * (uint32_t)min(8 * i + rr, p.M - 1 - tfirst) * (uint32_t)p.x_ld + 16 * tpart(i);
    }
  };
  // pieces 4 half .. of a panel of chunk c; a partial last chunk, zero-filled, through registers
  auto copy = [&](int slot, int c, int half, __amdgpu_buffer_rsrc_t from, const uint32_t (&off)[8],
                  auto part) {
    unsigned char* base = slot_at(slot) + wave * 8192;
#pragma unroll
    for (int i = 4 * half; i < 4 * half + 4; ++i) {
      if (RAGGED && c == whole) {
        u32x4 v = u32x4{0, 0, 0, 0};
        if (c * kKC + 8 * part(i) < K) v = __builtin_amdgcn_raw_buffer_load_b128(from, off[i], c * 128, 0);
        *reinterpret_cast<u32x4*>(base + i * 1024 + lane * 16) = v;
      } else {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (lds_void*)(base + i * 1024), 16, off[i], c * 128, 0, 0);
      }
    }
  };
  auto copy_w = [&](int slot, int c, int half) { copy(slot, c, half, wsrc, woff, wpart); };
  auto copy_t = [&](int slot, int c, int half) { copy(slot, c, half, tsrc, toff, tpart); };

  // Results: fragment by token fragment (64 rows of the tile at a time) through two LDS slots, fp32,
  // 16-byte slots XORed with the row; then 8 columns of a row per thread, whole lines of a row
  // together, the residuals of the next four rows in flight.
  constexpr int G = GATED ? 16 : 32, ROWS = 256 / G, PASSES = 64 / ROWS;   // threads of a row, rows of a pass
  constexpr int R = 4;   // rows of a thread at a time
  auto barrier = [&] { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); };
  auto results = [&](unsigned char* low, unsigned char* high, int m0, int n0) {
    int tid = threadIdx.x;   // (addresses are computed here, not held through the item's loop)
    asm volatile("" : "+v"(tid));
    const int group = tid % G, row0 = tid / G, r = tid & 31, h = tid >> 5 & 1;
    const int n = n0 + 8 * group;
    const bool on = n < p.N;
    float bh[8], bu[8];
    load_bias(p, min(n, p.N - 1), 0, bh);
    if (GATED) load_bias(p, min(n, p.N - 1), p.N, bu);
    auto token = [&](int g, int k) {   // row k of this thread's four in group g of passes
      const int lr = (g * R + k) % PASSES * ROWS + row0;
      return m0 + 128 * (lr >> 5) + 32 * (g * R / PASSES) + (lr & 31);
    };
    Residual<8> res[R];
    auto fetch = [&](int g, int k) {
      if (p.residual && on && token(g, k) < p.M) res[k].load(p, token(g, k), n);
    };
#pragma unroll
    for (int k = 0; k < R; ++k) fetch(0, k);
#pragma unroll
    for (int ph = 0; ph < 4; ++ph) {
      unsigned char* const mine = (wm ? high : low) + r * 1024;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int col = GATED ? 128 * (i >> 1) + 64 * wn + 32 * (i & 1) + 16 * h + 4 * k
                                : 128 * wn + 32 * i + 16 * h + 4 * k;
          *reinterpret_cast<f32x4*>(mine + 16 * ((col >> 2) ^ r)) =
              f32x4{acc[i][ph][4 * k], acc[i][ph][4 * k + 1], acc[i][ph][4 * k + 2], acc[i][ph][4 * k + 3]};
        }
        __builtin_amdgcn_sched_barrier(0);   // (16 sums at a time leave the accumulation registers)
      }
      barrier();
#pragma unroll 1
      for (int g = ph * (PASSES / R); g < (ph + 1) * (PASSES / R); ++g) {
        float v[R][8], u[R][8];
#pragma unroll
        for (int k = 0; k < R; ++k) {
          const int lr = (g * R + k) % PASSES * ROWS + row0;
          const unsigned char* src = (lr & 32 ? high : low) + (lr & 31) * 1024;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const f32x4 a = *reinterpret_cast<const f32x4*>(src + 16 * ((2 * group + half) ^ (lr & 31)));
            f32x4 b = f32x4{0.f, 0.f, 0.f, 0.f};
            if (GATED) b = *reinterpret_cast<const f32x4*>(src + 16 * ((32 + 2 * group + half) ^ (lr & 31)));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              v[k][4 * half + e] = a[e];
              u[k][4 * half + e] = b[e];
            }
          }
        }
        int m[R];
#pragma unroll
        for (int k = 0; k < R; ++k) m[k] = on ? token(g, k) : p.M;
        finish<GATED>(p, m, n, v, u, bh, bu, res, [&] {
          if (g + 1 < 4 * PASSES / R) {
#pragma unroll
            for (int k = 0; k < R; ++k) fetch(g + 1, k);
          }
        });
      }
      barrier();
    }
  };

  BlockWalk walk((p.M + kBig - 1) / kBig, (p.N + COLS - 1) / COLS);
  int mtile, ntile;
  if (!walk.next(mtile, ntile)) return;
  sources(mtile * kBig, ntile * COLS);
  int slot = 0;   // of the present chunk's weights
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    copy_w(0, 0, half);
    copy_t(1, 0, half);
  }
#pragma unroll
  for (int half = 0; half < 2; ++half) copy_w(2, 1, half);   // (nch >= 2)
  wait_vmcnt<8>();
  barrier();
  for (;;) {
    const int m0 = mtile * kBig, n0 = ntile * COLS;
    bool more = false;
    copy_t(slot + 3, 1, 0);
    read(slot, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.0f;
#pragma unroll 1
    for (int c = 0; c < nch; ++c) {
      const int ahead = c + 2 < nch ? c + 2 : c + 2 - nch;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        if (s == 1 && c == nch - 2) {   // the copies that follow are the next item's (repeats without one)
          more = walk.next(mtile, ntile);
          sources(mtile * kBig, ntile * COLS);
        }
        if (s == 3) {   // all but the 8 copies of the weights of chunk c + 2 have landed
          asm volatile("s_waitcnt vmcnt(8) lgkmcnt(0)\n\ts_barrier" ::: "memory");
          if (c + 1 < nch) copy_t(slot, ahead, 0);   // (an item's last chunk leaves its slots to the results)
          read(slot + 2, 0);
        } else {
          if (s == 0) copy_t(slot + 3, c + 1 < nch ? c + 1 : 0, 1);
          else copy_w(slot + 4, ahead, s - 1);
          read(slot, s + 1);
        }
        multiply(s);
        // one fragment read beside each of the first eight MFMAs, a copy beside every second
        if (!RAGGED) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      slot = slot + 2 < kBigSlots ? slot + 2 : slot + 2 - kBigSlots;
    }
    const int last = slot + 3;   // (two back)
    results(slot_at(last), slot_at(last + 1), m0, n0);
    if (!more) break;
  }
  wait_vmcnt<0>();   // copies into LDS that are still in flight end with the workgroup
#endif
}

template <bool GATED, bool RAGGED>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1))) void big_kernel(GemmArgs p) {
  __shared__ __align__(16) unsigned char lds[kBigSlots * kBigSlot];
  big_products<GATED, RAGGED>(p, lds);
}

template <bool GATED>
hipError_t launch_big(const GemmArgs& a, hipStream_t s) {
  const int cols = GATED ? kBig / 2 : kBig;
  const long items = (long)((a.M + kBig - 1) / kBig) * ((a.N + cols - 1) / cols);
  const dim3 grid((unsigned)walk_grid(items, kBigSlots * kBigSlot)), threads(256);
  if (a.K % kKC == 0) hipLaunchKernelGGL((big_kernel<GATED, false>), grid, threads, 0, s, a);
  else hipLaunchKernelGGL((big_kernel<GATED, true>), grid, threads, 0, s, a);
  return hipGetLastError();
}

// The variant of a product: the one that these estimates (us, fitted to bf16 results without an
// epilogue) make the fastest.  A chunk of all the tiles that the 256 CUs hold at once takes
//   64 x 64      0.20 (one tile per CU), 0.42 (two), more by the tile
//   128 x 128    0.39 (half of the CUs), 0.50, 0.68 (past two rounds of tiles)
//   256 x 256    1.25 (few tiles) .. 1.60 (all CUs)
//   32 x 16      0.07 (the few-token variant)
// K in parts fills idle CUs with 64 x 64 tiles, at the price of another launch and of fp32 sums
// that are written and read.  Measured, 32 x 16 / 64 x 64 / the best split of it / 128 x 128 /
// 256 x 256:
//   M     N     K
//   33    1024  2048     4.2    9.2    7.1   15.8     48
//   64    512   7168     9.6   24.2    9.6   43.9    141
//   40    4096  7168    18.5   24.5   15.4   43.5    141
//   160   1024  2048     7.3    9.3    8.8   16.4     49
//   640   2048  2048    35.9   13.8   20.1   17.2     50
//   640   4096  7168     218   64.4   69.8   47.0    142
//   2048  2048  2048     152   37.8   54.6   22.1     51
//   2048  7168  2048     504    116    187   77.7     61
//   8192  4096  7168    3845   1040   1118    567    373
// At 128 sizes (M 40 to 8192, N 64 to 7168, K 768 to 7168, gated and not) the pick was within 10 % of
// the fastest at all but five, the worst 22 %.  Up to 32 tokens the few-token variant takes one block
// of tokens, and no other was faster by more than 5 %.  Sizes decide, and whether 64 rows of x lie within
// the 32-bit byte offsets of the 256 x 256 variant (else 128 x 128, whose sums have another order); a
// call's workspace does not change its result.
enum Variant { kSkinny, kTile64, kTile128, kTile256 };
struct Choice {
  Variant variant;
  int splits;   // kTile64: parts of K
};
constexpr int kMaxSplits = 16;
Choice choose(int M, int N, int K, bool gated, int64_t x_ld) {
  if (M <= 32) return Choice{kSkinny, 1};
  const double rows = gated ? 2.0 * N : N, chunks = (K + kKC - 1) / kKC;
  auto tiles = [&](int m, int w) { return ceil((double)M / m) * ceil(rows / w); };
  Choice best{kTile64, 1};
  double cost = 1e30;
  auto offer = [&](Variant v, int splits, double us) {
    if (us < cost) {
      cost = us;
      best = Choice{v, splits};
    }
  };
  offer(kSkinny, 1, ceil(tiles(32, 16) / 256) * (2.1 + 0.07 * chunks));
  const double t64 = tiles(64, 64), t128 = tiles(128, 128), t256 = tiles(256, 256);
  auto time64 = [&](double items) {   // of a chunk of all of them
    return items <= 256 ? 0.2 : items <= 512 ? 0.42 : 0.00108 * items;
  };
  offer(kTile64, 1, 3.0 + chunks * time64(t64));
  for (int splits = 2; splits <= kMaxSplits && chunks / splits >= 4; splits *= 2)
    offer(kTile64, splits, (gated ? 7.5 : 5.5) + 0.15 * splits + ceil(chunks / splits) * time64(t64 * splits) +
                               8.0 * splits * M * rows / 3.5e6);   // (bytes, at 3.5 TB/s)
  offer(kTile128, 1, 3.0 + ceil(t128 / 256) * (2.0 + chunks * (t128 <= 128 ? 0.39 : t128 <= 512 ? 0.5 : 0.68)));
  if (K > kKC) {   // (the stream needs 2 chunks per item)
    const double full = t256 < 256 ? t256 / 256 : 1.0;
    offer(kTile256, 1, 5.0 + ceil(t256 / 256) * chunks * (1.25 + 0.35 * full * full * full) + 12.0 * full);
  }
  if (best.variant == kTile256 && x_ld > kBigMaxLd) best.variant = kTile128;
  return best;
}
int skinny_tokens(int M) { return M <= 8 ? 8 : M <= 16 ? 16 : 32; }

template <bool GATED>
hipError_t launch_sized(const GemmArgs& a, float* partial, hipStream_t s) {
  const Choice c = choose(a.M, a.N, a.K, GATED, a.x_ld);
  if (c.splits > 1) return launch_split<GATED>(a, c.splits, partial, s);
  if (c.variant == kSkinny) {
    const int tokens = skinny_tokens(a.M);
    return tokens == 8    ? launch_skinny<1, GATED>(a, s)
           : tokens == 16 ? launch_skinny<2, GATED>(a, s)
                          : launch_skinny<4, GATED>(a, s);
  }
  if (c.variant == kTile64) return launch_ring<64, 1, 4, 4, GATED>(a, s);
  if (c.variant == kTile256) return launch_big<GATED>(a, s);
  return launch_ring<128, 2, 4, 5, GATED>(a, s);
}

}  // namespace

size_t bf16_matmul_scratch_bytes(int M, int N, int K, bool gated) {
  const int splits = choose(M, N, K, gated, K).splits;   // (the same for every stride)
  return splits > 1 ? (size_t)splits * M * partial_ld(N, gated) * sizeof(float) : 0;
}

int bf16_matmul_tile_rows(int M, int N, int K, bool gated, int64_t x_ld) {
  const Variant v = choose(M, N, K, gated, x_ld).variant;
  return v == kSkinny ? skinny_tokens(M) : v == kTile64 ? 64 : v == kTile128 ? 128 : 256;
}

hipError_t launch_bf16_matmul(const GemmArgs& a, void* scratch, hipStream_t s) {
  float* partial = static_cast<float*>(scratch);
  return a.gated ? launch_sized<true>(a, partial, s) : launch_sized<false>(a, partial, s);
}

}  // namespace moe
