// int8 matrix products on MFMA (v_mfma_i32_16x16x64_i8): sums in int32, exact for
// K <= 131,072 (mend_wrapped), scaled once at the end in fp32 by the scale of the token
// row and the scale of the weight row (output channel).
//
// Workgroup tile: BM token rows x 64 WN weight rows, K in chunks of 128 values (one
// 128-byte line per row).  Both operands are copied global -> LDS in 1 KiB pieces of 8 rows
// x one line, whose 16-byte parts are XOR-swizzled so that an MFMA fragment (16 rows x 64 K
// values, 16 per lane) is one conflict-free ds_read_b128.  A ring of S stages
// keeps S - 1 chunks in flight; each wave waits for its own copies and a bare barrier
// publishes them.  Only a partial last chunk goes through registers (zero-filled).
//
// UP: tokens gathered through the plan, gate and up rows of 32 WN act columns, SwiGLU, act
// in fp32 (below).  DOWN: act rows of the plan, results in fp32 to their picks' rows of y.
// DENSE: plain rows.
#include <math.h>

#include <type_traits>

#include "device_common.h"
#include "launchers.h"
#include "tiled_common.h"

namespace moe {

namespace {

typedef __attribute__((ext_vector_type(4))) int i32x4;

__device__ __forceinline__ i32x4 mfma_i8(u32x4 a, u32x4 b, i32x4 c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a),
                                               __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

// Sums of K <= 131,072 products of any two int8 codes in int32.  They reach from -128 * 127 K
// > -2^31 to 128^2 K <= 2^31: only that last one, at K = kWrapK, wraps, to a value that no other
// sum has.  (A test of K, not one of every sum: 253 against 256 us at 8192 x 4096 x 7168.)
constexpr int kWrapK = 131072;
template <int N>
__device__ __forceinline__ void mend_wrapped(int K, const i32x4 (&sum)[N], float (&v)[4 * N]) {
  if (K != kWrapK) return;
#pragma unroll
  for (int q = 0; q < 4 * N; ++q)
    if (sum[q >> 2][q & 3] == INT32_MIN) v[q] = 0x1p31f;
}

constexpr int kKC = 128;   // K values per chunk
constexpr int kStreamPolicy = 2;   // nontemporal
enum Mode { kUp, kDown, kDense };

struct I8Args {
  const int8_t* tok;
  const float* tok_scale;
  const int8_t* w;
  const float* w_scale;
  const int32_t* sorted_ids;
  const int32_t* block_expert;
  const int2* tiles;
  const int32_t* num_tiles;
  int act_rows;   // rows of a 128-column block of act
  int n_ntiles, M, K, ncols, top_k, block;   // ncols: act columns (UP), output columns
  float* act;
  float* y;
  void* out;
};

// LDS rows are one 128-byte line of a chunk each; 16-byte slot q of row r holds the part
// q ^ f(r) of the line, with f chosen so that the 16 rows of a fragment read (which also
// differ in r % 2) meet no bank twice.  Token fragments are 16 consecutive rows.  Weight
// fragment j of a wave's 32 (UP: gate, and as many up) or 64 rows holds rows
// SPAN (i / 4) + 4 j + i % 4, i = 0 .. 15, SPAN = 8 or 16: a lane's results of all the
// fragments then are SPAN consecutive columns, stored 16 bytes at a time.
__device__ __forceinline__ int token_swizzle(int r) { return (r >> 1) & 7; }
template <int SPAN>
__device__ __forceinline__ int weight_swizzle(int r) {
  return ((r >> 1) & 1) | ((r / SPAN) & 3) << 1;
}

__device__ __forceinline__ void load16(const float* src, float (&w)[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 g = reinterpret_cast<const float4*>(src)[j];
    w[4 * j] = g.x;
    w[4 * j + 1] = g.y;
    w[4 * j + 2] = g.z;
    w[4 * j + 3] = g.w;
  }
}
__device__ __forceinline__ void store16(float* dst, const float (&v)[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    reinterpret_cast<float4*>(dst)[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
}
__device__ __forceinline__ void store16(uint16_t* dst, const float (&v)[16]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    u32x4 u;
#pragma unroll
    for (int q = 0; q < 4; ++q) u[q] = pack_bf16x2(v[8 * j + 2 * q], v[8 * j + 2 * q + 1]);
    st16(dst + 8 * j, u);
  }
}

// __expf is exp2 of a rounded product: within about (1.5 |z| + 2) 2^-24 of itself; the reciprocal
// within 2^-23.
__device__ __forceinline__ float silu_fast(float z) {
  return z * __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}

// act of this lane's 8 columns from c on: silu(gate) * up of the scaled sums, 0 past the last
// column.  ws: the gate rows' scales, the up rows' p.ncols behind them.
__device__ __forceinline__ void scaled_act(i32x4 g0, i32x4 g1, i32x4 u0, i32x4 u1, float xs,
                                           const float* ws, int c, int ncols, float (&a)[8]) {
  const bool in = c < ncols;
  const float4* g4 = reinterpret_cast<const float4*>(ws + (in ? c : 0));
  const float4* u4 = reinterpret_cast<const float4*>(ws + ncols + (in ? c : 0));
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float4 gw = g4[h], uw = u4[h];
    const float gs[4] = {gw.x, gw.y, gw.z, gw.w}, us[4] = {uw.x, uw.y, uw.z, uw.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float v = silu_fast((float)(h ? g1 : g0)[q] * (xs * gs[q])) *
                      ((float)(h ? u1 : u0)[q] * (xs * us[q]));
      a[4 * h + q] = in ? v : 0.0f;
    }
  }
}

// act leaves the up product in fp32: the codes that it is quantized to next are roundings of
// its quotients, and a shorter act would move them (bf16 one in ten by one, 16 bits under an
// exponent of 32 columns one in 2,000: layer outputs 0.6 % and 0.12 % off in relative L2).
// a: act of this lane's 8 columns from c on.
// Layout [ceil(I / 128)][rows][128]: what a workgroup writes is one piece of memory.
__device__ __forceinline__ void store_act(const I8Args& p, int row, int c, const float (&a)[8]) {
  float* dst = p.act + ((size_t)(c >> 7) * p.act_rows + row) * 128 + (c & 127);
  if (c < p.ncols) {   // nontemporal: kept out of the way of the weights' stream
#pragma unroll
    for (int h = 0; h < 2; ++h)
      __builtin_nontemporal_store(f32x4{a[4 * h], a[4 * h + 1], a[4 * h + 2], a[4 * h + 3]},
                                  reinterpret_cast<f32x4*>(dst) + h);
  }
}

// 16 results of pick i, columns n0 on.  y is fp32 at every size: bf16 picks (the other weight
// formats' y) put the outputs of the M=2048, k=16 layer 0.20 % off in relative L2, fp32 ones
// 0.166 %, which is their own rounding, for 165 us more of 2,880.
__device__ __forceinline__ void store_y(const I8Args& p, int i, int n0, const float (&v)[16]) {
  store16(p.y + (size_t)i * p.ncols + n0, v);
}

// 16 results of a dense row that starts at `row` (in values), columns n0 on
template <bool F32>
__device__ __forceinline__ void store_dense(const I8Args& p, size_t row, int n0,
                                            const float (&v)[16]) {
  if (n0 + 15 < p.ncols && p.ncols % 8 == 0) {
    if (F32) store16(static_cast<float*>(p.out) + row + n0, v);
    else store16(static_cast<uint16_t*>(p.out) + row + n0, v);
    return;
  }
#pragma unroll
  for (int q = 0; q < 16; ++q)
    if (n0 + q < p.ncols) {
      if (F32) static_cast<float*>(p.out)[row + n0 + q] = v[q];
      else static_cast<uint16_t*>(p.out)[row + n0 + q] = (uint16_t)f32_to_bf16_rne(v[q]);
    }
}

template <int BM, int WN, int WM>
struct I8Cfg {
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

template <int BM, int WN, int WM, int S, Mode MODE, bool F32, int WPOL>
__global__ __launch_bounds__(64 * WN * WM) void i8_gemm_kernel(I8Args p) {
  using C = I8Cfg<BM, WN, WM>;
  constexpr bool UP = MODE == kUp;
  static_assert((S - 2) * C::PPW <= 63, "the copies in flight must fit the vmcnt counter");
  static_assert(S * C::PIECES * 1024 <= 160 * 1024, "the ring must fit the LDS");
  __shared__ __align__(16) unsigned char lds[S * C::PIECES * 1024];
  constexpr int SPAN = UP ? 8 : 16;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int li = lane & 15, lg = lane >> 4;
  const int wn = wave % WN, wm = wave / WN;
  const int K = p.K;

  TiledWalk walk(MODE == kDense ? (p.M + BM - 1) / BM : *p.num_tiles, p.n_ntiles);
  int ntile, ti;
  while (walk.next(ntile, ti)) {
    int start, nlive, e = 0;
    if (MODE == kDense) {
      start = ti * BM;
      nlive = min(BM, p.M - start);
    } else {
      const int2 tile = p.tiles[ti];
      start = tile.x;
      nlive = tile.y;
      e = p.block_expert[start / p.block];
    }
    const int mt_active = (nlive + 15) >> 4;
    const int col0 = UP ? ntile * 32 * WN : ntile * 64 * WN;
    const size_t wrow0 = MODE == kDense ? 0 : (size_t)e * (UP ? 2 * p.ncols : p.ncols);

    // piece f of a chunk: LDS rows 8f .. 8f + 7 (weight rows first); lane l copies slot l % 8
    // of row 8f + l / 8.  Rows without data point at a valid row; their results are never
    // stored.
    const int8_t* src[C::PPW];
    bool on[C::PPW];
    int q16[C::PPW];
#pragma unroll
    for (int i = 0; i < C::PPW; ++i) {
      const int f = wave * C::PPW + i;
      const int lr = 8 * f + (lane >> 3);
      if (lr < 64 * WN) {
        q16[i] = 16 * ((lane & 7) ^ weight_swizzle<SPAN>(lr));
        const bool up = UP && lr >= 32 * WN;
        const int col = col0 + (up ? lr - 32 * WN : lr);
        const int row = up ? p.ncols + col : col;
        on[i] = col < p.ncols;
        src[i] = p.w + (wrow0 + (on[i] ? row : 0)) * K + q16[i];
      } else {
        const int r = lr - 64 * WN;
        q16[i] = 16 * ((lane & 7) ^ token_swizzle(r));
        on[i] = r < nlive;
        int row = start + (on[i] ? r : 0);
        if (UP) row = p.sorted_ids[row] / p.top_k;
        src[i] = p.tok + (size_t)row * K + q16[i];
      }
    }
    const int nch = (K + kKC - 1) / kKC;
    const int ndma = K / kKC;   // whole chunks
    auto issue = [&](int c) {
      unsigned char* base = lds + (size_t)(c % S) * C::PIECES * 1024;
      if (c < ndma) {
#pragma unroll
        for (int i = 0; i < C::PPW; ++i) {
          const int f = wave * C::PPW + i;
          if (f < 2 * C::WT)
            __builtin_amdgcn_global_load_lds((global_void*)(src[i] + (size_t)c * kKC),
                                             (lds_void*)(base + f * 1024), 16, 0, WPOL);
          else
            __builtin_amdgcn_global_load_lds((global_void*)(src[i] + (size_t)c * kKC),
                                             (lds_void*)(base + f * 1024), 16, 0, 0);
        }
      } else {
#pragma unroll
        for (int i = 0; i < C::PPW; ++i) {
          const int f = wave * C::PPW + i;
          const u32x4 v = (on[i] && c * kKC + q16[i] < K) ? ld16(src[i] + (size_t)c * kKC)
                                                          : u32x4{0, 0, 0, 0};
          *reinterpret_cast<u32x4*>(base + (size_t)f * 1024 + lane * 16) = v;
        }
      }
    };
    const int wrow = (UP ? 32 : 64) * wn + SPAN * (li >> 2) + (li & 3);
    const int wslot = weight_swizzle<SPAN>(wrow), tslot = token_swizzle(li);
    auto frag = [&](int c, int row, int slot) -> u32x4 {
      return *reinterpret_cast<const u32x4*>(lds + (size_t)(c % S) * C::PIECES * 1024 + row * 128 +
                                             slot * 16);
    };
    auto wfrag = [&](int c, int j, int ks) {
      const int row = UP ? wrow + 4 * (j & 1) + (j >> 1) * 32 * WN : wrow + 4 * j;
      return frag(c, row, (lg + 4 * ks) ^ wslot);
    };

    i32x4 acc[4][C::MTW];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int s = 0; s < C::MTW; ++s) acc[j][s] = i32x4{0, 0, 0, 0};
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
          for (int j = 0; j < 4; ++j) wa[j] = wfrag(c, j, ks);
#pragma unroll
          for (int s = 0; s < C::MTW; ++s) {
            if (s < my_active) {
              const u32x4 xb = frag(c, 64 * WN + 16 * (wm * C::MTW + s) + li, (lg + 4 * ks) ^ tslot);
#pragma unroll
              for (int j = 0; j < 4; ++j) acc[j][s] = mfma_i8(wa[j], xb, acc[j][s]);
            }
          }
        }
      }
    }

    // lane (li, lg) holds token row li of each token tile and SPAN columns from n0 on
    const float* ws = p.w_scale + wrow0;
    const int n0 = col0 + (UP ? 32 : 64) * wn + SPAN * lg;
#pragma unroll
    for (int s = 0; s < C::MTW; ++s) {
      const int r = 16 * (wm * C::MTW + s) + li;
      if (s >= my_active || r >= nlive) continue;
      const int row = start + r;
      if (UP) {
        float a[8];
        const float xs = p.tok_scale[p.sorted_ids[row] / p.top_k];
        scaled_act(acc[0][s], acc[1][s], acc[2][s], acc[3][s], xs, ws, n0, p.ncols, a);
        store_act(p, row, n0, a);
      } else if (n0 < p.ncols) {
        const float xs = p.tok_scale[row];
        const i32x4 v4[4] = {acc[0][s], acc[1][s], acc[2][s], acc[3][s]};
        float v[16], w[16];
        if (MODE == kDown || n0 + 15 < p.ncols) {
          load16(ws + n0, w);
        } else {
#pragma unroll
          for (int q = 0; q < 16; ++q) w[q] = ws[min(n0 + q, p.ncols - 1)];
        }
#pragma unroll
        for (int q = 0; q < 16; ++q) v[q] = (float)v4[q >> 2][q & 3];
        if (MODE == kDense) mend_wrapped(K, v4, v);
#pragma unroll
        for (int q = 0; q < 16; ++q) v[q] *= xs * w[q];
        if (MODE == kDense) {
          store_dense<F32>(p, (size_t)row * p.ncols, n0, v);
        } else {
          store_y(p, p.sorted_ids[row], n0, v);
        }
      }
    }
    __syncthreads();   // the next item's first copies reuse the ring
  }
}

template <int BM, int WN, int WM, int S, Mode MODE, bool F32, int WPOL>
hipError_t launch(I8Args& a, long token_tiles, hipStream_t s) {
  const int per = MODE == kUp ? 32 * WN : 64 * WN;
  a.n_ntiles = (a.ncols + per - 1) / per;
  const long grid =
      walk_grid(token_tiles * a.n_ntiles, S * I8Cfg<BM, WN, WM>::PIECES * 1024);
  hipLaunchKernelGGL((i8_gemm_kernel<BM, WN, WM, S, MODE, F32, WPOL>), dim3((unsigned)grid),
                     dim3(64 * WN * WM), 0, s, a);
  return hipGetLastError();
}

// Grouped products, and dense ones of many rows, of more than 4 chunks.
//
// 256 weight rows (UP: 128 act columns) per workgroup of 8 waves, 4 along the weight rows and
// 2 along the tokens, against up to ROWS token rows of an expert at once, so that its weights
// are read once.  The workgroup walks its items as one stream of steps (a chunk of an item
// each, rounded up to a multiple of D; the added steps compute nothing): in step c it
//   copies the tokens of step c + D into a ring of D + 1 LDS stages,
//   moves the weights of step c + 1 from registers into one of two LDS stages and
//   loads those of step c + 1 + D into the registers they leave,
//   multiplies chunk c.
// The copies of the next item's first D + 1 steps start in the last steps of the present
// one.  Weights and tokens return in order, so both run D steps ahead; the registers hold
// the weights in flight because the LDS cannot hold both rings (two LDS rings: tokens one
// step ahead, whose L2 latency then set the pace).  Without the stream each item paid about
// 12 us of latencies: item data, first chunks, scales (M=2048, H=7168, I=2048, E=256, 29
// items a workgroup in the down product).
// Measured: dense 8192 x 4096 x 7168 215 to 220 us (2.2 POP/s, MFMAs busy half the cycles: a
// step's fragment reads and its barrier stand beside them), 224 with a partial last chunk (K =
// 7152); the layer at M=8 450 + 232 us (6.7 TB/s of weights), at M=2048 1,640 + 1,020 us (7.5 and
// 3.8 GB of weights, 8.2 and 4.1 read in all, with the tokens' lines from the L2 and 0.29 GB of act
// or 0.94 GB of results written at the same time; MFMAs busy 28 and 24 %).
// The 256-row up kernels spill 3 registers a lane, and 17 with a partial last chunk: reloads that
// wait for all copies in flight, once an item.
template <int ROWS_, int D_>
struct Ring {
  static constexpr int ROWS = ROWS_, D = D_;
  static constexpr int MTW = ROWS / 32;           // token row tiles per wave
  static constexpr int TPW = ROWS / 64;           // token pieces (8 rows) per wave per chunk
  static constexpr int PW = 4;                    // weight pieces per wave per chunk
  static constexpr int WSTAGE = 256 * 128, TSTAGE = ROWS * 128;
  static constexpr int LDS = 2 * WSTAGE + (D + 1) * TSTAGE;
  static_assert(D % 2 == 0, "a step's weight stage is its parity");
  static_assert(LDS <= 160 * 1024, "the rings must fit the LDS");
  static_assert(PW + (D - 1) * (TPW + PW) <= 63, "the copies in flight must fit the vmcnt counter");
};

#ifdef __HIP_DEVICE_COMPILE__   // the host pass knows no buffer descriptors
// Buffer descriptor of raw bytes from a wave-uniform pointer on, without a bound.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const int8_t* base) {
  const uint64_t b = (uint64_t)base;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)b);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)(b >> 32));
  return __builtin_amdgcn_make_buffer_rsrc((void*)((uint64_t)hi << 32 | lo), 0, -1, 0x00020000);
}

// Vector memory operations stay on their side of it; the mask lets everything else (ALU, MFMA,
// LDS reads and writes) pass.
__device__ __forceinline__ void keep_memory_order() { __builtin_amdgcn_sched_barrier(0x78f); }

struct GroupedItem {
  int start, nlive, e, col0;
};

template <Mode MODE, typename R, int WPOL, bool F32, bool RAGGED>
__device__ __forceinline__ void grouped_products(const I8Args& p, unsigned char* lds) {
  constexpr bool UP = MODE == kUp;
  constexpr int D = R::D, PW = R::PW, TPW = R::TPW, MTW = R::MTW;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int li = lane & 15, lg = lane >> 4;
  const int wn = wave & 3, wm = wave >> 2;
  const int K = p.K;
  unsigned char* const tlds = lds + 2 * R::WSTAGE;

  TiledWalk walk(MODE == kDense ? (p.M + R::ROWS - 1) / R::ROWS : *p.num_tiles, p.n_ntiles);
  auto next_item = [&](GroupedItem& it) -> bool {
    int ntile, ti;
    if (!walk.next(ntile, ti)) return false;
    const int l = ntile * walk.ntiles_live + ti;   // expert by expert: its N tiles share its
    ti = l / p.n_ntiles;                           // token rows through the XCD's L2
    if (MODE == kDense) {
      it.start = ti * R::ROWS;
      it.nlive = min(R::ROWS, p.M - it.start);
      it.e = 0;
    } else {
      const int2 tile = p.tiles[ti];
      it.start = tile.x;
      it.nlive = tile.y;
      it.e = p.block_expert[tile.x / p.block];
    }
    it.col0 = (l % p.n_ntiles) * (UP ? 128 : 256);
    return true;
  };

  // A piece is 8 LDS rows (UP: 128 gate rows, then 128 up rows); lane l copies slot l % 8 of
  // row l / 8.  Weight rows past the last column repeat it; they and token rows past nlive
  // are never stored.  Buffer loads: scalar base and step offset, a 32-bit offset
  // a lane.  (Beside copies of the global_load_lds form the compiler waits for everything in
  // flight.)
  const int rr = lane >> 3;
  constexpr int SPAN = UP ? 8 : 16;
  auto wpart = [&](int i) { return 16 * ((lane & 7) ^ weight_swizzle<SPAN>(32 * wave + 8 * i + rr)); };
  auto tpart = [&](int i) { return 16 * ((lane & 7) ^ token_swizzle((wave * TPW + i) * 8 + rr)); };
  struct Src {
    __amdgpu_buffer_rsrc_t w, t;
    uint32_t woff[PW], toff[TPW];
  };
  auto sources = [&](const GroupedItem& it, Src& q) {
    const int wcol = it.col0 + (UP ? 32 * wn : 32 * wave);   // the wave's first weight row
    const size_t row0 = (size_t)it.e * (UP ? 2 * p.ncols : p.ncols) + (UP && wm ? p.ncols : 0) +
                        min(wcol, p.ncols - 1);
    q.w = buffer_of(p.w + row0 * K);
    q.t = buffer_of(UP ? p.tok : p.tok + (size_t)it.start * K);
#pragma unroll
    for (int i = 0; i < PW; ++i)
      q.woff[i] = (uint32_t)max(0, min(8 * i + rr, p.ncols - 1 - wcol)) * (uint32_t)K + wpart(i);
#pragma unroll
    for (int i = 0; i < TPW; ++i) {
      const int lr = (wave * TPW + i) * 8 + rr;
      const int r = min(lr, it.nlive - 1);
      const uint32_t row = UP ? (uint32_t)p.sorted_ids[it.start + r] / (uint32_t)p.top_k : r;
      q.toff[i] = row * (uint32_t)K + tpart(i);
    }
  };

  const int nch = (K + kKC - 1) / kKC;
  const int steps = (nch + D - 1) / D * D;
  // RAGGED, a partial last chunk (a variant of its own: 256-row tiles have no registers to spare
  // for it): parts behind column K repeat the chunk's first part, and those of the weights
  // become zeros on their way to LDS.
  const int rest = K - (nch - 1) * kKC;
  auto partial = [&](int c) { return RAGGED && c >= nch - 1; };
  auto behind = [&](int part) { return part >= rest ? part : 0; };
  u32x4 wreg[D][PW];
  int tput = 0;   // token stage that the next copy fills
  int tget = 0;   // token stage of the present step
  auto load_w = [&](const Src& q, int c, u32x4 (&dst)[PW]) {
    const int off = min(c, nch - 1) * kKC;
    uint32_t o[PW];
#pragma unroll
    for (int i = 0; i < PW; ++i) o[i] = q.woff[i];
    if (partial(c)) {
#pragma unroll
      for (int i = 0; i < PW; ++i) o[i] -= behind(wpart(i));
    }
#pragma unroll
    for (int i = 0; i < PW; ++i)
      dst[i] = __builtin_amdgcn_raw_buffer_load_b128(q.w, o[i], off, WPOL);
    keep_memory_order();
  };
  auto put_w = [&](int stage, int c, const u32x4 (&v)[PW]) {   // v: chunk c
    unsigned char* base = lds + stage * R::WSTAGE + wave * PW * 1024 + lane * 16;
    if (partial(c)) {
#pragma unroll
      for (int i = 0; i < PW; ++i)
        *reinterpret_cast<u32x4*>(base + i * 1024) = wpart(i) >= rest ? u32x4{0, 0, 0, 0} : v[i];
      return;
    }
#pragma unroll
    for (int i = 0; i < PW; ++i) *reinterpret_cast<u32x4*>(base + i * 1024) = v[i];
  };
  auto copy_t = [&](const Src& q, int c) {
    const int off = min(c, nch - 1) * kKC;
    unsigned char* base = tlds + tput * R::TSTAGE + wave * TPW * 1024;
    tput = tput == D ? 0 : tput + 1;
    uint32_t o[TPW];
#pragma unroll
    for (int i = 0; i < TPW; ++i) o[i] = q.toff[i];
    if (partial(c)) {
#pragma unroll
      for (int i = 0; i < TPW; ++i) o[i] -= behind(tpart(i));
    }
#pragma unroll
    for (int i = 0; i < TPW; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(q.t, (lds_void*)(base + i * 1024), 16, o[i], off, 0, 0);
    keep_memory_order();
  };
  const int wrow = (UP ? 32 : 64) * wn + SPAN * (li >> 2) + (li & 3);
  const int woff16 = wrow * 128 + 16 * (lg ^ weight_swizzle<SPAN>(wrow));
  const int toff16 = (16 * wm + li) * 128 + 16 * (lg ^ token_swizzle(li));
  auto at = [&](const unsigned char* q) { return *reinterpret_cast<const u32x4*>(q); };
  // fragments of K half ks: slot lg + 4 ks, that is byte 64 ks flipped
  auto wfrag = [&](const unsigned char* stage, int j, int ks) {
    return at(stage + (woff16 ^ (64 * ks)) + (UP ? 512 * (j & 1) + 16384 * (j >> 1) : 512 * j));
  };
  auto tfrag = [&](const unsigned char* stage, int s, int ks) {
    return at(stage + (toff16 ^ (64 * ks)) + 4096 * s);
  };

  i32x4 acc[4][MTW];
  auto clear = [&] {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int s = 0; s < MTW; ++s) acc[j][s] = i32x4{0, 0, 0, 0};
  };
  // Products of a step, token tile by token tile (both K halves of one: 8 MFMAs) up to the
  // item's last, each tile's fragments read while the tile before is multiplied; `between`
  // runs after the first tile, whose products cover its waits.
  auto compute = [&](const GroupedItem& it, int c, auto between) {
    const unsigned char* wb = lds + (c & 1) * R::WSTAGE;
    const unsigned char* tb = tlds + tget * R::TSTAGE;
    tget = tget == D ? 0 : tget + 1;
    const int active = c < nch ? (((it.nlive + 15) >> 4) - wm + 1) >> 1 : 0;
    u32x4 wa[2][4], xb[2][2];
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
      for (int j = 0; j < 4; ++j) wa[ks][j] = wfrag(wb, j, ks);
      xb[0][ks] = tfrag(tb, 0, ks);
    }
#pragma unroll
    for (int s = 0; s < MTW; ++s) {
      if (s + 1 < MTW) {
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) xb[(s + 1) & 1][ks] = tfrag(tb, s + 1, ks);
      }
      __builtin_amdgcn_sched_barrier(0);   // keeps the reads ahead
      if (s < active) {
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[j][s] = mfma_i8(wa[ks][j], xb[s & 1][ks], acc[j][s]);
      }
      if (s == 0) between();
      else if (s + 1 < MTW && s >= active) break;
    }
  };
  // The next step's tokens have to be in LDS: all but what was issued after them, which is the
  // weights of their own step and the tokens and weights of the D - 1 steps that follow it.  A
  // load issued before its step's copies would make this count too large, so keep_memory_order
  // holds the order of the source.
  auto publish = [&] {
    wait_vmcnt<PW + (D - 1) * (TPW + PW)>();
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  };
  auto store = [&](const GroupedItem& it) {
    const float* ws = p.w_scale + (size_t)it.e * (UP ? 2 * p.ncols : p.ncols);
    const int n0 = it.col0 + (UP ? 32 : 64) * wn + SPAN * lg;
    int id[MTW];   // every load of a kind before its first use: one latency, not one per row
    float xs[MTW];
#pragma unroll
    for (int s = 0; s < MTW; ++s) {
      const int row = it.start + min(16 * (2 * s + wm) + li, it.nlive - 1);
      id[s] = MODE == kDense ? 0 : p.sorted_ids[row];
      if (!UP) xs[s] = p.tok_scale[row];
    }
    if (UP) {
#pragma unroll
      for (int s = 0; s < MTW; ++s) xs[s] = p.tok_scale[id[s] / p.top_k];
#pragma unroll
      for (int s = 0; s < MTW; ++s) {
        const int r = 16 * (2 * s + wm) + li;
        if (r >= it.nlive) continue;
        float a[8];
        scaled_act(acc[0][s], acc[1][s], acc[2][s], acc[3][s], xs[s], ws, n0, p.ncols, a);
        store_act(p, it.start + r, n0, a);
      }
    } else if (n0 < p.ncols) {
      float w[16];
      if (MODE == kDown || n0 + 15 < p.ncols) {
        load16(ws + n0, w);
      } else {
#pragma unroll
        for (int q = 0; q < 16; ++q) w[q] = ws[min(n0 + q, p.ncols - 1)];
      }
#pragma unroll
      for (int s = 0; s < MTW; ++s) {
        const int r = 16 * (2 * s + wm) + li;
        if (r >= it.nlive) continue;
        const i32x4 v4[4] = {acc[0][s], acc[1][s], acc[2][s], acc[3][s]};
        float v[16];
#pragma unroll
        for (int q = 0; q < 16; ++q) v[q] = (float)v4[q >> 2][q & 3];
        if (MODE == kDense) mend_wrapped(K, v4, v);
#pragma unroll
        for (int q = 0; q < 16; ++q) v[q] *= xs[s] * w[q];
        if (MODE == kDense) {
          store_dense<F32>(p, (size_t)(it.start + r) * p.ncols, n0, v);
          continue;
        }
        store_y(p, id[s], n0, v);
      }
    }
  };

  GroupedItem cur, nxt;
  if (!next_item(cur)) return;
  Src qc, qn;
  sources(cur, qc);
  {
    u32x4 first[PW];
    load_w(qc, 0, first);
#pragma unroll
    for (int d = 0; d < D; ++d) {
      copy_t(qc, d);
      load_w(qc, 1 + d, wreg[d]);
    }
    put_w(0, 0, first);
  }
  clear();
  publish();   // (the first stage of weights too: older than the tokens)
  for (;;) {
    nxt = cur;
    const bool more = next_item(nxt);   // without another item the last copies are repeats
    sources(nxt, qn);
    int c = 0;
    for (; c + 2 * D < steps; c += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        compute(cur, c + d, [&] {
          copy_t(qc, c + d + D);
          put_w((d + 1) & 1, c + d + 1, wreg[d]);
          load_w(qc, c + d + 1 + D, wreg[d]);
        });
        publish();
      }
    }
    // the last 2 D steps reach into the next item
#pragma unroll
    for (int d = 0; d < D; ++d) {
      compute(cur, c + d, [&] {
        copy_t(qc, c + d + D);
        put_w((d + 1) & 1, c + d + 1, wreg[d]);
        if (d + 1 < D) load_w(qc, c + d + 1 + D, wreg[d]);
        else load_w(qn, 0, wreg[d]);
      });
      publish();
    }
    c += D;
#pragma unroll
    for (int d = 0; d < D; ++d) {
      compute(cur, c + d, [&] {
        copy_t(qn, d);
        put_w((d + 1) & 1, d + 1 < D ? c + d + 1 : 0, wreg[d]);
        load_w(qn, d + 1, wreg[d]);
      });
      publish();
    }
    store(cur);
    if (!more) break;
    clear();
    cur = nxt;
    qc = qn;
  }
  wait_vmcnt<0>();   // copies into LDS that are still in flight end with the workgroup
}
#endif

constexpr int kGroupedLds = 160 * 1024;

template <Mode MODE, typename R, int WPOL, bool F32, bool RAGGED>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void i8_grouped_kernel(
    I8Args p) {
  __shared__ __align__(16) unsigned char lds[R::LDS];
#ifdef __HIP_DEVICE_COMPILE__
  grouped_products<MODE, R, WPOL, F32, RAGGED>(p, lds);
#endif
}

using RingFew = Ring<64, 4>;
using RingMid = Ring<128, 4>;
using RingMany = Ring<256, 2>;

template <Mode MODE, typename R, int WPOL, bool F32 = false>
hipError_t launch_grouped(I8Args& a, long token_tiles, hipStream_t s) {
  const int per = MODE == kUp ? 128 : 256;
  a.n_ntiles = (a.ncols + per - 1) / per;
  // one workgroup per CU, whatever its LDS would allow: 512 threads of up to 256 registers
  const long grid = walk_grid(token_tiles * a.n_ntiles, kGroupedLds);
  if (a.K % kKC == 0)
    hipLaunchKernelGGL((i8_grouped_kernel<MODE, R, WPOL, F32, false>), dim3((unsigned)grid), dim3(512),
                       0, s, a);
  else
    hipLaunchKernelGGL((i8_grouped_kernel<MODE, R, WPOL, F32, true>), dim3((unsigned)grid), dim3(512),
                       0, s, a);
  return hipGetLastError();
}

// Dense products of few rows: 16 weight rows x 16 MT token rows per workgroup, the 128-wide
// units of K dealt over its 8 waves, whose int32 sums meet in LDS.  Fragments come straight
// from memory (a weight row's line is read by one wave), BATCH units at a time in flight.
// Bound by the latency of one pass over the weights: 16 rows per workgroup, so that N = 4096
// fills the 256 CUs (8 x 4096 x 7168 8.6 us, 29 MB; 77 x 1537 x 2064 6.7 us).
template <int MT, bool F32>
__global__ __launch_bounds__(512) void i8_skinny_kernel(I8Args p, int mblocks, int per_xcd) {
  constexpr int WAVES = 8, BATCH = MT == 1 ? 4 : MT == 2 ? 2 : 1;
  __shared__ int part[WAVES][MT][4][kWave];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int li = lane & 15, lg = lane >> 4;
  // the token blocks of a weight tile run on one XCD
  const int slot = blockIdx.x / kXcds, item = (blockIdx.x % kXcds) * per_xcd + slot;
  if (slot >= per_xcd || item >= p.n_ntiles * mblocks) return;
  const int n0 = item / mblocks * 16, m0 = item % mblocks * (16 * MT);
  const int K = p.K, units = (K + kKC - 1) / kKC, whole = K / kKC;
  const int8_t* wrow = p.w + (size_t)min(n0 + li, p.ncols - 1) * K + 16 * lg;
  const int8_t* trow[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) trow[t] = p.tok + (size_t)min(m0 + 16 * t + li, p.M - 1) * K + 16 * lg;
  i32x4 acc[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) acc[t] = i32x4{0, 0, 0, 0};
  for (int u0 = wave; u0 < units; u0 += WAVES * BATCH) {
    u32x4 w[BATCH][2], x[BATCH][MT][2];
#pragma unroll
    for (int b = 0; b < BATCH; ++b) {
      const int u = u0 + WAVES * b;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // behind column K zeros meet zeros
        const bool in = u < whole || (u < units && u * kKC + 64 * h + 16 * lg < K);
        const size_t off = (size_t)u * kKC + 64 * h;
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
        for (int t = 0; t < MT; ++t) acc[t] = mfma_i8(w[b][h], x[b][t][h], acc[t]);
  }
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int q = 0; q < 4; ++q) part[wave][t][q][lane] = acc[t][q];
  __syncthreads();
  // thread -> token r, column c: lane 16 (c / 4) + r % 16, result c % 4 of token tile r / 16
  for (int i = threadIdx.x; i < 256 * MT; i += 64 * WAVES) {
    const int r = i >> 4, c = i & 15;
    if (m0 + r >= p.M || n0 + c >= p.ncols) continue;
    uint32_t sum = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w)
      sum += (uint32_t)part[w][r >> 4][c & 3][16 * (c >> 2) + (r & 15)];
    const float all = K == kWrapK && (int)sum == INT32_MIN ? 0x1p31f : (float)(int)sum;
    const float v = all * (p.tok_scale[m0 + r] * p.w_scale[n0 + c]);
    const size_t o = (size_t)(m0 + r) * p.ncols + n0 + c;
    if (F32) static_cast<float*>(p.out)[o] = v;
    else static_cast<uint16_t*>(p.out)[o] = (uint16_t)f32_to_bf16_rne(v);
  }
}

template <int MT, bool F32>
hipError_t launch_skinny(I8Args& a, hipStream_t s) {
  a.n_ntiles = (a.ncols + 15) / 16;
  const int mblocks = (a.M + 16 * MT - 1) / (16 * MT);
  const int64_t per_xcd = ((int64_t)a.n_ntiles * mblocks + kXcds - 1) / kXcds;
  hipLaunchKernelGGL((i8_skinny_kernel<MT, F32>), dim3((unsigned)(per_xcd * kXcds)), dim3(512), 0, s,
                     a, mblocks, (int)per_xcd);
  return hipGetLastError();
}

// Variants of the dense product, by the time that a 128-wide step of K takes each (us,
// measured at K = 7168, N = 4096 with the chip full; the sums of the steps' latencies count
// where it is not):
//   workgroups of 16 weight rows, K over the waves, 64 tokens: 0.08 + 0.29 per 256 of them
//     (M=64: 21 us against 26.6 for 64 x 64 tiles; M=128: 35 against 27)
//   64 x 64 tiles, two workgroups a CU: 0.48 up to 256 of them, then 0.64 per 512
//     (M=256: 28 us against 41; M=512: 36 against 49; M=1024: 69 against 54)
//   step streams of 64, 128, 256 tokens x 256 weight rows: 0.88, 1.33, 2.09 per 256
//     (M=1024: 54, 61, 88 us; M=2048: 98, 74, 92; M=3500: 178, 136, 117)
// At 63 sizes (M 64 to 8192; N x K 4096 x 7168, 4096 x 2048, 1024 x 7168, 1024 x 2048, 7168 x
// 2048, 2048 x 640, 8192 x 1024, 4096 x 512, 4096 x 256) the pick is the fastest or within 8 % of
// it in 58, within 15 % in four (M=2048, N=4096, K=7168 72 us against 62.5 for 128 tokens), and
// 27 % slower in one (M=512, N=8192, K=1024: 19.4 us against 15.2 for 64 x 64 tiles).
template <bool F32>
hipError_t launch_dense(I8Args& a, hipStream_t s) {
  if (a.M <= 16) return launch_skinny<1, F32>(a, s);
  if (a.M <= 32) return launch_skinny<2, F32>(a, s);
  auto tiles = [&](int m, int n) {
    return (double)((a.M + m - 1) / m) * (double)((a.ncols + n - 1) / n);
  };
  const double t64 = tiles(64, 64);
  double best = t64 <= 256 ? 0.48 : 0.64 * ceil(t64 / 512);
  int pick = 0;
  auto offer = [&](int which, double cost) {
    if (cost < best) {
      best = cost;
      pick = which;
    }
  };
  offer(1, 0.08 + 0.29 * tiles(64, 16) / 256);
  if (a.K > 4 * kKC) {   // (the stream needs 2 D chunks per item)
    offer(64, 0.88 * ceil(tiles(64, 256) / 256));
    offer(128, 1.33 * ceil(tiles(128, 256) / 256));
    offer(256, 2.09 * ceil(tiles(256, 256) / 256));
  }
  switch (pick) {
    case 1: return launch_skinny<4, F32>(a, s);
    case 64: return launch_grouped<kDense, RingFew, 0, F32>(a, (a.M + 63L) / 64, s);
    case 128: return launch_grouped<kDense, RingMid, 0, F32>(a, (a.M + 127L) / 128, s);
    case 256: return launch_grouped<kDense, RingMany, 0, F32>(a, (a.M + 255L) / 256, s);
    default: return launch<64, 1, 4, 4, kDense, F32, 0>(a, (a.M + 63L) / 64, s);
  }
}

template <Mode MODE>
hipError_t launch_expert(I8Args& a, long tiles, int tile_rows, hipStream_t s) {
  if (a.K > 4 * kKC) {   // the stream needs 2 D chunks per item
    if (tile_rows == 64) return launch_grouped<MODE, RingFew, kStreamPolicy>(a, tiles, s);
    if (tile_rows == 128) return launch_grouped<MODE, RingMid, kStreamPolicy>(a, tiles, s);
    return launch_grouped<MODE, RingMany, kStreamPolicy>(a, tiles, s);
  }
  if (tile_rows == 64) return launch<64, 4, 1, 3, MODE, false, kStreamPolicy>(a, tiles, s);
  if (tile_rows == 128) return launch<128, 8, 1, 2, MODE, false, 0>(a, tiles, s);
  return launch<256, 4, 2, 2, MODE, false, 0>(a, tiles, s);
}

}  // namespace

hipError_t launch_i8_matmul(const int8_t* a, const float* a_scale, const int8_t* w,
                            const float* w_scale, int M, int N, int K, void* out, bool f32,
                            hipStream_t s) {
  I8Args p{};
  p.tok = a;
  p.tok_scale = a_scale;
  p.w = w;
  p.w_scale = w_scale;
  p.M = M;
  p.K = K;
  p.ncols = N;
  p.top_k = p.block = 1;
  p.out = out;
  return f32 ? launch_dense<true>(p, s) : launch_dense<false>(p, s);
}

static I8Args grouped(const int8_t* tok, const float* tok_scale, const int8_t* w,
                      const float* w_scale, const int32_t* sorted_ids,
                      const int32_t* block_expert, const int2* tiles, const int32_t* num_tiles,
                      int K, int ncols, int top_k, int block) {
  I8Args p{};
  p.tok = tok;
  p.tok_scale = tok_scale;
  p.w = w;
  p.w_scale = w_scale;
  p.sorted_ids = sorted_ids;
  p.block_expert = block_expert;
  p.tiles = tiles;
  p.num_tiles = num_tiles;
  p.K = K;
  p.ncols = ncols;
  p.top_k = top_k;
  p.block = block;
  return p;
}

hipError_t launch_i8_up(const int8_t* x, const float* x_scale, const int8_t* w13,
                        const float* w13_scale, const int32_t* sorted_ids,
                        const int32_t* block_expert, const int2* tiles, const int32_t* num_tiles,
                        int max_tiles, int tile_rows, int H, int I, int top_k,
                        int block, float* act, int act_rows,
                        hipStream_t s) {
  I8Args p = grouped(x, x_scale, w13, w13_scale, sorted_ids, block_expert, tiles, num_tiles, H, I,
                     top_k, block);
  p.act = act;
  p.act_rows = act_rows;
  return launch_expert<kUp>(p, max_tiles, tile_rows, s);
}

hipError_t launch_i8_down(const int8_t* act, const float* act_scale, const int8_t* w2,
                          const float* w2_scale, const int32_t* sorted_ids,
                          const int32_t* block_expert, const int2* tiles,
                          const int32_t* num_tiles, int max_tiles, int tile_rows, int H, int I,
                          int top_k, int block, float* y, hipStream_t s) {
  I8Args p = grouped(act, act_scale, w2, w2_scale, sorted_ids, block_expert, tiles, num_tiles, I,
                     H, top_k, block);
  p.y = y;
  return launch_expert<kDown>(p, max_tiles, tile_rows, s);
}

}  // namespace moe
