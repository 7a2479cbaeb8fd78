// int8 matrix products on MFMA (v_mfma_i32_16x16x64_i8): sums in int32, exact for
// K <= 131,072 (127^2 K < 2^31), scaled once at the end in fp32 by the scale of the token
// row and the scale of the weight row (output channel).
//
// Workgroup tile: BM token rows x 64 WN weight rows, K in chunks of 128 values (one
// 128-byte line per row).  Both operands are copied global -> LDS in 1 KiB pieces of 8 rows
// x one line; inside a row the 16-byte pieces are XOR-swizzled so that an MFMA fragment (16
// rows x 64 K values, 16 per lane) is one conflict-free ds_read_b128.  A ring of S stages
// keeps S - 1 chunks in flight; each wave waits for its own copies and a bare barrier
// publishes them.  Only a partial last chunk goes through registers (zero-filled).
//
// UP: tokens gathered through the plan, gate and up rows of 32 WN act columns, SwiGLU, act
// as block floats (below).  DOWN: act rows of the plan, results to the split y rows.  DENSE: plain rows.
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
  int n_ntiles, M, K, ncols, top_k, block;   // ncols: act columns (UP), output columns
  int16_t* act;
  uint8_t* act_exps;
  uint16_t* y;
  float* y0;
  void* out;
};

template <int BM, int WN, int WM>
struct I8Cfg {
  static constexpr int THREADS = 64 * WN * WM;
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

    // piece f of a chunk: rows 8h .. 8h + 7 (h = f % 2) of row tile f / 2 (weight tiles
    // first); lane l copies 16 bytes of row 8h + l / 8 into slot l % 8, which holds K piece
    // (l % 8) ^ (row % 8) ^ h.  Rows without data point at a valid row; their results are
    // never stored.
    const int8_t* src[C::PPW];
    bool on[C::PPW];
    int q16[C::PPW];
#pragma unroll
    for (int i = 0; i < C::PPW; ++i) {
      const int f = wave * C::PPW + i;
      const int rt = f >> 1, h = f & 1;
      const int rr = 8 * h + (lane >> 3);
      q16[i] = 16 * ((lane & 7) ^ (lane >> 3) ^ h);
      if (rt < C::WT) {
        int col, row;
        if (UP) {
          const bool up = rt >= C::WT / 2;
          col = col0 + (up ? rt - C::WT / 2 : rt) * 16 + rr;
          row = up ? p.ncols + col : col;
        } else {
          row = col = col0 + rt * 16 + rr;
        }
        on[i] = col < p.ncols;
        src[i] = p.w + (wrow0 + (on[i] ? row : 0)) * K + q16[i];
      } else {
        const int r = 16 * (rt - C::WT) + rr;
        on[i] = r < nlive;
        int row = start + (on[i] ? r : 0);
        if (UP) row = p.sorted_ids[row] / p.top_k;
        src[i] = p.tok + (size_t)row * K + q16[i];
      }
    }
    int wtile[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      wtile[j] = UP ? ((j < 2) ? 2 * wn + j : C::WT / 2 + 2 * wn + j - 2) : 4 * wn + j;

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
    const int frag_off = (li >> 3) * 1024 + (li & 7) * 128;
    auto frag = [&](int c, int t, int ks) -> u32x4 {
      const int q = (lg + 4 * ks) ^ (li & 7) ^ (li >> 3);
      return *reinterpret_cast<const u32x4*>(lds + (size_t)(c % S) * C::PIECES * 1024 + t * 2048 +
                                             frag_off + q * 16);
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
          for (int j = 0; j < 4; ++j) wa[j] = frag(c, wtile[j], ks);
#pragma unroll
          for (int s = 0; s < C::MTW; ++s) {
            if (s < my_active) {
              const u32x4 xb = frag(c, C::WT + wm * C::MTW + s, ks);
#pragma unroll
              for (int j = 0; j < 4; ++j) acc[j][s] = mfma_i8(wa[j], xb, acc[j][s]);
            }
          }
        }
      }
    }

    // lane (li, lg) holds weight rows 4 lg .. 4 lg + 3 of each weight tile, token row li
    const float* ws = p.w_scale + wrow0;
#pragma unroll
    for (int s = 0; s < C::MTW; ++s) {
      const int r = 16 * (wm * C::MTW + s) + li;
      if (s >= my_active || r >= nlive) continue;
      if (UP) {
        // act leaves as block floats: the wave's 32 columns of a row share a power of two
        // (byte E: value = int16 * 2^(E - 140), the largest below 2^14), because rounding
        // act to bf16 first moves one int8 code in ten by one (the layer's output 0.6 % off
        // in relative L2 instead of 0.2 %) and fp32 is twice the bytes.
        const float xs = p.tok_scale[p.sorted_ids[start + r] / p.top_k];
        float a[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int n = col0 + wn * 32 + h * 16 + 4 * lg;
          const bool in = n < p.ncols;
          const float4 g = *reinterpret_cast<const float4*>(ws + (in ? n : 0));
          const float4 u = *reinterpret_cast<const float4*>(ws + p.ncols + (in ? n : 0));
          const float gs[4] = {g.x, g.y, g.z, g.w}, us[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float v = silu_f32((float)acc[h][s][q] * (xs * gs[q])) *
                            ((float)acc[2 + h][s][q] * (xs * us[q]));
            a[h][q] = in ? v : 0.0f;
          }
        }
        uint32_t m = 0;   // magnitudes' bits order as they do, infinities and NaN last
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int q = 0; q < 4; ++q) m = max(m, __float_as_uint(a[h][q]) & 0x7fffffffu);
        // lanes of the same row (lg = 0 .. 3) are all live or all not
        m = max(m, (uint32_t)__shfl_xor((int)m, 16, kWave));
        m = max(m, (uint32_t)__shfl_xor((int)m, 32, kWave));
        const uint32_t E = max(m >> 23, 14u);
        const float mult = E == 255u ? 0.0f : __uint_as_float((267u - E) << 23);   // 2^(140 - E)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int n = col0 + wn * 32 + h * 16 + 4 * lg;
          int c[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) c[q] = E == 255u ? 0 : (int)rintf(a[h][q] * mult);
          if (n < p.ncols)
            *reinterpret_cast<uint2*>(p.act + (size_t)(start + r) * p.ncols + n) =
                uint2{(uint32_t)(c[0] & 0xffff) | (uint32_t)c[1] << 16,
                      (uint32_t)(c[2] & 0xffff) | (uint32_t)c[3] << 16};
        }
        const int b = (col0 >> 5) + wn;
        if (lg == 0 && 32 * b < p.ncols)
          p.act_exps[(size_t)(start + r) * ((p.ncols + 31) >> 5) + b] = (uint8_t)E;
      } else {
        const float xs = p.tok_scale[start + r];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int n = col0 + wn * 64 + j * 16 + 4 * lg;
          if (MODE == kDown) {
            if (n < p.ncols) {
              const float4 g = *reinterpret_cast<const float4*>(ws + n);
              store_y4(p.y, p.y0, y_row(p.sorted_ids[start + r], p.top_k, p.ncols), n,
                       (float)acc[j][s][0] * (xs * g.x), (float)acc[j][s][1] * (xs * g.y),
                       (float)acc[j][s][2] * (xs * g.z), (float)acc[j][s][3] * (xs * g.w));
            }
          } else {
            const size_t o = (size_t)(start + r) * p.ncols + n;
            if (n + 3 < p.ncols && p.ncols % 4 == 0) {
              const float4 g = *reinterpret_cast<const float4*>(ws + n);
              const float4 v =
                  make_float4((float)acc[j][s][0] * (xs * g.x), (float)acc[j][s][1] * (xs * g.y),
                              (float)acc[j][s][2] * (xs * g.z), (float)acc[j][s][3] * (xs * g.w));
              if (F32)
                *reinterpret_cast<float4*>(static_cast<float*>(p.out) + o) = v;
              else
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + o) =
                    uint2{pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w)};
            } else {
#pragma unroll
              for (int q = 0; q < 4; ++q)
                if (n + q < p.ncols) {
                  const float v = (float)acc[j][s][q] * (xs * ws[n + q]);
                  if (F32) static_cast<float*>(p.out)[o + q] = v;
                  else static_cast<uint16_t*>(p.out)[o + q] = (uint16_t)f32_to_bf16_rne(v);
                }
            }
          }
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
  const long tt = (M + 63L) / 64;
  return f32 ? launch<64, 4, 1, 3, kDense, true, 0>(p, tt, s)
             : launch<64, 4, 1, 3, kDense, false, 0>(p, tt, s);
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
                        int max_tiles, int tile_rows, bool stream_weights, int H, int I, int top_k,
                        int block, int16_t* act, uint8_t* act_exps, hipStream_t s) {
  I8Args p = grouped(x, x_scale, w13, w13_scale, sorted_ids, block_expert, tiles, num_tiles, H, I,
                     top_k, block);
  p.act = act;
  p.act_exps = act_exps;
  if (tile_rows == 64)
    return stream_weights ? launch<64, 4, 1, 3, kUp, false, kStreamPolicy>(p, max_tiles, s)
                          : launch<64, 4, 1, 3, kUp, false, 0>(p, max_tiles, s);
  return launch<128, 8, 1, 2, kUp, false, 0>(p, max_tiles, s);
}

hipError_t launch_i8_down(const int8_t* act, const float* act_scale, const int8_t* w2,
                          const float* w2_scale, const int32_t* sorted_ids,
                          const int32_t* block_expert, const int2* tiles,
                          const int32_t* num_tiles, int max_tiles, int tile_rows,
                          bool stream_weights, int H, int I, int top_k, int block, uint16_t* y,
                          float* y0, hipStream_t s) {
  I8Args p = grouped(act, act_scale, w2, w2_scale, sorted_ids, block_expert, tiles, num_tiles, I,
                     H, top_k, block);
  p.y = y;
  p.y0 = y0;
  if (tile_rows == 64)
    return stream_weights ? launch<64, 8, 1, 2, kDown, false, kStreamPolicy>(p, max_tiles, s)
                          : launch<64, 8, 1, 2, kDown, false, 0>(p, max_tiles, s);
  return launch<128, 8, 1, 2, kDown, false, 0>(p, max_tiles, s);
}

}  // namespace moe
