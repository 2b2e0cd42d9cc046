// Attention of each sequence's newest tokens over its 4-bit cache.
//
//   S_t = scale q . K_t,  p = softmax over the visible t,  out = sum_t p_t V_t
//   K_t = lo + s u (per group of channels), V_t likewise, u = 0..15
//
// so a group's share of S_t is scale (s sum q u + lo sum q), and of out
// sum_t (p_t s_t) u_t + sum_t p_t lo_t: the matrix products only ever see the
// codes u and never a rebuilt K or V.
//
// Bound by the cache's bytes as long as the unpacking keeps up: at 6.5 TB/s an
// SM takes in about 49 codes per clock. What keeps the instruction count near
// one per two codes:
//  - Two codes are masked out of a word in place and OR'ed under the exponent
//    of 1024 in one operation; a packed subtraction leaves u - 8 (16 times that
//    for the upper 4 bits of a byte) as exact fp16, and lo + 8 s replaces lo.
//    Without the subtraction the masked bits are fp16 subnormals, exact too, and
//    mma takes them: but it aligns products by their nominal exponents, and the
//    result was 2e-4 off at 67000 tokens (fp16 rounds by 2e-4), now 2e-7.
//  - The order of a contraction is free, so the packed order of a row is the
//    order of the mma fragments (kv_cache.cu): a lane's K words feed its
//    A fragments without a shuffle, and two tokens' V words give the pairs of
//    the second product with one byte permute per 4 pairs.
//  - Tokens are the 16 rows of the first product and the contraction of the
//    second, query rows the 8 columns: S^T = K q^T and out^T = V^T p^T.
//  - Of the 8 columns 4 are query rows and 4 repeat them: in the second
//    product the repeats carry what rounding p s to fp16 lost. The result
//    then has fp32's error although mma takes fp16, at no extra mma for up to
//    4 query rows per KV head (32 / 8 and 40 / 10 heads).
// The tcgen05 tensor cores would need the codes expanded to 8 or 16 bits in
// shared memory first, 2 to 4 times the cache's bytes of shared-memory writes
// and reads, for products that mma.sync does within the bytes' time.
//
// A warp takes 32 tokens at a time straight from global memory into registers
// (the next 32 load while these are computed), the warps of a CTA take such
// tiles in turn and join their sums once, at the end. Nothing in the loop
// waits for another warp. Few (sequence, head) pairs are split over the
// tokens; a second kernel joins the splits.
#include <climits>

#include "kernel_common.cuh"
#include "kv_cache.hpp"
#include "ops_common.cuh"

namespace stagq {
namespace {

__device__ uint32_t g_status;

using kernels::grid_dependency_wait;
using kernels::grid_launch_dependents;
using kernels::kFull;

constexpr int kWarps = 4;
constexpr int kTile = 32;            // tokens of a warp's tile
constexpr int kMaxSplits = 256;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// Two codes in their halves' lowest 4 bits (HIGH: the 4 above) as fp16 u - 8
// (HIGH: 16 times that), exact: 0x6400 | u is the half 1024 + u.
template <bool HIGH>
__device__ __forceinline__ uint32_t centered(uint32_t w) {
  const uint32_t v = (w & (HIGH ? 0x00F000F0u : 0x000F000Fu)) | 0x64006400u;
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(HIGH ? 0x64806480u : 0x64086408u));
  return r;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

template <int WORDS>
__device__ __forceinline__ void load_words(uint32_t (&w)[WORDS], const uint8_t* p) {
  static_assert(WORDS == 1 || WORDS == 2 || WORDS % 4 == 0, "one vector load, or several of 16 bytes");
  if constexpr (WORDS == 1) {
    w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
  } else if constexpr (WORDS == 2) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    w[0] = v.x;
    w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < WORDS / 4; ++i) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
      w[4 * i] = v.x;
      w[4 * i + 1] = v.y;
      w[4 * i + 2] = v.z;
      w[4 * i + 3] = v.w;
    }
  }
}

// One warp's 32 tokens as a lane (g = lane / 4, t = lane mod 4) holds them:
// K codes of tokens 4 g .. 4 g + 3 (channels 32 j + 8 t + 0..7), V codes of
// tokens 8 t .. 8 t + 7 (channels 32 j + 4 g + 0..3), and both pairs of
// tokens 4 g .. 4 g + 3.
template <int D, int NG>
struct Tile {
  uint32_t k[4][D / 32];
  uint32_t v[8][D / 64];
  uint32_t mk[4 * NG], mv[4 * NG];
  bool ok;  // the page of tokens 4 g .. 4 g + 3 is in the pool
};

// Query positions of row r: token r / per of the n_new newest sees the tokens
// before `limit`.
__device__ __forceinline__ int row_limit(const KvAttnArgs& a, int len, int r) {
  return len - (a.n_new - 1 - r / a.per);
}

__device__ __forceinline__ int clamped_len(const KvAttnArgs& a, int b) {
  const int len = a.lens[b];
  return len < 0 ? 0 : min(len, a.max_len);
}

template <int D, int NG, int NT>
__global__ void __launch_bounds__(kWarps * 32, NT == 1 ? 3 : 2) kv_attention_kernel(const __grid_constant__ KvAttnArgs a) {
  constexpr int J = D / 32;       // blocks of 32 channels
  constexpr int JG = J / NG;      // blocks of a group
  constexpr int ROWS = 4 * NT;
  __shared__ float s_o[kWarps][ROWS][D];
  __shared__ float s_m[kWarps][ROWS], s_l[kWarps][ROWS];

  grid_launch_dependents();
  grid_dependency_wait();
  const KvView& kv = a.kv;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  int unit = blockIdx.x;
  const int split = unit % a.splits;
  unit /= a.splits;
  const int rb = unit % a.row_blocks;
  const int bh = unit / a.row_blocks;
  const int b = bh / kv.heads, h = bh - b * kv.heads;
  const int r0 = rb * ROWS;
  const int len = clamped_len(a, b);
  if (threadIdx.x == 0 && len != a.lens[b]) atomicOr(&g_status, kOpsBadPage);
  const int limmax = max(0, row_limit(a, len, min(r0 + ROWS, a.rows) - 1));  // of the block's last row

  // this CTA's tiles: an even share of the sequence's, whole rounds of warps apart from the last
  const int tiles = (limmax + kTile - 1) / kTile;
  const int share = (tiles + a.splits - 1) / a.splits;
  const int tile_end = min(tiles, (split + 1) * share);
  int tile = split * share + warp;

  // q in fp16, each row scaled by a power of two so that its largest value is
  // in [2^10, 2^11): exact for fp16 and bf16 alike (and q / 16 too), down to
  // values 2^-34 of the row's largest.
  uint32_t qf[NT][J][4];
  float cf[NT][2], qs[NT][2][NG];
  int lim[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = r0 + 4 * nt + (g & 3);
    float x[J][8];
    float amax = 0.0f;
    bool fine = true;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      uint16_t raw[8] = {};
      if (r < a.rows) {
        const int tok = r / a.per;
        ops::load8(a.q + (static_cast<int64_t>(b) * a.n_new + tok) * a.q_stride + (h * a.per + r - tok * a.per) * D + 32 * j + 8 * t,
                   a.vec, raw);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[j][i] = ops::load16(raw[i], kv.bf16);
        fine = fine && isfinite(x[j][i]);
        amax = fmaxf(amax, fabsf(x[j][i]));
      }
    }
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
      amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, d));
      fine = __shfl_xor_sync(kFull, fine ? 1 : 0, d) && fine;
    }
    const int e = fine && amax > 0.0f ? max(-126, static_cast<int>(__float_as_uint(amax) >> 23) - 127 - 10) : 0;
    const float down = pow2(-e);
    const float c = fine ? a.scale_log2 * pow2(e) : __uint_as_float(0x7FC00000u);
    float sum[NG];
#pragma unroll
    for (int n = 0; n < NG; ++n) sum[n] = 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[j][i] = fine ? x[j][i] * down : 0.0f;
        sum[j / JG] += x[j][i];
      }
      // word nibbles 0, 4 | 1, 5 (16 times) | 2, 6 | 3, 7 (16 times)
      qf[nt][j][0] = pack_half2(x[j][0], x[j][4]);
      qf[nt][j][1] = pack_half2(x[j][1] * 0.0625f, x[j][5] * 0.0625f);
      qf[nt][j][2] = pack_half2(x[j][2], x[j][6]);
      qf[nt][j][3] = pack_half2(x[j][3] * 0.0625f, x[j][7] * 0.0625f);
    }
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      sum[n] += __shfl_xor_sync(kFull, sum[n], 1);
      sum[n] += __shfl_xor_sync(kFull, sum[n], 2);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // this lane's columns 2 t + i are rows (2 t + i) mod 4 of the tile
      const int row = (2 * t + i) & 3;
      cf[nt][i] = __shfl_sync(kFull, c, 4 * row);
#pragma unroll
      for (int n = 0; n < NG; ++n) qs[nt][i][n] = __shfl_sync(kFull, sum[n], 4 * row);
      const int rr = r0 + 4 * nt + row;
      lim[nt][i] = rr < a.rows ? row_limit(a, len, rr) : limmax;
    }
  }
  int lim_min = lim[0][0];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) lim_min = min(lim_min, min(lim[nt][0], lim[nt][1]));
  lim_min = __reduce_min_sync(kFull, lim_min);

  float o[J][2][NT][4];
  float m[NT][2], l[NT][2], lsum[NT][2][NG];
  int e_run[NG];                 // exponent field that p s is scaled by, 15 at least
#pragma unroll
  for (int n = 0; n < NG; ++n) e_run[n] = 15;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      m[nt][i] = -INFINITY;
      l[nt][i] = 0.0f;
#pragma unroll
      for (int n = 0; n < NG; ++n) lsum[nt][i][n] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[j][0][nt][c] = o[j][1][nt][c] = 0.0f;
  }

  const int last_page = max(0, (limmax - 1) >> kv.page_shift);
  const int32_t* table = kv.table + b * kv.table_stride;
  const uint8_t* head = kv.pages + static_cast<int64_t>(2 * h) * kv.block_bytes;
  const int meta_off = kv.page * (D / 2);
  // page numbers of tile `i`'s tokens 4 g and 8 t (those past the end: the last page)
  auto load_pages = [&](int i, int& pk, int& pv) {
    pk = __ldg(table + min((i * kTile + 4 * g) >> kv.page_shift, last_page));
    pv = __ldg(table + min((i * kTile + 8 * t) >> kv.page_shift, last_page));
  };
  auto load_tile = [&](int i, int pk, int pv, Tile<D, NG>& x) {
    x.ok = pk >= 0 && pk < kv.n_pages;
    pk = x.ok ? pk : 0;
    pv = pv >= 0 && pv < kv.n_pages ? pv : 0;
    const uint8_t* kb = head + pk * kv.page_stride;
    const uint8_t* vb = head + pv * kv.page_stride + kv.block_bytes;
    const int sk = (i * kTile + 4 * g) & (kv.page - 1), sv = (i * kTile + 8 * t) & (kv.page - 1);
#pragma unroll
    for (int n = 0; n < 4; ++n) load_words<J>(x.k[n], kb + (sk + n) * (D / 2) + t * (D / 8));
    load_words<4 * NG>(x.mk, kb + meta_off + sk * (4 * NG));
#pragma unroll
    for (int n = 0; n < 8; ++n) load_words<J / 2>(x.v[n], vb + (sv + n) * (D / 2) + g * (D / 16));
    load_words<4 * NG>(x.mv, head + pk * kv.page_stride + kv.block_bytes + meta_off + sk * (4 * NG));
  };

  Tile<D, NG> cur;
  int pk = 0, pv = 0;
  if (tile < tile_end) {
    load_pages(tile, pk, pv);
    load_tile(tile, pk, pv, cur);
    if (tile + kWarps < tile_end) load_pages(tile + kWarps, pk, pv);
  }
  while (tile < tile_end) {
    Tile<D, NG> nxt = cur;
    const int next = tile + kWarps;
    if (next < tile_end) {
      load_tile(next, pk, pv, nxt);
      if (next + kWarps < tile_end) load_pages(next + kWarps, pk, pv);
    }
    const int tok0 = tile * kTile + 4 * g;
    const uint32_t bad = __ballot_sync(kFull, !cur.ok && tok0 < limmax);
    if (bad && lane == 0) atomicOr(&g_status, kOpsBadPage);
    const bool edge = (tile + 1) * kTile > lim_min || bad;  // some row does not see all of the tile
    if (edge) {
      // tokens that no row sees may hold anything: their pairs count as zero
#pragma unroll
      for (int n = 0; n < 4; ++n)
        if (!cur.ok || tok0 + n >= limmax) {
#pragma unroll
          for (int c = 0; c < NG; ++c) cur.mk[n * NG + c] = cur.mv[n * NG + c] = 0u;
        }
    }

    // S^T: rows g and g + 8 of product `mt` are tokens 4 g + 2 mt and the next
    float s[NT][2][4];  // [column][token]
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      float acc[NT][NG][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int n = 0; n < NG; ++n) acc[nt][n][0] = acc[nt][n][1] = acc[nt][n][2] = acc[nt][n][3] = 0.0f;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const uint32_t w0 = cur.k[2 * mt][j], w1 = cur.k[2 * mt + 1][j];
        const uint32_t a0 = centered<false>(w0), a1 = centered<false>(w1), a2 = centered<true>(w0), a3 = centered<true>(w1);
        const uint32_t b0 = centered<false>(w0 >> 8), b1 = centered<false>(w1 >> 8), b2 = centered<true>(w0 >> 8),
                       b3 = centered<true>(w1 >> 8);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma16816(acc[nt][j / JG], a0, a1, a2, a3, qf[nt][j][0], qf[nt][j][1]);
          mma16816(acc[nt][j / JG], b0, b1, b2, b3, qf[nt][j][2], qf[nt][j][3]);
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float sum = 0.0f;
#pragma unroll
            for (int c = 0; c < NG; ++c) {
              const uint32_t w = cur.mk[(2 * mt + n) * NG + c];
              const float sc = ops::load16(static_cast<uint16_t>(w), kv.bf16);
              const float lo = fmaf(sc, 8.0f, ops::load16(static_cast<uint16_t>(w >> 16), kv.bf16));
              sum += fmaf(sc, acc[nt][c][2 * n + i], lo * qs[nt][i][c]);
            }
            s[nt][i][2 * mt + n] = sum * cf[nt][i];
          }
    }
    if (edge) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int n = 0; n < 4; ++n)
            if (!cur.ok || tok0 + n >= lim[nt][i]) s[nt][i][n] = -INFINITY;
    }
    if (a.scores && t < 2) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          *reinterpret_cast<float4*>(a.scores + (static_cast<int64_t>(bh) * a.rows_pad + r0 + 4 * nt + 2 * t + i) * a.score_stride +
                                     tok0) = make_float4(s[nt][i][0], s[nt][i][1], s[nt][i][2], s[nt][i][3]);
    }

    // running maximum; sums are rescaled only when one of the warp's rises
    float top[NT][2];
    bool rises = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = fmaxf(fmaxf(s[nt][i][0], s[nt][i][1]), fmaxf(s[nt][i][2], s[nt][i][3]));
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, d));
        top[nt][i] = fmaxf(m[nt][i], x);
        rises = rises || top[nt][i] > m[nt][i];
      }
    if (__any_sync(kFull, rises)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float f = top[nt][i] > m[nt][i] ? ex2(m[nt][i] - top[nt][i]) : 1.0f;  // the first time: 0
          m[nt][i] = top[nt][i];
          l[nt][i] *= f;
#pragma unroll
          for (int n = 0; n < NG; ++n) lsum[nt][i][n] *= f;
#pragma unroll
          for (int j = 0; j < J; ++j) {
            o[j][0][nt][i] *= f;
            o[j][0][nt][2 + i] *= f;
            o[j][1][nt][i] *= f;
            o[j][1][nt][2 + i] *= f;
          }
        }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float base = m[nt][i] == -INFINITY ? 0.0f : m[nt][i];  // a row that has seen nothing yet
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          s[nt][i][n] = ex2(s[nt][i][n] - base);
          l[nt][i] += s[nt][i][n];
        }
      }

#pragma unroll
    for (int c = 0; c < NG; ++c) {
      float sv[4], lo[4];
      uint32_t top_s = 0;
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const uint32_t w = cur.mv[n * NG + c];
        sv[n] = ops::load16(static_cast<uint16_t>(w), kv.bf16);
        lo[n] = fmaf(sv[n], 8.0f, ops::load16(static_cast<uint16_t>(w >> 16), kv.bf16));
        const uint32_t bits = __float_as_uint(fabsf(sv[n]));
        if (bits < 0x7F800000u) top_s = max(top_s, bits);
      }
      // p s is held as p s 2^(14 - e), e the exponent of the largest s so far
      const int e_new = static_cast<int>(__reduce_max_sync(kFull, top_s) >> 23);
      if (e_new > e_run[c]) {
        const float f = e_new - e_run[c] > 126 ? 0.0f : pow2(e_run[c] - e_new);
#pragma unroll
        for (int j = c * JG; j < (c + 1) * JG; ++j)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              o[j][0][nt][i] *= f;
              o[j][1][nt][i] *= f;
            }
        e_run[c] = e_new;
      }
      const float f = __uint_as_float(static_cast<uint32_t>(268 - e_run[c]) << 23);
      uint32_t pf[NT][4];  // B fragments of both products, k = token
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          float x[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const bool hidden = edge && tok0 + n >= lim[nt][i];  // 0 times a NaN that other rows see
            x[i] = hidden ? 0.0f : s[nt][i][n] * (sv[n] * f);
            lsum[nt][i][c] += hidden ? 0.0f : s[nt][i][n] * lo[n];
          }
          const __half2 hi = __floats2half2_rn(x[0], x[1]);
          const float2 back = __half22float2(hi);
          const uint32_t rest = pack_half2(x[0] - back.x, x[1] - back.y);
          pf[nt][n] = transpose8x8(t < 2 ? *reinterpret_cast<const uint32_t*>(&hi) : rest);
        }
      }
#pragma unroll
      for (int j = c * JG; j < (c + 1) * JG; ++j)
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          // tokens 8 t + 2 mt and 8 t + 4 + 2 mt, then the ones after each
          constexpr uint32_t kLow = 0x5410u, kHigh = 0x7632u;
          const uint32_t sel = (j & 1) ? kHigh : kLow;
          const uint32_t p0 = __byte_perm(cur.v[2 * mt][j / 2], cur.v[2 * mt + 4][j / 2], sel);
          const uint32_t p1 = __byte_perm(cur.v[2 * mt + 1][j / 2], cur.v[2 * mt + 5][j / 2], sel);
          const uint32_t a0 = centered<false>(p0), a1 = centered<true>(p0), a2 = centered<false>(p1), a3 = centered<true>(p1);
          const uint32_t b0 = centered<false>(p0 >> 8), b1 = centered<true>(p0 >> 8), b2 = centered<false>(p1 >> 8),
                         b3 = centered<true>(p1 >> 8);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma16816(o[j][0][nt], a0, a1, a2, a3, pf[nt][2 * mt], pf[nt][2 * mt + 1]);
            mma16816(o[j][1][nt], b0, b1, b2, b3, pf[nt][2 * mt], pf[nt][2 * mt + 1]);
          }
        }
    }
    cur = nxt;
    tile = next;
  }

  // the warp's sums to shared memory, in natural units
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) {
        l[nt][i] += __shfl_xor_sync(kFull, l[nt][i], d);
#pragma unroll
        for (int n = 0; n < NG; ++n) lsum[nt][i][n] += __shfl_xor_sync(kFull, lsum[nt][i][n], d);
      }
      const int row = 4 * nt + 2 * t + i;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        float x[4] = {o[j][0][nt][i], o[j][0][nt][2 + i] * 0.0625f, o[j][1][nt][i], o[j][1][nt][2 + i] * 0.0625f};
        const float up = pow2(e_run[j / JG] - 127 - 14);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          x[n] += __shfl_xor_sync(kFull, x[n], 2);  // the columns of the rounding's rest
          x[n] = fmaf(x[n], up, lsum[nt][i][j / JG]);
        }
        if (t < 2) *reinterpret_cast<float4*>(&s_o[warp][row][32 * j + 4 * g]) = make_float4(x[0], x[1], x[2], x[3]);
      }
      if (t < 2 && g == 0) {
        s_m[warp][row] = m[nt][i];
        s_l[warp][row] = l[nt][i];
      }
    }
  __syncthreads();
  const bool direct = a.splits == 1 && !a.scores;
  for (int idx = threadIdx.x; idx < ROWS * D; idx += kWarps * 32) {
    const int row = idx / D, d = idx - row * D, r = r0 + row;
    float top = s_m[0][row];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_m[w][row]);
    const float base = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f, den = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = ex2(s_m[w][row] - base);
      sum += f * s_o[w][row][d];
      den += f * s_l[w][row];
    }
    if (r >= a.rows) continue;
    if (direct) {
      const int tok = r / a.per;
      a.out[(static_cast<int64_t>(b) * a.n_new + tok) * a.out_stride + (h * a.per + r - tok * a.per) * D + d] =
          ops::store16(den == 0.0f ? 0.0f : sum / den, kv.bf16);
    } else {
      const int64_t at = (static_cast<int64_t>(bh) * a.rows_pad + r) * a.splits + split;
      a.part_o[at * D + d] = sum;
      if (d == 0) a.part_ml[at] = make_float2(top, den);
    }
  }
}

// Joins the splits: the first batch * heads * rows CTAs each write one output
// row; the others add the weights exp2(S - lse) of 4 * blockDim tokens of one
// (sequence, head) to the mass, every element by one thread in one order.
template <int D>
__global__ void __launch_bounds__(128) kv_join_kernel(const __grid_constant__ KvAttnArgs a) {
  __shared__ float s_w[kMaxSplits];
  __shared__ float s_lse[STAGQ_KV_MAX_NEW * STAGQ_KV_MAX_SHARE];
  grid_launch_dependents();
  grid_dependency_wait();
  const KvView& kv = a.kv;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t n_rows = static_cast<int64_t>(a.batch) * kv.heads * a.rows;
  if (blockIdx.x < n_rows) {
    const int bh = blockIdx.x / a.rows, r = blockIdx.x - bh * a.rows;
    const int b = bh / kv.heads, h = bh - b * kv.heads;
    const int64_t at = (static_cast<int64_t>(bh) * a.rows_pad + r) * a.splits;
    float top = -INFINITY;
    for (int s = lane; s < a.splits; s += 32) top = fmaxf(top, a.part_ml[at + s].x);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, d));
    const float base = top == -INFINITY ? 0.0f : top;
    float den = 0.0f;
    for (int s = lane; s < a.splits; s += 32) {
      const float2 ml = a.part_ml[at + s];
      const float f = ex2(ml.x - base);
      if (warp == 0) s_w[s] = f;
      den += f * ml.y;
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) den += __shfl_xor_sync(kFull, den, d);
    __syncthreads();
    const int d = threadIdx.x;
    if (d >= D) return;
    float sum = 0.0f;
#pragma unroll 8
    for (int s = 0; s < a.splits; ++s) sum += s_w[s] * a.part_o[(at + s) * D + d];
    const int tok = r / a.per;
    a.out[(static_cast<int64_t>(b) * a.n_new + tok) * a.out_stride + (h * a.per + r - tok * a.per) * D + d] =
        ops::store16(den == 0.0f ? 0.0f : sum / den, kv.bf16);
    return;
  }
  const int chunks = (a.max_len + 511) / 512;
  const int unit = static_cast<int>(blockIdx.x - n_rows);
  const int bh = unit / chunks, t0 = (unit - bh * chunks) * 512;
  const int b = bh / kv.heads, h = bh - b * kv.heads;
  const int len = clamped_len(a, b);
  if (t0 >= len) return;
  for (int r = warp; r < a.rows; r += 4) {
    const int64_t at = (static_cast<int64_t>(bh) * a.rows_pad + r) * a.splits;
    float top = -INFINITY;
    for (int s = lane; s < a.splits; s += 32) top = fmaxf(top, a.part_ml[at + s].x);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, d));
    const float base = top == -INFINITY ? 0.0f : top;
    float den = 0.0f;
    for (int s = lane; s < a.splits; s += 32) {
      const float2 ml = a.part_ml[at + s];
      den += ex2(ml.x - base) * ml.y;
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) den += __shfl_xor_sync(kFull, den, d);
    if (lane == 0) s_lse[r] = base + log2f(den);
  }
  __syncthreads();
  float* mass = a.mass + b * a.mass_stride_b + h * a.mass_stride_h;
  const float* scores = a.scores + static_cast<int64_t>(bh) * a.rows_pad * a.score_stride;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int tok = t0 + 128 * i + threadIdx.x;
    if (tok >= len) break;
    float sum = 0.0f;
    for (int r = 0; r < a.rows; ++r)
      if (tok < row_limit(a, len, r)) sum += ex2(scores[r * a.score_stride + tok] - s_lse[r]);
    mass[tok] += sum;
  }
}

template <int D, int NG, int NT>
cudaError_t launch_attention(const KvAttnArgs& a, cudaStream_t s) {
  const int64_t ctas = static_cast<int64_t>(a.batch) * a.kv.heads * a.row_blocks * a.splits;
  cudaError_t e = launch_op(kv_attention_kernel<D, NG, NT>, dim3(static_cast<unsigned>(ctas)), dim3(kWarps * 32), 0, s, a);
  if (e != cudaSuccess || (a.splits == 1 && !a.scores)) return e;
  int64_t join = static_cast<int64_t>(a.batch) * a.kv.heads * a.rows;
  if (a.scores) join += static_cast<int64_t>(a.batch) * a.kv.heads * ((a.max_len + 511) / 512);
  return launch_op(kv_join_kernel<D>, dim3(static_cast<unsigned>(join)), dim3(128), 0, s, a);
}

template <int D, int NG>
cudaError_t launch_nt(const KvAttnArgs& a, int nt, cudaStream_t s) {
  return nt == 1 ? launch_attention<D, NG, 1>(a, s) : launch_attention<D, NG, 2>(a, s);
}

int64_t align256(int64_t v) { return (v + 255) / 256 * 256; }

}  // namespace

// Four query rows of a KV head per CTA, eight where there are more than four
// (the cache is then read once per eight rows). The tokens are split until the
// CTAs fill the GPU three times over (three fit an SM), but a split keeps
// one tile for each warp.
KvAttnPlan plan_kv_attention(int batch, int heads, int q_heads, int n_new, int dim, int max_len, bool mass,
                             int num_sms) {
  KvAttnPlan p{};
  const int rows = q_heads / heads * n_new;
  p.nt = rows <= 4 ? 1 : 2;
  p.row_blocks = (rows + 4 * p.nt - 1) / (4 * p.nt);
  p.rows_pad = p.row_blocks * 4 * p.nt;
  const int64_t units = static_cast<int64_t>(batch) * heads * p.row_blocks;
  const int64_t tiles = (static_cast<int64_t>(max_len) + kTile - 1) / kTile;
  int64_t splits = (static_cast<int64_t>(num_sms) * (p.nt == 1 ? 3 : 2)) / units;
  const int64_t most = (tiles + kWarps - 1) / kWarps;
  if (splits > most) splits = most;
  if (splits > kMaxSplits) splits = kMaxSplits;
  if (splits < 1) splits = 1;
  p.splits = static_cast<int>(splits);
  p.score_stride = mass ? tiles * kTile : 0;
  if (p.splits > 1 || mass) {
    const int64_t parts = static_cast<int64_t>(batch) * heads * p.rows_pad * p.splits;
    p.off_ml = 0;
    p.off_o = align256(parts * 8);
    p.off_scores = p.off_o + align256(parts * dim * 4);
    p.bytes = p.off_scores + align256(static_cast<int64_t>(batch) * heads * p.rows_pad * p.score_stride * 4);
  }
  return p;
}

cudaError_t launch_kv_attention(const KvAttnArgs& a, const KvAttnPlan& p, cudaStream_t s) {
  const int ng = a.kv.dim / a.kv.group;
  if (a.kv.dim == 128)
    return ng == 1 ? launch_nt<128, 1>(a, p.nt, s) : ng == 2 ? launch_nt<128, 2>(a, p.nt, s) : launch_nt<128, 4>(a, p.nt, s);
  return ng == 1 ? launch_nt<64, 1>(a, p.nt, s) : launch_nt<64, 2>(a, p.nt, s);
}

cudaError_t take_status_kv_attention(uint32_t* word) {
  cudaError_t e = cudaMemcpyFromSymbol(word, g_status, sizeof(uint32_t));
  if (e != cudaSuccess || !*word) return e;
  const uint32_t zero = 0;
  return cudaMemcpyToSymbol(g_status, &zero, sizeof(zero));
}

}  // namespace stagq
