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
// A warp takes 32 tokens at a time. Each has a ring of tiles in shared memory
// of its own, filled by bulk copies (4 per tile, one per lane, 8 where a page
// holds half a tile) two tiles ahead: no registers wait for memory, so 16 warps
// fit an SM. The four warps of a CTA take tiles in turn and join their sums at
// the end; nothing in the loop waits for another warp.
//
// The work is cut into rounds of 128 tokens (a tile per warp) of a unit
// (sequence, KV head, block of query rows), numbered unit after unit, and every
// CTA takes an equal run of that numbering, read off the lengths on the
// device. A ragged batch, one long sequence and many short ones thus fill the
// GPU alike. A unit that one CTA covers is written out; the others leave a
// partial sum (at most two per CTA), and a second kernel joins those.
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
// (HIGH: 16 times that), exact: 0x6400 | u is the half 1024 + u. `exponent` is
// 0x64006400 in a register: with two immediates the masking and the OR would
// be two instructions.
template <bool HIGH>
__device__ __forceinline__ uint32_t centered(uint32_t w, uint32_t exponent) {
  uint32_t v, r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(w), "n"(HIGH ? 0x00F000F0 : 0x000F000F), "r"(exponent));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(HIGH ? 0x64806480u : 0x64086408u));
  return r;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Both values toward zero, hi in the upper half.
__device__ __forceinline__ uint32_t pack_half2_rz(float lo, float hi) {
  uint32_t r;
  asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// The pair (scale, lowest) of a group.
template <bool BF>
__device__ __forceinline__ float pair_scale(uint32_t w) {
  return BF ? __uint_as_float(w << 16) : __low2float(*reinterpret_cast<const __half2*>(&w));
}
template <bool BF>
__device__ __forceinline__ float pair_low(uint32_t w) {
  return BF ? __uint_as_float(w & 0xFFFF0000u) : __high2float(*reinterpret_cast<const __half2*>(&w));
}
// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

template <int WORDS>
__device__ __forceinline__ void load_words(uint32_t (&w)[WORDS], const uint8_t* p) {
  static_assert(WORDS == 1 || WORDS == 2 || WORDS == 4, "one vector load");
  if constexpr (WORDS == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (WORDS == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x;
    w[1] = v.y;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
  }
}

constexpr int kStages = 3;
constexpr uint64_t kWaitLimitNs = 2000000000ull;

// A tile in shared memory: codes of K and of V (32 rows of D / 2 bytes each),
// pairs of K and of V.
template <int D, int NG>
struct TileLayout {
  static constexpr int kCodes = kTile * D / 2, kPairs = kTile * 4 * NG;
  static constexpr int kV = kCodes, kPairsK = 2 * kCodes, kPairsV = 2 * kCodes + kPairs;
  static constexpr int kBytes = 2 * (kCodes + kPairs);
};
// Row r of a product's 16 (8 for each half) is token tau(r) of the tile's 16:
// with 64-byte rows, the K rows that 8 lanes read at a time then lie in
// different halves of the banks, and so do two of the four V rows.
__device__ __forceinline__ int tau(int r) { return r ^ ((r >> 1) & 1); }

// Query positions of row r: token r / per of the n_new newest sees the tokens
// before `limit`.
__device__ __forceinline__ int row_limit(const KvAttnArgs& a, int len, int r) {
  return len - (a.n_new - 1 - r / a.per);
}

__device__ __forceinline__ int clamped_len(const KvAttnArgs& a, int b) {
  const int len = a.lens[b];
  return len < 0 ? 0 : min(len, a.max_len);
}

// Rounds of 128 tokens of sequence b (one head, one block of query rows).
__device__ __forceinline__ int rounds_of(const KvAttnArgs& a, int b) {
  return (clamped_len(a, b) + kWarps * kTile - 1) / (kWarps * kTile);
}
// The rounds of the sequences before b, and of all of them. The lanes of a
// warp take 32 sequences at a time.
__device__ __forceinline__ int64_t rounds_before(const KvAttnArgs& a, int b, int lane) {
  int64_t n = 0;
  for (int i = lane; i < b; i += 32) n += rounds_of(a, i);
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) n += __shfl_xor_sync(kFull, n, d);
  return n;
}
// CTAs that get a run of `total` rounds, of at least one round each, and the
// first round of CTA c's.
__device__ __forceinline__ int busy_ctas(int64_t total, int ctas) { return total < ctas ? static_cast<int>(total) : ctas; }
__device__ __forceinline__ int64_t run_start(int64_t total, int c, int busy) { return total * c / busy; }

template <int D, int NG, int NT, bool BF>
__global__ void __launch_bounds__(kWarps * 32, NT == 1 ? 4 : 2) kv_attention_kernel(const __grid_constant__ KvAttnArgs a) {
  constexpr int J = D / 32;       // blocks of 32 channels
  constexpr int JG = J / NG;      // blocks of a group
  constexpr int ROWS = 4 * NT;
  using L = TileLayout<D, NG>;
  static_assert(kStages * L::kBytes >= ROWS * D * 4, "the warps' sums take the rings' place");
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_m[kWarps][ROWS], s_l[kWarps][ROWS];
  __shared__ __align__(8) uint64_t s_full[kWarps][kStages];
  __shared__ uint32_t s_ok[kWarps][kStages];  // by lane: whether its piece's page is in the pool
  float (*s_o)[ROWS][D] = reinterpret_cast<float (*)[ROWS][D]>(smem);

  grid_launch_dependents();
  grid_dependency_wait();
  const KvView& kv = a.kv;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int units_b = kv.heads * a.row_blocks;  // units of a sequence

  uint8_t* ring = smem + warp * (kStages * L::kBytes);
  const uint32_t ring_addr = kernels::smem_addr(ring), full_addr = kernels::smem_addr(&s_full[warp][0]);
  if (lane < kStages) kernels::mbar_init(full_addr + 8 * lane, 1);
  kernels::fence_barrier_init();
  __syncthreads();
  uint32_t filled = 0, used = 0;  // tiles that this warp has asked for, and waited for
  bool dead = false;              // a wait ran out: nothing more is asked for or waited for
  // What lane l copies of a tile: piece l / 4 of its tokens (two pieces where a
  // page holds half a tile), K codes, V codes, K pairs or V pairs.
  const int piece_tokens = min(kv.page, kTile), piece = kv.page < kTile ? (lane >> 2) & 1 : 0;
  const int kind = lane & 3, row_bytes = kind < 2 ? D / 2 : 4 * NG;
  const bool copies = lane < 4 * (kTile / piece_tokens);
  const uint32_t copy_dst = (kind == 0 ? 0 : kind == 1 ? L::kV : kind == 2 ? L::kPairsK : L::kPairsV) +
                            piece * piece_tokens * row_bytes;
  const int copy_src = (kind & 1) * kv.block_bytes + (kind < 2 ? 0 : kv.page * (D / 2));
  const int copy_bytes = piece_tokens * row_bytes;

  for (int i = blockIdx.x; i < a.batch; i += gridDim.x) {  // sequences without a token have no unit
    const int n = a.lens[i];
    if (threadIdx.x == 0 && (n < 0 || n > a.max_len)) atomicOr(&g_status, kOpsBadPage);
    if (n <= 0)
      for (int c = threadIdx.x; c < a.n_new * a.q_heads * D; c += kWarps * 32) {
        const int tok = c / (a.q_heads * D);
        a.out[(static_cast<int64_t>(i) * a.n_new + tok) * a.out_stride + c - tok * a.q_heads * D] = 0;
      }
  }

  // this CTA's run of rounds, and the sequence b that it starts in
  const int64_t total = rounds_before(a, a.batch, lane) * units_b;
  const int busy = busy_ctas(total, gridDim.x);
  if (static_cast<int>(blockIdx.x) >= busy) return;
  int64_t at = run_start(total, blockIdx.x, busy);
  const int64_t run_end = run_start(total, blockIdx.x + 1, busy);
  int b = 0;
  int64_t before = 0;  // rounds before sequence b
  for (int b0 = 0;; b0 += 32) {
    const int64_t n = b0 + lane < a.batch ? static_cast<int64_t>(rounds_of(a, b0 + lane)) * units_b : 0;
    int64_t sum = n;  // of this lane's sequence and those before it
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(kFull, sum, d);
      if (lane >= d) sum += o;
    }
    const uint32_t past = __ballot_sync(kFull, before + sum > at);
    if (past) {
      const int l = __ffs(past) - 1;
      b = b0 + l;
      before += __shfl_sync(kFull, sum - n, l);
      break;
    }
    before += __shfl_sync(kFull, sum, 31);
  }
  bool first_segment = true;
  for (; at < run_end; first_segment = false) {
  int rounds = rounds_of(a, b);
  while (at >= before + static_cast<int64_t>(rounds) * units_b) {
    before += static_cast<int64_t>(rounds) * units_b;
    rounds = rounds_of(a, ++b);
  }
  const int unit = static_cast<int>((at - before) / rounds);  // of the sequence
  const int round0 = static_cast<int>((at - before) - static_cast<int64_t>(unit) * rounds);
  const int n_rounds = static_cast<int>(min(static_cast<int64_t>(rounds - round0), run_end - at));
  at += n_rounds;
  const int h = unit / a.row_blocks, rb = unit - h * a.row_blocks;
  const int bh = b * kv.heads + h;
  const int r0 = rb * ROWS;
  const int len = clamped_len(a, b);
  const int limmax = max(0, row_limit(a, len, min(r0 + ROWS, a.rows) - 1));  // of the block's last row
  const int tile_end = min((limmax + kTile - 1) / kTile, (round0 + n_rounds) * kWarps);
  int tile = round0 * kWarps + warp;

  const int last_page = max(0, (limmax - 1) >> kv.page_shift);
  const int32_t* table = kv.table + b * kv.table_stride;
  const uint8_t* head = kv.pages + static_cast<int64_t>(2 * h) * kv.block_bytes + copy_src;
  // page number of the lane's piece of tile i (past the end: the last page)
  auto page_of = [&](int i) { return __ldg(table + min((i * kTile + piece * piece_tokens) >> kv.page_shift, last_page)); };
  auto ask = [&](int i, int pid) {
    const int s = filled % kStages;
    const bool ok = pid >= 0 && pid < kv.n_pages;
    const uint32_t okm = __ballot_sync(kFull, ok);
    if (lane == 0) {
      s_ok[warp][s] = okm;
      kernels::mbar_arrive_expect_tx(full_addr + 8 * s, L::kBytes);
    }
    __syncwarp();
    if (copies)
      kernels::bulk_load(ring_addr + s * L::kBytes + copy_dst,
                         head + (ok ? pid : 0) * kv.page_stride + ((i * kTile + piece * piece_tokens) & (kv.page - 1)) * row_bytes,
                         copy_bytes, full_addr + 8 * s);
    ++filled;
  };
  int ahead = tile, pid = 0;  // the next tile to ask for, and its lane's page
  if (ahead < tile_end) pid = page_of(ahead);
  for (int i = 0; i < kStages - 1; ++i)
    if (ahead < tile_end && !dead) {
      ask(ahead, pid);
      ahead += kWarps;
      if (ahead < tile_end) pid = page_of(ahead);
    }

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
        x[j][i] = ops::load16(raw[i], BF);
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

  uint32_t exponent;
  asm volatile("mov.b32 %0, 0x64006400;" : "=r"(exponent));
  const uint32_t rest_mask = t < 2 ? 0u : 0xFFFFE000u;
  const int tau_g = tau(g), tau_v = tau(2 * t), tau_w = tau(2 * t + 1);
  for (; tile < tile_end && !dead; tile += kWarps) {
    if (ahead < tile_end) {
      ask(ahead, pid);
      ahead += kWarps;
      if (ahead < tile_end) pid = page_of(ahead);
    }
    const int stage = used % kStages;
    dead = !__all_sync(kFull, kernels::mbar_wait(full_addr + 8 * stage, (used / kStages) & 1, kWaitLimitNs));
    ++used;
    if (dead) {
      if (lane == 0) atomicOr(&g_status, kOpsTimeout);
      for (; used < filled; ++used)  // the copies in flight land before the CTA goes
        kernels::mbar_wait(full_addr + 8 * (used % kStages), (used / kStages) & 1, kWaitLimitNs);
      break;
    }
    const uint8_t* x = ring + stage * L::kBytes;
    const uint32_t okm = s_ok[warp][stage];
    const int tok0 = tile * kTile + tau_g;  // this lane's tokens: tok0 + 8 n
    const bool bad = okm != kFull;
    if (bad && lane == 0) atomicOr(&g_status, kOpsBadPage);
    const bool edge = (tile + 1) * kTile > lim_min || bad;  // some row does not see all of the tile
    const bool ok[2] = {(okm & 1u) != 0, (okm & 16u) != 0};  // of the tile's first and last 16 tokens
    uint32_t mk[4][NG], mv[4][NG];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      load_words<NG>(mk[n], x + L::kPairsK + (tau_g + 8 * n) * (4 * NG));
      load_words<NG>(mv[n], x + L::kPairsV + (tau_g + 8 * n) * (4 * NG));
    }
    if (edge) {
      // tokens that no row sees may hold anything: their pairs count as zero
#pragma unroll
      for (int n = 0; n < 4; ++n)
        if (!ok[n >> 1] || tok0 + 8 * n >= limmax) {
#pragma unroll
          for (int c = 0; c < NG; ++c) mk[n][c] = mv[n][c] = 0u;
        }
    }

    // S^T: rows g and g + 8 of product `mt` are the lane's tokens 2 mt and 2 mt + 1
    float s[NT][2][4];  // [column][token]
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      float acc[NT][NG][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int n = 0; n < NG; ++n) acc[nt][n][0] = acc[nt][n][1] = acc[nt][n][2] = acc[nt][n][3] = 0.0f;
      uint32_t k0[J], k1[J];
      load_words<J>(k0, x + (tau_g + 16 * mt) * (D / 2) + t * (D / 8));
      load_words<J>(k1, x + (tau_g + 16 * mt + 8) * (D / 2) + t * (D / 8));
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const uint32_t w0 = k0[j], w1 = k1[j];
        const uint32_t a0 = centered<false>(w0, exponent), a1 = centered<false>(w1, exponent), a2 = centered<true>(w0, exponent), a3 = centered<true>(w1, exponent);
        const uint32_t b0 = centered<false>(w0 >> 8, exponent), b1 = centered<false>(w1 >> 8, exponent), b2 = centered<true>(w0 >> 8, exponent),
                       b3 = centered<true>(w1 >> 8, exponent);
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
              const uint32_t w = mk[2 * mt + n][c];
              const float sc = pair_scale<BF>(w);
              const float lo = fmaf(sc, 8.0f, pair_low<BF>(w));
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
            if (!ok[n >> 1] || tok0 + 8 * n >= lim[nt][i]) s[nt][i][n] = -INFINITY;
    }
    if (a.scores && t < 2) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int n = 0; n < 4; ++n)
            a.scores[(static_cast<int64_t>(bh) * a.rows_pad + r0 + 4 * nt + 2 * t + i) * a.score_stride + tok0 + 8 * n] = s[nt][i][n];
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

    // V of contraction steps 2 t and 2 t + 1 (mt, half by half): channels 32 j + 4 g + 0..3
    uint32_t v[4][2][J / 2];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      load_words<J / 2>(v[n][0], x + L::kV + (tau_v + 8 * n) * (D / 2) + g * (D / 16));
      load_words<J / 2>(v[n][1], x + L::kV + (tau_w + 8 * n) * (D / 2) + g * (D / 16));
    }
#pragma unroll
    for (int c = 0; c < NG; ++c) {
      float sv[4], lo[4];
      uint32_t top_s = 0;  // bits of the largest scale, which has no sign
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const uint32_t w = mv[n][c];
        sv[n] = pair_scale<BF>(w);
        lo[n] = fmaf(sv[n], 8.0f, pair_low<BF>(w));
        top_s = max(top_s, w & 0xFFFFu);
      }
      // p s is held as p s 2^(14 - e), e the exponent of the largest finite s so far
      top_s = __reduce_max_sync(kFull, top_s);
      constexpr uint32_t kInf = BF ? 0x7F80u : 0x7C00u;
      if (top_s >= kInf) {
        top_s = 0;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const uint32_t v = mv[n][c] & 0xFFFFu;
          top_s = max(top_s, v < kInf ? v : 0u);
        }
        top_s = __reduce_max_sync(kFull, top_s);
      }
      const int e_new = static_cast<int>(__float_as_uint(pair_scale<BF>(top_s)) >> 23);
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
            const bool hidden = edge && tok0 + 8 * n >= lim[nt][i];  // 0 times a NaN that other rows see
            x[i] = hidden ? 0.0f : s[nt][i][n] * (sv[n] * f);
            lsum[nt][i][c] += hidden ? 0.0f : s[nt][i][n] * lo[n];
            // columns 4..7 take what fp16's 11 bits, cut toward zero, leave
            x[i] -= __uint_as_float(__float_as_uint(x[i]) & rest_mask);
          }
          pf[nt][n] = transpose8x8(pack_half2_rz(x[0], x[1]));
        }
      }
#pragma unroll
      for (int j = c * JG; j < (c + 1) * JG; ++j)
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          constexpr uint32_t kLow = 0x5410u, kHigh = 0x7632u;
          const uint32_t sel = (j & 1) ? kHigh : kLow;
          const uint32_t p0 = __byte_perm(v[2 * mt][0][j / 2], v[2 * mt][1][j / 2], sel);
          const uint32_t p1 = __byte_perm(v[2 * mt + 1][0][j / 2], v[2 * mt + 1][1][j / 2], sel);
          const uint32_t a0 = centered<false>(p0, exponent), a1 = centered<true>(p0, exponent), a2 = centered<false>(p1, exponent), a3 = centered<true>(p1, exponent);
          const uint32_t b0 = centered<false>(p0 >> 8, exponent), b1 = centered<true>(p0 >> 8, exponent), b2 = centered<false>(p1 >> 8, exponent),
                         b3 = centered<true>(p1 >> 8, exponent);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma16816(o[j][0][nt], a0, a1, a2, a3, pf[nt][2 * mt], pf[nt][2 * mt + 1]);
            mma16816(o[j][1][nt], b0, b1, b2, b3, pf[nt][2 * mt], pf[nt][2 * mt + 1]);
          }
        }
    }
    __syncwarp();  // the stage may be filled again
  }
  __syncthreads();  // every ring is idle: the sums take their place

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
  const bool whole = n_rounds == rounds;
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
    if (whole) {
      const int tok = r / a.per;
      a.out[(static_cast<int64_t>(b) * a.n_new + tok) * a.out_stride + (h * a.per + r - tok * a.per) * D + d] =
          ops::store16(den == 0.0f ? 0.0f : sum / den, BF);
      if (a.scores && d == 0) a.unit_ml[static_cast<int64_t>(bh) * a.rows_pad + r] = make_float2(top, den);
    } else {
      const int64_t slot = (2 * static_cast<int64_t>(blockIdx.x) + (first_segment ? 0 : 1)) * ROWS + row;
      a.part_o[slot * D + d] = sum;
      if (d == 0) a.part_ml[slot] = make_float2(top, den);
    }
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // bulk copies will overwrite what was read here
  __syncthreads();
  }
}

// The partial sums of unit `unit` of sequence b: those of CTAs first .. last,
// the first's in slot `slot` and the others' in slot 0. False if one CTA wrote
// the unit out (or there is none).
struct Parts {
  int first, last, slot;
};
__device__ __forceinline__ bool parts_of(const KvAttnArgs& a, int b, int unit, int lane, Parts& p) {
  const int rounds = rounds_of(a, b);
  if (rounds == 0) return false;
  const int units_b = a.kv.heads * a.row_blocks;
  const int64_t total = rounds_before(a, a.batch, lane) * units_b;
  const int64_t lo = rounds_before(a, b, lane) * units_b + static_cast<int64_t>(unit) * rounds, hi = lo + rounds;
  const int busy = busy_ctas(total, a.ctas);
  // CTA c holds round x if run_start(c) <= x < run_start(c + 1): the largest c with total c / busy < x + 1
  auto holder = [&](int64_t x) { return static_cast<int>(((x + 1) * busy - 1) / total); };
  p.first = holder(lo);
  p.last = holder(hi - 1);
  if (p.first == p.last) return false;
  // slot 0 if the unit is the first that the CTA works on
  p.slot = run_start(total, p.first, busy) >= lo ? 0 : 1;
  return true;
}

// Joins the partial sums: CTAs before `n_units` each write the output rows of a
// unit; the others (tracked calls) add the weights exp2(S - lse) of 512 tokens
// of one (sequence, head) to the mass, every element by one thread in one
// order.
template <int D, int ROWS>
__global__ void __launch_bounds__(512) kv_join_kernel(const __grid_constant__ KvAttnArgs a) {
  constexpr int GROUPS = 512 / D;  // partial sums read at a time
  __shared__ float s_sum[GROUPS][D];
  __shared__ float s_lse[STAGQ_KV_MAX_NEW * STAGQ_KV_MAX_SHARE];
  grid_launch_dependents();
  grid_dependency_wait();
  const KvView& kv = a.kv;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n_units = a.batch * kv.heads * a.row_blocks;
  // a row's maximum, and its denominator, over the partial sums of its unit
  auto row_sum = [&](const Parts& p, int row, float& top, float& den) {
    top = -INFINITY;
    for (int c = p.first + lane; c <= p.last; c += 32)
      top = fmaxf(top, a.part_ml[(2 * static_cast<int64_t>(c) + (c == p.first ? p.slot : 0)) * ROWS + row].x);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, d));
    const float base = top == -INFINITY ? 0.0f : top;
    den = 0.0f;
    for (int c = p.first + lane; c <= p.last; c += 32) {
      const float2 ml = a.part_ml[(2 * static_cast<int64_t>(c) + (c == p.first ? p.slot : 0)) * ROWS + row];
      den += ex2(ml.x - base) * ml.y;
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) den += __shfl_xor_sync(kFull, den, d);
  };
  Parts p;
  if (static_cast<int64_t>(blockIdx.x) < static_cast<int64_t>(n_units) * ROWS) {
    const int u = blockIdx.x / ROWS, row = blockIdx.x - u * ROWS;
    const int b = u / (kv.heads * a.row_blocks), unit = u - b * kv.heads * a.row_blocks;
    const int h = unit / a.row_blocks, r = (unit - h * a.row_blocks) * ROWS + row;
    if (r >= a.rows || !parts_of(a, b, unit, lane, p)) return;
    float top, den;
    row_sum(p, row, top, den);
    const float base = top == -INFINITY ? 0.0f : top;
    const int group = threadIdx.x / D, d = threadIdx.x - group * D;
    float sum = 0.0f;
#pragma unroll 4
    for (int c = p.first + group; c <= p.last; c += GROUPS) {
      const int64_t slot = (2 * static_cast<int64_t>(c) + (c == p.first ? p.slot : 0)) * ROWS + row;
      sum += ex2(a.part_ml[slot].x - base) * a.part_o[slot * D + d];
    }
    s_sum[group][d] = sum;
    __syncthreads();
    if (threadIdx.x >= D) return;
#pragma unroll
    for (int i = 1; i < GROUPS; ++i) sum += s_sum[i][d];
    const int tok = r / a.per;
    a.out[(static_cast<int64_t>(b) * a.n_new + tok) * a.out_stride + (h * a.per + r - tok * a.per) * D + d] =
        ops::store16(den == 0.0f ? 0.0f : sum / den, kv.bf16);
    return;
  }
  const int chunks = (a.max_len + 511) / 512;
  const int which = static_cast<int>(blockIdx.x - static_cast<int64_t>(n_units) * ROWS);
  const int bh = which / chunks, tok = (which - bh * chunks) * 512 + threadIdx.x;
  const int b = bh / kv.heads, h = bh - b * kv.heads;
  const int len = clamped_len(a, b);
  if (tok - static_cast<int>(threadIdx.x) >= len) return;
  for (int rb = 0; rb < a.row_blocks; ++rb) {
    const bool parts = parts_of(a, b, h * a.row_blocks + rb, lane, p);
    for (int row = warp; row < ROWS && rb * ROWS + row < a.rows; row += 16) {
      float top, den;
      if (parts) {
        row_sum(p, row, top, den);
      } else {
        const float2 ml = a.unit_ml[static_cast<int64_t>(bh) * a.rows_pad + rb * ROWS + row];
        top = ml.x;
        den = ml.y;
      }
      if (lane == 0) s_lse[rb * ROWS + row] = (top == -INFINITY ? 0.0f : top) + log2f(den);
    }
  }
  __syncthreads();
  if (tok >= len) return;
  const float* scores = a.scores + static_cast<int64_t>(bh) * a.rows_pad * a.score_stride + tok;
  float sum = 0.0f;
#pragma unroll 4
  for (int r = 0; r < a.rows; ++r)
    if (tok < row_limit(a, len, r)) sum += ex2(scores[r * a.score_stride] - s_lse[r]);
  a.mass[b * a.mass_stride_b + h * a.mass_stride_h + tok] += sum;
}

template <int D, int NG, int NT, bool BF>
cudaError_t launch_attention(const KvAttnArgs& a, cudaStream_t s) {
  constexpr int smem = kWarps * kStages * TileLayout<D, NG>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(kv_attention_kernel<D, NG, NT, BF>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  e = launch_op(kv_attention_kernel<D, NG, NT, BF>, dim3(a.ctas), dim3(kWarps * 32), smem, s, a);
  if (e != cudaSuccess || !a.part_o) return e;
  int64_t join = static_cast<int64_t>(a.batch) * a.kv.heads * a.row_blocks * 4 * NT;
  if (a.scores) join += static_cast<int64_t>(a.batch) * a.kv.heads * ((a.max_len + 511) / 512);
  return launch_op(kv_join_kernel<D, 4 * NT>, dim3(static_cast<unsigned>(join)), dim3(512), 0, s, a);
}

template <int D, int NG>
cudaError_t launch_nt(const KvAttnArgs& a, int nt, cudaStream_t s) {
  if (a.kv.bf16) return nt == 1 ? launch_attention<D, NG, 1, true>(a, s) : launch_attention<D, NG, 2, true>(a, s);
  return nt == 1 ? launch_attention<D, NG, 1, false>(a, s) : launch_attention<D, NG, 2, false>(a, s);
}

int64_t align256(int64_t v) { return (v + 255) / 256 * 256; }

}  // namespace

// Four query rows of a KV head per unit, eight where there are more than four
// (the cache is then read once per eight rows). As many CTAs as fit the GPU at
// once, but no more than there can be rounds. Units of one round need no join.
KvAttnPlan plan_kv_attention(int batch, int heads, int q_heads, int n_new, int dim, int max_len, bool mass,
                             int num_sms) {
  KvAttnPlan p{};
  const int rows = q_heads / heads * n_new;
  p.nt = rows <= 4 ? 1 : 2;
  p.row_blocks = (rows + 4 * p.nt - 1) / (4 * p.nt);
  p.rows_pad = p.row_blocks * 4 * p.nt;
  const int64_t units = static_cast<int64_t>(batch) * heads * p.row_blocks;
  const int64_t rounds = (static_cast<int64_t>(max_len) + kWarps * kTile - 1) / (kWarps * kTile);
  const int64_t fit = static_cast<int64_t>(num_sms) * (p.nt == 1 ? 4 : 2);
  p.score_stride = mass ? rounds * kWarps * kTile : 0;
  if (rounds == 1 && !mass) {
    p.ctas = static_cast<int>(units);
    return p;
  }
  p.ctas = static_cast<int>(units * rounds < fit ? units * rounds : fit);
  const int64_t slots = 2 * static_cast<int64_t>(p.ctas) * 4 * p.nt;
  p.off_ml = 0;
  p.off_o = align256(slots * 8);
  p.off_unit = p.off_o + align256(slots * dim * 4);
  const int64_t rows_all = static_cast<int64_t>(batch) * heads * p.rows_pad;
  p.off_scores = p.off_unit + (mass ? align256(rows_all * 8) : 0);
  p.bytes = p.off_scores + align256(rows_all * p.score_stride * 4);
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
