// Attention of each sequence's newest tokens over its 4-bit cache.
//
//   S_t = scale q . K_t,  p = softmax over the visible t,  out = sum_t p_t V_t
//   K_t = lo + s u (per group of channels), V_t likewise, u = 0..15
//
// so a group's share of S_t is scale (s sum q u + lo sum q), and of out
// sum_t (p_t s_t) u_t + sum_t p_t lo_t: the matrix products only ever see the
// codes u and never a rebuilt K or V.
//
// The cache's bytes would bound it if the unpacking kept up: at 6.5 TB/s an SM
// takes in about 49 codes per clock. Measured, long sequences stream 3.4 TB/s:
// issue slots 58 % and the ALU pipe 55 % busy, no unit full, 12 warps per SM
// that each wait on their own chain of steps. What keeps the instruction count
// near one per two codes:
//  - V: two codes are masked out of a word in place and OR'ed under the exponent
//    of 1024 in one operation; a packed subtraction leaves u - 8 (16 times that
//    for the upper 4 bits of a byte) as exact fp16, and lo + 8 s replaces lo.
//    The sums over the tokens then stay small: with u itself, whose mean is
//    7.5, the result was 4e-4 off at 67000 tokens (fp16 rounds by 2e-4).
//  - K: the same bits without the OR are fp16 subnormals, 16 u 2^-24, exact
//    too, and mma takes them at full rate; nothing needs to be subtracted. It
//    aligns products by their nominal exponents, which drops what lies below
//    2^-18 of the row's largest q. For q of even size that is less than the
//    rounding of s q u + lo q adds (weights off by 7e-7); where one channel is
//    2^10 times the others and more, weights were off by 2.4e-5, against 4e-6
//    for the same sums without the drop.
//  - The order of a contraction is free, so the packed order of a row is the
//    order of the mma fragments (kv_cache.cu): a lane's K words feed its
//    A fragments without a shuffle, and two tokens' V words give the pairs of
//    the second product with one byte permute per 4 pairs.
//  - Tokens are the 16 rows of the first product and the contraction of the
//    second, query rows the 8 columns: S^T = K q^T and out^T = V^T p^T.
//  - Of the 8 columns 4 are query rows and 4 repeat them: in the second
//    product the repeats carry what rounding p s to fp16 lost, at no extra mma
//    for up to 4 query rows per KV head (32 / 8 and 40 / 10 heads). Together
//    the parts hold 22 bits of p s above 2^-9 of the largest scale s that the
//    row has met in the group, and below that all but 2^-30 of that scale per
//    token (and no more than 2^-22 of its largest p s, where that is less). The
//    scaling is each row's own: a token that a row does not see, or hardly,
//    may have any V.
// The tcgen05 tensor cores would need the codes expanded to 8 or 16 bits in
// shared memory first, 2 to 4 times the cache's bytes of shared-memory writes
// and reads, for products that mma.sync does within the bytes' time.
//
// A warp takes 32 tokens at a time. Each has a ring of tiles in shared memory
// of its own, filled by bulk copies (4 per tile, one per lane, 8 where a page
// holds half a tile) one tile ahead: no registers wait for memory, so 12
// warps of 168 registers fit an SM. The four warps of a CTA take tiles in turn and join their sums at
// the end; nothing in the loop waits for another warp.
//
// The work is cut into rounds of 128 tokens (a tile per warp) of a unit
// (sequence, KV head, block of query rows). Two ways to share it, chosen from
// the sizes (plan_kv_attention):
//  - A cluster of up to 8 CTAs per unit, an equal part of its rounds each, that
//    joins its sums through distributed shared memory: one launch, for calls
//    of little work.
//  - As many CTAs as fit the GPU. The rounds are numbered unit after unit and
//    every CTA takes an equal run of the numbering, read off the lengths on the
//    device, so that a ragged batch, one long sequence and many short ones fill
//    the GPU alike. A unit that one CTA covers is written out; the others leave
//    a partial sum (at most two per CTA), and a second kernel joins those.
#include <algorithm>
#include <cmath>

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
constexpr int kMaxCluster = 8;
constexpr int kMassTokens = 2048;   // tokens of a CTA of the join that adds to the mass

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

// Both products by one instruction.
__device__ __forceinline__ void mul2(float& x, float& y, float a, float b) {
  asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\t"
      "mul.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}

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

// CTAs of an SM: 168 registers a thread for 4 query rows, 255 for 8. (With 128
// registers 4 CTAs fit and one group per head does not spill, but 16 ragged
// sequences up to 8192 tokens then took 33.1 us instead of 31.9: the runs of
// tiles are shorter against what starts and ends them.)
constexpr int resident_ctas(int nt) { return nt > 1 ? 2 : 3; }

constexpr int kStages = 2;
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
// How `total` rounds (positive) are dealt to the CTAs: runs of `base` rounds,
// the first `rem` CTAs one more; CTAs from `busy` on get none.
struct Runs {
  int base, rem, busy;
  __device__ Runs(int total, int ctas) {
    busy = min(total, ctas);
    base = total / busy;
    rem = total - base * busy;
  }
  __device__ int start(int c) const { return c * base + min(c, rem); }
  // the CTA whose run holds round x
  __device__ int holder(int x) const {
    const int longer = rem * (base + 1);
    return x < longer ? x / (base + 1) : rem + (x - longer) / base;
  }
};

__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive;\n\tbarrier.cluster.wait;" ::: "memory");
}
__device__ __forceinline__ float load_peer(uint32_t addr, uint32_t rank) {
  uint32_t peer;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(peer) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(peer) : "memory");
  return v;
}

__device__ __forceinline__ float4 load_peer4(uint32_t addr, uint32_t rank) {
  uint32_t peer;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(peer) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(peer) : "memory");
  return v;
}

template <int D, int NG, int NT, bool BF>
__global__ void __launch_bounds__(kWarps * 32, resident_ctas(NT)) kv_attention_kernel(const __grid_constant__ KvAttnArgs a) {
  constexpr int J = D / 32;       // blocks of 32 channels
  constexpr int JG = J / NG;      // blocks of a group
  constexpr int ROWS = 4 * NT;
  using L = TileLayout<D, NG>;
  static_assert(kStages * L::kBytes >= 2 * ROWS * D * 4, "the warps' sums take the rings' place");
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_m[kWarps][ROWS], s_l[kWarps][ROWS];
  __shared__ __align__(8) uint64_t s_full[kWarps][kStages + 1];  // the last: nothing completes it (test hook)
  __shared__ uint32_t s_ok[kWarps][kStages];  // by lane: whether its piece's page is in the pool
  __shared__ float s_top[ROWS], s_den[ROWS];  // of the CTA, for its cluster
  __shared__ __align__(16) uint16_t s_q[ROWS][D];
  __shared__ float s_cf[ROWS], s_qs[ROWS][NG];
  float (*s_o)[2 * ROWS][D] = reinterpret_cast<float (*)[2 * ROWS][D]>(smem);  // 8 columns for 4 rows

  grid_launch_dependents();
  grid_dependency_wait();
  const KvView& kv = a.kv;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int units_b = kv.heads * a.row_blocks;  // units of a sequence

  uint8_t* ring = smem + warp * (kStages * L::kBytes);
  const uint32_t ring_addr = kernels::smem_addr(ring), full_addr = kernels::smem_addr(&s_full[warp][0]);
  if (lane <= kStages) kernels::mbar_init(full_addr + 8 * lane, 1);
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

  int at = 0, run_end = 1;  // this CTA's run of rounds; with clusters: one pass
  int b = 0, before = 0;    // the sequence of round `at`, and the rounds before it
  Runs runs(1, 1);
  if (a.cluster == 0) {
    for (int i = blockIdx.x; i < a.batch; i += gridDim.x) {  // sequences without a token have no unit
      const int n = a.lens[i];
      if (threadIdx.x == 0 && (n < 0 || n > a.max_len)) atomicOr(&g_status, kOpsBadPage);
      if (n <= 0)
        for (int c = threadIdx.x; c < a.n_new * a.q_heads * D; c += kWarps * 32) {
          const int tok = c / (a.q_heads * D);
          a.out[(static_cast<int64_t>(i) * a.n_new + tok) * a.out_stride + c - tok * a.q_heads * D] = 0;
        }
    }
    int total = 0;
    for (int i = lane; i < a.batch; i += 32) total += rounds_of(a, i) * units_b;
    total = __reduce_add_sync(kFull, total);
    if (total == 0) return;
    runs = Runs(total, gridDim.x);
    if (static_cast<int>(blockIdx.x) >= runs.busy) return;
    at = runs.start(blockIdx.x);
    run_end = runs.start(blockIdx.x + 1);
    for (int b0 = 0;; b0 += 32) {
      const int n = b0 + lane < a.batch ? rounds_of(a, b0 + lane) * units_b : 0;
      int sum = n;  // of this lane's sequence and those before it
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(kFull, sum, d);
        if (lane >= d) sum += o;
      }
      const uint32_t past = __ballot_sync(kFull, before + sum > at);
      if (b0 >= a.batch) return;
      if (past) {
        const int l = __ffs(past) - 1;
        b = b0 + l;
        before += __shfl_sync(kFull, sum - n, l);
        break;
      }
      before += __shfl_sync(kFull, sum, 31);
    }
  }
  bool first_segment = true;
  for (; at < run_end; first_segment = false) {
  int rounds, unit, round0, n_rounds, part = 0;
  if (a.cluster == 0) {
    rounds = rounds_of(a, b);
    while (at >= before + rounds * units_b) {
      before += rounds * units_b;
      if (++b >= a.batch) return;  // here and below: lengths that changed under the call write nothing out of bounds
      rounds = rounds_of(a, b);
    }
    unit = (at - before) / rounds;  // of the sequence
    if (unit >= units_b) return;
    round0 = at - before - unit * rounds;
    n_rounds = min(rounds - round0, run_end - at);
    if (round0 == 0 && threadIdx.x == 0 && a.part_o)  // where the join finds the unit's partial sums
      a.parts[b * units_b + unit] = make_int4(blockIdx.x, runs.holder(at + rounds - 1), first_segment ? 0 : 1, 0);
    at += n_rounds;
  } else {
    unit = blockIdx.x / a.cluster;
    part = blockIdx.x - unit * a.cluster;
    b = unit / units_b;
    unit -= b * units_b;
    if (threadIdx.x == 0 && (a.lens[b] < 0 || a.lens[b] > a.max_len)) atomicOr(&g_status, kOpsBadPage);
    rounds = rounds_of(a, b);
    round0 = rounds * part / a.cluster;
    n_rounds = rounds * (part + 1) / a.cluster - round0;
    at = run_end;
  }
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
  auto page_of = [&](int i) { return table[min((i * kTile + piece * piece_tokens) >> kv.page_shift, last_page)]; };
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
                         head + static_cast<uint64_t>(static_cast<uint32_t>(ok ? pid : 0)) * kv.page_stride + ((i * kTile + piece * piece_tokens) & (kv.page - 1)) * row_bytes,
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
  // in [2^10, 2^11): exact for fp16 and bf16 alike, down to values 2^-24 of the
  // row's largest. A warp takes a row, a lane one channel of each 32; each
  // eight channels lie in the order of the fragments: 0, 4, 1, 5, 2, 6, 3, 7.
#pragma unroll
  for (int row = warp; row < ROWS; row += kWarps) {
    const int r = r0 + row, tok = r / a.per;
    const uint16_t* q = a.q + (static_cast<int64_t>(b) * a.n_new + tok) * a.q_stride + (h * a.per + r - tok * a.per) * D;
    float x[J], sum[NG];
    uint32_t top = 0;  // bits of the largest magnitude
#pragma unroll
    for (int j = 0; j < J; ++j) {
      x[j] = r < a.rows ? ops::load16(q[32 * j + lane], BF) : 0.0f;
      top = max(top, __float_as_uint(x[j]) & 0x7FFFFFFFu);
    }
    top = __reduce_max_sync(kFull, top);
    const bool fine = top < 0x7F800000u;
    const int e = fine && top ? max(-126, static_cast<int>(top >> 23) - 127 - 10) : 0;
    const float down = fine ? pow2(-e) : 0.0f;
#pragma unroll
    for (int n = 0; n < NG; ++n) sum[n] = 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      x[j] = fine ? x[j] * down : 0.0f;
      sum[j / JG] += x[j];
      s_q[row][32 * j + (lane & ~7) + 2 * (lane & 3) + ((lane >> 2) & 1)] = __half_as_ushort(__float2half_rn(x[j]));
    }
#pragma unroll
    for (int n = 0; n < NG; ++n)
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) sum[n] += __shfl_xor_sync(kFull, sum[n], d);
    if (lane == 0) {
      const float c = fine ? a.scale_log2 * pow2(e) : __uint_as_float(0x7FC00000u);
      s_cf[row] = c;
#pragma unroll
      for (int n = 0; n < NG; ++n) s_qs[row][n] = sum[n] * c;
    }
  }
  __syncthreads();
  uint32_t qf[NT][J][4];
  float cf[NT][2], qs[NT][2][NG];  // softmax scale of a column, and that times its sums of q
  int lim[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int j = 0; j < J; ++j) load_words<4>(qf[nt][j], reinterpret_cast<const uint8_t*>(&s_q[4 * nt + (g & 3)][32 * j + 8 * t]));
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // this lane's columns 2 t + i are rows (2 t + i) mod 4 of the tile
      const int row = 4 * nt + ((2 * t + i) & 3);
      cf[nt][i] = s_cf[row] * 1048576.0f;  // codes count as 2^-20
#pragma unroll
      for (int n = 0; n < NG; ++n) qs[nt][i][n] = s_qs[row][n];
      lim[nt][i] = r0 + row < a.rows ? row_limit(a, len, r0 + row) : limmax;
    }
  }
  int lim_min = lim[0][0];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) lim_min = min(lim_min, min(lim[nt][0], lim[nt][1]));
  lim_min = __reduce_min_sync(kFull, lim_min);

  float o[J][2][NT][4];
  float m[NT][2], l[NT][2], lsum[NT][2][NG];
  float fit[NT][2][NG];          // what p s is scaled by, 2^118 at most
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      m[nt][i] = -INFINITY;
      l[nt][i] = 0.0f;
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        lsum[nt][i][n] = 0.0f;
        fit[nt][i][n] = pow2(118);
      }
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
  auto give_up = [&]() {
    dead = true;
    if (lane == 0) atomicOr(&g_status, kOpsTimeout);
    for (; used < filled; ++used)  // the copies in flight land before the sums take their place
      kernels::mbar_wait(full_addr + 8 * (used % kStages), (used / kStages) & 1, kWaitLimitNs);
  };
  if (__builtin_expect(a.stall_ns != 0, 0) && tile < tile_end && !dead &&  // test hook
      !__all_sync(kFull, kernels::mbar_wait(full_addr + 8 * kStages, 0, a.stall_ns)))
    give_up();
  for (; tile < tile_end && !dead; tile += kWarps) {
    if (ahead < tile_end) {
      ask(ahead, pid);
      ahead += kWarps;
      if (ahead < tile_end) pid = page_of(ahead);
    }
    const int stage = used % kStages;
    if (!__all_sync(kFull, kernels::mbar_wait(full_addr + 8 * stage, (used / kStages) & 1, kWaitLimitNs))) {
      give_up();
      break;
    }
    ++used;
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
    float acc[2][NT][NG][4];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int n = 0; n < NG; ++n) acc[mt][nt][n][0] = acc[mt][nt][n][1] = acc[mt][nt][n][2] = acc[mt][nt][n][3] = 0.0f;
      uint32_t k0[J], k1[J];
      load_words<J>(k0, x + (tau_g + 16 * mt) * (D / 2) + t * (D / 8));
      load_words<J>(k1, x + (tau_g + 16 * mt + 8) * (D / 2) + t * (D / 8));
#pragma unroll
      for (int j = 0; j < J; ++j) {
        constexpr uint32_t M = 0x00F000F0u;
        const uint32_t a0 = (k0[j] << 4) & M, a1 = (k1[j] << 4) & M, a2 = k0[j] & M, a3 = k1[j] & M;
        const uint32_t b0 = (k0[j] >> 4) & M, b1 = (k1[j] >> 4) & M, b2 = (k0[j] >> 8) & M, b3 = (k1[j] >> 8) & M;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma16816(acc[mt][nt][j / JG], a0, a1, a2, a3, qf[nt][j][0], qf[nt][j][1]);
          mma16816(acc[mt][nt][j / JG], b0, b1, b2, b3, qf[nt][j][2], qf[nt][j][3]);
        }
      }
    }
    // scores less the reference m of their row, in powers of two
    float s[NT][2][4];  // [column][token]
    auto score = [&](const float (&ref)[NT][2]) {
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int c = 0; c < NG; ++c) {
          const float sc = pair_scale<BF>(mk[n][c]), lo = pair_low<BF>(mk[n][c]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              s[nt][i][n] = fmaf(acc[n >> 1][nt][c][2 * (n & 1) + i], sc * cf[nt][i],
                                 fmaf(lo, qs[nt][i][c], c == 0 ? -ref[nt][i] : s[nt][i][n]));
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
    };
    score(m);
    // The reference is no maximum: it follows only when a score exceeds it by
    // 2^8 (from -inf, the start, any score does), so p is below 2^8 and most
    // tiles need no reduction over the warp and no rescaling.
    bool rises = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        rises = rises || fmaxf(fmaxf(s[nt][i][0], s[nt][i][1]), fmaxf(s[nt][i][2], s[nt][i][3])) > 8.0f;
    if (__any_sync(kFull, rises)) {
      float zero[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) zero[nt][0] = zero[nt][1] = 0.0f;
      score(zero);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float x = fmaxf(fmaxf(s[nt][i][0], s[nt][i][1]), fmaxf(s[nt][i][2], s[nt][i][3]));
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, d));
          const float top = fmaxf(m[nt][i], x);
          const float f = top > m[nt][i] ? ex2(m[nt][i] - top) : 1.0f;  // the first time: 0
          m[nt][i] = top;
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
      float ref[NT][2];  // a row that has seen nothing yet: all its scores are -inf
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) ref[nt][i] = m[nt][i] == -INFINITY ? 0.0f : m[nt][i];
      score(ref);
    }
    if (a.scores && t < 2) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int n = 0; n < 4; ++n)
            a.scores[(static_cast<int64_t>(bh) * a.rows_pad + r0 + 4 * nt + 2 * t + i) * a.score_stride + tok0 + 8 * n] =
                s[nt][i][n] + (m[nt][i] == -INFINITY ? 0.0f : m[nt][i]);
    }

#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          s[nt][i][n] = ex2(s[nt][i][n]);
          l[nt][i] += s[nt][i][n];
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
      // A row's p s is held as p s 2^(6 - e), where s < 2^(e + 1) for the scales
      // that it has met: below 2^15, for p is below 2^8. When an s is larger, e
      // follows, of the rows that see the token, and no further than 2^8 past the
      // row's largest p s: a token of small weight costs the others no bits.
      float sv[4], lo[4], fit_top = 0.0f;
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        sv[n] = pair_scale<BF>(mv[n][c]);
        lo[n] = fmaf(sv[n], 8.0f, pair_low<BF>(mv[n][c]));
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) fit_top = fmaxf(fit_top, fmaxf(fit[nt][0][c], fit[nt][1][c]));
      const float large = fmaxf(fmaxf(sv[0], sv[1]), fmaxf(sv[2], sv[3])) * fit_top;
      if (__any_sync(kFull, large >= 128.0f)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            constexpr uint32_t kInf = 0x7F800000u;
            uint32_t top_s = 0, top_ps = 0;  // bits of the row's largest s and p s
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              const uint32_t of_s = __float_as_uint(fabsf(sv[n])), of_ps = __float_as_uint(fabsf(s[nt][i][n] * sv[n]));
              if (of_s >= kInf || (edge && tok0 + 8 * n >= lim[nt][i])) continue;
              top_s = max(top_s, of_s);
              top_ps = max(top_ps, of_ps < kInf ? of_ps : of_s);
            }
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) {
              top_s = max(top_s, __shfl_xor_sync(kFull, top_s, d));
              top_ps = max(top_ps, __shfl_xor_sync(kFull, top_ps, d));
            }
            const int e = 260 - static_cast<int>(__float_as_uint(fit[nt][i][c]) >> 23);
            const int e_new = min(static_cast<int>(top_s >> 23), static_cast<int>(top_ps >> 23) + 8);
            if (e_new > e) {  // the same in all lanes of the row
              const float down = e_new - e > 126 ? 0.0f : pow2(e - e_new);
#pragma unroll
              for (int j = c * JG; j < (c + 1) * JG; ++j) {
                o[j][0][nt][i] *= down;
                o[j][0][nt][2 + i] *= down;
                o[j][1][nt][i] *= down;
                o[j][1][nt][2 + i] *= down;
              }
              fit[nt][i][c] = __uint_as_float(static_cast<uint32_t>(260 - e_new) << 23);
            }
          }
      }
      uint32_t pf[NT][4];  // B fragments of both products, k = token
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          float x[2] = {s[nt][0][n], s[nt][1][n]};
          mul2(x[0], x[1], fit[nt][0][c], fit[nt][1][c]);  // finite whatever s is
          mul2(x[0], x[1], sv[n], sv[n]);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const bool hidden = edge && tok0 + 8 * n >= lim[nt][i];  // 0 times a NaN that other rows see
            if (hidden) x[i] = 0.0f;
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

  // the warp's sums to shared memory, in natural units: columns 4..7 of four
  // rows hold what their rounding left, and the lowest values' part is theirs too
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
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const float up = __uint_as_float((254u << 23) - __float_as_uint(fit[nt][i][j / JG]));  // 1 / fit
        const float up16 = up * 0.0625f, low = t < 2 ? 0.0f : lsum[nt][i][j / JG];
        *reinterpret_cast<float4*>(&s_o[warp][8 * nt + 2 * t + i][32 * j + 4 * g]) =
            make_float4(fmaf(o[j][0][nt][i], up, low), fmaf(o[j][0][nt][2 + i], up16, low), fmaf(o[j][1][nt][i], up, low),
                        fmaf(o[j][1][nt][2 + i], up16, low));
      }
      if (t < 2 && g == 0) {
        s_m[warp][4 * nt + 2 * t + i] = m[nt][i];
        s_l[warp][4 * nt + 2 * t + i] = l[nt][i];
      }
    }
  __syncthreads();
  const bool whole = n_rounds == rounds;
  const bool direct = a.cluster == 0 ? whole : a.cluster == 1;
  auto put = [&](int r, int d, float4 sum, float den) {  // 4 channels from d on
    const int tok = r / a.per;
    uint16_t* out = a.out + (static_cast<int64_t>(b) * a.n_new + tok) * a.out_stride + (h * a.per + r - tok * a.per) * D + d;
    const float f = den == 0.0f ? 0.0f : 1.0f / den;
    const uint32_t y[2] = {ops::store16x2(sum.x * f, sum.y * f, BF), ops::store16x2(sum.z * f, sum.w * f, BF)};
    if (a.vec_out) {
      *reinterpret_cast<uint2*>(out) = make_uint2(y[0], y[1]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) out[i] = static_cast<uint16_t>(y[i >> 1] >> (16 * (i & 1)));
    }
  };
  for (int idx = threadIdx.x; idx < ROWS * D / 4; idx += kWarps * 32) {
    const int row = idx / (D / 4), d = 4 * (idx - row * (D / 4)), r = r0 + row;
    const int col = 8 * (row >> 2) + (row & 3);
    float top = s_m[0][row];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_m[w][row]);
    const float base = top == -INFINITY ? 0.0f : top;
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float den = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = ex2(s_m[w][row] - base);
      const float4 hi = *reinterpret_cast<const float4*>(&s_o[w][col][d]), lo = *reinterpret_cast<const float4*>(&s_o[w][col + 4][d]);
      sum.x = fmaf(f, hi.x + lo.x, sum.x);
      sum.y = fmaf(f, hi.y + lo.y, sum.y);
      sum.z = fmaf(f, hi.z + lo.z, sum.z);
      sum.w = fmaf(f, hi.w + lo.w, sum.w);
      den = fmaf(f, s_l[w][row], den);
    }
    if (direct) {
      if (r < a.rows) {
        put(r, d, sum, den);
        if (a.scores && d == 0) a.unit_ml[static_cast<int64_t>(bh) * a.rows_pad + r] = make_float2(top, den);
      }
    } else if (a.cluster == 0) {
      const int slot = (2 * blockIdx.x + (first_segment ? 0 : 1)) * ROWS + row;
      *reinterpret_cast<float4*>(a.part_o + static_cast<int64_t>(slot) * D + d) = sum;
      if (d == 0) a.part_ml[slot] = make_float2(top, den);
    } else {
      *reinterpret_cast<float4*>(&s_o[0][col][d]) = sum;  // this thread alone reads and writes these elements
      if (d == 0) {
        s_top[row] = top;
        s_den[row] = den;
      }
    }
  }
  if (a.cluster > 1) {
    cluster_sync_all();
    const uint32_t o_addr = kernels::smem_addr(&s_o[0][0][0]), top_addr = kernels::smem_addr(s_top), den_addr = kernels::smem_addr(s_den);
    for (int idx = threadIdx.x * a.cluster + part; idx < ROWS * D / 4; idx += a.cluster * kWarps * 32) {
      const int row = idx / (D / 4), d = 4 * (idx - row * (D / 4));
      if (r0 + row >= a.rows) continue;
      const uint32_t at_o = o_addr + 4 * ((8 * (row >> 2) + (row & 3)) * D + d);
      float m_p[kMaxCluster], l_p[kMaxCluster], top = -INFINITY;
      float4 o_p[kMaxCluster];
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) {
        m_p[c] = -INFINITY;
        l_p[c] = 0.0f;
        o_p[c] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (c < a.cluster) {
          m_p[c] = load_peer(top_addr + 4 * row, c);
          l_p[c] = load_peer(den_addr + 4 * row, c);
          o_p[c] = load_peer4(at_o, c);
        }
        top = fmaxf(top, m_p[c]);
      }
      const float base = top == -INFINITY ? 0.0f : top;
      float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float den = 0.0f;
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) {
        const float f = ex2(m_p[c] - base);
        sum.x = fmaf(f, o_p[c].x, sum.x);
        sum.y = fmaf(f, o_p[c].y, sum.y);
        sum.z = fmaf(f, o_p[c].z, sum.z);
        sum.w = fmaf(f, o_p[c].w, sum.w);
        den = fmaf(f, l_p[c], den);
      }
      put(r0 + row, d, sum, den);
    }
    cluster_sync_all();  // no CTA leaves while a peer reads its sums
    return;
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // bulk copies will overwrite what was read here
  __syncthreads();
  }
}

// Joins the partial sums: CTAs before n_units * ROWS each write one output row;
// the others (tracked calls) add the weights exp2(S - lse) of kMassTokens tokens
// of one (sequence, head) to the mass, every element by one thread in one order.
template <int D, int ROWS>
__global__ void __launch_bounds__(512) kv_join_kernel(const __grid_constant__ KvAttnArgs a) {
  constexpr int GROUPS = 512 / D;  // partial sums read at a time
  __shared__ float s_sum[GROUPS][D], s_top[GROUPS], s_den[GROUPS];
  __shared__ float s_lse[STAGQ_KV_MAX_NEW * STAGQ_KV_MAX_SHARE];
  grid_launch_dependents();
  grid_dependency_wait();
  const KvView& kv = a.kv;
  const int units_b = kv.heads * a.row_blocks, n_units = a.batch * units_b;
  // slot of row `row` in CTA c's partial sum of a unit
  auto slot_of = [&](const int4& p, int c, int row) { return (2 * c + (c == p.x ? p.z : 0)) * ROWS + row; };
  if (static_cast<int64_t>(blockIdx.x) < static_cast<int64_t>(n_units) * ROWS) {
    const int u = blockIdx.x / ROWS, row = blockIdx.x - u * ROWS;
    const int b = u / units_b, unit = u - b * units_b;
    const int h = unit / a.row_blocks, r = (unit - h * a.row_blocks) * ROWS + row;
    if (r >= a.rows || a.lens[b] <= 0) return;
    const int4 p = a.parts[u];
    if (p.x == p.y || p.x < 0 || p.x > p.y || p.y >= a.ctas) return;  // one CTA wrote the unit out
    const int group = threadIdx.x / D, d = threadIdx.x - group * D;
    float top = -INFINITY, den = 0.0f, sum = 0.0f;
    for (int c0 = p.x + group; c0 <= p.y; c0 += 4 * GROUPS) {
      float2 ml[4];
      float o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = c0 + i * GROUPS;
        ml[i] = make_float2(-INFINITY, 0.0f);
        o[i] = 0.0f;
        if (c <= p.y) {
          const int slot = slot_of(p, c, row);
          ml[i] = a.part_ml[slot];
          o[i] = a.part_o[static_cast<int64_t>(slot) * D + d];
        }
      }
      const float now = fmaxf(fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)), top);
      const float base = now == -INFINITY ? 0.0f : now, f = ex2(top - base);
      sum *= f;
      den *= f;
      top = now;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float w = ex2(ml[i].x - base);
        sum += w * o[i];
        den += w * ml[i].y;
      }
    }
    s_sum[group][d] = sum;
    if (d == 0) {
      s_top[group] = top;
      s_den[group] = den;
    }
    __syncthreads();
    if (threadIdx.x >= D) return;
    top = s_top[0];
#pragma unroll
    for (int i = 1; i < GROUPS; ++i) top = fmaxf(top, s_top[i]);
    const float base = top == -INFINITY ? 0.0f : top;
    sum = den = 0.0f;
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) {
      const float w = ex2(s_top[i] - base);
      sum += w * s_sum[i][d];
      den += w * s_den[i];
    }
    const int tok = r / a.per;
    a.out[(static_cast<int64_t>(b) * a.n_new + tok) * a.out_stride + (h * a.per + r - tok * a.per) * D + d] =
        ops::store16(den == 0.0f ? 0.0f : sum / den, kv.bf16);
    return;
  }
  const int chunks = (a.max_len + kMassTokens - 1) / kMassTokens;
  const int which = static_cast<int>(blockIdx.x - static_cast<int64_t>(n_units) * ROWS);
  const int bh = which / chunks, t0 = (which - bh * chunks) * kMassTokens;
  const int b = bh / kv.heads, h = bh - b * kv.heads;
  const int len = clamped_len(a, b);
  if (t0 >= len) return;
  // a thread's tokens: t0 + threadIdx.x + 512 i. Four rows' scores, the first
  // of them while the rows' denominators are found.
  constexpr int PER = kMassTokens / 512;
  const float* scores = a.scores + static_cast<int64_t>(bh) * a.rows_pad * a.score_stride + t0 + threadIdx.x;
  float s[4][PER], sum[PER], old[PER];
  auto load_rows = [&](int r0) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int limit = r0 + r < a.rows ? row_limit(a, len, r0 + r) : 0;
#pragma unroll
      for (int i = 0; i < PER; ++i)
        s[r][i] = t0 + static_cast<int>(threadIdx.x) + 512 * i < limit ? scores[(r0 + r) * a.score_stride + 512 * i] : -INFINITY;
    }
  };
  load_rows(0);
  float* mass = a.mass + b * a.mass_stride_b + h * a.mass_stride_h + t0 + threadIdx.x;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    old[i] = t0 + static_cast<int>(threadIdx.x) + 512 * i < len ? mass[512 * i] : 0.0f;
    sum[i] = 0.0f;
  }
  const int lane = threadIdx.x & 31;
  for (int r = threadIdx.x >> 5; r < a.rows; r += 16) {
    const int rb = r / ROWS, row = r - rb * ROWS;
    int4 p = a.parts[b * units_b + h * a.row_blocks + rb];
    if (p.x < 0 || p.x > p.y || p.y >= a.ctas) p.x = p.y;  // not a record: the lengths changed under the call
    float top, den;
    if (p.x == p.y) {
      const float2 ml = a.unit_ml[static_cast<int64_t>(bh) * a.rows_pad + r];
      top = ml.x;
      den = ml.y;
    } else {
      top = -INFINITY;
      den = 0.0f;
      for (int c = p.x + lane; c <= p.y; c += 32) {
        const float2 ml = a.part_ml[slot_of(p, c, row)];
        const float now = fmaxf(top, ml.x), base = now == -INFINITY ? 0.0f : now;
        den = den * ex2(top - base) + ml.y * ex2(ml.x - base);
        top = now;
      }
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const float t2 = __shfl_xor_sync(kFull, top, d), d2 = __shfl_xor_sync(kFull, den, d);
        const float now = fmaxf(top, t2), base = now == -INFINITY ? 0.0f : now;
        den = den * ex2(top - base) + d2 * ex2(t2 - base);
        top = now;
      }
    }
    // (a row that sees nothing: its scores are all -inf, whatever stands here)
    if (lane == 0) s_lse[r] = den == 0.0f ? 0.0f : (top == -INFINITY ? 0.0f : top) + log2f(den);
  }
  __syncthreads();
  for (int r0 = 0; r0 < a.rows; r0 += 4) {
    if (r0) load_rows(r0);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float lse = s_lse[min(r0 + r, a.rows - 1)];
#pragma unroll
      for (int i = 0; i < PER; ++i)  // a token that the row does not see stays out of a row whose lse is NaN
        sum[i] += s[r][i] == -INFINITY ? 0.0f : ex2(s[r][i] - lse);
    }
  }
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (t0 + static_cast<int>(threadIdx.x) + 512 * i < len) mass[512 * i] = old[i] + sum[i];
}

template <int D, int NG, int NT, bool BF>
cudaError_t launch_attention(const KvAttnArgs& a, cudaStream_t s) {
  constexpr int smem = kWarps * kStages * TileLayout<D, NG>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(kv_attention_kernel<D, NG, NT, BF>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.ctas);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.cluster > 1 ? a.cluster : 1;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.cluster > 1 ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kv_attention_kernel<D, NG, NT, BF>, a);
  if (e != cudaSuccess || !a.part_o) return e;
  int64_t join = static_cast<int64_t>(a.batch) * a.kv.heads * a.row_blocks * 4 * NT;
  if (a.scores) join += static_cast<int64_t>(a.batch) * a.kv.heads * ((a.max_len + kMassTokens - 1) / kMassTokens);
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
// (the cache is then read once per eight rows). A round takes about 1.4 us in a
// CTA that has its SM to itself and 2.2 us where all of them are full. Clusters
// of S CTAs per unit (S up to 8, no more than the rounds, all resident at once
// where that goes) take ceil(rounds / S) rounds after one another, of the
// longest sequence; the even split takes an equal share of all rounds (of a
// batch, about 0.6 times the longest sequence's each), and a second launch of
// about 5 us.
KvAttnPlan plan_kv_attention(int batch, int heads, int q_heads, int n_new, int dim, int max_len, bool mass,
                             int num_sms) {
  KvAttnPlan p{};
  const int rows = q_heads / heads * n_new;
  p.nt = rows <= 4 ? 1 : 2;
  p.row_blocks = (rows + 4 * p.nt - 1) / (4 * p.nt);
  p.rows_pad = p.row_blocks * 4 * p.nt;
  const int64_t units = static_cast<int64_t>(batch) * heads * p.row_blocks;
  const int64_t rounds = (static_cast<int64_t>(max_len) + kWarps * kTile - 1) / (kWarps * kTile);
  const int64_t fit = static_cast<int64_t>(num_sms) * resident_ctas(p.nt);
  p.score_stride = mass ? rounds * kWarps * kTile : 0;
  if (!mass) {
    int64_t s = 1;
    while (s < kMaxCluster && s < rounds && units * s * 2 <= fit) s *= 2;
    auto round_us = [&](int64_t ctas) { return std::max(1.4, 2.2 * std::min<int64_t>(ctas, fit) / fit); };
    const double waves = static_cast<double>((units * s + fit - 1) / fit);
    const double clusters_us = waves * static_cast<double>((rounds + s - 1) / s) * round_us(units * s);
    const double work = static_cast<double>(units * rounds) * (batch > 1 ? 0.6 : 1.0);
    const double even_us = std::ceil(work / fit) * round_us(units * rounds) + 5.0;
    if (rounds == 1 || clusters_us <= even_us) {
      p.cluster = static_cast<int>(s);
      p.ctas = static_cast<int>(units * s);
      return p;
    }
  }
  p.ctas = static_cast<int>(units * rounds < fit ? units * rounds : fit);
  const int64_t slots = 2 * static_cast<int64_t>(p.ctas) * 4 * p.nt;
  const int64_t rows_all = static_cast<int64_t>(batch) * heads * p.rows_pad;
  p.off_ml = align256(units * 16);  // the units' parts come first
  p.off_o = p.off_ml + align256(slots * 8);
  p.off_unit = p.off_o + align256(slots * dim * 4);
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
