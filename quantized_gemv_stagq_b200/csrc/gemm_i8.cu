// The 8-bit linear: rows rounded to int8 with a scale each, and the product of
// two such matrices.
//
//   q_ik = rint(127 x_ik / a_i), a_i = max_k |x_ik|, scale_i = a_i / 127
//   y_ij = scale_i wscale_j sum_k q_ik w_jk        (the sum exact in int32)
//
// The product runs on the tcgen05 tensor cores (kind::i8). TMA brings 128-byte
// K blocks of both operands into a ring of 128B-swizzled stages; one thread
// issues the MMAs; the other warps read the int32 accumulators from TMEM, scale
// and store. Two kernels, chosen from the sizes by plan_gemm_i8:
//  - gemm_i8_kernel, few tokens: 128 output channels are the accumulator's
//    lanes and 16, 32 or 64 tokens its columns, so few tokens cost few columns.
//    A CTA has one tile, and two CTAs share an SM. Bound by the weights' bytes;
//    a cluster of up to 8 CTAs shares one tile's K so that all SMs stream, and
//    adds its partial sums through distributed shared memory. They are
//    integers, so the split changes no bit of the result.
//  - gemm_i8_pair_kernel, many tokens: persistent pairs of CTAs (cta_group::2)
//    on tiles of 256 tokens and 128 or 256 channels, tokens as lanes, with two
//    accumulators, so that a tile's epilogue runs under the next tile's MMAs.
//    Bound by the tensor cores.
#include <cuda.h>

#include <algorithm>

#include "gemm_i8.hpp"
#include "kernel_common.cuh"
#include "ops_common.cuh"

namespace stagq {
namespace {

__device__ uint32_t g_status;

using kernels::fence_barrier_init;
using kernels::grid_dependency_wait;
using kernels::grid_launch_dependents;
using kernels::kFull;
using kernels::mbar_arrive_expect_tx;
using kernels::mbar_init;
using kernels::mbar_wait_unless;
using kernels::smem_addr;

// -------------------------------------------------------------- quantising

constexpr int kQuantThreads = 256;

// The 8-bit values of eight elements by the 64-bit quotient.
__device__ __noinline__ uint2 quantize_exact(uint4 v, float amax, bool bf16) {
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t pair = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    const double f = ops::load16(static_cast<uint16_t>(pair >> (16 * (i & 1))), bf16);
    w[i >> 2] |= (static_cast<uint32_t>(static_cast<int>(rint(f * 127.0 / static_cast<double>(amax)))) & 255u) << (8 * (i & 3));
  }
  return make_uint2(w[0], w[1]);
}

// One row per CTA, held in registers between its maximum and its rounding, so
// x is read once: 2 bytes in and 1 out per element, bound by bytes. Two
// elements at a time share the maximum of their magnitudes' bits. q comes from
// an approximate reciprocal and is checked by the remainder 127 x - q a, which
// fp32 has exactly (18 bits against 18): no division, and ties are settled by
// it too. Rows whose a is out of fp32's reach for that divide in 64 bits.
template <int STEPS, bool BF>
__global__ void __launch_bounds__(kQuantThreads) quantize_i8_kernel(const __grid_constant__ QuantizeI8Args a) {
  __shared__ uint32_t s_top[kQuantThreads / 32];
  grid_launch_dependents();
  grid_dependency_wait();
  const int row = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint16_t* x = a.x + static_cast<int64_t>(row) * a.x_stride;
  uint32_t v[STEPS][4];
  uint32_t top = 0;  // bits of the largest magnitude, in either half
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int c = (s * kQuantThreads + threadIdx.x) * 8;
    if (a.vec && c + 8 <= a.in) {
      const uint4 w = *reinterpret_cast<const uint4*>(x + c);
      v[s][0] = w.x;
      v[s][1] = w.y;
      v[s][2] = w.z;
      v[s][3] = w.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[s][i] = ops::pack2(c + 2 * i < a.in ? x[c + 2 * i] : static_cast<uint16_t>(0),
                             c + 2 * i + 1 < a.in ? x[c + 2 * i + 1] : static_cast<uint16_t>(0));
    }
  }
#pragma unroll
  for (int s = 0; s < STEPS; ++s)
#pragma unroll
    for (int i = 0; i < 4; ++i) top = __vmaxu2(top, v[s][i] & 0x7FFF7FFFu);
  top = max(top & 0xFFFFu, top >> 16);
  top = __reduce_max_sync(kFull, top);
  if (lane == 0) s_top[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kQuantThreads / 32; ++w) top = max(top, s_top[w]);
  const bool bad = top >= (BF ? 0x7F80u : 0x7C00u);
  const float amax = ops::load16(static_cast<uint16_t>(top), BF);
  if (threadIdx.x == 0) a.scale[row] = bad ? __uint_as_float(0x7FC00000u) : amax / 127.0f;
  const bool zero = bad || top == 0;
  const float inv = 127.0f / amax;
  int8_t* q = a.q + static_cast<int64_t>(row) * a.ld;
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int c = (s * kQuantThreads + threadIdx.x) * 8;
    if (c >= a.ld) break;
    uint32_t w[2] = {0u, 0u};
    if (!zero) {
      constexpr float kRound = 12582912.0f;  // 1.5 * 2^23: a sum with it is rounded to a whole number
      if (amax > 1e-30f && amax < 1e36f) {
        uint32_t bits[8];
        float far = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float f = ops::load16(static_cast<uint16_t>(v[s][i >> 1] >> (16 * (i & 1))), BF);
          const float r = fmaf(f, inv, kRound);
          bits[i] = __float_as_uint(r);  // its lowest byte is q
          far = fmaxf(far, fabsf(fmaf(kRound - r, amax, 127.0f * f)));
        }
        if (far * 2.0f >= amax) {  // a tie, or one off next to a half
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float f = ops::load16(static_cast<uint16_t>(v[s][i >> 1] >> (16 * (i & 1))), BF);
            const float rest = 2.0f * fmaf(kRound - __uint_as_float(bits[i]), amax, 127.0f * f);
            const bool odd = bits[i] & 1u;
            bits[i] += (rest > amax || (rest == amax && odd)) - (rest < -amax || (rest == -amax && odd));
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
          w[i] = __byte_perm(__byte_perm(bits[4 * i], bits[4 * i + 1], 0x0040),
                             __byte_perm(bits[4 * i + 2], bits[4 * i + 3], 0x0040), 0x5410);
      } else {
        const uint2 exact = quantize_exact(make_uint4(v[s][0], v[s][1], v[s][2], v[s][3]), amax, BF);
        w[0] = exact.x;
        w[1] = exact.y;
      }
    }
    *reinterpret_cast<uint2*>(q + c) = make_uint2(w[0], w[1]);
  }
}

// ----------------------------------------------------------------- product

constexpr int kBM = 128;               // output channels of a tile
constexpr int kBK = 128;               // bytes of a K block: one swizzle row
constexpr int kGemmThreads = 192;      // TMA warp, MMA warp, four epilogue warps
constexpr uint64_t kWaitLimitNs = 2000000000ull;

__host__ __device__ constexpr int stage_bytes(int bn) { return (kBM + bn) * kBK; }
// Stages of the ring: two CTAs share an SM.
__host__ __device__ constexpr int stage_count(int bn) { return bn == 16 ? 6 : bn == 32 ? 5 : 4; }
__host__ __device__ constexpr int tmem_cols(int bn) { return bn < 32 ? 32 : bn; }
constexpr int kBarrierBytes = 256;
__host__ __device__ constexpr size_t gemm_smem(int bn) {
  return 1024 + static_cast<size_t>(stage_count(bn)) * stage_bytes(bn) + kBarrierBytes;
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// Shared-memory descriptor of a K-major tile of 128-byte rows, 128B swizzle:
// 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
// kind::i8 instruction descriptor: int32 accumulator, both operands signed 8
// bits and K-major.
constexpr uint32_t instr_desc(int bn, int bm) {
  return (2u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(bn >> 3) << 17) | (static_cast<uint32_t>(bm >> 4) << 24);
}
__device__ __forceinline__ void mma_i8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// The same on a pair of CTAs: copies that complete on the first CTA's barrier,
// MMAs on both shared memories, commits that arrive in both CTAs.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void mma_i8_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void mma_commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
// To the first CTA alone.
__device__ __forceinline__ void mma_commit_pair_here(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_load16(uint32_t addr, int (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive;\n\tbarrier.cluster.wait;" ::: "memory");
}
__device__ __forceinline__ int load_peer(uint32_t addr, uint32_t rank) {
  uint32_t peer;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(peer) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(peer) : "memory");
  return v;
}

// A sum is scaled by its channel first, whose weights are of one size; tokens
// (bf16) may be far from 1, and their scale times the sum out of fp32's range.
__device__ __forceinline__ void store_y(const GemmI8Args& a, int64_t at, float y) {
  if (a.y_f32)
    static_cast<float*>(a.y)[at] = y;
  else
    static_cast<uint16_t*>(a.y)[at] = ops::store16(y, a.y_bf16);
}

template <int BN>
__global__ void __launch_bounds__(kGemmThreads) gemm_i8_kernel(const __grid_constant__ GemmI8Args a,
                                                              const __grid_constant__ CUtensorMap wmap,
                                                              const __grid_constant__ CUtensorMap xmap) {
  constexpr int STAGES = stage_count(BN);
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem;
  __shared__ uint32_t s_stop;
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t ring = (raw + 1023u) & ~1023u;  // a swizzled tile starts on 1024 bytes
  uint8_t* ring_ptr = smem_raw + (ring - raw);
  const uint32_t bars = ring + STAGES * stage_bytes(BN);
  auto full = [&](int s) { return bars + 8 * s; };
  auto empty = [&](int s) { return bars + 8 * (STAGES + s); };
  const uint32_t acc_full = bars + 8 * (2 * STAGES), drained = bars + 8 * (2 * STAGES + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    prefetch_map(&wmap);
    prefetch_map(&xmap);
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(drained, 1);
    s_stop = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&s_tmem)),
                 "r"(tmem_cols(BN))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = s_tmem;
  volatile uint32_t* stop = &s_stop;
  grid_launch_dependents();
  grid_dependency_wait();  // x and the weights may come from earlier kernels; y may still be read

  // cluster rank `part` of `split` takes K blocks k0 .. k1 - 1 of the tile
  const int part = blockIdx.x % a.split;
  const int k0 = static_cast<int>(static_cast<int64_t>(a.kblocks) * part / a.split);
  const int k1 = static_cast<int>(static_cast<int64_t>(a.kblocks) * (part + 1) / a.split);
  const int tile = blockIdx.x / a.split, m0 = (tile % a.m_tiles) * kBM, n0 = (tile / a.m_tiles) * BN;
  auto give_up = [&]() {
    s_stop = 1;
    __threadfence_block();
    atomicOr(&g_status, kOpsTimeout);
  };

  // Test hook: one of the roles waits for what nothing completes, which one by the block's number.
  auto stalled = [&](int role) {
    return a.stall_ns && static_cast<int>(blockIdx.x % 3) == role && !kernels::mbar_wait(drained, 0, a.stall_ns);
  };
  uint32_t issued = 0;  // K blocks that this thread has asked for

  if (warp == 0) {
    if (lane == 0) {
      bool ok = !stalled(0);
      for (int k = k0; k < k1 && ok; ++k) {
        const int s = issued % STAGES;
        ok = mbar_wait_unless(empty(s), ((issued / STAGES) & 1) ^ 1, kWaitLimitNs, stop);
        if (!ok) break;
        const uint32_t dst = ring + s * stage_bytes(BN);
        mbar_arrive_expect_tx(full(s), stage_bytes(BN));
        tma_load_2d(dst, &wmap, k * kBK, m0, full(s));
        tma_load_2d(dst + kBM * kBK, &xmap, k * kBK, n0, full(s));
        ++issued;
      }
      if (!ok) give_up();
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = instr_desc(BN, kBM);
      bool ok = !stalled(1);
      for (int k = k0; k < k1 && ok; ++k) {
        const int it = k - k0, s = it % STAGES;
        ok = mbar_wait_unless(full(s), (it / STAGES) & 1, kWaitLimitNs, stop);
        if (!ok) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint64_t ad = smem_desc(ring + s * stage_bytes(BN)), bd = smem_desc(ring + s * stage_bytes(BN) + kBM * kBK);
#pragma unroll
        for (int i = 0; i < kBK / 32; ++i)  // 32 bytes of K per MMA: 2 units of the descriptor's address
          mma_i8(tmem, ad + 2 * i, bd + 2 * i, idesc, it > 0 || i > 0);
        mma_commit(empty(s));
      }
      if (ok)
        mma_commit(acc_full);
      else
        give_up();
    }
  } else {
    const int quarter = warp & 3;  // the TMEM lanes that this warp may read
    const int row = quarter * 32 + lane, o = m0 + row, cols = min(BN, a.n - n0);
    bool ok = !stalled(2) && mbar_wait_unless(acc_full, 0, kWaitLimitNs, stop);
    ok = __all_sync(kFull, ok);
    if (!ok) {
      if (lane == 0) give_up();
    } else {
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t addr = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
      const float ws = o < a.out ? a.ws[o] : 0.0f;
      for (int c0 = 0; c0 < cols; c0 += 16) {
        int v[16];
        tmem_load16(addr + c0, v);
        if (a.split > 1) {
          // the ring is free: every MMA that read it has completed
          int* red = reinterpret_cast<int*>(ring_ptr);
#pragma unroll
          for (int i = 0; i < 16; ++i) red[(c0 + i) * kBM + row] = v[i];
        } else if (o < a.out) {
          float xs[16];  // all loads before the first store, which might be to the same place for all the compiler knows
#pragma unroll
          for (int i = 0; i < 16; ++i) xs[i] = c0 + i < cols ? a.xs[n0 + c0 + i] : 0.0f;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (c0 + i < cols) store_y(a, static_cast<int64_t>(n0 + c0 + i) * a.y_stride + o, static_cast<float>(v[i]) * ws * xs[i]);
        }
      }
    }
  }
  if (a.split > 1) {
    __syncwarp();
    cluster_sync_all();
    if (warp >= 2 && !*stop) {
      const int row = (warp & 3) * 32 + lane, o = m0 + row, cols = min(BN, a.n - n0);
      if (o < a.out) {
        const float ws = a.ws[o];
        // four columns' sums of every CTA at a time: a load from a peer takes as long as one from L2
        for (int c0 = part; c0 < cols; c0 += 4 * a.split) {
          int v[4][8];
          float xs[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) xs[i] = c0 + i * a.split < cols ? a.xs[n0 + c0 + i * a.split] : 0.0f;
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int r = 0; r < 8; ++r)
              v[i][r] = r < a.split && c0 + i * a.split < cols ? load_peer(ring + ((c0 + i * a.split) * kBM + row) * 4, r) : 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = c0 + i * a.split;
            if (c >= cols) break;
            int sum = 0;
#pragma unroll
            for (int r = 0; r < 8; ++r) sum += v[i][r];
            store_y(a, static_cast<int64_t>(n0 + c) * a.y_stride + o, static_cast<float>(sum) * ws * xs[i]);
          }
        }
      }
    }
    __syncwarp();
    cluster_sync_all();  // no CTA leaves while a peer reads its sums
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  if (*stop) {
    // A wait ran out, in whichever warp: the copies and MMAs in flight end
    // before shared memory and TMEM go. (Else the epilogue has seen the MMAs
    // complete, and they have consumed every copy.)
    if (threadIdx.x == 0)
      for (uint32_t j = issued < STAGES ? 0 : issued - STAGES; j < issued; ++j)
        kernels::mbar_wait(full(j % STAGES), (j / STAGES) & 1, kWaitLimitNs);
    if (threadIdx.x == 32) {
      mma_commit(drained);
      kernels::mbar_wait(drained, 0, kWaitLimitNs);
    }
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  }
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(tmem_cols(BN)));
}

// Many tokens: two CTAs of a cluster share a tile of 256 tokens x BN channels
// (cta_group::2). Each loads its 128 tokens and half of the channels; the MMAs,
// issued by the first, read both halves of the channels from both shared
// memories. Each keeps its 128 tokens of the accumulator in its own TMEM, a
// token per lane, so that a thread holds consecutive channels of one row of y
// and stores 16 bytes at a time; eight warps do that under the next tile's MMAs
// (with 2-byte stores by four warps they did not keep up with K = 4096).
// Barriers that the MMAs wait for are the first CTA's.
//
// BN = 256 reads 512 rows of operands per 65536 products and K element, BN = 128
// 384 per 32768: at K = 14336 and 4096 tokens and channels the latter was bound
// by L2 (2.8 GB: 237 us, against 175).
constexpr int pair_stage_bytes(int bn) { return (kBM + bn / 2) * kBK; }
constexpr int pair_stages(int bn) { return bn == 128 ? 8 : 6; }
constexpr size_t pair_smem(int bn) { return 1024 + static_cast<size_t>(pair_stages(bn)) * pair_stage_bytes(bn) + kBarrierBytes; }

__device__ __forceinline__ uint32_t in_first_cta(uint32_t addr) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
  return r;
}

__device__ __forceinline__ void store_peer(uint32_t addr, uint32_t rank, uint32_t v) {
  uint32_t peer;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(peer) : "r"(addr), "r"(rank));
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(peer), "r"(v) : "memory");
}
// Counts bytes as arrived that no copy will bring.
__device__ __forceinline__ void mbar_complete_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

constexpr int kPairThreads = 320;  // TMA warp, MMA warp, eight epilogue warps

// 16 consecutive channels of 32 rows of y, a row per lane, from int32 sums.
// `at`: the lane's first element; `left` channels exist; `rows`: lanes whose row
// exists. Where every row is aligned to 16 bytes a lane stores its own; else the
// warp turns the block round in shared memory and stores two rows' 16 channels at
// a time.
struct __align__(16) TurnBuffer {
  float v[32][17];
};
__device__ __forceinline__ void store_rows(const GemmI8Args& a, int64_t at, const int (&v)[16], float xs, const float* ws,
                                           int left, int rows, int lane, TurnBuffer& turn) {
  float y[16];
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    const float4 w = *reinterpret_cast<const float4*>(ws + i);
    y[i] = static_cast<float>(v[i]) * w.x * xs;
    y[i + 1] = static_cast<float>(v[i + 1]) * w.y * xs;
    y[i + 2] = static_cast<float>(v[i + 2]) * w.z * xs;
    y[i + 3] = static_cast<float>(v[i + 3]) * w.w * xs;
  }
  if (a.wide && left >= 16) {
    if (lane >= rows) return;
    if (a.y_f32) {
      float4* dst = reinterpret_cast<float4*>(static_cast<float*>(a.y) + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) dst[i] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
    } else {
      uint32_t p[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = ops::store16x2(y[2 * i], y[2 * i + 1], a.y_bf16);
      uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.y) + at);
      dst[0] = make_uint4(p[0], p[1], p[2], p[3]);
      dst[1] = make_uint4(p[4], p[5], p[6], p[7]);
    }
    return;
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 16; ++i) turn.v[lane][i] = y[i];
  __syncwarp();
  const int c = lane & 15, r0 = lane >> 4;
  const int64_t base = __shfl_sync(kFull, at, 0) + c;
  if (c < left) {
#pragma unroll 4
    for (int r = r0; r < min(rows, 32); r += 2) store_y(a, base + r * a.y_stride, turn.v[r][c]);
  }
}

template <int BN>
__global__ void __launch_bounds__(kPairThreads) gemm_i8_pair_kernel(const __grid_constant__ GemmI8Args a,
                                                                   const __grid_constant__ CUtensorMap wmap,
                                                                   const __grid_constant__ CUtensorMap xmap) {
  constexpr int STAGES = pair_stages(BN), STAGE = pair_stage_bytes(BN), ACC = 2;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem;
  __shared__ uint32_t s_stop;
  __shared__ uint32_t s_issued[2];                  // the first CTA's: K blocks that each CTA has asked for
  __shared__ __align__(16) float s_ws[8][BN / 2];  // scales of an epilogue warp's channels
  __shared__ TurnBuffer s_turn[8];
  const uint32_t ring = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t bars = ring + STAGES * STAGE;
  auto full = [&](int s) { return bars + 8 * s; };
  auto empty = [&](int s) { return bars + 8 * (STAGES + s); };
  auto acc_full = [&](int s) { return bars + 8 * (2 * STAGES + s); };
  auto acc_empty = [&](int s) { return bars + 8 * (2 * STAGES + ACC + s); };
  const uint32_t drained = bars + 8 * (2 * STAGES + 2 * ACC);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x & 1;

  if (threadIdx.x == 0) {
    prefetch_map(&wmap);
    prefetch_map(&xmap);
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full(s), 1);    // the first CTA's: both CTAs' copies complete on it
      mbar_init(empty(s), 1);   // in both: the MMAs' commit arrives
    }
    for (int s = 0; s < ACC; ++s) {
      mbar_init(acc_full(s), 1);
      mbar_init(acc_empty(s), 512);  // the first CTA's: both CTAs' epilogue threads
    }
    mbar_init(drained, 1);
    s_stop = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&s_tmem)), "r"(2 * BN)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers are set up
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = s_tmem;
  volatile uint32_t* stop = &s_stop;
  grid_launch_dependents();
  grid_dependency_wait();

  const int n_work = a.m_tiles * a.n_tiles, first = blockIdx.x >> 1, step = gridDim.x >> 1;
  auto give_up = [&]() {  // both CTAs stop: neither gets on without the other
    s_stop = 1;
    __threadfence_block();
    store_peer(smem_addr(&s_stop), rank ^ 1, 1);
    atomicOr(&g_status, kOpsTimeout);
  };
  // Test hook: one of the roles waits for what nothing completes, which one by the pair's number.
  auto stalled = [&](int role) {
    return a.stall_ns && first % 4 == role && !kernels::mbar_wait(drained, 0, a.stall_ns);
  };

  if (warp == 0) {
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = !stalled(rank);
      for (int w = first; w < n_work && ok; w += step) {
        const int m0 = (w % a.m_tiles) * 2 * kBM + rank * kBM, c0 = (w / a.m_tiles) * BN + rank * (BN / 2);
        for (int k = 0; k < a.kblocks; ++k, ++it) {
          const int s = it % STAGES;
          if (!mbar_wait_unless(empty(s), ((it / STAGES) & 1) ^ 1, kWaitLimitNs, stop)) {
            ok = false;
            break;
          }
          const uint32_t dst = ring + s * STAGE, bar = in_first_cta(full(s));
          if (rank == 0) mbar_arrive_expect_tx(full(s), 2 * STAGE);
          tma_load_2d_pair(dst, &xmap, k * kBK, m0, bar);
          tma_load_2d_pair(dst + kBM * kBK, &wmap, k * kBK, c0, bar);
        }
      }
      if (!ok) give_up();
      store_peer(smem_addr(&s_issued[rank]), 0, it);
    }
  } else if (warp == 1) {
    if (rank == 0 && lane == 0) {
      constexpr uint32_t idesc = instr_desc(BN, 2 * kBM);
      uint32_t it = 0, tile = 0;
      bool ok = !stalled(2);
      for (int w = first; w < n_work && ok; w += step, ++tile) {
        const int buf = tile % ACC;
        if (!mbar_wait_unless(acc_empty(buf), ((tile / ACC) & 1) ^ 1, kWaitLimitNs, stop)) {
          ok = false;
          break;
        }
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        for (int k = 0; k < a.kblocks; ++k, ++it) {
          const int s = it % STAGES;
          if (!mbar_wait_unless(full(s), (it / STAGES) & 1, kWaitLimitNs, stop)) {
            ok = false;
            break;
          }
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint64_t ad = smem_desc(ring + s * STAGE), bd = smem_desc(ring + s * STAGE + kBM * kBK);
#pragma unroll
          for (int i = 0; i < kBK / 32; ++i) mma_i8_pair(tmem + buf * BN, ad + 2 * i, bd + 2 * i, idesc, k > 0 || i > 0);
          mma_commit_pair(empty(s));
        }
        if (ok) mma_commit_pair(acc_full(buf));
      }
      if (!ok) give_up();
    }
  } else {
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    float* scales = s_ws[warp - 2];
    uint32_t tile = 0;
    bool ok = !__any_sync(kFull, stalled(3));
    if (!ok && lane == 0) give_up();
    for (int w = first; w < n_work && ok; w += step, ++tile) {
      const int tok = (w % a.m_tiles) * 2 * kBM + rank * kBM + quarter * 32 + lane;
      const int o0 = (w / a.m_tiles) * BN + half * (BN / 2);
      const int buf = tile % ACC;
      __syncwarp();
#pragma unroll
      for (int i = lane; i < BN / 2; i += 32) scales[i] = o0 + i < a.out ? a.ws[o0 + i] : 0.0f;
      __syncwarp();
      ok = mbar_wait_unless(acc_full(buf), (tile / ACC) & 1, kWaitLimitNs, stop);
      ok = __all_sync(kFull, ok);
      if (!ok) {
        if (lane == 0) give_up();
        break;
      }
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t addr = tmem + buf * BN + half * (BN / 2) + (static_cast<uint32_t>(quarter * 32) << 16);
      const float xs = tok < a.n ? a.xs[tok] : 0.0f;
      const int64_t row = static_cast<int64_t>(tok) * a.y_stride;
      const int rows = a.n - (tok - lane);  // that exist from the warp's first on
      for (int c = 0; c < BN / 2 && o0 + c < a.out; c += 16) {
        int v[16];
        tmem_load16(addr + c, v);
        store_rows(a, row + o0 + c, v, xs, scales + c, a.out - o0 - c, rows, lane, s_turn[warp - 2]);
      }
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      mbar_arrive_cluster(in_first_cta(acc_empty(buf)));
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  cluster_sync_all();  // neither CTA's memory goes while the other's MMAs or copies use it
  if (*stop) {
    // A wait ran out, in whichever warp of the two CTAs (both see it: it was
    // noted before the barrier above). The MMAs and both CTAs' copies in flight
    // end before memory goes. The copies complete on the first CTA's barriers,
    // which expect both CTAs' bytes of a block that it asked for; a block that
    // only one of the two asked for is evened out here.
    if (rank == 0 && threadIdx.x == 0) {
      const uint32_t n0 = s_issued[0], n1 = s_issued[1], n = max(n0, n1);
      for (uint32_t j = n < STAGES ? 0 : n - STAGES; j < n; ++j) {
        if (j >= n0)
          mbar_arrive_expect_tx(full(j % STAGES), STAGE);
        else if (j >= n1)
          mbar_complete_tx(full(j % STAGES), STAGE);
        kernels::mbar_wait(full(j % STAGES), (j / STAGES) & 1, kWaitLimitNs);
      }
    }
    if (rank == 0 && threadIdx.x == 32) {
      mma_commit_pair_here(drained);
      kernels::mbar_wait(drained, 0, kWaitLimitNs);
    }
    __syncthreads();
    cluster_sync_all();
  }
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * BN));
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

// rows x ld bytes, read in boxes of box_rows x 128 bytes; rows past the end read as zero.
bool encode_rows(CUtensorMap* map, const int8_t* p, int64_t rows, int ld, int box_rows) {
  EncodeTiled fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(ld), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld)};
  const cuuint32_t box[2] = {kBK, static_cast<cuuint32_t>(box_rows)}, unit[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(p), dims, strides, box, unit,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

using GemmKernel = void (*)(GemmI8Args, CUtensorMap, CUtensorMap);

cudaError_t launch_gemm(GemmKernel kernel, size_t smem, int cluster, const GemmI8Args& a, const GemmI8Plan& p,
                        const CUtensorMap& wmap, const CUtensorMap& xmap, cudaStream_t s) {
  // per device and cheap; must be set before the first launch on each
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(p.grid);
  cfg.blockDim = dim3(p.pair ? kPairThreads : kGemmThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, wmap, xmap);
}

}  // namespace

// Up to 64 tokens: the smallest tile that holds them, and clusters as wide as
// all CTAs still fit the GPU (two per SM) with four K blocks each. Above, the
// cheaper of that with 64-token tiles and of the pairs, by what was measured: a
// K block takes a pair 0.36 us (BN = 256) or 0.29 us (BN = 128), a 64-token CTA
// 2 ns for every CTA there is (what L2 delivers), 0.15 us at least, and the two
// kernels 5.3 and 7.5 us besides. (256 x 14336 x 4096: 28.6 us with 64-token
// tiles, 36.8 with pairs; 512 x 4096 x 4096: 18.1 and 15.6.)
GemmI8Plan plan_gemm_i8(int n, int out, int kblocks, int num_sms) {
  GemmI8Plan p{};
  const int64_t m_tiles = (out + kBM - 1) / kBM;
  p.bn = n <= 16 ? 16 : n <= 32 ? 32 : 64;
  p.split = 1;
  const int64_t tiles = m_tiles * ((n + p.bn - 1) / p.bn);
  while (p.split < 8 && tiles * p.split * 2 <= 2 * num_sms && kblocks >= 4 * p.split * 2) p.split *= 2;
  p.grid = static_cast<int>(tiles * p.split);
  if (n <= 64) return p;

  const int64_t pairs = num_sms / 2, m_pairs = (n + 2 * kBM - 1) / (2 * kBM);
  auto pair_tiles = [&](int bn) { return m_pairs * ((out + bn - 1) / bn); };
  auto pair_us = [&](int bn, double block_us) {
    return 5.3 + (pair_tiles(bn) + pairs - 1) / pairs * kblocks * block_us;
  };
  const double us256 = pair_us(256, 0.36), us128 = pair_us(128, 0.29);
  const double ctas = static_cast<double>(std::min<int64_t>(tiles * p.split, 2 * num_sms));
  const double us64 = 7.5 + static_cast<double>((tiles * p.split + 2 * num_sms - 1) / (2 * num_sms)) *
                      ((kblocks + p.split - 1) / p.split) * std::max(0.15, 0.002 * ctas);
  if (us64 <= us128 && us64 <= us256) return p;
  p.split = 1;
  p.pair = 1;
  p.bn = us128 < us256 ? 128 : 256;
  p.grid = static_cast<int>(2 * std::min<int64_t>(pair_tiles(p.bn), pairs));
  return p;
}

namespace {

template <bool BF>
cudaError_t launch_quantize(const QuantizeI8Args& a, int steps, cudaStream_t s) {
  const dim3 grid(a.n), block(kQuantThreads);
  if (steps <= 2) return launch_op(quantize_i8_kernel<2, BF>, grid, block, 0, s, a);
  if (steps <= 4) return launch_op(quantize_i8_kernel<4, BF>, grid, block, 0, s, a);
  if (steps <= 8) return launch_op(quantize_i8_kernel<8, BF>, grid, block, 0, s, a);
  return launch_op(quantize_i8_kernel<16, BF>, grid, block, 0, s, a);
}

}  // namespace

cudaError_t launch_quantize_i8(const QuantizeI8Args& a, cudaStream_t s) {
  const int steps = (a.ld + kQuantThreads * 8 - 1) / (kQuantThreads * 8);
  return a.bf16 ? launch_quantize<true>(a, steps, s) : launch_quantize<false>(a, steps, s);
}

cudaError_t launch_gemm_i8(GemmI8Args a, const GemmI8Plan& p, const int8_t* xq, const int8_t* wq, int ld,
                           cudaStream_t s, bool* encode_failed) {
  a.kblocks = ld / kBK;
  if (p.pair) {
    a.m_tiles = (a.n + 2 * kBM - 1) / (2 * kBM);
    a.n_tiles = (a.out + p.bn - 1) / p.bn;
  } else {
    a.m_tiles = (a.out + kBM - 1) / kBM;
    a.n_tiles = (a.n + p.bn - 1) / p.bn;
  }
  a.split = p.split;
  a.wide = reinterpret_cast<uintptr_t>(a.y) % 16 == 0 && a.y_stride * (a.y_f32 ? 4 : 2) % 16 == 0;
  CUtensorMap wmap, xmap;
  *encode_failed = !encode_rows(&wmap, wq, a.out, ld, p.pair ? p.bn / 2 : kBM) || !encode_rows(&xmap, xq, a.n, ld, p.pair ? kBM : p.bn);
  if (*encode_failed) return cudaSuccess;
  if (p.pair) {
    if (p.bn == 128) return launch_gemm(gemm_i8_pair_kernel<128>, pair_smem(128), 2, a, p, wmap, xmap, s);
    return launch_gemm(gemm_i8_pair_kernel<256>, pair_smem(256), 2, a, p, wmap, xmap, s);
  }
  switch (p.bn) {
    case 16: return launch_gemm(gemm_i8_kernel<16>, gemm_smem(16), p.split, a, p, wmap, xmap, s);
    case 32: return launch_gemm(gemm_i8_kernel<32>, gemm_smem(32), p.split, a, p, wmap, xmap, s);
    default: return launch_gemm(gemm_i8_kernel<64>, gemm_smem(64), p.split, a, p, wmap, xmap, s);
  }
}

cudaError_t take_status_i8(uint32_t* word) {
  cudaError_t e = cudaMemcpyFromSymbol(word, g_status, sizeof(uint32_t));
  if (e != cudaSuccess || !*word) return e;
  const uint32_t zero = 0;
  return cudaMemcpyToSymbol(g_status, &zero, sizeof(zero));
}

}  // namespace stagq
