// The 8-bit linear: rows rounded to int8 with a scale each, and the product of
// two such matrices.
//
//   q_ik = rint(127 x_ik / a_i), a_i = max_k |x_ik|, scale_i = a_i / 127
//   y_ij = scale_i wscale_j sum_k q_ik w_jk        (the sum exact in int32)
//
// The product runs on the tcgen05 tensor cores (kind::i8): the weights' 128
// output channels are the accumulator's 128 lanes, BN tokens its columns, so
// few tokens cost few columns and the weights are always the wide operand.
// TMA brings 128-byte K blocks of both operands into a ring of 128B-swizzled
// stages; one thread issues the MMAs; four warps read the int32 accumulators
// from TMEM, scale and store (32 consecutive channels of one token per store).
//
// Many tokens (BN = 128 or 256): persistent CTAs, one per SM, two accumulators,
// so that a tile's epilogue runs under the next tile's MMAs. Bound by the
// tensor cores. Few tokens (BN = 16, 32, 64): bound by the weights' bytes; a
// cluster of up to 8 CTAs shares one tile's K so that all SMs stream, and adds
// its partial sums through distributed shared memory. The partial sums are
// integers, so the split changes no bit of the result.
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
// Stages of the ring: two CTAs share an SM up to 64 tokens, one has it to itself above.
__host__ __device__ constexpr int stage_count(int bn) {
  return bn == 16 ? 6 : bn == 32 ? 5 : bn == 64 ? 4 : bn == 128 ? 6 : 4;
}
__host__ __device__ constexpr int acc_count(int bn) { return bn >= 128 ? 2 : 1; }
__host__ __device__ constexpr int tmem_cols(int bn) { return bn * acc_count(bn) < 32 ? 32 : bn * acc_count(bn); }
constexpr int kBarrierBytes = 256;
__host__ __device__ constexpr size_t gemm_smem(int bn) {
  return 1024 + static_cast<size_t>(stage_count(bn)) * stage_bytes(bn) + kBarrierBytes;
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
constexpr uint32_t instr_desc(int bn) {
  return (2u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(bn >> 3) << 17) | (static_cast<uint32_t>(kBM >> 4) << 24);
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
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
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
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ int load_peer(uint32_t addr, uint32_t rank) {
  uint32_t peer;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(peer) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(peer) : "memory");
  return v;
}

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
  constexpr int STAGES = stage_count(BN), ACC = acc_count(BN);
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem;
  __shared__ uint32_t s_stop;
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t ring = (raw + 1023u) & ~1023u;  // a swizzled tile starts on 1024 bytes
  uint8_t* ring_ptr = smem_raw + (ring - raw);
  const uint32_t bars = ring + STAGES * stage_bytes(BN);
  auto full = [&](int s) { return bars + 8 * s; };
  auto empty = [&](int s) { return bars + 8 * (STAGES + s); };
  auto acc_full = [&](int s) { return bars + 8 * (2 * STAGES + s); };
  auto acc_empty = [&](int s) { return bars + 8 * (2 * STAGES + ACC + s); };
  const uint32_t drained = bars + 8 * (2 * STAGES + 2 * ACC);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int s = 0; s < ACC; ++s) {
      mbar_init(acc_full(s), 1);
      mbar_init(acc_empty(s), 128);
    }
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
  const int n_work = a.m_tiles * a.n_tiles, first = blockIdx.x / a.split, step = gridDim.x / a.split;
  auto give_up = [&]() {
    s_stop = 1;
    __threadfence_block();
    atomicOr(&g_status, kOpsTimeout);
  };

  if (warp == 0) {
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int w = first; w < n_work && ok; w += step) {
        const int m0 = (w % a.m_tiles) * kBM, n0 = (w / a.m_tiles) * BN;
        for (int k = k0; k < k1; ++k, ++it) {
          const int s = it % STAGES;
          if (!mbar_wait_unless(empty(s), ((it / STAGES) & 1) ^ 1, kWaitLimitNs, stop)) {
            ok = false;
            break;
          }
          const uint32_t dst = ring + s * stage_bytes(BN);
          mbar_arrive_expect_tx(full(s), stage_bytes(BN));
          tma_load_2d(dst, &wmap, k * kBK, m0, full(s));
          tma_load_2d(dst + kBM * kBK, &xmap, k * kBK, n0, full(s));
        }
      }
      if (!ok) {
        give_up();
        // let the copies in flight land before the CTA's shared memory goes
        for (uint32_t j = it < STAGES ? 0 : it - STAGES; j < it; ++j)
          kernels::mbar_wait(full(j % STAGES), (j / STAGES) & 1, kWaitLimitNs);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = instr_desc(BN);
      uint32_t it = 0, tile = 0;
      bool ok = true;
      for (int w = first; w < n_work && ok; w += step, ++tile) {
        const int buf = tile % ACC;
        if (!mbar_wait_unless(acc_empty(buf), ((tile / ACC) & 1) ^ 1, kWaitLimitNs, stop)) {
          ok = false;
          break;
        }
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        for (int k = k0; k < k1; ++k, ++it) {
          const int s = it % STAGES;
          if (!mbar_wait_unless(full(s), (it / STAGES) & 1, kWaitLimitNs, stop)) {
            ok = false;
            break;
          }
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint64_t ad = smem_desc(ring + s * stage_bytes(BN)), bd = smem_desc(ring + s * stage_bytes(BN) + kBM * kBK);
#pragma unroll
          for (int i = 0; i < kBK / 32; ++i)  // 32 bytes of K per MMA: 2 units of the descriptor's address
            mma_i8(tmem + buf * BN, ad + 2 * i, bd + 2 * i, idesc, k > k0 || i > 0);
          mma_commit(empty(s));
        }
        if (ok) mma_commit(acc_full(buf));
      }
      if (!ok) {
        give_up();
        mma_commit(drained);  // no MMA may still read the ring or write TMEM when the CTA goes
        kernels::mbar_wait(drained, 0, kWaitLimitNs);
      }
    }
  } else {
    const int quarter = warp & 3;  // the TMEM lanes that this warp may read
    const int row = quarter * 32 + lane;
    uint32_t tile = 0;
    bool ok = true;
    for (int w = first; w < n_work && ok; w += step, ++tile) {
      const int o = (w % a.m_tiles) * kBM + row, n0 = (w / a.m_tiles) * BN;
      const int cols = min(BN, a.n - n0);
      const int buf = tile % ACC;
      ok = mbar_wait_unless(acc_full(buf), (tile / ACC) & 1, kWaitLimitNs, stop);
      ok = __all_sync(kFull, ok);
      if (!ok) {
        if (lane == 0) give_up();
        break;
      }
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t addr = tmem + buf * BN + (static_cast<uint32_t>(quarter * 32) << 16);
      const float ws = o < a.out ? __ldg(a.ws + o) : 0.0f;
      for (int c0 = 0; c0 < cols; c0 += 16) {
        int v[16];
        tmem_load16(addr + c0, v);
        if (a.split > 1) {
          // the ring is free: every MMA that read it has completed
          int* red = reinterpret_cast<int*>(ring_ptr);
#pragma unroll
          for (int i = 0; i < 16; ++i) red[(c0 + i) * kBM + row] = v[i];
        } else if (o < a.out) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (c0 + i < cols)
              store_y(a, static_cast<int64_t>(n0 + c0 + i) * a.y_stride + o,
                      static_cast<float>(v[i]) * __ldg(a.xs + n0 + c0 + i) * ws);
        }
      }
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      mbar_arrive(acc_empty(buf));
    }
  }
  if (a.split > 1) {  // one tile per cluster
    __syncwarp();
    cluster_sync_all();
    if (warp >= 2 && !*stop) {
      const int row = (warp & 3) * 32 + lane;
      const int o = (first % a.m_tiles) * kBM + row, n0 = (first / a.m_tiles) * BN;
      const int cols = min(BN, a.n - n0);
      if (o < a.out) {
        const float ws = __ldg(a.ws + o);
        for (int c = part; c < cols; c += a.split) {
          int sum = 0;
          for (int r = 0; r < a.split; ++r) sum += load_peer(ring + (c * kBM + row) * 4, r);
          store_y(a, static_cast<int64_t>(n0 + c) * a.y_stride + o, static_cast<float>(sum) * __ldg(a.xs + n0 + c) * ws);
        }
      }
    }
    __syncwarp();
    cluster_sync_all();  // no CTA leaves while a peer reads its sums
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(tmem_cols(BN)));
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

template <int BN>
cudaError_t launch_bn(const GemmI8Args& a, const GemmI8Plan& p, const CUtensorMap& wmap, const CUtensorMap& xmap,
                      cudaStream_t s) {
  // per device and cheap; must be set before the first launch on each
  cudaError_t e = cudaFuncSetAttribute(gemm_i8_kernel<BN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(gemm_smem(BN)));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(p.grid);
  cfg.blockDim = dim3(kGemmThreads);
  cfg.dynamicSmemBytes = gemm_smem(BN);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, gemm_i8_kernel<BN>, a, wmap, xmap);
}

}  // namespace

// The smallest tile that holds the tokens up to 128, then 256 if that fills
// the SMs as well. Up to 64 tokens the CTAs of a tile are doubled while all of
// them still fit the GPU (two per SM) and keep four K blocks each.
GemmI8Plan plan_gemm_i8(int n, int out, int kblocks, int num_sms) {
  GemmI8Plan p{};
  const int64_t m_tiles = (out + kBM - 1) / kBM;
  auto tiles = [&](int bn) { return m_tiles * ((n + bn - 1) / bn); };
  p.split = 1;
  if (n <= 64) {
    p.bn = n <= 16 ? 16 : n <= 32 ? 32 : 64;
    while (p.split < 8 && tiles(p.bn) * p.split * 2 <= 2 * num_sms && kblocks >= 4 * p.split * 2) p.split *= 2;
    p.grid = static_cast<int>(tiles(p.bn) * p.split);
    return p;
  }
  const int64_t w128 = (tiles(128) + num_sms - 1) / num_sms, w256 = (tiles(256) + num_sms - 1) / num_sms;
  p.bn = w128 <= 2 * w256 - 1 ? 128 : 256;
  p.grid = static_cast<int>(std::min<int64_t>(tiles(p.bn), num_sms));
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
  a.m_tiles = (a.out + kBM - 1) / kBM;
  a.n_tiles = (a.n + p.bn - 1) / p.bn;
  a.split = p.split;
  CUtensorMap wmap, xmap;
  *encode_failed = !encode_rows(&wmap, wq, a.out, ld, kBM) || !encode_rows(&xmap, xq, a.n, ld, p.bn);
  if (*encode_failed) return cudaSuccess;
  switch (p.bn) {
    case 16: return launch_bn<16>(a, p, wmap, xmap, s);
    case 32: return launch_bn<32>(a, p, wmap, xmap, s);
    case 64: return launch_bn<64>(a, p, wmap, xmap, s);
    case 128: return launch_bn<128>(a, p, wmap, xmap, s);
    default: return launch_bn<256>(a, p, wmap, xmap, s);
  }
}

cudaError_t take_status_i8(uint32_t* word) {
  cudaError_t e = cudaMemcpyFromSymbol(word, g_status, sizeof(uint32_t));
  if (e != cudaSuccess || !*word) return e;
  const uint32_t zero = 0;
  return cudaMemcpyToSymbol(g_status, &zero, sizeof(zero));
}

}  // namespace stagq
