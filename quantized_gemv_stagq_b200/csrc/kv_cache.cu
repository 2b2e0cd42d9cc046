// Writing, reading and thinning out a 4-bit cache.
//
// A group of `group` consecutive channels of one token and head is stored as
//   lo = min x,  s = RN16((max x - min x) / 15),  u = clamp(rint((x - lo) / s), 0, 15),
// and stands for lo + s u (s = 0: u = 0). The quotient that decides u is the
// binary64 one: fp32 gives the same u unless it falls within 1e-4 of a half,
// and only those elements take the 64-bit division. A group that holds an
// infinity or a NaN is stored with s = lo = NaN, so it reads back as NaN and
// spoils no other group.
//
// Code order inside a row of dim / 2 bytes (attention reads it in one load per
// lane, see kv_attention.cu): a K row holds channel 32 j + 8 t + n in nibble n
// of the 4 bytes at t dim / 8 + 4 j (t = 0..3); a V row holds channel
// 32 j + 4 g + n in nibble n of the 2 bytes at g dim / 16 + 2 j (g = 0..7).
#include "kv_cache.hpp"
#include "kernel_common.cuh"
#include "ops_common.cuh"

namespace stagq {
namespace {

__device__ uint32_t g_status;

using kernels::grid_dependency_wait;
using kernels::grid_launch_dependents;
using kernels::kFull;

// Block of (page of position pos, head, which) of sequence b; null if the
// position or the page number is outside the table or the pool.
__device__ __forceinline__ uint8_t* kv_block(const KvView& kv, int64_t b, int64_t pos, int head, int which) {
  if (pos < 0 || (pos >> kv.page_shift) >= kv.table_width) return nullptr;
  const int pid = kv.table[b * kv.table_stride + (pos >> kv.page_shift)];
  if (pid < 0 || pid >= kv.n_pages) return nullptr;
  return kv.pages + static_cast<int64_t>(pid) * kv.page_stride + static_cast<int64_t>(2 * head + which) * kv.block_bytes;
}

// ------------------------------------------------------------------ append

// Bound by bytes: 4 per channel read (K and V), about 1 written. dim / 8 lanes
// take a row (one token, head, K or V), 8 consecutive channels each, so that a
// row's code bytes leave in one coalesced store.
__global__ void __launch_bounds__(256) kv_append_kernel(const __grid_constant__ KvRowsArgs a) {
  grid_launch_dependents();
  grid_dependency_wait();
  const KvView& kv = a.kv;
  const int lanes = kv.dim >> 3;                       // 8 or 16 lanes per row
  const int64_t row = (blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x) / lanes;
  const int c8 = threadIdx.x & (lanes - 1);            // its channels: 8 c8 .. 8 c8 + 7
  const int64_t unit = row >> 1;                       // (token row, head)
  const int which = static_cast<int>(row & 1);
  const bool in = unit < a.n_rows * kv.heads;
  const int64_t tok = in ? unit / kv.heads : 0;
  const int head = in ? static_cast<int>(unit - tok * kv.heads) : 0;
  const int64_t b = tok / a.n;
  const int start = a.starts[b];
  const int64_t pos = start < 0 ? -1 : start + (tok - b * a.n);
  uint8_t* block = kv_block(kv, b, pos, head, which);
  if (in && !block && start >= 0 && c8 == 0) atomicOr(&g_status, kOpsBadPage);
  const bool live = in && block;

  uint16_t raw[8];
  const uint16_t* src = static_cast<const uint16_t*>(which ? a.v : a.k) + tok * (which ? a.v_stride : a.k_stride) +
                        head * kv.dim + 8 * c8;
  if (live) {
    ops::load8(src, a.vec, raw);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) raw[i] = 0;
  }
  float x[8], lo, hi;
  bool fine = true;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = ops::load16(raw[i], kv.bf16);
    fine = fine && isfinite(x[i]);
    lo = i ? fminf(lo, x[i]) : x[0];
    hi = i ? fmaxf(hi, x[i]) : x[0];
  }
  const int glanes = kv.group >> 3;
  for (int d = 1; d < glanes; d <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(kFull, lo, d));
    hi = fmaxf(hi, __shfl_xor_sync(kFull, hi, d));
    fine = __shfl_xor_sync(kFull, fine ? 1 : 0, d) && fine;
  }
  if (!live) return;

  const uint16_t s16 = ops::store16_from_double((static_cast<double>(hi) - static_cast<double>(lo)) / 15.0, kv.bf16);
  const float s = ops::load16(s16, kv.bf16);
  const float inv = 1.0f / s;
  uint32_t word = 0;
  if (fine && s > 0.0f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float t = (x[i] - lo) * inv;
      float u = rintf(t);
      // t is within 16 * 3 * 2^-24 of the quotient; also taken when t is not finite
      if (!(fabsf(t - u) <= 0.4999f))
        u = static_cast<float>(rint((static_cast<double>(x[i]) - static_cast<double>(lo)) / static_cast<double>(s)));
      word |= static_cast<uint32_t>(fminf(u, 15.0f)) << (4 * i);
    }
  }
  const int slot = static_cast<int>(pos & (kv.page - 1));
  uint8_t* codes = block + slot * (kv.dim >> 1);
  const int j = c8 >> 2, t = c8 & 3;
  if (which == 0) {
    *reinterpret_cast<uint32_t*>(codes + t * (kv.dim >> 3) + 4 * j) = word;
  } else {
    *reinterpret_cast<uint16_t*>(codes + (2 * t) * (kv.dim >> 4) + 2 * j) = static_cast<uint16_t>(word);
    *reinterpret_cast<uint16_t*>(codes + (2 * t + 1) * (kv.dim >> 4) + 2 * j) = static_cast<uint16_t>(word >> 16);
  }
  if ((c8 & (glanes - 1)) == 0) {
    const uint16_t nan = kv.bf16 ? 0x7FC0 : 0x7E00;
    const uint16_t lo16 = ops::store16(lo, kv.bf16);   // exact: lo is one of the inputs
    uint32_t* meta = reinterpret_cast<uint32_t*>(block + kv.page * (kv.dim >> 1)) + slot * (kv.dim / kv.group);
    meta[8 * c8 / kv.group] = fine ? ops::pack2(s16, lo16) : ops::pack2(nan, nan);
  }
}

// -------------------------------------------------------------------- read

// The values of positions starts[b] + i, i < n; rows at or past lens[b], and
// rows whose page is bad, are zero. Lanes as in kv_append_kernel.
__global__ void __launch_bounds__(256) kv_read_kernel(const __grid_constant__ KvRowsArgs a) {
  grid_launch_dependents();
  grid_dependency_wait();
  const KvView& kv = a.kv;
  const int lanes = kv.dim >> 3;
  const int64_t row = (blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x) / lanes;
  const int c8 = threadIdx.x & (lanes - 1);
  const int64_t unit = row >> 1;
  const int which = static_cast<int>(row & 1);
  if (unit >= a.n_rows * kv.heads) return;
  const int64_t tok = unit / kv.heads;
  const int head = static_cast<int>(unit - tok * kv.heads);
  const int64_t b = tok / a.n;
  const int64_t pos = (a.starts ? a.starts[b] : 0) + (tok - b * a.n);
  float x[8] = {};
  const bool inside = pos >= 0 && (!a.lens || pos < a.lens[b]);
  uint8_t* block = inside ? kv_block(kv, b, pos, head, which) : nullptr;
  if (inside && !block && c8 == 0) atomicOr(&g_status, kOpsBadPage);
  if (block) {
    const int slot = static_cast<int>(pos & (kv.page - 1));
    const uint8_t* codes = block + slot * (kv.dim >> 1);
    const int j = c8 >> 2, t = c8 & 3;
    uint32_t word;
    if (which == 0) {
      word = *reinterpret_cast<const uint32_t*>(codes + t * (kv.dim >> 3) + 4 * j);
    } else {
      word = ops::pack2(*reinterpret_cast<const uint16_t*>(codes + (2 * t) * (kv.dim >> 4) + 2 * j),
                        *reinterpret_cast<const uint16_t*>(codes + (2 * t + 1) * (kv.dim >> 4) + 2 * j));
    }
    const uint32_t m = (reinterpret_cast<const uint32_t*>(block + kv.page * (kv.dim >> 1)) +
                        slot * (kv.dim / kv.group))[8 * c8 / kv.group];
    const float s = ops::load16(static_cast<uint16_t>(m), kv.bf16), lo = ops::load16(static_cast<uint16_t>(m >> 16), kv.bf16);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fmaf(s, static_cast<float>((word >> (4 * i)) & 15u), lo);
  }
  const int64_t at = tok * (which ? a.v_stride : a.k_stride) + head * kv.dim + 8 * c8;
  void* base = which ? a.v : a.k;
  if (a.f32) {
    float* dst = static_cast<float*>(base) + at;
    if (a.vec) {
      reinterpret_cast<float4*>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
      reinterpret_cast<float4*>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) dst[i] = x[i];
    }
  } else {
    uint16_t* dst = static_cast<uint16_t*>(base) + at;
    uint16_t y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = ops::store16(x[i], kv.bf16);
    if (a.vec) {
      *reinterpret_cast<uint4*>(dst) =
          make_uint4(ops::pack2(y[0], y[1]), ops::pack2(y[2], y[3]), ops::pack2(y[4], y[5]), ops::pack2(y[6], y[7]));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) dst[i] = y[i];
    }
  }
}

// ------------------------------------------------------------------- evict

constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;
constexpr int kBins = 256;

// Order of the masses as unsigned numbers: -inf < ... < -0 = +0 < ... < +inf < NaN.
__device__ __forceinline__ uint32_t mass_key(float m) {
  if (isnan(m)) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(m == 0.0f ? 0.0f : m);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// kept[b, h, :] for one (sequence, head) per CTA: the `want` largest masses of
// the first `old` tokens, ties to the lowest index, then the recent tokens, all
// in their order. A radix selection finds the want-th largest key 8 bits at a
// time; every lane counts into its own copy of the histogram (256 x 32
// counters), so equal keys, which a mass of mostly one exponent is full of, do
// not queue on one shared-memory word. Two passes then number the kept tokens.
__global__ void __launch_bounds__(kSelThreads) kv_select_kernel(const __grid_constant__ KvEvictArgs a) {
  __shared__ int hist[kBins][32];
  __shared__ int total[kBins];
  __shared__ int n_above[kSelWarps], n_equal[kSelWarps];
  __shared__ uint32_t s_prefix;
  __shared__ int s_want;
  grid_launch_dependents();
  grid_dependency_wait();
  const int b = blockIdx.x / a.src.heads, h = blockIdx.x - b * a.src.heads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int len = a.lens[b];
  if (len > a.max_len || len < 0) {
    if (tid == 0) atomicOr(&g_status, kOpsBadPage);
    len = len < 0 ? 0 : a.max_len;
  }
  int32_t* kept = a.kept + static_cast<int64_t>(blockIdx.x) * a.budget;
  const int n_kept = min(len, a.budget);
  if (h == 0 && tid == 0) a.new_lens[b] = n_kept;
  for (int i = n_kept + tid; i < a.budget; i += kSelThreads) kept[i] = -1;
  if (len <= a.budget) {
    for (int i = tid; i < len; i += kSelThreads) kept[i] = i;
    return;
  }
  const int old = len - a.recent, want = a.budget - a.recent;
  for (int i = tid; i < a.recent; i += kSelThreads) kept[want + i] = old + i;
  if (want == 0) return;

  const float* mass = a.mass + b * a.mass_stride_b + h * a.mass_stride_h;
  if (tid == 0) {
    s_prefix = 0;
    s_want = want;
  }
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < kBins * 32; i += kSelThreads) (&hist[0][0])[i] = 0;
    __syncthreads();
    const uint32_t prefix = s_prefix, mask = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
    const int left = s_want;
    for (int i = tid; i < old; i += kSelThreads) {
      const uint32_t key = mass_key(mass[i]);
      if (((key ^ prefix) & mask) == 0) atomicAdd(&hist[(key >> shift) & 255u][lane], 1);
    }
    __syncthreads();
    for (int i = warp; i < kBins; i += kSelWarps) {
      const int n = __reduce_add_sync(kFull, hist[i][lane]);
      if (lane == 0) total[i] = n;
    }
    __syncthreads();
    if (warp == 0) {  // lane l: bins 255 - 8 l .. 248 - 8 l, from the largest down
      int mine = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) mine += total[255 - 8 * lane - i];
      int before = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(kFull, before, d);
        if (lane >= d) before += o;
      }
      before -= mine;
      if (before < left && before + mine >= left) {  // one lane
        int bin = 255 - 8 * lane;
        while (before + total[bin] < left) before += total[bin--];
        s_prefix = prefix | (static_cast<uint32_t>(bin) << shift);
        s_want = left - before;
      }
    }
    __syncthreads();
  }
  // keys above the threshold are kept, and the first s_want equal to it
  const uint32_t thr = s_prefix;
  const int n_eq = s_want;
  const int per = (old + kSelWarps * 32 - 1) / (kSelWarps * 32) * 32;  // tokens of one warp, in order
  const int lo = warp * per, hi = min(lo + per, old);
  int above = 0, equal = 0;
  for (int i = lo + lane; i < hi; i += 32) {
    const uint32_t key = mass_key(mass[i]);
    above += key > thr;
    equal += key == thr;
  }
  above = __reduce_add_sync(kFull, above);
  equal = __reduce_add_sync(kFull, equal);
  if (lane == 0) {
    n_above[warp] = above;
    n_equal[warp] = equal;
  }
  __syncthreads();
  int a0 = 0, e0 = 0;
  for (int w = 0; w < warp; ++w) {
    a0 += n_above[w];
    e0 += n_equal[w];
  }
  const uint32_t below = (1u << lane) - 1u;
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t key = i < hi ? mass_key(mass[i]) : 0u;
    const bool up = i < hi && key > thr, eq = i < hi && key == thr;
    const uint32_t mu = __ballot_sync(kFull, up), me = __ballot_sync(kFull, eq);
    const int na = a0 + __popc(mu & below), ne = e0 + __popc(me & below);
    if (up || (eq && ne < n_eq)) kept[na + min(ne, n_eq)] = i;
    a0 += __popc(mu);
    e0 += __popc(me);
  }
}

// Copies the kept tokens' K and V rows to the destination pages and their
// masses to new_mass. Four lanes per token, a quarter of its code bytes each.
// Bound by bytes: kept rows read and written once.
__global__ void __launch_bounds__(256) kv_move_kernel(const __grid_constant__ KvEvictArgs a) {
  grid_launch_dependents();
  grid_dependency_wait();
  const KvView& kv = a.src;
  const int per_cta = 64;
  const int chunks = (a.new_cap + per_cta - 1) / per_cta;
  const int bh = blockIdx.x / chunks;
  const int i = (blockIdx.x - bh * chunks) * per_cta + (threadIdx.x >> 2), t = threadIdx.x & 3;
  const int b = bh / kv.heads, h = bh - b * kv.heads;
  if (i >= a.new_cap) return;
  const int from = i < a.budget ? a.kept[static_cast<int64_t>(bh) * a.budget + i] : -1;
  if (t == 0)
    a.new_mass[b * a.new_mass_stride_b + h * a.new_mass_stride_h + i] =
        from >= 0 ? a.mass[b * a.mass_stride_b + h * a.mass_stride_h + from] : 0.0f;
  if (from < 0) return;
  const uint8_t* src = kv_block(kv, b, from, h, 0);
  uint8_t* dst = kv_block(a.dst, b, i, h, 0);
  if (!src || !dst) {
    if (t == 0) atomicOr(&g_status, kOpsBadPage);
    return;
  }
  const int half = kv.dim >> 1, ng = kv.dim / kv.group;
  const int s0 = from & (kv.page - 1), s1 = i & (kv.page - 1);
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const uint8_t* sb = src + which * kv.block_bytes;
    uint8_t* db = dst + which * kv.block_bytes;
    if (kv.dim == 128)
      reinterpret_cast<uint4*>(db + s1 * half)[t] = reinterpret_cast<const uint4*>(sb + s0 * half)[t];
    else
      reinterpret_cast<uint2*>(db + s1 * half)[t] = reinterpret_cast<const uint2*>(sb + s0 * half)[t];
    if (t < ng)
      reinterpret_cast<uint32_t*>(db + kv.page * half)[s1 * ng + t] =
          reinterpret_cast<const uint32_t*>(sb + kv.page * half)[s0 * ng + t];
  }
}

}  // namespace

cudaError_t launch_kv_append(const KvRowsArgs& a, cudaStream_t s) {
  const int64_t threads = a.n_rows * a.kv.heads * 2 * (a.kv.dim / 8);
  return launch_op(kv_append_kernel, dim3(static_cast<unsigned>((threads + 255) / 256)), dim3(256), 0, s, a);
}

cudaError_t launch_kv_read(const KvRowsArgs& a, cudaStream_t s) {
  const int64_t threads = a.n_rows * a.kv.heads * 2 * (a.kv.dim / 8);
  return launch_op(kv_read_kernel, dim3(static_cast<unsigned>((threads + 255) / 256)), dim3(256), 0, s, a);
}

cudaError_t launch_kv_evict(const KvEvictArgs& a, cudaStream_t s) {
  cudaError_t e = launch_op(kv_select_kernel, dim3(a.batch * a.src.heads), dim3(kSelThreads), 0, s, a);
  if (e != cudaSuccess) return e;
  const int64_t chunks = (a.new_cap + 63) / 64;
  return launch_op(kv_move_kernel, dim3(static_cast<unsigned>(chunks * a.batch * a.src.heads)), dim3(256), 0, s, a);
}

cudaError_t take_status_kv(uint32_t* word) {
  cudaError_t e = cudaMemcpyFromSymbol(word, g_status, sizeof(uint32_t));
  if (e != cudaSuccess || !*word) return e;
  const uint32_t zero = 0;
  return cudaMemcpyToSymbol(g_status, &zero, sizeof(zero));
}

}  // namespace stagq
