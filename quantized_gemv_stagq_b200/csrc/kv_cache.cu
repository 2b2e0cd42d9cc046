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
#include <climits>

#include "kv_cache.hpp"
#include "kernel_common.cuh"
#include "ops_common.cuh"

namespace stagq {
namespace {

__device__ uint32_t g_status;

using kernels::grid_dependency_wait;
using kernels::grid_launch_dependents;
using kernels::kFull;

// K block of (page of position pos, head) of sequence b; null if the position
// or the page number is outside the table or the pool. The sizes of a pool's
// parts fit 32 bits, so that each offset is one widening multiplication.
__device__ __forceinline__ uint8_t* kv_block(const KvView& kv, int b, int pos, int head) {
  const int page = pos >> kv.page_shift;
  if (pos < 0 || page >= kv.table_width) return nullptr;
  const int pid = kv.table[b * kv.table_stride + page];
  if (pid < 0 || pid >= kv.n_pages) return nullptr;
  return kv.pages + static_cast<uint64_t>(static_cast<uint32_t>(pid)) * kv.page_stride + static_cast<uint32_t>(2 * head * kv.block_bytes);
}

// Append and read: dim / 8 lanes take a token's K and V rows of one head, 8
// consecutive channels each, so that a row's code bytes move in one coalesced
// access. Items are numbered (token, head, lane) and found again by
// multiplications (Divider): the kernels are bound by bytes only as long as
// finding an item costs less than moving it, which is also why an item is K
// and V (one page lookup for both).
struct Item {
  int tok, head, c8;  // token row of the call; c8: channels 8 c8 .. 8 c8 + 7
};
__device__ __forceinline__ Item item_of(const KvRowsArgs& a, int tok0, uint32_t i) {
  const uint32_t t = a.per_token.divide(i), rest = i - t * a.per_token.d;
  const int shift = a.kv.dim == 128 ? 4 : 3;  // lanes per row
  return {tok0 + static_cast<int>(t), static_cast<int>(rest >> shift), static_cast<int>(rest) & ((1 << shift) - 1)};
}

constexpr int kRowThreads = 256;

__device__ __forceinline__ uint64_t row_offset(int row, uint32_t stride) {
  return static_cast<uint64_t>(static_cast<uint32_t>(row)) * stride;
}
// start + i, which stays past every table where it would overflow.
__device__ __forceinline__ int position(int start, int i) { return start > INT_MAX - i ? INT_MAX : start + i; }
constexpr float kWhole = 12582912.0f;  // 1.5 * 2^23: a sum with it is rounded to a whole number

// ------------------------------------------------------------------ append

// The rounding error of d = x - y in fp32 (Moller and Knuth's two-sum): 0 if d is exact.
__device__ __forceinline__ float difference_error(float x, float y, float d) {
  const float z = d - x;
  return (x - (d - z)) - (y + z);
}

// RN16((hi - lo) / 15). fp32 gives it unless it lies within 8 ulp of a tie
// between two 16-bit values (its error is below 4); there the remainder's sign,
// which one multiply-add has exactly, decides. Where hi - lo is not exact or
// fp32's own spacing widens, 64 bits do.
template <bool BF>
__device__ __forceinline__ uint16_t scale16(float lo, float hi) {
  const float d = hi - lo, s = d * (1.0f / 15.0f);
  const uint32_t bits = __float_as_uint(s), tie = BF ? 0x8000u : 0x1000u;
  const int cut = static_cast<int>(bits & (2 * tie - 1)) - static_cast<int>(tie);
  if (s > (BF ? 1e-36f : 6.2e-5f) && s < 1e37f) {
    if (cut > 8 || cut < -8) return ops::store16(s, BF);
    if (difference_error(hi, lo, d) == 0.0f) {
      const uint32_t middle = (bits & ~(2 * tie - 1)) | tie;
      const float rest = fmaf(-15.0f, __uint_as_float(middle), d);
      return ops::store16(__uint_as_float(rest > 0.0f ? middle + 1 : rest < 0.0f ? middle - 1 : middle), BF);
    }
  }
  return ops::store16_from_double((static_cast<double>(hi) - static_cast<double>(lo)) / 15.0, BF);
}

// The codes of eight channels by the 64-bit quotient.
__device__ __noinline__ uint32_t exact_codes(uint4 v, float lo, float s, bool bf16) {
  uint32_t word = 0;
  for (int k = 0; k < 8; ++k) {
    const uint32_t pair = k < 2 ? v.x : k < 4 ? v.y : k < 6 ? v.z : v.w;
    const double x = ops::load16(static_cast<uint16_t>(pair >> (16 * (k & 1))), bf16);
    const double u = rint((x - static_cast<double>(lo)) / static_cast<double>(s));
    word |= static_cast<uint32_t>(fmin(u, 15.0)) << (4 * k);
  }
  return word;
}

template <bool BF>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t r;
  if (BF)
    asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <bool BF>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  if (BF)
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint4 load8_packed(const uint16_t* p, bool vec) {
  if (vec) return *reinterpret_cast<const uint4*>(p);
  return make_uint4(ops::pack2(p[0], p[1]), ops::pack2(p[2], p[3]), ops::pack2(p[4], p[5]), ops::pack2(p[6], p[7]));
}

// Codes (nibble k: channel k of the lane's eight) and the group's pair. All
// lanes of the warp take part; a group is `glanes` neighbouring ones.
template <bool BF>
__device__ __forceinline__ uint32_t round8(const uint4& v, int glanes, uint32_t& pair) {
  uint32_t lo2 = min2<BF>(min2<BF>(v.x, v.y), min2<BF>(v.z, v.w));
  uint32_t hi2 = max2<BF>(max2<BF>(v.x, v.y), max2<BF>(v.z, v.w));
  uint32_t top = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
  for (int d = 1; d < glanes; d <<= 1) {
    lo2 = min2<BF>(lo2, __shfl_xor_sync(kFull, lo2, d));
    hi2 = max2<BF>(hi2, __shfl_xor_sync(kFull, hi2, d));
    top = __vmaxu2(top, __shfl_xor_sync(kFull, top, d));
  }
  const bool fine = max(top & 0xFFFFu, top >> 16) < (BF ? 0x7F80u : 0x7C00u);
  if (!fine) {
    pair = BF ? 0x7FC07FC0u : 0x7E007E00u;
    return 0u;
  }
  const float lo = fminf(ops::load16(static_cast<uint16_t>(lo2), BF), ops::load16(static_cast<uint16_t>(lo2 >> 16), BF));
  const float hi = fmaxf(ops::load16(static_cast<uint16_t>(hi2), BF), ops::load16(static_cast<uint16_t>(hi2 >> 16), BF));
  const uint16_t s16 = scale16<BF>(lo, hi);
  const float s = ops::load16(s16, BF);
  pair = ops::pack2(s16, ops::store16(lo, BF));  // exact: lo is one of the inputs
  if (s == 0.0f) return 0u;
  const float inv = __frcp_rn(s);
  if (s < (BF ? 1e-36f : 6.2e-5f) || !(hi - lo < 1e37f)) return exact_codes(v, lo, s, BF);
  // The quotient of d = x - lo and s, correctly rounded by Markstein's method (a
  // correctly rounded reciprocal, one correction), so that ties, which are
  // common where K and V have few bits, are exact halves and round to even. It
  // is checked by the remainder d - u s, which a multiply-add has exactly if d
  // is exact: more than s / 2 means a quotient next to a half that rounded to
  // it. d is exact if no element lies more than 2^16 (fp16: 2^13) below the
  // group's largest, 24 bits spanning them; if not, a remainder near s / 2
  // decides nothing. Either leaves the lane's eight to 64 bits.
  uint32_t word = 0;
  float far = 0.0f;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 7; k >= 0; --k) {
    const float d = ops::load16(static_cast<uint16_t>(w[k >> 1] >> (16 * (k & 1))), BF) - lo;
    const float q0 = d * inv;
    const float r = fmaf(fmaf(-q0, s, d), inv, q0) + kWhole;
    far = fmaxf(far, fabsf(fmaf(kWhole - r, s, d)));
    word = word * 16u + __float_as_uint(r);  // the lowest 4 bits of r are the code
  }
  word -= 0x4B400000u * 0x11111111u;
  if (far >= s * 0.49999f) {
    uint32_t low = 0xFFFFFFFFu;  // the smallest magnitudes' bits less 1 (zero: the largest)
#pragma unroll
    for (int k = 0; k < 4; ++k) low = __vminu2(low, __vsub2(w[k] & 0x7FFF7FFFu, 0x00010001u));
    const int smallest = min(min(low & 0xFFFFu, low >> 16), static_cast<uint32_t>(ops::store16(fabsf(lo), BF) - 1) & 0xFFFFu);
    const int largest = static_cast<int>(max(top & 0xFFFFu, top >> 16));
    if (far > s * 0.5f || smallest < largest - (BF ? 16 * 128 : 13 * 1024)) word = exact_codes(v, lo, s, BF);
  }
  return word;
}

// Bound by bytes: 4 per channel read (K and V), about 1 written.
template <bool BF>
__global__ void __launch_bounds__(kRowThreads) kv_append_kernel(const __grid_constant__ KvRowsArgs a) {
  grid_launch_dependents();
  grid_dependency_wait();
  const KvView& kv = a.kv;
  const int tok0 = blockIdx.x * a.cta_tokens;
  const uint32_t n_items = min(a.cta_tokens, static_cast<int>(a.n_rows) - tok0) * a.per_token.d;
  const int glanes = kv.group >> 3;
  for (uint32_t i0 = 0; i0 < n_items; i0 += kRowThreads) {
    const uint32_t i = i0 + threadIdx.x;
    const bool in = i < n_items;
    const Item it = item_of(a, tok0, in ? i : 0);
    const int c = it.head * kv.dim + 8 * it.c8;
    const uint4 k = load8_packed(static_cast<const uint16_t*>(a.k) + row_offset(it.tok, a.k_stride) + c, a.vec);
    const uint4 v = load8_packed(static_cast<const uint16_t*>(a.v) + row_offset(it.tok, a.v_stride) + c, a.vec);
    const int b = static_cast<int>(a.per_sequence.divide(it.tok));
    const int start = a.starts[b];
    const int pos = position(start, it.tok - b * a.n);
    uint8_t* block = kv_block(kv, b, start < 0 ? -1 : pos, it.head);
    if (in && !block && start >= 0 && it.c8 == 0) atomicOr(&g_status, kOpsBadPage);
    uint32_t pair_k, pair_v;
    const uint32_t word_k = round8<BF>(k, glanes, pair_k), word_v = round8<BF>(v, glanes, pair_v);
    // V: the lane of blocks j and j ^ 1 swap halves, so that each has 4 bytes in a row
    const int j = it.c8 >> 2, t = it.c8 & 3;
    const uint32_t other = __shfl_xor_sync(kFull, word_v, 4);
    const uint32_t bytes_v = j & 1 ? __byte_perm(other, word_v, 0x7632) : __byte_perm(word_v, other, 0x5410);
    if (!in || !block) continue;
    const int slot = pos & (kv.page - 1), half = kv.dim >> 1;
    uint8_t* at = block + slot * half;
    *reinterpret_cast<uint32_t*>(at + t * (kv.dim >> 3) + 4 * j) = word_k;
    at += kv.block_bytes;
    *reinterpret_cast<uint32_t*>(at + (2 * t + (j & 1)) * (kv.dim >> 4) + 2 * (j & ~1)) = bytes_v;
    if ((it.c8 & (glanes - 1)) == 0) {
      uint8_t* meta = block + kv.page * half + 4 * (slot * a.groups + (it.c8 >> a.group_shift));
      *reinterpret_cast<uint32_t*>(meta) = pair_k;
      *reinterpret_cast<uint32_t*>(meta + kv.block_bytes) = pair_v;
    }
  }
}

// -------------------------------------------------------------------- read

template <bool BF, bool F32>
__device__ __forceinline__ void write8(void* base, int64_t at, uint32_t word, uint32_t pair, bool vec) {
  const float s = ops::load16(static_cast<uint16_t>(pair), BF), lo = ops::load16(static_cast<uint16_t>(pair >> 16), BF);
  float x[8];
#pragma unroll
  for (int k = 0; k < 8; ++k)  // a code under the exponent of 2^23 is 2^23 + u
    x[k] = fmaf(s, __uint_as_float(((word >> (4 * k)) & 15u) | 0x4B000000u) - 8388608.0f, lo);
  if (F32) {
    float* dst = static_cast<float*>(base) + at;
    if (vec) {
      reinterpret_cast<float4*>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
      reinterpret_cast<float4*>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) dst[k] = x[k];
    }
  } else {
    uint16_t* dst = static_cast<uint16_t*>(base) + at;
    uint32_t y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] = ops::store16x2(x[2 * k], x[2 * k + 1], BF);
    if (vec) {
      *reinterpret_cast<uint4*>(dst) = make_uint4(y[0], y[1], y[2], y[3]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) dst[k] = static_cast<uint16_t>(y[k >> 1] >> (16 * (k & 1)));
    }
  }
}

// The values of positions starts[b] + i, i < n; rows at or past lens[b], and
// rows whose page is bad, are zero (code 0, scale 0, lowest 0).
template <bool BF, bool F32>
__global__ void __launch_bounds__(kRowThreads) kv_read_kernel(const __grid_constant__ KvRowsArgs a) {
  grid_launch_dependents();
  grid_dependency_wait();
  const KvView& kv = a.kv;
  const int tok0 = blockIdx.x * a.cta_tokens;
  const uint32_t n_items = min(a.cta_tokens, static_cast<int>(a.n_rows) - tok0) * a.per_token.d;
  const int half = kv.dim >> 1;
#pragma unroll 2
  for (uint32_t i = threadIdx.x; i < n_items; i += kRowThreads) {
    const Item it = item_of(a, tok0, i);
    const int b = static_cast<int>(a.per_sequence.divide(it.tok));
    const int pos = position(a.starts ? a.starts[b] : 0, it.tok - b * a.n);
    const bool inside = pos >= 0 && (!a.lens || pos < a.lens[b]);
    const uint8_t* block = inside ? kv_block(kv, b, pos, it.head) : nullptr;
    if (inside && !block && it.c8 == 0) atomicOr(&g_status, kOpsBadPage);
    uint32_t word_k = 0, word_v = 0, pair_k = 0, pair_v = 0;
    if (block) {
      const int slot = pos & (kv.page - 1);
      const int j = it.c8 >> 2, t = it.c8 & 3;
      const uint8_t* at = block + slot * half;
      word_k = *reinterpret_cast<const uint32_t*>(at + t * (kv.dim >> 3) + 4 * j);
      at += kv.block_bytes;
      word_v = ops::pack2(*reinterpret_cast<const uint16_t*>(at + (2 * t) * (kv.dim >> 4) + 2 * j),
                          *reinterpret_cast<const uint16_t*>(at + (2 * t + 1) * (kv.dim >> 4) + 2 * j));
      const uint8_t* meta = block + kv.page * half + 4 * (slot * a.groups + (it.c8 >> a.group_shift));
      pair_k = *reinterpret_cast<const uint32_t*>(meta);
      pair_v = *reinterpret_cast<const uint32_t*>(meta + kv.block_bytes);
    }
    const int c = it.head * kv.dim + 8 * it.c8;
    write8<BF, F32>(a.k, row_offset(it.tok, a.k_stride) + c, word_k, pair_k, a.vec);
    write8<BF, F32>(a.v, row_offset(it.tok, a.v_stride) + c, word_v, pair_v, a.vec);
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

__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive;\n\tbarrier.cluster.wait;" ::: "memory");
}
__device__ __forceinline__ int load_peer(const int* p, uint32_t rank) {
  uint32_t peer;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(peer) : "r"(kernels::smem_addr(p)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(peer) : "memory");
  return v;
}

// kept[b, h, :] for one (sequence, head) per cluster of a.share CTAs: the `want`
// largest masses of the first `old` tokens, ties to the lowest index, then the
// recent tokens, all in their order. The CTAs take consecutive slices of the
// tokens. A radix selection finds the want-th largest key 8 bits at a time;
// every lane counts into its own copy of the histogram (256 x 32 counters), so
// equal keys, which a mass of mostly one exponent is full of, do not queue on
// one shared-memory word, and the CTAs add their histograms through distributed
// shared memory. Then every 32 tokens count their kept ones, a scan over the
// counts and the CTAs numbers them, and the kept positions are written. Up to
// KEYS * 1024 tokens of a slice are read once and stay in registers; KEYS = 0
// (share 1) reads them again in each of the six passes (they come from L2).
// Bound by instructions, 6 passes of about 10 a key, hence the sharing: 64
// heads of 32768 tokens, moved too, take 38 us with one CTA each and 30 with two.
template <int KEYS>
__global__ void __launch_bounds__(kSelThreads) kv_select_kernel(const __grid_constant__ KvEvictArgs a) {
  __shared__ int hist[kBins][32];
  __shared__ int total[2][kBins];  // of this CTA, in turn by pass: peers may still read the last one's
  __shared__ int all[kBins];
  __shared__ int2 sums[kSelWarps];
  __shared__ int s_kept[2];        // this CTA's tokens above the threshold, and equal to it
  __shared__ uint32_t s_prefix;
  __shared__ int s_want;
  grid_launch_dependents();
  grid_dependency_wait();
  const int unit = blockIdx.x / a.share, rank = blockIdx.x - unit * a.share;
  const int b = unit / a.src.heads, h = unit - b * a.src.heads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int len = a.lens[b];
  if (len > a.max_len || len < 0) {
    if (tid == 0) atomicOr(&g_status, kOpsBadPage);
    len = len < 0 ? 0 : a.max_len;
  }
  int32_t* kept = a.kept + static_cast<int64_t>(unit) * a.budget;
  const int n_kept = min(len, a.budget);
  if (rank == 0) {
    if (h == 0 && tid == 0) a.new_lens[b] = n_kept;
    for (int i = n_kept + tid; i < a.budget; i += kSelThreads) kept[i] = -1;
  }
  // (the CTAs of a cluster leave together: at once, or after the last barrier)
  const int old_all = len - a.recent, want = a.budget - a.recent;
  const bool select = len > a.budget && want > 0;
  if (rank == 0) {
    if (len <= a.budget)
      for (int i = tid; i < len; i += kSelThreads) kept[i] = i;
    else
      for (int i = tid; i < a.recent; i += kSelThreads) kept[want + i] = old_all + i;
  }
  if (a.share == 1 && !select) return;

  const int per = select ? (old_all + 32 * a.share - 1) / (32 * a.share) * 32 : 0;
  const int first = select ? min(rank * per, old_all) : 0, old = select ? min(per, old_all - first) : 0;
  const float* mass = a.mass + b * a.mass_stride_b + h * a.mass_stride_h + first;
  constexpr int HELD = KEYS > 0 ? KEYS : 1;
  uint32_t keys[HELD];
  if (KEYS > 0) {
#pragma unroll
    for (int k = 0; k < HELD; ++k) {
      const int i = k * kSelThreads + tid;
      keys[k] = i < old ? mass_key(mass[i]) : 0u;
    }
  }
  // f(key) for the thread's tokens: tid, tid + 1024, ... of the slice
  auto each = [&](auto&& f) {
    if (KEYS > 0) {
#pragma unroll
      for (int k = 0; k < HELD; ++k)
        if (k * kSelThreads + tid < old) f(keys[k]);
    } else {
      for (int i = tid; i < old; i += kSelThreads) f(mass_key(mass[i]));
    }
  };
  if (tid == 0) {
    s_prefix = 0;
    s_want = want;
  }
  for (int shift = 24; shift >= 0; shift -= 8) {
    int* mine_total = total[(shift >> 3) & 1];
    for (int i = tid; i < kBins * 32; i += kSelThreads) (&hist[0][0])[i] = 0;
    __syncthreads();
    const uint32_t prefix = s_prefix, mask = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
    const int left = s_want;
    each([&](uint32_t key) {
      if (((key ^ prefix) & mask) == 0) atomicAdd(&hist[(key >> shift) & 255u][lane], 1);
    });
    __syncthreads();
    for (int i = warp; i < kBins; i += kSelWarps) {
      const int n = __reduce_add_sync(kFull, hist[i][lane]);
      if (lane == 0) mine_total[i] = n;
    }
    const int* sum_total = mine_total;
    if (a.share > 1) {
      cluster_sync_all();
      if (tid < kBins) {
        int n = 0;
        for (int r = 0; r < a.share; ++r) n += load_peer(mine_total + tid, r);
        all[tid] = n;
      }
      sum_total = all;
    }
    __syncthreads();
    if (warp == 0) {  // lane l: bins 255 - 8 l .. 248 - 8 l, from the largest down
      int mine = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) mine += sum_total[255 - 8 * lane - i];
      int before = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(kFull, before, d);
        if (lane >= d) before += o;
      }
      before -= mine;
      if (before < left && before + mine >= left) {  // one lane (none if nothing is selected)
        int bin = 255 - 8 * lane;
        while (before + sum_total[bin] < left) before += sum_total[bin--];
        s_prefix = prefix | (static_cast<uint32_t>(bin) << shift);
        s_want = left - before;
      }
    }
    __syncthreads();
  }
  // keys above the threshold are kept, and the first n_eq equal to it. The
  // tokens of a warp lie 32 together, `blocks` of them in all; blocks are
  // scanned 1024 at a time, thread i holding block base + i.
  const uint32_t thr = s_prefix;
  const int n_eq = s_want;
  const uint32_t below = (1u << lane) - 1u;
  const int blocks = (old + 31) / 32;
  int2* count = reinterpret_cast<int2*>(&hist[0][0]);  // 1024 pairs (above, equal)
  int2 carry = make_int2(0, 0);
  // With several CTAs there is one round of blocks, and the CTAs before this
  // one have kept `carry` first.
  for (int base = 0; base < max(blocks, 1); base += kSelThreads) {
    // block base + 32 k + warp: tokens from 32 times that on, the thread's k-th key where base = 0
    auto block_key = [&](int k, int& i) {
      i = (base + 32 * k + warp) * 32 + lane;
      return KEYS > 0 ? (k < HELD ? keys[k] : 0u) : i < old ? mass_key(mass[i]) : 0u;
    };
    constexpr int ROUNDS = KEYS > 0 ? HELD : 32;
    count[tid] = make_int2(0, 0);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < ROUNDS; ++k) {
      int i;
      const uint32_t key = block_key(k, i);
      const uint32_t up = __ballot_sync(kFull, i < old && key > thr), eq = __ballot_sync(kFull, i < old && key == thr);
      if (lane == 0) count[32 * k + warp] = make_int2(__popc(up), __popc(eq));
    }
    __syncthreads();
    const int2 mine = count[tid];
    int2 sum = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(kFull, sum.x, d), y = __shfl_up_sync(kFull, sum.y, d);
      if (lane >= d) {
        sum.x += x;
        sum.y += y;
      }
    }
    if (lane == 31) sums[warp] = sum;
    __syncthreads();
    int2 before = make_int2(0, 0), whole = make_int2(0, 0);
    for (int w = 0; w < kSelWarps; ++w) {
      const int2 o = sums[w];
      if (w < warp) {
        before.x += o.x;
        before.y += o.y;
      }
      whole.x += o.x;
      whole.y += o.y;
    }
    if (a.share > 1) {
      if (tid == 0) {
        s_kept[0] = whole.x;
        s_kept[1] = whole.y;
      }
      cluster_sync_all();
      for (int r = 0; r < rank; ++r) {
        carry.x += load_peer(&s_kept[0], r);
        carry.y += load_peer(&s_kept[1], r);
      }
    }
    count[tid] = make_int2(carry.x + before.x + sum.x - mine.x, carry.y + before.y + sum.y - mine.y);
    carry.x += whole.x;
    carry.y += whole.y;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < ROUNDS; ++k) {
      int i;
      const uint32_t key = block_key(k, i);
      const bool up = i < old && key > thr, eq = i < old && key == thr;
      const int2 at = count[32 * k + warp];
      const int ne = at.y + __popc(__ballot_sync(kFull, eq) & below);
      const int na = at.x + __popc(__ballot_sync(kFull, up) & below);
      if (up || (eq && ne < n_eq)) kept[na + min(ne, n_eq)] = first + i;
    }
    __syncthreads();
  }
  if (a.share > 1) cluster_sync_all();  // no CTA leaves while a peer reads its counts
}

// Copies the kept tokens' K and V rows to the destination pages and their
// masses to new_mass. Four lanes per token, a quarter of its code bytes each;
// kMoveTokens tokens per thread load before any is stored. Bound by bytes: kept
// rows read and written once.
constexpr int kMoveTokens = 2;

// The row of a kept token whose own page is not in the pool: zeros, as a read
// of it gives, and not what the fresh page held. t: quarter of the row.
template <int W>
__device__ __noinline__ void zero_row(const KvView& kv, uint8_t* block, int pos, int t) {
  if (!block) return;
  const int slot = pos & (kv.page - 1), half = kv.dim >> 1, ng = kv.dim / kv.group;
  for (int which = 0; which < 2; ++which, block += kv.block_bytes) {
    for (int w = 0; w < W; ++w) reinterpret_cast<uint32_t*>(block + slot * half)[t * W + w] = 0u;
    if (t < ng) reinterpret_cast<uint32_t*>(block + kv.page * half)[slot * ng + t] = 0u;
  }
}

template <int D>
__global__ void __launch_bounds__(256) kv_move_kernel(const __grid_constant__ KvEvictArgs a) {
  constexpr int W = D / 32;  // words of a quarter row
  grid_launch_dependents();
  grid_dependency_wait();
  const KvView& kv = a.src;
  constexpr int kPerCta = 64 * kMoveTokens;
  const int chunks = (a.new_cap + kPerCta - 1) / kPerCta;
  const int bh = blockIdx.x / chunks;
  const int i0 = (blockIdx.x - bh * chunks) * kPerCta + (threadIdx.x >> 2), t = threadIdx.x & 3;
  const int b = bh / kv.heads, h = bh - b * kv.heads;
  const int half = kv.dim >> 1, ng = kv.dim / kv.group;
  int from[kMoveTokens];
  uint8_t* dst[kMoveTokens];
  uint32_t codes[kMoveTokens][2][W], meta[kMoveTokens][2];
  float m[kMoveTokens];
#pragma unroll
  for (int k = 0; k < kMoveTokens; ++k) {
    const int i = i0 + 64 * k;
    from[k] = i < a.budget ? a.kept[static_cast<int64_t>(bh) * a.budget + i] : -1;
  }
#pragma unroll
  for (int k = 0; k < kMoveTokens; ++k) {
    m[k] = 0.0f;
    dst[k] = nullptr;
    if (from[k] < 0) continue;
    m[k] = a.mass[b * a.mass_stride_b + h * a.mass_stride_h + from[k]];
    const uint8_t* src = kv_block(kv, b, from[k], h);
    dst[k] = src ? kv_block(a.dst, b, i0 + 64 * k, h) : nullptr;
    if (!dst[k]) {
      if (t == 0) atomicOr(&g_status, kOpsBadPage);
      if (!src) zero_row<W>(a.dst, kv_block(a.dst, b, i0 + 64 * k, h), i0 + 64 * k, t);
      continue;
    }
    const int slot = from[k] & (kv.page - 1);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const uint8_t* p = src + which * kv.block_bytes;
#pragma unroll
      for (int w = 0; w < W; w += 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(p + slot * half + (t * W + w) * 4);
        codes[k][which][w] = v.x;
        codes[k][which][w + 1] = v.y;
      }
      if (t < ng) meta[k][which] = reinterpret_cast<const uint32_t*>(p + kv.page * half)[slot * ng + t];
    }
  }
#pragma unroll
  for (int k = 0; k < kMoveTokens; ++k) {
    const int i = i0 + 64 * k;
    if (t == 0 && i < a.new_cap) a.new_mass[b * a.new_mass_stride_b + h * a.new_mass_stride_h + i] = m[k];
    if (!dst[k]) continue;
    const int slot = i & (kv.page - 1);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      uint8_t* p = dst[k] + which * kv.block_bytes;
#pragma unroll
      for (int w = 0; w < W; w += 2)
        *reinterpret_cast<uint2*>(p + slot * half + (t * W + w) * 4) = make_uint2(codes[k][which][w], codes[k][which][w + 1]);
      if (t < ng) reinterpret_cast<uint32_t*>(p + kv.page * half)[slot * ng + t] = meta[k][which];
    }
  }
}

}  // namespace

namespace {

// Tokens of a CTA: up to four items per thread, but CTAs for the whole GPU first.
int row_ctas(KvRowsArgs& a, int num_sms) {
  a.groups = a.kv.dim / a.kv.group;
  a.group_shift = a.kv.group == 128 ? 4 : a.kv.group == 64 ? 3 : 2;
  a.per_token = Divider(static_cast<uint32_t>(a.kv.heads * (a.kv.dim / 8)));
  a.per_sequence = Divider(static_cast<uint32_t>(a.n));
  const int64_t items = a.n_rows * a.per_token.d;
  int64_t per_cta = items / (num_sms * 8);
  per_cta = per_cta < kRowThreads ? kRowThreads : per_cta > 4 * kRowThreads ? 4 * kRowThreads : per_cta;
  a.cta_tokens = static_cast<int32_t>((per_cta + a.per_token.d - 1) / a.per_token.d);
  return static_cast<int>((a.n_rows + a.cta_tokens - 1) / a.cta_tokens);
}

}  // namespace

cudaError_t launch_kv_append(KvRowsArgs a, int num_sms, cudaStream_t s) {
  const dim3 grid(row_ctas(a, num_sms)), block(kRowThreads);
  return a.kv.bf16 ? launch_op(kv_append_kernel<true>, grid, block, 0, s, a) : launch_op(kv_append_kernel<false>, grid, block, 0, s, a);
}

cudaError_t launch_kv_read(KvRowsArgs a, int num_sms, cudaStream_t s) {
  const dim3 grid(row_ctas(a, num_sms)), block(kRowThreads);
  if (a.f32)
    return a.kv.bf16 ? launch_op(kv_read_kernel<true, true>, grid, block, 0, s, a) : launch_op(kv_read_kernel<false, true>, grid, block, 0, s, a);
  return a.kv.bf16 ? launch_op(kv_read_kernel<true, false>, grid, block, 0, s, a) : launch_op(kv_read_kernel<false, false>, grid, block, 0, s, a);
}

namespace {

template <int KEYS>
cudaError_t launch_select(const KvEvictArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.batch * a.src.heads * a.share);
  cfg.blockDim = dim3(kSelThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.share;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.share > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kv_select_kernel<KEYS>, a);
}

}  // namespace

// CTAs of a selection: doubled while they fit the GPU and keep more than 4096
// tokens each, and while a slice does not fit the registers (up to 8).
cudaError_t launch_kv_evict(KvEvictArgs a, int num_sms, cudaStream_t s) {
  const int64_t units = static_cast<int64_t>(a.batch) * a.src.heads;
  a.share = 1;
  while (a.share < 8 && ((units * a.share * 2 <= num_sms && a.max_len > a.share * 2 * 4096) || a.max_len > a.share * 32 * kSelThreads))
    a.share *= 2;
  int64_t slice = (static_cast<int64_t>(a.max_len) + 32 * a.share - 1) / (32 * a.share) * 32;
  if (slice > 32 * kSelThreads || units * a.share > (1 << 30)) {
    a.share = 1;
    slice = a.max_len;
  }
  cudaError_t e = slice <= 4 * kSelThreads    ? launch_select<4>(a, s)
                  : slice <= 16 * kSelThreads ? launch_select<16>(a, s)
                  : slice <= 32 * kSelThreads ? launch_select<32>(a, s)
                                              : launch_select<0>(a, s);
  if (e != cudaSuccess) return e;
  const int64_t chunks = (a.new_cap + 64 * kMoveTokens - 1) / (64 * kMoveTokens);
  const dim3 grid(static_cast<unsigned>(chunks * a.batch * a.src.heads));
  return a.src.dim == 128 ? launch_op(kv_move_kernel<128>, grid, dim3(256), 0, s, a)
                          : launch_op(kv_move_kernel<64>, grid, dim3(256), 0, s, a);
}

cudaError_t take_status_kv(uint32_t* word) {
  cudaError_t e = cudaMemcpyFromSymbol(word, g_status, sizeof(uint32_t));
  if (e != cudaSuccess || !*word) return e;
  const uint32_t zero = 0;
  return cudaMemcpyToSymbol(g_status, &zero, sizeof(zero));
}

}  // namespace stagq
