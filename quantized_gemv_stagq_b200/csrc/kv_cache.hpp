// Arguments of the 4-bit cache's kernels, and their launchers.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "stagq.h"

namespace stagq {

// The pool and one call's page table. A (page, head, K | V) block holds
// `page` rows of dim / 2 code bytes, then `page` rows of dim / group pairs
// (scale, lowest) of the cache's 16-bit type.
struct KvView {
  uint8_t* pages;
  const int32_t* table;
  int64_t table_stride;    // entries between the table rows of two sequences
  uint32_t page_stride;    // bytes of a page (all heads, K and V)
  int32_t block_bytes;     // bytes of a (page, head, K | V) block
  int32_t n_pages, table_width, heads, dim, group, page, page_shift;
  int32_t bf16;
};

// Division of numbers below 2^31 by d >= 1 without a division (Granlund and
// Montgomery): with s = ceil(log2 d) and m = ceil(2^(31 + s) / d), x / d is
// (x m) >> (31 + s), as m d - 2^(31 + s) < d <= 2^s; that is the upper word of
// 2 x m, shifted by s.
struct Divider {
  uint32_t d = 1, m = 0x80000000u, shift = 0;
  Divider() = default;
  explicit Divider(uint32_t by) : d(by) {
    while ((1ull << shift) < by) ++shift;
    m = static_cast<uint32_t>(((1ull << (31 + shift)) + by - 1) / by);
  }
#ifdef __CUDACC__
  __device__ __forceinline__ uint32_t divide(uint32_t x) const { return __umulhi(2 * x, m) >> shift; }
#endif
};

struct KvRowsArgs {        // append and read
  KvView kv;
  void* k;                 // 16-bit rows (fp32 for a read with STAGQ_Y_F32)
  void* v;
  uint32_t k_stride, v_stride;  // elements between two rows
  const int32_t* starts;   // null: 0
  const int32_t* lens;     // read only; null: no bound
  int64_t n_rows;          // batch * n
  int32_t n, f32, vec;     // tokens per sequence; fp32 output; 16-byte accesses allowed
  // set by the launchers: tokens of a CTA, groups per row, log2 of a group's lanes
  int32_t cta_tokens, groups, group_shift;
  Divider per_token, per_sequence;  // items of a token; token rows of a sequence
};

struct KvAttnArgs {
  KvView kv;
  const uint16_t* q;
  uint16_t* out;
  int64_t q_stride, out_stride;
  const int32_t* lens;
  float* mass;             // null: not tracked
  int64_t mass_stride_b, mass_stride_h;
  int4* parts;             // by unit: first and last CTA with a part of it, the first's slot
  float* part_o;           // partial sums: [ctas][2][rows of a block][dim]; null: no unit is shared
  float2* part_ml;         // their maxima and denominators
  float2* unit_ml;         // tracked: the same of the rows that one CTA finished, [batch * heads][rows_pad]
  float* scores;           // [batch * heads][rows_pad][score_stride]
  int64_t score_stride;
  int32_t batch, q_heads, per, n_new, rows, rows_pad, row_blocks, ctas, max_len, vec_out;
  int32_t cluster;         // CTAs per unit, or 0: the even split
  float scale_log2;        // softmax scale times log2(e)
  uint32_t stall_ns;       // test hook: a wait of this length that runs out
};

struct KvEvictArgs {
  KvView src, dst;
  const int32_t* lens;
  const float* mass;
  float* new_mass;
  int32_t* kept;
  int32_t* new_lens;
  int64_t mass_stride_b, mass_stride_h, new_mass_stride_b, new_mass_stride_h;
  int32_t batch, max_len, budget, recent, new_cap;
  int32_t share;           // set by the launcher: CTAs that share a head's selection
};

struct KvAttnPlan {
  int nt;                  // query rows per CTA: 4 * nt
  int row_blocks, ctas, rows_pad, cluster;
  int64_t score_stride;
  int64_t off_ml, off_o, off_unit, off_scores, bytes;  // workspace layout
};

KvAttnPlan plan_kv_attention(int batch, int heads, int q_heads, int n_new, int dim, int max_len, bool mass,
                             int num_sms);

cudaError_t launch_kv_append(KvRowsArgs a, int num_sms, cudaStream_t s);
cudaError_t launch_kv_read(KvRowsArgs a, int num_sms, cudaStream_t s);
cudaError_t launch_kv_attention(const KvAttnArgs& a, const KvAttnPlan& p, cudaStream_t s);
cudaError_t launch_kv_evict(KvEvictArgs a, int num_sms, cudaStream_t s);

}  // namespace stagq
