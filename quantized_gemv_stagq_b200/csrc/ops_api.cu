// C ABI of the operators beside the GEMV: argument checks and launches. See
// include/stagq.h for the contract of each function.
#include <atomic>
#include <climits>
#include <cmath>
#include <string>

#include "gemm_i8.hpp"
#include "host_common.hpp"
#include "kv_cache.hpp"
#include "ops_common.cuh"

namespace stagq {
namespace {

int bad(const char* what) { return fail(STAGQ_EINVAL, what); }

int launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return STAGQ_OK;
  cudaGetLastError();  // reported here; not left for the caller's next call
  return fail(STAGQ_ECUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
// Rows of 16-bit (or wider) values that wide accesses may take.
bool wide(const void* p, int64_t stride, int size) { return aligned(p, 16) && stride * size % 16 == 0; }

constexpr int kMaxDevices = 64;

// Multiprocessors of the current device `device`; 0 if the query fails.
int sm_count(int device) {
  static std::atomic<int> known[kMaxDevices];  // a racing first call stores the same number
  if (!known[device]) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    known[device] = n;
  }
  return known[device];
}

std::atomic<uint32_t> g_stall_ns[kMaxDevices];  // stagq_debug_stall_ops

// Error text, or null.
const char* cache_error(const stagq_kv_cache* c) {
  if (!c) return "null cache";
  if (c->dim != 64 && c->dim != 128) return "dim must be 64 or 128";
  if (c->group != 32 && c->group != 64 && c->group != 128) return "group must be 32, 64 or 128";
  if (c->group > c->dim) return "group exceeds dim";
  if (c->page < 16 || c->page > 1024 || (c->page & (c->page - 1))) return "page must be a power of two, 16..1024";
  if (c->heads < 1 || c->heads > 4096) return "heads outside 1..4096";
  if (c->flags & ~STAGQ_BF16) return "unknown cache flags";
  if (c->device < 0 || c->device >= kMaxDevices) return "device index outside 0..63";
  return nullptr;
}
const char* pool_error(const stagq_kv_cache* c) {
  if (const char* e = cache_error(c)) return e;
  if (!c->pages || !aligned(c->pages, 16)) return "pages must be a 16-byte aligned device pointer";
  if (c->n_pages < 1) return "the pool has no page";
  return nullptr;
}
const char* table_error(const stagq_kv_cache* c, const stagq_kv_table* t) {
  if (!t || !t->pages) return "null page table";
  if (t->batch < 1 || t->width < 1 || t->row_stride < t->width) return "bad page table shape";
  if (static_cast<int64_t>(t->width) * c->page > STAGQ_KV_MAX_TOKENS) return "page table covers more than STAGQ_KV_MAX_TOKENS";
  return nullptr;
}

KvView view_of(const stagq_kv_cache* c, const stagq_kv_table* t) {
  KvView v{};
  v.pages = static_cast<uint8_t*>(c->pages);
  v.table = t->pages;
  v.table_stride = t->row_stride;
  v.block_bytes = c->page * (c->dim / 2 + 4 * (c->dim / c->group));
  v.page_stride = 2u * c->heads * v.block_bytes;  // at most 2 * 4096 * 1024 * 80 bytes
  v.n_pages = c->n_pages;
  v.table_width = t->width;
  v.heads = c->heads;
  v.dim = c->dim;
  v.group = c->group;
  v.page = c->page;
  while ((1 << v.page_shift) < c->page) ++v.page_shift;
  v.bf16 = (c->flags & STAGQ_BF16) ? 1 : 0;
  return v;
}

// Append and read take the same rows.
const char* rows_error(const stagq_kv_cache* c, const stagq_kv_table* t, int32_t n, const void* k, int64_t ks,
                       const void* v, int64_t vs) {
  if (const char* e = pool_error(c)) return e;
  if (const char* e = table_error(c, t)) return e;
  if (n < 1 || n > STAGQ_KV_MAX_TOKENS) return "n outside 1..STAGQ_KV_MAX_TOKENS";
  if (!k || !v) return "null k or v";
  const int64_t row = static_cast<int64_t>(c->heads) * c->dim;
  if (ks < row || vs < row) return "k or v rows overlap (stride below heads * dim)";
  if (ks > INT_MAX || vs > INT_MAX) return "k or v rows lie 2^31 elements apart or more";
  if (static_cast<int64_t>(t->batch) * n > INT_MAX) return "too many rows for one call";
  return nullptr;
}

}  // namespace
}  // namespace stagq

using namespace stagq;

extern "C" int64_t stagq_i8_row_bytes(int32_t in) {
  if (in < 1 || in > STAGQ_MAX_IN) return -1;
  return (in + STAGQ_I8_ROW_MULTIPLE - 1) / STAGQ_I8_ROW_MULTIPLE * STAGQ_I8_ROW_MULTIPLE;
}

extern "C" int stagq_quantize_i8(const void* x, int64_t x_stride, int32_t n, int32_t in, uint32_t flags, int8_t* q,
                                 float* scale, int device, void* cuda_stream) {
  const int64_t ld = stagq_i8_row_bytes(in);
  if (ld < 0) return bad("in outside 1..STAGQ_MAX_IN");
  if (n < 1) return bad("n must be positive");
  if (!x || !q || !scale) return bad("null x, q or scale");
  if (x_stride < in) return bad("rows of x overlap (stride below in)");
  if (!aligned(q, 16)) return bad("q must be 16-byte aligned");
  if (flags & ~STAGQ_BF16) return bad("unknown flags");
  if (device < 0 || device >= kMaxDevices) return bad("device index outside 0..63");
  OpsDevice guard(device);
  if (!guard.ok) return fail(STAGQ_ECUDA, "cudaSetDevice failed");
  QuantizeI8Args a{};
  a.x = static_cast<const uint16_t*>(x);
  a.x_stride = x_stride;
  a.q = q;
  a.scale = scale;
  a.n = n;
  a.in = in;
  a.ld = static_cast<int32_t>(ld);
  a.bf16 = (flags & STAGQ_BF16) ? 1 : 0;
  a.vec = wide(x, x_stride, 2);
  return launched(launch_quantize_i8(a, static_cast<cudaStream_t>(cuda_stream)), "quantize launch");
}

extern "C" int stagq_gemm_i8(const int8_t* xq, const float* xscale, int32_t n, const int8_t* wq, const float* wscale,
                             int32_t out, int32_t in, void* y, int64_t y_stride, uint32_t flags, int device,
                             void* cuda_stream) {
  const int64_t ld = stagq_i8_row_bytes(in);
  if (ld < 0) return bad("in outside 1..STAGQ_MAX_IN");
  if (n < 1 || out < 1) return bad("n and out must be positive");
  if (!xq || !xscale || !wq || !wscale || !y) return bad("null argument");
  if (!aligned(xq, 16) || !aligned(wq, 16)) return bad("xq and wq must be 16-byte aligned");
  if (y_stride < out) return bad("rows of y overlap (stride below out)");
  if (flags & ~(STAGQ_Y_F32 | STAGQ_BF16)) return bad("unknown flags");
  if ((flags & STAGQ_Y_F32) && (flags & STAGQ_BF16)) return bad("y cannot be both fp32 and bf16");
  if (device < 0 || device >= kMaxDevices) return bad("device index outside 0..63");
  if ((static_cast<int64_t>(n) + 15) / 16 * ((static_cast<int64_t>(out) + 127) / 128) > INT_MAX / 16)
    return bad("n * out too large for one call");
  OpsDevice guard(device);
  if (!guard.ok) return fail(STAGQ_ECUDA, "cudaSetDevice failed");
  const int sms = sm_count(device);
  if (!sms) return fail(STAGQ_ENODEV, "no usable device");
  GemmI8Args a{};
  a.xs = xscale;
  a.ws = wscale;
  a.y = y;
  a.y_stride = y_stride;
  a.n = n;
  a.out = out;
  a.y_f32 = (flags & STAGQ_Y_F32) ? 1 : 0;
  a.y_bf16 = (flags & STAGQ_BF16) ? 1 : 0;
  a.stall_ns = g_stall_ns[device];
  bool encode_failed = false;
  const GemmI8Plan p = plan_gemm_i8(n, out, static_cast<int>(ld / STAGQ_I8_ROW_MULTIPLE), sms);
  const cudaError_t e = launch_gemm_i8(a, p, xq, wq, static_cast<int>(ld), static_cast<cudaStream_t>(cuda_stream), &encode_failed);
  if (encode_failed) return fail(STAGQ_ECUDA, "cuTensorMapEncodeTiled refused xq or wq");
  return launched(e, "int8 product launch");
}

extern "C" int64_t stagq_kv_page_bytes(const stagq_kv_cache* c) {
  if (const char* e = cache_error(c)) {
    set_error(e);
    return -1;
  }
  return 2 * static_cast<int64_t>(c->heads) * c->page * (c->dim / 2 + 4 * (c->dim / c->group));
}

extern "C" int stagq_kv_append(const stagq_kv_cache* c, const stagq_kv_table* t, const int32_t* starts, const void* k,
                               int64_t k_stride, const void* v, int64_t v_stride, int32_t n, void* cuda_stream) {
  if (const char* e = rows_error(c, t, n, k, k_stride, v, v_stride)) return bad(e);
  if (!starts) return bad("null starts");
  OpsDevice guard(c->device);
  if (!guard.ok) return fail(STAGQ_ECUDA, "cudaSetDevice failed");
  KvRowsArgs a{};
  a.kv = view_of(c, t);
  a.k = const_cast<void*>(k);
  a.v = const_cast<void*>(v);
  a.k_stride = static_cast<uint32_t>(k_stride);
  a.v_stride = static_cast<uint32_t>(v_stride);
  a.starts = starts;
  a.n = n;
  a.n_rows = static_cast<int64_t>(t->batch) * n;
  a.vec = wide(k, k_stride, 2) && wide(v, v_stride, 2);
  const int sms = sm_count(c->device);
  if (!sms) return fail(STAGQ_ENODEV, "no usable device");
  return launched(launch_kv_append(a, sms, static_cast<cudaStream_t>(cuda_stream)), "append launch");
}

extern "C" int stagq_kv_read(const stagq_kv_cache* c, const stagq_kv_table* t, const int32_t* starts,
                             const int32_t* lens, void* k, int64_t k_stride, void* v, int64_t v_stride, int32_t n,
                             uint32_t flags, void* cuda_stream) {
  if (const char* e = rows_error(c, t, n, k, k_stride, v, v_stride)) return bad(e);
  if (flags & ~STAGQ_Y_F32) return bad("unknown flags");
  OpsDevice guard(c->device);
  if (!guard.ok) return fail(STAGQ_ECUDA, "cudaSetDevice failed");
  KvRowsArgs a{};
  a.kv = view_of(c, t);
  a.k = k;
  a.v = v;
  a.k_stride = static_cast<uint32_t>(k_stride);
  a.v_stride = static_cast<uint32_t>(v_stride);
  a.starts = starts;
  a.lens = lens;
  a.n = n;
  a.n_rows = static_cast<int64_t>(t->batch) * n;
  a.f32 = (flags & STAGQ_Y_F32) ? 1 : 0;
  a.vec = wide(k, k_stride, a.f32 ? 4 : 2) && wide(v, v_stride, a.f32 ? 4 : 2);
  const int sms = sm_count(c->device);
  if (!sms) return fail(STAGQ_ENODEV, "no usable device");
  return launched(launch_kv_read(a, sms, static_cast<cudaStream_t>(cuda_stream)), "read launch");
}

namespace {

const char* attention_error(const stagq_kv_cache* c, int32_t batch, int32_t max_len, int32_t q_heads, int32_t n_new) {
  if (const char* e = cache_error(c)) return e;
  if (batch < 1) return "batch must be positive";
  if (max_len < 1 || max_len > STAGQ_KV_MAX_TOKENS) return "max_len outside 1..STAGQ_KV_MAX_TOKENS";
  if (q_heads < 1 || q_heads % c->heads) return "q_heads must be a multiple of the cache's heads";
  if (q_heads / c->heads > STAGQ_KV_MAX_SHARE) return "more than STAGQ_KV_MAX_SHARE query heads per KV head";
  if (n_new < 1 || n_new > STAGQ_KV_MAX_NEW) return "n_new outside 1..STAGQ_KV_MAX_NEW";
  // the join's grid: rows in blocks of up to 8, and 2048 tokens of a head per CTA (counted here as 512)
  const int64_t heads = static_cast<int64_t>(batch) * c->heads;
  if (heads * (q_heads / c->heads * n_new + 8 + (static_cast<int64_t>(max_len) + 511) / 512) > INT_MAX) return "too many rows for one call";
  // rounds of 128 tokens, numbered through all units
  if (heads * (q_heads / c->heads * n_new + 8) > INT_MAX / ((static_cast<int64_t>(max_len) + 127) / 128 + 8)) return "too many rows for one call";
  return nullptr;
}

}  // namespace

extern "C" int64_t stagq_kv_attention_workspace(const stagq_kv_cache* c, int32_t batch, int32_t max_len,
                                                int32_t q_heads, int32_t n_new, int tracked) {
  if (const char* e = attention_error(c, batch, max_len, q_heads, n_new)) {
    set_error(e);
    return -1;
  }
  const int sms = sm_count(c->device);
  if (!sms) {
    set_error("no usable device");
    return -1;
  }
  return plan_kv_attention(batch, c->heads, q_heads, n_new, c->dim, max_len, tracked != 0, sms).bytes;
}

extern "C" int stagq_kv_attention(const stagq_kv_cache* c, const stagq_kv_table* t, const int32_t* lens,
                                  int32_t max_len, const void* q, int64_t q_stride, int32_t q_heads, int32_t n_new,
                                  float scale, void* out, int64_t out_stride, float* mass, int64_t mass_stride_b,
                                  int64_t mass_stride_h, void* workspace, int64_t workspace_bytes, void* cuda_stream) {
  if (const char* e = pool_error(c)) return bad(e);
  if (const char* e = table_error(c, t)) return bad(e);
  if (const char* e = attention_error(c, t->batch, max_len, q_heads, n_new)) return bad(e);
  if (!lens || !q || !out) return bad("null lens, q or out");
  if (max_len > static_cast<int64_t>(t->width) * c->page) return bad("max_len exceeds the page table");
  const int64_t row = static_cast<int64_t>(q_heads) * c->dim;
  if (q_stride < row || out_stride < row) return bad("q or out rows overlap (stride below q_heads * dim)");
  if (!std::isfinite(scale)) return bad("scale must be finite");
  if (mass && (mass_stride_h < max_len || (t->batch > 1 && mass_stride_b < mass_stride_h * (c->heads - 1) + max_len)))
    return bad("mass rows overlap (strides below max_len)");
  OpsDevice guard(c->device);
  if (!guard.ok) return fail(STAGQ_ECUDA, "cudaSetDevice failed");
  const int sms = sm_count(c->device);
  if (!sms) return fail(STAGQ_ENODEV, "no usable device");
  const KvAttnPlan p = plan_kv_attention(t->batch, c->heads, q_heads, n_new, c->dim, max_len, mass != nullptr, sms);
  if (p.bytes && (!workspace || !aligned(workspace, 256) || workspace_bytes < p.bytes))
    return bad("workspace must be 256-byte aligned and hold stagq_kv_attention_workspace() bytes");
  KvAttnArgs a{};
  a.kv = view_of(c, t);
  a.q = static_cast<const uint16_t*>(q);
  a.out = static_cast<uint16_t*>(out);
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.lens = lens;
  a.mass = mass;
  a.mass_stride_b = mass_stride_b;
  a.mass_stride_h = mass_stride_h;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (p.bytes) {
    a.parts = reinterpret_cast<int4*>(ws);
    a.part_ml = reinterpret_cast<float2*>(ws + p.off_ml);
    a.part_o = reinterpret_cast<float*>(ws + p.off_o);
    if (mass) {
      a.unit_ml = reinterpret_cast<float2*>(ws + p.off_unit);
      a.scores = reinterpret_cast<float*>(ws + p.off_scores);
    }
  }
  a.score_stride = p.score_stride;
  a.batch = t->batch;
  a.q_heads = q_heads;
  a.per = q_heads / c->heads;
  a.n_new = n_new;
  a.rows = a.per * n_new;
  a.rows_pad = p.rows_pad;
  a.row_blocks = p.row_blocks;
  a.ctas = p.ctas;
  a.cluster = p.cluster;
  a.max_len = max_len;
  a.vec_out = aligned(out, 8) && out_stride % 4 == 0;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.stall_ns = g_stall_ns[c->device];
  return launched(launch_kv_attention(a, p, static_cast<cudaStream_t>(cuda_stream)), "attention launch");
}

extern "C" int stagq_kv_evict(const stagq_kv_cache* c, const stagq_kv_table* t, const int32_t* lens, int32_t max_len,
                              const float* mass, int64_t mass_stride_b, int64_t mass_stride_h, int32_t budget,
                              int32_t recent, const stagq_kv_table* fresh, int32_t* kept, int32_t* new_lens,
                              float* new_mass, int64_t new_mass_stride_b, int64_t new_mass_stride_h, int32_t new_cap,
                              void* cuda_stream) {
  if (const char* e = pool_error(c)) return bad(e);
  if (const char* e = table_error(c, t)) return bad(e);
  if (const char* e = table_error(c, fresh)) return bad(e);
  if (fresh->batch != t->batch) return bad("the two tables differ in batch");
  if (!lens || !mass || !kept || !new_lens || !new_mass) return bad("null argument");
  if (max_len < 1 || max_len > static_cast<int64_t>(t->width) * c->page) return bad("max_len outside 1..width * page");
  if (budget < 1 || budget > static_cast<int64_t>(fresh->width) * c->page) return bad("budget outside 1..the fresh table's tokens");
  if (recent < 0 || recent > budget) return bad("recent outside 0..budget");
  if (new_cap < budget) return bad("new_mass holds fewer than budget entries");
  if (new_cap > STAGQ_KV_MAX_TOKENS) return bad("new_cap exceeds STAGQ_KV_MAX_TOKENS");
  if (mass_stride_h < max_len || new_mass_stride_h < new_cap) return bad("mass rows overlap");
  if (t->batch > 1 && (mass_stride_b < mass_stride_h * (c->heads - 1) + max_len ||
                       new_mass_stride_b < new_mass_stride_h * (c->heads - 1) + new_cap))
    return bad("mass rows overlap");
  const int64_t heads = static_cast<int64_t>(t->batch) * c->heads;
  if (heads > INT_MAX || heads * ((static_cast<int64_t>(new_cap) + 63) / 64) > INT_MAX) return bad("too many rows for one call");
  // heads read lens, masses and pages while others already write theirs
  if (new_lens == lens || new_mass == mass || fresh->pages == t->pages) return bad("new_lens, new_mass and fresh must not be lens, mass and the table");
  OpsDevice guard(c->device);
  if (!guard.ok) return fail(STAGQ_ECUDA, "cudaSetDevice failed");
  KvEvictArgs a{};
  a.src = view_of(c, t);
  a.dst = view_of(c, fresh);
  a.lens = lens;
  a.mass = mass;
  a.new_mass = new_mass;
  a.kept = kept;
  a.new_lens = new_lens;
  a.mass_stride_b = mass_stride_b;
  a.mass_stride_h = mass_stride_h;
  a.new_mass_stride_b = new_mass_stride_b;
  a.new_mass_stride_h = new_mass_stride_h;
  a.batch = t->batch;
  a.max_len = max_len;
  a.budget = budget;
  a.recent = recent;
  a.new_cap = new_cap;
  const int sms = sm_count(c->device);
  if (!sms) return fail(STAGQ_ENODEV, "no usable device");
  return launched(launch_kv_evict(a, sms, static_cast<cudaStream_t>(cuda_stream)), "evict launch");
}

extern "C" int stagq_ops_check(int device) {
  if (device < 0 || device >= kMaxDevices) return bad("device index outside 0..63");
  OpsDevice guard(device);
  if (!guard.ok) return fail(STAGQ_ECUDA, "cudaSetDevice failed");
  cudaError_t e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return launched(e, "work on the device failed");
  e = cudaGetLastError();
  if (e != cudaSuccess) return launched(e, "pending CUDA error");
  uint32_t i8 = 0, kv = 0, at = 0;
  if ((e = take_status_i8(&i8)) != cudaSuccess || (e = take_status_kv(&kv)) != cudaSuccess ||
      (e = take_status_kv_attention(&at)) != cudaSuccess)
    return launched(e, "status read");
  const uint32_t word = i8 | kv | at;
  if (word & kOpsTimeout) return fail(STAGQ_ETIMEOUT, "an operator's kernel gave up a bounded wait");
  if (word & kOpsBadPage) return fail(STAGQ_EFORMAT, "a page number, position or length lies outside the pool, the table or max_len");
  return STAGQ_OK;
}

extern "C" int stagq_debug_stall_ops(int device, uint32_t stall_ns) {
  if (device < 0 || device >= kMaxDevices) return bad("device index outside 0..63");
  g_stall_ns[device] = stall_ns;
  return STAGQ_OK;
}

extern "C" int stagq_debug_gemm_i8_plan(int32_t n, int32_t out, int32_t in, int32_t num_sms, int32_t* plan) {
  const int64_t ld = stagq_i8_row_bytes(in);
  if (ld < 0 || n < 1 || out < 1 || num_sms < 2 || !plan) return bad("bad sizes or null plan");
  const GemmI8Plan p = plan_gemm_i8(n, out, static_cast<int>(ld / STAGQ_I8_ROW_MULTIPLE), num_sms);
  plan[0] = p.bn;
  plan[1] = p.split;
  plan[2] = p.pair;
  plan[3] = p.grid;
  return STAGQ_OK;
}

extern "C" int stagq_debug_kv_attention_plan(const stagq_kv_cache* c, int32_t batch, int32_t max_len, int32_t q_heads,
                                             int32_t n_new, int tracked, int32_t num_sms, int32_t* plan) {
  if (const char* e = attention_error(c, batch, max_len, q_heads, n_new)) return bad(e);
  if (num_sms < 1 || !plan) return bad("no multiprocessors or null plan");
  const KvAttnPlan p = plan_kv_attention(batch, c->heads, q_heads, n_new, c->dim, max_len, tracked != 0, num_sms);
  plan[0] = 4 * p.nt;
  plan[1] = p.row_blocks;
  plan[2] = p.ctas;
  plan[3] = p.cluster;
  return STAGQ_OK;
}
