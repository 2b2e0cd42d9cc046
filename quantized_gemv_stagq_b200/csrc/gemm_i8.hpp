// Arguments of the 8-bit linear's kernels, and their launchers.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

namespace stagq {

struct QuantizeI8Args {
  const uint16_t* x;
  int64_t x_stride;   // elements between rows
  int8_t* q;          // rows of ld bytes
  float* scale;
  int32_t n, in, ld, bf16, vec;
};

struct GemmI8Args {
  const float* xs;
  const float* ws;
  void* y;
  int64_t y_stride;   // elements between rows
  int32_t n, out, kblocks;           // kblocks: 128-byte blocks of a row
  // tiles of 128 channels and of BN tokens, and the CTAs of a cluster that
  // share one; for pairs, tiles of 256 tokens and of BN channels
  int32_t m_tiles, n_tiles, split;
  int32_t wide;                      // every row of y is aligned to 16 bytes
  int32_t y_f32, y_bf16;
  uint32_t stall_ns;                 // test hook: a wait of this length that runs out
};

// The tile and split that plan_gemm_i8 chose.
struct GemmI8Plan {
  int bn;     // tokens per tile
  int split;  // CTAs of a cluster that share a tile's K
  int pair;   // two CTAs share a tile of 256 channels
  int grid;
};

GemmI8Plan plan_gemm_i8(int n, int out, int kblocks, int num_sms);
cudaError_t launch_quantize_i8(const QuantizeI8Args& a, cudaStream_t s);
// xq: n rows, wq: out rows, both of ld bytes. `encode_failed` is set when the
// driver refused a tensor map.
cudaError_t launch_gemm_i8(GemmI8Args a, const GemmI8Plan& p, const int8_t* xq, const int8_t* wq, int ld,
                           cudaStream_t s, bool* encode_failed);

}  // namespace stagq
