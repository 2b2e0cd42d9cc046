// Shared by the serving operators that stand beside the GEMV (8-bit linear,
// 4-bit cache): conversions of the 16-bit types, the launch helper, and the
// status bits that stagq_ops_check reports.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "stagq.h"

namespace stagq {

// Bits of an operator's status word (one word per translation unit and device).
constexpr uint32_t kOpsTimeout = 1u;   // a bounded wait ran out
constexpr uint32_t kOpsBadPage = 2u;   // a page number or position outside the pool or the table

// Reads and clears one translation unit's status word on the current device.
cudaError_t take_status_i8(uint32_t* word);
cudaError_t take_status_kv(uint32_t* word);
cudaError_t take_status_kv_attention(uint32_t* word);

namespace ops {

// One 16-bit value, fp16 or bf16, as fp32 (exact).
__device__ __forceinline__ float load16(uint16_t v, bool bf16) {
  return bf16 ? __uint_as_float(static_cast<uint32_t>(v) << 16) : __half2float(__ushort_as_half(v));
}
__device__ __forceinline__ uint16_t store16(float v, bool bf16) {
  return bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
}
// Two values rounded and packed by one instruction, lo in the lower half.
__device__ __forceinline__ uint32_t store16x2(float lo, float hi, bool bf16) {
  uint32_t r;
  if (bf16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// binary64 to fp16 or bf16 with one rounding: to fp32 by round-to-odd (a
// truncation whose lost bits set the last one), which keeps a tie a tie and a
// near tie a near tie, then to nearest even. fp32 has 13 bits more than fp16.
__device__ __forceinline__ uint16_t store16_from_double(double d, bool bf16) {
  float f = __double2float_rz(d);
  if (static_cast<double>(f) != d) f = __uint_as_float(__float_as_uint(f) | 1u);
  return store16(f, bf16);
}
__device__ __forceinline__ uint32_t pack2(uint16_t lo, uint16_t hi) {
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}
// Eight consecutive 16-bit values from p; one 16-byte load where `vec` (p is
// then 16-byte aligned).
__device__ __forceinline__ void load8(const uint16_t* p, bool vec, uint16_t (&v)[8]) {
  if (vec) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = static_cast<uint16_t>(a[i]);
      v[2 * i + 1] = static_cast<uint16_t>(a[i] >> 16);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = p[i];
  }
}

}  // namespace ops

// Restores the caller's current device on scope exit.
struct OpsDevice {
  int prev = -1;
  bool ok = false;
  explicit OpsDevice(int dev) {
    ok = cudaGetDevice(&prev) == cudaSuccess && (prev == dev || cudaSetDevice(dev) == cudaSuccess);
    if (prev == dev) prev = -1;
    if (!ok) cudaGetLastError();  // reported by the call; not left for the caller's next one
  }
  ~OpsDevice() {
    if (prev >= 0) cudaSetDevice(prev);
  }
};

// Launches `kern` with programmatic dependent launch: its CTAs may become
// resident while the previous kernel of the stream drains. Every operator
// kernel therefore waits for the previous grid in every thread before it
// touches memory.
template <typename... P, typename... A>
cudaError_t launch_op(void (*kern)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

}  // namespace stagq
