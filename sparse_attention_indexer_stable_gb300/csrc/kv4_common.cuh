// kv4_common.cuh -- what the kernels of the 4-bit key/value cache share: the
// element conversions, asynchronous copies, and the launch helper.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "dcp_kv4.h"

namespace dcp {
namespace kv4 {

constexpr int kBlock = 16;  // elements that share a scale

// The cache as the kernels see it.  A slot's rows start at
// (slot * heads + head) * bytes per head row; 64-bit, since a plane may pass
// 4 GB.
struct Planes {
  uint8_t* k_codes;
  uint8_t* v_codes;
  uint8_t* k_scales;
  uint8_t* v_scales;
  uint32_t num_pages;
  int page_shift;
  int heads;
  float k_unit, v_unit;

  __device__ uint64_t num_slots() const { return (uint64_t)num_pages << page_shift; }
};

// Waits until the stream's previous kernel is complete and visible, then lets
// the next one be scheduled (it waits here in its turn).
__device__ __forceinline__ void grid_dependency_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Four bytes of two codes each -> four fp16 pairs, the low nibble in the low
// half.  Exact.
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t (&d)[4]) {
  asm("{\n .reg .b8 a, b, c, e;\n mov.b32 {a, b, c, e}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, e;\n}"
      : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
      : "r"(w));
}

// Two e4m3 scales -> an fp16 pair, the low byte in the low half.  Exact.
__device__ __forceinline__ uint32_t scales_to_half(uint32_t pair) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"((uint16_t)pair));
  return d;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// a times the low, or the high, half of s.
__device__ __forceinline__ uint32_t hmul2_low(uint32_t a, uint32_t s) {
  const __half2 r = __hmul2_rn(*reinterpret_cast<const __half2*>(&a),
                               __low2half2(*reinterpret_cast<const __half2*>(&s)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hmul2_high(uint32_t a, uint32_t s) {
  const __half2 r = __hmul2_rn(*reinterpret_cast<const __half2*>(&a),
                               __high2half2(*reinterpret_cast<const __half2*>(&s)));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// tanh by 1 - 2 / (e^2x + 1), and near 0, where that cancels, by the odd
// series to x^9: relative error below 2^-20 (the series' at 0.35 2^-21, the
// quotient's approximations 2^-22 of 1).
__device__ __forceinline__ float tanh_score(float x) {
  const float a = fabsf(x), q = x * x;
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(exp2_approx(a * 2.8853900817779268f) + 1.0f));
  const float far = copysignf(fmaf(-2.0f, r, 1.0f), x);
  float near = fmaf(q, 62.0f / 2835.0f, -17.0f / 315.0f);
  near = fmaf(q, near, 2.0f / 15.0f);
  near = fmaf(q, near, -1.0f / 3.0f);
  near = fmaf(x * q, near, x);
  return a < 0.35f ? near : far;  // NaN goes through `far`
}

// base + row * stride, in one wide multiply-add.
__device__ __forceinline__ const uint8_t* row_at(const uint8_t* base, uint32_t row,
                                                 uint32_t stride) {
  const uint8_t* r;
  asm("mad.wide.u32 %0, %1, %2, %3;" : "=l"(r) : "r"(row), "r"(stride), "l"(base));
  return r;
}

// Asynchronous copy of N bytes (4, 8 or 16) into shared memory; zeros where
// !ok, with nothing read.
template <int N>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool ok) {
  const int n = ok ? N : 0;
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N),
                 "r"(n)
                 : "memory");
}

// 16 bytes of which the last may be zeros: `bytes` (0 to 16) are read.
__device__ __forceinline__ void cp_async_some(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}

// The same without the choice.
template <int N>
__device__ __forceinline__ void cp_async_all(uint32_t dst, const void* src) {
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N)
                 : "memory");
}

__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}

template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float load_element(const void* p, int64_t i, int dtype) {
  if (dtype == DCP_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  if (dtype == DCP_F16) return __half2float(static_cast<const __half*>(p)[i]);
  return static_cast<const float*>(p)[i];
}

__device__ __forceinline__ uint32_t pack_pair(float lo, float hi, int dtype) {
  if (dtype == DCP_BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Launches with programmatic stream serialization: the grid may be scheduled
// while the stream's previous kernel drains; every kernel here waits for it
// (griddepcontrol.wait) before it touches global memory.
template <typename... KArgs, typename... Args>
inline cudaError_t launch(void (*kernel)(KArgs...), dim3 grid, int block, size_t smem, int cluster,
                          cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace kv4
}  // namespace dcp
