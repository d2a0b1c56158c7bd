// What the dense packed-sequence kernels share.
#pragma once
#include <cuda_runtime.h>

#include "common.cuh"
#include "kernels.h"

namespace msa {

// Checks cu_q and cu_k, writes seqs, items and n_items (see DenseArgs).
cudaError_t launch_dense_plan(const DenseArgs &a, cudaStream_t st);

// Programmatic dependent launch: wait for the kernel before this one in the
// stream, and let the next one start its own prologue.
__device__ __forceinline__ void grid_dep_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void grid_dep_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Packed fp32 pairs (one instruction for two values).
__device__ __forceinline__ uint64_t pack_f2(float2 a) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
  return r;
}
__device__ __forceinline__ float2 unpack_f2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ float2 f2_fma(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(pack_f2(a)), "l"(pack_f2(b)), "l"(pack_f2(c)));
  return unpack_f2(d);
}
__device__ __forceinline__ float2 f2_add(float2 a, float2 b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pack_f2(a)), "l"(pack_f2(b)));
  return unpack_f2(d);
}
__device__ __forceinline__ float2 f2_mul(float2 a, float2 b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pack_f2(a)), "l"(pack_f2(b)));
  return unpack_f2(d);
}
__device__ __forceinline__ float2 f2_dup(float a) { return make_float2(a, a); }

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// 2^x of two values on the FMA pipe: x = n + f with n the nearest whole number
// (adding 1.5 * 2^23 leaves n in the low mantissa bits), 2^f by a degree-4
// polynomial whose largest relative error on [-1/2, 1/2] is 2.6e-6 (its
// coefficients: a Remez exchange on that error), n added to the exponent.
// For -126 <= x <= 126; smaller x is raised to -126.
__device__ __forceinline__ float2 f2_exp2_poly(float2 x) {
  x.x = fmaxf(x.x, -126.f);
  x.y = fmaxf(x.y, -126.f);
  const float2 magic = f2_dup(12582912.f);
  const float2 t = f2_add(x, magic);
  const float2 f = f2_add(x, f2_mul(f2_add(t, f2_dup(-12582912.f)), f2_dup(-1.f)));
  float2 p = f2_fma(f2_dup(0.009570102207362652f), f, f2_dup(0.05591785907745361f));
  p = f2_fma(p, f, f2_dup(0.240247443318367f));
  p = f2_fma(p, f, f2_dup(0.6931217908859253f));
  p = f2_fma(p, f, f2_dup(0.9999992847442627f));
  return make_float2(__int_as_float(__float_as_int(p.x) + (__float_as_int(t.x) << 23)),
                     __int_as_float(__float_as_int(p.y) + (__float_as_int(t.y) << 23)));
}

}  // namespace msa
