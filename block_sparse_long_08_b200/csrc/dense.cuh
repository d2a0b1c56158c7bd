// What the dense packed-sequence kernels share.
#pragma once
#include <cuda_runtime.h>

#include "common.cuh"
#include "kernels.h"

namespace msa {

// Checks cu_q and cu_k, writes seqs, the list of items of `per` queries and,
// when a.items_k is given, that of key tiles and stat (see DenseArgs).
cudaError_t launch_dense_plan(const DenseArgs &a, int per, int num_sms, cudaStream_t st);

// Programmatic dependent launch: wait for the kernel before this one in the
// stream, and let the next one start its own prologue.
__device__ __forceinline__ void grid_dep_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void grid_dep_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Registers per thread of a warpgroup, out of those the block was launched with.
template <uint32_t N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <uint32_t N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
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

// Four 16-byte granules per lane, transposed among the lanes of a quad: lane
// l's granule j becomes lane j's granule l.
__device__ __forceinline__ void quad_transpose(uint4 (&g)[4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int bit = 1; bit <= 2; bit <<= 1) {
    const bool up = lane & bit;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & bit) continue;
      uint4 &lo = g[i], &hi = g[i | bit];
      uint4 t = up ? lo : hi;
      t.x = __shfl_xor_sync(0xffffffffu, t.x, bit);
      t.y = __shfl_xor_sync(0xffffffffu, t.y, bit);
      t.z = __shfl_xor_sync(0xffffffffu, t.z, bit);
      t.w = __shfl_xor_sync(0xffffffffu, t.w, bit);
      if (up) lo = t; else hi = t;
    }
  }
}
// 32 fp32 values of this lane's row times f, as bf16, to granules g0 .. g0+3 of
// the row.  A lane per row would touch 32 lines with every store, 16 bytes
// of each; the quad's transpose makes it eight lines, 64 bytes of each.
// row_ptr(j): where row j of the quad's four (tile rows row & ~3 ..) begins,
// or null when it is not to be written.  All lanes of the warp take part.
template <typename RowPtr>
__device__ __forceinline__ void quad_store32(const float *v, float f, int g0, RowPtr row_ptr) {
  uint4 g[4];
#pragma unroll
  for (int c = 0; c < 4; ++c)
    g[c] = make_uint4(pack_bf16x2(v[8 * c] * f, v[8 * c + 1] * f), pack_bf16x2(v[8 * c + 2] * f, v[8 * c + 3] * f),
                      pack_bf16x2(v[8 * c + 4] * f, v[8 * c + 5] * f),
                      pack_bf16x2(v[8 * c + 6] * f, v[8 * c + 7] * f));
  quad_transpose(g);
  const int l = threadIdx.x & 3;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint16_t *p = row_ptr(j);
    if (p) reinterpret_cast<uint4 *>(p)[g0 + l] = g[j];
  }
}

}  // namespace msa
