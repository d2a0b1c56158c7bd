// Backward pass of dense causal attention over packed sequences.
//   P = exp(scale q.k - lse), dP = dout . v, D = dout . out, dZ = P (dP - D)
//   dq = scale sum dZ k,  dk += scale dZ q,  dv += P dout.
#include <cuda.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "dense.cuh"
#include "kernels.h"

namespace msa {

namespace {

// The sequence that owns packed row r (by the starts in seqs[].x or, for
// keys, seqs[].z): the last with start <= r.  False when r lies in none.
template <bool KEY>
__device__ __forceinline__ bool find_seq(const DenseArgs &a, int r, int4 &s) {
  int lo = 0, hi = a.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((KEY ? a.seqs[mid].z : a.seqs[mid].x) <= r) lo = mid; else hi = mid - 1;
  }
  s = a.seqs[lo];
  return KEY ? (r >= s.z && r < s.z + s.w) : (r >= s.x && r < s.x + s.y);
}

__device__ __forceinline__ float4 row4(const uint16_t *p, size_t row, int lane) {
  const uint2 w = reinterpret_cast<const uint2 *>(p + row * kHeadDim)[lane];
  return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
}
__device__ __forceinline__ float dot4(const float4 &x, const float4 &y) {
  float z = x.x * y.x + x.y * y.y + x.z * y.z + x.w * y.w;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  return z;
}
__device__ __forceinline__ void axpy4(float4 &y, float a, const float4 &x) {
  y.x = fmaf(a, x.x, y.x);
  y.y = fmaf(a, x.y, y.y);
  y.z = fmaf(a, x.z, y.z);
  y.w = fmaf(a, x.w, y.w);
}
__device__ __forceinline__ void put_row4(uint16_t *p, size_t row, int lane, const float4 &x, float f) {
  reinterpret_cast<uint2 *>(p + row * kHeadDim)[lane] =
      make_uint2(pack_bf16x2(x.x * f, x.y * f), pack_bf16x2(x.z * f, x.w * f));
}

// dq: one warp per (query row, head).
__global__ void __launch_bounds__(256) dense_bwd_dq_kernel(const DenseArgs a) {
  const long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int r = int(w / a.H), h = int(w % a.H), g = h / (a.H / a.G);
  int4 s;
  if (r >= a.nq || !find_seq<false>(a, r, s)) return;
  const int n_vis = s.w - s.y + (r - s.x) + 1;
  const float4 q = row4(a.q, size_t(w), lane), go = row4(a.dout, size_t(w), lane);
  const float D = dot4(go, row4(a.out, size_t(w), lane));
  const float lse2 = a.lse[w] * 1.4426950408889634f;
  float4 dq = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int x = 0; x < n_vis; ++x) {
    const size_t kr = size_t(s.z + x) * a.G + g;
    const float4 k = row4(a.k, kr, lane);
    const float p = exp2f(dot4(q, k) * a.scale_log2 - lse2);
    axpy4(dq, p * (dot4(go, row4(a.v, kr, lane)) - D), k);
  }
  put_row4(a.dq, size_t(w), lane, dq, a.scale);
}

// dk, dv: one warp per (key row, KV head), over the query rows that see it.
__global__ void __launch_bounds__(256) dense_bwd_dkv_kernel(const DenseArgs a) {
  const long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int r = int(w / a.G), g = int(w % a.G), R = a.H / a.G;
  int4 s;
  if (r >= a.nk || !find_seq<true>(a, r, s)) return;
  const float4 k = row4(a.k, size_t(w), lane), v = row4(a.v, size_t(w), lane);
  float4 dk = make_float4(0.f, 0.f, 0.f, 0.f), dv = dk;
  // query i sees key x = r - s.z when x <= nk - nq + i
  for (int i = max(0, (r - s.z) - (s.w - s.y)); i < s.y; ++i)
    for (int h = g * R; h < (g + 1) * R; ++h) {
      const size_t qr = size_t(s.x + i) * a.H + h;
      const float4 q = row4(a.q, qr, lane), go = row4(a.dout, qr, lane);
      const float D = dot4(go, row4(a.out, qr, lane));
      const float p = exp2f(dot4(q, k) * a.scale_log2 - a.lse[qr] * 1.4426950408889634f);
      axpy4(dv, p, go);
      axpy4(dk, p * (dot4(go, v) - D), q);
    }
  put_row4(a.dk, size_t(w), lane, dk, a.scale);
  put_row4(a.dv, size_t(w), lane, dv, 1.f);
}

unsigned warps_grid(long long warps) { return unsigned((warps + 7) / 8); }

}  // namespace

cudaError_t launch_dense_varlen_backward(const DenseArgs &a, int num_sms, cudaStream_t st) {
  (void)num_sms;
  cudaError_t e = launch_dense_plan(a, st);
  if (e != cudaSuccess) return e;
  if (a.nq > 0) dense_bwd_dq_kernel<<<warps_grid((long long)a.nq * a.H), 256, 0, st>>>(a);
  if (a.nk > 0) dense_bwd_dkv_kernel<<<warps_grid((long long)a.nk * a.G), 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace msa
