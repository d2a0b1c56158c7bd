// Dense attention over paged caches: the cache append with position rotation
// and single-token attention.
//
//   paged_append_kernel  rotates the keys and queries of new tokens by their
//                 position and writes keys and values into their cache rows.
//   paged_decode_kernel  out = softmax(scale q K^T) V of one query row per
//                 (sequence, head) over the sequence's cached tokens.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cfloat>

#include "common.cuh"
#include "kernels.h"

namespace msa {

namespace {

// ------------------------------------------------------------------ append
constexpr int kAppThreads = 256;
constexpr int kAppTokens = 4;        // most tokens per CTA

// Sixteen bf16 values of one head row, as two 16-byte granules, to fp32.
__device__ __forceinline__ void unpack16(const uint4 &a, const uint4 &b, float (&x)[16]) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = bf16_lo(w[i]);
    x[2 * i + 1] = bf16_hi(w[i]);
  }
}
__device__ __forceinline__ uint4 pack8(const float *x) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}
// Eight E4M3 codes of x * inv (round to nearest even, saturated).
__device__ __forceinline__ uint2 codes8(const float *x, float inv) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float2 lo = make_float2(x[4 * h] * inv, x[4 * h + 1] * inv);
    const float2 hi = make_float2(x[4 * h + 2] * inv, x[4 * h + 3] * inv);
    w[h] = uint32_t(__nv_cvt_float2_to_fp8x2(lo, __NV_SATFINITE, __NV_E4M3)) |
           (uint32_t(__nv_cvt_float2_to_fp8x2(hi, __NV_SATFINITE, __NV_E4M3)) << 16);
  }
  return make_uint2(w[0], w[1]);
}

// Sequence that owns packed row r by cu[0..B]: the last b with cu[b] <= r.
__device__ __forceinline__ int seq_of_row(const int32_t *cu, int B, int r) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu[mid] <= r) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// A token's rows (H query heads, G key heads, G value heads of 256 bytes)
// are shared out over groups of eight lanes, one head row each; lane j takes
// the values of rotation pairs 8j..8j+7 (or, behind rot, sixteen values that
// pass through), so a pair never leaves its thread and in-place calls are
// safe.  The token's 64 cosines and sines are made once in shared memory:
// the angle t * inv_freq needs 64 bits (at a million tokens fp32 would be
// off by 0.06 rad), and per head row that product would outweigh the copy.
template <bool FP8, bool INTER>
__global__ void __launch_bounds__(kAppThreads) paged_append_kernel(const AppendArgs a, int T) {
  __shared__ float2 s_cs[kAppTokens][64];
  __shared__ int s_pos[kAppTokens];
  __shared__ long long s_slot[kAppTokens];   // cache row, -1: nothing to do
  const int tid = threadIdx.x;
  const int row0 = blockIdx.x * T;
  if (tid < T) {
    const int r = row0 + tid;
    int pos = -1;
    long long slot = -1;
    bool bad = false;
    if (r < a.n_rows) {
      int b = r, c0 = r, c1 = r + 1;
      if (a.cu) {
        b = seq_of_row(a.cu, a.B, r);
        c0 = a.cu[b];
        c1 = a.cu[b + 1];
      }
      const int len = a.seq_lens[b];
      // behind the last sequence, or a padding sequence: skipped in silence
      if (r >= c0 && r < c1 && len != 0) {
        if (c0 < 0 || c1 > a.n_rows || len < c1 - c0 || len > a.Lmax) {
          bad = true;
        } else {
          pos = len - (c1 - r);
          const int pg = a.c.table[size_t(b) * a.c.max_pages + (pos >> a.c.page_log2)];
          if (pg < 0 || pg >= a.c.num_pages)
            bad = true;
          else
            slot = ((long long)pg << a.c.page_log2) + (pos & ((1 << a.c.page_log2) - 1));
        }
      }
    }
    // every descent of cu is seen by the row that starts behind it or, when
    // no row does, leaves rows unowned: the first CTA looks at them all
    if (bad) atomicCAS(a.status, 0, kStatusBadInput);
    s_pos[tid] = pos;
    s_slot[tid] = slot;
  }
  if (a.cu && blockIdx.x == 0) {
    bool bad = false;
    for (int b = tid; b < a.B; b += kAppThreads)
      bad |= a.cu[b] < 0 || a.cu[b + 1] < a.cu[b] || a.cu[b + 1] > a.n_rows;
    if (bad) atomicCAS(a.status, 0, kStatusBadInput);
  }
  __syncthreads();
  const int half = a.rot >> 1;
  for (int x = tid; x < T * 64; x += kAppThreads) {
    const int i = x & 63;
    if (i < half && s_slot[x >> 6] >= 0) {
      // turns of the angle, less the whole ones, in 64 bits
      const double turns = double(s_pos[x >> 6]) * double(a.inv_freq[i]) * 0.15915494309189535;
      const float frac = float(turns - rint(turns));
      float s, c;
      sincospif(2.f * frac, &s, &c);
      s_cs[x >> 6][i] = make_float2(c, s);
    }
  }
  __syncthreads();
  const int j = tid & 7;                       // sixteen values of a head row
  const int nh = a.H + 2 * a.G;
  const bool turn = 16 * j < a.rot;
  // first values of the thread's two granules
  const int e0 = (turn && !INTER) ? 8 * j : 16 * j;
  const int e1 = (turn && !INTER) ? half + 8 * j : 16 * j + 8;
  for (int idx = tid >> 3; idx < T * nh; idx += kAppThreads / 8) {
    const int t = idx / nh, h = idx % nh;
    const long long slot = s_slot[t];
    if (slot < 0) continue;                    // the eight lanes of a row agree
    const size_t r = size_t(row0 + t);
    const bool is_v = h >= a.H + a.G, is_q = h < a.H;
    const int g = is_q ? 0 : (is_v ? h - a.H - a.G : h - a.H);
    const uint16_t *src = is_q ? a.q + (r * a.H + h) * kHeadDim
                               : (is_v ? a.v : a.k) + (r * a.G + g) * kHeadDim;
    const uint4 x0 = *reinterpret_cast<const uint4 *>(src + e0);
    const uint4 x1 = *reinterpret_cast<const uint4 *>(src + e1);
    float x[16];
    unpack16(x0, x1, x);
    if (turn && !is_v) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 cs = s_cs[t][8 * j + i];
        constexpr int step = INTER ? 2 : 1, mate = INTER ? 1 : 8;
        const float u = x[step * i], w = x[step * i + mate];
        x[step * i] = u * cs.x - w * cs.y;
        x[step * i + mate] = w * cs.x + u * cs.y;
      }
    }
    if (is_q || (a.k_out && !is_v)) {
      uint16_t *dst = is_q ? a.q_out + (r * a.H + h) * kHeadDim : a.k_out + (r * a.G + g) * kHeadDim;
      *reinterpret_cast<uint4 *>(dst + e0) = pack8(x);
      *reinterpret_cast<uint4 *>(dst + e1) = pack8(x + 8);
    }
    if (is_q) continue;
    const size_t crow = size_t(slot) * a.G + g;
    if (FP8) {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(x[i]));
      const unsigned mask = 0xFFu << ((tid & 31) & ~7);
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) m = fmaxf(m, __shfl_xor_sync(mask, m, o));
      const float scale = m > 0.f ? m / 448.f : 1.f;
      const float inv = 1.f / scale;
      uint8_t *dst = static_cast<uint8_t *>(is_v ? a.c.v : a.c.k) + crow * kHeadDim;
      *reinterpret_cast<uint2 *>(dst + e0) = codes8(x, inv);
      *reinterpret_cast<uint2 *>(dst + e1) = codes8(x + 8, inv);
      if (j == 0) (is_v ? a.c.v_scale : a.c.k_scale)[crow] = scale;
    } else {
      uint16_t *dst = static_cast<uint16_t *>(is_v ? a.c.v : a.c.k) + crow * kHeadDim;
      *reinterpret_cast<uint4 *>(dst + e0) = pack8(x);
      *reinterpret_cast<uint4 *>(dst + e1) = pack8(x + 8);
    }
  }
}

// ------------------------------------------------------------------ decode
// Four values (dims 4 lane .. 4 lane + 3) of cache row `crow`, in fp32.
template <bool FP8>
__device__ __forceinline__ float4 cache_row4(const void *base, const float *scale, size_t crow,
                                             int lane) {
  if (FP8) {
    const uint32_t w = reinterpret_cast<const uint32_t *>(static_cast<const uint8_t *>(base) +
                                                          crow * kHeadDim)[lane];
    const float s = scale[crow];
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half_raw h = __nv_cvt_fp8_to_halfraw(uint8_t(w >> (8 * i)), __NV_E4M3);
      f[i] = __half2float(__half(h)) * s;
    }
    return make_float4(f[0], f[1], f[2], f[3]);
  }
  const uint2 w = reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(base) +
                                                  crow * kHeadDim)[lane];
  return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
}

// One CTA per (sequence, KV head); its four warps take the tokens in turn,
// each with its own running maximum and sum per head, joined at the end.
template <int R, bool FP8>
__global__ void __launch_bounds__(128) paged_decode_kernel(const PagedDecodeArgs a) {
  __shared__ float s_m[4][R], s_l[4][R];
  __shared__ float s_o[4][R][kHeadDim];
  const int b = blockIdx.x, g = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int n = a.seq_lens[b];
  if (n < 0 || n > a.Lmax) {
    if (threadIdx.x == 0) atomicCAS(a.status, 0, kStatusBadInput);
    n = 0;
  }
  float m[R], l[R];
  float4 o[R], q[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const uint2 w = reinterpret_cast<const uint2 *>(a.q + (size_t(b) * a.H + g * R + r) * kHeadDim)[lane];
    q[r] = make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
    m[r] = -INFINITY;
    l[r] = 0.f;
    o[r] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int s = warp; s < n; s += 4) {
    const int pg = a.c.table[size_t(b) * a.c.max_pages + (s >> a.c.page_log2)];
    if (pg < 0 || pg >= a.c.num_pages) {
      if (lane == 0) atomicCAS(a.status, 0, kStatusBadInput);
      continue;
    }
    const size_t crow =
        ((size_t(pg) << a.c.page_log2) + (s & ((1 << a.c.page_log2) - 1))) * a.G + g;
    const float4 k = cache_row4<FP8>(a.c.k, a.c.k_scale, crow, lane);
    const float4 v = cache_row4<FP8>(a.c.v, a.c.v_scale, crow, lane);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float z = q[r].x * k.x + q[r].y * k.y + q[r].z * k.z + q[r].w * k.w;
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) z += __shfl_xor_sync(0xffffffffu, z, x);
      const float mn = fmaxf(m[r], z);
      const float al = m[r] == -INFINITY ? 0.f : exp2f((m[r] - mn) * a.scale_log2);
      const float p = exp2f((z - mn) * a.scale_log2);
      m[r] = mn;
      l[r] = l[r] * al + p;
      o[r].x = o[r].x * al + p * v.x;
      o[r].y = o[r].y * al + p * v.y;
      o[r].z = o[r].z * al + p * v.z;
      o[r].w = o[r].w * al + p * v.w;
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (lane == 0) { s_m[warp][r] = m[r]; s_l[warp][r] = l[r]; }
    *reinterpret_cast<float4 *>(&s_o[warp][r][4 * lane]) = o[r];
  }
  __syncthreads();
  for (int x = threadIdx.x; x < R * kHeadDim; x += 128) {
    const int r = x / kHeadDim, d = x % kHeadDim;
    float M = -INFINITY;
    for (int w = 0; w < 4; ++w) M = fmaxf(M, s_m[w][r]);
    float L = 0.f, O = 0.f;
    for (int w = 0; w < 4; ++w) {
      const float e = s_m[w][r] == -INFINITY ? 0.f : exp2f((s_m[w][r] - M) * a.scale_log2);
      L += e * s_l[w][r];
      O += e * s_o[w][r][d];
    }
    const size_t row = size_t(b) * a.H + g * R + r;
    reinterpret_cast<__nv_bfloat16 *>(a.out)[row * kHeadDim + d] =
        __float2bfloat16(L > 0.f ? O / L : 0.f);
    if (d == 0 && a.lse) a.lse[row] = L > 0.f ? M * a.scale + logf(L) : -INFINITY;
  }
}

template <int R>
cudaError_t launch_decode_r(const PagedDecodeArgs &a, cudaStream_t st) {
  const dim3 grid(a.B, a.G);
  if (a.c.k_scale)
    paged_decode_kernel<R, true><<<grid, 128, 0, st>>>(a);
  else
    paged_decode_kernel<R, false><<<grid, 128, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_append(const AppendArgs &a, int num_sms, cudaStream_t st) {
  const int T = a.n_rows <= 8 * num_sms ? 1 : kAppTokens;
  const int grid = ceil_div(a.n_rows, T);
  auto kern = a.c.k_scale ? (a.interleaved ? paged_append_kernel<true, true> : paged_append_kernel<true, false>)
                          : (a.interleaved ? paged_append_kernel<false, true> : paged_append_kernel<false, false>);
  kern<<<grid, kAppThreads, 0, st>>>(a, T);
  return cudaGetLastError();
}

cudaError_t launch_paged_decode(const PagedDecodeArgs &a, int num_sms, cudaStream_t st) {
  (void)num_sms;
  switch (a.H / a.G) {
    case 1: return launch_decode_r<1>(a, st);
    case 2: return launch_decode_r<2>(a, st);
    case 4: return launch_decode_r<4>(a, st);
    case 8: return launch_decode_r<8>(a, st);
    case 16: return launch_decode_r<16>(a, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace msa
