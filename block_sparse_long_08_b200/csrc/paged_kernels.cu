// Dense attention over paged caches: the cache append with position rotation
// and single-token attention.
//
//   paged_append_kernel  rotates the keys and queries of new tokens by their
//                 position and writes keys and values into their cache rows.
//   paged_decode_kernel, paged_join_kernel  out = softmax(scale q K^T) V of
//                 one query row per (sequence, head) over the sequence's
//                 cached tokens, split over the SMs and joined.
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace msa {

namespace {

// ------------------------------------------------------------------ append
constexpr int kAppThreads = 256;
constexpr int kAppTokens = 8;        // most tokens per CTA (35K prompt tokens: 4 151 us, 8 147 us)

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
// Four E4M3 codes (round to nearest even, saturated).
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  return uint32_t(__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3)) |
         (uint32_t(__nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3)) << 16);
}
// Sixteen E4M3 codes of x / scale.  y = x (1 / scale) is within 3 * 2^-24 of
// the quotient, so where y (1 -+ 2^-21) have one code it is the quotient's;
// only a row with a value next to the middle of two codes (or whose 1 / scale
// may overflow) is divided.  11.5K prompt tokens: 31.1 us, all divided 32.6.
__device__ __forceinline__ void codes16(const float (&x)[16], float scale, uint32_t (&w)[4]) {
  const float inv = 1.f / scale, lo = inv * (1.f - 0x1p-21f), hi = inv * (1.f + 0x1p-21f);
  bool sure = scale >= 0x1p-120f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = codes4(x[4 * i] * lo, x[4 * i + 1] * lo, x[4 * i + 2] * lo, x[4 * i + 3] * lo);
    sure &= w[i] == codes4(x[4 * i] * hi, x[4 * i + 1] * hi, x[4 * i + 2] * hi, x[4 * i + 3] * hi);
  }
  if (sure) return;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = codes4(__fdiv_rn(x[4 * i], scale), __fdiv_rn(x[4 * i + 1], scale), __fdiv_rn(x[4 * i + 2], scale),
                  __fdiv_rn(x[4 * i + 3], scale));
}

// Sequence that owns packed row r by cu[0..B]: the last b with cu[b] <= r.
// A warp looks at 32 places at once (the loads depend on each other, and a
// call's first microseconds are spent here).
__device__ __forceinline__ int seq_of_row(const int32_t *cu, int B, int r) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B;                 // b lies in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const int at = lo + min(lane * step, n - 1);
    const unsigned le = __ballot_sync(0xffffffffu, lane * step < n && cu[at] <= r);
    const int k = le ? 31 - __clz(le) : 0;
    lo += k * step;
    n = min(step, n - k * step);
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
  if (tid < 32 * T) {                // a warp per token
    const int w = tid >> 5, r = row0 + w;
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
    if (bad && (tid & 31) == 0) atomicCAS(a.status, 0, kStatusBadInput);
    s_pos[w] = pos;
    s_slot[w] = slot;
  }
  // a descent of cu may leave rows that no sequence owns: the last CTA looks
  // at them all
  if (a.cu && blockIdx.x == gridDim.x - 1) {
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
      uint8_t *dst = static_cast<uint8_t *>(is_v ? a.c.v : a.c.k) + crow * kHeadDim;
      uint32_t w[4];
      codes16(x, scale, w);
      *reinterpret_cast<uint2 *>(dst + e0) = make_uint2(w[0], w[1]);
      *reinterpret_cast<uint2 *>(dst + e1) = make_uint2(w[2], w[3]);
      if (j == 0) (is_v ? a.c.v_scale : a.c.k_scale)[crow] = scale;
    } else {
      uint16_t *dst = static_cast<uint16_t *>(is_v ? a.c.v : a.c.k) + crow * kHeadDim;
      *reinterpret_cast<uint4 *>(dst + e0) = pack8(x);
      *reinterpret_cast<uint4 *>(dst + e1) = pack8(x + 8);
    }
  }
}

// ------------------------------------------------------------------ decode
// The bytes of the cache bound this: 2 len G d of them per sequence, about R
// products of each, far under the ridge; so mma.sync (heads as the 16 rows)
// suffices for the products and the design is about keeping HBM busy.
//   Work    The 64-key tiles of all sequences, in order, are cut into equal
//           runs: no CTA waits for a longer sequence, whatever the lengths.
//           A run goes to a group of G CTAs, one per KV head: they walk the
//           same tokens side by side, whose rows (and 8-bit scales, 4 bytes
//           of a sector each) lie next to each other.  A sequence inside one
//           run is finished by its CTAs; of one that crosses runs every CTA
//           leaves a part (O, maximum, sum in fp32) and paged_join_kernel
//           adds them up.
//   Loads   Each of the four warps owns 16 keys of a tile and runs its own
//           cp.async ring over them (no block barrier inside a run).  Pages
//           hold a multiple of 16 tokens, so a warp's step lies in one page.
//   Sums    Per warp a running maximum, moved when a step exceeds it by more
//           than 2^8 in P, and a sum, both fp32.  For the product with V
//           P is the sum of two bf16 terms, off by 2^-16 of it: with up to
//           eight heads the second term takes the product's idle rows, which
//           costs nothing; with sixteen it takes products of its own (16 x
//           32K tokens, 128 heads on 8: 337 us against 330).  8-bit: P times
//           the value's scale as f16, the codes' own type in the product,
//           against a reference of its own that lets the weights run up to
//           2^15: f16 keeps their 11 bits down to 2^-25 of the largest, and
//           none above 2^-36 of it is lost.
constexpr int kPdTile = 64;                 // keys per tile, 16 per warp
constexpr int kPdThreads = 128;
constexpr int kPdMaxGrid = 1024;            // CTAs, and so parts, at most
constexpr int kPdRow = kHeadDim + 2;        // floats per head of a part: O, maximum, sum
// 8-bit: the reference of the weights is moved when one passes 2^kPdWTop, to
// where it is 2^kPdWRef.
constexpr float kPdWTop = 15.f, kPdWRef = 11.f;

template <int R, bool FP8>
struct PdCfg {
  // a stage: 16 K rows and 16 V rows (8-bit: and their scales)
  static constexpr int KB = 16 * kHeadDim * (FP8 ? 1 : 2);
  static constexpr int STAGE = 2 * KB + (FP8 ? 128 : 0);
  // An 8-bit cache's limit is the warps' instructions (codes to f16); with up
  // to eight heads the products run with the keys as the 16 rows and the
  // heads as the 8 columns, half as many of them, and V's codes go from their
  // rows into fragments without a detour through shared memory.
  static constexpr bool KM = FP8 && R <= 8;
  static constexpr int NST = 3;
  static constexpr int CTAS = KM ? 4 : FP8 ? 3 : 2;   // per SM (8-bit, 96 x <= 16K tokens: 4 321 us, 3 326 us)
  static constexpr int SCR = FP8 && !KM ? 4096 : 0;   // a step's V rows as f16
  static constexpr int WARP = NST * STAGE + SCR;
  static constexpr int OFF_O = 4 * WARP;       // [R][128] fp32
  static constexpr int OFF_ML = OFF_O + R * kHeadDim * 4;   // [4][16] maxima, [4][16] sums
  static constexpr int OFF_VIS = OFF_ML + 2 * 4 * 16 * 4;   // [4][NST] visible keys
  static constexpr int OFF_SL = OFF_VIS + 4 * NST * 4;   // [4][16] factors of the heads' scores (8-bit, not KM)
  static constexpr int SMEM = OFF_SL + 256;
  static_assert(CTAS * (SMEM + 1024) <= 228 * 1024, "CTAs per SM");
};

__device__ __forceinline__ void cpa16(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cpa4(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cpa_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cpa_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two E4M3 codes (low byte first) as two f16 values (exact).
__device__ __forceinline__ uint32_t f16x2_of_e4m3x2(uint32_t two) {
  uint32_t r;
  const uint16_t in = static_cast<uint16_t>(two);
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(in));
  return r;
}
// Two bf16 values times f as two f16 values.
__device__ __forceinline__ uint32_t f16x2_of_bf16x2(uint32_t w, float f) {
  const __half2 h = __floats2half2_rn(bf16_lo(w) * f, bf16_hi(w) * f);
  return *reinterpret_cast<const uint32_t *>(&h);
}
// The exponent field of the power of two that brings x into [2^14, 2^15), at most
// 2^112: what a query row is multiplied by before it is rounded to f16, so that
// f16 holds rows of any size (elements down to 2^-28 of the row's largest keep
// their bits, the others are off by 2^-39 of it).  2^(254 - field - 127) undoes it.
__device__ __forceinline__ uint32_t f16_lift(float x) { return min(268u - (__float_as_uint(x) >> 23), 239u); }

// Byte of 16-byte granule gr of row r in a stage: rows of 256 bytes (8-bit:
// 128), granules permuted so that eight rows of one granule (8-bit: two
// neighbouring rows of four granules, and four even or odd rows of two) fall
// into different banks.
template <bool FP8>
__device__ __forceinline__ uint32_t swz(int r, int gr) {
  return FP8 ? r * 128 + ((gr ^ (((r & 6) ^ ((r & 1) << 2)))) << 4) : r * 256 + ((gr ^ (r & 7)) << 4);
}
// An 8 x 8 matrix of 16-bit values (row lane / 4, columns 2 (lane % 4), + 1) transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// The fp32 at this CTA's shared address `a` in CTA `rank` of the cluster.
__device__ __forceinline__ float ld_cluster(uint32_t a, uint32_t rank) {
  uint32_t r;
  float v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(r) : "memory");
  return v;
}

// Tokens of a sequence that are attended: 0 when its length is not allowed.
__device__ __forceinline__ int pd_len(const PagedDecodeArgs &a, int b) {
  const int n = a.seq_lens[b];
  return (n < 0 || n > a.Lmax) ? 0 : n;
}

// A place in the list of tiles: (sequence, tile).
struct PdCur {
  int b, t, len;
  __device__ __forceinline__ int tiles() const { return (len + kPdTile - 1) / kPdTile; }
  __device__ __forceinline__ void seek(const PagedDecodeArgs &a) {   // the next sequence with tokens
    while (b < a.B && (len = pd_len(a, b)) == 0) ++b;
  }
  __device__ __forceinline__ void next(const PagedDecodeArgs &a) {
    if (++t < tiles()) return;
    t = 0;
    ++b;
    seek(a);
  }
};

// One chunk of 128 sequences from b0: this thread's tile count, those before
// it in the chunk, and the chunk's total.
__device__ __forceinline__ void pd_scan(const PagedDecodeArgs &a, int b0, long long *s_w, long long &mine,
                                        long long &before, long long &total) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = b0 + tid;
  mine = b < a.B ? (pd_len(a, b) + kPdTile - 1) / kPdTile : 0;
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) s_w[warp] = inc;
  __syncthreads();
  long long base = 0;
  total = 0;
  for (int w = 0; w < 4; ++w) {
    if (w < warp) base += s_w[w];
    total += s_w[w];
  }
  before = base + inc - mine;
  __syncthreads();
}

// CL: the short form.  A cluster of eight CTAs takes one (sequence, KV head),
// an eighth of its tiles each, and joins the parts through distributed shared
// memory: one launch, for calls so short that the second one is felt.
template <int R, bool FP8, bool CL>
__global__ void __launch_bounds__(kPdThreads, (PdCfg<R, FP8>::CTAS)) paged_decode_kernel(const PagedDecodeArgs a) {
  using C = PdCfg<R, FP8>;
  extern __shared__ __align__(128) uint8_t dsm[];
  __shared__ long long s_w[4];
  __shared__ int s_start[2];
  __shared__ float2 s_part[16];        // CL: maximum and sum of each head's part
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g4 = lane >> 2, c = lane & 3;
  if (!CL) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- this CTA's run of tiles [u0, u1)
  long long T = 0, mine, before, total;
  for (int b0 = 0; !CL && b0 < a.B; b0 += 128) {
    pd_scan(a, b0, s_w, mine, before, total);
    T += total;
  }
  const int groups = gridDim.x / a.G;
  const int n_grp = int(T < groups ? T : groups);         // groups that get a run
  const int cta = blockIdx.x, grp = CL ? 0 : cta / a.G, g = CL ? (cta >> 3) % a.G : cta % a.G;
  long long u0 = grp < n_grp ? T * grp / n_grp : 0, u1 = grp < n_grp ? T * (grp + 1) / n_grp : 0;
  if (CL) {
    const int b = (cta >> 3) / a.G, rank = cta & 7, nt = (pd_len(a, b) + kPdTile - 1) / kPdTile;
    u0 = nt * rank / 8;
    u1 = nt * (rank + 1) / 8;
    if (tid == 0) { s_start[0] = b; s_start[1] = int(u0); }
    if (tid < 16) s_part[tid] = make_float2(-INFINITY, 0.f);
  } else if (grp < n_grp) {
    long long base = 0;
    for (int b0 = 0; b0 < a.B; b0 += 128) {
      if (a.B > 128) pd_scan(a, b0, s_w, mine, before, total);   // (else the one scan stands)
      if (u0 >= base + before && u0 < base + before + mine) {
        s_start[0] = b0 + tid;
        s_start[1] = int(u0 - base - before);
      }
      base += total;
      if (base > u0) break;
    }
  }
  __syncthreads();

  int4 meta = make_int4(-1, 0, 0, 0);   // {b, g, parts} of the pair that this CTA's run leaves unfinished
  float *s_o = reinterpret_cast<float *>(dsm + C::OFF_O);
  if (CL ? u0 < u1 : grp < n_grp) {
    const uint32_t sm = static_cast<uint32_t>(__cvta_generic_to_shared(dsm)) + warp * C::WARP;
    uint8_t *smp = dsm + warp * C::WARP;
    float *s_m = reinterpret_cast<float *>(dsm + C::OFF_ML), *s_l = s_m + 64;
    volatile int *s_vis = reinterpret_cast<volatile int *>(dsm + C::OFF_VIS) + warp * C::NST;
    volatile float *s_sl = reinterpret_cast<volatile float *>(dsm + C::OFF_SL) + warp * 16;
    const int pmask = (1 << a.c.page_log2) - 1;
    PdCur ld;
    ld.b = s_start[0]; ld.t = s_start[1];
    ld.len = pd_len(a, ld.b);
    PdCur cu = ld;
    // (no call has 2^31 tiles to a CTA)
    const int n_u = int(u1 - u0);
    int u_ld = 0;
    const int32_t *tab = a.c.table + size_t(ld.b) * a.c.max_pages;
    auto page_of = [&](const PdCur &x) {
      const int key = x.t * kPdTile + warp * 16;
      return key < x.len ? tab[key >> a.c.page_log2] : 0;
    };
    int pg = page_of(ld);
    // this lane's granule: row r0 (then every ROWS-th) of a step, granule gr
    constexpr int GR = FP8 ? 8 : 16, ROWS = 32 / GR, EB = FP8 ? 1 : 2;
    const int r0 = lane / GR, gr = lane % GR;
    const uint32_t rowb = uint32_t(a.G) * (kHeadDim * EB);          // bytes between tokens
    const uint8_t *k0p = static_cast<const uint8_t *>(a.c.k) + size_t(g) * (kHeadDim * EB) + gr * 16;
    const uint8_t *v0p = static_cast<const uint8_t *>(a.c.v) + size_t(g) * (kHeadDim * EB) + gr * 16;
    const float *s0p = FP8 ? (lane < 16 ? a.c.k_scale : a.c.v_scale) + g : nullptr;
    // copies of this warp's 16 keys of the next tile into ring stage st
    auto issue = [&](int st) {
      if (u_ld < n_u) {
        const int key = ld.t * kPdTile + warp * 16;
        int vis = min(16, max(0, ld.len - key));
        if (vis > 0 && (pg < 0 || pg >= a.c.num_pages)) {
          vis = 0;
          if (lane == 0) atomicCAS(a.status, 0, kStatusBadInput);
        }
        // (nothing is read where vis is 0: the token stays inside the pool)
        const unsigned long long tok = vis > 0 ? ((unsigned long long)pg << a.c.page_log2) + (key & pmask) : 0;
        const uint32_t dst = sm + st * C::STAGE;
        if (vis == 16) {
          const unsigned long long off = (tok + r0) * rowb;
          const uint8_t *kp = k0p + off, *vp = v0p + off;
#pragma unroll
          for (int i = 0; i < 16 / ROWS; ++i, kp += ROWS * rowb, vp += ROWS * rowb) {
            const uint32_t d = swz<FP8>(r0 + ROWS * i, gr);
            cpa16(dst + d, kp, 16u);
            cpa16(dst + C::KB + d, vp, 16u);
          }
          if (FP8) cpa4(dst + 2 * C::KB + lane * 4, s0p + (tok + (lane & 15)) * a.G, 4u);
        } else {
          // rows behind the visible ones are filled with zeros, not read
#pragma unroll 1
          for (int i = 0; i < 16 / ROWS; ++i) {
            const int r = r0 + ROWS * i;
            const uint32_t d = swz<FP8>(r, gr), n = r < vis ? 16u : 0u;
            const unsigned long long off = (tok + (r < vis ? r : 0)) * rowb;
            cpa16(dst + d, k0p + off, n);
            cpa16(dst + C::KB + d, v0p + off, n);
          }
          if (FP8) {
            const int r = lane & 15;
            cpa4(dst + 2 * C::KB + lane * 4, s0p + (tok + (r < vis ? r : 0)) * a.G, r < vis ? 4u : 0u);
          }
        }
        if (lane == 0) s_vis[st] = vis;
        if (++u_ld < n_u) {
          const int b = ld.b;
          ld.next(a);
          if (ld.b != b) tab = a.c.table + size_t(ld.b) * a.c.max_pages;
          pg = page_of(ld);   // used at the next issue
        }
      }
      cpa_commit();
    };
#pragma unroll
    for (int st = 0; st < C::NST - 1; ++st) issue(st);

    // running state of the pair: rows g4 and g4 + 8 of the 16 head rows
    // (8-bit: O is kept against mw, the others against m)
    // (KM: heads 2c and 2c + 1 in place of rows g4 and g4 + 8; O's value e of
    // tile d is dim 16 g4 + 2 d + e / 2 of head 2c + e % 2)
    float o[C::KM ? 8 : 16][4], m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f, mw0 = -INFINITY, mw1 = -INFINITY;
#pragma unroll
    for (int d = 0; d < (C::KM ? 8 : 16); ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[d][e] = 0.f;
    uint32_t qf[8][4];
    float sl0 = 0.f, sl1 = 0.f;                     // KM: a.scale_log2 with the lift of this lane's heads undone
    bool fresh = true;                              // a new pair: its queries are to be loaded
    bool head = cu.t > 0;                           // the pair began in an earlier run
    int pair_left = 0;
    int st = 0;
    for (int u = 0; u < n_u; ++u) {
      if (fresh) {
        fresh = false;
        pair_left = cu.tiles() - cu.t;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (C::KM && (e & 1)) continue;   // the B operand's two registers: e 0 and 2
            const int r = g4 + (e & 1) * 8;
            // bf16: dims 16 kk + 2c, +1 (e < 2) and + 8; 8-bit: the order in
            // which a lane's sixteen codes of a granule feed four k steps
            const int d = FP8 ? 16 * (c + 4 * (kk >> 2)) + 4 * (kk & 3) + (e >> 1) * 2 : kk * 16 + 2 * c + (e >> 1) * 8;
            uint32_t w = 0;
            if (r < R) w = *reinterpret_cast<const uint32_t *>(a.q + (size_t(cu.b) * a.H + g * R + r) * kHeadDim + d);
            qf[kk][e] = w;
          }
        if (FP8) {   // to f16, each head's row lifted by its own power of two
          float x[2] = {0.f, 0.f};
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!C::KM || !(e & 1))
                x[e & 1] = fmaxf(x[e & 1], fmaxf(fabsf(bf16_lo(qf[kk][e])), fabsf(bf16_hi(qf[kk][e]))));
#pragma unroll
          for (int i = 1; i < 4; i <<= 1) {
            x[0] = fmaxf(x[0], __shfl_xor_sync(0xffffffffu, x[0], i));
            if (!C::KM) x[1] = fmaxf(x[1], __shfl_xor_sync(0xffffffffu, x[1], i));
          }
          const uint32_t up[2] = {f16_lift(x[0]), f16_lift(x[1])};
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!C::KM || !(e & 1)) qf[kk][e] = f16x2_of_bf16x2(qf[kk][e], __uint_as_float(up[e & 1] << 23));
          const float d0 = __uint_as_float((254u - up[0]) << 23) * a.scale_log2;
          const float d1 = __uint_as_float((254u - up[1]) << 23) * a.scale_log2;
          // KM: this lane loaded head g4, its scores are of heads 2c and 2c + 1.
          // Else through shared memory: the sixteen-head form has no two registers
          // to spare (kept there it spills: 16 x 32K tokens 170 us, 149 this way)
          sl0 = __shfl_sync(0xffffffffu, d0, 8 * c);
          sl1 = __shfl_sync(0xffffffffu, d0, 8 * c + 4);
          if (!C::KM && c == 0) { s_sl[g4] = d0; s_sl[g4 + 8] = d1; }
        }
      }
      cpa_wait<C::NST - 2>();
      __syncwarp();
      const int vis = s_vis[st];
      const uint32_t kb = sm + st * C::STAGE, vb = kb + C::KB;
      if (C::KM && vis > 0) {
        const uint8_t *ks = smp + st * C::STAGE;
        const float *sc = reinterpret_cast<const float *>(ks + 2 * C::KB);
        // S^T: rows are keys g4 and g4 + 8, columns heads 2c and 2c + 1
        float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 r0 = *reinterpret_cast<const uint4 *>(ks + swz<true>(g4, c + 4 * h));
          const uint4 r1 = *reinterpret_cast<const uint4 *>(ks + swz<true>(g4 + 8, c + 4 * h));
          const uint32_t w0[4] = {r0.x, r0.y, r0.z, r0.w}, w1[4] = {r1.x, r1.y, r1.z, r1.w};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint32_t ka[4] = {f16x2_of_e4m3x2(w0[x]), f16x2_of_e4m3x2(w1[x]), f16x2_of_e4m3x2(w0[x] >> 16),
                                    f16x2_of_e4m3x2(w1[x] >> 16)};
            mma_f16(s, ka, qf[4 * h + x][0], qf[4 * h + x][2]);
          }
        }
        const float k0 = sc[g4], k1 = sc[g4 + 8];
        const float v0 = sc[16 + g4], v1 = sc[24 + g4];
        // log2 units (the factors first: the scale brings the lift's undoing back into range)
        s[0] *= k0 * sl0; s[1] *= k0 * sl1; s[2] *= k1 * sl0; s[3] *= k1 * sl1;
        if (vis < 16) {
          if (g4 >= vis) s[0] = s[1] = -INFINITY;
          if (g4 + 8 >= vis) s[2] = s[3] = -INFINITY;
        }
        const float lv0 = __log2f(fabsf(v0)), lv1 = __log2f(fabsf(v1));
        float x0 = fmaxf(s[0], s[2]), x1 = fmaxf(s[1], s[3]);
        float y0 = fmaxf(s[0] + lv0, s[2] + lv1), y1 = fmaxf(s[1] + lv0, s[3] + lv1);
#pragma unroll
        for (int i = 4; i < 32; i <<= 1) {
          x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, i));
          x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, i));
          y0 = fmaxf(y0, __shfl_xor_sync(0xffffffffu, y0, i));
          y1 = fmaxf(y1, __shfl_xor_sync(0xffffffffu, y1, i));
        }
        // two references as below: m for the sums, mw for the weights that
        // multiply V's codes (P |scale|, f16); both in log2 units here
        const bool up0 = m0 == -INFINITY || x0 - m0 > 8.f, up1 = m1 == -INFINITY || x1 - m1 > 8.f;
        const bool wu0 = y0 > -INFINITY && (mw0 == -INFINITY || y0 - mw0 > kPdWTop);
        const bool wu1 = y1 > -INFINITY && (mw1 == -INFINITY || y1 - mw1 > kPdWTop);
        if (__any_sync(0xffffffffu, up0 || up1 || wu0 || wu1)) {
          if (up0) { l0 *= m0 == -INFINITY ? 0.f : fast_exp2(m0 - x0); m0 = x0; }
          if (up1) { l1 *= m1 == -INFINITY ? 0.f : fast_exp2(m1 - x1); m1 = x1; }
          const float al0 = wu0 ? (mw0 == -INFINITY ? 0.f : fast_exp2(mw0 - (y0 - kPdWRef))) : 1.f;
          const float al1 = wu1 ? (mw1 == -INFINITY ? 0.f : fast_exp2(mw1 - (y1 - kPdWRef))) : 1.f;
          if (wu0) mw0 = y0 - kPdWRef;
          if (wu1) mw1 = y1 - kPdWRef;
#pragma unroll
          for (int d = 0; d < 8; ++d) {
            o[d][0] *= al0; o[d][2] *= al0;
            o[d][1] *= al1; o[d][3] *= al1;
          }
        }
        l0 += fast_exp2(s[0] - m0) + fast_exp2(s[2] - m0);
        l1 += fast_exp2(s[1] - m1) + fast_exp2(s[3] - m1);
        const float n0 = mw0 == -INFINITY ? 0.f : -mw0, n1 = mw1 == -INFINITY ? 0.f : -mw1;
        const __half2 p0 = __floats2half2_rn(copysignf(fast_exp2(s[0] + lv0 + n0), v0),
                                             copysignf(fast_exp2(s[1] + lv0 + n1), v0));
        const __half2 p1 = __floats2half2_rn(copysignf(fast_exp2(s[2] + lv1 + n0), v1),
                                             copysignf(fast_exp2(s[3] + lv1 + n1), v1));
        const uint32_t b0 = transpose8(*reinterpret_cast<const uint32_t *>(&p0));
        const uint32_t b1 = transpose8(*reinterpret_cast<const uint32_t *>(&p1));
        // O^T += V^T P^T: this lane's dims are 16 g4 .. + 15 (rows g4 and g4 + 8
        // of the eight tiles), its keys 2c, 2c + 1, 2c + 8, 2c + 9
        const uint8_t *vr = ks + C::KB;
        const uint4 q0 = *reinterpret_cast<const uint4 *>(vr + swz<true>(2 * c, g4));
        const uint4 q1 = *reinterpret_cast<const uint4 *>(vr + swz<true>(2 * c + 1, g4));
        const uint4 q2 = *reinterpret_cast<const uint4 *>(vr + swz<true>(2 * c + 8, g4));
        const uint4 q3 = *reinterpret_cast<const uint4 *>(vr + swz<true>(2 * c + 9, g4));
        const uint32_t w0[4] = {q0.x, q0.y, q0.z, q0.w}, w1[4] = {q1.x, q1.y, q1.z, q1.w};
        const uint32_t w2[4] = {q2.x, q2.y, q2.z, q2.w}, w3[4] = {q3.x, q3.y, q3.z, q3.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t e0 = __byte_perm(w0[j], w1[j], h ? 0x7362 : 0x5140);
            const uint32_t e1 = __byte_perm(w2[j], w3[j], h ? 0x7362 : 0x5140);
            const uint32_t va[4] = {f16x2_of_e4m3x2(e0), f16x2_of_e4m3x2(e0 >> 16), f16x2_of_e4m3x2(e1),
                                    f16x2_of_e4m3x2(e1 >> 16)};
            mma_f16(o[2 * j + h], va, b0, b1);
          }
      }
      if (!C::KM && vis > 0) {
        const float unit = FP8 ? 1.f : a.scale_log2;   // of the scores below, in log2
        float s[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[i][e] = 0.f;
        float vs[2][2] = {{1.f, 1.f}, {1.f, 1.f}};
        if (FP8) {
          const uint8_t *ks = smp + st * C::STAGE;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = i * 8 + g4;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint4 w = *reinterpret_cast<const uint4 *>(ks + swz<true>(r, c + 4 * h));
              const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int x = 0; x < 4; ++x)
                mma_f16(s[i], qf[4 * h + x], f16x2_of_e4m3x2(ww[x]), f16x2_of_e4m3x2(ww[x] >> 16));
            }
          }
          const float *sc = reinterpret_cast<const float *>(ks + 2 * C::KB);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float2 k2 = *reinterpret_cast<const float2 *>(sc + i * 8 + 2 * c);
            const float2 v2 = *reinterpret_cast<const float2 *>(sc + 16 + i * 8 + 2 * c);
            const float f0 = s_sl[g4], f1 = s_sl[g4 + 8];   // (log2 units, as above)
            s[i][0] *= k2.x * f0; s[i][1] *= k2.y * f0; s[i][2] *= k2.x * f1; s[i][3] *= k2.y * f1;
            vs[i][0] = v2.x; vs[i][1] = v2.y;
          }
          // V's codes as f16 rows in the scratch: the two granules that a
          // granule of codes makes lie 128 bytes apart (no bank conflicts)
          const uint8_t *vr = smp + st * C::STAGE + C::KB;
          uint8_t *scr = smp + C::NST * C::STAGE;
          __syncwarp();   // the last step's reads of the scratch
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = (lane >> 3) + 4 * i, gr = lane & 7;
            const uint4 w = *reinterpret_cast<const uint4 *>(vr + swz<true>(r, gr));
            uint4 *d = reinterpret_cast<uint4 *>(scr + r * 256 + ((gr ^ (r & 7)) << 4));
            d[0] = make_uint4(f16x2_of_e4m3x2(w.x), f16x2_of_e4m3x2(w.x >> 16), f16x2_of_e4m3x2(w.y),
                              f16x2_of_e4m3x2(w.y >> 16));
            d[8] = make_uint4(f16x2_of_e4m3x2(w.z), f16x2_of_e4m3x2(w.z >> 16), f16x2_of_e4m3x2(w.w),
                              f16x2_of_e4m3x2(w.w >> 16));
          }
          __syncwarp();
        } else {
          // matrices: (keys 0-7, dims 0-7), (keys 0-7, dims 8-15), (keys 8-15, ...), ...
          const int r = (lane & 7) + ((lane >> 4) << 3), h = (lane >> 3) & 1;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            uint32_t b[4];
            ldsm4(b, kb + r * 256 + (((2 * kk + h) ^ (r & 7)) << 4));
            mma_bf16(s[0], qf[kk], b[0], b[1]);
            mma_bf16(s[1], qf[kk], b[2], b[3]);
          }
        }
        if (vis < 16) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (i * 8 + 2 * c + (e & 1) >= vis) s[i][e] = -INFINITY;
        }
        float x0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
        float x1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
#pragma unroll
        for (int i = 1; i < 4; i <<= 1) {
          x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, i));
          if (R > 8) x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, i));
        }
        if (R <= 8) x1 = m1;   // rows 8-15 hold no head: their zeros move nothing
        // (a step with a visible key has a finite maximum, so m0 and m1 are finite behind it)
        const bool up0 = m0 == -INFINITY || (x0 - m0) * unit > 8.f;
        const bool up1 = R > 8 && (m1 == -INFINITY || (x1 - m1) * unit > 8.f);
        if (__any_sync(0xffffffffu, up0 || up1)) {
          const float al0 = up0 ? (m0 == -INFINITY ? 0.f : fast_exp2((m0 - x0) * unit)) : 1.f;
          const float al1 = up1 ? (m1 == -INFINITY ? 0.f : fast_exp2((m1 - x1) * unit)) : 1.f;
          if (up0) m0 = x0;
          if (up1) m1 = x1;
          l0 *= al0;
          l1 *= al1;
          if (!FP8) {
#pragma unroll
            for (int d = 0; d < 16; ++d) {
              o[d][0] *= al0; o[d][1] *= al0;
              o[d][2] *= R > 8 ? al1 : al0; o[d][3] *= R > 8 ? al1 : al0;
            }
          }
        }
        const float n0 = -m0 * unit, n1 = R > 8 ? -m1 * unit : 0.f;
        uint32_t pa[4], pb[4];
        float lv[2][2], w0 = 0.f, w1 = 0.f;
        if (FP8) {
          // the weights that multiply V's codes are P |scale|, in f16, against
          // a reference of their own (log2), whatever the scales
          float y0 = -INFINITY, y1 = -INFINITY;
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              lv[i][e] = __log2f(fabsf(vs[i][e]));
              y0 = fmaxf(y0, fmaf(s[i][e], unit, lv[i][e]));
              if (R > 8) y1 = fmaxf(y1, fmaf(s[i][2 + e], unit, lv[i][e]));
            }
#pragma unroll
          for (int i = 1; i < 4; i <<= 1) {
            y0 = fmaxf(y0, __shfl_xor_sync(0xffffffffu, y0, i));
            if (R > 8) y1 = fmaxf(y1, __shfl_xor_sync(0xffffffffu, y1, i));
          }
          const bool wu0 = y0 > -INFINITY && (mw0 == -INFINITY || y0 - mw0 > kPdWTop);
          const bool wu1 = R > 8 && y1 > -INFINITY && (mw1 == -INFINITY || y1 - mw1 > kPdWTop);
          if (__any_sync(0xffffffffu, wu0 || wu1)) {
            const float al0 = wu0 ? (mw0 == -INFINITY ? 0.f : fast_exp2(mw0 - (y0 - kPdWRef))) : 1.f;
            const float al1 = wu1 ? (mw1 == -INFINITY ? 0.f : fast_exp2(mw1 - (y1 - kPdWRef))) : 1.f;
            if (wu0) mw0 = y0 - kPdWRef;
            if (wu1) mw1 = y1 - kPdWRef;
#pragma unroll
            for (int d = 0; d < 16; ++d) {
              o[d][0] *= al0; o[d][1] *= al0;
              if (R > 8) { o[d][2] *= al1; o[d][3] *= al1; }
            }
          }
          w0 = mw0 == -INFINITY ? 0.f : -mw0;
          w1 = mw1 == -INFINITY ? 0.f : -mw1;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int h = 0; h < (R > 8 ? 2 : 1); ++h) {   // rows g4, then g4 + 8
            const float z0 = s[i][2 * h] * unit, z1 = s[i][2 * h + 1] * unit;
            const float n = h ? n1 : n0, w = h ? w1 : w0;
            const float p0 = fast_exp2(z0 + n), p1 = fast_exp2(z1 + n);
            if (h) l1 += p0 + p1; else l0 += p0 + p1;
            if (FP8) {
              const __half2 x = __floats2half2_rn(copysignf(fast_exp2(z0 + lv[i][0] + w), vs[i][0]),
                                                  copysignf(fast_exp2(z1 + lv[i][1] + w), vs[i][1]));
              pa[2 * i + h] = *reinterpret_cast<const uint32_t *>(&x);
            } else {
              // P in two bf16 terms; the second takes the rows that hold no head
              const uint32_t hi = pack_bf16x2(p0, p1);
              const uint32_t lo = pack_bf16x2(p0 - bf16_lo(hi), p1 - bf16_hi(hi));
              pa[2 * i + h] = hi;
              if (R <= 8) pa[2 * i + 1] = lo; else pb[2 * i + h] = lo;
            }
          }
        // matrices: (keys 0-7, dims d), (keys 8-15, dims d), (keys 0-7, dims d + 8), ...
        const int r = lane & 15, h = lane >> 4;
        const uint32_t vrow = (FP8 ? sm + C::NST * C::STAGE : vb) + r * 256;
#pragma unroll
        for (int d = 0; d < 16; d += 2) {
          uint32_t b[4];
          if (FP8) {
            ldsm4_t(b, vrow + (((d >> 1) ^ (r & 7)) << 4) + h * 128);
            mma_f16(o[d], pa, b[0], b[1]);
            mma_f16(o[d + 1], pa, b[2], b[3]);
          } else {
            ldsm4_t(b, vrow + (((d + h) ^ (r & 7)) << 4));
            mma_bf16(o[d], pa, b[0], b[1]);
            mma_bf16(o[d + 1], pa, b[2], b[3]);
            if (R > 8) {
              mma_bf16(o[d], pb, b[0], b[1]);
              mma_bf16(o[d + 1], pb, b[2], b[3]);
            }
          }
        }
      }
      __syncwarp();
      issue(st == 0 ? C::NST - 1 : st - 1);   // into the stage that was read last time
      st = st + 1 == C::NST ? 0 : st + 1;

      // ---- the pair's end, or the run's: join the four warps
      const bool done = --pair_left == 0;
      if (done || u + 1 == n_u) {
        const int h0 = C::KM ? 2 * c : g4, h1 = C::KM ? 2 * c + 1 : g4 + 8;   // this lane's heads
#pragma unroll
        for (int i = C::KM ? 4 : 1; i < (C::KM ? 32 : 4); i <<= 1) {
          l0 += __shfl_xor_sync(0xffffffffu, l0, i);
          l1 += __shfl_xor_sync(0xffffffffu, l1, i);
        }
        if (FP8) {   // from log2 units back to those of the scores
          m0 /= a.scale_log2;
          m1 /= a.scale_log2;
        }
        if (C::KM ? g4 == 0 : c == 0) {
          s_m[warp * 16 + h0] = m0; s_m[warp * 16 + h1] = m1;
          s_l[warp * 16 + h0] = l0; s_l[warp * 16 + h1] = l1;
        }
        __syncthreads();
        float M0 = -INFINITY, M1 = -INFINITY;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          M0 = fmaxf(M0, s_m[w * 16 + h0]);
          M1 = fmaxf(M1, s_m[w * 16 + h1]);
        }
        // O's unit, 2^(scale m) (8-bit: 2^mw), to 2^(scale M)
        const float unit0 = FP8 ? mw0 : m0 * a.scale_log2, unit1 = FP8 ? mw1 : m1 * a.scale_log2;
        const float f0 = unit0 == -INFINITY ? 0.f : fast_exp2(unit0 - M0 * a.scale_log2);
        const float f1 = unit1 == -INFINITY ? 0.f : fast_exp2(unit1 - M1 * a.scale_log2);
        if (!FP8 && R <= 8) {   // the products of P's two terms (an infinite value's second one is NaN)
#pragma unroll
          for (int d = 0; d < 16; ++d) {
            o[d][0] = fabsf(o[d][0]) == INFINITY ? o[d][0] : o[d][0] + o[d][2];
            o[d][1] = fabsf(o[d][1]) == INFINITY ? o[d][1] : o[d][1] + o[d][3];
          }
        }
        // warp by warp, so that the sum's order is always the same
        for (int w = 0; w < 4; ++w) {
          if (C::KM && w == warp) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (2 * c + h >= R) continue;
              float4 *x = reinterpret_cast<float4 *>(s_o + (2 * c + h) * kHeadDim + 16 * g4);
              const float f = h ? f1 : f0;
#pragma unroll
              for (int d = 0; d < 4; ++d) {
                const float4 y = w ? x[d] : make_float4(0.f, 0.f, 0.f, 0.f);
                x[d] = make_float4(y.x + o[2 * d][h] * f, y.y + o[2 * d][2 + h] * f, y.z + o[2 * d + 1][h] * f,
                                   y.w + o[2 * d + 1][2 + h] * f);
              }
            }
          }
          if (!C::KM && w == warp) {
#pragma unroll
            for (int d = 0; d < 16; ++d) {
              if (g4 < R) {
                float2 *x = reinterpret_cast<float2 *>(s_o + g4 * kHeadDim + d * 8 + 2 * c);
                const float2 y = w ? *x : make_float2(0.f, 0.f);
                *x = make_float2(y.x + o[d][0] * f0, y.y + o[d][1] * f0);
              }
              if (g4 + 8 < R) {
                float2 *x = reinterpret_cast<float2 *>(s_o + (g4 + 8) * kHeadDim + d * 8 + 2 * c);
                const float2 y = w ? *x : make_float2(0.f, 0.f);
                *x = make_float2(y.x + o[d][2] * f1, y.y + o[d][3] * f1);
              }
            }
          }
          __syncthreads();
        }
        const bool whole = done && !head;
        // an unfinished pair: slot 0 when it began in an earlier run, else 1
        float *part = a.parts + size_t(2 * cta + (head ? 0 : 1)) * R * kPdRow;
        for (int r = 0; r < R; ++r) {
          float M = -INFINITY, L = 0.f;
#pragma unroll
          for (int w = 0; w < 4; ++w) M = fmaxf(M, s_m[w * 16 + r]);
#pragma unroll
          for (int w = 0; w < 4; ++w)
            L += s_m[w * 16 + r] == -INFINITY ? 0.f : s_l[w * 16 + r] * fast_exp2((s_m[w * 16 + r] - M) * a.scale_log2);
          const float x = s_o[r * kHeadDim + tid];
          if (CL) {
            if (tid == 0) s_part[r] = make_float2(M, L);
          } else if (whole) {
            const size_t orow = size_t(cu.b) * a.H + g * R + r;
            reinterpret_cast<__nv_bfloat16 *>(a.out)[orow * kHeadDim + tid] = __float2bfloat16(L == 0.f ? 0.f : x / L);
            if (tid == 0 && a.lse) a.lse[orow] = L == 0.f ? -INFINITY : M * a.scale + logf(L);
          } else {
            part[r * kPdRow + tid] = x;
            if (tid == 0) { part[r * kPdRow + kHeadDim] = M; part[r * kPdRow + kHeadDim + 1] = L; }
          }
        }
        if (!CL && !done && !head) {
          // the pair ends with tile u + pair_left: parts up to the group whose run holds that
          const long long e = u0 + u + 1 + pair_left;
          meta = make_int4(cu.b, g, int((e * n_grp + T - 1) / T - 1) - grp + 1, 0);
        }
        __syncthreads();   // s_o, s_m and s_l are free again
        m0 = m1 = mw0 = mw1 = -INFINITY;
        l0 = l1 = 0.f;
#pragma unroll
        for (int d = 0; d < (C::KM ? 8 : 16); ++d)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[d][e] = 0.f;
        fresh = true;
        head = false;
      }
      if (u + 1 < n_u) cu.next(a);
    }
    cpa_wait<0>();
  }
  if (CL) {
    // every CTA of the cluster joins the heads r = rank, rank + 8
    asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
    for (int r = cta & 7; r < R; r += 8) {
      const uint32_t po = static_cast<uint32_t>(__cvta_generic_to_shared(s_o + r * kHeadDim + tid));
      const uint32_t pm = static_cast<uint32_t>(__cvta_generic_to_shared(s_part + r));
      float m[8], l[8], x[8];
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        m[p] = ld_cluster(pm, p);
        l[p] = ld_cluster(pm + 4, p);
        x[p] = ld_cluster(po, p);
      }
      float M = -INFINITY, L = 0.f, O = 0.f;
#pragma unroll
      for (int p = 0; p < 8; ++p) M = fmaxf(M, m[p]);
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        const float f = m[p] == -INFINITY ? 0.f : fast_exp2((m[p] - M) * a.scale_log2);
        L = fmaf(f, l[p], L);
        O = m[p] == -INFINITY ? O : fmaf(f, x[p], O);   // (a CTA without tiles left x unwritten)
      }
      const size_t orow = size_t((cta >> 3) / a.G) * a.H + g * R + r;
      reinterpret_cast<__nv_bfloat16 *>(a.out)[orow * kHeadDim + tid] = __float2bfloat16(L == 0.f ? 0.f : O / L);
      if (tid == 0 && a.lse) a.lse[orow] = L == 0.f ? -INFINITY : M * a.scale + logf(L);
    }
    asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
    if ((cta & 7) == 0 && g == 0 && tid == 0) {
      const int n = a.seq_lens[(cta >> 3) / a.G];
      if (n < 0 || n > a.Lmax) atomicCAS(a.status, 0, kStatusBadInput);
    }
    return;
  }
  if (tid == 0) a.meta[cta] = meta;
  // sequences without tokens: out 0, lse -inf (and a word about bad lengths)
  for (int b = cta * 4 + warp; b < a.B; b += gridDim.x * 4) {
    const int n = a.seq_lens[b];
    if (n > 0 && n <= a.Lmax) continue;
    if (n != 0 && lane == 0) atomicCAS(a.status, 0, kStatusBadInput);
    for (int x = lane; x < a.H * (kHeadDim / 8); x += 32)
      reinterpret_cast<uint4 *>(a.out + size_t(b) * a.H * kHeadDim)[x] = make_uint4(0u, 0u, 0u, 0u);
    if (a.lse)
      for (int x = lane; x < a.H; x += 32) a.lse[size_t(b) * a.H + x] = -INFINITY;
  }
}

// Joins the parts of the pair that CTA blockIdx.x of the decode left
// unfinished (its slot 1, then slot 0 of the following groups' CTAs of the
// same KV head), for one head:
// out = sum_p 2^(s (M_p - M)) O_p / sum_p 2^(s (M_p - M)) L_p.
__global__ void __launch_bounds__(512) paged_join_kernel(const PagedDecodeArgs a, int R) {
  __shared__ float s_x[4][kHeadDim], s_l[4], s_max[16];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int cta = blockIdx.x, r = blockIdx.y, tid = threadIdx.x;
  const int4 meta = a.meta[cta];
  if (meta.x < 0) return;
  const int n = meta.z;
  auto part = [&](int p) { return a.parts + (size_t(p == 0 ? 2 * cta + 1 : 2 * (cta + p * a.G)) * R + r) * kPdRow; };
  float M = -INFINITY;
  for (int p = tid; p < n; p += 512) M = fmaxf(M, __ldcg(part(p) + kHeadDim));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if ((tid & 31) == 0) s_max[tid >> 5] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 16; ++w) M = fmaxf(M, s_max[w]);
  const int grp = tid >> 7, d = tid & 127;
  float x = 0.f, l = 0.f;
#pragma unroll 4
  for (int p = grp; p < n; p += 4) {
    const float *q = part(p);
    const float mp = __ldcg(q + kHeadDim), lp = __ldcg(q + kHeadDim + 1), op = __ldcg(q + d);
    const float f = mp == -INFINITY ? 0.f : fast_exp2((mp - M) * a.scale_log2);
    x = fmaf(f, op, x);
    l = fmaf(f, lp, l);
  }
  s_x[grp][d] = x;
  if (d == 0) s_l[grp] = l;
  __syncthreads();
  if (grp) return;
  x = (s_x[0][d] + s_x[1][d]) + (s_x[2][d] + s_x[3][d]);
  l = (s_l[0] + s_l[1]) + (s_l[2] + s_l[3]);
  const size_t orow = size_t(meta.x) * a.H + meta.y * R + r;
  reinterpret_cast<__nv_bfloat16 *>(a.out)[orow * kHeadDim + d] = __float2bfloat16(l == 0.f ? 0.f : x / l);
  if (d == 0 && a.lse) a.lse[orow] = l == 0.f ? -INFINITY : M * a.scale + logf(l);
}

template <int R, bool FP8>
cudaError_t launch_decode_rt(const PagedDecodeArgs &a, int num_sms, cudaStream_t st) {
  constexpr int smem = PdCfg<R, FP8>::SMEM;
  // The short form, in microseconds against the split one (in a graph): 1
  // sequence, 2 KV heads of 2000 tokens 8.8 / 10.1; 4, 8 of 1000 8.0 / 11.2, of
  // 4000 13.4 / 16.7; but 8, 8 of 1000 14.3 / 13.8 and 1, 8 of 8000 15.7 / 14.3.
  if (a.B <= 32 / a.G && a.Lmax <= 4096) {
    auto kern = paged_decode_kernel<R, FP8, true>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(a.B) * a.G * 8);
    cfg.blockDim = dim3(kPdThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 8;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a);
  }
  auto kern = paged_decode_kernel<R, FP8, false>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  // groups of one CTA per KV head: as many as are resident at once, no more
  // than there can be tiles (Lmax tokens in each sequence)
  const long long most = (long long)a.B * ((a.Lmax + kPdTile - 1) / kPdTile);
  long long groups = PdCfg<R, FP8>::CTAS * num_sms / a.G;
  if (groups > kPdMaxGrid / a.G) groups = kPdMaxGrid / a.G;
  if (groups > most) groups = most;
  if (groups < 1) groups = 1;
  const int grid = int(groups) * a.G;
  kern<<<grid, kPdThreads, smem, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, R);
  cfg.blockDim = dim3(512);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_join_kernel, a, R);
}

template <int R>
cudaError_t launch_decode_r(const PagedDecodeArgs &a, int num_sms, cudaStream_t st) {
  return a.c.k_scale ? launch_decode_rt<R, true>(a, num_sms, st) : launch_decode_rt<R, false>(a, num_sms, st);
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
  switch (a.H / a.G) {
    case 1: return launch_decode_r<1>(a, num_sms, st);
    case 2: return launch_decode_r<2>(a, num_sms, st);
    case 4: return launch_decode_r<4>(a, num_sms, st);
    case 8: return launch_decode_r<8>(a, num_sms, st);
    case 16: return launch_decode_r<16>(a, num_sms, st);
    default: return cudaErrorInvalidValue;
  }
}

size_t paged_decode_parts_floats(int R) { return size_t(2) * kPdMaxGrid * R * kPdRow; }
int paged_decode_max_ctas() { return kPdMaxGrid; }

}  // namespace msa
