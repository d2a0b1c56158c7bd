// Dense causal attention over packed sequences, forward.
//   out = softmax(scale Q K^T) V per (sequence, head), the i-th of n query
//   rows of a sequence with m keys seeing its first m - n + i + 1 keys.
//
//   dense_plan_kernel  checks cu_q and cu_k (a batch that is not ascending
//                 inside the buffers is refused whole), writes each
//                 sequence's {q0, nq, k0, nk} and the list of work items.
//   dense_fwd_kernel   one work item is 256/R consecutive queries x the R
//                 heads of one KV head: two 128-row tiles, A and B, that
//                 sweep the same key tiles (128 keys) once:
//                   S = Q K^T           UMMA into the tile's 128 TMEM columns
//                   P = exp2(S - mr)    as bf16 over S's first 64 columns,
//                                       mr a running reference maximum
//                   O += P V            UMMA, A operand P from TMEM
//
// The tensor work of one (tile, key tile) is 2 x 128^3 products, 1024 cycles;
// its 128 x 128 exponentials take 1024 cycles of the SM's 16-a-cycle unit.
// The two tiles take turns: one's softmax runs under the other's products.
// A tile's chain (softmax 1700 cycles, then O += P V and the next S, 1400
// with the hand-overs) sets the pace: S and P share TMEM columns (2 x 128 for
// S and 2 x 128 for O are all there is), so S cannot run ahead.
// Measured: 32K tokens, 8 heads on 1 KV head, 1.70 ms from idle (1294
// TFLOP/s, 0.78 of burst bf16) and 1.91 ms in a long power-capped run.
// Tried and slower, each against its own start:
//   - a quarter of the exponentials as polynomials on the FMA pipe, 1.98 ms
//     against 1.94 (a packed FMA takes two issue slots);
//   - P handed over in halves, 1.81 against 1.70 (the issuer waits inside a
//     tile while the other tile's product could go);
//   - two softmax warpgroups per tile, 2.61 against 2.12;
//   - an issuer per tile, 2.26 against 1.71 (both chains then finish late);
//   - S held back to interleave it with the other tile's O, 3.22 against 2.12
//     (the tiles fall into step);
//   - S in two buffers of 64 keys, ahead of the products into O: 2.83 against
//     1.65, with an issuer per tile 1.82 (a product of N = 64 takes the issuer
//     as long as one of 128);
//   - the next item's first S right behind each tile's last product, 1.82
//     against 1.67.
// P is rounded to bf16 for its product with V (both operands of a UMMA have one
// type); the row's sum takes it unrounded, in fp32.
//
// Roles (one persistent CTA per SM, four warpgroups):
//   warp 0     TMA producer: the tiles' Q, then K and V of each key tile, into
//              a ring of five 32 KB tiles.
//   warp 1     TMEM owner; one thread issues the UMMAs.  Per key tile j:
//              O_A += P_A V_j, S_A of j+1, O_B += P_B V_j, S_B of j+1.  UMMAs
//              complete in issue order, so S_A may overwrite P_A behind the
//              product that reads it, and a finished S_A(j+1) means a
//              finished O_A(j).  What this thread does between two UMMAs is
//              on the critical path: descriptors are stepped, not encoded,
//              and the ring position is kept, not divided out (-15% time).
//   warp 2     clears the rows of V behind a sequence's last key.
//   warps 4-7, 8-11  softmax of tile A and tile B, one row per thread.  mr
//              moves only when a tile raises the row's maximum by more than
//              2^8 in P; O and the row's sum are then scaled in place, a few
//              times per row at most.
//   warps 12-15  epilogue of both tiles: O / l as bf16 and lse, while the
//              softmax is at the next item.
#include <cuda.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "dense.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace msa {

namespace {

// ------------------------------------------------------------------ plan
constexpr int kPlanBins = 1024;

// Sum of v over the block's earlier threads, and the block's total.
__device__ __forceinline__ int block_exclusive(int v, int *s_warp, int &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  __syncthreads();   // s_warp may still be read by the last call
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    int w = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += x;
    }
    s_warp[lane] = w;
  }
  __syncthreads();
  total = s_warp[31];
  return inc - v + (warp ? s_warp[warp - 1] : 0);
}

// {-lse log2 e, -D} of rows row0 .. (D = dout . out), two rows per warp and
// step, 16 bytes of out and of dout per lane; two steps' loads are in flight.
__device__ __forceinline__ void row_stats(const DenseArgs &a, long long first, long long stride, int lane) {
  const long long rows = (long long)a.nq * a.H;
  const int half = lane >> 4;
  for (long long r0 = first * 4; r0 < rows; r0 += stride * 4) {
    uint4 x[2], y[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const long long r = min(r0 + 2 * i + half, rows - 1);
      x[i] = reinterpret_cast<const uint4 *>(a.out + r * kHeadDim)[lane & 15];
      y[i] = reinterpret_cast<const uint4 *>(a.dout + r * kHeadDim)[lane & 15];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t xs[4] = {x[i].x, x[i].y, x[i].z, x[i].w}, ys[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s = fmaf(bf16_lo(xs[e]), bf16_lo(ys[e]), s);
        s = fmaf(bf16_hi(xs[e]), bf16_hi(ys[e]), s);
      }
#pragma unroll
      for (int m = 8; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
      const long long r = r0 + 2 * i + half;
      if ((lane & 15) == 0 && r < rows) a.stat[r] = make_float2(-a.lse[r] * 1.4426950408889634f, -s);
    }
  }
}

// One CTA per list: the items of `per` queries (block 0) and the key tiles of
// 128 keys (block 1, for the backward); the other blocks make the backward's
// row statistics meanwhile.  Items are sorted by their number of
// key tiles (query tiles of qpi queries), in at most 1024 steps of equal
// width (a counting sort; the order inside a step does not matter, an item's
// result depends on nothing but the item).
__global__ void __launch_bounds__(1024) dense_plan_kernel(const DenseArgs a, int per, int qpi) {
  if (blockIdx.x > 1) {
    row_stats(a, (long long)(blockIdx.x - 2) * 32 + (threadIdx.x >> 5), (long long)(gridDim.x - 2) * 32,
              threadIdx.x & 31);
    return;
  }
  const bool keys = blockIdx.x == 1;
  int *prefix = keys ? a.prefix_k : a.prefix;
  int2 *items = keys ? a.items_k : a.items;
  const int max_items = keys ? a.max_items_k : a.max_items;
  if (keys) per = 128;
  __shared__ int s_warp[32];
  __shared__ int s_bin[kPlanBins];
  const int tid = threadIdx.x;
  grid_dep_launch();
  int bad = 0, most = 0;
  for (int b = tid; b < a.B; b += 1024) {
    const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1], k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
    bad |= q0 < 0 || q1 < q0 || q1 > a.nq || k0 < 0 || k1 < k0 || k1 > a.nk;
    most = max(most, keys ? (q1 - q0 + qpi - 1) / qpi : (k1 - k0 + 127) / 128);
  }
  bad = __syncthreads_or(bad);
  if (bad && tid == 0 && !keys) atomicCAS(a.status, 0, kStatusBadInput);
  s_bin[tid] = 0;
  // the longest sequence sets the width of a step
  for (int o = 16; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
  if ((tid & 31) == 0) s_warp[tid >> 5] = most;
  __syncthreads();
  for (int w = 0; w < 32; ++w) most = max(most, s_warp[w]);
  const int width = most / kPlanBins + 1;
  int base = 0;
  for (int b0 = 0; b0 < a.B; b0 += 1024) {
    const int b = b0 + tid;
    int4 s = make_int4(0, 0, 0, 0);
    if (b < a.B && !bad) {
      s.x = a.cu_q[b];
      s.y = a.cu_q[b + 1] - s.x;
      s.z = a.cu_k[b];
      s.w = a.cu_k[b + 1] - s.z;
    }
    int total;
    const int before = block_exclusive(ceil_div(keys ? s.w : s.y, per), s_warp, total);
    if (b < a.B) {
      if (!keys) a.seqs[b] = s;
      prefix[b] = base + before;
    }
    base += total;
  }
  if (tid == 0) *(keys ? a.n_items_k : a.n_items) = base;
  if (tid == 0 && keys) *a.next_q = 0;
  __syncthreads();
  __threadfence_block();
  // item x: its sequence (the last b with prefix[b] <= x) and place in it
  auto item_of = [&](int x, int &bin) {
    int lo = 0, hi = a.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (prefix[mid] <= x) lo = mid; else hi = mid - 1;
    }
    const int n = a.cu_q[lo + 1] - a.cu_q[lo], m = a.cu_k[lo + 1] - a.cu_k[lo];
    const int at = x - prefix[lo];
    // queries that see the key tile, in tiles; or keys of the item's last row, in tiles
    const int cost = keys ? (n - max(0, at * 128 - (m - n)) + qpi - 1) / qpi
                          : (m - n + min(n, (at + 1) * per) + 127) / 128;
    bin = kPlanBins - 1 - min(kPlanBins - 1, max(0, cost) / width);
    return make_int2(lo, at);
  };
  for (int x = tid; x < base; x += 1024) {
    int bin;
    item_of(x, bin);
    atomicAdd(&s_bin[bin], 1);
  }
  __syncthreads();
  int total;
  const int mine = s_bin[tid];
  const int first = block_exclusive(mine, s_warp, total);
  s_bin[tid] = first;
  __syncthreads();
  for (int x = tid; x < base; x += 1024) {
    int bin;
    const int2 it = item_of(x, bin);
    const int at = atomicAdd(&s_bin[bin], 1);
    if (at < max_items) items[at] = it;
  }
}

// ------------------------------------------------------------------ forward
constexpr int kFThreads = 512;
constexpr int kFRegsRest = 64, kFRegsSoftmax = 192;   // 256 threads each: 512 * 128 in all
constexpr int kFTile = 32768;                    // 128 rows x 256 B
constexpr int kFNkv = 5;                         // K/V ring depth
constexpr int kFSQ = 0;                          // two Q tiles
constexpr int kFSKV = 2 * kFTile;
constexpr int kFSmem = kFSKV + kFNkv * kFTile;
// barriers
constexpr int kFQFull = 0, kFQEmpty = 2, kFKvFull = 4, kFKvEmpty = 4 + kFNkv,
              kFSFull = 4 + 2 * kFNkv, kFPFull = kFSFull + 2, kFOFull = kFPFull + 2,
              kFOEmpty = kFOFull + 2, kFLFull = kFOEmpty + 2, kFLEmpty = kFLFull + 2, kFDrain = kFLEmpty + 2, kFVReq = kFDrain + 1, kFVClean = kFVReq + 1,
              kFNumBars = kFVClean + 1;
constexpr int kFCtlMisc = kFNumBars * 8;         // tmem holder, abort flag
constexpr int kFCtlX = (kFCtlMisc + 8 + 15) & ~15;   // [2][128] row sums, [2][128] reference maxima
constexpr int kFCtlSmall = kFCtlX + 4 * 128 * 4;      // FSmall
constexpr int kFBytes = kFCtlSmall + 32 * 16 + 33 * 4;
constexpr int kFStatic = 3 * 1024;   // static shared memory of the control block
static_assert(kFBytes <= kFStatic, "control block");
static_assert(kFSmem + kFStatic <= 232448, "shared memory budget");
// TMEM columns: S (then P) of tile A and B, O of A and B
constexpr uint32_t kFTmS = 0, kFTmO = 256;

struct FItem {
  int g, q0, k0, m;     // KV head, first packed query row, first key row, keys
  int n;                // queries of both tiles
  int hi0;              // last visible key of the first query
  int n_kt_a, n_kt_b;   // key tiles of each tile
  __device__ __forceinline__ int n_kt(int x) const { return x ? n_kt_b : n_kt_a; }
};

// The plan of a small call, made by every CTA for itself (a.fused): at most 32
// sequences, their items in order.
struct FSmall {
  int4 seq[32];
  int pre[33];          // items before sequence b
};

// Round r's item of this CTA (snake order over the CTAs), false at the end.
// Items come longest first (in a small call: within each sequence) and every
// KV head of one before the next.
template <int R>
__device__ __forceinline__ bool dense_item(const DenseArgs &a, const FSmall &sm, int r, int n_work, FItem &w) {
  constexpr int QPI = 128 / R;
  const int u = r * gridDim.x + ((r & 1) ? (gridDim.x - 1 - blockIdx.x) : blockIdx.x);
  if (u >= n_work) return false;
  int2 it;
  int4 s;
  if (a.fused) {
    const int i = u / a.G;
    it.x = 0;
#pragma unroll
    for (int step = 16; step > 0; step >>= 1)
      if (it.x + step < a.B && sm.pre[it.x + step] <= i) it.x += step;
    it.y = sm.pre[it.x + 1] - 1 - i;
    s = sm.seq[it.x];
  } else {
    it = a.items[u / a.G];
    s = a.seqs[it.x];
  }
  w.g = u % a.G;
  const int t0 = it.y * 2 * QPI;
  w.q0 = s.x + t0;
  w.k0 = s.z;
  w.m = s.w;
  w.n = min(2 * QPI, s.y - t0);
  w.hi0 = s.w - s.y + t0;
  const int last_a = w.hi0 + min(w.n, QPI) - 1, last_b = w.hi0 + w.n - 1;
  w.n_kt_a = last_a >= 0 ? (last_a >> 7) + 1 : 0;
  w.n_kt_b = (w.n > QPI && last_b >= 0) ? (last_b >> 7) + 1 : 0;
  return true;
}

template <int R>
__global__ void __launch_bounds__(kFThreads, 1)
    dense_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const DenseArgs a) {
  constexpr int QPI = 128 / R;
  // the tiles fill the dynamic memory; 3 KB of static memory before them, so
  // that they start on a 1024-byte boundary without slack
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ __align__(1024) uint8_t ctl[kFStatic];
  const uint32_t s_base = smem_u32(smem);
  if (s_base & 1023) {   // the tiles' swizzle needs it
    if (threadIdx.x == 0) atomicCAS(a.status, 0, kStatusTimeout);
    return;
  }
  float *s_l = reinterpret_cast<float *>(ctl + kFCtlX), *s_m = s_l + 256;
  const uint32_t bar0 = smem_u32(ctl);
  auto bar = [&](int i) { return bar0 + 8u * uint32_t(i); };
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(ctl + kFCtlMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(ctl + kFCtlMisc + 4);

  const int tid = threadIdx.x;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int lane = tid & 31;
  if (tid == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(bar(kFQFull + x), 1);
      mbar_init(bar(kFQEmpty + x), 1);
      mbar_init(bar(kFSFull + x), 1);
      mbar_init(bar(kFPFull + x), 128);
      mbar_init(bar(kFOFull + x), 1);
      mbar_init(bar(kFOEmpty + x), 128);
      mbar_init(bar(kFLFull + x), 128);
      mbar_init(bar(kFLEmpty + x), 128);
    }
    for (int x = 0; x < kFNkv; ++x) {
      mbar_init(bar(kFKvFull + x), 1);
      mbar_init(bar(kFKvEmpty + x), 1);
    }
    mbar_init(bar(kFDrain), 1);
    mbar_init(bar(kFVReq), 1);
    mbar_init(bar(kFVClean), 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_holder), 512);
    tmem_relinquish();
  }
  FSmall &sm = *reinterpret_cast<FSmall *>(ctl + kFCtlSmall);
  if (a.fused && warp == 2) {
    int4 s = make_int4(0, 0, 0, 0);
    bool bad = false;
    if (lane < a.B) {
      const int q0 = a.cu_q[lane], q1 = a.cu_q[lane + 1], k0 = a.cu_k[lane], k1 = a.cu_k[lane + 1];
      bad = q0 < 0 || q1 < q0 || q1 > a.nq || k0 < 0 || k1 < k0 || k1 > a.nk;
      s = make_int4(q0, q1 - q0, k0, k1 - k0);
    }
    bad = __any_sync(0xffffffffu, bad);
    if (bad && lane == 0 && blockIdx.x == 0) atomicCAS(a.status, 0, kStatusBadInput);
    int n = bad ? 0 : (s.y + 2 * QPI - 1) / (2 * QPI);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, n, o);
      if (lane >= o) n += x;
    }
    sm.seq[lane] = s;
    sm.pre[lane + 1] = n;
    if (lane == 0) sm.pre[0] = 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  grid_dep_wait();   // the plan (where there is one)
  const int n_work = (a.fused ? sm.pre[a.B] : *a.n_items) * a.G;

  if (warp < 4) {
    regs_dec<kFRegsRest>();
    if (warp == 0 && lane == 0) {
      // -------------------------------------------------------- TMA producer
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
      uint32_t kseq = 0, qn[2] = {0, 0};
      bool ok = true;
      FItem w;
      for (int r = 0; ok && dense_item<R>(a, sm, r, n_work, w); ++r) {
        const int n_kt = max(w.n_kt_a, w.n_kt_b);
        for (int step = 0; step < 2 * n_kt && ok; ++step) {
          const int e = int(kseq % kFNkv);
          ok = mbar_wait(bar(kFKvEmpty + e), ((kseq / kFNkv) & 1) ^ 1, abort_flag, a.status);
          if (!ok) break;
          mbar_arrive_expect_tx(bar(kFKvFull + e), kFTile);
          const void *tm = (step & 1) ? static_cast<const void *>(&tm_v) : static_cast<const void *>(&tm_k);
          const uint32_t dst = s_base + kFSKV + e * kFTile;
          const int key0 = w.k0 + (step >> 1) * 128;
          tma_load_3d(dst, tm, bar(kFKvFull + e), 0, w.g, key0);
          tma_load_3d(dst + 16384, tm, bar(kFKvFull + e), 64, w.g, key0);
          ++kseq;
          if (step > 0) continue;
          // Q behind the first K: its tiles are free only once the last item's
          // scores are done
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (!ok || w.n_kt(x) == 0) continue;
            ok = mbar_wait(bar(kFQEmpty + x), (qn[x] & 1) ^ 1, abort_flag, a.status);
            if (!ok) continue;
            mbar_arrive_expect_tx(bar(kFQFull + x), kFTile);
            const uint32_t dq = s_base + kFSQ + x * kFTile;
            tma_load_3d(dq, &tm_q, bar(kFQFull + x), 0, w.g * R, w.q0 + x * QPI);
            tma_load_3d(dq + 16384, &tm_q, bar(kFQFull + x), 64, w.g * R, w.q0 + x * QPI);
            ++qn[x];
          }
        }
      }
      // copies still in flight land before the CTA may exit
      for (uint32_t x = 0; x < kFNkv; ++x)
        if (kseq > x) {
          const uint32_t last = kseq - 1 - x;
          mbar_wait_drain(bar(kFKvFull + last % kFNkv), (last / kFNkv) & 1);
        }
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (qn[x]) mbar_wait_drain(bar(kFQFull + x), (qn[x] - 1) & 1);
    } else if (warp == 1 && lane == 0) {
      // -------------------------------------------------------- MMA issuer
      constexpr uint32_t idesc_s = idesc_bf16_f32(128, 128, 0, 0);
      constexpr uint32_t idesc_o = idesc_bf16_f32(128, 128, 0, 1);
      // operand descriptors: Q and K K-major, V MN-major
      constexpr uint32_t kDescHi = sdesc_hi(1024);
      const uint32_t q_lo = sdesc_lo(s_base + kFSQ, 16), k_lo = sdesc_lo(s_base + kFSKV, 16),
                     v_lo = sdesc_lo(s_base + kFSKV, 16384);
      // ring position of the next entry to be consumed, and its phase
      uint32_t e = 0, ph = 0;
      uint32_t qn0 = 0, qn1 = 0, pn0 = 0, pn1 = 0, cn = 0;   // phases: items and key tiles of A, B
      bool ok = true, issued = false;
      FItem w;
      auto step = [&](uint32_t &ek) {            // takes the next ring entry, once it is full
        ok = ok && mbar_wait(bar(kFKvFull) + 8u * e, ph, abort_flag, a.status);
        ek = e;
        if (++e == kFNkv) { e = 0; ph ^= 1; }
      };
      // S of tile x from ring entry ek
      auto issue_s = [&](int x, uint32_t ek, bool last_j, bool last_user) {
        const uint32_t dq = q_lo + x * (kFTile >> 4), dk = k_lo + ek * (kFTile >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t off = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
          umma_f16_ss_w(tmem_base + kFTmS + x * 128, dq + off, kDescHi, dk + off, kDescHi, idesc_s,
                        kk > 0);
        }
        umma_commit(bar(kFSFull + x));
        if (last_user) umma_commit(bar(kFKvEmpty) + 8u * ek);
        if (last_j) umma_commit(bar(kFQEmpty + x));
        issued = true;
      };
      for (int r = 0; ok && dense_item<R>(a, sm, r, n_work, w); ++r) {
        const int na = w.n_kt_a, nb = w.n_kt_b, n_kt = max(na, nb);
        if (n_kt == 0) continue;
        uint32_t ek, ev;
        step(ek);
        if (na > 0) {
          ok = ok && mbar_wait(bar(kFQFull), qn0, abort_flag, a.status);
          if (ok) issue_s(0, ek, na == 1, nb == 0);
        }
        if (nb > 0) {
          ok = ok && mbar_wait(bar(kFQFull + 1), qn1, abort_flag, a.status);
          if (ok) issue_s(1, ek, nb == 1, true);
        }
        for (int j = 0; j < n_kt && ok; ++j) {
          step(ev);
          if (j + 1 < n_kt) step(ek);
          if (j + 1 == n_kt && w.m - j * 128 < 128) {   // V's rows behind the last key are cleared
            mbar_arrive(bar(kFVReq));
            ok = ok && mbar_wait(bar(kFVClean), cn, abort_flag, a.status);
            cn ^= 1;
          }
          const uint32_t dv = v_lo + ev * (kFTile >> 4);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int mine = x ? nb : na;
            uint32_t &pn = x ? pn1 : pn0, &qn = x ? qn1 : qn0;
            if (j >= mine) continue;
            if (j == 0) ok = ok && mbar_wait(bar(kFOEmpty + x), qn ^ 1, abort_flag, a.status);
            ok = ok && mbar_wait(bar(kFPFull + x), pn, abort_flag, a.status);
            if (!ok) break;
            pn ^= 1;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)   // 16 keys per step, 8 columns of P
              umma_f16_ts_w(tmem_base + kFTmO + x * 128, tmem_base + kFTmS + x * 128 + kk * 8,
                            dv + ((kk * 2048) >> 4), kDescHi, idesc_o, (j > 0 || kk > 0));
            if (j + 1 < mine) {
              issue_s(x, ek, j + 2 == mine, x == (j + 1 < nb ? 1 : 0));
            } else {
              umma_commit(bar(kFOFull + x));
              qn ^= 1;
            }
            if (x == (j < nb ? 1 : 0)) umma_commit(bar(kFKvEmpty) + 8u * ev);
          }
        }
      }
      // every UMMA issued has completed before TMEM can be released
      if (issued) {
        umma_commit(bar(kFDrain));
        mbar_wait_drain(bar(kFDrain), 0);
      }
    } else if (warp == 2) {
      // -------------------------------------------------------- V cleaner
      // Rows of a V tile behind the sequence's last key belong to others:
      // their weights are 0, but 0 times a NaN there would not be.  Only an
      // item's last key tile can have such rows.  The MMA issuer asks once the
      // tile has landed (so both look at the same use of its ring entry).
      uint32_t kseq = 0, cn = 0;
      bool ok = true;
      FItem w;
      for (int r = 0; ok && dense_item<R>(a, sm, r, n_work, w); ++r) {
        const int n_kt = max(w.n_kt_a, w.n_kt_b);
        kseq += 2 * n_kt;
        const int rem = w.m - (n_kt - 1) * 128;
        if (n_kt == 0 || rem >= 128) continue;
        const uint32_t seq = kseq - 1;
        ok = mbar_wait(bar(kFVReq), cn, abort_flag, a.status) &&
             mbar_wait(bar(kFKvFull + seq % kFNkv), (seq / kFNkv) & 1, abort_flag, a.status);
        cn ^= 1;
        if (!__all_sync(0xffffffffu, ok)) break;
        uint8_t *sv = smem + kFSKV + (seq % kFNkv) * kFTile;
        for (int i = rem * 8 + lane; i < 1024; i += 32) {
          *reinterpret_cast<uint4 *>(sv + i * 16) = make_uint4(0u, 0u, 0u, 0u);
          *reinterpret_cast<uint4 *>(sv + 16384 + i * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kFVClean));
      }
    }
  } else if (warp < 12) {
    // ---------------------------------------------------------- softmax
    regs_inc<kFRegsSoftmax>();
    const int x = (warp - 4) >> 2;              // tile A or B
    const int row = (warp & 3) * 32 + lane;     // tile row = TMEM lane
    const uint32_t tm_lane = tmem_base + (uint32_t((warp & 3) * 32) << 16);
    const uint32_t tm_s = tm_lane + kFTmS + x * 128, tm_o = tm_lane + kFTmO + x * 128;
    const int qi = row / R;
    const float2 sc2 = f2_dup(a.scale_log2);
    uint32_t sn = 0, ln = 0;
    bool ok = true;
    FItem w;
    for (int r = 0; ok && dense_item<R>(a, sm, r, n_work, w); ++r) {
      const bool valid = x * QPI + qi < w.n;
      const int n_kt = w.n_kt(x);
      const int hi = valid ? w.hi0 + x * QPI + qi : -1;     // last visible key
      if (n_kt == 0) continue;                       // no row of the tile sees a key
      float mr = -INFINITY;                          // reference maximum, raw scores
      float2 l2 = make_float2(0.f, 0.f), l3 = l2;
      for (int j = 0; j < n_kt; ++j) {
        ok = mbar_wait(bar(kFSFull + x), sn & 1, abort_flag, a.status);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        ++sn;
        tc_fence_after();
        float v[128];
        {
          float t0[32], t1[32], t2[32], t3[32];
          tmem_ld32(tm_s, t0);
          tmem_ld32(tm_s + 32, t1);
          tmem_ld32(tm_s + 64, t2);
          tmem_ld32(tm_s + 96, t3);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            v[c] = t0[c];
            v[32 + c] = t1[c];
            v[64 + c] = t2[c];
            v[96 + c] = t3[c];
          }
        }
        const int lim = hi - j * 128;                // last visible column
        const bool masked = __any_sync(0xffffffffu, lim < 127);
        if (masked) {
#pragma unroll
          for (int c = 0; c < 128; ++c) v[c] = (c <= lim) ? v[c] : -INFINITY;
        }
        float mc[4];
#pragma unroll
        for (int c4 = 0; c4 < 4; ++c4) mc[c4] = max3(v[32 * c4], v[32 * c4 + 1], v[32 * c4 + 2]);
#pragma unroll
        for (int c = 3; c + 2 <= 31; c += 2)
#pragma unroll
          for (int c4 = 0; c4 < 4; ++c4) mc[c4] = max3(mc[c4], v[32 * c4 + c], v[32 * c4 + c + 1]);
        float tmx = fmaxf(max3(mc[0], mc[1], v[31]), max3(mc[2], mc[3], v[63]));
        tmx = max3(tmx, v[95], v[127]);
        const bool resc = tmx > -INFINITY && (mr == -INFINITY || (tmx - mr) * a.scale_log2 > 8.f);
        if (__any_sync(0xffffffffu, resc)) {
          const float alpha = resc ? (mr == -INFINITY ? 0.f : fast_exp2((mr - tmx) * a.scale_log2)) : 1.f;
          if (resc) mr = tmx;
          l2 = f2_mul(l2, f2_dup(alpha));
          l3 = f2_mul(l3, f2_dup(alpha));
          if (j > 0) {
            // S of this tile is complete, so the products into O before it are
#pragma unroll 1
            for (int c = 0; c < 128; c += 32) {
              float t0[32];
              tmem_ld32(tm_o + c, t0);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) t0[e] *= alpha;
              tmem_st32(tm_o + c, t0);
            }
          }
        }
        const float2 nmb2 = f2_dup(mr == -INFINITY ? 0.f : -mr * a.scale_log2);
        // P as bf16 over S's first 64 columns (S is all in registers)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t pw[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const int c = h * 64 + 2 * e;
            const float2 z = f2_fma(make_float2(v[c], v[c + 1]), sc2, nmb2);
            const float2 p = make_float2(fast_exp2(z.x), fast_exp2(z.y));
            if (e & 1) l3 = f2_add(l3, p); else l2 = f2_add(l2, p);
            pw[e] = pack_bf16x2(p.x, p.y);
          }
          tmem_st32u(tm_s + h * 32, pw);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(kFPFull + x));
      }
      if (!ok) break;
      // the sum and the maximum go to the epilogue, once it has read the last
      // item's (this item's products may still wait for O then)
      ok = mbar_wait(bar(kFLEmpty + x), ln ^ 1, abort_flag, a.status);
      if (!__all_sync(0xffffffffu, ok)) break;
      ln ^= 1;
      s_l[x * 128 + row] = (l2.x + l3.x) + (l2.y + l3.y);
      s_m[x * 128 + row] = mr;
      mbar_arrive(bar(kFLFull + x));
    }
  } else {
    // ---------------------------------------------------------- epilogue
    regs_dec<kFRegsRest>();
    const int row = (warp & 3) * 32 + lane;          // tile row = TMEM lane
    const uint32_t tm_lane = tmem_base + (uint32_t((warp & 3) * 32) << 16);
    const int qi = row / R, hh = row % R;
    uint32_t on0 = 0, on1 = 0;
    bool ok = true;
    FItem w;
    for (int r = 0; ok && dense_item<R>(a, sm, r, n_work, w); ++r) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const bool valid = x * QPI + qi < w.n;
        const size_t orow = size_t(w.q0 + x * QPI + qi) * a.H + w.g * R + hh;
        uint4 *dst = reinterpret_cast<uint4 *>(a.out + orow * kHeadDim);
        if (w.n_kt(x) == 0) {                        // no row of the tile sees a key
          if (valid) {
#pragma unroll
            for (int c = 0; c < 16; ++c) dst[c] = make_uint4(0u, 0u, 0u, 0u);
            if (a.lse) a.lse[orow] = -INFINITY;
          }
          continue;
        }
        uint32_t &on = x ? on1 : on0;
        ok = ok && mbar_wait(bar(kFLFull + x), on, abort_flag, a.status) &&
             mbar_wait(bar(kFOFull + x), on, abort_flag, a.status);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        on ^= 1;
        const float l = s_l[x * 128 + row], mr = s_m[x * 128 + row];
        mbar_arrive(bar(kFLEmpty + x));
        const float inv = l == 0.f ? 0.f : 1.f / l;   // (a NaN stays one)
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          float o[32];
          tmem_ld32(tm_lane + kFTmO + x * 128 + c * 32, o);
          tmem_wait_ld();
          quad_store32(o, inv, 4 * c, [&](int j) {
            const int rw = (row & ~3) + j, i = x * QPI + rw / R;
            return i < w.n ? a.out + (size_t(w.q0 + i) * a.H + w.g * R + rw % R) * kHeadDim : nullptr;
          });
        }
        tc_fence_before();
        mbar_arrive(bar(kFOEmpty + x));
        if (valid && a.lse) a.lse[orow] = l == 0.f ? -INFINITY : mr * a.scale + logf(l);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

template <int R>
cudaError_t launch_fwd_r(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                         const DenseArgs &a, int num_sms, cudaStream_t st) {
  auto kern = dense_fwd_kernel<R>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kFSmem);
  if (e != cudaSuccess) return e;
  const long long work = (long long)a.max_items * a.G;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(work < num_sms ? work : num_sms));
  cfg.blockDim = dim3(kFThreads);
  cfg.dynamicSmemBytes = kFSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.fused ? 0 : 1;   // (only the plan may still run when this kernel starts)
  return cudaLaunchKernelEx(&cfg, kern, tq, tk, tv, a);
}

}  // namespace

cudaError_t launch_dense_plan(const DenseArgs &a, int per, int num_sms, cudaStream_t st) {
  int grid = 1;
  if (a.items_k) {   // the backward: the key tiles' list, and the rows' statistics
    const long long blocks = ((long long)a.nq * a.H + 127) / 128;
    grid = 2 + int(blocks < 2 * num_sms ? blocks : 2 * num_sms);
  }
  dense_plan_kernel<<<grid, 1024, 0, st>>>(a, per, 128 / (a.H / a.G));
  return cudaGetLastError();
}

cudaError_t launch_dense_varlen(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                                const DenseArgs &a, int num_sms, cudaStream_t st) {
  DenseArgs b = a;
  // Up to two rounds of items the order matters less than the plan's launch
  // (512 tokens in three prompts, 8 heads: 16.3 us against 19.5).
  b.fused = a.B <= 32 && (long long)a.max_items * a.G <= 2 * num_sms;
  if (!b.fused) {
    cudaError_t e = launch_dense_plan(a, dense_item_queries(a.H / a.G), num_sms, st);
    if (e != cudaSuccess) return e;
  }
  switch (a.H / a.G) {
    case 1: return launch_fwd_r<1>(tq, tk, tv, b, num_sms, st);
    case 2: return launch_fwd_r<2>(tq, tk, tv, b, num_sms, st);
    case 4: return launch_fwd_r<4>(tq, tk, tv, b, num_sms, st);
    case 8: return launch_fwd_r<8>(tq, tk, tv, b, num_sms, st);
    case 16: return launch_fwd_r<16>(tq, tk, tv, b, num_sms, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace msa
