// Backward pass of dense causal attention over packed sequences.
//   P = exp(scale q.k - lse), dP = dout . v, D = dout . out, dZ = P (dP - D)
//   dq = scale sum dZ k,  dk += scale dZ q,  dv += P dout.
//
//   dense_plan_kernel  (dense_kernels.cu) the lists of work items, and
//                 {-lse log2 e, -D} of every (query row, head).
//   dense_dkv_kernel   key tiles outer: one work item is 128 keys of a KV
//                 head and every 128-row query tile (128/R queries x R heads)
//                 that sees one of them.  Transposed products, so that what
//                 the softmax makes is the A operand from TMEM:
//                   S^T = K Q^T, dP^T = V dO^T   (TMEM lanes are keys)
//                   dV += P^T dO, dK += dZ^T Q   (P^T and dZ^T over dP^T)
//   dense_dq_kernel    query tiles outer: one item is a 128-row query tile:
//                   S = Q K^T, dP = dO V^T, dQ += dZ K  (dZ over S).
//
// S and dP are computed in both kernels: 7 products where one kernel with
// atomics on dq would need 5.  In return no gradient is summed by atomics (the
// result repeats bit for bit) and nothing of dq's size is kept in fp32.
// P and dZ are rounded to bf16 for their products (Q, K and dO are bf16, and
// both operands of a UMMA have one type).  Every element's rounding is its own,
// of the size of the results' last one: with random rows of 1000 keys and more
// dq and dk are 2.4e-3 of their norm off where a single rounding at the end
// gives 1.7e-3, dv 2.3e-3.  D is an fp32 sum over out as bf16, as the caller
// holds it, and what that rounding costs does not shrink where dP and D nearly
// cancel: dq and dk are 3.5e-3 off for sequences of two tokens, 3.0e-3 of
// eight, and 3.7e-3 (5.2e-3) for 1000 tokens whose queries are four (eight)
// times as large.
// Measured: 8192 tokens, 32 heads on 8, 1.34 ms from idle (7 products of 128^3
// per tile pair; 1026 TFLOP/s, 0.62 of burst bf16, over the 5 counted); 7.3K tokens in seven
// documents, 16 heads on 4, 136-158 us.  Over that whole 8192-token call, items'
// starts and ends among them, a tile pair takes dkv 2860 cycles for 2048 of
// products (four of 512) and dq 2130 for 1536; in the steady state (read with
// clock()) 2560 and 1880.  The softmax's chain (exponentials 1024 of the MUFU
// unit, loads and stores of TMEM around them) bounds both.
// Tried and not faster: exponentials as polynomials on the FMA pipe, K and V
// (Q and dO) released before the last product, dq stored under the next item's
// first products, halves of a dq tile skipped where no row sees them.
// Roles in both kernels (one persistent CTA per SM, three warpgroups): warp 0
// loads by TMA, warp 1 issues UMMAs, warps 2-3 help, warps 4-11 are the
// softmax: two warpgroups, one TMEM lane per thread, 64 of the 128 columns
// each; each writes its bf16 results over its own half of what it read.
#include <cuda.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "dense.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace msa {

namespace {

constexpr int kBThreads = 384;
constexpr int kBTile = 32768;                       // 128 rows x 256 B
// Seven tiles: two that stay for an item, a ring of three for the streamed
// tile that two products far apart read (dkv: Q, dq: K) and one of two for the
// other (dkv: dO, dq: V).  They fill the dynamic shared memory; barriers and
// statistics lie in 3 KB of static memory before it, so that the tiles start
// on a 1024-byte boundary without slack.
constexpr int kBSKeep = 0, kBSLong = 2 * kBTile, kBSShort = 5 * kBTile, kBSmem = 7 * kBTile;
constexpr int kBCtl = 3 * 1024;
static_assert(kBSmem + kBCtl <= 232448, "shared memory budget");
// A place in a ring of n stages and the phase of its use.
struct RingPos {
  uint32_t s = 0, ph = 0;
  __device__ __forceinline__ void next(uint32_t n) {
    if (++s == n) { s = 0; ph ^= 1; }
  }
};
constexpr int kBRegsRest = 72, kBRegsSoftmax = 216;   // 128 * 72 + 256 * 216 = 384 * 168
constexpr uint32_t kBDescHi = sdesc_hi(1024);

// D (+)= A B^T over 128 elements of the head dim, both operands K-major tiles.
__device__ __forceinline__ void mma_tiles(uint32_t d, uint32_t a_lo, uint32_t b_lo) {
  constexpr uint32_t idesc = idesc_bf16_f32(128, 128, 0, 0);
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    const uint32_t off = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
    umma_f16_ss_w(d, a_lo + off, kBDescHi, b_lo + off, kBDescHi, idesc, kk > 0);
  }
}
// D (+)= A B: A from TMEM (bf16 pairs, the first 64 of the 128 summed-over
// indices from column `a`, the others from a + 64), B a tile whose rows are
// summed over.
__device__ __forceinline__ void mma_from_tmem(uint32_t d, uint32_t a, uint32_t b_lo, bool add) {
  constexpr uint32_t idesc = idesc_bf16_f32(128, 128, 0, 1);
#pragma unroll
  for (int kk = 0; kk < 8; ++kk)
    umma_f16_ts_w(d, a + (kk >> 2) * 64 + (kk & 3) * 8, b_lo + ((kk * 2048) >> 4), kBDescHi, idesc,
                  add || kk > 0);
}

__device__ __forceinline__ void load64(uint32_t taddr, float (&v)[64]) {
  float t0[32], t1[32];
  tmem_ld32(taddr, t0);
  tmem_ld32(taddr + 32, t1);
  tmem_wait_ld();
#pragma unroll
  for (int c = 0; c < 32; ++c) {
    v[c] = t0[c];
    v[32 + c] = t1[c];
  }
}
// 64 values as bf16 pairs into 32 columns.
__device__ __forceinline__ void store64(uint32_t taddr, const float (&v)[64]) {
  uint32_t w[32];
#pragma unroll
  for (int e = 0; e < 32; ++e) w[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
  tmem_st32u(taddr, w);
  tmem_wait_st();
}
__device__ __forceinline__ void load_tile(uint32_t dst, const void *tm, uint32_t bar, int y, int z) {
  tma_load_3d(dst, tm, bar, 0, y, z);
  tma_load_3d(dst + 16384, tm, bar, 64, y, z);
}
// Rows [row0, 128) of a tile to zero (one or two warps, thread `t` of `n`).
__device__ __forceinline__ void clear_rows(uint8_t *tile, int row0, int t, int n) {
  for (int i = row0 * 8 + t; i < 1024; i += n) {
    *reinterpret_cast<uint4 *>(tile + i * 16) = make_uint4(0u, 0u, 0u, 0u);
    *reinterpret_cast<uint4 *>(tile + 16384 + i * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
}
// This CTA's work item in round r (snake order), or -1.
__device__ __forceinline__ int round_item(int r, int n_work) {
  const int u = r * gridDim.x + ((r & 1) ? (gridDim.x - 1 - blockIdx.x) : blockIdx.x);
  return u < n_work ? u : -1;
}

// ------------------------------------------------------------------ dk, dv
struct KvItem {
  int g, key0, keys;      // first packed key row, keys of the tile that exist
  int q0, n, qt0, n_qt;   // the sequence's first query row and queries; its query tiles that see the tile
  int rel;                // key (of the tile) that query 0 sees last: 128 kt - off subtracted
};
template <int R>
__device__ __forceinline__ bool kv_item(const DenseArgs &a, int r, int n_work, KvItem &w) {
  constexpr int QPI = 128 / R;
  const int u = round_item(r, n_work);
  if (u < 0) return false;
  const int2 it = a.items_k[u / a.G];
  const int4 s = a.seqs[it.x];
  w.g = u % a.G;
  w.key0 = s.z + it.y * 128;
  w.keys = min(128, s.w - it.y * 128);
  w.q0 = s.x;
  w.n = s.y;
  w.rel = s.w - s.y - it.y * 128;              // query i sees keys 0 .. rel + i of the tile
  const int first = max(0, -w.rel);             // first query that sees a key of the tile
  w.qt0 = first / QPI;
  w.n_qt = first < s.y ? (s.y + QPI - 1) / QPI - w.qt0 : 0;
  return true;
}

// barriers
constexpr int kVKvFull = 0, kVKvEmpty = 1, kVQFull = 2, kVQEmpty = 5, kVOFull = 8, kVOEmpty = 10,
              kVStFull = 12, kVStEmpty = 14, kVSFull = 16, kVDpFull = 17, kVPFull = 18, kVZFull = 19,
              kVAccFull = 20, kVAccEmpty = 21, kVDrain = 22, kVSFree = 23, kVNumBars = 24;
constexpr int kVMisc = kVNumBars * 8;                // tmem holder, abort flag
constexpr int kVStat = (kVMisc + 8 + 15) & ~15;      // [2 stages][128] -lse log2 e, [2][128] -D
static_assert(kVStat + 4 * 128 * 4 <= kBCtl, "control block");
constexpr uint32_t kVTmS = 0, kVTmDP = 128, kVTmDV = 256, kVTmDK = 384;

// S is free as soon as the softmax has it in registers, and P and dZ both go
// over dP (each warpgroup's 64 columns of it take its 32 of P and its 32 of
// dZ once it has read them), so the order of the UMMAs is
//   dV += P_i dO_i | dK += dZ_i Q_i, dP_i+1, S_i+2
// (the bar: behind P_i, behind dZ_i) and the exponentials of tile i+1 run
// under all of it.
template <int R>
__global__ void __launch_bounds__(kBThreads, 1)
    dense_dkv_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                     const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const DenseArgs a) {
  constexpr int QPI = 128 / R;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ __align__(1024) uint8_t ctl[kBCtl];
  const uint32_t s_base = smem_u32(smem);
  if (s_base & 1023) {   // the tiles' swizzle needs it
    if (threadIdx.x == 0) atomicCAS(a.status, 0, kStatusTimeout);
    return;
  }
  const uint32_t bar0 = smem_u32(ctl);
  auto bar = [&](int i) { return bar0 + 8u * uint32_t(i); };
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(ctl + kVMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(ctl + kVMisc + 4);
  float *s_nl = reinterpret_cast<float *>(ctl + kVStat), *s_nd = s_nl + 256;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kVNumBars; ++i)
      mbar_init(bar(i), i == kVStFull || i == kVStFull + 1 ? 64
                        : (i == kVStEmpty || i == kVStEmpty + 1 || i == kVPFull || i == kVZFull || i == kVAccEmpty ||
                         i == kVSFree)
                            ? 256
                            : 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_holder), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = *tmem_holder;
  const int n_work = *a.n_items_k * a.G;
  KvItem w;
  grid_dep_launch();   // dense_dq_kernel may follow wherever a CTA of this one ends

  if (warp < 4) {
    regs_dec<kBRegsRest>();
    if (warp == 0 && lane == 0) {
      // -------------------------------------------------------- TMA producer
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_do);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
      uint32_t it = 0, seq = 0, nq = 0;              // items; tiles of dO and of Q
      RingPos q, o;
      bool ok = true;
      for (int r = 0; ok && kv_item<R>(a, r, n_work, w); ++r) {
        if (w.n_qt == 0) continue;
        for (int i = 0; i < w.n_qt && ok; ++i, ++seq) {
          const int row = w.q0 + (w.qt0 + i) * QPI;
          ok = mbar_wait(bar(kVQEmpty + q.s), q.ph ^ 1, abort_flag, a.status);
          if (!ok) break;
          mbar_arrive_expect_tx(bar(kVQFull + q.s), kBTile);
          load_tile(s_base + kBSLong + q.s * kBTile, &tm_q, bar(kVQFull + q.s), w.g * R, row);
          q.next(3);
          ++nq;
          ok = mbar_wait(bar(kVOEmpty + o.s), o.ph ^ 1, abort_flag, a.status);
          if (!ok) break;
          mbar_arrive_expect_tx(bar(kVOFull + o.s), kBTile);
          load_tile(s_base + kBSShort + o.s * kBTile, &tm_do, bar(kVOFull + o.s), w.g * R, row);
          o.next(2);
          if (i > 0) continue;
          // K and V behind the first tiles: theirs are free only once the last
          // item is done
          ok = mbar_wait(bar(kVKvEmpty), (it & 1) ^ 1, abort_flag, a.status);
          if (!ok) { ++seq; break; }
          mbar_arrive_expect_tx(bar(kVKvFull), 2 * kBTile);
          load_tile(s_base + kBSKeep, &tm_k, bar(kVKvFull), w.g, w.key0);
          load_tile(s_base + kBSKeep + kBTile, &tm_v, bar(kVKvFull), w.g, w.key0);
          ++it;
        }
      }
      // copies still in flight land before the CTA may exit
      if (it) mbar_wait_drain(bar(kVKvFull), (it - 1) & 1);
      for (uint32_t x = 1; x <= 3; ++x)
        if (nq >= x) mbar_wait_drain(bar(kVQFull + (nq - x) % 3), ((nq - x) / 3) & 1);
      for (uint32_t x = 1; x <= 2; ++x)
        if (seq >= x) mbar_wait_drain(bar(kVOFull + ((seq - x) & 1)), ((seq - x) >> 1) & 1);
    } else if (warp == 1 && lane == 0) {
      // -------------------------------------------------------- MMA issuer
      const uint32_t k_lo = sdesc_lo(s_base + kBSKeep, 16), v_lo = sdesc_lo(s_base + kBSKeep + kBTile, 16);
      // Q and dO as K-major operands and, summed over their rows, as MN-major ones
      const uint32_t qk_lo = sdesc_lo(s_base + kBSLong, 16), qm_lo = sdesc_lo(s_base + kBSLong, 16384);
      const uint32_t ok_lo = sdesc_lo(s_base + kBSShort, 16), om_lo = sdesc_lo(s_base + kBSShort, 16384);
      constexpr uint32_t T = kBTile >> 4;
      uint32_t it = 0, ph = 0;
      RingPos q, o;
      bool ok = true;
      for (int r = 0; ok && kv_item<R>(a, r, n_work, w); ++r) {
        if (w.n_qt == 0) continue;
        ok = mbar_wait(bar(kVKvFull), it & 1, abort_flag, a.status) &&
             mbar_wait(bar(kVQFull + q.s), q.ph, abort_flag, a.status);
        if (!ok) break;
        // S of the first two tiles, dP of the first; qn runs ahead with S
        RingPos qn = q;
        auto issue_s = [&]() {
          mma_tiles(tm + kVTmS, k_lo, qk_lo + qn.s * T);
          umma_commit(bar(kVSFull));
          qn.next(3);
        };
        issue_s();
        ok = mbar_wait(bar(kVOFull + o.s), o.ph, abort_flag, a.status);
        if (!ok) break;
        mma_tiles(tm + kVTmDP, v_lo, ok_lo + o.s * T);
        umma_commit(bar(kVDpFull));
        if (w.n_qt > 1) {
          ok = mbar_wait(bar(kVQFull + qn.s), qn.ph, abort_flag, a.status) &&
               mbar_wait(bar(kVSFree), ph, abort_flag, a.status);
          if (!ok) break;
          tc_fence_after();
          issue_s();
        }
        ok = mbar_wait(bar(kVAccEmpty), (it & 1) ^ 1, abort_flag, a.status);
        for (int i = 0; i < w.n_qt && ok; ++i, ph ^= 1) {
          const uint32_t qs = q.s, os = o.s;
          q.next(3);
          o.next(2);
          ok = mbar_wait(bar(kVPFull), ph, abort_flag, a.status);
          if (!ok) break;
          tc_fence_after();
          mma_from_tmem(tm + kVTmDV, tm + kVTmDP, om_lo + os * T, i > 0);
          umma_commit(bar(kVOEmpty + os));
          if (i + 1 < w.n_qt) ok = mbar_wait(bar(kVOFull + o.s), o.ph, abort_flag, a.status);
          ok = ok && mbar_wait(bar(kVZFull), ph, abort_flag, a.status);
          if (!ok) break;
          tc_fence_after();
          mma_from_tmem(tm + kVTmDK, tm + kVTmDP + 32, qm_lo + qs * T, i > 0);
          umma_commit(bar(kVQEmpty + qs));
          if (i + 1 < w.n_qt) {
            mma_tiles(tm + kVTmDP, v_lo, ok_lo + o.s * T);
            umma_commit(bar(kVDpFull));
          }
          // the softmax's read of S_i+1 (of the last tile too, so that every
          // phase of the barrier is waited for)
          if (i + 2 < w.n_qt) ok = mbar_wait(bar(kVQFull + qn.s), qn.ph, abort_flag, a.status);
          if (i + 1 < w.n_qt) ok = ok && mbar_wait(bar(kVSFree), ph ^ 1, abort_flag, a.status);
          if (!ok) break;
          if (i + 2 < w.n_qt) {
            tc_fence_after();
            issue_s();
          }
        }
        if (!ok) break;
        umma_commit(bar(kVAccFull));
        umma_commit(bar(kVKvEmpty));
        ++it;
      }
      umma_commit(bar(kVDrain));
      mbar_wait_drain(bar(kVDrain), 0);
    } else if (warp >= 2) {
      // -------------------------------------------------------- helpers
      // each query tile's statistics; and in a sequence's last tile the rows
      // behind its last query, which belong to others: their P and dZ are 0,
      // but 0 times a NaN there would not be
      const int ht = tid - 64;
      uint32_t seq = 0;
      bool ok = true;
      for (int r = 0; ok && kv_item<R>(a, r, n_work, w); ++r) {
        for (int i = 0; i < w.n_qt; ++i, ++seq) {
          const int st = seq & 1, qa = (w.qt0 + i) * QPI;
          ok = mbar_wait(bar(kVStEmpty + st), ((seq >> 1) & 1) ^ 1, abort_flag, a.status);
          if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
#pragma unroll
          for (int x = ht; x < 128; x += 64) {
            const int qi = qa + x / R;
            const float2 v = qi < w.n ? a.stat[size_t(w.q0 + qi) * a.H + w.g * R + x % R] : make_float2(0.f, 0.f);
            s_nl[st * 128 + x] = v.x;
            s_nd[st * 128 + x] = v.y;
          }
          if (w.n - qa < QPI) {
            ok = mbar_wait(bar(kVQFull + seq % 3), (seq / 3) & 1, abort_flag, a.status) &&
                 mbar_wait(bar(kVOFull + st), (seq >> 1) & 1, abort_flag, a.status);
            if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
            clear_rows(smem + kBSLong + (seq % 3) * kBTile, (w.n - qa) * R, ht, 64);
            clear_rows(smem + kBSShort + st * kBTile, (w.n - qa) * R, ht, 64);
            fence_proxy_async_smem();
          }
          mbar_arrive(bar(kVStFull + st));
        }
      }
    }
  } else {
    // ---------------------------------------------------------- softmax
    regs_inc<kBRegsSoftmax>();
    const int hc = (warp - 4) >> 2;                  // query rows 64 hc .. of each tile
    const int key = (warp & 3) * 32 + lane;          // TMEM lane
    const uint32_t tl = tm + (uint32_t((warp & 3) * 32) << 16);
    const float2 sc2 = f2_dup(a.scale_log2);
    uint32_t seq = 0, it = 0;
    bool ok = true;
    for (int r = 0; ok && kv_item<R>(a, r, n_work, w); ++r) {
      const size_t grow = size_t(w.key0 + key) * a.G + w.g;
      uint16_t *dk = a.dk + grow * kHeadDim + hc * 64, *dv = a.dv + grow * kHeadDim + hc * 64;
      if (w.n_qt == 0) {                             // no query sees a key of the tile
        if (key < w.keys) {
#pragma unroll
          for (int c = 0; c < 8; ++c)
            reinterpret_cast<uint4 *>(dk)[c] = reinterpret_cast<uint4 *>(dv)[c] = make_uint4(0u, 0u, 0u, 0u);
        }
        continue;
      }
      for (int i = 0; i < w.n_qt; ++i, ++seq) {
        const int st = seq & 1, qa = (w.qt0 + i) * QPI;
        ok = mbar_wait(bar(kVStFull + st), (seq >> 1) & 1, abort_flag, a.status) &&
             mbar_wait(bar(kVSFull), seq & 1, abort_flag, a.status);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        tc_fence_after();
        float p[64];
        load64(tl + kVTmS + hc * 64, p);
        tc_fence_before();
        mbar_arrive(bar(kVSFree));
        // rows that see this key: queries >= key - rel, up to the last one; in
        // the queries of this warpgroup's half (64 / R of them, R rows each)
        constexpr int QH = 64 / R;
        const int lo = key - w.rel - qa - hc * QH, hi = w.n - qa - hc * QH;
        const bool tail = hi < QH;
        const bool masked = __any_sync(0xffffffffu, lo > 0 || tail);
        if (masked && __all_sync(0xffffffffu, lo >= min(hi, QH))) {   // no row sees a key of this warp
#pragma unroll
          for (int c = 0; c < 64; ++c) p[c] = 0.f;
        } else {
          const float4 *nl = reinterpret_cast<const float4 *>(s_nl + st * 128 + hc * 64);
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const float4 x = nl[c];
            const float2 z0 = f2_fma(make_float2(p[4 * c], p[4 * c + 1]), sc2, make_float2(x.x, x.y));
            const float2 z1 = f2_fma(make_float2(p[4 * c + 2], p[4 * c + 3]), sc2, make_float2(x.z, x.w));
            p[4 * c] = fast_exp2(z0.x);
            p[4 * c + 1] = fast_exp2(z0.y);
            p[4 * c + 2] = fast_exp2(z1.x);
            p[4 * c + 3] = fast_exp2(z1.y);
          }
          if (masked) {
#pragma unroll
            for (int c = 0; c < 64; ++c) p[c] = (c / R >= lo && c / R < hi) ? p[c] : 0.f;
          }
        }
        ok = mbar_wait(bar(kVDpFull), seq & 1, abort_flag, a.status);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        tc_fence_after();
        float z[64];
        load64(tl + kVTmDP + hc * 64, z);
        store64(tl + kVTmDP + hc * 64, p);
        tc_fence_before();
        mbar_arrive(bar(kVPFull));
        const float4 *nd = reinterpret_cast<const float4 *>(s_nd + st * 128 + hc * 64);
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float4 x = nd[c];
          const float2 z0 = f2_mul(f2_add(make_float2(z[4 * c], z[4 * c + 1]), make_float2(x.x, x.y)),
                                   make_float2(p[4 * c], p[4 * c + 1]));
          const float2 z1 = f2_mul(f2_add(make_float2(z[4 * c + 2], z[4 * c + 3]), make_float2(x.z, x.w)),
                                   make_float2(p[4 * c + 2], p[4 * c + 3]));
          z[4 * c] = z0.x; z[4 * c + 1] = z0.y;
          z[4 * c + 2] = z1.x; z[4 * c + 3] = z1.y;
        }
        if (tail) {   // (dP of the rows behind the last query may be anything)
#pragma unroll
          for (int c = 0; c < 64; ++c) z[c] = c / R < hi ? z[c] : 0.f;
        }
        store64(tl + kVTmDP + hc * 64 + 32, z);
        tc_fence_before();
        mbar_arrive(bar(kVZFull));
        mbar_arrive(bar(kVStEmpty + st));
      }
      if (!ok) break;
      ok = mbar_wait(bar(kVAccFull), it & 1, abort_flag, a.status);
      if (!__all_sync(0xffffffffu, ok)) break;
      ++it;
      tc_fence_after();
      const size_t row4 = size_t(w.key0 + (key & ~3)) * a.G + w.g;   // the quad's first key
      const int left = w.keys - (key & ~3);
#pragma unroll 1
      for (int m = 0; m < 2; ++m) {
        float x[64];
        load64(tl + (m ? kVTmDK : kVTmDV) + hc * 64, x);
        if (m) {
          tc_fence_before();
          mbar_arrive(bar(kVAccEmpty));
        }
        uint16_t *out = (m ? a.dk : a.dv) + row4 * kHeadDim;
        auto ptr = [&](int j) { return j < left ? out + size_t(j) * a.G * kHeadDim : nullptr; };
        quad_store32(x, m ? a.scale : 1.f, hc * 8, ptr);
        quad_store32(x + 32, m ? a.scale : 1.f, hc * 8 + 4, ptr);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tm, 512);
  }
}

// ------------------------------------------------------------------ dq
struct QItem {
  int g, q0, n, hi0, key0, m, n_kt;   // first packed query row, queries of the tile, last key of the first
};
template <int R>
__device__ __forceinline__ bool q_item(const DenseArgs &a, int u, int n_work, QItem &w) {
  constexpr int QPI = 128 / R;
  if (u >= n_work) return false;
  const int2 it = a.items[u / a.G];
  const int4 s = a.seqs[it.x];
  w.g = u % a.G;
  w.q0 = s.x + it.y * QPI;
  w.n = min(QPI, s.y - it.y * QPI);
  w.hi0 = s.w - s.y + it.y * QPI;
  w.key0 = s.z;
  w.m = s.w;
  const int last = w.hi0 + w.n - 1;
  w.n_kt = last >= 0 ? (last >> 7) + 1 : 0;
  return true;
}

constexpr int kGQFull = 0, kGQEmpty = 1, kGKFull = 2, kGKEmpty = 5, kGVFull = 8, kGVEmpty = 10, kGSFull = 12,
              kGDpFull = 14, kGZFull = 15, kGAccFull = 16, kGAccEmpty = 17, kGReq = 18, kGClean = 19, kGDrain = 20,
              kGItFull = 21, kGItEmpty = 23, kGNumBars = 25;
constexpr int kGMisc = kGNumBars * 8;                // tmem holder, abort flag, two item numbers
constexpr uint32_t kGTmS = 0, kGTmDP = 256, kGTmDQ = 384;   // S: two buffers of 128 columns

// S of key tile j+1 runs under the softmax of tile j; dP of tile j+1 and
// dQ += dZ K of tile j under the exponentials of tile j+1.
//
// This kernel needs nothing that dense_dkv_kernel makes, so it is launched as
// its programmatic dependent: its CTAs take over an SM as soon as one of the
// other's has ended there.  They start at different times, hence items are
// handed out by a counter (by the producer, through a mailbox of two), which
// evens out dk's and dv's long items: 7.3K tokens in seven documents 180 ->
// 166 us for the whole backward.  Before it ends it waits for the other
// kernel, so that what follows in the stream finds both done.
template <int R>
__global__ void __launch_bounds__(kBThreads, 1)
    dense_dq_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const DenseArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ __align__(1024) uint8_t ctl[kBCtl];
  const uint32_t s_base = smem_u32(smem);
  if (s_base & 1023) {   // the tiles' swizzle needs it
    if (threadIdx.x == 0) atomicCAS(a.status, 0, kStatusTimeout);
    return;
  }
  const uint32_t bar0 = smem_u32(ctl);
  auto bar = [&](int i) { return bar0 + 8u * uint32_t(i); };
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(ctl + kGMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(ctl + kGMisc + 4);
  volatile int *s_item = reinterpret_cast<volatile int *>(ctl + kGMisc + 8);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kGNumBars; ++i) mbar_init(bar(i), (i == kGZFull || i == kGAccEmpty) ? 256 : (i == kGItEmpty || i == kGItEmpty + 1) ? 10 : 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_holder), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = *tmem_holder;
  const int n_work = *a.n_items * a.G;
  QItem w;
  // The n-th item of this CTA, for its ten readers (one lane of the issuer,
  // the cleaner and eight softmax warps): `all` of the warp's lanes call.
  auto next_item = [&](uint32_t n, bool all) {
    const uint32_t x = n & 1;
    bool ok = mbar_wait(bar(kGItFull + x), (n >> 1) & 1, abort_flag, a.status);
    const int it = s_item[x];
    if (all) ok = __all_sync(0xffffffffu, ok);
    if (ok && (!all || lane == 0)) mbar_arrive(bar(kGItEmpty + x));
    return ok ? it : 0x7fffffff;
  };

  if (warp < 4) {
    regs_dec<kBRegsRest>();
    if (warp == 0 && lane == 0) {
      // -------------------------------------------------------- TMA producer
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_do);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
      uint32_t it = 0, seq = 0, nk = 0;              // items; tiles of V and of K
      RingPos k, v;
      bool ok = true;
      for (uint32_t n = 0; ok; ++n) {
        ok = mbar_wait(bar(kGItEmpty + (n & 1)), ((n >> 1) & 1) ^ 1, abort_flag, a.status);
        if (!ok) break;
        const int item = atomicAdd(a.next_q, 1);
        s_item[n & 1] = item;
        mbar_arrive(bar(kGItFull + (n & 1)));
        if (!q_item<R>(a, item, n_work, w)) break;
        if (w.n_kt == 0) continue;
        for (int j = 0; j < w.n_kt && ok; ++j, ++seq) {
          ok = mbar_wait(bar(kGKEmpty + k.s), k.ph ^ 1, abort_flag, a.status);
          if (!ok) break;
          mbar_arrive_expect_tx(bar(kGKFull + k.s), kBTile);
          load_tile(s_base + kBSLong + k.s * kBTile, &tm_k, bar(kGKFull + k.s), w.g, w.key0 + j * 128);
          k.next(3);
          ++nk;
          ok = mbar_wait(bar(kGVEmpty + v.s), v.ph ^ 1, abort_flag, a.status);
          if (!ok) break;
          mbar_arrive_expect_tx(bar(kGVFull + v.s), kBTile);
          load_tile(s_base + kBSShort + v.s * kBTile, &tm_v, bar(kGVFull + v.s), w.g, w.key0 + j * 128);
          v.next(2);
          if (j > 0) continue;
          // Q and dO behind the first tiles (see above)
          ok = mbar_wait(bar(kGQEmpty), (it & 1) ^ 1, abort_flag, a.status);
          if (!ok) { ++seq; break; }
          mbar_arrive_expect_tx(bar(kGQFull), 2 * kBTile);
          load_tile(s_base + kBSKeep, &tm_q, bar(kGQFull), w.g * R, w.q0);
          load_tile(s_base + kBSKeep + kBTile, &tm_do, bar(kGQFull), w.g * R, w.q0);
          ++it;
        }
      }
      if (it) mbar_wait_drain(bar(kGQFull), (it - 1) & 1);
      for (uint32_t x = 1; x <= 3; ++x)
        if (nk >= x) mbar_wait_drain(bar(kGKFull + (nk - x) % 3), ((nk - x) / 3) & 1);
      for (uint32_t x = 1; x <= 2; ++x)
        if (seq >= x) mbar_wait_drain(bar(kGVFull + ((seq - x) & 1)), ((seq - x) >> 1) & 1);
    } else if (warp == 1 && lane == 0) {
      // -------------------------------------------------------- MMA issuer
      const uint32_t q_lo = sdesc_lo(s_base + kBSKeep, 16), do_lo = sdesc_lo(s_base + kBSKeep + kBTile, 16);
      const uint32_t kk_lo = sdesc_lo(s_base + kBSLong, 16), km_lo = sdesc_lo(s_base + kBSLong, 16384);
      const uint32_t vk_lo = sdesc_lo(s_base + kBSShort, 16);
      constexpr uint32_t T = kBTile >> 4;
      uint32_t it = 0, seq = 0, cn = 0;
      RingPos k, v;
      bool ok = true;
      for (uint32_t n = 0; ok && q_item<R>(a, next_item(n, false), n_work, w); ++n) {
        if (w.n_kt == 0) continue;
        ok = mbar_wait(bar(kGQFull), it & 1, abort_flag, a.status) &&
             mbar_wait(bar(kGKFull + k.s), k.ph, abort_flag, a.status);
        if (!ok) break;
        mma_tiles(tm + kGTmS + (seq & 1) * 128, q_lo, kk_lo + k.s * T);
        umma_commit(bar(kGSFull + (seq & 1)));
        ok = mbar_wait(bar(kGVFull + v.s), v.ph, abort_flag, a.status);
        if (!ok) break;
        mma_tiles(tm + kGTmDP, do_lo, vk_lo + v.s * T);
        umma_commit(bar(kGDpFull));
        umma_commit(bar(kGVEmpty + v.s));
        v.next(2);
        ok = mbar_wait(bar(kGAccEmpty), (it & 1) ^ 1, abort_flag, a.status);
        for (int j = 0; j < w.n_kt && ok; ++j, ++seq) {
          const uint32_t st = seq & 1, ks = k.s;
          const bool more = j + 1 < w.n_kt;
          k.next(3);
          if (more) {
            ok = mbar_wait(bar(kGKFull + k.s), k.ph, abort_flag, a.status);
            if (!ok) break;
            mma_tiles(tm + kGTmS + (st ^ 1) * 128, q_lo, kk_lo + k.s * T);
            umma_commit(bar(kGSFull + (st ^ 1)));
            ok = mbar_wait(bar(kGVFull + v.s), v.ph, abort_flag, a.status);
          } else if (w.m - j * 128 < 128) {   // K's rows behind the last key are cleared
            mbar_arrive(bar(kGReq));
            ok = mbar_wait(bar(kGClean), cn & 1, abort_flag, a.status);
            ++cn;
          }
          ok = ok && mbar_wait(bar(kGZFull), seq & 1, abort_flag, a.status);
          if (!ok) break;
          tc_fence_after();
          if (more) {
            mma_tiles(tm + kGTmDP, do_lo, vk_lo + v.s * T);
            umma_commit(bar(kGDpFull));
            umma_commit(bar(kGVEmpty + v.s));
            v.next(2);
          }
          mma_from_tmem(tm + kGTmDQ, tm + kGTmS + st * 128, km_lo + ks * T, j > 0);
          umma_commit(bar(kGKEmpty + ks));
        }
        if (!ok) break;
        umma_commit(bar(kGAccFull));
        umma_commit(bar(kGQEmpty));
        ++it;
      }
      umma_commit(bar(kGDrain));
      mbar_wait_drain(bar(kGDrain), 0);
    } else if (warp == 2) {
      // -------------------------------------------------------- K cleaner
      // (dZ of the keys behind the last is 0, but 0 times a NaN would not
      // be).  The issuer asks when the item's last tile has landed and the
      // score products that read it are issued or done.
      uint32_t seq = 0, cn = 0;
      bool ok = true;
      for (uint32_t n = 0; ok && q_item<R>(a, next_item(n, true), n_work, w); ++n) {
        seq += w.n_kt;
        const int rem = w.m - (w.n_kt - 1) * 128;
        if (w.n_kt == 0 || rem >= 128) continue;
        const uint32_t last = seq - 1;
        ok = mbar_wait(bar(kGReq), cn & 1, abort_flag, a.status) &&
             mbar_wait(bar(kGKFull + last % 3), (last / 3) & 1, abort_flag, a.status);
        ++cn;
        if (!__all_sync(0xffffffffu, ok)) break;
        clear_rows(smem + kBSLong + (last % 3) * kBTile, rem, lane, 32);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kGClean));
      }
    }
  } else {
    // ---------------------------------------------------------- softmax
    regs_inc<kBRegsSoftmax>();
    const int hc = (warp - 4) >> 2;                  // keys 64 hc .. of each tile
    const int row = (warp & 3) * 32 + lane;          // TMEM lane
    const uint32_t tl = tm + (uint32_t((warp & 3) * 32) << 16);
    const int qi = row / R, hh = row % R;
    const float2 sc2 = f2_dup(a.scale_log2);
    uint32_t seq = 0, it = 0;
    bool ok = true;
    for (uint32_t n = 0; ok && q_item<R>(a, next_item(n, true), n_work, w); ++n) {
      const bool valid = qi < w.n;
      const size_t qrow = size_t(w.q0 + qi) * a.H + w.g * R + hh;
      uint16_t *dq = a.dq + qrow * kHeadDim + hc * 64;
      if (w.n_kt == 0) {                             // no row of the tile sees a key
        if (valid) {
#pragma unroll
          for (int c = 0; c < 8; ++c) reinterpret_cast<uint4 *>(dq)[c] = make_uint4(0u, 0u, 0u, 0u);
        }
        continue;
      }
      const float2 stt = valid ? a.stat[qrow] : make_float2(0.f, 0.f);
      const float2 nl2 = f2_dup(stt.x), nd2 = f2_dup(stt.y);
      for (int j = 0; j < w.n_kt; ++j, ++seq) {
        const uint32_t ts = tl + kGTmS + (seq & 1) * 128 + hc * 64;
        ok = mbar_wait(bar(kGSFull + (seq & 1)), (seq >> 1) & 1, abort_flag, a.status);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        tc_fence_after();
        float p[64];
        load64(ts, p);
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
          const float2 x = f2_fma(make_float2(p[c], p[c + 1]), sc2, nl2);
          p[c] = fast_exp2(x.x);
          p[c + 1] = fast_exp2(x.y);
        }
        ok = mbar_wait(bar(kGDpFull), seq & 1, abort_flag, a.status);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        tc_fence_after();
        float z[64];
        load64(tl + kGTmDP + hc * 64, z);
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
          const float2 x = f2_mul(f2_add(make_float2(z[c], z[c + 1]), nd2), make_float2(p[c], p[c + 1]));
          z[c] = x.x;
          z[c + 1] = x.y;
        }
        const int lim = (valid ? w.hi0 + qi : -1) - j * 128 - hc * 64;   // last visible column
        if (__any_sync(0xffffffffu, lim < 63)) {
#pragma unroll
          for (int c = 0; c < 64; ++c) z[c] = c <= lim ? z[c] : 0.f;
        }
        store64(ts, z);
        tc_fence_before();
        mbar_arrive(bar(kGZFull));
      }
      if (!ok) break;
      ok = mbar_wait(bar(kGAccFull), it & 1, abort_flag, a.status);
      if (!__all_sync(0xffffffffu, ok)) break;
      ++it;
      tc_fence_after();
      float x[64];
      load64(tl + kGTmDQ + hc * 64, x);
      tc_fence_before();
      mbar_arrive(bar(kGAccEmpty));
      auto ptr = [&](int j) {
        const int rw = (row & ~3) + j, i = rw / R;
        return i < w.n ? a.dq + (size_t(w.q0 + i) * a.H + w.g * R + rw % R) * kHeadDim : nullptr;
      };
      quad_store32(x, a.scale, hc * 8, ptr);
      quad_store32(x + 32, a.scale, hc * 8 + 4, ptr);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tm, 512);
  }
  grid_dep_wait();
}

template <int R>
cudaError_t launch_bwd_r(const CUtensorMap &tq, const CUtensorMap &tdo, const CUtensorMap &tk,
                         const CUtensorMap &tv, const DenseArgs &a, int num_sms, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(dense_dkv_kernel<R>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBSmem);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(dense_dq_kernel<R>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBSmem);
  if (e != cudaSuccess) return e;
  const long long wk = (long long)a.max_items_k * a.G, wq = (long long)a.max_items * a.G;
  if (a.nk > 0)
    dense_dkv_kernel<R><<<unsigned(wk < num_sms ? wk : num_sms), kBThreads, kBSmem, st>>>(tq, tdo, tk, tv, a);
  e = cudaGetLastError();
  if (e != cudaSuccess || a.nq == 0) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(wq < num_sms ? wq : num_sms));
  cfg.blockDim = dim3(kBThreads);
  cfg.dynamicSmemBytes = kBSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.nk > 0 ? 1 : 0;   // without keys it follows the plan, which it needs
  return cudaLaunchKernelEx(&cfg, dense_dq_kernel<R>, tq, tdo, tk, tv, a);
}

}  // namespace

cudaError_t launch_dense_varlen_backward(const CUtensorMap &tq, const CUtensorMap &tdo, const CUtensorMap &tk,
                                         const CUtensorMap &tv, const DenseArgs &a, int num_sms,
                                         cudaStream_t st) {
  cudaError_t e = launch_dense_plan(a, 128 / (a.H / a.G), num_sms, st);
  if (e != cudaSuccess) return e;
  switch (a.H / a.G) {
    case 1: return launch_bwd_r<1>(tq, tdo, tk, tv, a, num_sms, st);
    case 2: return launch_bwd_r<2>(tq, tdo, tk, tv, a, num_sms, st);
    case 4: return launch_bwd_r<4>(tq, tdo, tk, tv, a, num_sms, st);
    case 8: return launch_bwd_r<8>(tq, tdo, tk, tv, a, num_sms, st);
    case 16: return launch_bwd_r<16>(tq, tdo, tk, tv, a, num_sms, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace msa
