// spec_tree_attention_shared and spec_tree_attention_window for units of at most 16 query rows (single tokens,
// short chains, small groups) on the tcgen05 tensor cores: bf16, head_dim 128.
//
// Such a unit is bound by its keys' and values' bytes: 64 KB a tile of 128 keys take ~2800 clocks of an SM's
// share of HBM.  With the rows on the TMEM lanes, as attention_span_tc.cu has them, 16 threads would form 128
// exponentials each, one after another; here S^T = K Q^T (M = 128 keys on the lanes, N = 16 rows), so that a
// thread has one key and 16 exponentials, and O^T += V^T P^T (M = 128 columns of the head, V read as an
// MN-major operand).  P goes to shared memory key by key, as two bf16 pieces of a weight (together 2^-16 of
// it), the second in columns of O of its own: N = 32, and V is read once.
// Two groups of four warps take alternate key tiles, each with references, sums and accumulators of its own;
// a further group joins the two and writes a unit's rows while the next one is under way.
//   warp 0 Q, K by TMA; warp 2 V; warp 1 issues S^T, warp 3 O^T; warps 4-7, 8-11 softmax; 12-15 output;
//   warp 16 walks the items, and lays out what a unit's rows see.
// References: weights are formed against the row's reference at hand.  bf16 has fp32's exponents, so a weight
// of 2^60 is as good as one of 2^-1; only beyond that, and at a row's first visible key, the group agrees on
// a new one (one vote a tile, no maxima).
//
// The waits on mbarriers are bounded; one that runs out raises the abort flag.  The groups of four warps meet
// at hardware barriers as well, so their warps leave together: every such barrier carries a vote on it.
#include <cudaTypedefs.h>
#include <math.h>

#include "attention_span.cuh"
#include "tc_ptx.cuh"

namespace spec {
namespace span {
namespace rows {

constexpr int kD = 128;
constexpr int kN = 16;                        // query rows of a unit
constexpr int kKeys = 128;
constexpr int kThreads = 544;
constexpr int kAtom = 16384;                  // 128 rows x 128 B
constexpr int kTile = 2 * kAtom;
constexpr int kQAtom = kN * 128;              // Q: 16 rows x 64 columns, two of them
constexpr int kKStages = 3;
constexpr int kVStages = 2;
constexpr int kItems = 4;
constexpr int kSmemP = 2 * 2 * kQAtom;        // behind two Q buffers: P of each group, 128 B a key
constexpr int kSmemK = kSmemP + 2 * kAtom;
constexpr int kSmemV = kSmemK + kKStages * kTile;
constexpr int kSmemCtl = kSmemV + kVStages * kTile;
constexpr uint32_t kTmemCols = 256;           // S^T: group, buffer: 4 x 16; O^T from 64 on: unit parity, group: 4 x 32
constexpr uint32_t kTmemO = 64;
constexpr long long kWaitLimit = 4000000000LL;     // clock cycles (~2 s)
constexpr float kFar = 60.f;                       // log2 units
static_assert(kSmemP % 1024 == 0 && kSmemK % 1024 == 0, "swizzled tiles on 1024-byte bounds");

// An item, and what its rows see: prefix keys from lo on (and the sinks), tree keys by bit.
struct RowsItem {
  Item it;
  int lo[kN];
  uint32_t anc[kN];
  int nrows, lo_max;
};

struct Control {
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[kKStages], k_empty[kKStages], v_full[kVStages], v_empty[kVStages];
  uint64_t s_full[2][2], s_free[2][2], p_full[2], pv_done[2];
  uint64_t sum_full[2], o_full[2], o_free[2];      // by unit parity
  uint64_t item_full[kItems], item_empty[kItems], drain[2];
  alignas(16) RowsItem item[kItems];
  float sum[2][2][4][kN];         // unit parity, group, warp
  float ref[2][2][kN];
  float top[2][4][kN];            // group, warp: maxima when a reference moves
  Range range;
  uint32_t tmem;
  int abort;
  RangeScratch report;
};
constexpr int kSmemBytes = kSmemCtl + int(sizeof(Control));
static_assert(kSmemBytes <= 232448, "fits one CTA's shared memory");

__device__ __forceinline__ bool lane0_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  bool r = true;
  if ((threadIdx.x & 31) == 0) r = tc::mbar_wait(bar, parity, abort, kWaitLimit);
  return __shfl_sync(0xffffffffu, r ? 1 : 0, 0) != 0;
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  const bool ok = tc::mbar_wait(bar, parity, abort, kWaitLimit);
  return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
// the 128 threads of a group vote at its barrier
__device__ __forceinline__ bool group_any(int bar, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "barrier.cta.red.or.aligned.pred q, %1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r) : "r"(bar), "r"(v ? 1u : 0u) : "memory");
  return r != 0;
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(a), "f"(b));
  return r;
}
// Sums of v[n] over the warp's lanes: lanes 2 n and 2 n + 1 get that of n (16 shuffles).
__device__ __forceinline__ float reduce16(float (&v)[kN], int lane) {
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) {
    const bool up = (lane & (2 * o)) != 0;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float give = up ? v[i] : v[i + o];
      const float keep = up ? v[i + o] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, 2 * o);
    }
  }
  return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
}

__global__ void __launch_bounds__(kThreads, 1)
span_rows_kernel(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mK,
                 const __grid_constant__ CUtensorMap mV, const __grid_constant__ CUtensorMap mKt,
                 const __grid_constant__ CUtensorMap mVt, Dev a, int q_tokens, int kv_rows) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sP = smem + kSmemP;
  uint8_t* sK = smem + kSmemK;
  uint8_t* sV = smem + kSmemV;
  Control& c = *reinterpret_cast<Control*>(smem + kSmemCtl);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&c.q_full[i], 1);
      tc::mbar_init(&c.q_empty[i], 1);
      for (int b = 0; b < 2; ++b) {
        tc::mbar_init(&c.s_full[i][b], 1);
        tc::mbar_init(&c.s_free[i][b], 4);
      }
      tc::mbar_init(&c.p_full[i], 4);
      tc::mbar_init(&c.pv_done[i], 1);
      tc::mbar_init(&c.sum_full[i], 8);
      tc::mbar_init(&c.o_full[i], 1);
      tc::mbar_init(&c.o_free[i], 4);
      tc::mbar_init(&c.drain[i], 1);
    }
    for (int s = 0; s < kKStages; ++s) {
      tc::mbar_init(&c.k_full[s], 1);
      tc::mbar_init(&c.k_empty[s], 1);
    }
    for (int s = 0; s < kVStages; ++s) {
      tc::mbar_init(&c.v_full[s], 1);
      tc::mbar_init(&c.v_empty[s], 1);
    }
    for (int i = 0; i < kItems; ++i) {
      tc::mbar_init(&c.item_full[i], 1);
      tc::mbar_init(&c.item_empty[i], 16);        // warps 0-3, eight of the softmax, four of the output
    }
    c.abort = (tc::smem_u32(smem) & 1023u) ? 1 : 0;      // the swizzle wants 1024-byte bounds
    tc::fence_mbar_init();
  }
  if (warp == 0) {
    tc::tmem_alloc(&c.tmem, kTmemCols);
    tc::tmem_relinquish();
  } else if (warp == 2 && lane == 0) {
    tc::prefetch_tensormap(&mQ);
    tc::prefetch_tensormap(&mK);
    tc::prefetch_tensormap(&mV);
    tc::prefetch_tensormap(&mKt);
    tc::prefetch_tensormap(&mVt);
  }
  pdl_wait();
  pdl_trigger();
  if (warp == 16) {
    const Range mine = warp_range(a, blockIdx.x, *reinterpret_cast<RangeScratch*>(sK));
    if (lane == 0) c.range = mine;
  }
  tc::tc_fence_before();
  tc::fence_proxy_async_smem();      // the scratch lies where TMA writes next
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = c.tmem;
  volatile int* abort_flag = &c.abort;
  const bool layout_ok = *abort_flag == 0;
  int ni = 0;                        // items taken so far
  auto take = [&](bool one_lane) -> bool {
    uint64_t* bar = &c.item_full[ni % kItems];
    const uint32_t parity = (ni / kItems) & 1;
    return one_lane ? tc::mbar_wait(bar, parity, abort_flag, kWaitLimit) : warp_wait(bar, parity, abort_flag);
  };
  auto give_back = [&](bool one_lane) {
    if (!one_lane) __syncwarp();
    if (one_lane || lane == 0) tc::mbar_arrive(&c.item_empty[ni % kItems]);
    ++ni;
  };
  if (!layout_ok) {
    // fall through to the end: the range is reported
  } else if (warp == 16) {
    // ===================================================================== items
    const Range R = c.range;
    Walker w;
    if (lane == 0) w.start(R);
    bool more = true, ok = true;
    for (int n = 0; more && ok; ++n) {
      const int s = n % kItems;
      if (n >= kItems) ok = lane0_wait(&c.item_empty[s], (n / kItems - 1) & 1, abort_flag);
      if (!ok) break;
      RowsItem& r = c.item[s];
      if (lane == 0) {
        more = w.next(a, R, r.it);
        if (!more) r.it.j0 = r.it.j1 = -1;
      }
      more = __shfl_sync(0xffffffffu, more ? 1 : 0, 0) != 0;
      __syncwarp();
      if (more) {
        const Item& it = r.it;
        const int nrows = it.T * a.G;
        if (lane < kN) {
          int lo = it.lo;
          uint32_t anc = 0;
          if (lane < nrows && it.end > it.P) {
            const uint32_t* arow = a.anc + size_t(it.o + lane / a.G) * a.W;
            if (a.window > 0) {
              uint32_t words[8];
              lo = window_words(a, arow, it.P, words);
              anc = words[0];
            } else {
              anc = arow[0];
            }
            anc &= (1u << it.T) - 1u;       // T <= 16 here
          }
          r.lo[lane] = lo;
          r.anc[lane] = anc;
        }
        if (lane == 0) {
          r.nrows = nrows;
          r.lo_max = a.window > 0 ? int(max(0LL, (long long)it.P + it.T - a.window)) : it.lo;
        }
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&c.item_full[s]);
    }
    if (!ok && lane == 0) *abort_flag = 1;
  } else if (warp == 0 || warp == 2) {
    // ===================================================================== TMA producers
    const bool is_k = warp == 0;
    const CUtensorMap* page_map = is_k ? &mK : &mV;
    const CUtensorMap* tile_map = is_k ? &mKt : &mVt;
    const int nstage = is_k ? kKStages : kVStages;
    uint8_t* ring = is_k ? sK : sV;
    uint64_t* full = is_k ? c.k_full : c.v_full;
    uint64_t* empty = is_k ? c.k_empty : c.v_empty;
    const int npg = kKeys / a.bs, page_bytes = a.bs * 128;
    int kt = 0, qn = 0;
    bool ok = true;
    while (ok) {
      ok = take(false);
      if (!ok || c.item[ni % kItems].it.j1 < 0) break;
      const Item it = c.item[ni % kItems].it;
      give_back(false);
      const int32_t* table = a.block_table + size_t(it.table) * a.max_blocks;
      // the physical page of this lane's page of tile j: -1 if no row sees it (read as zeros), -2 if bad
      auto tile_page = [&](int j) -> int {
        if (lane >= npg) return -1;
        const int first = key_base(a, it.nt0, it.w0, j) + lane * a.bs;
        if (!page_needed(first, a.bs, it.lo, it.sink, it.end)) return -1;
        const int pb = table[first / a.bs];
        if (pb >= 0 && pb < a.num_blocks) return pb;
        flag(a, it.req, it.nreq, SPEC_REQ_BAD_BLOCK);
        return -2;
      };
      int pb = tile_page(it.j0);
      if (is_k) {
        const int b = qn & 1;
        if (qn > 1) ok = lane0_wait(&c.q_empty[b], ((qn >> 1) - 1) & 1, abort_flag);
        if (!ok) break;
        if (lane == 0) {
          uint8_t* dst = smem + b * 2 * kQAtom;
          tc::mbar_arrive_expect_tx(&c.q_full[b], 2 * q_tokens * a.G * 128);
          tc::tma_load_3d(dst, &mQ, 0, it.h * a.G, it.o, &c.q_full[b]);
          tc::tma_load_3d(dst + kQAtom, &mQ, 64, it.h * a.G, it.o, &c.q_full[b]);
        }
        ++qn;
      }
      for (int j = it.j0; ok && j < it.j1; ++j, ++kt) {
        const int ahead = j + 1 < it.j1 ? tile_page(j + 1) : -1;
        const int st = kt % nstage, use = kt / nstage;
        if (use > 0) ok = lane0_wait(&empty[st], (use - 1) & 1, abort_flag);
        if (!ok) break;
        const int pb0 = __shfl_sync(0xffffffffu, pb, 0);
        const bool run = __all_sync(0xffffffffu, lane >= npg || pb == pb0 + lane) && pb0 >= 0;
        if (lane == 0) tc::mbar_arrive_expect_tx(&full[st], kTile);
        __syncwarp();
        uint8_t* dst = ring + st * kTile;
        if (run) {
          if (lane == 0) {
            tc::tma_load_4d(dst, tile_map, 0, 0, it.h, pb0, &full[st]);
            tc::tma_load_4d(dst + kAtom, tile_map, 64, 0, it.h, pb0, &full[st]);
          }
        } else if (lane < npg) {
          const int row = pb >= 0 ? (pb * a.H_kv + it.h) * a.bs : kv_rows;      // past the cache: zeros
          tc::tma_load_2d(dst + lane * page_bytes, page_map, 0, row, &full[st]);
          tc::tma_load_2d(dst + kAtom + lane * page_bytes, page_map, 64, row, &full[st]);
        }
        __syncwarp();
        pb = ahead;
      }
    }
    if (lane == 0) {
      if (!ok) *abort_flag = 1;
      // no copy may be in flight when the CTA ends
      volatile int never = 0;
      for (int k = max(0, kt - nstage); k < kt; ++k)
        tc::mbar_wait(&full[k % nstage], (k / nstage) & 1, &never, kWaitLimit / 8);
      for (int k = max(0, qn - 2); k < qn; ++k)
        tc::mbar_wait(&c.q_full[k & 1], (k >> 1) & 1, &never, kWaitLimit / 8);
    }
  } else if (warp == 1 || warp == 3) {
    // ===================================================================== MMA issuers
    const bool is_qk = warp == 1;
    if (elect_one()) {
      const uint32_t id_qk = tc::idesc_bf16_f32(128, kN, false, false);
      const uint32_t id_pv = tc::idesc_bf16_f32(128, 2 * kN, true, true);
      const uint64_t dQ0 = tc::smem_desc(tc::smem_u32(smem), 16, 1024), dK0 = tc::smem_desc(tc::smem_u32(sK), 16, 1024);
      const uint64_t dV0 = tc::smem_desc(tc::smem_u32(sV), kAtom, 1024), dP0 = tc::smem_desc(tc::smem_u32(sP), kAtom, 1024);
      int kt = 0, li = 0, gn[2] = {0, 0};      // tiles; items; tiles of each group
      bool ok = true;
      for (; ok; ++li) {
        ok = take(true);
        const Item& it = c.item[ni % kItems].it;
        if (!ok || it.j1 < 0) break;
        const int nt = it.j1 - it.j0;
        give_back(true);
        if (is_qk) {
          ok = tc::mbar_wait(&c.q_full[li & 1], (li >> 1) & 1, abort_flag, kWaitLimit);
          for (int k = 0; ok && k < nt; ++k, ++kt) {
            const int g = k & 1, n = g == 0 ? gn[0]++ : gn[1]++, buf = n & 1, st = kt % kKStages;
            // (the third wait: the product before in V's stage, so that whoever has S of a tile finds the stage
            // free of older tiles, and the phase of its barrier is the tile's own)
            ok = tc::mbar_wait(&c.k_full[st], (kt / kKStages) & 1, abort_flag, kWaitLimit) &&
                 (kt < kVStages || tc::mbar_wait(&c.v_empty[kt % kVStages], (kt / kVStages - 1) & 1, abort_flag, kWaitLimit)) &&
                 (n < 2 || tc::mbar_wait(&c.s_free[g][buf], ((n >> 1) - 1) & 1, abort_flag, kWaitLimit));
            if (!ok) break;
            tc::tc_fence_after();
            const uint64_t dk = dK0 + uint64_t(st) * (kTile >> 4), dq = dQ0 + uint64_t(li & 1) * (2 * kQAtom >> 4);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              tc::mma_bf16_ss(tmem + 16 * (2 * g + buf), dk + uint64_t(((kk >> 2) * kAtom + (kk & 3) * 32) >> 4),
                              dq + uint64_t(((kk >> 2) * kQAtom + (kk & 3) * 32) >> 4), id_qk, kk > 0 ? 1u : 0u);
            tc::mma_commit(&c.s_full[g][buf]);
            tc::mma_commit(&c.k_empty[st]);
            if (k + 1 == nt) tc::mma_commit(&c.q_empty[li & 1]);
          }
        } else {
          const int par = li & 1;
          // the output warps have to have read what this parity's accumulators held
          if (li > 1) ok = tc::mbar_wait(&c.o_free[par], ((li >> 1) - 1) & 1, abort_flag, kWaitLimit);
          for (int k = 0; ok && k < nt; ++k, ++kt) {
            const int g = k & 1, n = g == 0 ? gn[0]++ : gn[1]++, st = kt % kVStages;
            ok = tc::mbar_wait(&c.p_full[g], n & 1, abort_flag, kWaitLimit) &&
                 tc::mbar_wait(&c.v_full[st], (kt / kVStages) & 1, abort_flag, kWaitLimit);
            if (!ok) break;
            tc::tc_fence_after();
            const uint64_t dv = dV0 + uint64_t(st) * (kTile >> 4), dp = dP0 + uint64_t(g) * (kAtom >> 4);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)      // 16 keys: 2048 bytes of V and of P
              tc::mma_bf16_ss(tmem + kTmemO + 32 * (2 * par + g), dv + uint64_t(kk * (2048 >> 4)), dp + uint64_t(kk * (2048 >> 4)),
                              id_pv, kk > 0 || k > 1 ? 1u : 0u);
            tc::mma_commit(&c.v_empty[st]);
            tc::mma_commit(&c.pv_done[g]);
          }
          if (ok) tc::mma_commit(&c.o_full[par]);
        }
      }
      if (!ok) *abort_flag = 1;
      // TMEM may not be freed under a product
      tc::mma_commit(&c.drain[is_qk ? 0 : 1]);
      volatile int never = 0;
      tc::mbar_wait(&c.drain[is_qk ? 0 : 1], 0, &never, kWaitLimit / 8);
    }
  } else if (warp >= 12) {
    // ===================================================================== output
    if (warp == 12 && reports(c.range, gridDim.x)) write_recs(a, c.report);
    const int q4 = warp & 3, d = q4 * 32 + lane;       // this thread's column of the head
    const uint32_t lane_addr = uint32_t(q4 * 32) << 16;
    bool ok = true;
    for (int li = 0; ok; ++li) {
      ok = take(false);
      if (!ok || c.item[ni % kItems].it.j1 < 0) break;
      const RowsItem& r = c.item[ni % kItems];
      const Item& it = r.it;
      const int par = li & 1;
      const bool two = it.j1 - it.j0 > 1;
      ok = warp_wait(&c.o_full[par], (li >> 1) & 1, abort_flag) && warp_wait(&c.sum_full[par], (li >> 1) & 1, abort_flag);
      if (!ok) break;
      tc::tc_fence_after();
      uint32_t o0[32], o1[32];
      tc::tmem_ld32(tmem + lane_addr + kTmemO + 32 * (2 * par), o0);
      if (two) tc::tmem_ld32(tmem + lane_addr + kTmemO + 32 * (2 * par + 1), o1);
      tc::tmem_ld_wait();
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        if (n < r.nrows) {
          const float r0 = c.ref[par][0][n], r1 = two ? c.ref[par][1][n] : -INFINITY;
          const float M = fmaxf(r0, r1);
          // (without a reference the sum is 0, or NaN of a row that saw nothing else)
          const float s0 = (c.sum[par][0][0][n] + c.sum[par][0][1][n]) + (c.sum[par][0][2][n] + c.sum[par][0][3][n]);
          const float s1 = two ? (c.sum[par][1][0][n] + c.sum[par][1][1][n]) + (c.sum[par][1][2][n] + c.sum[par][1][3][n]) : 0.f;
          const float w0 = r0 == -INFINITY ? s0 : ex2(r0 - M), w1 = r1 == -INFINITY ? s1 : ex2(r1 - M);
          float l = 0.f, v = 0.f;
          if (w0 != 0.f) {
            l = w0 * s0;
            v = w0 * (__uint_as_float(o0[n]) + __uint_as_float(o0[kN + n]));
          }
          if (w1 != 0.f) {
            l += w1 * s1;
            v += w1 * (__uint_as_float(o1[n]) + __uint_as_float(o1[kN + n]));
          }
          v = l == 0.f ? 0.f : v / l;
          const float lse2 = l == 0.f ? -INFINITY : M + log2f(l);
          const int t = n / a.G;
          const size_t out = size_t(it.o + t) * a.H_q + it.h * a.G + (n - t * a.G);
          if (it.slot == -1) {
            static_cast<__nv_bfloat16*>(a.o)[out * kD + d] = __float2bfloat16_rn(v);
            if (d == 0 && a.lse) a.lse[out] = lse2 * 0.6931471805599453f;
          } else if (it.slot >= 0) {
            a.part_o[(size_t(it.slot) * a.part_rows + n) * kD + d] = v;
            if (d == 0) a.part_lse[size_t(it.slot) * a.part_rows + n] = lse2;
          } else {
            const size_t at = size_t(it.slot == -2 ? 0 : 1) * a.N * a.H_q + out;
            a.row_o[at * kD + d] = v;
            if (d == 0) a.row_lse[at] = lse2;
          }
        }
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&c.o_free[par]);
      give_back(false);
    }
    if (!ok) *abort_flag = 1;
  } else {
    // ===================================================================== softmax
    const int g = (warp - 4) >> 2, q4 = warp & 3, kl = q4 * 32 + lane;     // group; this thread's key of a tile
    const int bar = 1 + g;
    const uint32_t lane_addr = uint32_t(q4 * 32) << 16;
    const float sl2 = a.scale_log2;
    uint8_t* sPg = sP + g * kAtom;
    int sn = 0, kt0 = 0;       // tiles of this group; tiles before the item
    bool ok = true;
    for (int li = 0;; ++li) {
      ok = take(false);
      if (group_any(bar, !ok)) { ok = false; break; }
      const RowsItem& r = c.item[ni % kItems];
      if (r.it.j1 < 0) break;
      const int par = li & 1, j0 = r.it.j0, nt = r.it.j1 - j0, nt0 = r.it.nt0, skip = r.it.w0 - nt0, P = r.it.P, nrows = r.nrows;
      const int lo_max = r.lo_max;
      float neg[kN], sum[kN];      // -reference (+inf: none yet; -inf: not a row); sums
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        neg[n] = n < nrows ? INFINITY : -INFINITY;
        sum[n] = 0.f;
      }
      bool leave = false;
      for (int k = g; k < nt; k += 2, ++sn) {
        const int j = j0 + k, kb = (j < nt0 ? j : j + skip) * kKeys, key = kb + kl;
        const bool masked = !(kb + kKeys <= P && (kb >= lo_max || kb + kKeys <= a.sinks));
        uint32_t vis = (1u << kN) - 1u;
        if (masked) {
          vis = 0;
          const int tree = key - P;
#pragma unroll
          for (int n = 0; n < kN; ++n) {
            const bool v = tree < 0 ? key >= r.lo[n] || key < a.sinks : tree < 32 && ((r.anc[n] >> (tree & 31)) & 1u);
            vis |= n < nrows && v ? 1u << n : 0u;
          }
        }
        ok = ok && warp_wait(&c.s_full[g][sn & 1], (sn >> 1) & 1, abort_flag);
        bool broken = false;         // V of this thread's key is not finite
        if (ok && masked) {
          // V's rows, 32 a warp, eight lanes a row.  S of this tile was issued after the product that read the
          // older tile in V's stage.
          const int gv = kt0 + k, st = gv % kVStages;
          ok = warp_wait(&c.v_full[st], (gv / kVStages) & 1, abort_flag);
          if (ok) {
            uint8_t* tile = sV + st * kTile + (q4 * 32 + (lane >> 3)) * 128 + (lane & 7) * 16;
            const int key0 = kb + q4 * 32 + (lane >> 3), end = r.it.end, sink = r.it.sink, lo = r.it.lo;
            uint32_t word = 0;
            bool wrote = false;
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
              uint8_t* p = tile + half * kAtom;
              uint32_t hits = 0;           // bit i: an exponent of all ones in row 4 i + lane / 8
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const uint4 x = *reinterpret_cast<const uint4*>(p + i * 512);
                const int kk = key0 + 4 * i;
                const bool seen = kk < sink || (kk >= lo && kk < end);
                // the addition carries into a half word's sign bit from an exponent of all ones only
                const uint32_t t = ((x.x & 0x7f807f80u) + 0x00800080u) | ((x.y & 0x7f807f80u) + 0x00800080u) |
                                   ((x.z & 0x7f807f80u) + 0x00800080u) | ((x.w & 0x7f807f80u) + 0x00800080u);
                if (!seen) {
                  *reinterpret_cast<uint4*>(p + i * 512) = make_uint4(0, 0, 0, 0);
                  wrote = true;
                } else if (t & 0x80008000u) {
                  hits |= 1u << i;
                }
              }
              if (__any_sync(0xffffffffu, hits != 0u)) {
#pragma unroll 1
                for (int i = 0; i < 8; ++i) {
                  const bool hit = (hits >> i) & 1u;
                  if (hit) {
                    uint32_t* w = reinterpret_cast<uint32_t*>(p + i * 512);
                    for (int e = 0; e < 4; ++e) {
                      if ((w[e] & 0x7f80u) == 0x7f80u) w[e] &= 0xffff0000u;
                      if ((w[e] & 0x7f800000u) == 0x7f800000u) w[e] &= 0xffffu;
                    }
                    wrote = true;
                  }
                  const uint32_t lanes = __ballot_sync(0xffffffffu, hit);
                  for (int e = 0; e < 4; ++e) word |= ((lanes >> (8 * e)) & 0xffu) ? 1u << (4 * i + e) : 0u;
                }
              }
            }
            if (wrote) tc::fence_proxy_async_smem();
            broken = (word >> lane) & 1u;      // a warp looks at its own lanes' keys
          }
        }
        uint32_t x[kN];
        if (ok) {
          tc::tc_fence_after();
          tc::tmem_ld16(tmem + lane_addr + 16 * (2 * g + (sn & 1)), x);
          tc::tmem_ld_wait();
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&c.s_free[g][sn & 1]);
        } else {
#pragma unroll
          for (int n = 0; n < kN; ++n) x[n] = 0;
        }
        if (masked) {
#pragma unroll
          for (int n = 0; n < kN; ++n) {
            // a masked score is the most negative number there is, so that it stays one when a reference is
            // taken off; a row that sees a key whose V is not finite becomes NaN
            if (!((vis >> n) & 1u)) x[n] = __float_as_uint(-3.0e38f);
            else if (broken) x[n] = __float_as_uint(NAN);
          }
        }
        // exponents; beyond kFar (a row's first visible key: +inf) the references move
        float y[kN];
        auto exponents = [&] {
          const uint64_t slv = f2_pack(sl2, sl2);
#pragma unroll
          for (int n = 0; n < kN; n += 2)
            f2_unpack(f2_fma(f2_pack(__uint_as_float(x[n]), __uint_as_float(x[n + 1])), slv, f2_pack(neg[n], neg[n + 1])), y[n], y[n + 1]);
          if (masked) {
#pragma unroll
            for (int n = 0; n < kN; ++n) y[n] = (vis >> n) & 1u ? y[n] : -INFINITY;
          }
        };
        exponents();
        float ym = fmaxf(y[0], y[1]);
#pragma unroll
        for (int n = 2; n < kN; n += 2) ym = fmax3(ym, y[n], y[n + 1]);
        if (group_any(bar, ym > kFar || !ok)) {
          if (group_any(bar, !ok)) { leave = true; break; }
          // the group's maxima of all rows
#pragma unroll
          for (int n = 0; n < kN; ++n) {
            const float v = n < nrows && ((vis >> n) & 1u) ? __uint_as_float(x[n]) * sl2 : -INFINITY;
            const float t = warp_max(v);
            if (lane == 0) c.top[g][q4][n] = t;
          }
          ok = k == g || warp_wait(&c.pv_done[g], (sn - 1) & 1, abort_flag);
          if (group_any(bar, !ok)) { leave = true; break; }       // and the maxima are there
          tc::tc_fence_after();
          float f[kN];
#pragma unroll
          for (int n = 0; n < kN; ++n) {
            const float t = fmaxf(fmaxf(c.top[g][0][n], c.top[g][1][n]), fmaxf(c.top[g][2][n], c.top[g][3][n]));
            f[n] = 1.f;
            if (n < nrows && t > -neg[n]) {
              f[n] = neg[n] == INFINITY ? 1.f : ex2(-neg[n] - t);
              neg[n] = -t;
            }
            sum[n] *= f[n];
          }
          if (k != g) {
            uint32_t o[32];
            const uint32_t to = tmem + lane_addr + kTmemO + 32 * (2 * par + g);
            tc::tmem_ld32(to, o);
            tc::tmem_ld_wait();
#pragma unroll
            for (int n = 0; n < 32; ++n) o[n] = __float_as_uint(__uint_as_float(o[n]) * f[n & (kN - 1)]);
            tc::tmem_st32(to, o);
            tc::tmem_st_wait();
          }
          exponents();
          if (group_any(bar, false)) { leave = true; break; }     // the maxima have been read
        }
        uint32_t hi[kN / 2], lo[kN / 2];
#pragma unroll
        for (int n = 0; n < kN; n += 2) {
          const float p0 = ex2(y[n]), p1 = ex2(y[n + 1]);
          sum[n] += p0;
          sum[n + 1] += p1;
          hi[n / 2] = pack_bf16(p0, p1);
          lo[n / 2] = pack_bf16(p0 - bf16_lo(hi[n / 2]), p1 - bf16_hi(hi[n / 2]));
        }
        // the product that read this group's last P
        if (sn > 0) ok = ok && warp_wait(&c.pv_done[g], (sn - 1) & 1, abort_flag);
        uint8_t* prow = sPg + kl * 128;
        const int sw = kl & 7;
        *reinterpret_cast<uint4*>(prow + ((0 ^ sw) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(prow + ((1 ^ sw) << 4)) = make_uint4(hi[4], hi[5], hi[6], hi[7]);
        *reinterpret_cast<uint4*>(prow + ((2 ^ sw) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        *reinterpret_cast<uint4*>(prow + ((3 ^ sw) << 4)) = make_uint4(lo[4], lo[5], lo[6], lo[7]);
        tc::fence_proxy_async_smem();
        tc::tc_fence_before();
        __syncwarp();
        // (after a wait that ran out nothing reads P any more: the next vote ends the group)
        if (lane == 0) tc::mbar_arrive(&c.p_full[g]);
      }
      if (leave) { ok = false; break; }
      // the unit's sums; the output warps have to have read the ones before of this parity
      const float total = reduce16(sum, lane);
      bool fine = li < 2 || warp_wait(&c.o_free[par], ((li >> 1) - 1) & 1, abort_flag);
      fine = fine && ok;
      if ((lane & 1) == 0) c.sum[par][g][q4][lane >> 1] = total;
      if (q4 == 0 && lane < kN) {
        float v = neg[0];
#pragma unroll
        for (int n = 1; n < kN; ++n) v = lane == n ? neg[n] : v;
        c.ref[par][g][lane] = -v;
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&c.sum_full[par]);
      ok = fine;
      kt0 += nt;
      give_back(false);
      if (group_any(bar, !ok)) { ok = false; break; }
    }
    if (!ok) *abort_flag = 1;
  }
  tc::tc_fence_before();
  __syncthreads();
  if (*abort_flag && tid == 0) {
    // every request of the range is unreliable after a wait that ran out
    const Range R = c.range;
    Walker w;
    w.start(R);
    Item it;
    while (w.next(a, R, it)) flag(a, it.req, it.nreq, SPEC_REQ_TIMEOUT);
  }
  tc::tc_fence_after();
  if (warp == 0) tc::tmem_dealloc(tmem, kTmemCols);
}

}  // namespace rows

spec_status_t launch_span_rows(const Dev& d, const TcMaps& m, cudaStream_t s) {
  static DeviceOnce raised;
  const spec_status_t st = raise_dyn_smem_once(rows::span_rows_kernel, rows::kSmemBytes, raised);
  if (st != SPEC_OK) return st;
  return launch_result(launch_pdl(rows::span_rows_kernel, dim3(d.ctas), dim3(rows::kThreads), size_t(rows::kSmemBytes), s,
                                  m.q_rows, m.k_page, m.v_page, m.k_tile, m.v_tile, d, m.q_rows_tokens, m.kv_rows));
}

}  // namespace span
}  // namespace spec
