// spec_tree_attention_window for at most 16 query rows a request and head (single tokens, short chains) on the
// tcgen05 tensor cores: bf16, head_dim 128.
//
// Such a unit is bound by its keys' and values' bytes: 64 KB a tile of 128 keys take ~2800 clocks of an SM's
// share of HBM.  With the rows on the TMEM lanes, as attention_span_tc.cu has them, 16 threads would form 128
// exponentials each, one after another; here S^T = K Q^T (M = 128 keys on the lanes, N = 16 rows), so that a
// thread has one key and 16 exponentials, and O^T += V^T P^T (M = 128 columns of the head, V read as an
// MN-major operand).  P goes to shared memory key by key, as two bf16 pieces of a weight (together 2^-16 of
// it), the second in columns of O of its own: N = 32, and V is read once.
// Two groups of four warps take alternate key tiles, each with references, sums and accumulators of its own;
// a further group joins the two and writes a unit's rows while the next one is under way.
//   warp 0 Q and K by TMA, warp 2 V; warp 1 issues S^T two tiles ahead of O^T, across units; warp 3 walks the
//   items and lays out what a unit's rows see; warps 4-7, 8-11 softmax; 12-15 output.
// References: weights are formed against the row's reference at hand.  bf16 has fp32's exponents, so a weight
// of 2^60 is as good as one of 2^-1; only beyond that, and at a row's first visible key, the group agrees on
// a new one (one vote a tile, no maxima), once a tile: the new one is the largest score rounded down, so that it
// may lie below that score by a step of fp32 in the end, which at 2^30 is more than 60.  Weights stop at 2^60, which
// moves scores by less than that step; the fused product is rounded once in it as well.
//
// What runs once a unit (a reference's first setting, the output, masks) is kept short in instructions rather
// than in steps: it comes from beyond the instruction cache every time.  The output unrolled over 16 rows with
// its divisions and addresses took 5000 .. 28000 clocks a unit, as below 1000.
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
constexpr int kThreads = 512;                 // 128 registers a thread
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
constexpr uint32_t kTmemCols = 256;           // S^T: a group's 16; O^T from 64 on: unit parity, group: 4 x 32
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
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint64_t sum_full[2], o_full[2], o_free[2];      // by unit parity
  uint64_t item_full[kItems], item_empty[kItems], drain;
  alignas(16) RowsItem item[kItems];
  float sum[2][2][4][kN];         // unit parity, group, warp
  float ref[2][2][kN];
  alignas(16) float top[2][4][kN];      // group, warp: maxima when a reference moves
  Range range;
  Entry first;
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(RangeScratch) <= size_t(kKStages * kTile), "the search's scratch lies in the tiles");
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
// 32 lanes x 8 consecutive 32-bit columns
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
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
// Sums (or maxima) of v[n] over the warp's lanes: lanes 2 n and 2 n + 1 get that of n (16 shuffles).
template <bool kMax>
__device__ __forceinline__ float reduce16(float (&v)[kN], int lane) {
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) {
    const bool up = (lane & (2 * o)) != 0;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float give = up ? v[i] : v[i + o];
      const float keep = up ? v[i + o] : v[i];
      const float got = __shfl_xor_sync(0xffffffffu, give, 2 * o);
      v[i] = kMax ? fmaxf(keep, got) : keep + got;
    }
  }
  const float got = __shfl_xor_sync(0xffffffffu, v[0], 1);
  return kMax ? fmaxf(v[0], got) : v[0] + got;
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
      tc::mbar_init(&c.s_full[i], 1);
      tc::mbar_init(&c.p_full[i], 4);
      tc::mbar_init(&c.pv_done[i], 1);
      tc::mbar_init(&c.sum_full[i], 8);
      tc::mbar_init(&c.o_full[i], 1);
      tc::mbar_init(&c.o_free[i], 4);
    }
    tc::mbar_init(&c.drain, 1);
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
      tc::mbar_init(&c.item_empty[i], 15);        // warps 0, 1, 2, eight of the softmax, four of the output
    }
    c.abort = (tc::smem_u32(smem) & 1023u) ? 1 : 0;      // the swizzle wants 1024-byte bounds
    tc::fence_mbar_init();
  }
  if (warp == 0) {
    tc::tmem_alloc(&c.tmem, kTmemCols);
    tc::tmem_relinquish();
  } else if (warp == 1 && lane == 0) {
    tc::prefetch_tensormap(&mQ);
    tc::prefetch_tensormap(&mK);
    tc::prefetch_tensormap(&mV);
    tc::prefetch_tensormap(&mKt);
    tc::prefetch_tensormap(&mVt);
  }
  pdl_wait();
  pdl_trigger();
  find_range(a, *reinterpret_cast<RangeScratch*>(sK), c.range, c.first);
  tc::tc_fence_before();
  tc::fence_proxy_async_smem();      // the scratch lies where TMA writes next
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = c.tmem;
  volatile int* abort_flag = &c.abort;
  const bool layout_ok = *abort_flag == 0;
  int ni = 0;                        // items taken so far
  auto take = [&]() -> bool { return warp_wait(&c.item_full[ni % kItems], (ni / kItems) & 1, abort_flag); };
  auto give_back = [&] {
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&c.item_empty[ni % kItems]);
    ++ni;
  };
  if (!layout_ok) {
    // fall through to the end: the range is reported
    if (warp == 12 && reports(c.range, gridDim.x)) clear_recs(a);
  } else if (warp == 3) {
    // ===================================================================== items
    const Range R = c.range;
    Walker w;
    if (lane == 0) w.start(R, &c.first);
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
          if (lane < nrows) {
            anc = mask_word(a.anc + size_t(it.o + lane / a.G) * a.W, 0, it.T);      // T <= 16 here
            lo = window_words(a, &anc, 1, it.P);
          }
          r.lo[lane] = lo;
          r.anc[lane] = anc;
        }
        if (lane == 0) {
          r.nrows = nrows;
          r.lo_max = int(max(0LL, (long long)it.P + it.T - a.window));
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
      ok = take();
      if (!ok || c.item[ni % kItems].it.j1 < 0) break;
      const Item it = c.item[ni % kItems].it;
      give_back();
      const int32_t* table = a.block_table + size_t(it.table) * a.max_blocks;
      // the physical page of this lane's page of tile j: -1 if no row sees it (read as zeros), -2 if bad
      auto tile_page = [&](int j) -> int {
        if (lane >= npg) return -1;
        const int first = key_base(a, it.nt0, it.w0, j) + lane * a.bs;
        if (!page_needed(first, a.bs, it.lo, it.sink, it.end)) return -1;
        const int pb = table[first / a.bs];
        if (pb >= 0 && pb < a.num_blocks) return pb;
        flag(a, it.req, 1, SPEC_REQ_BAD_BLOCK);
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
  } else if (warp == 1) {
    // ===================================================================== MMA issuer
    // One thread issues S(0) S(1) | O(t) S(t+2) | ..: a group's S goes over the one that its P came from, and
    // whoever has S of tile t + 2 knows that O's product of tile t is done and V's stage free.
    if (elect_one()) {
      const uint32_t id_qk = tc::idesc_bf16_f32(128, kN, false, false);
      const uint32_t id_pv = tc::idesc_bf16_f32(128, 2 * kN, true, true);
      const uint64_t dQ0 = tc::smem_desc(tc::smem_u32(smem), 16, 1024), dK0 = tc::smem_desc(tc::smem_u32(sK), 16, 1024);
      const uint64_t dV0 = tc::smem_desc(tc::smem_u32(sV), kAtom, 1024), dP0 = tc::smem_desc(tc::smem_u32(sP), kAtom, 1024);
      bool ok = true;
      // the scores' place in the stream: item, tile of it, its tiles; tiles before; and the output's
      int qi = -1, qk = 0, qnt = 0, qt = 0, pi = -1, pk = 0, pnt = 0, pt = 0;
      bool q_end = false, p_end = false;
      auto item_tiles = [&](int i, int& nt) -> bool {       // of item i; false: the stream ends
        ok = ok && tc::mbar_wait(&c.item_full[i % kItems], (i / kItems) & 1, abort_flag, kWaitLimit);
        if (!ok) return false;
        const Item& it = c.item[i % kItems].it;
        nt = it.j1 - it.j0;
        return it.j1 >= 0;
      };
      auto score = [&] {
        if (q_end) return;
        if (qk == qnt) {
          qk = 0;
          if (!item_tiles(++qi, qnt)) { q_end = true; return; }
          ok = tc::mbar_wait(&c.q_full[qi & 1], (qi >> 1) & 1, abort_flag, kWaitLimit);
        }
        const int st = qt % kKStages;
        ok = ok && tc::mbar_wait(&c.k_full[st], (qt / kKStages) & 1, abort_flag, kWaitLimit);
        if (!ok) return;
        tc::tc_fence_after();
        const uint64_t dk = dK0 + uint64_t(st) * (kTile >> 4), dq = dQ0 + uint64_t(qi & 1) * (2 * kQAtom >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          tc::mma_bf16_ss(tmem + 16 * (qt & 1), dk + uint64_t(((kk >> 2) * kAtom + (kk & 3) * 32) >> 4),
                          dq + uint64_t(((kk >> 2) * kQAtom + (kk & 3) * 32) >> 4), id_qk, kk > 0 ? 1u : 0u);
        tc::mma_commit(&c.s_full[qt & 1]);
        tc::mma_commit(&c.k_empty[st]);
        ++qt;
        if (++qk == qnt) tc::mma_commit(&c.q_empty[qi & 1]);
      };
      while (ok && !p_end) {
        if (pk == pnt) {
          pk = 0;
          if (!item_tiles(++pi, pnt)) { p_end = true; break; }
          // the output warps have to have read what this parity's accumulators held
          if (pi > 1) ok = tc::mbar_wait(&c.o_free[pi & 1], ((pi >> 1) - 1) & 1, abort_flag, kWaitLimit);
        }
        while (ok && !q_end && qt < pt + 2) score();
        const int g = pt & 1, st = pt % kVStages, par = pi & 1;
        ok = ok && tc::mbar_wait(&c.p_full[g], (pt >> 1) & 1, abort_flag, kWaitLimit) &&
             tc::mbar_wait(&c.v_full[st], (pt / kVStages) & 1, abort_flag, kWaitLimit);
        if (!ok) break;
        tc::tc_fence_after();
        const uint64_t dv = dV0 + uint64_t(st) * (kTile >> 4), dp = dP0 + uint64_t(g) * (kAtom >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)      // 16 keys: 2048 bytes of V and of P
          tc::mma_bf16_ss(tmem + kTmemO + 32 * (2 * par + g), dv + uint64_t(kk * (2048 >> 4)), dp + uint64_t(kk * (2048 >> 4)),
                          id_pv, kk > 0 || pk > 1 ? 1u : 0u);
        tc::mma_commit(&c.v_empty[st]);
        tc::mma_commit(&c.pv_done[g]);
        ++pt;
        if (++pk == pnt) {
          tc::mma_commit(&c.o_full[par]);
          tc::mbar_arrive(&c.item_empty[pi % kItems]);
        }
      }
      if (!ok) *abort_flag = 1;
      // TMEM may not be freed under a product
      tc::mma_commit(&c.drain);
      volatile int never = 0;
      tc::mbar_wait(&c.drain, 0, &never, kWaitLimit / 8);
    }
  } else if (warp >= 12) {
    // ===================================================================== output
    if (warp == 12 && reports(c.range, gridDim.x)) write_recs(a, c.range.ordered);
    const int q4 = warp & 3, d = q4 * 32 + lane;       // this thread's column of the head
    const uint32_t lane_addr = uint32_t(q4 * 32) << 16;
    bool ok = true;
    int kt0 = 0;                                       // tiles before the item
    for (int li = 0; ok; ++li) {
      ok = take();
      if (!ok || c.item[ni % kItems].it.j1 < 0) break;
      const RowsItem& r = c.item[ni % kItems];
      const Item& it = r.it;
      const int par = li & 1;
      const int nt = it.j1 - it.j0;
      const bool has0 = nt > 1 || (kt0 & 1) == 0, has1 = nt > 1 || (kt0 & 1) == 1;     // groups with a tile of it
      kt0 += nt;
      ok = warp_wait(&c.o_full[par], (li >> 1) & 1, abort_flag) && warp_wait(&c.sum_full[par], (li >> 1) & 1, abort_flag);
      if (!ok) break;
      tc::tc_fence_after();
      // lane n: row n's weights of the groups, log-sum-exp and place
      const int n0 = lane & (kN - 1), nrows = r.nrows;
      float f0 = 0.f, f1 = 0.f, lse2;
      {
        const float r0 = has0 ? c.ref[par][0][n0] : -INFINITY, r1 = has1 ? c.ref[par][1][n0] : -INFINITY;
        // (without a reference the sum is 0, or NaN of a row that saw nothing else)
        const float s0 = has0 ? (c.sum[par][0][0][n0] + c.sum[par][0][1][n0]) + (c.sum[par][0][2][n0] + c.sum[par][0][3][n0]) : 0.f;
        const float s1 = has1 ? (c.sum[par][1][0][n0] + c.sum[par][1][1][n0]) + (c.sum[par][1][2][n0] + c.sum[par][1][3][n0]) : 0.f;
        const float M = fmaxf(r0, r1);
        const bool any0 = r0 != -INFINITY || s0 != 0.f, any1 = r1 != -INFINITY || s1 != 0.f;      // something seen
        const float w0 = r0 == -INFINITY ? s0 : ex2(r0 - M), w1 = r1 == -INFINITY ? s1 : ex2(r1 - M);
        const float l = (any0 ? w0 * s0 : 0.f) + (any1 ? w1 * s1 : 0.f);
        const float inv = l == 0.f ? 0.f : 1.f / l;
        f0 = any0 ? w0 * inv : -1.f;       // -1: what the group has does not count (a weight of 0 lets a NaN through)
        f1 = any1 ? w1 * inv : -1.f;
        lse2 = l == 0.f ? -INFINITY : M + __log2f(l);
      }
      const int t = n0 / a.G;
      const size_t row = size_t(it.o + t) * a.H_q + it.h * a.G + (n0 - t * a.G);
      const bool direct = it.slot == -1;       // else a piece: a request on its own has no other places
      const size_t at = direct ? row : size_t(it.slot) * a.part_rows + n0;
      if (q4 == 0 && lane < nrows && lane < kN) {
        if (!direct) a.part_lse[at] = lse2;
        else if (a.lse) a.lse[at] = lse2 * 0.6931471805599453f;
      }
      char* base = direct ? static_cast<char*>(a.o) : reinterpret_cast<char*>(a.part_o);
      const unsigned long long mine = reinterpret_cast<unsigned long long>(base) + at * kD * (direct ? 2 : 4);
      const uint32_t to = tmem + lane_addr + kTmemO + 64 * par;
#pragma unroll 1
      for (int n8 = 0; n8 < nrows; n8 += 8) {
        // eight rows at a time: both pieces of both groups
        uint32_t x[4][8];
        tmem_ld8(to + n8, x[0]);
        tmem_ld8(to + kN + n8, x[1]);
        tmem_ld8(to + 32 + n8, x[2]);
        tmem_ld8(to + 32 + kN + n8, x[3]);
        tc::tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float a0 = __shfl_sync(0xffffffffu, f0, n8 + i), a1 = __shfl_sync(0xffffffffu, f1, n8 + i);
          const unsigned long long dst = __shfl_sync(0xffffffffu, mine, n8 + i);
          float v = a0 < 0.f ? 0.f : a0 * (__uint_as_float(x[0][i]) + __uint_as_float(x[1][i]));
          if (!(a1 < 0.f)) v = fmaf(a1, __uint_as_float(x[2][i]) + __uint_as_float(x[3][i]), v);
          if (n8 + i < nrows) {
            if (direct) *(reinterpret_cast<__nv_bfloat16*>(dst) + d) = __float2bfloat16_rn(v);
            else *(reinterpret_cast<float*>(dst) + d) = v;
          }
        }
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&c.o_free[par]);
      give_back();
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
      ok = take();
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
      for (int k = (g ^ kt0) & 1; k < nt; k += 2, ++sn) {       // tiles alternate across units
        const int j = j0 + k, kb = (j < nt0 ? j : j + skip) * kKeys, key = kb + kl;
        const bool masked = !(kb + kKeys <= P && (kb >= lo_max || kb + kKeys <= a.sinks));
        uint32_t vis = (1u << kN) - 1u;
        if (masked) {
          vis = 0;
          const int tree = key - P;
#pragma unroll 1
          for (int n = 0; n < nrows; ++n) {
            const bool v = tree < 0 ? key >= r.lo[n] || key < a.sinks : tree < 32 && ((r.anc[n] >> (tree & 31)) & 1u);
            vis |= v ? 1u << n : 0u;
          }
        }
        ok = ok && warp_wait(&c.s_full[g], sn & 1, abort_flag);
        uint32_t x[kN];
        if (ok) {
          tc::tc_fence_after();
          tc::tmem_ld16(tmem + lane_addr + 16 * g, x);
          tc::tmem_ld_wait();
        } else {
#pragma unroll
          for (int n = 0; n < kN; ++n) x[n] = 0;
        }
        // Exponents; beyond kFar (a row's first visible key: +inf) the references move, and they are formed
        // again.  A masked key has the exponent -inf.
        float y[kN];
        for (bool moved = false;; moved = true) {
          const uint64_t slv = f2_pack(sl2, sl2);
          float ym = -INFINITY;
#pragma unroll
          for (int n = 0; n < kN; n += 2) {
            f2_unpack(f2_fma(f2_pack(__uint_as_float(x[n]), __uint_as_float(x[n + 1])), slv, f2_pack(neg[n], neg[n + 1])), y[n], y[n + 1]);
            if (masked) {
              y[n] = (vis >> n) & 1u ? y[n] : -INFINITY;
              y[n + 1] = (vis >> (n + 1)) & 1u ? y[n + 1] : -INFINITY;
            }
            ym = fmax3(ym, y[n], y[n + 1]);
          }
          if (moved) {
            // (a NaN stays; +inf, of products beyond fp32, becomes one)
#pragma unroll
            for (int n = 0; n < kN; ++n) y[n] = y[n] > kFar ? (y[n] < INFINITY ? kFar : NAN) : y[n];
            break;
          }
          if (!group_any(bar, ym > kFar || !ok)) break;
          // the group's maxima of all rows
          float v[kN];
#pragma unroll
          for (int n = 0; n < kN; ++n) v[n] = (vis >> n) & 1u ? __uint_as_float(x[n]) : -INFINITY;
          const float mine = __fmul_rd(reduce16<true>(v, lane), sl2);
          if ((lane & 1) == 0) c.top[g][q4][lane >> 1] = mine;
          if (ok && k > 1) ok = warp_wait(&c.pv_done[g], (sn - 1) & 1, abort_flag);
          if (group_any(bar, !ok)) { leave = true; break; }       // and the maxima are there
          tc::tc_fence_after();
          float f[kN];
#pragma unroll
          for (int n = 0; n < kN; n += 4) {
            float t[4];
            *reinterpret_cast<float4*>(t) = *reinterpret_cast<const float4*>(&c.top[g][0][n]);
#pragma unroll
            for (int w = 1; w < 4; ++w) {
              const float4 u = *reinterpret_cast<const float4*>(&c.top[g][w][n]);
              t[0] = fmaxf(t[0], u.x); t[1] = fmaxf(t[1], u.y); t[2] = fmaxf(t[2], u.z); t[3] = fmaxf(t[3], u.w);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              // (not a row: neg = -inf, nothing is above +inf; no reference yet: 2^-inf = 0 of a sum of 0)
              const bool up = t[i] > -neg[n + i];
              f[n + i] = up && neg[n + i] != INFINITY ? ex2(-neg[n + i] - t[i]) : 1.f;
              neg[n + i] = up ? -t[i] : neg[n + i];
              sum[n + i] *= f[n + i];
            }
          }
          if (k > 1) {
#pragma unroll 1
            for (int piece = 0; piece < 2; ++piece) {
              uint32_t o[kN];
              const uint32_t to = tmem + lane_addr + kTmemO + 32 * (2 * par + g) + kN * piece;
              tc::tmem_ld16(to, o);
              tc::tmem_ld_wait();
#pragma unroll
              for (int n = 0; n < kN; ++n) o[n] = __float_as_uint(__uint_as_float(o[n]) * f[n]);
              tc::tmem_st16(to, o);
            }
            tc::tmem_st_wait();
          }
        }
        if (leave) break;
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
        if (ok && masked) {
          // V's rows, 32 a warp, eight lanes a row; by now V has mostly come.  S of this tile was issued after the
          // product that read the older tile in V's stage.
          const int gv = kt0 + k, st = gv % kVStages;
          ok = warp_wait(&c.v_full[st], (gv / kVStages) & 1, abort_flag);
          if (ok) {
            uint8_t* tile = sV + st * kTile + (q4 * 32 + (lane >> 3)) * 128 + (lane & 7) * 16;
            const int key0 = kb + q4 * 32 + (lane >> 3), end = r.it.end, sink = r.it.sink, lo = r.it.lo;
            uint32_t word = 0;
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
                  }
                  const uint32_t lanes = __ballot_sync(0xffffffffu, hit);
                  for (int e = 0; e < 4; ++e) word |= ((lanes >> (8 * e)) & 0xffu) ? 1u << (4 * i + e) : 0u;
                }
              }
            }
            // a key whose V is not finite: NaN for the rows that see it (a warp's lanes have the keys it looked at)
            if ((word >> lane) & 1u) {
#pragma unroll 1
              for (int n = 0; n < nrows; ++n)
                if ((vis >> n) & 1u) *reinterpret_cast<uint16_t*>(prow + (((n >> 3) ^ sw) << 4) + (n & 7) * 2) = 0x7fff;
            }
          }
        }
        tc::fence_proxy_async_smem();
        tc::tc_fence_before();
        __syncwarp();
        // (after a wait that ran out nothing reads P any more: the next vote ends the group)
        if (lane == 0) tc::mbar_arrive(&c.p_full[g]);
      }
      if (leave) { ok = false; break; }
      // the unit's sums; the output warps have to have read the ones before of this parity
      const float total = reduce16<false>(sum, lane);
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
      give_back();
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
    w.start(R, nullptr);
    Item it;
    while (w.next(a, R, it)) flag(a, it.req, 1, SPEC_REQ_TIMEOUT);
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
