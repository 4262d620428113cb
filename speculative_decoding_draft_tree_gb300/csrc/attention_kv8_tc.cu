// spec_tree_attention_kv8 on the tcgen05 tensor cores: bf16 queries, head_dim 128.
//
// attn_kv8_rows_kernel: units of at most 8 or 16 query rows (T x G: single tokens and short chains).
// S^T = K Q^T (M = 128 slots on the TMEM lanes, N = the rows' hi pieces, then their lo pieces), so
// that the softmax spends its lanes on keys; O^T += V^T P^T with V read as an MN-major operand and
// P^T's three pieces stacked the same way, each with columns of O of its own.  Bound by the codes'
// bytes: a tile's 32 KB take ~1400 clocks of an SM's share of HBM and the products a quarter of that,
// so what has to keep up is the softmax, whose step is a chain of latencies (wait, TMEM load, group
// vote, exponentials, stores).
// Two groups of four warps take alternate tiles, each with references, sums and an accumulator of
// its own, and a third warpgroup joins the two and writes a unit's rows while they go on with the
// next one (accumulators are double-buffered by unit).
// Warps: 0 copies K, 2 copies V, 1 issues the scores' products, 3 the output's, 4-7 and 8-11
// softmax, 12-15 split the queries and write the output, 16 brings the scales, 17 walks the items.
// Measured: 64 single tokens over 1024 .. 32768 slots (2.2 GB) 341 - 352 us, 6.4 TB/s, 93 - 96% of the
// copy rate; 16 chains of 6, 32 KV heads, 2048 slots (271 MB) 54 us, 5.0 TB/s; one token over 2047
// slots (4 MB) 11.0 us, all of it latency: the start, the walk to the first page, a tile, the join.
//
// attn_kv8_tile_kernel: longer units in tiles of 128 query rows (G heads x 128 / G tree tokens).
// S = Q K^T (M = N = 128, both pieces of Q into one accumulator) on the e4m3 codes; O += P V in fp16:
// four warps convert V's codes, which are fp16 values, in shared memory, ahead of the product, and P goes
// to TMEM as the A operand with one conversion a pair of weights.  Each product runs 512 clocks a tile,
// as two 8-bit pieces of P against the codes would, and P keeps fp16's 11 bits down to 2^-19 of a row's
// largest weight.  (e5m2 and e4m3 pieces kept three bits below 2^-13: a long flat rest beside one heavy
// key came out by up to an eighth wrong.  Three e5m2 pieces, right as well, took 367 and 1760 us on the
// two shapes below.)  A tile takes ~2600 clocks: the exponentials are 512 of them at 32 results a clock
// and SM, the conversion of V ~200, the products 1024, and no pipe is full; a step is a chain of waits,
// TMEM loads, votes and stores, which all warps take together, tile after tile.
// A row belongs to four threads of four warps, each with 32 of a tile's keys: they form weights against
// the present reference at once and vote on it meanwhile; where the vote says that it moves, they agree
// on the new one and form them again; ten binades of slack make that rare.  Three S buffers (TMEM columns
// 0-383, P over S) keep the scores of the next tiles coming while one is in the softmax and one in the
// output's product; O has columns 384-511.
// Warps: 0-3 as above, 4-19 softmax, 20-23 queries and output, 24 scales, 25 items, 28-31 V.
// Measured: 32 trees of 46 over 8192 slots (32 query heads on 8) 301 us, 656 TFLOP/s of scores and
// output; 64 ragged trees over 1024 .. 32768 slots (64 query heads on 8) 1465 us, 838 TFLOP/s.
// The bf16 cache takes 289 and 1554 us on these shapes.
//
// Scales: a score x is code product * (K scale of the slot's page * the row's query scale).  The
// reference is the largest y = x + log2(V scale), and the weight that goes into the product with V's
// codes is 2^(y - ref), which fills its format's range whatever the pages' scales are.  The row sum
// takes 2^(x - ref): in the rows kernel that is what the exponential forms, and the V scale is multiplied
// in; in the tile kernel, where that multiplication costs 4% (308 us against 296, 1530 against 1450),
// the exponential forms 2^(y - ref) and the sum divides by the scale again, which loses keys whose
// 2^(y - ref) is below 2^-126.
//
// The waits are bounded; one that runs out raises the CTA's abort flag, after which no wait
// blocks: the softmax groups, which meet at hardware barriers, still walk through their tiles, the
// other roles leave, and the range's requests get SPEC_REQ_TIMEOUT.
#include <math.h>

#include <mutex>

#include "attention_kv8_tc.cuh"

namespace spec {
namespace kv8tc {

namespace rows {
constexpr int kThreads = 640;
constexpr int kCtlRegs = 72;      // registers a thread (setmaxnreg): warps 0-3 and 16-19
constexpr int kSoftmaxRegs = 120; // warps 4-11
constexpr int kOutRegs = 96;      // warps 12-15, as launched
static_assert(128 * (2 * kCtlRegs + 2 * kSoftmaxRegs + kOutRegs) <= kThreads * 96, "register split");
constexpr int kKStages = 6;
constexpr int kVStages = 5;

template <int NR>
struct Layout {
  static constexpr int kPiece = NR * 128;                // bytes of one piece of the rows
  static constexpr int kPair = 2 * kPiece;               // Q: hi, then lo
  // P: hi, mid, lo, and with 8 rows a piece that is never written (the products take columns by 16;
  // what comes of it is not read)
  static constexpr int kPieces = NR == 8 ? 4 : 3;
  static constexpr int kTriple = kPieces * kPiece;
  static constexpr int kSmemQ = 0;                       // 2 buffers
  static constexpr int kSmemP = kSmemQ + 2 * kPair;      // 2 groups x 2 buffers
  static constexpr int kSmemK = kSmemP + 4 * kTriple;
  static constexpr int kSmemV = kSmemK + kKStages * kTile;
  static constexpr int kSmemBar = kSmemV + kVStages * kTile;
  static constexpr uint32_t kN = 2 * NR;                 // columns of a product of scores
  static constexpr uint32_t kNO = kPieces * NR;          // of the output
  static constexpr uint32_t kTmemO = 4 * kN;             // S: group, buffer; O: group, unit parity
  static constexpr uint32_t kOStride = NR == 8 ? 32 : 64;
  static constexpr uint32_t kTmemCols = NR == 8 ? 256 : 512;
  static_assert(kTmemO + 4 * kOStride <= kTmemCols && kNO <= kOStride && kNO % 16 == 0, "TMEM");
  static_assert(kSmemK % 1024 == 0, "swizzled tiles on 1024-byte bounds");
};

template <int NR>
struct Shared {
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[kKStages], k_empty[kKStages], v_full[kVStages], v_empty[kVStages];
  uint64_t s_full[2][2], s_free[2][2], p_full[2][2], pv_done[2][2];
  uint64_t sum_full[2], o_full[2], o_free[2];      // by unit parity
  uint64_t sc_full[kScaleRing], sc_empty[kScaleRing], drain[2];
  ScaleSlot sc[kScaleRing];
  alignas(16) float qmul[2][NR];
  float mx[2][4][NR];             // per group and warp: row maxima of an update
  float sum[2][2][4][NR];         // per unit parity, group and warp: row sums
  float add[2][2][NR];            // per unit parity and group: kShift - reference
  uint32_t tmem;
  int abort, r0, r1;              // r0 .. r1: the requests of the range
  ItemRing items;
};
template <int NR>
constexpr int smem_bytes() {
  return Layout<NR>::kSmemBar + int(sizeof(Shared<NR>)) + 1024;
}
static_assert(smem_bytes<16>() <= 232448, "fits one CTA's shared memory");
}  // namespace rows

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[N]) {
  if constexpr (N == 8) tmem_ld8(addr, r);
  else if constexpr (N == 16) tc::tmem_ld16(addr, r);
  else tc::tmem_ld32(addr, r);
}
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t addr, const uint32_t (&r)[N]) {
  if constexpr (N == 8) tmem_st8(addr, r);
  else tc::tmem_st16(addr, r);
}

// A V row of a tile in shared memory; a warp's lanes hold neighbouring rows and start at different
// vectors of them, in different banks.  (The stores are not unrolled: masked tiles are few.)
__device__ __forceinline__ void clear_row(uint8_t* row) {
  uint4* w = reinterpret_cast<uint4*>(row);
#pragma unroll 1
  for (int x = 0; x < 8; ++x) w[(x + threadIdx.x) & 7] = make_uint4(0, 0, 0, 0);
}
__device__ __forceinline__ bool has_nan(const uint8_t* row) {
  const uint4* w = reinterpret_cast<const uint4*>(row);
  uint32_t hit = 0;
#pragma unroll
  for (int x = 0; x < 8; ++x) {
    const uint4 v = w[(x + threadIdx.x) & 7];
    hit |= nan_bytes(v.x) | nan_bytes(v.y) | nan_bytes(v.z) | nan_bytes(v.w);
  }
  return hit != 0;
}
__device__ __forceinline__ void clear_nan(uint8_t* row) {
  uint32_t* w = reinterpret_cast<uint32_t*>(row);
#pragma unroll 1
  for (int x = 0; x < 32; ++x) w[x] &= ~((nan_bytes(w[x]) >> 7) * 255u);
}

template <int NR>
__global__ void __launch_bounds__(rows::kThreads, 1)
attn_kv8_rows_kernel(const __grid_constant__ CUtensorMap mK, const __grid_constant__ CUtensorMap mV,
                     const __grid_constant__ CUtensorMap mKw,
                     const __grid_constant__ CUtensorMap mVw, TcDev d) {
  using namespace rows;
  using L = Layout<NR>;
  constexpr int kN = int(L::kN);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* sQ = base + L::kSmemQ;
  uint8_t* sP = base + L::kSmemP;
  uint8_t* sK = base + L::kSmemK;
  uint8_t* sV = base + L::kSmemV;
  Shared<NR>& sh = *reinterpret_cast<Shared<NR>*>(base + L::kSmemBar);
  const AttnKv8Dev& a = d.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // what needs no input comes before the wait for the kernel before
  if (warp == 0) {
    tc::tmem_alloc(&sh.tmem, L::kTmemCols);
    tc::tmem_relinquish();
    if (lane == 0) {
      tc::prefetch_tensormap(&mK);
      tc::prefetch_tensormap(&mKw);
      tc::prefetch_tensormap(&mV);
      tc::prefetch_tensormap(&mVw);
    }
  } else if (warp == 1) {
    auto init = [&](uint64_t* bar, int n, int count) {
      if (lane < n) tc::mbar_init(bar + lane, count);
    };
    init(sh.q_full, 2, 4);                   // the output warps
    init(sh.q_empty, 2, 9);                  // the issuer's commit and the 8 softmax warps
    init(sh.k_full, kKStages, 1);
    init(sh.k_empty, kKStages, 1);
    init(sh.v_full, kVStages, 1);
    init(sh.v_empty, kVStages, 1);
    init(&sh.s_full[0][0], 4, 1);
    init(&sh.s_free[0][0], 4, 4);
    init(&sh.p_full[0][0], 4, 4);
    init(&sh.pv_done[0][0], 4, 1);
    init(sh.sum_full, 2, 8);
    init(sh.o_full, 2, 1);
    init(sh.o_free, 2, 4);
    init(sh.sc_full, kScaleRing, 1);
    init(sh.sc_empty, kScaleRing, 4);
    init(sh.drain, 2, 1);
    init(sh.items.full, kItemRing, 1);
    init(sh.items.empty, kItemRing, 17);     // warps 0-16
    if (lane == 0) sh.abort = 0;
    tc::fence_mbar_init();
  }
  tc::tc_fence_before();
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  tc::tc_fence_after();
  const uint32_t tmem = sh.tmem;
  volatile int* abort_flag = &sh.abort;

  if (warp < 4 || warp >= 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCtlRegs));
    if (warp == 0 || warp == 2) {
      const bool k = warp == 0;
      page_producer(d, sh.items, k ? &mK : &mV, k ? &mKw : &mVw, k ? kKStages : kVStages,
                    k ? sK : sV, k ? sh.k_full : sh.v_full, k ? sh.k_empty : sh.v_empty, k,
                    &sh.abort);
    } else if (warp == 16) {
      scale_producer(d, sh.items, sh.sc, sh.sc_full, sh.sc_empty, &sh.abort);
    } else if (warp == 17) {
      const Range R = warp_range(d);
      if (lane == 0) {
        sh.r0 = R.r0;
        sh.r1 = R.t0 < R.t1 ? R.r1 : -1;
        item_producer(d, R, sh.items, abort_flag);
        write_merge_record(d, R);
      }
      __syncwarp();
    } else if (warp == 1 || warp == 3) {
      // =================================================================== MMA issuers
      // the whole warp walks the tiles, so that addresses and descriptors are uniform values; one
      // elected lane issues
      const bool is_qk = warp == 1;
      const uint32_t id_qk = idesc_e4m3(128, kN, false, false);
      const uint32_t id_pv = idesc_e4m3(128, int(L::kNO), true, false) | kIdescBE5m2;
      const uint64_t dQ = tc::smem_desc(tc::smem_u32(sQ), 16, 1024);
      const uint64_t dP = tc::smem_desc(tc::smem_u32(sP), 16, 1024);
      const uint64_t dK = tc::smem_desc(tc::smem_u32(sK), 16, 1024);
      const uint64_t dV = tc::smem_desc(tc::smem_u32(sV), kTile, 1024);
      int kt = 0;                      // tiles so far; group = parity of the tile's number
      bool ok = true;
      Item it;
#pragma unroll 1
      for (int li = 0; ok && __all_sync(0xffffffffu, next_item(sh.items, li, it, abort_flag)); ++li) {
        const int par = li & 1;
        if (is_qk) ok = wait1(&sh.q_full[par], li >> 1, abort_flag);
        else if (li > 1) ok = wait1(&sh.o_free[par], (li >> 1) - 1, abort_flag);
#pragma unroll 1
        for (int j = it.j0; j < it.j1; ++j, ++kt) {
          const int g = kt & 1, b = (kt >> 1) & 1, use = kt >> 2;
          if (is_qk) {
            const int st = kt % kKStages;
            ok = ok && wait1(&sh.k_full[st], kt / kKStages, abort_flag) &&
                 (use == 0 || wait1(&sh.s_free[g][b], use - 1, abort_flag));
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc::tc_fence_after();
            const uint32_t tS = tmem + (g * 2 + b) * kN;
            const uint64_t ka = dK + uint64_t(st) * (kTile >> 4);
            const uint64_t qb = dQ + uint64_t(par) * (L::kPair >> 4);
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_e4m3_ss(tS, ka + 2 * k, qb + 2 * k, id_qk, k > 0 ? 1u : 0u);
              tc::mma_commit(&sh.s_full[g][b]);
              tc::mma_commit(&sh.k_empty[st]);
              if (j == it.j1 - 1) tc::mma_commit(&sh.q_empty[par]);
            }
            __syncwarp();
          } else {
            const int st = kt % kVStages;
            const bool first = j - it.j0 < 2;     // the group's first tile of the unit
            ok = ok && wait1(&sh.p_full[g][b], use, abort_flag) &&
                 wait1(&sh.v_full[st], kt / kVStages, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc::tc_fence_after();
            const uint32_t tO = tmem + L::kTmemO + (g * 2 + par) * L::kOStride;
            const uint64_t va = dV + uint64_t(st) * (kTile >> 4);
            const uint64_t pb = dP + uint64_t(g * 2 + b) * (L::kTriple >> 4);
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < 4; ++k)            // 32 slots a step: four groups of 8 V rows
                mma_e4m3_ss(tO, va + k * (4096 >> 4), pb + 2 * k, id_pv,
                            (k > 0 || !first) ? 1u : 0u);
              tc::mma_commit(&sh.v_empty[st]);
              tc::mma_commit(&sh.pv_done[g][b]);
              if (j == it.j1 - 1) tc::mma_commit(&sh.o_full[par]);
            }
            __syncwarp();
          }
        }
      }
      if (!ok) *abort_flag = 1;
      // nothing issued here may still run when TMEM is released (bounded, abort or not)
      if (elect_one()) tc::mma_commit(&sh.drain[is_qk ? 0 : 1]);
      __syncwarp();
      volatile int never = 0;
      tc::mbar_wait(&sh.drain[is_qk ? 0 : 1], 0, &never, kWaitLimit / 8);
      __syncwarp();
    }
  } else if (warp < 12) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ===================================================================== softmax
    const int grp = (warp - 4) >> 2, q = warp & 3;   // group; TMEM lane quarter
    const uint32_t lane_addr = uint32_t(q * 32) << 16;
    const int kl = q * 32 + lane;                    // this lane's slot of a tile
    const int si = kl >> d.log2bs;
    const int bar_g = 1 + grp;
    // With 16 rows P^T is stored two keys at a time: of each pair of rows a lane takes one, the even lane
    // the even row, for its key and its neighbour's (units of 16 rows over 8192 slots 67 us, 71 with
    // bytes; with 8 rows the exchange costs more than the stores, 54.9 against 54.0 us on the chains)
    const int odd = NR == 16 ? lane & 1 : 0, chunk = kl >> 4;
    uint8_t* const pcol = sP + grp * 2 * L::kTriple + odd * 128 + (kl & (NR == 16 ? 14 : 15));
    const uint32_t own_other = odd ? 0x3715u : 0x6240u;
    int kt = 0;
    bool ok = true;                                  // no early exit: see the file's comment
    Item it;
#pragma unroll 1
    for (int li = 0;; ++li) {
      // the group leaves together: an expired wait in one warp must not leave the others at a
      // barrier
      if (bar_any(bar_g, 128, !next_item(sh.items, li, it, abort_flag))) break;
      const int par = li & 1;
      const int T = it.T, P = it.P, kv_len = P + T;
      const int nt = it.j1 - it.j0;
      const uint32_t tO = tmem + lane_addr + L::kTmemO + (grp * 2 + par) * L::kOStride;
      const float4* qmul = reinterpret_cast<const float4*>(sh.qmul[par]);
      ok &= wait1(&sh.q_full[par], li >> 1, abort_flag);
      float add[NR], lsum[NR];
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        add[n] = INFINITY;
        lsum[n] = 0.f;
      }
      bool fresh = true;                             // nothing accumulated in this unit yet
#pragma unroll 1
      for (int i = (kt ^ grp) & 1; i < nt; i += 2, fresh = false) {
        const int kg = kt + i;                       // the tile's number in the CTA's stream
        const int b = (kg >> 1) & 1, use = kg >> 2;
        const int slot = kg % kScaleRing;
        ok &= wait1(&sh.sc_full[slot], kg / kScaleRing, abort_flag);
        const float ks = sh.sc[slot].k[si], lv = sh.sc[slot].lv[si], vs = sh.sc[slot].v[si];
        ok &= wait1(&sh.s_full[grp][b], use, abort_flag);
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sh.sc_empty[slot]);
        tc::tc_fence_after();
        uint32_t sv[kN];
        tmem_ld<kN>(tmem + lane_addr + (grp * 2 + b) * kN, sv);
        tc::tmem_ld_wait();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sh.s_free[grp][b]);
        const int key = (it.j0 + i) * kBN + kl;
        // scores in the exponent's units; rows that pad the unit have zero queries and are
        // carried along, so a tile inside the prefix needs no mask
        const bool masked = (it.j0 + i) * kBN + kBN > P;
        uint32_t vis = 0xFFFFFFFFu;
        if (masked && key >= P) {
          vis = 0;
          if (key < kv_len) {
            const uint32_t* anc = a.anc + size_t(it.o) * a.W + ((key - P) >> 5);
            const int sh_ = (key - P) & 31;
            uint32_t w[NR];
#pragma unroll
            for (int t = 0; t < NR; ++t) w[t] = t < T ? __ldg(anc + t * a.W) : 0u;
#pragma unroll
            for (int t = 0; t < NR; ++t)
              if ((w[t] >> sh_) & 1u) vis |= ((1u << a.G) - 1u) << (t * a.G);
          }
        }
        float x[NR], zmax = -INFINITY;
#pragma unroll
        for (int n4 = 0; n4 < NR / 4; ++n4) {
          const float4 qm = qmul[n4];
          const float m4[4] = {ks * qm.x, ks * qm.y, ks * qm.z, ks * qm.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int n = n4 * 4 + e;
            x[n] = (__uint_as_float(sv[n]) + __uint_as_float(sv[n + NR])) * m4[e];
          }
        }
        if (masked) {
#pragma unroll
          for (int n = 0; n < NR; ++n) x[n] = ((vis >> n) & 1u) ? x[n] : -INFINITY;
        }
        // against the references (none yet: +infinity, or NaN under a masked key)
#pragma unroll
        for (int n = 0; n < NR; ++n) zmax = fmaxf(zmax, x[n] + add[n]);
        if (bar_any(bar_g, 128, zmax + lv > kCeil)) {
          // some row's reference moves up to its maximum so far
          float y[NR];
#pragma unroll
          for (int n = 0; n < NR; ++n) y[n] = x[n] + lv;
          const float top = red_rows<NR, true>(y, lane);
          sh.mx[grp][q][red_row<NR>(lane)] = top;
          bar_sync(bar_g, 128);
          float factor[NR];
#pragma unroll
          for (int n = 0; n < NR; ++n) {
            const float ref = fmaxf(fmaxf(fmaxf(sh.mx[grp][0][n], sh.mx[grp][1][n]),
                                          fmaxf(sh.mx[grp][2][n], sh.mx[grp][3][n])),
                                    kShift - add[n]);
            const float now = kShift - ref;
            // (in two halves: pages of zeros before any other leave a sum that is far above the rest)
            const float half = add[n] == INFINITY ? 1.f : ex2(0.5f * (now - add[n]));
            factor[n] = half * half;
            add[n] = now;
            lsum[n] = lsum[n] * half * half;
          }
          if (!fresh) {                              // the group's accumulator holds something
            const int kp = kg - 2;                   // the group's tile before
            ok &= wait1(&sh.pv_done[grp][(kp >> 1) & 1], kp >> 2, abort_flag);
            __syncwarp();
            tc::tc_fence_after();
#pragma unroll
            for (int piece = 0; piece < 3; ++piece) {
              uint32_t ov[NR];
              tmem_ld<NR>(tO + piece * NR, ov);
              tc::tmem_ld_wait();
#pragma unroll
              for (int n = 0; n < NR; ++n)
                ov[n] = __float_as_uint(__uint_as_float(ov[n]) * factor[n]);
              tmem_st<NR>(tO + piece * NR, ov);
            }
            tc::tmem_st_wait();
          }
        }
        // weights: this slot's column of P^T, after the product that last read the buffer
        if (use > 0) ok &= wait1(&sh.pv_done[grp][b], use - 1, abort_flag);
        uint8_t* pc = pcol + b * L::kTriple;
#pragma unroll
        for (int n = 0; n < NR; n += 4) {
          float p[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            // (a row that has seen nothing: -infinity + infinity)
            const float e = x[n + u] == -INFINITY ? 0.f : ex2(x[n + u] + add[n + u]);
            lsum[n + u] = fmaf(e, kSumMul, lsum[n + u]);
            p[u] = e * vs;
          }
          const Split2 s0 = split_p2(p[0], p[1]), s1 = split_p2(p[2], p[3]);
          auto at = [&](int n) { return (n >> 3) * 1024 + (n & 7) * 128 + ((chunk ^ odd ^ (n & 7)) << 4); };
          if constexpr (NR == 16) {
            auto pairs = [&](uint32_t w) {           // bytes of rows (0, 1), (0, 1) or (2, 3)
              return __byte_perm(w, __shfl_xor_sync(0xffffffffu, w, 1), own_other);
            };
            auto put = [&](int o, uint32_t w) { *reinterpret_cast<uint16_t*>(pc + o) = uint16_t(w); };
            const uint32_t a0 = pairs(__byte_perm(s0.hi, s0.mid, 0x7531));
            const uint32_t a1 = pairs(__byte_perm(s1.hi, s1.mid, 0x7531));
            const uint32_t lo = pairs(__byte_perm(s0.lo, s1.lo, 0x7531));
            put(at(n), a0);
            put(at(n + 2), a1);
            put(L::kPiece + at(n), a0 >> 16);
            put(L::kPiece + at(n + 2), a1 >> 16);
            put(2 * L::kPiece + at(n), lo);
            put(2 * L::kPiece + at(n + 2), lo >> 16);
          } else {
            auto put = [&](int n, const Split2& s) {
              pc[at(n)] = uint8_t(s.hi >> 8);
              pc[at(n + 1)] = uint8_t(s.hi >> 24);
              pc[L::kPiece + at(n)] = uint8_t(s.mid >> 8);
              pc[L::kPiece + at(n + 1)] = uint8_t(s.mid >> 24);
              pc[2 * L::kPiece + at(n)] = uint8_t(s.lo >> 8);
              pc[2 * L::kPiece + at(n + 1)] = uint8_t(s.lo >> 24);
            };
            put(n, s0);
            put(n + 2, s1);
          }
        }
        // where keys are masked a NaN code of V times a zero weight must stay zero: stale rows past
        // the end are cleared, and a tree slot's NaN moves from V to the weights of the rows that
        // see it
        if (masked) {
          const int st = kg % kVStages;
          ok &= wait1(&sh.v_full[st], kg / kVStages, abort_flag);
          uint8_t* row = sV + st * kTile + kl * 128;
          uint32_t seen = 0u;                          // the rows that get a NaN
          if (key >= kv_len) {
            clear_row(row);
          } else if (key >= P && (~vis & ((1u << (T * a.G)) - 1u)) != 0 && has_nan(row)) {
            clear_nan(row);                            // (T G <= 16; some row does not see it)
            seen = vis;
          }
          if constexpr (NR == 16) __syncwarp();        // (the neighbour has stored this lane's weights)
          uint8_t* const own = sP + (grp * 2 + b) * L::kTriple + (kl & 15);
#pragma unroll 1
          for (int n = 0; seen >> n; ++n)
            if ((seen >> n) & 1u) own[(n >> 3) * 1024 + (n & 7) * 128 + ((chunk ^ (n & 7)) << 4)] = 0x7F;
        }
        tc::fence_proxy_async_smem();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sh.p_full[grp][b]);
      }
      // the unit's sums and references for the output warps
      const float total = red_rows<NR, false>(lsum, lane);
      if (li > 1) ok &= wait1(&sh.o_free[par], (li >> 1) - 1, abort_flag);
      sh.sum[par][grp][q][red_row<NR>(lane)] = total;
      if (q == 0 && lane == 0) {
#pragma unroll
        for (int n = 0; n < NR; ++n) sh.add[par][grp][n] = add[n];
      }
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(&sh.q_empty[par]);
        tc::mbar_arrive(&sh.sum_full[par]);
      }
      kt += nt;
    }
    if (!ok) *abort_flag = 1;
  } else {
    // ===================================================================== queries, output
    // Queries two units ahead, then the output of the unit that is done.
    const int q = warp & 3;
    const uint32_t lane_addr = uint32_t(q * 32) << 16;
    const int col = q * 32 + lane;
    bool ok = true;
    struct Unit {
      int o, T, h, slot;
    };
    auto fetch = [&](int li, Unit& u) -> bool {
      Item it;
      const bool has = __all_sync(0xffffffffu, next_item(sh.items, li, it, abort_flag));
      u.o = it.o;
      u.T = it.T;
      u.h = it.h;
      u.slot = it.slot;
      return has;
    };
    // a row to each half warp, 16 bytes a lane; the row's scale brings its largest element into
    // (224, 448]
    auto put_q = [&](int li, const Unit& u) {
      const int b = li & 1, c = lane & 15;
      uint8_t* p = sQ + b * L::kPair;
      if (li > 1) ok &= wait1(&sh.q_empty[b], (li >> 1) - 1, abort_flag);
#pragma unroll 1
      for (int n = q * 2 + (lane >> 4); n < NR; n += 8) {
        const int t = n / a.G, g = n - t * a.G;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (t < u.T)
          w = __ldg(reinterpret_cast<const uint4*>(
                        static_cast<const __nv_bfloat16*>(a.q) +
                        (size_t(u.o + t) * a.H_q + u.h * a.G + g) * kD) + c);
        float f[8], m = 0.f;
        elem<__nv_bfloat16>::unpack(w, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fabsf(f[e]) <= FLT_MAX ? fmaxf(m, fabsf(f[e])) : m;
#pragma unroll
        for (int s = 8; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
        const float sq = kv8::need_scale(m);
        uint2 hi, lo;
        split_q8(w, __uint_as_float((254u << 23) - __float_as_uint(sq)), hi, lo);
        const int off = (n >> 3) * 1024 + (n & 7) * 128 + (((c >> 1) ^ (n & 7)) << 4) + (c & 1) * 8;
        *reinterpret_cast<uint2*>(p + off) = hi;
        *reinterpret_cast<uint2*>(p + L::kPiece + off) = lo;
        if (c == 0) sh.qmul[b][n] = sq * a.scale_log2;
      }
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sh.q_full[b]);
    };
    Unit cur, next, after;
    bool has = fetch(0, cur), has_next = false;
    if (has) {
      put_q(0, cur);
      has_next = fetch(1, next);
      if (has_next) put_q(1, next);
    }
#pragma unroll 1
    for (int li = 0; has; ++li) {
      const bool has_after = has_next && fetch(li + 2, after);
      const int par = li & 1;
      const int nrows = cur.T * a.G;                 // <= NR
      ok &= wait1(&sh.sum_full[par], li >> 1, abort_flag);
      // lane n: row n's place, the weights of the two groups' accumulators, its log-sum-exp
      const int rn = lane < NR ? lane : 0, rt = rn / a.G;
      const int row = cur.slot < 0 ? (cur.o + rt) * a.H_q + cur.h * a.G + (rn - rt * a.G)
                                   : cur.slot * d.part_rows + rn;
      const float a0 = sh.add[par][0][rn], a1 = sh.add[par][1][rn];
      const float top = fminf(a0, a1);               // of the larger reference
      float w0 = a0 == INFINITY ? 0.f : ex2(0.5f * (top - a0));   // (their roots first, as above)
      float w1 = a1 == INFINITY ? 0.f : ex2(0.5f * (top - a1));
      float l0 = 0.f, l1 = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        l0 += sh.sum[par][0][w][rn];
        l1 += sh.sum[par][1][w][rn];
      }
      const float l = l0 * w0 * w0 + l1 * w1 * w1;
      const float inv = l == 0.f ? 0.f : kSumMul / l;    // (NaN stays NaN)
      const float lse2 = l == 0.f ? -INFINITY : log2f(l) + kSumShift - top;
      w0 *= w0 * inv;
      w1 *= w1 * inv;
      ok &= wait1(&sh.o_full[par], li >> 1, abort_flag);
      __syncwarp();
      tc::tc_fence_after();
      // (an accumulator that took no product in this unit has weight 0 and stale columns)
      uint32_t ov[3][NR];
      float v[NR];
      auto load_o = [&](int grp) {
#pragma unroll
        for (int piece = 0; piece < 3; ++piece)
          tmem_ld<NR>(tmem + lane_addr + L::kTmemO + (grp * 2 + par) * L::kOStride + piece * NR, ov[piece]);
        tc::tmem_ld_wait();
      };
      auto sum_o = [&](int n) {
        return (__uint_as_float(ov[2][n]) + __uint_as_float(ov[1][n])) + __uint_as_float(ov[0][n]);
      };
      load_o(0);
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        const float u = __shfl_sync(0xffffffffu, w0, n);
        v[n] = u != 0.f ? sum_o(n) * u : 0.f;
      }
      load_o(1);
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sh.o_free[par]);
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        const float u = __shfl_sync(0xffffffffu, w1, n);
        if (u != 0.f) v[n] = fmaf(sum_o(n), u, v[n]);
        const size_t at = size_t(__shfl_sync(0xffffffffu, row, n)) * kD + col;
        if (n < nrows) {
          if (cur.slot < 0) static_cast<__nv_bfloat16*>(a.o)[at] = __float2bfloat16_rn(v[n]);
          else d.part_o[at] = v[n];
        }
      }
      if (q == 0 && lane < nrows) {
        if (cur.slot >= 0) d.part_lse[row] = lse2;
        else if (a.lse) a.lse[row] = lse2 * 0.6931471805599453f;
      }
      if (has_after) put_q(li + 2, after);
      cur = next;
      next = after;
      has = has_next;
      has_next = has_after;
    }
    if (!ok) *abort_flag = 1;
  }
  tc::tc_fence_before();
  __syncthreads();
  if (*abort_flag)                           // every request of the range is unreliable
#pragma unroll 1
    for (int r = sh.r0 + tid; r <= sh.r1; r += kThreads) atomicOr(&a.req_status[r], SPEC_REQ_TIMEOUT);
  tc::tc_fence_after();
  if (warp == 0) tc::tmem_dealloc(tmem, L::kTmemCols);
}

// ------------------------------------------------------------------------------ long units
namespace tile {
constexpr int kRows = 128;
constexpr int kThreads = 1024;
// (40 / 80 / 56 registers: 32 trees of 46 over 8192 slots 296 us, over 2048 slots 122, ragged trees over
// 1024 .. 2048 slots 164; this split: 302, 119, 157; no split 328, 125, 161)
constexpr int kCtlRegs = 48;       // warps 0-3 and 24-27
constexpr int kSoftmaxRegs = 72;   // warps 4-19
constexpr int kOutRegs = 64;       // warps 20-23 and 28-31, as launched
static_assert(256 * kCtlRegs + 512 * kSoftmaxRegs + 256 * kOutRegs <= kThreads * 64, "register split");
// Weights are 2^(y - ref + kLift), in fp16; the reference moves when one passes 2^kTop.  11 bits are
// kept down to 2^-19 of a row's largest weight, and 2^-30 of it below.  (32 trees of 46, 64 ragged ones: lift
// 3 297 and 1443 us, 5 302 and 1448, 7 307 and 1495, 9 315 and 1520.)
constexpr float kLift = 5.f, kTop = 15.f;
constexpr int kKStages = 3;
constexpr int kVStages = 2;
constexpr int kPair = 2 * kTile;                         // Q's two pieces
constexpr int kHalves = 2 * kTile;                       // V in fp16: columns 0-63, then 64-127
constexpr int kSmemQ = 0;                                // 2 buffers
constexpr int kSmemK = kSmemQ + 2 * kPair;
constexpr int kSmemV = kSmemK + kKStages * kTile;
constexpr int kSmemW = kSmemV + kVStages * kTile;        // 2 buffers of fp16
constexpr int kSmemBar = kSmemW + 2 * kHalves;
constexpr int kBufs = 3;                                 // S, with P over it
constexpr uint32_t kTmemO = kBufs * 128;

struct Shared {
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[kKStages], k_empty[kKStages], v_full[kVStages], v_empty[kVStages];
  uint64_t w_full[2], w_empty[2];
  uint64_t s_full[kBufs], p_full[kBufs], pv_done[kBufs];
  uint64_t sum_full[2], sum_free[2], o_full, o_free;
  uint64_t sc_full[kScaleRing], sc_empty[kScaleRing], drain[2];
  ScaleSlot sc[kScaleRing];
  float qmul[2][kRows];
  float mx[4][kRows];             // per quarter of the keys: row maxima of an update
  float sum[2][4][kRows];         // per unit parity and quarter
  float add[2][kRows];            // per unit parity: kLift - reference
  uint32_t v_nan[2][4];           // per fp16 buffer of a masked tile: the slots whose V had a NaN
  uint32_t tmem;
  int abort, r0, r1;
  ItemRing items;
};
constexpr int kSmemBytes = kSmemBar + int(sizeof(Shared)) + 1024;
static_assert(kSmemBytes <= 232448, "fits one CTA's shared memory");
}  // namespace tile

// 32 ancestor bits of a row's words from tree index `pos` on (0 outside the row)
__device__ __forceinline__ uint32_t anc_window(const uint32_t* row, int W, int pos) {
  if (row == nullptr || pos <= -32 || pos >= 32 * W) return 0u;
  const int wi = pos >> 5, sh = pos & 31;                // wi >= -1
  const uint32_t lo = wi >= 0 ? __ldg(row + wi) : 0u;
  const uint32_t hi = wi + 1 < W ? __ldg(row + wi + 1) : 0u;
  return __funnelshift_r(lo, hi, sh);
}

__global__ void __launch_bounds__(tile::kThreads, 1)
attn_kv8_tile_kernel(const __grid_constant__ CUtensorMap mK, const __grid_constant__ CUtensorMap mV,
                     const __grid_constant__ CUtensorMap mKw,
                     const __grid_constant__ CUtensorMap mVw, TcDev d) {
  using namespace tile;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* sQ = base + kSmemQ;
  uint8_t* sK = base + kSmemK;
  uint8_t* sV = base + kSmemV;
  uint8_t* sW = base + kSmemW;
  Shared& sh = *reinterpret_cast<Shared*>(base + kSmemBar);
  const AttnKv8Dev& a = d.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == 0) {
    tc::tmem_alloc(&sh.tmem, 512);
    tc::tmem_relinquish();
    if (lane == 0) {
      tc::prefetch_tensormap(&mK);
      tc::prefetch_tensormap(&mKw);
      tc::prefetch_tensormap(&mV);
      tc::prefetch_tensormap(&mVw);
    }
  } else if (warp == 1) {
    auto init = [&](uint64_t* bar, int n, int count) {
      if (lane < n) tc::mbar_init(bar + lane, count);
    };
    init(sh.q_full, 2, 4);                   // the output warps
    init(sh.q_empty, 2, 17);                 // the issuer's commit and the 16 softmax warps
    init(sh.k_full, kKStages, 1);
    init(sh.k_empty, kKStages, 1);
    init(sh.v_full, kVStages, 1);
    init(sh.v_empty, kVStages, 4);           // the converting warps
    init(sh.w_full, 2, 4);
    init(sh.w_empty, 2, 1);
    init(sh.s_full, kBufs, 1);
    init(sh.p_full, kBufs, 16);
    init(sh.pv_done, kBufs, 1);
    init(sh.sum_full, 2, 16);
    init(sh.sum_free, 2, 4);
    init(&sh.o_full, 1, 1);
    init(&sh.o_free, 1, 4);
    init(sh.sc_full, kScaleRing, 1);
    init(sh.sc_empty, kScaleRing, 16);
    init(sh.drain, 2, 1);
    init(sh.items.full, kItemRing, 1);
    init(sh.items.empty, kItemRing, 29);     // warps 0-24 and 28-31
    if (lane == 0) sh.abort = 0;
    tc::fence_mbar_init();
  }
  tc::tc_fence_before();
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  tc::tc_fence_after();
  const uint32_t tmem = sh.tmem;
  volatile int* abort_flag = &sh.abort;

  if (warp < 4 || (warp >= 24 && warp < 28)) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCtlRegs));
    if (warp == 0 || warp == 2) {
      const bool k = warp == 0;
      page_producer(d, sh.items, k ? &mK : &mV, k ? &mKw : &mVw, k ? kKStages : kVStages,
                    k ? sK : sV, k ? sh.k_full : sh.v_full, k ? sh.k_empty : sh.v_empty, k,
                    &sh.abort);
    } else if (warp == 24) {
      scale_producer(d, sh.items, sh.sc, sh.sc_full, sh.sc_empty, &sh.abort);
    } else if (warp == 25) {
      const Range R = warp_range(d);
      if (lane == 0) {
        sh.r0 = R.r0;
        sh.r1 = R.t0 < R.t1 ? R.r1 : -1;
        item_producer(d, R, sh.items, abort_flag);
        write_merge_record(d, R);
      }
      __syncwarp();
    } else if (warp == 1 || warp == 3) {
      // =================================================================== MMA issuers
      // the whole warp walks the tiles, so that addresses and descriptors are uniform values; one
      // elected lane issues
      const bool is_qk = warp == 1;
      const uint32_t id_qk = idesc_e4m3(128, 128, false, false);
      const uint32_t id_pv = idesc_e4m3(128, 128, false, true);   // kind::f16: type fields 0, fp16
      const uint64_t dQ = tc::smem_desc(tc::smem_u32(sQ), 16, 1024);
      const uint64_t dK = tc::smem_desc(tc::smem_u32(sK), 16, 1024);
      const uint64_t dW = tc::smem_desc(tc::smem_u32(sW), kHalves / 2, 1024);
      int kt = 0;
      bool ok = true;
      Item it;
#pragma unroll 1
      for (int li = 0; ok && __all_sync(0xffffffffu, next_item(sh.items, li, it, abort_flag)); ++li) {
        const int par = li & 1;
        if (is_qk) ok = wait1(&sh.q_full[par], li >> 1, abort_flag);
        else if (li > 0) ok = wait1(&sh.o_free, li - 1, abort_flag);
#pragma unroll 1
        for (int j = it.j0; j < it.j1; ++j, ++kt) {
          const int b = kt % kBufs, use = kt / kBufs;
          if (is_qk) {
            const int st = kt % kKStages, slot = kt % kScaleRing;
            ok = ok && wait1(&sh.sc_full[slot], kt / kScaleRing, abort_flag) &&
                 wait1(&sh.k_full[st], kt / kKStages, abort_flag) &&
                 (use == 0 || wait1(&sh.pv_done[b], use - 1, abort_flag));
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc::tc_fence_after();
            const uint32_t tS = tmem + b * 128;
            const uint64_t kb = dK + uint64_t(st) * (kTile >> 4);
            const uint64_t qa = dQ + uint64_t(par) * (kPair >> 4);
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                mma_e4m3_ss(tS, qa + 2 * k, kb + 2 * k, id_qk, k > 0 ? 1u : 0u);
                mma_e4m3_ss(tS, qa + (kTile >> 4) + 2 * k, kb + 2 * k, id_qk, 1u);
              }
              tc::mma_commit(&sh.s_full[b]);
              tc::mma_commit(&sh.k_empty[st]);
              if (j == it.j1 - 1) tc::mma_commit(&sh.q_empty[par]);
            }
            __syncwarp();
          } else {
            const int wb = kt & 1;
            ok = __all_sync(0xffffffffu, ok && wait1(&sh.w_full[wb], kt >> 1, abort_flag) &&
                                             wait1(&sh.p_full[b], use, abort_flag));
            if (!ok) break;
            tc::tc_fence_after();
            const uint64_t vb = dW + uint64_t(wb) * (kHalves >> 4);
            const uint32_t tP = tmem + b * 128, acc = j > it.j0 ? 1u : 0u;
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < 8; ++k)          // 16 slots: 8 columns of P, 16 rows of V
                tc::mma_bf16_ts(tmem + kTmemO, tP + 32 * (k >> 1) + 8 * (k & 1), vb + k * (2048 >> 4),
                                id_pv, k > 0 ? 1u : acc);
              tc::mma_commit(&sh.w_empty[wb]);
              tc::mma_commit(&sh.pv_done[b]);
              if (j == it.j1 - 1) tc::mma_commit(&sh.o_full);
            }
            __syncwarp();
          }
        }
      }
      if (!ok) *abort_flag = 1;
      // nothing issued here may still run when TMEM is released (bounded, abort or not)
      if (elect_one()) tc::mma_commit(&sh.drain[is_qk ? 0 : 1]);
      __syncwarp();
      volatile int never = 0;
      tc::mbar_wait(&sh.drain[is_qk ? 0 : 1], 0, &never, kWaitLimit / 8);
      __syncwarp();
    }
  } else if (warp < 20) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ===================================================================== softmax
    const int part = (warp - 4) >> 2, q = warp & 3;  // quarter of a tile's keys; of its rows
    const uint32_t lane_addr = uint32_t(q * 32) << 16;
    const int m = q * 32 + lane;                     // this thread's row of the tile
    const int bar_q = 1 + q;                         // the four warps of these rows
    const int tl = m / a.G;
    int kt = 0;
    bool ok = true;                                  // no early exit: see the file's comment
    Item it;
#pragma unroll 1
    for (int li = 0;; ++li) {
      // the four leave together: an expired wait in one must not leave the others at a barrier
      if (bar_any(bar_q, 128, !next_item(sh.items, li, it, abort_flag))) break;
      const int par = li & 1;
      const int P = it.P, kv_len = it.P + it.T;
      const int t = it.mt * d.tpt + tl;
      const bool valid = tl < d.tpt && t < it.T;
      const uint32_t* arow = valid ? a.anc + size_t(it.o + t) * a.W : nullptr;
      // a quarter without a row only keeps the handshakes: its rows of P feed its rows of O
      const bool live = __any_sync(0xffffffffu, valid);
      ok &= wait1(&sh.q_full[par], li >> 1, abort_flag);
      const float qm = sh.qmul[par][m];
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sh.q_empty[par]);
      float add = INFINITY, lsum = 0.f;
#pragma unroll 1
      for (int j = it.j0; j < it.j1; ++j, ++kt) {
        const int b = kt % kBufs, use = kt / kBufs, slot = kt % kScaleRing;
        const int key0 = j * kBN + part * 32;
        ok &= wait1(&sh.s_full[b], use, abort_flag);   // (the issuer has waited for the scales)
        __syncwarp();
        tc::tc_fence_after();
        if (live) {
          const bool masked = j * kBN + kBN > P;
          const ScaleSlot& sc = sh.sc[slot];
          const uint32_t tS = tmem + lane_addr + b * 128 + part * 32;
          // the weights of this thread's 32 keys against the reference kLift - add, in fp16;
          // `top`: the largest exponent, `sum`: of the weights over the V scales
          float top, sum;
          uint32_t pk[16];
          auto seen = [&]() -> uint32_t {              // the keys that this row sees
            const int pre = P - key0, left = kv_len - key0;
            uint32_t vis = anc_window(arow, a.W, key0 - P);
            vis |= pre >= 32 ? 0xFFFFFFFFu : pre > 0 ? (1u << pre) - 1u : 0u;
            // (mask bits past the tree count for nothing)
            return vis & (left >= 32 ? 0xFFFFFFFFu : left > 0 ? (1u << left) - 1u : 0u);
          };
          auto weights = [&](float add) {
            const float shift = add == INFINITY ? 0.f : add;   // no key seen yet
            uint32_t x[32];
            tc::tmem_ld32(tS, x);
            tc::tmem_ld_wait();
            if (key0 + 32 > P) {
              const uint32_t vis = seen();
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((vis >> e) & 1u)) x[e] = __float_as_uint(-INFINITY);
            }
            top = -INFINITY;
            sum = 0.f;
#pragma unroll
            for (int g = 0; g < 2; ++g) {              // 16 keys of one page
              const int page = (part * 32 + 16 * g) >> d.log2bs;
              // (never 0, which would make a masked key's -infinity a NaN)
              const float mul = fmaxf(sc.k[page] * qm, FLT_MIN), lift = sc.lv[page] + shift;
              const uint64_t mul2 = f2_pack(mul, mul), lift2 = f2_pack(lift, lift);
              float s0 = 0.f, s1 = 0.f;
#pragma unroll
              for (int e = 0; e < 16; e += 4) {
                float z[4], p[4];
#pragma unroll
                for (int u = 0; u < 4; u += 2) {
                  const uint32_t* xe = &x[16 * g + e + u];
                  f2_unpack(f2_fma(f2_pack(__uint_as_float(xe[0]), __uint_as_float(xe[1])), mul2, lift2),
                            z[u], z[u + 1]);
                }
                top = fmax3(fmax3(top, z[0], z[1]), z[2], z[3]);
#pragma unroll
                for (int u = 0; u < 4; ++u) p[u] = ex2(z[u]);
                s0 += p[0] + p[1];
                s1 += p[2] + p[3];
                pk[g * 8 + e / 2] = pack_f16x2(p[0], p[1]);
                pk[g * 8 + e / 2 + 1] = pack_f16x2(p[2], p[3]);
              }
              sum = fmaf(s0 + s1, sc.iv[page], sum);
            }
            top -= shift;
          };
          // The weights are formed on the expectation that the tile does not move a row's reference,
          // and formed again where it does (they stay in registers until then: P lies over S).
          weights(add);
          if (bar_any(bar_q, 128, top + add > kTop)) {
            sh.mx[part][m] = top;
            bar_sync(bar_q, 128);
            const float ref = fmaxf(fmaxf(fmaxf(sh.mx[0][m], sh.mx[1][m]), fmaxf(sh.mx[2][m], sh.mx[3][m])),
                                    kLift - add);
            const float next = kLift - ref;
            const float factor = add == INFINITY ? 1.f : ex2(next - add);
            add = next;
            lsum *= factor;
            if (j > it.j0 && __any_sync(0xffffffffu, factor != 1.f)) {
              ok &= wait1(&sh.pv_done[(kt - 1) % kBufs], (kt - 1) / kBufs, abort_flag);
              __syncwarp();
              tc::tc_fence_after();
              uint32_t ov[32];                         // each of the four a quarter of the columns
              const uint32_t to = tmem + lane_addr + kTmemO + part * 32;
              tc::tmem_ld32(to, ov);
              tc::tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * factor);
              tc::tmem_st32(to, ov);
            }
            weights(add);
          }
          if (masked) {
            ok &= wait1(&sh.w_full[kt & 1], kt >> 1, abort_flag);
            const uint32_t v_nan = sh.v_nan[kt & 1][part];
            __syncwarp();
            if (v_nan != 0) {
              const uint32_t hit = v_nan & seen();
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const uint32_t n = (hit >> (2 * e)) & 3u;
                pk[e] |= ((n & 1u) | (n & 2u) << 15) * 0x7FFFu;
              }
            }
          }
          tc::tmem_st16(tS, pk);
          lsum += sum;
          tc::tmem_st_wait();
        }
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          tc::mbar_arrive(&sh.sc_empty[slot]);
          tc::mbar_arrive(&sh.p_full[b]);
        }
      }
      if (li > 1) ok &= wait1(&sh.sum_free[par], (li >> 1) - 1, abort_flag);
      sh.sum[par][part][m] = lsum;
      if (part == 0) sh.add[par][m] = add;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sh.sum_full[par]);
    }
    if (!ok) *abort_flag = 1;
  } else if (warp >= 28) {
    // ===================================================================== V to fp16
    // e4m3 values are fp16 values.  (The conversion by shifts and masks instead of cvt: 387 us against
    // 303 on 32 trees of 46; two warps instead of four 519, two vectors at a time 316; in halves of a
    // tile that the product waits for one by one 307.)
    // Eight lanes to a row, a 16-byte vector each, which becomes two (both tiles in 128-byte swizzle);
    // lanes of the upper columns store their second vector first, so that the eight hit all
    // banks.  Where keys are masked, a NaN code times a zero weight must stay zero: stale rows
    // past the end become zeros, and a tree slot's NaN becomes a bit in v_nan, from which the
    // softmax warps make it one in the weights of the rows that see it.
    const int cw = warp - 28, c = lane & 7, rq = lane >> 3;
    int kt = 0;
    bool ok = true;
    Item it;
#pragma unroll 1
    for (int li = 0; ok && __all_sync(0xffffffffu, next_item(sh.items, li, it, abort_flag)); ++li) {
#pragma unroll 1
      for (int j = it.j0; j < it.j1; ++j, ++kt) {
        const int st = kt % kVStages, wb = kt & 1;
        ok = __all_sync(0xffffffffu,
                        wait1(&sh.v_full[st], kt / kVStages, abort_flag) &&
                            (kt < 2 || wait1(&sh.w_empty[wb], (kt >> 1) - 1, abort_flag)));
        if (!ok) break;
        const uint8_t* const from = sV + st * kTile + (cw * 32 + rq) * 128;
        uint8_t* const to = sW + wb * kHalves + (c >> 2) * (kHalves / 2) + (cw * 32 + rq) * 128;
        const int live = it.P + it.T - j * kBN, tree = it.P - j * kBN;   // rows that exist; before the tree
        uint32_t found = 0u;
        uint4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
          v[u] = *reinterpret_cast<const uint4*>(from + u * 512 + ((c ^ ((u & 1) * 4 + rq)) << 4));
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sh.v_empty[st]);   // (the tile is in registers)
        if (tree < kBN) {
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const int r = cw * 32 + u * 4 + rq;
            if (r < tree) continue;
            uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w}, hit = 0u;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t n = nan_bytes(w[e]);
              hit |= n;
              w[e] = r >= live ? 0u : w[e] & ~((n >> 7) * 255u);
            }
            if (hit != 0u && r < live) found |= 1u << (u * 4 + rq);
            v[u] = make_uint4(w[0], w[1], w[2], w[3]);
          }
          found = __reduce_or_sync(0xffffffffu, found);
          if (lane == 0) sh.v_nan[wb][cw] = found;
        }
        const bool second = c >= 4;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
          uint32_t h[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            h[2 * e] = kv8::e4m3x2_to_f16x2(w[e] & 0xFFFFu);
            h[2 * e + 1] = kv8::e4m3x2_to_f16x2(w[e] >> 16);
          }
          uint8_t* const row = to + u * 512;
          const int even = ((2 * (c & 3)) ^ ((u & 1) * 4 + rq)) << 4;
          const uint4 h0 = make_uint4(h[0], h[1], h[2], h[3]), h1 = make_uint4(h[4], h[5], h[6], h[7]);
          *reinterpret_cast<uint4*>(row + (second ? even ^ 16 : even)) = second ? h1 : h0;
          *reinterpret_cast<uint4*>(row + (second ? even : even ^ 16)) = second ? h0 : h1;
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sh.w_full[wb]);
      }
    }
    if (!ok) *abort_flag = 1;
  } else {
    // ===================================================================== queries, output
    const int q = warp & 3;
    const uint32_t lane_addr = uint32_t(q * 32) << 16;
    const int m = q * 32 + lane;
    const int tl = m / a.G, gl = m - tl * a.G;       // token and head of this thread's output row
    bool ok = true;
    struct Unit {
      int o, T, h, mt, slot;
    };
    auto fetch = [&](int li, Unit& u) -> bool {
      Item it;
      const bool has = __all_sync(0xffffffffu, next_item(sh.items, li, it, abort_flag));
      u.o = it.o;
      u.T = it.T;
      u.h = it.h;
      u.mt = it.mt;
      u.slot = it.slot;
      return has;
    };
    // a row to each half warp, 16 bytes a lane, two rows of it in flight
    auto put_q = [&](int li, const Unit& u) {
      const int b = li & 1, c = lane & 15;
      uint8_t* p = sQ + b * kPair;
      if (li > 1) ok &= wait1(&sh.q_empty[b], (li >> 1) - 1, abort_flag);
      auto load = [&](int n) -> uint4 {
        const int rl = n / a.G, g = n - rl * a.G, t = u.mt * d.tpt + rl;
        if (n >= kRows || rl >= d.tpt || t >= u.T) return make_uint4(0, 0, 0, 0);
        return __ldg(reinterpret_cast<const uint4*>(
                         static_cast<const __nv_bfloat16*>(a.q) +
                         (size_t(u.o + t) * a.H_q + u.h * a.G + g) * kD) + c);
      };
      const int n0 = q * 2 + (lane >> 4);
      uint4 w0 = load(n0), w1 = load(n0 + 8), w2 = load(n0 + 16);
#pragma unroll 1
      for (int n = n0; n < kRows; n += 8) {
        const uint4 w = w0;
        w0 = w1;
        w1 = w2;
        w2 = load(n + 24);
        float f[8], mx = 0.f;
        elem<__nv_bfloat16>::unpack(w, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) mx = fabsf(f[e]) <= FLT_MAX ? fmaxf(mx, fabsf(f[e])) : mx;
#pragma unroll
        for (int s = 8; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
        const float sq = kv8::need_scale(mx);
        uint2 hi, lo;
        split_q8(w, __uint_as_float((254u << 23) - __float_as_uint(sq)), hi, lo);
        const int off = (n >> 3) * 1024 + (n & 7) * 128 + (((c >> 1) ^ (n & 7)) << 4) + (c & 1) * 8;
        *reinterpret_cast<uint2*>(p + off) = hi;
        *reinterpret_cast<uint2*>(p + kTile + off) = lo;
        if (c == 0) sh.qmul[b][n] = sq * a.scale_log2;
      }
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sh.q_full[b]);
    };
    Unit cur, next, after;
    bool has = fetch(0, cur), has_next = false;
    if (has) {
      put_q(0, cur);
      has_next = fetch(1, next);
      if (has_next) put_q(1, next);
    }
#pragma unroll 1
    for (int li = 0; has; ++li) {
      const bool has_after = has_next && fetch(li + 2, after);
      const int par = li & 1;
      const int t = cur.mt * d.tpt + tl;
      const bool valid = tl < d.tpt && t < cur.T;
      ok &= wait1(&sh.sum_full[par], li >> 1, abort_flag);
      const float l = (sh.sum[par][0][m] + sh.sum[par][1][m]) + (sh.sum[par][2][m] + sh.sum[par][3][m]);
      const float add = sh.add[par][m];
      const float inv = l == 0.f ? 0.f : kSumMul / l;    // (NaN stays NaN)
      const float lse2 = l == 0.f ? -INFINITY : log2f(l) + kSumShift - add;
      const size_t row = cur.slot < 0 ? size_t(cur.o + t) * a.H_q + cur.h * a.G + gl
                                      : size_t(cur.slot) * kRows + m;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sh.sum_free[par]);
      ok &= wait1(&sh.o_full, li, abort_flag);
      __syncwarp();
      tc::tc_fence_after();
#pragma unroll 1
      for (int c0 = 0; c0 < 128; c0 += 32) {
        uint32_t ov[32];
        __syncwarp();
        tc::tmem_ld32(tmem + lane_addr + kTmemO + c0, ov);
        tc::tmem_ld_wait();
        if (c0 == 96) {                              // O is read: the next unit may begin
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&sh.o_free);
        }
        // (a row that saw nothing may hold whatever P's other rows left: 0 by definition)
        if (!valid) continue;
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          float v[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) v[u] = l == 0.f ? 0.f : __uint_as_float(ov[e + u]) * inv;
          if (cur.slot < 0) {
            uint32_t w[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const __nv_bfloat162 z = __floats2bfloat162_rn(v[2 * u], v[2 * u + 1]);
              w[u] = *reinterpret_cast<const uint32_t*>(&z);
            }
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) + row * kD + c0 + e) =
                make_uint4(w[0], w[1], w[2], w[3]);
          } else {
            float4* o4 = reinterpret_cast<float4*>(d.part_o + row * kD + c0 + e);
            o4[0] = make_float4(v[0], v[1], v[2], v[3]);
            o4[1] = make_float4(v[4], v[5], v[6], v[7]);
          }
        }
      }
      if (valid) {
        if (cur.slot >= 0) d.part_lse[row] = lse2;
        else if (a.lse) a.lse[row] = lse2 * 0.6931471805599453f;
      }
      if (has_after) put_q(li + 2, after);
      cur = next;
      next = after;
      has = has_next;
      has_next = has_after;
    }
    if (!ok) *abort_flag = 1;
  }
  tc::tc_fence_before();
  __syncthreads();
  if (*abort_flag)                           // every request of the range is unreliable
#pragma unroll 1
    for (int r = sh.r0 + tid; r <= sh.r1; r += kThreads) atomicOr(&a.req_status[r], SPEC_REQ_TIMEOUT);
  tc::tc_fence_after();
  if (warp == 0) tc::tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------------------ join of pieces
// CTA (c, y): eight rows of the cut unit of record c, one a warp, lane l columns 4 l .. 4 l + 3.
// Four pieces' loads at a time are in flight.
__global__ void __launch_bounds__(256) attn_kv8_join_kernel(TcDev d) {
  pdl_wait();
  pdl_trigger();
  const MergeRec rec = d.recs[blockIdx.x];
  if (rec.np < 2) return;
  const AttnKv8Dev& a = d.a;
  const int lane = threadIdx.x & 31;
  const int m = blockIdx.y * 8 + (threadIdx.x >> 5);
  const int t = rec.mt * d.tpt + m / a.G, g = m % a.G;
  if (m >= d.tpt * a.G || t >= rec.T) return;
  float M = -INFINITY, sum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int p0 = 0; p0 < rec.np; p0 += 4) {
    float ls[4];
    float4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int p = p0 + u;
      ls[u] = -INFINITY;
      v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (p < rec.np) {
        const size_t row = size_t(p == 0 ? rec.slot0 : 2 * (int(blockIdx.x) + (p << d.pair))) * d.part_rows + m;
        ls[u] = d.part_lse[row];
        v[u] = reinterpret_cast<const float4*>(d.part_o + row * kD)[lane];
      }
    }
    float top = M;
    bool any = false;                                  // (a NaN counts, and makes the row NaN)
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      top = fmaxf(top, ls[u]);
      any = any || ls[u] != -INFINITY;
    }
    if (!any) continue;
    const float f = M == -INFINITY ? 0.f : ex2(M - top);
    sum *= f;
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] *= f;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float w = ls[u] == -INFINITY ? 0.f : ex2(ls[u] - top);
      sum += w;
      acc[0] = fmaf(w, v[u].x, acc[0]);
      acc[1] = fmaf(w, v[u].y, acc[1]);
      acc[2] = fmaf(w, v[u].z, acc[2]);
      acc[3] = fmaf(w, v[u].w, acc[3]);
    }
    M = top;
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const size_t row = size_t(rec.o + t) * a.H_q + rec.h * a.G + g;
  __nv_bfloat162 lo = __floats2bfloat162_rn(acc[0] * inv, acc[1] * inv);
  __nv_bfloat162 hi = __floats2bfloat162_rn(acc[2] * inv, acc[3] * inv);
  uint2 w;
  w.x = *reinterpret_cast<uint32_t*>(&lo);
  w.y = *reinterpret_cast<uint32_t*>(&hi);
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + row * kD + 4 * lane) = w;
  if (lane == 0 && a.lse)
    a.lse[row] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * 0.6931471805599453f;
}

// ------------------------------------------------------------------------------ host
struct WsLayout {
  size_t recs, part_o, part_lse, total;
};
static WsLayout ws_layout(int ctas, int part_rows) {
  WsLayout w;
  const size_t slots = 2 * size_t(ctas);
  size_t off = 0;
  w.recs = off;
  off = align_up(off + sizeof(MergeRec) * size_t(ctas), 256);
  w.part_o = off;
  off = align_up(off + sizeof(float) * slots * part_rows * kD, 256);
  w.part_lse = off;
  off = align_up(off + sizeof(float) * slots * part_rows, 256);
  w.total = off;
  return w;
}

static PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess && q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// a cache's rows of 128 codes, one page a box; and its pages, as many as fill a tile a box
static bool encode_maps(PFN_cuTensorMapEncodeTiled_v12000 enc, const AttnKv8Dev& a, const void* ptr,
                        CUtensorMap* page, CUtensorMap* wide) {
  const cuuint64_t rows = cuuint64_t(a.num_blocks) * a.H_kv * a.bs;
  const cuuint32_t one[4] = {1, 1, 1, 1};
  cuuint64_t dims[4] = {kD, rows, 0, 0}, strides[3] = {kD, 0, 0};
  cuuint32_t box[4] = {kD, cuuint32_t(a.bs), 0, 0};
  if (enc(page, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box, one,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return false;
  cuuint64_t dims4[4] = {kD, cuuint64_t(a.bs), cuuint64_t(a.H_kv), cuuint64_t(a.num_blocks)};
  cuuint64_t strides4[3] = {kD, cuuint64_t(a.bs) * kD, cuuint64_t(a.H_kv) * a.bs * kD};
  cuuint32_t box4[4] = {kD, cuuint32_t(a.bs), 1, cuuint32_t(kBN / a.bs)};
  return enc(wide, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(ptr), dims4, strides4, box4,
             one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Query rows of a unit's row tile: the smallest form that holds a request's rows.  Over 8192 slots,
// 16 requests, 8 KV heads: 8 rows 53.4 us in the form of 8, 63.1 in that of 16, 86.0 in tiles of
// 128; 16 rows 67.2 and 87.0.
static int rows_of(const AttnKv8Dev& a) {
  const int rows = a.T_max * a.G;
  return rows <= 8 ? 8 : rows <= 16 ? 16 : tile::kRows;
}

static int device_ctas() {
  const int sms = sm_count_current_device();
  return sms < kMaxCtas ? sms : kMaxCtas;
}

}  // namespace kv8tc

// Whether the tensor-core kernels take this call: their types and tile shapes, a row tile that holds
// a token's query heads, row coordinates of TMA in 32 bits.  (32 and 64 query heads of one KV head,
// 64 x 1 and 16 x 4 tokens over 8192 slots: 54 and 46 us here, 1120 and 1596 us on CUDA cores.)
bool attn_kv8_tc_takes(const AttnKv8Dev& a, bool bf16) {
  return bf16 && a.d == 128 && (a.bs == 16 || a.bs == 32 || a.bs == 64 || a.bs == 128) &&
         a.G <= kv8tc::tile::kRows &&
         (long long)a.num_blocks * a.H_kv * a.bs + 128 < (1LL << 31);
}

size_t attn_kv8_tc_workspace(const AttnKv8Dev& a) {
  using namespace kv8tc;
  return ws_layout(device_ctas(), rows_of(a)).total;
}

spec_status_t launch_attn_kv8_tc(const AttnKv8Dev& a, void* ws, size_t ws_bytes, cudaStream_t s) {
  using namespace kv8tc;
  const int ctas = device_ctas();
  if (ctas <= 0) return SPEC_ERR_CUDA;
  TcDev d;
  d.a = a;
  d.part_rows = rows_of(a);
  d.tpt = d.part_rows / a.G;
  d.log2bs = a.bs == 16 ? 4 : a.bs == 32 ? 5 : a.bs == 64 ? 6 : 7;
  d.kv_rows = a.num_blocks * a.H_kv * a.bs;
  d.ctas = ctas;
  d.min_tiles = 2;   // one token over 2047 slots: 11.1 us; 12.2 with 1, 11.5 with 4, 14.1 with 8
  d.pair = a.T_max * a.G > tile::kRows && ctas > 1;
  const WsLayout lay = ws_layout(ctas, d.part_rows);
  if (!ws || ws_bytes < lay.total || (reinterpret_cast<uintptr_t>(ws) & 255u))
    return SPEC_ERR_INVALID_ARG;
  char* w = static_cast<char*>(ws);
  d.recs = reinterpret_cast<MergeRec*>(w + lay.recs);
  d.part_o = reinterpret_cast<float*>(w + lay.part_o);
  d.part_lse = reinterpret_cast<float*>(w + lay.part_lse);
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return SPEC_ERR_CUDA;
  CUtensorMap mK, mV, mKw, mVw;
  if (!encode_maps(enc, a, a.k, &mK, &mKw) || !encode_maps(enc, a, a.v, &mV, &mVw))
    return SPEC_ERR_INVALID_ARG;
  static DeviceOnce raised8, raised16, raised_tile;
  spec_status_t st = raise_dyn_smem_once(attn_kv8_rows_kernel<8>, rows::smem_bytes<8>(), raised8);
  if (st == SPEC_OK)
    st = raise_dyn_smem_once(attn_kv8_rows_kernel<16>, rows::smem_bytes<16>(), raised16);
  if (st == SPEC_OK) st = raise_dyn_smem_once(attn_kv8_tile_kernel, tile::kSmemBytes, raised_tile);
  if (st != SPEC_OK) return st;
  cudaError_t e =
      d.part_rows == tile::kRows
          ? launch_pdl(attn_kv8_tile_kernel, dim3(ctas), dim3(tile::kThreads),
                       size_t(tile::kSmemBytes), s, mK, mV, mKw, mVw, d)
      : d.part_rows == 8
          ? launch_pdl(attn_kv8_rows_kernel<8>, dim3(ctas), dim3(rows::kThreads),
                       size_t(rows::smem_bytes<8>()), s, mK, mV, mKw, mVw, d)
          : launch_pdl(attn_kv8_rows_kernel<16>, dim3(ctas), dim3(rows::kThreads),
                       size_t(rows::smem_bytes<16>()), s, mK, mV, mKw, mVw, d);
  if (e == cudaSuccess)
    e = launch_pdl(attn_kv8_join_kernel, dim3(ctas, (d.part_rows + 7) / 8), dim3(256), 0, s, d);
  return launch_result(e);
}

}  // namespace spec
