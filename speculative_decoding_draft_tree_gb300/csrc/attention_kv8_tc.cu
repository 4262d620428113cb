// spec_tree_attention_kv8 on the tcgen05 tensor cores: bf16 queries, head_dim 128.
//
// attn_kv8_rows16_kernel: units of at most 16 query rows (T x G <= 16: single tokens and short
// chains).  S^T = K Q^T (M = 128 slots on the TMEM lanes, N = 16 rows), so that the softmax spends
// its lanes on keys; O^T += V^T P^T with V read as an MN-major operand.  Bound by the codes' bytes:
// a tile's 32 KB take ~1400 clocks of an SM's share of HBM, the two products a fraction of that,
// so what has to keep up is the softmax.  Its work is halved by two groups of four warps that
// take alternate tiles, each with its own references, sums and accumulator, joined per unit.
// Warps: 0 copies K, 2 copies V, 1 issues the scores' products, 3 the output's, 4-7 and 8-11 the
// softmax groups, 12 brings the queries and splits them in two pieces, 13 brings the scales.
//
// Scales: a score is code product * (K scale of the slot's page * the row's query scale); the V
// scale joins the exponent, y = score + log2(V scale), and the weight 2^(y - ref) goes into the
// product with V's codes while the row sum takes 2^(y - ref) / (V scale).  So the weights that
// enter the product fill e4m3's range whatever the pages' scales are.
//
// The waits are bounded; one that runs out raises the CTA's abort flag, after which no wait
// blocks: the softmax groups, which meet at hardware barriers, still walk through their tiles, the
// other roles leave, and the range's requests get SPEC_REQ_TIMEOUT.
#include <math.h>

#include <mutex>

#include "attention_kv8_tc.cuh"

namespace spec {
namespace kv8tc {

namespace r16 {
constexpr int kRows = 16;
constexpr int kThreads = 512;                            // 16 warps, two of them spare
constexpr int kCtlRegs = 96;                             // registers a thread (setmaxnreg):
constexpr int kSoftmaxRegs = 160;                        // two warpgroups each
static_assert(2 * 128 * (kCtlRegs + kSoftmaxRegs) <= kThreads * 128, "register split fits");
constexpr int kKStages = 6;
constexpr int kVStages = 5;
constexpr int kPiece = kRows * 128;                      // bytes of 16 rows of one piece
constexpr int kSmemQ = 0;                                // 2 buffers x (hi, lo)
constexpr int kSmemP = kSmemQ + 2 * 2 * kPiece;          // 2 groups x 2 buffers x (hi, lo)
constexpr int kSmemK = kSmemP + 2 * 2 * 2 * kPiece;
constexpr int kSmemV = kSmemK + kKStages * kTile;
constexpr int kSmemBar = kSmemV + kVStages * kTile;
constexpr uint32_t kTmemCols = 128;                      // S^T: 4 x 16, O^T: 2 x 16 from 64 on
constexpr uint32_t kTmemO = 64;
static_assert(kSmemK % 1024 == 0 && kSmemV % 1024 == 0, "swizzled tiles on 1024-byte bounds");

struct Shared {
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[kKStages], k_empty[kKStages], v_full[kVStages], v_empty[kVStages];
  uint64_t s_full[2][2], s_free[2][2], p_full[2][2], pv_done[2][2], o_free[2];
  uint64_t sc_full[kScaleRing], sc_empty[kScaleRing], drain[2];
  ScaleSlot sc[kScaleRing];
  alignas(16) float qmul[2][kRows];
  float mx[2][4][kRows];          // per group and warp: row maxima of an update
  float sum[2][2][4][kRows];      // per item parity, group and warp: row sums
  float add[2][2][kRows];         // per item parity and group: kShift - reference
  long long s64[20];
  int s32[2];
  uint32_t tmem;
  int abort;
};
constexpr int kSmemEnd = kSmemBar + int(sizeof(Shared));
constexpr int kSmemBytes = kSmemEnd + 1024;
static_assert(kSmemBytes <= 232448, "fits one CTA's shared memory");
}  // namespace r16

__global__ void __launch_bounds__(r16::kThreads, 1)
attn_kv8_rows16_kernel(const __grid_constant__ CUtensorMap mK,
                       const __grid_constant__ CUtensorMap mV,
                       const __grid_constant__ CUtensorMap mKw,
                       const __grid_constant__ CUtensorMap mVw, TcDev d) {
  using namespace r16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* sQ = base + kSmemQ;
  uint8_t* sP = base + kSmemP;
  uint8_t* sK = base + kSmemK;
  uint8_t* sV = base + kSmemV;
  Shared& sh = *reinterpret_cast<Shared*>(base + kSmemBar);
  const AttnKv8Dev& a = d.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  pdl_trigger();
  const Range R = cta_range<kThreads>(d, sh.s64, sh.s32);
  if (tid == 0) write_merge_record(d, R);
  if (R.t0 >= R.t1) return;                  // uniform; nothing allocated yet
  if (tid == 0) {
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&sh.q_full[b], 1);
      tc::mbar_init(&sh.q_empty[b], 9);      // the issuer's commit and the 8 softmax warps
      for (int g = 0; g < 2; ++g) {
        tc::mbar_init(&sh.s_full[g][b], 1);
        tc::mbar_init(&sh.s_free[g][b], 4);
        tc::mbar_init(&sh.p_full[g][b], 4);
        tc::mbar_init(&sh.pv_done[g][b], 1);
      }
      tc::mbar_init(&sh.o_free[b], 8);
      tc::mbar_init(&sh.drain[b], 1);
    }
    for (int s = 0; s < kKStages; ++s) {
      tc::mbar_init(&sh.k_full[s], 1);
      tc::mbar_init(&sh.k_empty[s], 1);
    }
    for (int s = 0; s < kVStages; ++s) {
      tc::mbar_init(&sh.v_full[s], 1);
      tc::mbar_init(&sh.v_empty[s], 1);
    }
    for (int s = 0; s < kScaleRing; ++s) {
      tc::mbar_init(&sh.sc_full[s], 1);
      tc::mbar_init(&sh.sc_empty[s], 4);
    }
    sh.abort = 0;
    tc::fence_mbar_init();
  }
  if (warp == 0) {
    tc::tmem_alloc(&sh.tmem, kTmemCols);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = sh.tmem;
  volatile int* abort_flag = &sh.abort;

  if (warp < 4 || warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCtlRegs));
  if (warp == 0) {
    page_producer(d, R, &mK, &mKw, kKStages, sK, sh.k_full, sh.k_empty, true, &sh.abort);
  } else if (warp == 2) {
    page_producer(d, R, &mV, &mVw, kVStages, sV, sh.v_full, sh.v_empty, false, &sh.abort);
  } else if (warp == 13) {
    scale_producer(d, R, sh.sc, sh.sc_full, sh.sc_empty, &sh.abort);
  } else if (warp == 12) {
    // ===================================================================== queries
    // lanes 0-15 and 16-31 a row each, eight rows a half: a row's scale brings its largest element
    // into (224, 448]
    const int c = lane & 15;
    ItemIter iter;
    iter.start(d, R);
    Item it;
    bool ok = true;
    for (int li = 0; ok && iter.next(d, R, it); ++li) {
      const int b = li & 1, use = li >> 1;
      uint4 w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int n = 2 * k + (lane >> 4), t = n / a.G, g = n - t * a.G;
        w[k] = make_uint4(0, 0, 0, 0);
        if (t < it.T)
          w[k] = __ldg(reinterpret_cast<const uint4*>(
                     static_cast<const __nv_bfloat16*>(a.q) +
                     (size_t(it.o + t) * a.H_q + it.h * a.G + g) * kD) + c);
      }
      if (use > 0 && !lane0_wait(&sh.q_empty[b], use - 1, abort_flag)) {
        ok = false;
        break;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int n = 2 * k + (lane >> 4);
        float f[8], m = 0.f;
        elem<__nv_bfloat16>::unpack(w[k], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fabsf(f[e]) <= FLT_MAX ? fmaxf(m, fabsf(f[e])) : m;
#pragma unroll
        for (int s = 8; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
        const float sq = kv8::need_scale(m);
        uint2 hi, lo;
        split_q8(w[k], __uint_as_float((254u << 23) - __float_as_uint(sq)), hi, lo);
        const int off = (n >> 3) * 1024 + (n & 7) * 128 + (((c >> 1) ^ (n & 7)) << 4) + (c & 1) * 8;
        uint8_t* p = sQ + b * 2 * kPiece;
        *reinterpret_cast<uint2*>(p + off) = hi;
        *reinterpret_cast<uint2*>(p + kPiece + off) = lo;
        if (c == 0) sh.qmul[b][n] = sq * a.scale_log2;
      }
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sh.q_full[b]);
    }
    if (!ok && lane == 0) *abort_flag = 1;
    __syncwarp();
  } else if (warp == 1 || warp == 3) {
    // ===================================================================== MMA issuers
    if (lane == 0) {
      const bool is_qk = warp == 1;
      const uint32_t id_qk = idesc_e4m3(128, kRows, false, false);
      const uint32_t id_pv = idesc_e4m3(128, kRows, true, false);
      const uint64_t dQ = tc::smem_desc(tc::smem_u32(sQ), 16, 1024);
      const uint64_t dP = tc::smem_desc(tc::smem_u32(sP), 16, 1024);
      const uint64_t dK = tc::smem_desc(tc::smem_u32(sK), 16, 1024);
      const uint64_t dV = tc::smem_desc(tc::smem_u32(sV), kTile, 1024);
      int kt = 0, cnt[2] = {0, 0};     // tiles; tiles of each group
      bool ok = true;
      ItemIter iter;
      iter.start(d, R);
      Item it;
      for (int li = 0; ok && iter.next(d, R, it); ++li) {
        if (is_qk && !wait1(&sh.q_full[li & 1], li >> 1, abort_flag)) {
          ok = false;
          break;
        }
        for (int j = it.j0; j < it.j1; ++j, ++kt) {
          const int g = (j - it.j0) & 1, c = g ? cnt[1] : cnt[0], b = c & 1, use = c >> 1;
          if (is_qk) {
            const int st = kt % kKStages;
            if (!wait1(&sh.k_full[st], kt / kKStages, abort_flag) ||
                (use > 0 && !wait1(&sh.s_free[g][b], use - 1, abort_flag))) {
              ok = false;
              break;
            }
            tc::tc_fence_after();
            const uint32_t tS = tmem + (g * 2 + b) * kRows;
            const uint64_t ka = dK + uint64_t(st) * (kTile >> 4);
            const uint64_t qb = dQ + uint64_t(li & 1) * (2 * kPiece >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) {      // 32 elements a step: hi and lo against one K step
              mma_e4m3_ss(tS, ka + 2 * k, qb + 2 * k, id_qk, k > 0 ? 1u : 0u);
              mma_e4m3_ss(tS, ka + 2 * k, qb + (kPiece >> 4) + 2 * k, id_qk, 1u);
            }
            tc::mma_commit(&sh.s_full[g][b]);
            tc::mma_commit(&sh.k_empty[st]);
            if (j == it.j1 - 1) tc::mma_commit(&sh.q_empty[li & 1]);
          } else {
            const int st = kt % kVStages;
            const bool first = j - it.j0 < 2;   // the group's first tile of the item
            if (!wait1(&sh.p_full[g][b], use, abort_flag) ||
                !wait1(&sh.v_full[st], kt / kVStages, abort_flag) ||
                (first && li > 0 && !wait1(&sh.o_free[g], li - 1, abort_flag))) {
              ok = false;
              break;
            }
            tc::tc_fence_after();
            const uint32_t tO = tmem + kTmemO + g * kRows;
            const uint64_t va = dV + uint64_t(st) * (kTile >> 4);
            const uint64_t pb = dP + uint64_t(g * 2 + b) * (2 * kPiece >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) {      // 32 slots a step: four groups of 8 V rows
              mma_e4m3_ss(tO, va + k * (4096 >> 4), pb + 2 * k, id_pv, (k > 0 || !first) ? 1u : 0u);
              mma_e4m3_ss(tO, va + k * (4096 >> 4), pb + (kPiece >> 4) + 2 * k, id_pv, 1u);
            }
            tc::mma_commit(&sh.v_empty[st]);
            tc::mma_commit(&sh.pv_done[g][b]);
          }
          if (g) ++cnt[1];
          else ++cnt[0];
        }
      }
      if (!ok) *abort_flag = 1;
      // nothing issued here may still run when TMEM is released (bounded, abort or not)
      tc::mma_commit(&sh.drain[is_qk ? 0 : 1]);
      volatile int never = 0;
      tc::mbar_wait(&sh.drain[is_qk ? 0 : 1], 0, &never, kWaitLimit / 8);
    }
    __syncwarp();
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ===================================================================== softmax, epilogue
    const int grp = (warp - 4) >> 2, q = warp & 3;   // group; TMEM lane quarter
    const uint32_t lane_addr = uint32_t(q * 32) << 16;
    const int kl = q * 32 + lane;                    // this lane's slot of a tile; its d of O^T
    const int si = kl >> d.log2bs;
    const int bar_g = 1 + grp;
    int kt = 0, cnt[2] = {0, 0};
    bool ok = true;                                  // no early exit: see the file's comment
    ItemIter iter;
    iter.start(d, R);
    Item it;
    for (int li = 0; iter.next(d, R, it); ++li) {
      const int o = it.o, T = it.T, P = it.P, kv_len = P + T;
      const int nrows = T * a.G;                     // <= 16
      const int nt = it.j1 - it.j0;
      ok = warp_wait(&sh.q_full[li & 1], li >> 1, abort_flag) && ok;
      const float4* qmul = reinterpret_cast<const float4*>(sh.qmul[li & 1]);
      float add[kRows], lsum[kRows];
#pragma unroll
      for (int n = 0; n < kRows; ++n) {
        add[n] = INFINITY;
        lsum[n] = 0.f;
      }
      for (int i = grp; i < nt; i += 2) {
        const int kg = kt + i;                       // the tile's number in the CTA's stream
        const int c = cnt[grp], b = c & 1, use = c >> 1;
        const int slot = kg % kScaleRing;
        ok = warp_wait(&sh.sc_full[slot], kg / kScaleRing, abort_flag) && ok;
        const float ks = sh.sc[slot].k[si], lv = sh.sc[slot].lv[si], iv = sh.sc[slot].iv[si];
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sh.sc_empty[slot]);
        ok = warp_wait(&sh.s_full[grp][b], use, abort_flag) && ok;
        tc::tc_fence_after();
        uint32_t sv[kRows];
        tc::tmem_ld16(tmem + lane_addr + (grp * 2 + b) * kRows, sv);
        tc::tmem_ld_wait();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sh.s_free[grp][b]);
        const int key = (it.j0 + i) * kBN + kl;
        uint32_t vis = 0;
        if (key < P) {
          vis = (1u << nrows) - 1u;
        } else if (key < kv_len) {
          const int s = key - P;
          for (int t = 0; t < T; ++t) {
            const uint32_t w = a.anc[size_t(o + t) * a.W + (s >> 5)];
            if ((w >> (s & 31)) & 1u) vis |= ((1u << a.G) - 1u) << (t * a.G);
          }
        }
        float z[kRows], zmax = -INFINITY;
#pragma unroll
        for (int n4 = 0; n4 < kRows / 4; ++n4) {
          const float4 qm = qmul[n4];
          const float m4[4] = {ks * qm.x, ks * qm.y, ks * qm.z, ks * qm.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int n = n4 * 4 + e;
            z[n] = fmaf(__uint_as_float(sv[n]), m4[e], lv + add[n]);
            z[n] = ((vis >> n) & 1u) ? z[n] : -INFINITY;
            zmax = fmaxf(zmax, z[n]);
          }
        }
        if (bar_any(bar_g, 128, zmax > kCeil)) {
          // some row's reference moves up to its maximum so far
#pragma unroll
          for (int n = 0; n < kRows; ++n)
            z[n] = ((vis >> n) & 1u)
                       ? fmaf(__uint_as_float(sv[n]), ks * sh.qmul[li & 1][n], lv) : -INFINITY;
          const float top = reduce16<true>(z, lane);
          if (!(lane & 1)) sh.mx[grp][q][row16(lane)] = top;
          bar_sync(bar_g, 128);
          float factor[kRows];
#pragma unroll
          for (int n = 0; n < kRows; ++n) {
            const float ref = fmaxf(fmaxf(fmaxf(sh.mx[grp][0][n], sh.mx[grp][1][n]),
                                          fmaxf(sh.mx[grp][2][n], sh.mx[grp][3][n])),
                                    kShift - add[n]);
            const float now = kShift - ref;
            factor[n] = add[n] == INFINITY ? 1.f : ex2(now - add[n]);
            add[n] = now;
            lsum[n] *= factor[n];
            z[n] = ((vis >> n) & 1u) ? z[n] + now : -INFINITY;
          }
          if (i >= 2) {                              // the group's accumulator holds something
            ok = warp_wait(&sh.pv_done[grp][(c - 1) & 1], (c - 1) >> 1, abort_flag) && ok;
            tc::tc_fence_after();
            uint32_t ov[kRows];
            tc::tmem_ld16(tmem + lane_addr + kTmemO + grp * kRows, ov);
            tc::tmem_ld_wait();
#pragma unroll
            for (int n = 0; n < kRows; ++n)
              ov[n] = __float_as_uint(__uint_as_float(ov[n]) * factor[n]);
            tc::tmem_st16(tmem + lane_addr + kTmemO + grp * kRows, ov);
            tc::tmem_st_wait();
          }
        }
        // weights: this slot's column of P^T, after the product that last read the buffer
        if (c >= 2) ok = warp_wait(&sh.pv_done[grp][b], use - 1, abort_flag) && ok;
        uint8_t* pc = sP + (grp * 2 + b) * 2 * kPiece + (kl & 15);
        const int chunk = kl >> 4;
#pragma unroll
        for (int n = 0; n < kRows; n += 2) {
          const float p0 = z[n] == -INFINITY ? 0.f : ex2(z[n]);
          const float p1 = z[n + 1] == -INFINITY ? 0.f : ex2(z[n + 1]);
          lsum[n] = fmaf(p0, iv, lsum[n]);
          lsum[n + 1] = fmaf(p1, iv, lsum[n + 1]);
          uint32_t hi, lo;
          split_p2(p0, p1, hi, lo);
          const int o0 = (n >> 3) * 1024 + (n & 7) * 128 + ((chunk ^ (n & 7)) << 4);
          const int o1 = (n >> 3) * 1024 + ((n & 7) + 1) * 128 + ((chunk ^ ((n & 7) + 1)) << 4);
          pc[o0] = uint8_t(hi);
          pc[o1] = uint8_t(hi >> 8);
          pc[kPiece + o0] = uint8_t(lo);
          pc[kPiece + o1] = uint8_t(lo >> 8);
        }
        // the unit's last tile: stale V rows past the end (NaN codes) times zero must stay zero
        if ((it.j0 + i) * kBN + kBN > kv_len) {
          const int st = kg % kVStages;
          ok = warp_wait(&sh.v_full[st], kg / kVStages, abort_flag) && ok;
          if (key >= kv_len) {
            uint4* row = reinterpret_cast<uint4*>(sV + st * kTile + kl * 128);
#pragma unroll
            for (int x = 0; x < 8; ++x) row[x] = make_uint4(0, 0, 0, 0);
          }
        }
        tc::fence_proxy_async_smem();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sh.p_full[grp][b]);
        if (grp) ++cnt[1];
        else ++cnt[0];
      }
      // the other group's tiles of the item
      if (grp) cnt[0] += (nt + 1) >> 1;
      else cnt[1] += nt >> 1;
      // join: row sums over lanes and warps, references of both groups
      const float total = reduce16<false>(lsum, lane);
      if (!(lane & 1)) sh.sum[li & 1][grp][q][row16(lane)] = total;
      if (q == 0 && lane == 0) {
#pragma unroll
        for (int n = 0; n < kRows; ++n) sh.add[li & 1][grp][n] = add[n];
      }
      bar_sync(3, 256);
      uint32_t o0[kRows], o1[kRows];
      ok = warp_wait(&sh.pv_done[0][(cnt[0] - 1) & 1], (cnt[0] - 1) >> 1, abort_flag) && ok;
      if (nt > 1) ok = warp_wait(&sh.pv_done[1][(cnt[1] - 1) & 1], (cnt[1] - 1) >> 1, abort_flag) && ok;
      tc::tc_fence_after();
      tc::tmem_ld16(tmem + lane_addr + kTmemO, o0);
      tc::tmem_ld16(tmem + lane_addr + kTmemO + kRows, o1);
      tc::tmem_ld_wait();
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(&sh.q_empty[li & 1]);
        tc::mbar_arrive(&sh.o_free[0]);
        tc::mbar_arrive(&sh.o_free[1]);
      }
#pragma unroll
      for (int n = 0; n < kRows; ++n) {
        if ((n & 1) != grp || n >= nrows) continue;   // each group writes every other row
        const float a0 = sh.add[li & 1][0][n], a1 = sh.add[li & 1][1][n];
        const float top = fminf(a0, a1);              // of the larger reference
        const float w0 = a0 == INFINITY ? 0.f : ex2(top - a0);
        const float w1 = a1 == INFINITY ? 0.f : ex2(top - a1);
        float l0 = 0.f, l1 = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          l0 += sh.sum[li & 1][0][w][n];
          l1 += sh.sum[li & 1][1][w][n];
        }
        const float l = l0 * w0 + l1 * w1;
        const float inv = l > 0.f ? 1.f / l : 0.f;
        // an accumulator that took no product in this item holds the one before's
        float v = w0 > 0.f ? __uint_as_float(o0[n]) * w0 : 0.f;
        if (w1 > 0.f) v = fmaf(__uint_as_float(o1[n]), w1, v);
        v = l > 0.f ? v * inv : 0.f;
        const float lse2 = l > 0.f ? log2f(l) - top : -INFINITY;
        const int t = n / a.G, g = n - t * a.G;
        if (it.slot < 0) {
          const size_t row = size_t(o + t) * a.H_q + it.h * a.G + g;
          static_cast<__nv_bfloat16*>(a.o)[row * kD + kl] = __float2bfloat16_rn(v);
          if (q == 0 && lane == 0 && a.lse) a.lse[row] = lse2 * 0.6931471805599453f;
        } else {
          const size_t row = size_t(it.slot) * d.part_rows + n;
          d.part_o[row * kD + kl] = v;
          if (q == 0 && lane == 0) d.part_lse[row] = lse2;
        }
      }
      kt += nt;
    }
    if (!ok) *abort_flag = 1;
  }
  tc::tc_fence_before();
  __syncthreads();
  if (*abort_flag && tid == 0) {
    ItemIter iter;
    iter.start(d, R);
    Item it;
    while (iter.next(d, R, it)) atomicOr(&a.req_status[it.r], SPEC_REQ_TIMEOUT);
  }
  tc::tc_fence_after();
  if (warp == 0) tc::tmem_dealloc(tmem, kTmemCols);
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
  for (int p0 = 0; p0 < rec.np; p0 += 4) {
    float ls[4];
    float4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int p = p0 + u;
      ls[u] = -INFINITY;
      v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (p < rec.np) {
        const size_t row = size_t(p == 0 ? rec.slot0 : 2 * (rec.ca + p)) * d.part_rows + m;
        ls[u] = d.part_lse[row];
        v[u] = reinterpret_cast<const float4*>(d.part_o + row * kD)[lane];
      }
    }
    float top = M;
#pragma unroll
    for (int u = 0; u < 4; ++u) top = fmaxf(top, ls[u]);
    if (top == -INFINITY) continue;
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
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  const size_t row = size_t(rec.o + t) * a.H_q + rec.h * a.G + g;
  __nv_bfloat162 lo = __floats2bfloat162_rn(acc[0] * inv, acc[1] * inv);
  __nv_bfloat162 hi = __floats2bfloat162_rn(acc[2] * inv, acc[3] * inv);
  uint2 w;
  w.x = *reinterpret_cast<uint32_t*>(&lo);
  w.y = *reinterpret_cast<uint32_t*>(&hi);
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + row * kD + 4 * lane) = w;
  if (lane == 0 && a.lse)
    a.lse[row] = sum > 0.f ? (M + log2f(sum)) * 0.6931471805599453f : -INFINITY;
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

static int rows_of(const AttnKv8Dev& a) { return r16::kRows; }

static int device_ctas() {
  const int sms = sm_count_current_device();
  return sms < kMaxCtas ? sms : kMaxCtas;
}

}  // namespace kv8tc

// Whether the tensor-core kernels take this call.
bool attn_kv8_tc_takes(const AttnKv8Dev& a, bool bf16) {
  return bf16 && a.d == 128 && (a.bs == 16 || a.bs == 32 || a.bs == 64 || a.bs == 128) &&
         a.G <= 16 && (long long)a.T_max * a.G <= 16 &&
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
  d.min_tiles = 2;
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
  static DeviceOnce raised16;
  spec_status_t st = raise_dyn_smem_once(attn_kv8_rows16_kernel, r16::kSmemBytes, raised16);
  if (st != SPEC_OK) return st;
  cudaError_t e = launch_pdl(attn_kv8_rows16_kernel, dim3(ctas), dim3(r16::kThreads),
                             size_t(r16::kSmemBytes), s, mK, mV, mKw, mVw, d);
  if (e == cudaSuccess)
    e = launch_pdl(attn_kv8_join_kernel, dim3(ctas, (d.part_rows + 7) / 8), dim3(256), 0, s, d);
  return launch_result(e);
}

}  // namespace spec
