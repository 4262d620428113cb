// The partition of spec_tree_attention_kv8's work over persistent CTAs, the page copies and the
// tensor-core forms that its kernels share.
//
// Work unit = (request r, KV head h, tile of query rows); its K/V is read in tiles of 128 slots.
// The units are laid end to end (request, head, row tile) as one stream of K/V tiles that is cut
// into equal contiguous ranges, one per CTA.  A unit cut by a range boundary is computed in
// pieces: each writes its normalised output and log-sum-exp, and the CTA holding the first piece
// leaves a record from which a second launch joins them.
// Where requests have several row tiles, CTAs work in pairs (`pair`): a stream element is two
// units, one for each CTA of the pair -- two row tiles of one head, which read the same K/V tiles
// at the same pace, so that the second reader finds them in L2; or, of an odd last row tile, two
// heads.  (Without the pairs the row tiles' passes over a long cache lie too far apart for L2, and
// K and V come from HBM once a row tile: 64 ragged trees, 432 rows a head, 1376 us with, 1437
// without.)
//
// K's codes go to tcgen05.mma kind::f8f6f4 as they are.  A bf16 query keeps its precision as the sum of
// two 8-bit pieces, both multiplied into the same fp32 accumulator: e4m3(x) + e4m3(x - e4m3(x)), exact
// (4 + 4 significant bits) but for elements 2^-18 of the row's largest.  fp8 products run at twice the
// bf16 rate, so the two pieces cost what one bf16 product does.
// V's codes go there as they are too in the kernel of short units, against weights that are the sum of
// three e5m2 pieces (split_p2), 10 bits over 22 binades and 2^-17 of the range below: V is read where
// TMA put it, one byte an element; converting it first would move 6 bytes of shared memory an element
// against 2, more than the SM has at HBM speed.  The kernel of long units, whose tiles take several
// times as long as HBM needs for them, converts V to fp16 for weights in fp16.
#pragma once

#include <cudaTypedefs.h>

#include "attention_kv8.cuh"
#include "tc_ptx.cuh"

namespace spec {
namespace kv8tc {

constexpr int kD = 128;
constexpr int kBN = 128;                          // slots of a K/V tile
constexpr int kTile = kBN * kD;                   // bytes
constexpr long long kWaitLimit = 4000000000LL;    // clock cycles (~2 s)
constexpr int kMaxCtas = 1024;
// Weights enter the products as 2^(y - ref + kShift); the reference, a maximum seen before, moves
// when a y passes it by more than 2, so that they stay below 2^15 <= 57344 and a row's largest is at
// least 2^kShift.  Two binades of slack: with one, the chains' units spent more on moving
// references than on weights.
constexpr float kShift = 13.f;
constexpr float kCeil = 15.f;
// Row sums are kept times 2^-kSumShift: of weights up to 2^15 over V scales down to 2^-100, a million
// keys' sum stays finite.
constexpr float kSumShift = 10.f;
constexpr float kSumMul = 1.f / 1024.f;
constexpr float kMinVScale = 7.888609052210118e-31f;   // 2^-100

struct MergeRec {
  int np, h, mt, o, T, slot0;
};

struct TcDev {
  AttnKv8Dev a;
  int tpt;              // tree tokens of a row tile
  int log2bs;
  int kv_rows;          // a row past the cache: TMA fills zeros there
  int ctas, min_tiles;
  int pair;             // 1: CTAs 2 c, 2 c + 1 share range c
  int part_rows;        // rows of a piece
  MergeRec* recs;       // [ctas]
  float* part_o;        // [2 ctas][part_rows][128]
  float* part_lse;      // [2 ctas][part_rows], log2
};

struct ReqGeom {
  int o, T, P, mts, nts, units;
};
__device__ __forceinline__ ReqGeom req_geom(const TcDev& d, int r) {
  ReqGeom g;
  g.o = d.a.node_offset[r];
  g.T = d.a.node_offset[r + 1] - g.o;
  g.P = d.a.prefix_len[r];
  const bool ok = kv8_live(d.a, r, g.T, g.P) == Kv8Live::yes && g.o >= 0 && g.o + g.T <= d.a.N;
  g.mts = ok ? (g.T + d.tpt - 1) / d.tpt : 0;
  g.nts = ok ? (g.P + g.T + kBN - 1) / kBN : 0;
  g.units = d.pair ? d.a.H_kv * (g.mts >> 1) + (g.mts & 1) * ((d.a.H_kv + 1) >> 1)
                   : d.a.H_kv * g.mts;
  return g;
}
// This CTA's range and its place in it.
__device__ __forceinline__ int range_id(const TcDev& d) { return int(blockIdx.x) >> d.pair; }
// Head and row tile of the u-th stream element for this CTA; h = H_kv: none.
__device__ __forceinline__ void unit_of(const TcDev& d, const ReqGeom& g, int u, int& h, int& mt) {
  if (!d.pair) {
    h = u / g.mts;
    mt = u - h * g.mts;
    return;
  }
  const int rank = blockIdx.x & 1, twos = g.mts >> 1, whole = d.a.H_kv * twos;
  if (u < whole) {
    h = u / twos;
    mt = 2 * (u - h * twos) + rank;
  } else {
    h = min(2 * (u - whole) + rank, d.a.H_kv);
    mt = g.mts - 1;
  }
}

// `total` tiles in C ranges, the first `rem` of them one tile longer than `quot`
struct Cut {
  long long quot;
  int rem;
};
struct Range {
  long long total, t0, t1;   // tiles of the stream; this CTA's
  int C;                     // ranges
  Cut cut;
  int r0, r1;                // requests holding tiles t0 and t1 - 1
  long long rbeg0, rbeg1;    // their first tiles
};
// quotient of a 64-bit count, which fits 32 bits but in absurd calls
__device__ __noinline__ long long div64(long long n, long long m) { return n / m; }
__device__ __forceinline__ long long div_count(long long n, long long m) {
  return (n | m) >> 31 ? div64(n, m) : (long long)(uint32_t(n) / uint32_t(m));
}
__device__ __forceinline__ Cut make_cut(long long total, int C) {
  Cut k;
  k.quot = div_count(total, C);
  k.rem = int(total - k.quot * C);
  return k;
}
__device__ __forceinline__ long long range_start(const Cut& k, int c) {
  return k.quot * c + min(c, k.rem);
}
__device__ __forceinline__ int range_of(const Cut& k, long long t) {
  const long long longer = (k.quot + 1) * k.rem;
  return t < longer ? int(div_count(t, k.quot + 1)) : k.rem + int(div_count(t - longer, k.quot));
}

// The walking warp's range (every lane gets it): pass 1 sums the requests' tiles, pass 2 scans them
// for the requests that hold the range's ends.  The first kHeld requests' counts stay in registers.
__device__ __forceinline__ Range warp_range(const TcDev& d) {
  constexpr int kHeld = 2;           // chunks of 32 requests
  const int lane = threadIdx.x & 31;
  auto tiles_of = [&](int r) -> long long {
    if (r >= d.a.B) return 0;
    const ReqGeom g = req_geom(d, r);
    if (blockIdx.x == 0 && g.units == 0 && kv8_live(d.a, r, g.T, g.P) == Kv8Live::beyond_table)
      atomicOr(&d.a.req_status[r], SPEC_REQ_BAD_BLOCK);
    return (long long)g.units * g.nts;
  };
  long long held[kHeld], total = 0;
#pragma unroll
  for (int c = 0; c < kHeld; ++c) {
    held[c] = tiles_of(c * 32 + lane);
    total += held[c];
  }
#pragma unroll 2
  for (int r = kHeld * 32 + lane; r < d.a.B; r += 32) total += tiles_of(r);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  Range R;
  R.total = total;
  R.C = int(max(1LL, min((long long)(d.ctas >> d.pair), div_count(total, d.min_tiles))));
  R.cut = make_cut(total, R.C);
  R.t0 = R.t1 = 0;
  R.r0 = R.r1 = 0;
  R.rbeg0 = R.rbeg1 = 0;
  const int id = range_id(d);
  if (total == 0 || id >= R.C) return R;
  R.t0 = range_start(R.cut, id);
  R.t1 = range_start(R.cut, id + 1);
  long long base = 0;
#pragma unroll 1
  for (int c = 0; c * 32 < d.a.B; ++c) {
    const int r = c * 32 + lane;
    long long n = 0;
#pragma unroll
    for (int k = 0; k < kHeld; ++k) n = c == k ? held[k] : n;
    if (c >= kHeld) n = tiles_of(r);
    long long hi = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, hi, o);
      if (lane >= o) hi += x;
    }
    hi += base;
    const long long lo = hi - n;
    const uint32_t m0 = __ballot_sync(0xffffffffu, n > 0 && lo <= R.t0 && R.t0 < hi);
    const uint32_t m1 = __ballot_sync(0xffffffffu, n > 0 && lo <= R.t1 - 1 && R.t1 - 1 < hi);
    if (m0) {
      R.r0 = c * 32 + __ffs(m0) - 1;
      R.rbeg0 = __shfl_sync(0xffffffffu, lo, __ffs(m0) - 1);
    }
    if (m1) {
      R.r1 = c * 32 + __ffs(m1) - 1;
      R.rbeg1 = __shfl_sync(0xffffffffu, lo, __ffs(m1) - 1);
      break;
    }
    base = __shfl_sync(0xffffffffu, hi, 31);
  }
  return R;
}

// Tiles [j0, j1) of unit (r, h, row tile mt).
struct Item {
  int r, h, mt, j0, j1;
  int slot;               // >= 0: a piece of a cut unit, written to part_o[slot]
  int o, T, P;
};
struct ItemIter {
  long long t, rbeg, rend;
  int r;
  ReqGeom g;
  __device__ __forceinline__ void start(const TcDev& d, const Range& R) {
    t = R.t0;
    r = R.r0;
    rbeg = rend = R.rbeg0;
    if (t < R.t1) {
      g = req_geom(d, r);
      rend = rbeg + (long long)g.units * g.nts;
    }
  }
  __device__ __forceinline__ bool next(const TcDev& d, const Range& R, Item& it) {
#pragma unroll 1
    while (t < R.t1) {
#pragma unroll 1
      while (t >= rend) {
        if (r + 1 >= d.a.B) return false;
        ++r;
        g = req_geom(d, r);
        rbeg = rend;
        rend = rbeg + (long long)g.units * g.nts;
      }
      const long long off = t - rbeg;
      const int u = int(div_count(off, g.nts));
      it.r = r;
      unit_of(d, g, u, it.h, it.mt);
      it.j0 = int(off - (long long)u * g.nts);
      it.j1 = int(min((long long)g.nts, (long long)it.j0 + (R.t1 - t)));
      it.o = g.o;
      it.T = g.T;
      it.P = g.P;
      const bool partial = it.j0 > 0 || it.j1 < g.nts;
      it.slot = partial ? (t == R.t0 ? 2 * int(blockIdx.x) : 2 * int(blockIdx.x) + 1) : -1;
      t += it.j1 - it.j0;
      if (it.h < d.a.H_kv) return true;
    }
    return false;
  }
};

// One lane walks the range and hands the items to the other roles through a ring in shared memory,
// so that the loads and divisions of the walk are done once and ahead of time (each role walking
// for itself made the kernel 137 KB of instructions, more than the instruction cache holds: every
// unit began with a few microseconds of misses).  r < 0 ends the stream.
constexpr int kItemRing = 4;
struct ItemRing {
  uint64_t full[kItemRing], empty[kItemRing];
  Item item[kItemRing];
};

// One lane of each CTA: the record of its unit of the range's last tile, if that unit starts in
// this range and continues past it.  Piece p > 0 starts range id + p: slot 2 (CTA + (p << pair)).
__device__ __forceinline__ void write_merge_record(const TcDev& d, const Range& R) {
  MergeRec rec;
  rec.np = rec.h = rec.mt = rec.o = rec.T = rec.slot0 = 0;
  if (R.t0 < R.t1) {
    const ReqGeom g = req_geom(d, R.r1);
    const int u = int(div_count(R.t1 - 1 - R.rbeg1, g.nts));
    const long long ubeg = R.rbeg1 + (long long)u * g.nts;
    unit_of(d, g, u, rec.h, rec.mt);
    if (ubeg >= R.t0 && ubeg + g.nts > R.t1 && rec.h < d.a.H_kv) {
      rec.np = range_of(R.cut, ubeg + g.nts - 1) - range_id(d) + 1;
      rec.o = g.o;
      rec.T = g.T;
      rec.slot0 = 2 * int(blockIdx.x) + (ubeg > R.t0 ? 1 : 0);
    }
  }
  d.recs[blockIdx.x] = rec;
}

// ------------------------------------------------------------------------------ waits
// One look at a barrier's phase that lets the hardware suspend the thread for up to ~20 us: a
// waiting warp leaves its issue slots to the others.  (Polling took a quarter of all instructions.)
__device__ __forceinline__ bool try_wait_suspended(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok) : "r"(tc::smem_u32(bar)), "r"(parity), "r"(20000u) : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool wait1(uint64_t* bar, int parity, volatile int* abort) {
  if (tc::mbar_try_wait(bar, uint32_t(parity & 1))) return true;
  const long long t0 = clock64();
#pragma unroll 1
  while (!try_wait_suspended(bar, uint32_t(parity & 1)))
    if (*abort || clock64() - t0 > kWaitLimit) return false;
  return true;
}
// one lane waits, the warp gets the outcome
__device__ __forceinline__ bool lane0_wait(uint64_t* bar, int parity, volatile int* abort) {
  bool r = true;
  if ((threadIdx.x & 31) == 0) r = wait1(bar, parity, abort);
  return __shfl_sync(0xffffffffu, r ? 1 : 0, 0) != 0;
}

// ------------------------------------------------------------------------------ items
// the walking lane
__device__ __forceinline__ void item_producer(const TcDev& d, const Range& R, ItemRing& ring,
                                              volatile int* abort) {
  ItemIter iter;
  iter.start(d, R);
  Item it;
  bool more = true;
#pragma unroll 1
  for (int li = 0; more; ++li) {
    more = iter.next(d, R, it);
    if (!more) it.r = -1;
    const int s = li % kItemRing;
    if (li >= kItemRing && !wait1(&ring.empty[s], li / kItemRing - 1, abort)) return;
    ring.item[s] = it;
    tc::mbar_arrive(&ring.full[s]);
  }
}
// The li-th item, for every lane of a warp; false at the end of the stream or on an expired wait.
// `arrivals` of the ring's empty barrier: one a warp.
__device__ __forceinline__ bool next_item(ItemRing& ring, int li, Item& it, volatile int* abort) {
  const int s = li % kItemRing;
  const bool ok = wait1(&ring.full[s], li / kItemRing, abort);
  it = ring.item[s];
  __syncwarp();
  if ((threadIdx.x & 31) == 0) tc::mbar_arrive(&ring.empty[s]);
  return ok && it.r >= 0;
}

// ------------------------------------------------------------------------------ page copies
// One warp brings the K (or V) tiles of the CTA's items into a ring of stages.  Lanes below
// 128 / bs hold the tile's page ids, fetched a tile ahead; consecutive pages come as one 16 KB
// box, others as a box each.  Pages past the request or with a bad id are read from a row past
// the cache, which TMA fills with zeros.  Every copy issued is waited for before return.
__device__ __forceinline__ void page_producer(const TcDev& d, ItemRing& items,
                                              const CUtensorMap* map, const CUtensorMap* wide,
                                              int nstage, uint8_t* ring, uint64_t* full,
                                              uint64_t* empty, bool flag_bad, int* abort_flag) {
  const int lane = threadIdx.x & 31;
  const int bs = d.a.bs, ppt = kBN >> d.log2bs, page_bytes = bs * kD;
  int st = 0, use = 0, issued = 0;         // the stage and how often the ring has gone round
  bool ok = true;
  Item it;
#pragma unroll 1
  for (int li = 0; ok && __all_sync(0xffffffffu, next_item(items, li, it, abort_flag)); ++li) {
    const int nblk = (it.P + it.T + bs - 1) >> d.log2bs;
    const int32_t* table = d.a.block_table + size_t(it.r) * d.a.max_blocks;
    auto page_of = [&](int j) -> int {     // -1: past the request or the item
      const int lb = j * ppt + lane;
      return lane < ppt && j < it.j1 && lb < nblk ? __ldg(table + lb) : -1;
    };
    int cur = page_of(it.j0), next = page_of(it.j0 + 1);
#pragma unroll 1
    for (int j = it.j0; j < it.j1; ++j) {
      const int after = page_of(j + 2);
      if (use > 0 && !lane0_wait(empty + st, use - 1, abort_flag)) {
        ok = false;
        break;
      }
      const bool good = cur >= 0 && cur < d.a.num_blocks;
      if (flag_bad && !good && lane < ppt && j * ppt + lane < nblk)
        atomicOr(&d.a.req_status[it.r], SPEC_REQ_BAD_BLOCK);
      const int first = __shfl_sync(0xffffffffu, cur, 0);
      const bool run = __all_sync(0xffffffffu, lane >= ppt || (good && cur == first + lane));
      if (lane == 0) tc::mbar_arrive_expect_tx(full + st, kTile);
      __syncwarp();
      uint8_t* dst = ring + st * kTile;
      if (run) {
        if (lane == 0) tc::tma_load_4d(dst, wide, 0, 0, it.h, first, full + st);
      } else if (lane < ppt) {
        const int row = good ? (cur * d.a.H_kv + it.h) * bs : d.kv_rows;
        tc::tma_load_2d(dst + lane * page_bytes, map, 0, row, full + st);
      }
      __syncwarp();
      cur = next;
      next = after;
      ++issued;
      if (++st == nstage) {
        st = 0;
        ++use;
      }
    }
  }
  if (lane == 0) {
    if (!ok) *reinterpret_cast<volatile int*>(abort_flag) = 1;
    // the copies of the last round: `st` and after belong to the round before
    const int n = min(issued, nstage);
#pragma unroll 1
    for (int k = 1; k <= n; ++k) {
      const int s = st - k < 0 ? st - k + nstage : st - k;
      const int u = st - k < 0 ? use - 1 : use;
      tc::mbar_wait(full + s, u & 1, abort_flag, kWaitLimit / 8);
    }
  }
  __syncwarp();
}

// The scales of each tile's pages into a ring: k[i] = K scale, v[i] = V scale, lv[i] its log2, iv[i] its
// reciprocal (times kSumMul), i < 128 / bs.  One warp, four tiles at a time (lanes 8 u .. 8 u + 7: tile u), far
// enough ahead of the softmax to hide its dependent loads.
struct ScaleSlot {
  float k[8], v[8], lv[8], iv[8];
};
constexpr int kScaleRing = 16;
__device__ __forceinline__ void scale_producer(const TcDev& d, ItemRing& items, ScaleSlot* ring,
                                               uint64_t* full, uint64_t* empty, int* abort_flag) {
  const int lane = threadIdx.x & 31;
  const int ppt = kBN >> d.log2bs, i = lane & 7, sub = lane >> 3;
  int kt = 0;
  bool ok = true;
  Item it;
#pragma unroll 1
  for (int li = 0; ok && __all_sync(0xffffffffu, next_item(items, li, it, abort_flag)); ++li) {
    const int nblk = (it.P + it.T + d.a.bs - 1) >> d.log2bs;
    const int32_t* table = d.a.block_table + size_t(it.r) * d.a.max_blocks;
    auto page_of = [&](int j) -> int {
      const int lb = (j + sub) * ppt + i;
      int pb = -1;
      if (i < ppt && j + sub < it.j1 && lb < nblk) pb = table[lb];
      return pb >= 0 && pb < d.a.num_blocks ? pb : -1;
    };
    // the scales of the four tiles ahead and the page ids of the four after those are in flight
    float ks_n, vs_n;
    auto scales_of = [&](int pb) {
      ks_n = vs_n = 0.f;
      if (pb >= 0) {
        ks_n = d.a.k_scale[size_t(pb) * d.a.H_kv + it.h];
        vs_n = d.a.v_scale[size_t(pb) * d.a.H_kv + it.h];
      }
    };
    scales_of(page_of(it.j0));
    int ahead = page_of(it.j0 + 4);
#pragma unroll 1
    for (int j = it.j0; j < it.j1; j += 4) {
      const float ks = ks_n;
      float vs = vs_n;
      scales_of(ahead);
      ahead = page_of(j + 8);
      const int n = min(4, it.j1 - j);
#pragma unroll 1
      for (int u = 0; u < n; ++u) {
        const int use = (kt + u) / kScaleRing;
        if (use > 0 && !lane0_wait(empty + (kt + u) % kScaleRing, use - 1, abort_flag)) ok = false;
      }
      if (!ok) break;
      if (sub < n) {
        ScaleSlot* o = ring + (kt + sub) % kScaleRing;
        // a V scale of 0 (a block of zeros) has no logarithm
        vs = fmaxf(vs, kMinVScale);
        o->k[i] = ks;
        o->v[i] = vs;
        o->iv[i] = kSumMul / vs;
        o->lv[i] = log2f(vs);
      }
      __syncwarp();
      if (lane < n) tc::mbar_arrive(full + (kt + lane) % kScaleRing);
      kt += n;
    }
  }
  if (lane == 0 && !ok) *reinterpret_cast<volatile int*>(abort_flag) = 1;
  __syncwarp();
}

// ------------------------------------------------------------------------------ number forms
// eight bf16 query elements, scaled, as two pieces of eight e4m3 codes each
__device__ __forceinline__ void split_q8(const uint4& w, float inv, uint2& hi, uint2& lo) {
  float f[8];
  elem<__nv_bfloat16>::unpack(w, f);
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] *= inv;
  hi.x = kv8::pack_e4m3x4(f[0], f[1], f[2], f[3]);
  hi.y = kv8::pack_e4m3x4(f[4], f[5], f[6], f[7]);
  float b[4];
  kv8::unpack_e4m3x4(hi.x, b);
  lo.x = kv8::pack_e4m3x4(f[0] - b[0], f[1] - b[1], f[2] - b[2], f[3] - b[3]);
  kv8::unpack_e4m3x4(hi.y, b);
  lo.y = kv8::pack_e4m3x4(f[4] - b[0], f[5] - b[1], f[6] - b[2], f[7] - b[3]);
}
// Softmax weights as three e5m2 pieces of their fp16 value, hi + mid + lo.  An e5m2 code is the upper
// byte of an fp16: a rounding add and a mask give a piece, and the subtractions are exact.  hi is
// rounded to nearest (within 2^-3 of the weight), mid cut off (2^-2 of what is left; a NaN stays one
// there), lo to nearest (2^-3 of the rest): over all fp16 values the sum is within 2^-10 of a weight
// of at least 2^-7 and within 2^-17 of a smaller one.  (Pieces with more bits and less range, e4m3, lose
// the weights below 2^-16 of a row's largest: of one key with most of the weight before a long flat
// rest, the rest.)
struct Split2 {
  uint32_t hi, mid, lo;   // two weights: the codes are bytes 1 and 3
};
__device__ __forceinline__ Split2 split_p2(float a, float b) {
  Split2 s;
  asm("{\n\t.reg .b32 w, r;\n\t"
      "cvt.rn.f16x2.f32 w, %4, %3;\n\t"
      "add.u32 %0, w, 0x00800080;\n\tand.b32 %0, %0, 0xFF00FF00;\n\t"
      "sub.rn.f16x2 r, w, %0;\n\t"
      "and.b32 %1, r, 0xFF00FF00;\n\t"
      "sub.rn.f16x2 r, r, %1;\n\t"
      "add.u32 %2, r, 0x00800080;\n\t}"
      : "=&r"(s.hi), "=&r"(s.mid), "=&r"(s.lo) : "f"(a), "f"(b));
  return s;
}
// two weights in fp16
__device__ __forceinline__ uint32_t pack_f16x2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(a), "f"(b));
  return r;
}

// bit 7 of each byte of w that holds e4m3's NaN (0x7F, 0xFF)
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

// 32 lanes x 8 consecutive 32-bit columns
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
        "r"(r[7])
      : "memory");
}

// one lane of a converged warp, the same each time
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(p));
  return p != 0;
}

// D[tmem] (+)= A[smem] * B[smem], kind::f8f6f4 (e4m3 codes, fp32 accumulate), K = 32
__device__ __forceinline__ void mma_e4m3_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor of kind::f8f6f4: fp32 accumulator (bits 4-5 = 1), A and B e4m3 (both
// type fields 0), major-ness in bits 15 / 16 (1 = MN-major), N >> 3 in bits 17-22, M >> 4 in 24-28.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | (uint32_t(a_mn) << 15) | (uint32_t(b_mn) << 16) | (uint32_t(N >> 3) << 17) |
         (uint32_t(M >> 4) << 24);
}

constexpr uint32_t kIdescBE5m2 = 1u << 10;   // B's type field: e5m2

// Reductions of NR values a lane over the 32 lanes: each of the first exchanges halves what a lane
// holds, about NR shuffles instead of 5 NR.  Lane l ends with the result of row red_row<NR>(l).
template <int NR>
__device__ __forceinline__ int red_row(int lane) {
  int r = 0;
#pragma unroll
  for (int w = NR / 2, b = 16; w >= 1; w /= 2, b /= 2) r += (lane & b) ? w : 0;
  return r;
}
template <int NR, bool kMax>
__device__ __forceinline__ float red_rows(const float (&v)[NR], int lane) {
  auto op = [](float x, float y) { return kMax ? fmaxf(x, y) : x + y; };
  float a[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) a[i] = v[i];
  int b = 16;
#pragma unroll
  for (int w = NR / 2; w >= 1; w /= 2, b /= 2) {
    const bool up = lane & b;
#pragma unroll
    for (int i = 0; i < w; ++i) {
      const float keep = up ? a[i + w] : a[i], send = up ? a[i] : a[i + w];
      a[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, b));
    }
  }
#pragma unroll 1
  for (; b >= 1; b /= 2) a[0] = op(a[0], __shfl_xor_sync(0xffffffffu, a[0], b));
  return a[0];
}

// OR of a predicate over the `n` threads of named barrier `id`
__device__ __forceinline__ bool bar_any(int id, int n, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\t"
      "setp.ne.u32 a, %3, 0;\n\t"
      "barrier.cta.red.or.pred b, %1, %2, a;\n\t"
      "selp.u32 %0, 1, 0, b;\n\t}"
      : "=r"(r) : "r"(id), "r"(n), "r"(p ? 1u : 0u) : "memory");
  return r != 0;
}
__device__ __forceinline__ void bar_sync(int id, int n) {
  asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}

}  // namespace kv8tc
}  // namespace spec
