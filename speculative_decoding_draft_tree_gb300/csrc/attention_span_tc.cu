// spec_tree_attention_shared and spec_tree_attention_window on the tcgen05 tensor cores: bf16, head_dim 128.
//
// A unit is one or two tiles of 128 query rows (G heads x 128 / G tokens) under a KV head; the rows of a
// group's members lie in one unit, which is what a shared prefix gains: its keys and values meet full
// tiles, and are read once for 256 rows.  Tiles are 128 x 128 in S = Q K^T and O += P V; per row tile and
// key tile the two products take 1024 clocks of the tensor pipe (8192 flop a clock and SM), the
// exponentials 512 of theirs at 32 results a clock, and the operands' reads from shared memory 768 (Q and K
// for S, V alone for O since P is read from TMEM).  So two row tiles ("slots") alternate: while the
// products of one run, the other's softmax does.
//   pair unit  slot s has row tile s of a head, both read every key tile;
//   dual unit  slot s has a row tile of head h + s and key tiles of its own: for tiles of few rows, whose start,
//              join and end are most of their time and are shared so;
//   lone unit  the slots take the key tiles in turn, and the epilogue joins their halves.
// CTA (384 threads):
//   warp 0  Q and K by TMA (two stages of K), warp 2 V (two stages): 128-byte-swizzled boxes of a page,
//           or of all of a tile's pages when they follow one another; pages that no row sees come as zeros;
//   warp 1  one elected thread issues PV_0(k) QK_0(k+1) PV_1(k) QK_1(k+1) ..; P_s lies over S_s in TMEM, which
//           the issue order protects; a pair's PV starts on the first 64 keys while the softmax writes the rest;
//   warp 3  walks the CTA's range and hands the items to the others through a ring;
//   warps 4-7 and 8-11  softmax of slot 0 and 1, a row per thread, a pair unit's with all 128 scores in
//           registers; the reference moves when the maximum has grown by more than 2^8, and only then is O
//           rescaled.
// The product wants P in V's type.  A pair unit's weights are rounded to bf16 once (error of the output against
// 64 bits 0.0021 .. 0.0023 of it, 0.0017 being its own rounding's); the others' have the room for a second piece, what
// that rounding left (0.0017).  The sum takes the unrounded weights.
// A weight is 2 to a fused product less the reference, which was rounded for itself.  From references of 2^30 on
// that difference can leave fp32's range of exponents for the key that the reference came from; such a row's products are
// rounded first, by a function of its own that works in TMEM (8 groups of 8 samples 84.1 us, 83.3 without it; in line 85.6).
//
// Bound, for long pair units, by the chain of a slot: products 1024 clocks, loads of S and maxima 420, weights 800,
// waits; ~2650 clocks a key tile against 2048 of products alone (32 trees over 8192 shared slots: 169 us, and
// 191 with the issuing thread's code unrolled for each slot, which took 1430 clocks a slot to get through, and
// ranges cut without regard to masked tiles).  Short units are bound by what happens once in each: see the
// costs in attention_span.cu.
//
// Masked tiles (a window's edges, a tree, a last tile): masked scores become -inf before anything is
// formed from them.  Of V, whose product with a weight of zero would be NaN, the softmax warps look at the
// tile in shared memory first: rows that no query row sees are cleared, infinities and NaN elsewhere are
// taken out, and the scores of the rows that see their key become NaN.
//
// Waits are bounded; one that runs out raises the CTA's abort flag, every role leaves, TMEM is freed, and
// the requests of the CTA's range get SPEC_REQ_TIMEOUT.
#include <cudaTypedefs.h>
#include <math.h>

#include <mutex>

#include "attention_span.cuh"
#include "tc_ptx.cuh"

namespace spec {
namespace span {

constexpr int kD = 128;
constexpr int kRows = 128;                    // rows of an MMA tile
constexpr int kKeys = 128;
constexpr int kThreads = 384;
constexpr int kAtom = 16384;                  // 128 rows x 128 B
constexpr int kTile = 2 * kAtom;
constexpr int kKStages = 2;
constexpr int kVStages = 2;
constexpr int kItems = 4;                     // item ring
constexpr int kSmemK = 2 * kTile;             // Q: one tile per slot
constexpr int kSmemV = kSmemK + kKStages * kTile;
constexpr int kSmemOut = kSmemV + kVStages * kTile;     // 4 KB a softmax warp: output rows on their way out
constexpr int kSmemCtl = kSmemOut + 8 * 4096;
constexpr int kCtlRegs = 96, kSoftmaxRegs = 200;   // setmaxnreg: warps 0-3, warps 4-11
static_assert(kCtlRegs * 128 + kSoftmaxRegs * 256 <= kThreads * 168, "register split fits the launch");
constexpr long long kWaitLimit = 4000000000LL;     // clock cycles (~2 s)
constexpr float kLazy = 8.0f;                      // log2 units
constexpr float kCoarse = 1073741824.0f;           // 2^30: references from here on, their last place is 64 and more

struct Control {
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[kKStages], k_empty[kKStages], v_full[kVStages], v_empty[kVStages];
  uint64_t s_full[2], p_half[2], p_full[2], o_full[2], o_free[2];
  uint64_t exchange[4], vfix[3];                   // vfix: slot 0, slot 1, both
  uint64_t item_full[kItems], item_empty[kItems], drain;
  Item item[kItems];
  Range range;
  Entry first;
  alignas(16) uint32_t vbad[2][2][4];                          // tile parity, slot, 32 keys each: V not finite
  uint32_t tmem;
  int abort;
  float row[2][2][kRows];                          // slot, (reference, sum)
};
constexpr int kSmemBytes = kSmemCtl + int(sizeof(Control));
static_assert(kSmemBytes <= 232448, "fits one CTA's shared memory");
static_assert(sizeof(RangeScratch) <= size_t(kSmemOut), "the search's scratch lies in the tiles");

// One lane waits (bounded), the warp gets the outcome.
__device__ __forceinline__ bool lane0_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  bool r = true;
  if ((threadIdx.x & 31) == 0) r = tc::mbar_wait(bar, parity, abort, kWaitLimit);
  return __shfl_sync(0xffffffffu, r ? 1 : 0, 0) != 0;
}
// all lanes wait; the outcome is uniform, so that warp-wide TMEM accesses are made by all or none
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  const bool ok = tc::mbar_wait(bar, parity, abort, kWaitLimit);
  return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(a), "f"(b));
  return r;
}
// maximum of 32 values by three-input maxima
__device__ __forceinline__ float max32(const uint32_t (&x)[32]) {
  float m[11];
#pragma unroll
  for (int c = 0; c < 10; ++c)
    m[c] = fmax3(__uint_as_float(x[3 * c]), __uint_as_float(x[3 * c + 1]), __uint_as_float(x[3 * c + 2]));
  m[10] = fmaxf(__uint_as_float(x[30]), __uint_as_float(x[31]));
  return fmaxf(fmax3(fmax3(m[0], m[1], m[2]), fmax3(m[3], m[4], m[5]), fmax3(m[6], m[7], m[8])),
               fmaxf(m[9], m[10]));
}
// 32 weights 2^(x sl + add), summed in pairs into `acc`, as 16 columns of bf16 pairs in TMEM at `dst`; with
// kTwo what the rounding left, rounded again, in the 16 columns behind
template <bool kTwo>
__device__ __forceinline__ void weights32(const uint32_t (&x)[32], uint64_t sl, uint64_t add, uint64_t& acc,
                                          uint32_t dst) {
  uint32_t hi[16], lo[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float y0, y1;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), sl, add), y0, y1);
    const float p0 = ex2(y0), p1 = ex2(y1);
    acc = f2_add(acc, f2_pack(p0, p1));
    hi[i] = pack_bf16(p0, p1);
    if constexpr (kTwo) lo[i] = pack_bf16(p0 - bf16_lo(hi[i]), p1 - bf16_hi(hi[i]));
  }
  tc::tmem_st16(dst, hi);
  if constexpr (kTwo) tc::tmem_st16(dst + 16, lo);
}

// true for one lane of the warp, which the compiler knows to be one (what a lane number would not tell it:
// the products' operands then stay in uniform registers, and eight of them go out in 130 clocks, not 1000)
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// bits 0 .. n - 1
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }
// keys lo .. hi - 1 as bits of the 32 keys from key0 on
__device__ __forceinline__ uint32_t keys_in(int key0, int lo, int hi) {
  return below(hi - key0) & ~below(lo - key0);
}
// What a query row sees of its request.
struct RowView {
  const uint32_t* anc;    // its W ancestor words, null: no tree
  int W, lo, P, end;      // prefix keys lo .. P - 1, tree keys P .. end - 1
  int sunk;               // window: prefix keys below
  int first, deep;        // window: ancestors of depths below `first` are out of it, below `deep` sinks
};

// The row's visible keys among the 32 from key0 on.  Not inlined: masked tiles are few, and the code of a
// tile has to stay in the instruction cache.
__device__ __noinline__ uint32_t visible32(const RowView& v, int key0) {
  uint32_t w = keys_in(key0, v.lo, v.P) | keys_in(key0, 0, v.sunk);
  const int pos = key0 - v.P;
  if (pos > -32 && pos < 32 * v.W && v.anc != nullptr) {
    const int wi = pos >= 0 ? (pos >> 5) : -1, sh = pos - 32 * wi;
    const uint32_t lo = wi >= 0 ? __ldg(v.anc + wi) : 0u;
    const uint32_t hi = (sh != 0 && wi + 1 < v.W) ? __ldg(v.anc + wi + 1) : 0u;
    uint32_t t = (sh == 0 ? lo : ((lo >> sh) | (hi << (32 - sh)))) & keys_in(key0, v.P, v.end);
    if (v.first > 0 && t) {       // of the row's ancestors, in order of depth, the last `window` and the sinks
      int k = 0;
      for (int i = 0; i < v.W && 32 * i < pos; ++i) k += __popc(__ldg(v.anc + i) & below(pos - 32 * i));
      uint32_t keep = 0;
      for (uint32_t x = t; x; ++k) {
        const uint32_t b = x & (0u - x);
        if (k >= v.first || k < v.deep) keep |= b;
        x ^= b;
      }
      t = keep;
    }
    w |= t;
  }
  return w;
}

// The warp's 128 scores in TMEM at `at`: hidden ones become -infinity, and those of rows with a coarse reference (`mine`)
// their exponents, the largest key's 0.
__device__ __noinline__ void coarse_exponents(uint32_t at, float sl2, float ref, bool mine, uint4 vis) {
#pragma unroll 1
  for (int c = 0; c < kKeys; c += 16) {
    uint32_t r[16];
    tc::tmem_ld16(at + c, r);
    tc::tmem_ld_wait();
    const uint32_t seen = (c < 32 ? vis.x : c < 64 ? vis.y : c < 96 ? vis.z : vis.w) >> (c & 16);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float x = __uint_as_float(r[i]), y = mine ? __fadd_rn(__fmul_rn(x, sl2), -ref) : x;
      r[i] = __float_as_uint((seen >> i) & 1u ? y : -INFINITY);
    }
    tc::tmem_st16(at + c, r);
  }
  tc::tmem_st_wait();
}

__global__ void __launch_bounds__(kThreads, 1)
span_tc_kernel(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mQs,
               const __grid_constant__ CUtensorMap mK, const __grid_constant__ CUtensorMap mV,
               const __grid_constant__ CUtensorMap mKt, const __grid_constant__ CUtensorMap mVt, Dev a,
               int q_tokens, int qs_tokens, int kv_rows) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem;
  uint8_t* sK = smem + kSmemK;
  uint8_t* sV = smem + kSmemV;
  Control& c = *reinterpret_cast<Control*>(smem + kSmemCtl);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      tc::mbar_init(&c.q_full[s], 1);
      tc::mbar_init(&c.q_empty[s], 1);
      tc::mbar_init(&c.s_full[s], 1);
      tc::mbar_init(&c.p_half[s], 4);
      tc::mbar_init(&c.p_full[s], 4);
      tc::mbar_init(&c.o_full[s], 1);
      tc::mbar_init(&c.o_free[s], 8);
      tc::mbar_init(&c.vfix[s], 4);
    }
    tc::mbar_init(&c.vfix[2], 8);
    for (int s = 0; s < kKStages; ++s) {
      tc::mbar_init(&c.k_full[s], 1);
      tc::mbar_init(&c.k_empty[s], 1);
    }
    for (int s = 0; s < kVStages; ++s) {
      tc::mbar_init(&c.v_full[s], 1);
      tc::mbar_init(&c.v_empty[s], 1);
    }
    for (int q = 0; q < 4; ++q) tc::mbar_init(&c.exchange[q], 2);
    for (int i = 0; i < kItems; ++i) {
      tc::mbar_init(&c.item_full[i], 1);
      tc::mbar_init(&c.item_empty[i], 11);        // warps 0, 1, 2 and the eight of the softmax
    }
    tc::mbar_init(&c.drain, 1);
    c.abort = (tc::smem_u32(smem) & 1023u) ? 1 : 0;      // the swizzle wants 1024-byte bounds
    tc::fence_mbar_init();
  }
  if (warp == 0) {
    tc::tmem_alloc(&c.tmem, 512);
    tc::tmem_relinquish();
  } else if (warp == 2 && lane == 0) {
    tc::prefetch_tensormap(&mQ);
    tc::prefetch_tensormap(&mQs);
    tc::prefetch_tensormap(&mK);
    tc::prefetch_tensormap(&mV);
    tc::prefetch_tensormap(&mKt);
    tc::prefetch_tensormap(&mVt);
  }
  pdl_wait();
  pdl_trigger();
  find_range(a, *reinterpret_cast<RangeScratch*>(smem), c.range, c.first);
  tc::tc_fence_before();
  // the scratch was read and written through the generic proxy where TMA writes next
  tc::fence_proxy_async_smem();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = c.tmem;
  volatile int* abort_flag = &c.abort;
  const bool layout_ok = *abort_flag == 0;
  int ni = 0;                     // items taken so far
  // Waits for the next item, which stays in the ring until given back.
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
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCtlRegs));
    if (layout_ok && warp == 3) {
      // ===================================================================== items
      if (lane == 0) {
        const Range R = c.range;
        Walker w;
        w.start(R, &c.first);
        Item it;
        bool more = true, ok = true;
        for (int n = 0; more && ok; ++n) {
          more = w.next(a, R, it);
          if (!more) it.j0 = it.j1 = -1;
          const int s = n % kItems;
          if (n >= kItems) ok = tc::mbar_wait(&c.item_empty[s], (n / kItems - 1) & 1, abort_flag, kWaitLimit);
          if (ok) {
            c.item[s] = it;
            tc::mbar_arrive(&c.item_full[s]);
          }
        }
        if (!ok) *abort_flag = 1;
      }
    } else if (layout_ok && (warp == 0 || warp == 2)) {
      // ===================================================================== TMA producers
      const bool is_k = warp == 0;
      const CUtensorMap* page_map = is_k ? &mK : &mV;
      const CUtensorMap* tile_map = is_k ? &mKt : &mVt;
      const int nstage = is_k ? kKStages : kVStages;
      uint8_t* ring = is_k ? sK : sV;
      uint64_t* full = is_k ? c.k_full : c.v_full;
      uint64_t* empty = is_k ? c.k_empty : c.v_empty;
      const int npg = kKeys / a.bs, page_bytes = a.bs * 128;
      int kt = 0, qn[2] = {0, 0};
      bool ok = true;
      while (ok) {
        ok = take(false);
        if (!ok || c.item[ni % kItems].j1 < 0) break;
        const Item it = c.item[ni % kItems];
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
        const int pair = it.kind == kPair ? 1 : 0, dual = it.kind == kDual ? 1 : 0;
        if (is_k) {
          const bool grp = it.end == it.P;
          const int tokens = grp ? q_tokens : qs_tokens;
          for (int b = 0; ok && b <= (it.kind != kLone ? 1 : 0); ++b) {
            if (qn[b] > 0) ok = lane0_wait(&c.q_empty[b], (qn[b] - 1) & 1, abort_flag);
            if (!ok) break;
            if (lane == 0) {
              tc::mbar_arrive_expect_tx(&c.q_full[b], 2 * tokens * a.G * 128);
              const int tok = it.o + (it.mt + b * pair) * q_tokens, row = (it.h + b * dual) * a.G;
              uint8_t* dst = sQ + b * kTile;
              if (grp) {
                tc::tma_load_3d(dst, &mQ, 0, row, tok, &c.q_full[b]);
                tc::tma_load_3d(dst + kAtom, &mQ, 64, row, tok, &c.q_full[b]);
              } else {
                tc::tma_load_3d(dst, &mQs, 0, row, tok, &c.q_full[b]);
                tc::tma_load_3d(dst + kAtom, &mQs, 64, row, tok, &c.q_full[b]);
              }
            }
            ++qn[b];
          }
        }
        // a dual unit's tiles alternate between its heads, which lie in the same pages
        for (int j = it.j0; ok && j < it.j1; ++j) {
          const int ahead = j + 1 < it.j1 ? tile_page(j + 1) : -1;
          const int pb0 = __shfl_sync(0xffffffffu, pb, 0);
          const bool run = __all_sync(0xffffffffu, lane >= npg || pb == pb0 + lane) && pb0 >= 0;
          for (int h = it.h; h <= it.h + dual; ++h, ++kt) {
            const int st = kt % nstage, use = kt / nstage;
            if (use > 0) ok = lane0_wait(&empty[st], (use - 1) & 1, abort_flag);
            if (!ok) break;
            if (lane == 0) tc::mbar_arrive_expect_tx(&full[st], kTile);
            __syncwarp();
            uint8_t* dst = ring + st * kTile;
            if (run) {
              if (lane == 0) {
                tc::tma_load_4d(dst, tile_map, 0, 0, h, pb0, &full[st]);
                tc::tma_load_4d(dst + kAtom, tile_map, 64, 0, h, pb0, &full[st]);
              }
            } else if (lane < npg) {
              const int row = pb >= 0 ? (pb * a.H_kv + h) * a.bs : kv_rows;      // past the cache: zeros
              tc::tma_load_2d(dst + lane * page_bytes, page_map, 0, row, &full[st]);
              tc::tma_load_2d(dst + kAtom + lane * page_bytes, page_map, 64, row, &full[st]);
            }
            __syncwarp();
          }
          pb = ahead;
        }
      }
      if (lane == 0) {
        if (!ok) *abort_flag = 1;
        // no copy may be in flight when the CTA ends
        volatile int never = 0;
        for (int k = max(0, kt - nstage); k < kt; ++k)
          tc::mbar_wait(&full[k % nstage], (k / nstage) & 1, &never, kWaitLimit / 8);
        for (int b = 0; is_k && b < 2; ++b)
          if (qn[b] > 0) tc::mbar_wait(&c.q_full[b], (qn[b] - 1) & 1, &never, kWaitLimit / 8);
      }
    } else if (layout_ok && warp == 1 && elect_one()) {
      // ===================================================================== MMA issuer
      const uint32_t id_qk = tc::idesc_bf16_f32(128, 128, false, false);
      const uint32_t id_pv = tc::idesc_bf16_f32(128, 128, false, true);
      // descriptors of the first Q buffer, K stage and V stage; the others' lie kTile / 16 apart
      const uint64_t dQ0 = tc::smem_desc(tc::smem_u32(sQ), 16, 1024), dK0 = tc::smem_desc(tc::smem_u32(sK), 16, 1024);
      const uint64_t dV0 = tc::smem_desc(tc::smem_u32(sV), kAtom, 1024);
      constexpr uint64_t kStep = kTile >> 4;
      int g0 = 0, qn0 = 0, qn1 = 0, pn0 = 0, pn1 = 0, hn = 0, li = 0;
      bool ok = true;
      for (; ok; ++li) {
        ok = take(true);
        const Item& it = c.item[ni % kItems];
        if (!ok || it.j1 < 0) break;
        const int nt = it.j1 - it.j0;
        const bool pair = it.kind == kPair, both = it.kind != kLone;      // both: a row tile for each slot
        give_back(true);
        const int n0 = both ? nt : (nt + 1) >> 1, n1 = both ? nt : nt >> 1;
        ok = tc::mbar_wait(&c.q_full[0], qn0++ & 1, abort_flag, kWaitLimit);
        if (ok && both) ok = tc::mbar_wait(&c.q_full[1], qn1++ & 1, abort_flag, kWaitLimit);
        const int it_tiles = pair ? nt : n0 + n1;
        // P of a pair in one piece, two groups of four products a tile; else in two, four groups
        const int groups = pair ? 2 : 4;
        const uint32_t wide = pair ? 16 : 32;
        const uint64_t two = both ? kStep : 0;
        // PV_s(k) and QK_s(k + 1) in turn, from QK_s(0) on: one short body each for both slots
#pragma unroll 1
        for (int e = -2; ok && e < 2 * n0; ++e) {
          const int s = e & 1, k = e >> 1, n = s ? n1 : n0;
          const bool lead = !pair || s == 0, tail = !pair || s == 1;     // a stage's first and last reader
          const uint32_t tP = tmem + 128 * s;
          if (k >= 0 && k < n) {
            const int g = g0 + (pair ? k : 2 * k + s), st = g % kVStages;
            const uint32_t pp = ((s ? pn1 : pn0) + k) & 1;
            // a pair's product starts on the first 64 keys
            if (!tc::mbar_wait(pair ? &c.p_half[s] : &c.p_full[s], pair ? (hn + k) & 1 : pp, abort_flag, kWaitLimit) ||
                (lead && !tc::mbar_wait(&c.v_full[st], (g / kVStages) & 1, abort_flag, kWaitLimit)) ||
                // an item's first product overwrites O_s: the epilogue before has to have read it
                (k == 0 && li > 0 && !tc::mbar_wait(&c.o_free[s], (li - 1) & 1, abort_flag, kWaitLimit))) {
              ok = false;
              break;
            }
            const uint32_t tO = tmem + 256 + 128 * s;
            const uint64_t dv = dV0 + uint64_t(st) * kStep;
#pragma unroll 1
            for (int q = 0; q < groups; ++q) {
              if (pair && q == 1 && !tc::mbar_wait(&c.p_full[s], pp, abort_flag, kWaitLimit)) {
                ok = false;
                break;
              }
              tc::tc_fence_after();
              const uint32_t col = tP + 2 * wide * (q & 1) + 16 * (q >> 1);
              const uint64_t d = dv + uint64_t((q & 1) * (8192 >> 4));
              tc::mma_bf16_ts(tO, col, d, id_pv, q > 0 || k > 0 ? 1u : 0u);
              tc::mma_bf16_ts(tO, col + 8, d + (2048 >> 4), id_pv, 1u);
              tc::mma_bf16_ts(tO, col + wide, d + (4096 >> 4), id_pv, 1u);
              tc::mma_bf16_ts(tO, col + wide + 8, d + (6144 >> 4), id_pv, 1u);
            }
            if (!ok) break;
            if (tail) tc::mma_commit(&c.v_empty[st]);
            if (k + 1 == n) tc::mma_commit(&c.o_full[s]);
          }
          if (k + 1 < n) {
            const int g = g0 + (pair ? k + 1 : 2 * (k + 1) + s), st = g % kKStages;
            if (lead && !tc::mbar_wait(&c.k_full[st], (g / kKStages) & 1, abort_flag, kWaitLimit)) {
              ok = false;
              break;
            }
            tc::tc_fence_after();
            const uint64_t dq = dQ0 + (s ? two : 0), dk = dK0 + uint64_t(st) * kStep;
            uint64_t da[8], db[8];      // formed before the first product, so that the eight go back to back
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
              const uint64_t off = uint64_t(((kk >> 2) * kAtom + (kk & 3) * 32) >> 4);
              da[kk] = dq + off;
              db[kk] = dk + off;
            }
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) tc::mma_bf16_ss(tP, da[kk], db[kk], id_qk, kk > 0 ? 1u : 0u);
            tc::mma_commit(&c.s_full[s]);
            if (tail) tc::mma_commit(&c.k_empty[st]);
            if (k + 2 == n && s == (n1 == n0 ? 1 : 0)) {      // the unit's last scores
              tc::mma_commit(&c.q_empty[0]);
              if (both) tc::mma_commit(&c.q_empty[1]);
            }
          }
        }
        g0 += it_tiles;
        pn0 += n0;
        pn1 += n1;
        if (pair) hn += nt;
      }
      if (!ok) *abort_flag = 1;
      // TMEM may not be freed under a product: wait for all of them, also after an abort
      tc::mma_commit(&c.drain);
      volatile int never = 0;
      tc::mbar_wait(&c.drain, 0, &never, kWaitLimit / 8);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // (the merge reads the records whatever becomes of the CTAs)
    if (warp == 4 && reports(c.range, gridDim.x)) write_recs(a, c.range.ordered);
    if (layout_ok) {
      // ===================================================================== softmax, epilogue
      const int s = (warp - 4) >> 2, q4 = warp & 3;
      const int m = q4 * 32 + lane;                   // row of the slot's tile; also a key of V's check
      const uint32_t lane_addr = uint32_t(q4 * 32) << 16;
      const uint32_t tS = tmem + lane_addr + 128 * s, tO = tmem + lane_addr + 256;
      const int t_loc = m / a.G;
      const float sl2 = a.scale_log2;
      int sn = 0, on[2] = {0, 0}, xn = 0, vn1 = 0, vn2 = 0, g0 = 0;
      bool ok = true;
      while (ok) {
        ok = take(false);
        const Item& it = c.item[ni % kItems];
        if (!ok || it.j1 < 0) break;
        const int nt = it.j1 - it.j0, j0 = it.j0, nt0 = it.nt0, skip = it.w0 - it.nt0, P = it.P;
        const bool pair = it.kind == kPair, both = it.kind != kLone;
        const int n0 = both ? nt : (nt + 1) >> 1, n1 = both ? nt : nt >> 1;
        const int h = it.h + (it.kind == kDual ? s : 0);
        const int ns = s == 0 ? n0 : n1;
        const int t = (it.mt + (pair ? s : 0)) * q_tokens + t_loc;
        const bool valid = t_loc < q_tokens && t < it.T;
        const bool live = __any_sync(0xffffffffu, valid);   // else only handshakes and V's check
        RowView view;
        view.anc = nullptr;
        view.W = a.W;
        view.lo = it.lo;
        view.P = P;
        view.end = it.end;
        view.sunk = min(a.sinks, P);
        view.first = view.deep = 0;
        if (valid && it.end > P) {
          view.anc = a.anc + size_t(it.o + t) * a.W;
          if (a.window > 0) {
            int n = 0;
            for (int w = 0; w < a.W; ++w) n += __popc(mask_word(view.anc, w, it.T));
            view.first = max(0, n - a.window);
            view.deep = max(0, a.sinks - P);
            view.lo = int(min((long long)P, max(0LL, (long long)P + max(n - 1, 0) - a.window + 1)));
          }
        }
        if (!valid) view.lo = view.P = view.end = view.sunk = 0;
        const int lo_max = a.window > 0 ? int(max(0LL, (long long)P + it.T - a.window)) : it.lo;
        float ref = -INFINITY, l = 0.f;        // P_s is scaled by 2^-ref, O_s and l with it
        for (int k = 0; k < ns; ++k) {
          const int ti = pair ? k : 2 * k + s, j = j0 + (both ? k : 2 * k + s);      // in the ring; of the entry
          const int kb = (j < nt0 ? j : j + skip) * kKeys;
          const bool masked = !(kb + kKeys <= P && (kb >= lo_max || kb + kKeys <= a.sinks));
          uint32_t vis0 = ~0u, vis1 = ~0u, vis2 = ~0u, vis3 = ~0u;
          if (masked && live) {
            vis0 = visible32(view, kb);
            vis1 = visible32(view, kb + 32);
            vis2 = visible32(view, kb + 64);
            vis3 = visible32(view, kb + 96);
          }
          if (!warp_wait(&c.s_full[s], sn & 1, abort_flag)) { ok = false; break; }
          ++sn;
          tc::tc_fence_after();
          bool nan = false;        // the row sees a key whose V is not finite
          if (masked) {
            // V's rows, 32 a warp, eight lanes a row (of a pair unit one half of the columns in each slot).
            // S of this tile came after the products before, so V's stage holds no older tile that is
            // still to be read, and the phase waited for is the stage's next.
            const int gv = g0 + ti, st = gv % kVStages;
            if (!warp_wait(&c.v_full[st], (gv / kVStages) & 1, abort_flag)) { ok = false; break; }
            uint8_t* tile = sV + st * kTile + (q4 * 32 + (lane >> 3)) * 128 + (lane & 7) * 16;
            const int key0 = kb + q4 * 32 + (lane >> 3), end = it.end;
            const int sink = it.sink, lo = it.lo;
            uint32_t word = 0;
            bool wrote = false;
#pragma unroll 1
            for (int half = pair ? s : 0; half < (pair ? s + 1 : 2); ++half) {
              uint8_t* p = tile + half * kAtom;
              uint32_t hits = 0;           // bit i: an exponent of all ones in row 4 i + lane / 8
#pragma unroll 2
              for (int i = 0; i < 8; ++i) {
                const uint4 x = *reinterpret_cast<const uint4*>(p + i * 512);
                const int key = key0 + 4 * i;
                const bool seen = key < sink || (key >= lo && key < end);
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
                  for (int r = 0; r < 4; ++r) word |= ((lanes >> (8 * r)) & 0xffu) ? 1u << (4 * i + r) : 0u;
                }
              }
            }
            if (wrote) tc::fence_proxy_async_smem();
            if (lane == 0) c.vbad[k & 1][s][q4] = word;
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&c.vfix[pair ? 2 : s]);
            int& vn = pair ? vn2 : vn1;
            if (!warp_wait(&c.vfix[pair ? 2 : s], vn & 1, abort_flag)) { ok = false; break; }
            ++vn;
            const uint4 b0 = *reinterpret_cast<const uint4*>(c.vbad[k & 1][s]);
            const uint4 b1 = *reinterpret_cast<const uint4*>(c.vbad[k & 1][pair ? 1 - s : s]);
            nan = (((b0.x | b1.x) & vis0) | ((b0.y | b1.y) & vis1) | ((b0.z | b1.z) & vis2) | ((b0.w | b1.w) & vis3)) != 0u;
          }
          if (live) {
            auto hide = [&](uint32_t (&x)[32], uint32_t vis) {
#pragma unroll
              for (int i = 0; i < 32; ++i) x[i] = (vis >> i) & 1u ? x[i] : __float_as_uint(-INFINITY);
            };
            // the reference moves when the tile's maximum is 2^kLazy over it, and O_s and l follow
            auto refer = [&](float top) {
              if (!valid) top = -INFINITY;
              if (!__any_sync(0xffffffffu, top > ref + kLazy)) return;
              const bool up = top > ref + kLazy;
              const float f = up && ref != -INFINITY ? ex2(ref - top) : 1.f;
              // S of this tile was issued after the product before, which has therefore landed in O
              if (k > 0) {
#pragma unroll 1
                for (int c0 = 0; c0 < kD; c0 += 16) {
                  uint32_t r[16];
                  tc::tmem_ld16(tO + 128 * s + c0, r);
                  tc::tmem_ld_wait();
#pragma unroll
                  for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * f);
                  tc::tmem_st16(tO + 128 * s + c0, r);
                }
              }
              l *= f;
              ref = up ? top : ref;
            };
            uint64_t acc0 = f2_pack(0.f, 0.f), acc1 = acc0;
            // a row that has seen nothing yet: 2^(x - inf) = 0 for every key (masked: -inf - inf)
            uint64_t sl = 0, add = 0;
            bool coarse = false;
            auto scale = [&] {
              float v = ref == -INFINITY ? 1.f : sl2, w = nan ? NAN : ref == -INFINITY ? -INFINITY : -ref;
              const bool mine = fabsf(ref) >= kCoarse && ref != -INFINITY;
              coarse = __any_sync(0xffffffffu, mine);
              if (__builtin_expect(coarse, 0)) {
                coarse_exponents(tS, sl2, ref, mine, make_uint4(vis0, vis1, vis2, vis3));
                if (mine) {
                  v = 1.f;
                  w = nan ? NAN : 0.f;
                }
              }
              sl = f2_pack(v, v);
              add = f2_pack(w, w);
            };
            if (pair) {
              uint32_t x0[32], x1[32], x2[32], x3[32];
              auto load = [&] {
                tc::tmem_ld32(tS, x0);
                tc::tmem_ld32(tS + 32, x1);
                tc::tmem_ld32(tS + 64, x2);
                tc::tmem_ld32(tS + 96, x3);
                tc::tmem_ld_wait();
              };
              load();
              if (masked) {
                hide(x0, vis0);
                hide(x1, vis1);
                hide(x2, vis2);
                hide(x3, vis3);
              }
              refer(fmaxf(fmaxf(max32(x0), max32(x1)), fmaxf(max32(x2), max32(x3))) * sl2);
              scale();
              if (__builtin_expect(coarse, 0)) load();
              weights32<false>(x0, sl, add, acc0, tS);
              weights32<false>(x1, sl, add, acc1, tS + 16);
              tc::tmem_st_wait();
              tc::tc_fence_before();
              __syncwarp();
              if (lane == 0) tc::mbar_arrive(&c.p_half[s]);
              weights32<false>(x2, sl, add, acc0, tS + 32);
              weights32<false>(x3, sl, add, acc1, tS + 48);
            } else {
              // Two pieces of P, 32 keys at a time, read twice: a single unit is bound by its K/V's bytes or
              // by latency, and this is little code to fetch.
              float top = -INFINITY;
#pragma unroll 1
              for (int i = 0; i < 8; ++i) {
                const int q = i & 3;
                uint32_t x[32];
                tc::tmem_ld32(tS + 32 * q, x);
                tc::tmem_ld_wait();
                if (masked) hide(x, q == 0 ? vis0 : q == 1 ? vis1 : q == 2 ? vis2 : vis3);
                if (i < 4) {
                  top = fmaxf(top, max32(x));
                  if (i == 3) {
                    refer(top * sl2);
                    scale();
                  }
                } else {
                  weights32<true>(x, sl, add, acc0, tS + 32 * q);
                }
              }
            }
            float r0, r1, r2, r3;
            f2_unpack(acc0, r0, r1);
            f2_unpack(acc1, r2, r3);
            l += (r0 + r1) + (r2 + r3);
            tc::tmem_st_wait();
          }
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (pair && !live) tc::mbar_arrive(&c.p_half[s]);
            tc::mbar_arrive(&c.p_full[s]);
          }
        }
        if (!ok) break;
        // the products whose O this warp reads (both slots' of a single unit)
        for (int u = 0; ok && u < 2; ++u) {
          if ((u == 0 ? n0 : n1) == 0) continue;
          if (u == s || !both) ok = warp_wait(&c.o_full[u], on[u] & 1, abort_flag);
          ++on[u];
        }
        if (!ok) break;
        tc::tc_fence_after();
        float lt = l, M = ref, w0 = 0.f, w1 = 0.f;
        bool any0 = true, any1 = false;        // the row has seen something in slot 0's and 1's tiles of a lone unit
        int c_lo = 0, c_hi = kD;
        if (!both) {
          // exchange (reference, sum) with the other slot's warp of this quarter; 64 columns each
          c.row[s][0][m] = ref;
          c.row[s][1][m] = l;
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&c.exchange[q4]);
          if (!warp_wait(&c.exchange[q4], xn & 1, abort_flag)) { ok = false; break; }
          ++xn;
          const float mo = c.row[1 - s][0][m], lo = c.row[1 - s][1][m];
          const float m0 = s == 0 ? ref : mo, m1 = s == 0 ? mo : ref, l0 = s == 0 ? l : lo, l1 = s == 0 ? lo : l;
          // a slot that saw nothing but NaN has the reference -inf and the sum NaN
          any0 = m0 != -INFINITY || l0 != 0.f;
          any1 = n1 > 0 && (m1 != -INFINITY || l1 != 0.f);
          M = fmaxf(m0, m1);
          w0 = m0 != -INFINITY ? ex2(m0 - M) : 0.f;
          w1 = n1 > 0 && m1 != -INFINITY ? ex2(m1 - M) : 0.f;
          lt = l0 * w0 + (n1 > 0 ? l1 * w1 : 0.f);
          c_lo = 64 * s;
          c_hi = c_lo + 64;
        }
        const float inv = lt == 0.f ? 0.f : 1.f / lt;
        const float lse2 = lt == 0.f ? -INFINITY : M + log2f(lt);
        if (live) {
          // Rows leave through shared memory, 32 columns at a time, so that a store is of whole lines: row r's
          // 16-byte unit u lies at u ^ (r & 7).
          uint8_t* stage = smem + kSmemOut + (warp - 4) * 4096;
          const bool direct = it.slot == -1;
          const int nv = __popc(__ballot_sync(0xffffffffu, valid));    // the warp's rows 0 .. nv - 1
          const size_t slot_row = size_t(max(it.slot, 0)) * a.part_rows + (both ? s * kRows : 0);
          // where this lane's row of 128 columns begins, in elements of its buffer
          const size_t row_of = size_t(it.o + t) * a.H_q + h * a.G + (m - t_loc * a.G);
          const unsigned long long mine = (it.slot >= 0 ? slot_row + m : row_of) * kD;
          float* rows = it.slot >= 0 ? a.part_o : it.slot == -3 ? a.row_o + size_t(a.N) * a.H_q * kD : a.row_o;
          unsigned long long at[8];        // where rows 4 i + lane / 8 begin
#pragma unroll
          for (int i = 0; i < 8; ++i) at[i] = __shfl_sync(0xffffffffu, mine, 4 * i + (lane >> 3));
          const float wa = both ? inv : w0 * inv, wb = w1 * inv;
          any0 = any0 && lt != 0.f;            // (a weight of 0 lets a NaN through)
          const int u8 = lane & 7;
#pragma unroll 1
          for (int c0 = c_lo; c0 < c_hi; c0 += 32) {
            uint32_t r[32];
            float v[32];
            tc::tmem_ld32(tO + (both ? 128 * s : 0) + c0, r);
            tc::tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = any0 ? __uint_as_float(r[i]) * wa : 0.f;
            if (!both && n1 > 0) {
              tc::tmem_ld32(tO + 128 + c0, r);
              tc::tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = any1 ? fmaf(__uint_as_float(r[i]), wb, v[i]) : v[i];
            }
            if (direct) {
              const int h4 = (c0 >> 3) & 4;        // 64 columns make a row's 128 bytes
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                uint4 w;
                w.x = pack_bf16(v[8 * u], v[8 * u + 1]);
                w.y = pack_bf16(v[8 * u + 2], v[8 * u + 3]);
                w.z = pack_bf16(v[8 * u + 4], v[8 * u + 5]);
                w.w = pack_bf16(v[8 * u + 6], v[8 * u + 7]);
                *reinterpret_cast<uint4*>(stage + lane * 128 + (((u + h4) ^ (lane & 7)) << 4)) = w;
              }
              if (h4 == 0) continue;
            } else {
#pragma unroll
              for (int u = 0; u < 8; ++u)
                *reinterpret_cast<float4*>(stage + lane * 128 + ((u ^ (lane & 7)) << 4)) =
                    make_float4(v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]);
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int row = 4 * i + (lane >> 3);
              const uint4 w = *reinterpret_cast<const uint4*>(stage + row * 128 + ((u8 ^ (row & 7)) << 4));
              if (row < nv) {
                if (direct) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) + at[i] + c0 - 32 + 8 * u8) = w;
                else *reinterpret_cast<uint4*>(rows + at[i] + c0 + 4 * u8) = w;
              }
            }
            __syncwarp();
          }
          if (valid && (both || s == 0)) {
            if (it.slot >= 0) a.part_lse[slot_row + m] = lse2;
            else if (!direct) a.row_lse[(it.slot == -3 ? size_t(a.N) * a.H_q : 0) + row_of] = lse2;
            else if (a.lse) a.lse[row_of] = lse2 * 0.6931471805599453f;
          }
        }
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          tc::mbar_arrive(&c.o_free[0]);
          tc::mbar_arrive(&c.o_free[1]);
        }
        give_back(false);
        g0 += pair ? nt : n0 + n1;
      }
      if (!ok) *abort_flag = 1;
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (*abort_flag && tid == 0) {
    // every request of the range is unreliable after a wait that ran out
    const Range R = c.range;
    Walker w;
    w.start(R, nullptr);
    Item it;
    while (w.next(a, R, it)) flag(a, it.req, it.nreq, SPEC_REQ_TIMEOUT);
  }
  tc::tc_fence_after();
  if (warp == 0) tc::tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------------------ host
static PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// Whether the tensor cores take this call: their types and tiles, and row coordinates in 32 bits.
bool tc_takes(const spec_attn_params* p) {
  const int G = p->H_q / p->H_kv;
  return p->dtype == SPEC_BF16 && p->head_dim == kD && G <= kRows &&
         (p->block_size == 16 || p->block_size == 32 || p->block_size == 64 || p->block_size == 128);
}
int tc_row_tile(const spec_attn_params* p) {
  const int G = p->H_q / p->H_kv;
  return kRows / G * G;
}

static bool encode(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* map, const void* ptr, int rank,
                   const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapL2promotion l2) {
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(ptr), dims, strides, box, ones,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, l2, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

spec_status_t make_tc_maps(const spec_attn_params* p, TcMaps& m) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return SPEC_ERR_CUDA;
  const int G = p->H_q / p->H_kv;
  m.q_tokens = kRows / G;
  m.q_own_tokens = p->T_max < m.q_tokens ? p->T_max : m.q_tokens;
  m.q_rows_tokens = G <= 16 ? 16 / G : 1;
  m.kv_rows = p->num_blocks * p->H_kv * p->block_size;      // below 2^31 - 256, checked
  bool ok = true;
  CUtensorMap* q[3] = {&m.q, &m.q_own, &m.q_rows};
  const int tokens[3] = {m.q_tokens, m.q_own_tokens, m.q_rows_tokens};
  for (int i = 0; i < 3; ++i) {
    const cuuint64_t dims[3] = {cuuint64_t(kD), cuuint64_t(p->H_q), cuuint64_t(p->N)};
    const cuuint64_t strides[2] = {cuuint64_t(kD) * 2, cuuint64_t(p->H_q) * kD * 2};
    const cuuint32_t box[3] = {64, cuuint32_t(G), cuuint32_t(tokens[i])};
    ok = ok && encode(enc, q[i], p->q, 3, dims, strides, box, CU_TENSOR_MAP_L2_PROMOTION_L2_128B);
  }
  for (int v = 0; v < 2; ++v) {
    const void* cache = v ? p->v_cache : p->k_cache;
    {
      const cuuint64_t dims[2] = {cuuint64_t(kD), cuuint64_t(m.kv_rows)};
      const cuuint64_t strides[1] = {cuuint64_t(kD) * 2};
      const cuuint32_t box[2] = {64, cuuint32_t(p->block_size)};
      ok = ok && encode(enc, v ? &m.v_page : &m.k_page, cache, 2, dims, strides, box, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
    }
    {
      const cuuint64_t dims[4] = {cuuint64_t(kD), cuuint64_t(p->block_size), cuuint64_t(p->H_kv), cuuint64_t(p->num_blocks)};
      const cuuint64_t strides[3] = {cuuint64_t(kD) * 2, cuuint64_t(p->block_size) * kD * 2,
                                     cuuint64_t(p->H_kv) * p->block_size * kD * 2};
      const cuuint32_t box[4] = {64, cuuint32_t(p->block_size), 1, cuuint32_t(kKeys / p->block_size)};
      ok = ok && encode(enc, v ? &m.v_tile : &m.k_tile, cache, 4, dims, strides, box, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
    }
  }
  return ok ? SPEC_OK : SPEC_ERR_INVALID_ARG;
}

spec_status_t launch_span_tc(const Dev& d, const TcMaps& m, cudaStream_t s) {
  static DeviceOnce raised;
  const spec_status_t st = raise_dyn_smem_once(span_tc_kernel, kSmemBytes, raised);
  if (st != SPEC_OK) return st;
  return launch_result(launch_pdl(span_tc_kernel, dim3(d.ctas), dim3(kThreads), size_t(kSmemBytes), s, m.q, m.q_own,
                                  m.k_page, m.v_page, m.k_tile, m.v_tile, d, m.q_tokens, m.q_own_tokens, m.kv_rows));
}

}  // namespace span
}  // namespace spec
