// Work of the attention forms that read stretches of a request's cache (a shared prefix, a window and
// sinks): what a stretch is, how the stretches' tiles are laid end to end and cut into equal ranges,
// one a CTA, and where a CTA leaves the pieces that the merge puts together.
//
// Entries, in the order of the stream:
//   group g (shared form, two members at least and shared_len > 0): rows = all members' query rows,
//     keys [0, shared_len) by the first member's table row, every key visible to every row;
//   request r: rows = its query rows, keys [lo, P + T) and [0, sink) by its own table row.
// An entry has H_kv x (units) units; a unit is one or two row tiles of a KV head (`pairing`: two tiles
// read every K/V tile once) over all of the entry's key tiles.  A tile of a pair costs kPairCost, of a
// single row tile kSingleCost; ranges are equal in cost, and a tile belongs to the range that its first
// cost unit lies in.
#pragma once

#include "common.cuh"

namespace spec {
namespace span {

constexpr int kPairCost = 2, kSingleCost = 1;
constexpr int kMinCost = 8;              // cost of a range at least: small calls use fewer ranges
constexpr int kMaxCtas = 1024;
constexpr int kGroupCache = 4096;        // group offsets held in shared memory while ranges are found

struct Dev {
  const int32_t* block_table;
  const int32_t* prefix_len;
  const int32_t* node_offset;
  const uint32_t* anc;
  const int32_t* group_offset;   // shared form: [Gn + 1], else null
  const int32_t* shared_len;     // shared form: [Gn]
  const void* q;
  const void* k;
  const void* v;
  void* o;
  float* lse;
  int32_t* req_status;
  long long* ebeg;      // [Gn + B + 1]: cost before each entry, then the total (CTA 0, for the merge)
  float* part_o;        // [2 ctas][part_rows][d]: pieces of cut units
  float* part_lse;      // [2 ctas][part_rows]: their log2-sum-exps
  float* row_o;         // [2][N][H_q][d]: uncut units of the shared form; 0: group, 1: own
  float* row_lse;       // [2][N][H_q]
  int B, N, Gn, H_q, H_kv, G, d, bs, T_max, W, num_blocks, max_blocks, ctas;
  int window, sinks;    // window form; window = 0: none
  int rt;               // query rows of a row tile
  int bn;               // keys of a key tile
  int part_rows, pairing;
  float scale_log2;
};

// One entry: rows [0, T G) of tokens o .. o + T - 1; keys [0, sink) and [lo, end), those from P on
// under the ancestor mask; key tiles 0 .. nt0 - 1, then w0 ..: nt of them.
struct Entry {
  int o, T, P, end, lo, sink, table, nt0, w0, nt, mts;
  int group;            // >= 0: entry of a group; -1: a request on its own; -2 - g: a member of group g
};

__device__ __forceinline__ int units_of(const Dev& a, const Entry& e) {
  return a.pairing ? (e.mts + 1) >> 1 : e.mts;
}
// cost of one KV head of the entry
__device__ __forceinline__ long long head_cost(const Dev& a, const Entry& e) {
  const int per = a.pairing ? (e.mts >> 1) * kPairCost + (e.mts & 1) * kSingleCost : e.mts * kSingleCost;
  return (long long)e.nt * per;
}

// The group of request r: the g with off[g] <= r < off[g + 1], -1 if the offsets name none.
__device__ __forceinline__ int find_group(const int32_t* off, int Gn, int r) {
  int lo = 0, hi = Gn - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (off[mid] <= r) lo = mid; else hi = mid - 1;
  }
  return off[lo] <= r && r < off[lo + 1] ? lo : -1;
}

// Group g's tokens, if it is one that is computed together: two members at least, a shared part, and
// node offsets that lie in [0, N] (a member's own error leaves the others' results as they are).
__device__ __forceinline__ bool group_tokens(const Dev& a, const int32_t* off, int g, int& o, int& T, int& len) {
  const int r0 = off[g], r1 = off[g + 1];
  len = a.shared_len[g];
  if (r0 < 0 || r1 > a.B || r1 - r0 < 2 || len <= 0) return false;
  o = a.node_offset[r0];
  const int e = a.node_offset[r1];
  T = e - o;
  return o >= 0 && e <= a.N && T >= 1 && (long long)(len + a.bs - 1) / a.bs <= a.max_blocks;
}

__device__ __forceinline__ void key_tiles(const Dev& a, Entry& e) {
  e.nt0 = (e.sink + a.bn - 1) / a.bn;
  e.w0 = max(e.lo / a.bn, e.nt0);
  e.nt = e.nt0 + (e.end + a.bn - 1) / a.bn - e.w0;
  e.mts = (int)(((long long)e.T * a.G + a.rt - 1) / a.rt);
}

// Entry i of the stream (groups first).  `off`: the group offsets, possibly a copy.  mts = 0: no work.
// `bad`: SPEC_REQ_* bits that the request gets.  The bits that this library's attention sets itself
// (BAD_BLOCK, TIMEOUT) are ignored, and the others only take away a request's own units, so that all
// roles of all CTAs derive the same stream from the same inputs.
__device__ __forceinline__ Entry entry_of(const Dev& a, const int32_t* off, int i, int& bad) {
  Entry e;
  e.o = e.T = e.P = e.end = e.lo = e.sink = e.nt0 = e.w0 = e.nt = e.mts = e.table = 0;
  e.group = -1;
  bad = 0;
  if (i < a.Gn) {
    int o, T, len;
    if (!group_tokens(a, off, i, o, T, len)) return e;
    e.o = o;
    e.T = T;
    e.P = e.end = len;
    e.table = off[i];
    e.group = i;
    key_tiles(a, e);
    return e;
  }
  const int r = i - a.Gn;
  const int o = a.node_offset[r], T = a.node_offset[r + 1] - o, P = a.prefix_len[r];
  const int st = a.req_status[r] & ~(SPEC_REQ_BAD_BLOCK | SPEC_REQ_TIMEOUT);
  if (st != 0) return e;
  if (T < 1 || T > a.T_max || P < 0 || o < 0 || o + T > a.N) {
    bad = SPEC_REQ_BAD_SIZE;
    return e;
  }
  const long long end = (long long)P + T;
  if ((end + a.bs - 1) / a.bs > a.max_blocks || end > 0x7fffffffLL - 1024) {
    bad = SPEC_REQ_BAD_BLOCK;
    return e;
  }
  e.o = o;
  e.T = T;
  e.P = P;
  e.end = int(end);
  e.table = r;
  if (a.window > 0) {
    e.lo = max(0, P - a.window + 1);
    e.sink = min(a.sinks, e.lo);
  } else if (a.Gn > 0) {
    const int g = find_group(off, a.Gn, r);
    int go, gT, len;
    if (g < 0 || a.shared_len[g] < 0 || a.shared_len[g] > P) {
      bad = SPEC_REQ_BAD_SIZE;
      e.T = 0;
      return e;
    }
    if (group_tokens(a, off, g, go, gT, len)) {
      if (o < go || o + T > go + gT) {
        bad = SPEC_REQ_BAD_SIZE;
        e.T = 0;
        return e;
      }
      e.lo = len;
      e.group = -2 - g;
    } else if (off[g + 1] - off[g] >= 2 && a.shared_len[g] > 0) {   // the group's offsets are bad
      bad = SPEC_REQ_BAD_SIZE;
      e.T = 0;
      return e;
    }
  }
  key_tiles(a, e);
  return e;
}

__device__ __forceinline__ long long range_start(long long total, int C, int c) { return total * c / C; }
// the range holding cost position t (0 <= t < total)
__device__ __forceinline__ int range_of(long long t, long long total, int C) {
  const long long c = ((t + 1) * C + total - 1) / total - 1;
  return int(c < 0 ? 0 : (c >= C ? C - 1 : c));
}
__device__ __forceinline__ int ranges(const Dev& a, long long total) {
  return int(max(1LL, min((long long)a.ctas, total / kMinCost)));
}

// This CTA's share: cost positions [t0, t1), from entry e0, before which the cost is ebeg0.
struct Range {
  long long total, t0, t1, ebeg0;
  int C, e0;
};

// Scratch of the search; the group offsets are copied here when they fit.
struct RangeScratch {
  long long sum[34];
  long long found_beg;
  int found;
  int32_t off[kGroupCache + 1];
};

// All kThreads threads find the CTA's range.  CTA 0 also writes ebeg and reports the requests that
// cannot be worked on.  Contains __syncthreads.
template <int kThreads>
__device__ Range cta_range(const Dev& a, RangeScratch& s) {
  constexpr int kW = kThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int E = a.Gn + a.B;
  const int32_t* off = a.group_offset;
  if (a.Gn > 0 && a.Gn <= kGroupCache) {
    for (int i = tid; i <= a.Gn; i += kThreads) s.off[i] = a.group_offset[i];
    off = s.off;
    __syncthreads();
  }
  auto cost_of = [&](int i) -> long long {
    if (i >= E) return 0;
    int bad;
    const Entry e = entry_of(a, off, i, bad);
    if (bad && blockIdx.x == 0) atomicOr(&a.req_status[i - a.Gn], bad);
    return head_cost(a, e) * a.H_kv;
  };
  const long long mine0 = cost_of(tid);
  long long mine = mine0;
  for (int i = tid + kThreads; i < E; i += kThreads) mine += cost_of(i);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) s.sum[warp] = mine;
  if (tid == 0) s.found = -1;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kW; ++w) total += s.sum[w];
  if (blockIdx.x == 0 && tid == 0) a.ebeg[E] = total;
  Range R;
  R.total = total;
  R.C = ranges(a, total);
  R.t0 = R.t1 = R.ebeg0 = 0;
  R.e0 = 0;
  const int c = blockIdx.x;
  const bool work = total > 0 && c < R.C;
  if (work) {
    R.t0 = range_start(total, R.C, c);
    R.t1 = range_start(total, R.C, c + 1);
  }
  if (!work && c != 0) return R;
  long long base = 0;
  for (int i0 = 0; i0 < E; i0 += kThreads) {
    const int i = i0 + tid;
    const long long cost = i0 == 0 ? mine0 : cost_of(i);
    long long incl = cost;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    __syncthreads();   // s.sum is rewritten
    if (lane == 31) s.sum[warp] = incl;
    __syncthreads();
    long long before = base, chunk = 0;
#pragma unroll
    for (int w = 0; w < kW; ++w) {
      if (w < warp) before += s.sum[w];
      chunk += s.sum[w];
    }
    const long long hi = before + incl, lo = hi - cost;
    if (c == 0 && i < E) a.ebeg[i] = lo;
    if (work && cost > 0 && lo <= R.t0 && R.t0 < hi) {
      s.found = i;
      s.found_beg = lo;
    }
    base += chunk;
    if (c != 0 && base > R.t0) break;   // uniform
  }
  __syncthreads();
  if (work) {
    R.e0 = s.found;
    R.ebeg0 = s.found_beg;
    if (R.e0 < 0 || R.e0 >= E) R.t1 = R.t0;   // never: the scan finds the entry
  }
  __syncthreads();
  return R;
}

// Key tiles [j0, j1) of one unit.
struct Item {
  int o, T, P, end, lo, sink, table, nt0, w0;
  int h, mt, pair;       // KV head, first row tile, 1: two row tiles
  int j0, j1;
  int slot;              // >= 0: a piece of a cut unit, to part_o[slot]; -1: to o; -2, -3: to row_o[0], [1]
  int req, nreq;         // the requests that it concerns
  int pad;
};

// Walks the CTA's range.  One thread or a whole warp alike.
struct Walker {
  long long t, ebeg;     // next cost position; cost before the entry
  int i, bad;
  long long hcost;
  Entry e;
  const int32_t* off;    // group offsets
  __device__ __forceinline__ void start(const Dev& a, const Range& R) {
    t = R.t0;
    i = R.e0;
    ebeg = R.ebeg0;
    off = a.group_offset;
    hcost = 0;
    if (t < R.t1) {
      e = entry_of(a, off, i, bad);
      hcost = head_cost(a, e);
    }
  }
  __device__ __forceinline__ bool next(const Dev& a, const Range& R, Item& it) {
    while (t < R.t1) {
      while (t >= ebeg + hcost * a.H_kv) {
        ebeg += hcost * a.H_kv;
        if (++i >= a.Gn + a.B) return false;
        e = entry_of(a, off, i, bad);
        hcost = head_cost(a, e);
      }
      const long long in_entry = t - ebeg;
      const int h = int(in_entry / hcost);
      const long long in_head = in_entry - h * hcost;
      const int np = a.pairing ? e.mts >> 1 : 0;
      const long long pair_part = (long long)np * kPairCost * e.nt;
      const bool pair = in_head < pair_part;
      const int w = pair ? kPairCost : kSingleCost;
      const long long ucost = (long long)w * e.nt;
      const int u = int(pair ? in_head / ucost : (in_head - pair_part) / ucost);
      const long long ubeg = ebeg + h * hcost + (pair ? 0 : pair_part) + u * ucost;
      const int j0 = int((t - ubeg + w - 1) / w);
      const int j1 = int(min((long long)e.nt, (R.t1 - ubeg + w - 1) / w));
      t = min(R.t1, ubeg + ucost);
      if (j1 <= j0) continue;
      it.o = e.o; it.T = e.T; it.P = e.P; it.end = e.end; it.lo = e.lo; it.sink = e.sink;
      it.table = e.table; it.nt0 = e.nt0; it.w0 = e.w0;
      it.h = h;
      it.pair = pair ? 1 : 0;
      it.mt = pair ? 2 * u : 2 * np + u;
      it.j0 = j0;
      it.j1 = j1;
      const bool cut = j0 > 0 || j1 < e.nt;
      it.slot = cut ? 2 * int(blockIdx.x) + (ubeg > R.t0 ? 1 : 0)
                    : e.group >= 0 ? -2 : e.group == -1 ? -1 : -3;
      it.req = e.group >= 0 ? off[e.group] : i - a.Gn;
      it.nreq = e.group >= 0 ? off[e.group + 1] - it.req : 1;
      return true;
    }
    return false;
  }
};

__device__ __forceinline__ int key_base(const Dev& a, int nt0, int w0, int j) {
  return (j < nt0 ? j : w0 + j - nt0) * a.bn;
}
// a page that some row may see: it meets [0, sink) or [lo, end)
__device__ __forceinline__ bool page_needed(int first, int bs, int lo, int sink, int end) {
  return first < sink || (first + bs > lo && first < end);
}
__device__ __forceinline__ void flag(const Dev& a, int req, int nreq, int bits) {
  for (int r = req; r < req + nreq; ++r) atomicOr(&a.req_status[r], bits);
}

// The ancestor words of one query row under the window: of its n ancestors-or-self (depths 0 .. n - 1
// in increasing index, since parents come before children) those at depth k with n - 1 - k < window or
// P + k < sinks.  Returns the row's lower bound of visible prefix keys.
__device__ __forceinline__ int window_words(const Dev& a, const uint32_t* row, int P, uint32_t* out) {
  int n = 0;
  for (int w = 0; w < a.W; ++w) n += __popc(row[w]);
  const int first = n > a.window ? n - a.window : 0;       // depths below are out of the window
  const int sunk = a.sinks > P ? a.sinks - P : 0;          // depths below are sinks
  int k = 0;
  for (int w = 0; w < a.W; ++w) {
    uint32_t x = row[w], keep = 0;
    const int c = __popc(x);
    if (k >= first || k + c <= sunk) {
      keep = x;
      k += c;
    } else {
      while (x) {
        const uint32_t b = x & (0u - x);
        if (k >= first || k < sunk) keep |= b;
        x ^= b;
        ++k;
      }
    }
    out[w] = keep;
  }
  const int depth = n > 0 ? n - 1 : 0;
  const long long lo = (long long)P + depth - a.window + 1;
  return lo > 0 ? int(min(lo, (long long)P)) : 0;
}

}  // namespace span
}  // namespace spec
