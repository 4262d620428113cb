// Work of the attention forms that read stretches of a request's cache (a shared prefix, a window and
// sinks): what a stretch is, how the stretches' tiles are laid end to end and cut into equal ranges,
// one a CTA, and where a CTA leaves the pieces that the merge puts together.
//
// Entries, in the order of the stream:
//   group g (shared form, two members at least and shared_len > 0): rows = all members' query rows,
//     keys [0, shared_len) by the first member's table row, every key visible to every row;
//   request r: rows = its query rows, keys [lo, P + T) and [0, sink) by its own table row.
// An entry's units, each over all of its key tiles: with `pairing`, head by head, first its pair units (two row
// tiles, which read every K/V tile once), then, if its row tiles are odd in number, the last one; two heads
// make a block if that last tile has at most dual_rows rows, and share a dual unit for it; without `pairing`
// every row tile of every head.  A unit costs `cu`: cost_unit for its start and end and cost_masked for each
// tile under a mask; and cost_pair, cost_dual or cost_single for each key tile; ranges are equal in cost, and a
// tile belongs to the
// range that its first cost unit lies in.
#pragma once

#include <cuda.h>

#include "common.cuh"

namespace spec {
namespace span {

constexpr int kMaxCtas = 1024;
constexpr int kStartCache = 1024;      // requests whose inputs are held in shared memory at the start

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
  struct Rec* recs;     // [Gn + B]: the entries, for the merge
  long long* total;     // cost of the stream, for the merge
  float* part_o;        // [2 ctas][part_rows][d]: pieces of cut units
  float* part_lse;      // [2 ctas][part_rows]: their log2-sum-exps
  float* row_o;         // [2][N][H_q][d]: uncut units of the shared form; 0: group, 1: own
  float* row_lse;       // [2][N][H_q]
  int B, N, Gn, H_q, H_kv, G, d, bs, T_max, W, num_blocks, max_blocks, ctas;
  int window, sinks;    // window form; window = 0: none
  int rt;               // query rows of a row tile
  int bn;               // keys of a key tile
  int part_rows, pairing, dual_rows;
  int cost_pair, cost_dual, cost_single, cost_unit, cost_masked, cost_min;   // cost_min: of a range at least
  float scale_log2;
};

// What the merge has to know of an entry: where it lies in the stream, its tokens and tiles.
struct Rec {
  long long beg;
  int o, T, nt, mts, group, cu;
};

// One entry: rows [0, T G) of tokens o .. o + T - 1; keys [0, sink) and [lo, end), those from P on
// under the ancestor mask; key tiles 0 .. nt0 - 1, then w0 ..: nt of them.
struct Entry {
  int o, T, P, end, lo, sink, table, nt0, w0, nt, mts;
  int cu;               // cost of a unit besides its tiles
  int group;            // >= 0: entry of a group; -1: a request on its own; -2 - g: a member of group g
};

// An entry's (or a Rec's) blocks: of hb heads with `pairs` pair units each and then `rest` others; a last head
// that finds no second is a block of one.
struct Units {
  int hb, pairs, rest;
};
template <typename E>
__device__ __forceinline__ Units units_of(const Dev& a, const E& e) {
  if (!a.pairing) return Units{1, 0, e.mts};
  const int odd = e.mts & 1;
  return Units{odd && e.T * a.G - (e.mts - 1) * a.rt <= a.dual_rows ? 2 : 1, e.mts >> 1, odd};
}
__device__ __forceinline__ int block_heads(const Dev& a, const Units& n, int h) { return h + n.hb <= a.H_kv ? n.hb : 1; }
__device__ __forceinline__ int rest_cost(const Dev& a, int heads) { return heads == 2 ? a.cost_dual : a.cost_single; }
// cost before unit u of a block of so many heads, from its beginning
template <typename E>
__device__ __forceinline__ long long unit_begin(const Dev& a, const E& e, const Units& n, int heads, int u) {
  const int np = heads * n.pairs;
  return min(u, np) * ((long long)a.cost_pair * e.nt + e.cu) +
         max(u - np, 0) * ((long long)rest_cost(a, heads) * e.nt + e.cu);
}
template <typename E>
__device__ __forceinline__ long long block_cost(const Dev& a, const E& e, const Units& n, int heads) {
  return unit_begin(a, e, n, heads, heads * n.pairs + n.rest);
}
template <typename E>
__device__ __forceinline__ long long entry_cost(const Dev& a, const E& e) {
  const Units n = units_of(a, e);
  const long long one = block_cost(a, e, n, n.hb);
  if (n.hb == 1) return one * a.H_kv;
  return one * (a.H_kv >> 1) + ((a.H_kv & 1) ? block_cost(a, e, n, 1) : 0);
}

// The inputs that entries come from, possibly a copy.  Without `ordered` the groups' offsets go backwards somewhere, so
// that groups could overlap: none is worked on then, nor any request.
struct Inputs {
  const int32_t *node, *prefix, *status, *off, *shared;
  bool ordered;
};
__device__ __forceinline__ Inputs inputs_of(const Dev& a, bool ordered) {
  return Inputs{a.node_offset, a.prefix_len, a.req_status, a.group_offset, a.shared_len, ordered};
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

// Whether slots 0 .. end - 1 lie in a table row, and their tiles' bounds in 32 bits.
__device__ __forceinline__ bool fits(const Dev& a, long long end) {
  return (end + a.bs - 1) / a.bs <= a.max_blocks && end <= 0x7fffffffLL - 1024;
}

// Group g's tokens, if it is one that is computed together: two members at least, a shared part, and
// node offsets that lie in [0, N] (a member's own error leaves the others' results as they are).
__device__ __forceinline__ bool group_tokens(const Dev& a, const Inputs& in, int g, int& o, int& T, int& len) {
  const int r0 = in.off[g], r1 = in.off[g + 1];
  len = in.shared[g];
  if (r0 < 0 || r1 > a.B || r1 - r0 < 2 || len <= 0) return false;
  o = in.node[r0];
  const int e = in.node[r1];
  T = e - o;
  return o >= 0 && e <= a.N && T >= 1 && fits(a, len);
}

__device__ __forceinline__ void key_tiles(const Dev& a, Entry& e) {
  e.nt0 = (e.sink + a.bn - 1) / a.bn;
  e.w0 = max(e.lo / a.bn, e.nt0);
  e.nt = e.nt0 + (e.end + a.bn - 1) / a.bn - e.w0;
  e.mts = int(((long long)e.T * a.G + a.rt - 1) / a.rt);
  // tiles that some row does not see whole: the last ones, those at the lower edge, the sinks' last
  const int low = a.window > 0 ? int(max(0LL, (long long)e.P + e.T - a.window)) : e.lo;
  const int masked = (e.end + a.bn - 1) / a.bn - e.P / a.bn + (low + a.bn - 1) / a.bn - e.lo / a.bn + (e.sink % a.bn ? 1 : 0);
  e.cu = a.cost_unit + a.cost_masked * min(masked, e.nt);
}

// Entry i of the stream (groups first).  mts = 0: no work.
// `bad`: SPEC_REQ_* bits that the request gets.  The bits that this library's attention sets itself
// (BAD_BLOCK, TIMEOUT) are ignored, and the others only take away a request's own units, so that all
// roles of all CTAs derive the same stream from the same inputs.
__device__ __forceinline__ Entry entry_of(const Dev& a, const Inputs& in, int i, int& bad) {
  Entry e;
  e.o = e.T = e.P = e.end = e.lo = e.sink = e.nt0 = e.w0 = e.nt = e.mts = e.cu = e.table = 0;
  e.group = -1;
  bad = 0;
  if (i < a.Gn) {
    int o, T, len;
    if (!in.ordered || !group_tokens(a, in, i, o, T, len)) return e;
    e.o = o;
    e.T = T;
    e.P = e.end = len;
    e.table = in.off[i];
    e.group = i;
    key_tiles(a, e);
    return e;
  }
  const int r = i - a.Gn;
  const int o = in.node[r], T = in.node[r + 1] - o, P = in.prefix[r];
  const int st = in.status[r] & ~(SPEC_REQ_BAD_BLOCK | SPEC_REQ_TIMEOUT);
  if (st != 0) return e;
  if (T < 1 || T > a.T_max || P < 0 || o < 0 || o + T > a.N) {
    bad = SPEC_REQ_BAD_SIZE;
    return e;
  }
  const long long end = (long long)P + T;
  if (!fits(a, end)) {
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
    const int g = find_group(in.off, a.Gn, r);
    int go, gT, len;
    if (!in.ordered || g < 0 || in.shared[g] < 0 || in.shared[g] > P) {
      bad = SPEC_REQ_BAD_SIZE;
      e.T = 0;
      return e;
    }
    if (group_tokens(a, in, g, go, gT, len)) {
      if (o < go || o + T > go + gT) {
        bad = SPEC_REQ_BAD_SIZE;
        e.T = 0;
        return e;
      }
      e.lo = len;
      e.group = -2 - g;
    } else if (in.off[g + 1] - in.off[g] >= 2 && in.shared[g] > 0) {   // the group's offsets are bad
      bad = SPEC_REQ_BAD_SIZE;
      e.T = 0;
      return e;
    }
  }
  key_tiles(a, e);
  return e;
}

// The stream of `total` cost units in C ranges: the first `rem` have base + 1 units, the others base.
struct Cut {
  long long base;
  int C, rem;
};
__device__ __forceinline__ long long div_ll(long long a, long long b) {     // a, b >= 0
  return ((a | b) >> 32) == 0 ? (long long)(unsigned(a) / unsigned(b)) : a / b;
}
__device__ __forceinline__ Cut cut_of(const Dev& a, long long total) {
  Cut c;
  c.C = int(max(1LL, min((long long)a.ctas, div_ll(total, a.cost_min))));
  c.base = div_ll(total, c.C);
  c.rem = int(total - c.base * c.C);
  return c;
}
__device__ __forceinline__ long long range_start(const Cut& c, int i) { return i * c.base + min(i, c.rem); }
// the range holding cost position t (0 <= t < total)
__device__ __forceinline__ int range_of(const Cut& c, long long t) {
  const long long head = c.rem * (c.base + 1);
  return t < head ? int(div_ll(t, c.base + 1)) : c.rem + int(div_ll(t - head, max(1LL, c.base)));
}

// A CTA's share: cost positions [t0, t1), from entry e0, before which the cost is beg0.
struct Range {
  long long t0, t1, beg0;
  int e0, C;
  bool ordered;         // of the inputs
};

// Scratch of the search: the warps' costs and the inputs, where they fit.
struct RangeScratch {
  long long sum[32];
  int32_t node[kStartCache + 1], prefix[kStartCache], status[kStartCache], off[kStartCache + 1], shared[kStartCache];
};

__device__ __forceinline__ long long warp_scan(long long v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) >= o) v += x;
  }
  return v;
}

// All threads of the CTA find its range, an entry (or a run of entries) a thread, and `first`, the entry that it
// begins in, where a thread has only one (T = 0 else).  The inputs come in one round trip to memory, not in the
// chain that an entry's checks make of them.  The caller synchronises before it reads R.
__device__ __forceinline__ void find_range(const Dev& a, RangeScratch& s, Range& R, Entry& first) {
  const int E = a.Gn + a.B, nthr = blockDim.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Inputs in = inputs_of(a, true);
  bool back = false;
  if (a.B <= kStartCache) {              // Gn <= B
#pragma unroll 1
    for (int i = threadIdx.x; i <= a.B; i += nthr) {
      const bool r = i < a.B, g = i < a.Gn;
      const int32_t node = in.node[i], prefix = r ? in.prefix[i] : 0, status = r ? in.status[i] : 0;
      const int32_t off = i <= a.Gn && a.Gn > 0 ? in.off[i] : 0, next = g ? in.off[i + 1] : off, shared = g ? in.shared[i] : 0;
      s.node[i] = node;
      if (r) {
        s.prefix[i] = prefix;
        s.status[i] = status;
      }
      s.off[i] = off;
      back = back || off > next;
      if (g) s.shared[i] = shared;
    }
    in = Inputs{s.node, s.prefix, s.status, s.off, s.shared, true};
  } else {
#pragma unroll 1
    for (int i = threadIdx.x; i < a.Gn; i += nthr) back = back || in.off[i] > in.off[i + 1];
  }
  in.ordered = !__syncthreads_or(back);
  const int run = (E + nthr - 1) / nthr, i0 = min(E, int(threadIdx.x) * run), i1 = min(E, i0 + run);
  Entry e;
  e.T = 0;
  long long mine = 0;
#pragma unroll 1
  for (int i = i0; i < i1; ++i) {
    int bad;
    e = entry_of(a, in, i, bad);
    mine += entry_cost(a, e);
  }
  long long lo = warp_scan(mine);
  if (lane == 31) s.sum[warp] = lo;
  __syncthreads();
  lo -= mine;
  long long total = 0;
#pragma unroll 1
  for (int w = 0; w < nthr >> 5; ++w) {
    if (w == warp) lo += total;
    total += s.sum[w];
  }
  const Cut cut = cut_of(a, total);
  const bool none = total == 0 || int(blockIdx.x) >= cut.C;
  const long long t0 = none ? 0 : range_start(cut, blockIdx.x);
  if (none ? threadIdx.x == 0 : lo <= t0 && t0 < lo + mine) {
    int at = i0;
    if (!none && run > 1) {            // which of the thread's entries
#pragma unroll 1
      for (;; ++at) {
        int bad;
        e = entry_of(a, in, at, bad);
        const long long cost = entry_cost(a, e);
        if (t0 < lo + cost || at + 1 >= i1) break;
        lo += cost;
      }
    }
    R.t0 = t0;
    R.t1 = none ? 0 : range_start(cut, blockIdx.x + 1);
    R.beg0 = none ? 0 : lo;
    R.e0 = at;
    R.C = cut.C;
    R.ordered = in.ordered;
    first = e;
  }
}

// One warp of one CTA writes what the merge reads and flags the requests that cannot be worked on.  A CTA
// without a range does it if there is one, else the first.
__device__ __forceinline__ bool reports(const Range& R, int ctas) {
  return int(blockIdx.x) == (R.C < ctas ? ctas - 1 : 0);
}
__device__ __forceinline__ void write_recs(const Dev& a, bool ordered) {
  const int lane = threadIdx.x & 31;
  const Inputs in = inputs_of(a, ordered);
  long long sum = 0;
#pragma unroll 1
  for (int i0 = 0; i0 < a.Gn + a.B; i0 += 32) {
    const int i = i0 + lane;
    long long cost = 0;
    Rec r;
    if (i < a.Gn + a.B) {
      int bad;
      const Entry e = entry_of(a, in, i, bad);
      cost = entry_cost(a, e);
      if (bad) atomicOr(&a.req_status[i - a.Gn], bad);
      r.o = e.o; r.T = e.T; r.nt = e.nt; r.mts = e.mts; r.group = e.group; r.cu = e.cu;
    }
    const long long hi = warp_scan(cost) + sum;
    if (i < a.Gn + a.B) {
      r.beg = hi - cost;
      a.recs[i] = r;
    }
    sum = __shfl_sync(0xffffffffu, hi, 31);
  }
  if (lane == 0) *a.total = sum;
}

// For CTAs that give up at their start: records that leave the merge nothing to do.
__device__ __forceinline__ void clear_recs(const Dev& a) {
  for (int i = threadIdx.x & 31; i < a.Gn + a.B; i += 32) a.recs[i].mts = 0;
}

// Key tiles [j0, j1) of one unit.
enum { kLone, kPair, kDual };
struct Item {
  int o, T, P, end, lo, sink, table, nt0, w0;
  int h, mt, kind;       // first KV head and row tile; one of kLone, kPair, kDual
  int j0, j1;
  int slot;              // >= 0: a piece of a cut unit, to part_o[slot]; -1: to o; -2, -3: to row_o[0], [1]
  int req, nreq;         // the requests that it concerns
  int pad;
};

// Walks the CTA's range, one thread.
struct Walker {
  long long t, ubeg;     // next cost position; cost before the present unit
  long long eend;        // cost up to the entry's end
  int i, h, heads, u;    // entry; first head and heads of the block, unit in the block
  Units n;
  Entry e;
  bool known;            // e is the entry to enter next
  __device__ __forceinline__ void start(const Range& R, const Entry* first) {
    t = R.t0;
    i = R.e0 - 1;
    eend = R.beg0;      // next() enters e0
    known = first != nullptr && first->T > 0;
    if (known) e = *first;
  }
  __device__ __forceinline__ bool next(const Dev& a, const Range& R, Item& it) {
    while (t < R.t1) {
      while (t >= eend) {
        if (++i >= a.Gn + a.B) return false;
        if (!known) {
          int bad;
          e = entry_of(a, inputs_of(a, R.ordered), i, bad);
        }
        known = false;
        n = units_of(a, e);
        ubeg = eend;
        eend += entry_cost(a, e);
        h = u = 0;
        heads = block_heads(a, n, 0);
        if (t > ubeg && t < eend) {          // the range begins inside: the unit that holds t
          const long long bc = block_cost(a, e, n, n.hb);
          const int b = int(min((long long)(a.H_kv / n.hb), div_ll(t - ubeg, bc)));
          h = b * n.hb;
          heads = block_heads(a, n, h);
          ubeg += b * bc;
          const long long in = t - ubeg, rest = unit_begin(a, e, n, heads, heads * n.pairs);
          u = in < rest ? int(div_ll(in, (long long)a.cost_pair * e.nt + e.cu))
                        : heads * n.pairs + int(div_ll(in - rest, (long long)rest_cost(a, heads) * e.nt + e.cu));
          ubeg += unit_begin(a, e, n, heads, u);
        }
      }
      const int np = heads * n.pairs;
      int w = a.cost_pair;
      if (u < np) {
        const int hi = u / n.pairs;
        it.kind = kPair;
        it.h = h + hi;
        it.mt = 2 * (u - hi * n.pairs);
      } else {
        w = rest_cost(a, heads);
        it.kind = heads == 2 ? kDual : kLone;
        it.h = h;
        it.mt = 2 * n.pairs + u - np;
      }
      if (++u == np + n.rest) {
        u = 0;
        h += heads;
        heads = block_heads(a, n, h);
      }
      const long long first = ubeg + e.cu, uend = first + (long long)w * e.nt;      // the first tile's place
      const int j0 = int(max(0LL, div_ll(max(0LL, t - first + w - 1), w)));
      const int j1 = int(min((long long)e.nt, div_ll(max(0LL, R.t1 - first + w - 1), w)));
      t = min(R.t1, uend);
      ubeg = uend;
      if (j1 <= j0) continue;
      it.o = e.o; it.T = e.T; it.P = e.P; it.end = e.end; it.lo = e.lo; it.sink = e.sink;
      it.table = e.table; it.nt0 = e.nt0; it.w0 = e.w0;
      it.j0 = j0;
      it.j1 = j1;
      const bool cut = j0 > 0 || j1 < e.nt;
      it.slot = cut ? 2 * int(blockIdx.x) + (j0 == 0 && first > R.t0 ? 1 : 0)
                    : e.group >= 0 ? -2 : e.group == -1 ? -1 : -3;
      it.req = e.group >= 0 ? e.table : i - a.Gn;
      it.nreq = e.group >= 0 ? a.group_offset[e.group + 1] - it.req : 1;
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

// Word w of a mask row, without the bits behind a tree of T nodes, which count for nothing.
__device__ __forceinline__ uint32_t mask_word(const uint32_t* row, int w, int T) {
  const int n = T - 32 * w;
  return n <= 0 ? 0u : row[w] & (n >= 32 ? ~0u : (1u << n) - 1u);
}

// The ancestor words of one query row under the window, in place: of its n ancestors-or-self (depths 0 .. n - 1
// in increasing index, since parents come before children) those at depth k with n - 1 - k < window or
// P + k < sinks.  Returns the row's lower bound of visible prefix keys.
__device__ __forceinline__ int window_words(const Dev& a, uint32_t* row, int W, int P) {
  int n = 0;
  for (int w = 0; w < W; ++w) n += __popc(row[w]);
  const int first = n > a.window ? n - a.window : 0;       // depths below are out of the window
  const int sunk = a.sinks > P ? a.sinks - P : 0;          // depths below are sinks
  int k = 0;
  for (int w = 0; w < W; ++w) {
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
    row[w] = keep;
  }
  const int depth = n > 0 ? n - 1 : 0;
  const long long lo = (long long)P + depth - a.window + 1;
  return lo > 0 ? int(min(lo, (long long)P)) : 0;
}

// Tensor maps of a call on the tensor cores: q in boxes of a row tile's tokens, of at most T_max tokens and of
// a 16-row unit's tokens; the caches by page and by whole key tiles of consecutive pages.
struct TcMaps {
  CUtensorMap q, q_own, q_rows, k_page, v_page, k_tile, v_tile;
  int q_tokens, q_own_tokens, q_rows_tokens, kv_rows;
};

}  // namespace span
}  // namespace spec
