// spec_tree_attention_shared and spec_tree_attention_window: argument checks, workspaces, the kernel on
// the CUDA cores and the merge of pieces.  attention_span.cuh says how the work is laid out;
// attention_span_tc.cu and attention_span_rows.cu have the kernels on the tensor cores.
//
// Per query row, over its visible keys j: x_j = scale q.k_j, O = sum_j 2^(x_j - M) v_j / sum_j 2^(x_j - M)
// in base 2 (scale holds log2 e), LSE = ln 2 (M + log2 sum).  Pieces of a row merge by the same sums:
// O = sum_p 2^(L_p - M) O_p / sum_p 2^(L_p - M) with L_p the piece's log2-sum-exp.
#include <math.h>

#include "attention_span.cuh"

namespace spec {
namespace span {

// ------------------------------------------------------------------------------ CUDA cores
// Any head_dim up to 256 and any block size, fp32 and bf16.  A CTA takes 32 query rows by 64 keys at a
// time; thread (ty, tx) has rows 2 ty, 2 ty + 1, keys tx + 16 k of the scores and columns 4 tx + 64 c of
// the output, all in fp32.  Bound by its shared-memory reads (6 vectors for 32 multiply-adds of the
// scores).
constexpr int kSimtThreads = 256;
constexpr int kSimtRows = 32;
constexpr int kSimtKeys = 64;

struct SimtShared {
  RangeScratch scratch;
  Range range;
  Entry first;
  Item item;
  int more;
  int page[kSimtKeys];                 // cache row of a key's page row, -1: not needed
  int row_lo[kSimtRows];
  uint32_t anc[kSimtRows][8];
  uint64_t vis[kSimtRows];             // a masked tile's visible keys
  float p[kSimtRows][kSimtKeys + 4];
};

__host__ __device__ constexpr int simt_smem(int d) {
  return int(sizeof(SimtShared)) + 16 + 4 * (kSimtRows * d + 2 * kSimtKeys * (d + 4));
}

template <typename T>
__device__ __forceinline__ float4 load4(const T* p) {
  if constexpr (sizeof(T) == 4) {
    return *reinterpret_cast<const float4*>(p);
  } else {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
  }
}
template <typename T>
__device__ __forceinline__ void store4(T* p, float4 v) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = v;
  } else {
    __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
    uint2 w;
    w.x = *reinterpret_cast<uint32_t*>(&lo);
    w.y = *reinterpret_cast<uint32_t*>(&hi);
    *reinterpret_cast<uint2*>(p) = w;
  }
}

template <typename T>
__global__ void __launch_bounds__(kSimtThreads) span_simt_kernel(Dev a) {
  extern __shared__ uint8_t smem_raw[];
  SimtShared& s = *reinterpret_cast<SimtShared*>(smem_raw);
  float* sq = reinterpret_cast<float*>(smem_raw + ((sizeof(SimtShared) + 15) & ~size_t(15)));
  float* sk = sq + kSimtRows * a.d;
  const int ldk = a.d + 4;
  float* sv = sk + kSimtKeys * ldk;
  pdl_wait();
  pdl_trigger();
  find_range(a, s.scratch, s.range, s.first);
  __syncthreads();
  const Range R = s.range;
  if (threadIdx.x < 32 && reports(R, gridDim.x)) write_recs(a, R.ordered);
  if (R.t0 >= R.t1) return;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int d4 = a.d >> 2;
  const T* q = static_cast<const T*>(a.q);
  const T* kc = static_cast<const T*>(a.k);
  const T* vc = static_cast<const T*>(a.v);
  Walker walker;
  if (tid == 0) walker.start(R, &s.first);
  while (true) {
    if (tid == 0) s.more = walker.next(a, R, s.item) ? 1 : 0;
    __syncthreads();
    if (!s.more) return;
    const Item it = s.item;
    const int rows = min(kSimtRows, it.T * a.G - it.mt * kSimtRows);
    const bool tree = it.end > it.P;
    // the rows' queries, ancestor words and bounds
    for (int i = tid; i < kSimtRows * d4; i += kSimtThreads) {
      const int m = i / d4, c = i - m * d4;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (m < rows) {
        const int row = it.mt * kSimtRows + m, t = row / a.G, g = row - t * a.G;
        x = load4(q + (size_t(it.o + t) * a.H_q + it.h * a.G + g) * a.d + 4 * c);
      }
      reinterpret_cast<float4*>(sq)[m * d4 + c] = x;
    }
    if (tid < kSimtRows) {
      int lo = it.lo;
      for (int w = 0; w < 8; ++w) s.anc[tid][w] = 0;
      if (tid < rows && tree) {
        const uint32_t* arow = a.anc + size_t(it.o + (it.mt * kSimtRows + tid) / a.G) * a.W;
        for (int w = 0; w < a.W; ++w) s.anc[tid][w] = mask_word(arow, w, it.T);
        if (a.window > 0) lo = window_words(a, s.anc[tid], a.W, it.P);
      }
      s.row_lo[tid] = lo;
    }
    const int lo_max = a.window > 0 ? (int)max(0LL, (long long)it.P + it.T - a.window) : it.lo;
    const int32_t* table = a.block_table + size_t(it.table) * a.max_blocks;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    float4 acc[2][4];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[r][c] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = it.j0; j < it.j1; ++j) {
      const int kb = key_base(a, it.nt0, it.w0, j);
      const bool masked = !(kb + kSimtKeys <= it.P && (kb >= lo_max || (a.window > 0 && kb + kSimtKeys <= a.sinks)));
      if (tid < kSimtKeys) {
        const int key = kb + tid;
        int at = -1;
        if (key < it.sink || (key >= it.lo && key < it.end)) {
          const int pb = table[key / a.bs];
          if (pb < 0 || pb >= a.num_blocks) {
            flag(a, it.req, it.nreq, SPEC_REQ_BAD_BLOCK);
          } else {
            at = pb * a.bs * a.H_kv + it.h * a.bs + key % a.bs;   // < num_blocks * bs * H_kv, checked on the host
          }
        }
        s.page[tid] = at;
      }
      __syncthreads();
      for (int i = tid; i < kSimtKeys * d4; i += kSimtThreads) {
        const int n = i / d4, c = i - n * d4;
        const int at = s.page[n];
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
        if (at >= 0) {
          x = load4(kc + size_t(at) * a.d + 4 * c);
          y = load4(vc + size_t(at) * a.d + 4 * c);
        }
        *reinterpret_cast<float4*>(sk + n * ldk + 4 * c) = x;
        *reinterpret_cast<float4*>(sv + n * ldk + 4 * c) = y;
      }
      if (masked && tid < kSimtRows) {
        uint64_t v = 0;
        for (int n = 0; n < kSimtKeys; ++n) {
          const int key = kb + n, t = key - it.P;
          bool b = false;
          if (tid < rows && s.page[n] >= 0) {
            if (t < 0) b = key >= s.row_lo[tid] || (a.window > 0 && key < a.sinks);
            else b = t < 32 * a.W && ((s.anc[tid][t >> 5] >> (t & 31)) & 1u);
          }
          v |= uint64_t(b ? 1 : 0) << n;
        }
        s.vis[tid] = v;
      }
      __syncthreads();
      float x0[4] = {0.f, 0.f, 0.f, 0.f}, x1[4] = {0.f, 0.f, 0.f, 0.f};
      for (int c = 0; c < d4; ++c) {
        const float4 qa = reinterpret_cast<const float4*>(sq)[(2 * ty) * d4 + c];
        const float4 qb = reinterpret_cast<const float4*>(sq)[(2 * ty + 1) * d4 + c];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float4 kv = *reinterpret_cast<const float4*>(sk + (tx + 16 * k) * ldk + 4 * c);
          x0[k] = fmaf(qa.x, kv.x, x0[k]); x0[k] = fmaf(qa.y, kv.y, x0[k]);
          x0[k] = fmaf(qa.z, kv.z, x0[k]); x0[k] = fmaf(qa.w, kv.w, x0[k]);
          x1[k] = fmaf(qb.x, kv.x, x1[k]); x1[k] = fmaf(qb.y, kv.y, x1[k]);
          x1[k] = fmaf(qb.z, kv.z, x1[k]); x1[k] = fmaf(qb.w, kv.w, x1[k]);
        }
      }
      const uint64_t v0 = masked ? s.vis[2 * ty] : ~0ull, v1 = masked ? s.vis[2 * ty + 1] : ~0ull;
      float c0 = -INFINITY, c1 = -INFINITY;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        x0[k] = (v0 >> (tx + 16 * k)) & 1 ? x0[k] * a.scale_log2 : -INFINITY;
        x1[k] = (v1 >> (tx + 16 * k)) & 1 ? x1[k] * a.scale_log2 : -INFINITY;
        c0 = fmaxf(c0, x0[k]);
        c1 = fmaxf(c1, x1[k]);
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) {
        c0 = fmaxf(c0, __shfl_xor_sync(0xffffffffu, c0, o));
        c1 = fmaxf(c1, __shfl_xor_sync(0xffffffffu, c1, o));
      }
      const float n0 = fmaxf(m0, c0), n1 = fmaxf(m1, c1);
      const float f0 = m0 == -INFINITY ? 0.f : exp2f(m0 - n0), f1 = m1 == -INFINITY ? 0.f : exp2f(m1 - n1);
      float s0 = 0.f, s1 = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        // a masked score is -inf: weight 0, also while the row has seen nothing (its reference is -inf)
        const float p0 = (v0 >> (tx + 16 * k)) & 1 ? exp2f(x0[k] - n0) : 0.f;
        const float p1 = (v1 >> (tx + 16 * k)) & 1 ? exp2f(x1[k] - n1) : 0.f;
        s.p[2 * ty][tx + 16 * k] = p0;
        s.p[2 * ty + 1][tx + 16 * k] = p1;
        s0 += p0;
        s1 += p1;
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) {
        s0 += __shfl_xor_sync(0xffffffffu, s0, o);
        s1 += __shfl_xor_sync(0xffffffffu, s1, o);
      }
      l0 = l0 * f0 + s0;
      l1 = l1 * f1 + s1;
      m0 = n0;
      m1 = n1;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        acc[0][c].x *= f0; acc[0][c].y *= f0; acc[0][c].z *= f0; acc[0][c].w *= f0;
        acc[1][c].x *= f1; acc[1][c].y *= f1; acc[1][c].z *= f1; acc[1][c].w *= f1;
      }
      __syncwarp();   // a row's weights come from its own half warp
      for (int n = 0; n < kSimtKeys; ++n) {
        const float p0 = s.p[2 * ty][n], p1 = s.p[2 * ty + 1][n];
        const bool b0 = (v0 >> n) & 1, b1 = (v1 >> n) & 1;   // a masked NaN must not reach the row
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int col = 4 * tx + 64 * c;
          if (col >= a.d) continue;
          const float4 v = *reinterpret_cast<const float4*>(sv + n * ldk + col);
          if (b0) {
            acc[0][c].x = fmaf(p0, v.x, acc[0][c].x); acc[0][c].y = fmaf(p0, v.y, acc[0][c].y);
            acc[0][c].z = fmaf(p0, v.z, acc[0][c].z); acc[0][c].w = fmaf(p0, v.w, acc[0][c].w);
          }
          if (b1) {
            acc[1][c].x = fmaf(p1, v.x, acc[1][c].x); acc[1][c].y = fmaf(p1, v.y, acc[1][c].y);
            acc[1][c].z = fmaf(p1, v.z, acc[1][c].z); acc[1][c].w = fmaf(p1, v.w, acc[1][c].w);
          }
        }
      }
      __syncthreads();   // sk, sv and page are rewritten
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int m = 2 * ty + r;
      if (m >= rows) continue;
      const float l = r == 0 ? l0 : l1, M = r == 0 ? m0 : m1;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const float lse2 = l == 0.f ? -INFINITY : M + log2f(l);
      const int row = it.mt * kSimtRows + m, t = row / a.G, g = row - t * a.G;
      const size_t out = size_t(it.o + t) * a.H_q + it.h * a.G + g;
      float* part = nullptr;
      float* plse = nullptr;
      if (it.slot >= 0) {
        part = a.part_o + (size_t(it.slot) * a.part_rows + m) * a.d;
        plse = a.part_lse + size_t(it.slot) * a.part_rows + m;
      } else if (it.slot < -1) {
        const size_t at = size_t(it.slot == -2 ? 0 : 1) * a.N * a.H_q + out;
        part = a.row_o + at * a.d;
        plse = a.row_lse + at;
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int col = 4 * tx + 64 * c;
        if (col >= a.d) continue;
        const float4 v = make_float4(acc[r][c].x * inv, acc[r][c].y * inv, acc[r][c].z * inv, acc[r][c].w * inv);
        if (part) *reinterpret_cast<float4*>(part + col) = v;
        else store4(static_cast<T*>(a.o) + out * a.d + col, v);
      }
      if (tx == 0) {
        if (plse) *plse = lse2;
        else if (a.lse) a.lse[out] = lse2 * 0.6931471805599453f;
      }
    }
    __syncthreads();   // the item and the rows' words are rewritten
  }
}

// ------------------------------------------------------------------------------ merge
// CTA (r, h, z): rows kMergeRows z .. of request r under KV head h, kR rows a warp at a time.  A row's pieces:
// for a member of a group those of the group's unit, then those of its request's own unit, in stream order, so
// that the sum does not depend on who ran when.  Rows of requests on their own whose unit was not cut have been
// written already.  A piece's log-sum-exp is one fp32 number: at 2^k it weighs pieces to 2^(k - 24), which scores of
// thousands do not show.  Lane kR p + i holds the weight and the place of piece p (of 32 / kR at a time) of row i.
// Bound by a chain of loads (record, group's record, log-sum-exps, values), so rows that share the first two
// are taken by one CTA, two at a time (many rows: 32 trees under a window of 2048 95 us in all, 101 by one row a
// time), and a warp takes one row where there are few: 16 rows or less a request and head.
constexpr int kMergeFew = 16;
constexpr int kMergeRows = 32;

struct Pieces {
  int np, ca, slot0;        // np = 1: not cut
  int row;                  // of a slot, where the row tile begins
};
__device__ __forceinline__ Pieces pieces_of(const Dev& a, const Rec& e, const Cut& cut, int h, int mt) {
  const Units n = units_of(a, e);
  const int b = n.hb == 2 ? h >> 1 : h, heads = block_heads(a, n, b * n.hb), in = h - b * n.hb;
  const bool pair = mt < 2 * n.pairs;
  const int u = pair ? in * n.pairs + (mt >> 1) : heads * n.pairs + mt - 2 * n.pairs;
  const int w = pair ? a.cost_pair : rest_cost(a, heads);
  const int second = pair ? mt & 1 : heads == 2 ? in : 0;
  const long long first = e.beg + b * block_cost(a, e, n, n.hb) + unit_begin(a, e, n, heads, u) + e.cu;
  Pieces p;
  p.ca = range_of(cut, first);
  p.np = range_of(cut, first + (long long)(e.nt - 1) * w) - p.ca + 1;
  p.slot0 = 2 * p.ca + (first > range_start(cut, p.ca) ? 1 : 0);
  p.row = second * (a.part_rows / 2);
  return p;
}

template <typename T, int kR, int kCols>      // kCols: vectors of 128 columns of a row
__global__ void __launch_bounds__(256, kCols > 1 ? 2 : 4) span_merge_kernel(Dev a) {
  constexpr int kP = 32 / kR, kLoads = 4;      // pieces a round, vectors loaded together
  constexpr int kBatch = kLoads / kR;
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.x, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Rec own = a.recs[a.Gn + r];
  const long long total = *a.total;
  const int nrows = own.T * a.G;
  const int last = min(nrows, (int(blockIdx.z) + 1) * kMergeRows);
  if (own.mts == 0 || int(blockIdx.z) * kMergeRows + warp * kR >= last) return;
  const Cut cut = cut_of(a, total);
  const int g = own.group < -1 ? -2 - own.group : -1;
  Rec grp;
  if (g >= 0) grp = a.recs[g];
  const int i = lane % kR;
  Pieces po, pg;
  int mt_seen = -1, gmt_seen = -1;
#pragma unroll 1
  for (int m0 = int(blockIdx.z) * kMergeRows + warp * kR; m0 < last; m0 += 8 * kR) {
    // this lane's row and piece
    const int m = min(m0 + i, nrows - 1);
    const int mt = m / a.rt;
    if (mt != mt_seen) po = pieces_of(a, own, cut, h, mt);
    mt_seen = mt;
    if (g < 0 && !__any_sync(0xffffffffu, po.np > 1)) continue;
    const int t = m / a.G;
    const size_t out = size_t(own.o + t) * a.H_q + h * a.G + (m - t * a.G);
    // row of a piece's slot
    const int oc = m - mt * a.rt + po.row;
    int gc = 0, ng = 0;
    if (g >= 0) {
      const int gm = (own.o - grp.o) * a.G + m, gmt = gm / a.rt;
      if (gmt != gmt_seen) pg = pieces_of(a, grp, cut, h, gmt);
      gmt_seen = gmt;
      gc = gm - gmt * a.rt + pg.row;
      ng = pg.np;
    }
    const bool mine = m0 + i < last && (g >= 0 || po.np > 1);
    const int n = mine ? ng + po.np : 0;
    int most = n;
#pragma unroll
    for (int o = kR / 2; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
    // place of piece p of this lane's row, in rows of d values; bit 63: among row_o
    auto where = [&](int p) -> unsigned long long {
      const bool isg = p < ng;
      const int k = isg ? p : p - ng, np = isg ? pg.np : po.np;
      if (np == 1) return (1ULL << 63) | (size_t(isg ? 0 : 1) * a.N * a.H_q + out);
      return size_t(k == 0 ? (isg ? pg.slot0 : po.slot0) : 2 * ((isg ? pg.ca : po.ca) + k)) * a.part_rows + (isg ? gc : oc);
    };
    auto lse_at = [&](unsigned long long at) { return (at >> 63) ? a.row_lse[at & ~(1ULL << 63)] : a.part_lse[at]; };
    auto row_at = [&](unsigned long long at) {
      return reinterpret_cast<unsigned long long>((at >> 63) ? a.row_o + (at & ~(1ULL << 63)) * a.d : a.part_o + at * a.d);
    };
    // values of kBatch pieces from q0 of the round; a piece that the row does not have: zeros
    unsigned long long src = 0;
    float4 v[kLoads][kCols];
    auto load = [&](int q0) {
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        const int q = q0 + u / kR;
        const float* o = reinterpret_cast<const float*>(__shfl_sync(0xffffffffu, src, min(q, kP - 1) * kR + u % kR));
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          const int col = 4 * lane + 128 * c;
          v[u][c] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (o && q < kP && col < a.d) v[u][c] = *reinterpret_cast<const float4*>(o + col);
        }
      }
    };
    // the first pieces' values and the log-sum-exps are on their way together
    float M = -INFINITY, L0 = -INFINITY;
    if (lane / kR < n) {
      const unsigned long long at = where(lane / kR);
      M = L0 = lse_at(at);
      src = row_at(at);
    }
    load(0);
    for (int p = lane / kR + kP; p < n; p += kP) M = fmaxf(M, lse_at(where(p)));
#pragma unroll
    for (int o = kR; o < 32; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float sum = 0.f;
    float4 acc[kR][kCols];
#pragma unroll
    for (int k = 0; k < kR; ++k)
#pragma unroll
      for (int c = 0; c < kCols; ++c) acc[k][c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int p0 = 0; p0 < most; p0 += kP) {
      if (p0 > 0) {
        const int p = p0 + lane / kR;
        L0 = -INFINITY;
        src = 0;
        if (p < n) {
          const unsigned long long at = where(p);
          L0 = lse_at(at);
          src = row_at(at);
        }
      }
      // -1: nothing visible in this piece (M may be -inf as well), and what it holds does not count, not even a NaN
      const float wt = L0 == -INFINITY ? -1.f : exp2f(L0 - M);
      sum += wt < 0.f ? 0.f : wt;
      const int np = min(kP, most - p0);
#pragma unroll 1
      for (int q0 = 0; q0 < np; q0 += kBatch) {
        if (p0 + q0 > 0) load(q0);
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
          const int q = q0 + u / kR;
          const float w = __shfl_sync(0xffffffffu, wt, min(q, kP - 1) * kR + u % kR);
          if (w < 0.f || q >= np) continue;
#pragma unroll
          for (int c = 0; c < kCols; ++c) {
            float4& x = acc[u % kR][c];
            x.x = fmaf(w, v[u][c].x, x.x); x.y = fmaf(w, v[u][c].y, x.y);
            x.z = fmaf(w, v[u][c].z, x.z); x.w = fmaf(w, v[u][c].w, x.w);
          }
        }
      }
    }
#pragma unroll
    for (int o = kR; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int k = 0; k < kR; ++k) {
      const float f = __shfl_sync(0xffffffffu, inv, k);
      const unsigned long long at = __shfl_sync(0xffffffffu, (unsigned long long)out, k);
      if (!__shfl_sync(0xffffffffu, mine ? 1 : 0, k)) continue;
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        const int col = 4 * lane + 128 * c;
        if (col < a.d)
          store4(static_cast<T*>(a.o) + at * a.d + col,
                 make_float4(acc[k][c].x * f, acc[k][c].y * f, acc[k][c].z * f, acc[k][c].w * f));
      }
    }
    if (mine && lane < kR && a.lse) a.lse[out] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * 0.6931471805599453f;
  }
}

template <typename T>
static spec_status_t launch_merge(const Dev& a, cudaStream_t s) {
  const long long rows = (long long)a.T_max * a.G;
  const dim3 grid(a.B, a.H_kv, unsigned((rows + kMergeRows - 1) / kMergeRows));
  const bool few = rows <= kMergeFew, wide = a.d > 128;
  return launch_result(launch_pdl(few ? (wide ? span_merge_kernel<T, 1, 2> : span_merge_kernel<T, 1, 1>)
                                      : (wide ? span_merge_kernel<T, 2, 2> : span_merge_kernel<T, 2, 1>),
                                  grid, dim3(256), 0, s, a));
}

// ------------------------------------------------------------------------------ host
// Costs on the tensor cores, about 660 clocks each: measured, a key tile takes a pair unit 2650 clocks, two
// heads' a dual one 4000, one a lone one 2000, a unit's start and end 9000, and a tile under a mask 2500 more.
constexpr int kPairCost = 4, kDualCost = 6, kSingleCost = 3, kUnitCost = 14, kMaskedCost = 4, kMinCost = 16;
// The rows kernel's: a tile, a unit, a range.
// (a range of one unit with a tile or two: 1 token, window 1024 17.5 us, 18.7 with a minimum of 8)
constexpr int kRowsTileCost = 2, kRowsUnitCost = 2, kRowsMinCost = 6;
constexpr int kDualRows = 32;
constexpr int kFewRows = 16;       // query rows of a unit up to which the rows kernel takes it

// What the two calls have in common.
struct Args {
  const spec_attn_params* p;
  const int32_t* group_offset;
  const int32_t* shared_len;
  int num_groups, window, sinks;
};

bool tc_takes(const spec_attn_params* p);
int tc_row_tile(const spec_attn_params* p);
spec_status_t make_tc_maps(const spec_attn_params* p, TcMaps& m);
spec_status_t launch_span_tc(const Dev& d, const TcMaps& m, cudaStream_t s);
spec_status_t launch_span_rows(const Dev& d, const TcMaps& m, cudaStream_t s);

static spec_status_t check(const Args& x) {
  const spec_attn_params* p = x.p;
  if (p->dtype != SPEC_F32 && p->dtype != SPEC_BF16) return SPEC_ERR_INVALID_ARG;
  if (p->B < 1 || p->N < 0 || p->T_max < 1 || p->T_max > SPEC_MAX_TREE) return SPEC_ERR_INVALID_ARG;
  if (p->H_q < 1 || p->H_kv < 1 || p->H_q % p->H_kv || p->head_dim < 1 || p->block_size < 1 ||
      p->num_blocks < 1 || p->max_blocks_per_req < 1)
    return SPEC_ERR_INVALID_ARG;
  if (!(p->scale == p->scale) || isinf(p->scale)) return SPEC_ERR_INVALID_ARG;
  if (!p->block_table || !p->prefix_len || !p->node_offset || !p->req_status)
    return SPEC_ERR_INVALID_ARG;
  if (p->N > 0 && (!p->q || !p->k_cache || !p->v_cache || !p->o || !p->anc_mask))
    return SPEC_ERR_INVALID_ARG;
  if (p->N > 0 && (!aligned16(p->q) || !aligned16(p->k_cache) || !aligned16(p->v_cache) ||
                   !aligned16(p->o)))
    return SPEC_ERR_INVALID_ARG;
  const int es = p->dtype == SPEC_BF16 ? 2 : 4;
  if ((p->head_dim * es) % 16) return SPEC_ERR_INVALID_ARG;
  if (p->head_dim > 256) return SPEC_ERR_UNSUPPORTED;
  if ((long long)p->num_blocks * p->H_kv * p->block_size + 256 >= (1LL << 31)) return SPEC_ERR_UNSUPPORTED;
  if ((long long)p->N * p->H_q >= (1LL << 31) || p->H_kv > 65535) return SPEC_ERR_UNSUPPORTED;
  // the merge's grid
  if ((long long)p->T_max * (p->H_q / p->H_kv) > 65535LL * kMergeRows) return SPEC_ERR_UNSUPPORTED;
  return SPEC_OK;
}

// The kernel of a call: on the tensor cores the rows kernel for windows over at most 16 query rows a request
// and head (64 single tokens, 64 query heads on 8, window 4096: 171 us against 191 by the tile kernel; one
// token, window 1024: 17.5 against 25), else the tile kernel, which also takes a shared call's few-rowed requests
// beside their groups (8 groups of 8 single tokens, 32 heads on 8, 8192 shared: 94 us, 84 now; by one kernel for
// the groups and then the other 112); the CUDA-core kernel for everything else.
enum Kernel { kSimt, kTile, kFew };
struct Plan {
  Kernel kernel;
  int ctas, rt, bn, part_rows;
  size_t recs, sum, part_o, part_lse, row_o, row_lse, total;
};

static Plan plan(const Args& x) {
  const spec_attn_params* p = x.p;
  Plan w;
  const int sms = sm_count_current_device();
  const size_t d = size_t(p->head_dim), rows = size_t(p->N) * p->H_q;
  const bool few = x.num_groups == 0 && (long long)p->T_max * (p->H_q / p->H_kv) <= kFewRows;
  w.kernel = !tc_takes(p) ? kSimt : few ? kFew : kTile;
  w.ctas = sms;
  if (w.kernel == kSimt) {
    w.ctas = sms * (p->head_dim <= 64 ? 3 : p->head_dim <= 128 ? 2 : 1);   // resident at once
    w.rt = w.part_rows = kSimtRows;
    w.bn = kSimtKeys;
  } else if (w.kernel == kTile) {
    w.rt = tc_row_tile(p);
    w.bn = 128;
    w.part_rows = 256;
  } else {
    w.rt = w.part_rows = kFewRows;
    w.bn = 128;
  }
  if (w.ctas > kMaxCtas) w.ctas = kMaxCtas;
  size_t off = 0;
  w.recs = off; off = align_up(off + sizeof(Rec) * (size_t(x.num_groups) + p->B), 256);
  w.sum = off; off += 256;
  w.part_o = off; off = align_up(off + sizeof(float) * 2 * w.ctas * w.part_rows * d, 256);
  w.part_lse = off; off = align_up(off + sizeof(float) * 2 * w.ctas * w.part_rows, 256);
  w.row_o = w.row_lse = off;
  if (x.num_groups > 0) {
    w.row_o = off; off = align_up(off + sizeof(float) * 2 * rows * d, 256);
    w.row_lse = off; off = align_up(off + sizeof(float) * 2 * rows, 256);
  }
  w.total = off;
  return w;
}

static spec_status_t launch(const Args& x, void* ws, size_t ws_bytes, cudaStream_t s) {
  const spec_attn_params* p = x.p;
  const Plan w = plan(x);
  if (w.ctas <= 0) return SPEC_ERR_CUDA;
  if (!ws || ws_bytes < w.total || (reinterpret_cast<uintptr_t>(ws) & 255u)) return SPEC_ERR_INVALID_ARG;
  char* base = static_cast<char*>(ws);
  Dev d{};
  d.block_table = p->block_table;
  d.prefix_len = p->prefix_len;
  d.node_offset = p->node_offset;
  d.anc = p->anc_mask;
  d.group_offset = x.group_offset;
  d.shared_len = x.shared_len;
  d.q = p->q; d.k = p->k_cache; d.v = p->v_cache; d.o = p->o;
  d.lse = p->lse;
  d.req_status = p->req_status;
  d.recs = reinterpret_cast<Rec*>(base + w.recs);
  d.total = reinterpret_cast<long long*>(base + w.sum);
  d.part_o = reinterpret_cast<float*>(base + w.part_o);
  d.part_lse = reinterpret_cast<float*>(base + w.part_lse);
  d.row_o = reinterpret_cast<float*>(base + w.row_o);
  d.row_lse = reinterpret_cast<float*>(base + w.row_lse);
  d.B = p->B; d.N = p->N; d.Gn = x.num_groups; d.H_q = p->H_q; d.H_kv = p->H_kv; d.G = p->H_q / p->H_kv;
  d.d = p->head_dim; d.bs = p->block_size; d.T_max = p->T_max; d.W = (p->T_max + 31) / 32;
  d.num_blocks = p->num_blocks; d.max_blocks = p->max_blocks_per_req; d.ctas = w.ctas;
  d.window = x.window; d.sinks = x.sinks;
  d.rt = w.rt; d.bn = w.bn; d.part_rows = w.part_rows; d.pairing = w.kernel == kTile ? 1 : 0;
  // Two heads share a unit where its rows are few, its start, join and end then being most of it, and there are
  // requests enough for every CTA (64 single tokens, 32 heads on 8, 8192 shared by groups of 8: 83 us against 94);
  // not where the row tiles are fuller (32 trees, shared 8192: 169 against 166) or CTAs idle (4 requests: 26
  // against 23).
  d.dual_rows = (long long)p->B * p->H_kv >= 2LL * w.ctas ? kDualRows : 0;
  d.cost_pair = kPairCost;
  d.cost_dual = kDualCost;
  d.cost_single = w.kernel == kTile ? kSingleCost : w.kernel == kFew ? kRowsTileCost : 1;
  d.cost_unit = w.kernel == kTile ? kUnitCost : w.kernel == kFew ? kRowsUnitCost : 0;
  d.cost_masked = w.kernel == kTile ? kMaskedCost : 0;
  // CUDA cores: single tiles (3 requests of 9 fp32 tokens over 20 slots 28 us, 89 by ranges of four at least)
  d.cost_min = w.kernel == kTile ? kMinCost : w.kernel == kFew ? kRowsMinCost : 1;
  const float scale = p->scale > 0.f ? p->scale : 1.f / sqrtf(float(p->head_dim));
  d.scale_log2 = scale * 1.4426950408889634f;
  const bool bf16 = p->dtype == SPEC_BF16;
  spec_status_t st;
  if (w.kernel == kSimt) {
    static DeviceOnce raised_f32, raised_bf16;
    st = bf16 ? raise_dyn_smem_once(span_simt_kernel<__nv_bfloat16>, simt_smem(256), raised_bf16)
              : raise_dyn_smem_once(span_simt_kernel<float>, simt_smem(256), raised_f32);
    if (st == SPEC_OK)
      st = launch_result(launch_pdl(bf16 ? span_simt_kernel<__nv_bfloat16> : span_simt_kernel<float>,
                                    dim3(w.ctas), dim3(kSimtThreads), size_t(simt_smem(p->head_dim)), s, d));
  } else {
    TcMaps m;
    st = make_tc_maps(p, m);
    if (st == SPEC_OK) st = w.kernel == kFew ? launch_span_rows(d, m, s) : launch_span_tc(d, m, s);
  }
  if (st != SPEC_OK) return st;
  return bf16 ? launch_merge<__nv_bfloat16>(d, s) : launch_merge<float>(d, s);
}

static bool window_args(const spec_attn_window_params* p, Args& x) {
  if (!p || p->window < 1 || p->sinks < 0) return false;
  x = Args{&p->attn, nullptr, nullptr, 0, p->window, p->sinks};
  return true;
}
static bool shared_args(const spec_attn_shared_params* p, Args& x) {
  if (!p || p->num_groups < 1 || p->num_groups > p->attn.B || !p->group_offset || !p->shared_len) return false;
  x = Args{&p->attn, p->group_offset, p->shared_len, p->num_groups, 0, 0};
  return true;
}

}  // namespace span
}  // namespace spec

extern "C" {

size_t spec_attention_window_workspace_size(const spec_attn_window_params* p) {
  spec::span::Args x;
  if (!spec::span::window_args(p, x) || spec::span::check(x) != SPEC_OK) return 0;
  return spec::span::plan(x).total;
}

spec_status_t spec_tree_attention_window(const spec_attn_window_params* p, void* workspace,
                                         size_t ws_bytes, spec_stream_t stream) {
  spec::span::Args x;
  if (!spec::span::window_args(p, x)) return SPEC_ERR_INVALID_ARG;
  const spec_status_t st = spec::span::check(x);
  if (st != SPEC_OK || p->attn.N == 0) return st;
  return spec::span::launch(x, workspace, ws_bytes, (cudaStream_t)stream);
}

size_t spec_attention_shared_workspace_size(const spec_attn_shared_params* p) {
  spec::span::Args x;
  if (!spec::span::shared_args(p, x) || spec::span::check(x) != SPEC_OK) return 0;
  return spec::span::plan(x).total;
}

spec_status_t spec_tree_attention_shared(const spec_attn_shared_params* p, void* workspace,
                                         size_t ws_bytes, spec_stream_t stream) {
  spec::span::Args x;
  if (!spec::span::shared_args(p, x)) return SPEC_ERR_INVALID_ARG;
  const spec_status_t st = spec::span::check(x);
  if (st != SPEC_OK || p->attn.N == 0) return st;
  return spec::span::launch(x, workspace, ws_bytes, (cudaStream_t)stream);
}

}  // extern "C"
