// spec_beam_select: the best W of W x V continuations of each request; spec_beam_reorder: the paged cache
// follows the choice.
//
// Within a beam the rank is increasing in the logit, so a beam's W best tokens suffice, and they and the
// log-sum-exp come out of one pass over its row.
//   beam_rows_kernel  one CTA per (segment, row): every thread keeps the running maximum and sum of its
//                     elements (2^(x k2 - ref), k2 = log2 e / tau) and nothing else.  The W-th largest of
//                     the maxima of 32 groups of eight threads is a lower bound of the segment's W-th largest
//                     element, so only the few threads whose maximum reaches it hold candidates: their
//                     elements are read once more (they are still in L2; looked for by the second
//                     kernel, they made the whole take 63 us where it took 45 at the time), a warp for each such thread,
//                     and the elements that reach the bound are ranked by counting.  No list is kept while
//                     the row streams by.
//   beam_pick_kernel  one CTA per request: the beams' candidates ranked by (score + log p) / penalty in
//                     fp64, ties by beam and token.
// Bound by the rows' bytes when there are many rows (64 x 8 rows of 152064 bf16: 36.6 us, 4.3 TB/s), by two
// launches and the chain load -> maxima -> candidates when there are few (1 x 4 rows of 32000: 8.4 us; 16 x 5 of
// 128256 fp32: 17.8 us); few rows are cut in segments.
//
// Ranks of different beams meet in one list, so log p has to be good.  References are whole numbers (the
// maximum of x k2, rounded up), so that sums over threads and segments join by exact powers of two; log p =
// (x k2 - ref - log2 sum) ln 2 has the sum's error (about 1e-7: fp32 sums of a few hundred terms a thread, twice
// that precision beyond) and a relative 2^-25 of k2's rounding, whatever the logits' size: where the largest one, times
// k2, is 2^31 or more, the next ones in the type's order are 64 and more below it and weigh nothing beside it, so the sum is how
// often it occurs, and logits enter log p by their difference from it.
#include <math.h>

#include "common.cuh"

namespace spec {
namespace beam {

constexpr int kRowThreads = 256;           // 32 groups of eight
constexpr int kUnroll = 2;                 // 16-byte loads in flight per thread
constexpr int kList = 512;                 // candidates of a segment; more only where logits tie
constexpr int kPickThreads = 256;
static_assert(SPEC_MAX_BEAMS * SPEC_MAX_BEAMS <= kPickThreads && 16 * SPEC_MAX_BEAMS <= kPickThreads, "a thread per candidate, 16 per beam");
static_assert(SPEC_MAX_BEAMS <= 32, "as many groups as beams at least");
constexpr int kMaxSegLists = 64;           // segments x W
constexpr float kNoRef = -3.0e38f;         // reference of elements that are all -infinity

// log2 and a power in fp64 to about 1e-9, with few fp64 operations (a pow() takes 9 us of a request's
// latency here, these 1): z = 2^e (1 + s) / (1 - s), log2 z = e + 2 / ln 2 (s + s^3 / 3 + ..), |s| <= 0.2; terms
// from the second on are at most 0.014 of the first and are formed in fp32.
__device__ __forceinline__ double log2_of(double z) {          // finite, positive, normal
  const long long b = __double_as_longlong(z);
  int e = int(b >> 52) - 1023;
  double f = __longlong_as_double((b & 0xfffffffffffffLL) | 0x3ff0000000000000LL);
  if (f > 1.5) {
    f *= 0.5;
    ++e;
  }
  const double d = f + 1.0;
  double r = double(__frcp_rn(float(d)));
  r = r * (2.0 - d * r);                                        // one Newton step: 2^-46
  const double s = (f - 1.0) * r;
  const float q = float(s) * float(s);
  float t = 1.f / 15.f;
  t = fmaf(t, q, 1.f / 13.f); t = fmaf(t, q, 1.f / 11.f); t = fmaf(t, q, 1.f / 9.f);
  t = fmaf(t, q, 1.f / 7.f); t = fmaf(t, q, 1.f / 5.f); t = fmaf(t, q, 1.f / 3.f);
  return double(e) + 2.8853900817779268 * (s + s * double(t * q));
}
// 2^w = 2^n e^g, |g| <= ln 2 / 2, by the exponential series; terms from the third on in fp32
__device__ __forceinline__ double exp2_of(double w) {           // |w| < 1000
  const double n = rint(w), g = (w - n) * 0.693147180559945309417;
  const float h = float(g);
  float t = 1.f / 40320.f;
  t = fmaf(t, h, 1.f / 5040.f); t = fmaf(t, h, 1.f / 720.f); t = fmaf(t, h, 1.f / 120.f);
  t = fmaf(t, h, 1.f / 24.f); t = fmaf(t, h, 1.f / 6.f);
  const double y = 1.0 + g + g * g * (0.5 + double(t * h));
  return y * __longlong_as_double((long long)(1023 + int(n)) << 52);
}

struct Seg {
  dfloat sum;        // sum of 2^(x k2 - ref)
  float ref;
  int count;         // candidates; + kCoarseSeg: ref is the largest logit, which is coarse, and sum how often it occurs
};
constexpr int kCoarseSeg = 256;
// What stands for a part's largest logit where parts join: itself if it is coarse, 0 for others, -infinity for none.
// Coarse ones beside a larger one count for nothing.

struct SelectDev {
  const void* logits;
  const float* scores;
  const int32_t* lengths;
  const int32_t* finished;
  int32_t* parent;
  int32_t* token;
  float* out_score;
  int32_t* out_length;
  int32_t* out_finished;
  Seg* seg;          // [rows][S]
  float* cand_v;     // [rows][S][W]
  int32_t* cand_id;
  int64_t ld;
  int W, V, S, seg_vecs, eos;   // seg_vecs: 16-byte vectors of a segment
  float k2, coarse;             // coarse: logits of that magnitude and more are told apart by themselves, not by x k2
  double alpha;
};
// a finite or +infinite maximum that is; its row's sum is a count
__device__ __forceinline__ bool is_coarse(const SelectDev& a, float m) { return fabsf(m) >= a.coarse && m > -INFINITY; }

__device__ __forceinline__ bool ahead(float v, int id, float w, int jd) { return v > w || (v == w && id < jd); }

// a 16-byte vector's elements, those past V as -inf
template <typename T>
__device__ __forceinline__ void elements(const uint4& x, int first, int V, float* out) {
  elem<T>::unpack(x, out);
  if (first + elem<T>::per16 > V) {
#pragma unroll
    for (int k = 0; k < elem<T>::per16; ++k)
      if (first + k >= V) out[k] = -INFINITY;
  }
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads) beam_rows_kernel(SelectDev a) {
  constexpr int kE = elem<T>::per16;
  constexpr int kWarps = kRowThreads / 32;
  __shared__ float s_group[32], s_ref[kWarps], s_max[kWarps], s_v[kList], s_bv[kWarps];
  __shared__ dfloat s_sum[kWarps];
  __shared__ int s_id[kList], s_hot[kRowThreads], s_bi[kWarps];
  __shared__ int s_n, s_nhot;
  pdl_wait();
  pdl_trigger();
  const int row = blockIdx.y, sg = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const T* src = static_cast<const T*>(a.logits) + size_t(row) * a.ld;
  const int nvec = (a.V + kE - 1) / kE;
  const int v0 = sg * a.seg_vecs, v1 = min(nvec, v0 + a.seg_vecs);
  uint4 raw[kUnroll];
  auto fetch = [&](int b) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int v = b + u * kRowThreads;
      if (v < v1) raw[u] = ld_stream16(src + size_t(v) * kE);
    }
  };
  const int fin = a.finished[row];
  const float score = a.scores[row];
  fetch(v0 + tid);
  // a beam that offers no token of its row: nothing more of it is read
  if (fin != 0 || !(score > -INFINITY)) return;
  if (tid == 0) s_n = s_nhot = 0;
  float m = -INFINITY, ref = kNoRef, sum = 0.f;
  const uint64_t k2v = f2_pack(a.k2, a.k2);
  for (int b = v0 + tid; b < v1; b += kUnroll * kRowThreads) {
    float x[kUnroll * kE];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int v = b + u * kRowThreads;
      if (v < v1) {
        elements<T>(raw[u], v * kE, a.V, x + u * kE);
      } else {
#pragma unroll
        for (int k = 0; k < kE; ++k) x[u * kE + k] = -INFINITY;
      }
    }
    fetch(b + kUnroll * kRowThreads);
    float cm = x[0];
#pragma unroll
    for (int k = 1; k + 1 < kUnroll * kE; k += 2) cm = fmax3(cm, x[k], x[k + 1]);
    cm = fmaxf(cm, x[kUnroll * kE - 1]);
    if (cm > m) {
      m = cm;
      const float to = ceilf(cm * a.k2);
      if (!(fabsf(cm) < a.coarse)) {
        sum = sum != sum ? sum : 0.f;                        // what came before is nothing beside it
      } else if (to > ref) {
        // exact: whole numbers (a NaN stays; a coarse maximum's count does not)
        sum = ref != kNoRef ? sum * ex2(ref - to) : sum != sum ? sum : 0.f;
        ref = to;
      }
    }
    if (!(fabsf(m) < a.coarse)) {        // coarse, or -inf only so far; a NaN still has to show
#pragma unroll
      for (int k = 0; k < kUnroll * kE; ++k) sum = x[k] != x[k] ? x[k] : x[k] == m && m > -INFINITY ? sum + 1.f : sum;
      if (m == INFINITY) sum = NAN;
      continue;
    }
    const uint64_t neg = f2_pack(-ref, -ref);
    uint64_t acc[4] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f), f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
    for (int k = 0; k < kUnroll * kE; k += 2) {
      float y0, y1;
      f2_unpack(f2_fma(f2_pack(x[k], x[k + 1]), k2v, neg), y0, y1);
      acc[(k >> 1) & 3] = f2_add(acc[(k >> 1) & 3], f2_pack(ex2(y0), ex2(y1)));
    }
    float a0, a1, a2, a3;
    f2_unpack(f2_add(acc[0], acc[1]), a0, a1);
    f2_unpack(f2_add(acc[2], acc[3]), a2, a3);
    sum += (a0 + a1) + (a2 + a3);
  }
  // the segment's reference and sum
  float wm = 0.f;
  if (__any_sync(0xffffffffu, is_coarse(a, m))) {
    wm = warp_max(m);
    if (is_coarse(a, wm) ? m != wm : is_coarse(a, m)) sum = sum != sum ? sum : 0.f;
    if (is_coarse(a, wm)) ref = kNoRef;
    else wm = 0.f;
  }
  const float mref = warp_max(ref);
  const dfloat ws = warp_sum_df(df_make(ref == kNoRef ? sum : sum * ex2(ref - mref)));
  float gm = m;
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, o));
  if ((lane & 7) == 0) s_group[warp * 4 + (lane >> 3)] = gm;
  if (lane == 0) {
    s_ref[warp] = mref;
    s_max[warp] = wm == 0.f && mref == kNoRef ? -INFINITY : wm;
    s_sum[warp] = ws;
  }
  __syncthreads();
  // the W-th largest of the groups' maxima, ties by group (an equal element passes the test below alike);
  // each warp finds it for itself
  float thr;
  {
    const float mine = s_group[lane];
    int rank = 0;
#pragma unroll
    for (int g = 0; g < 32; ++g) {
      const float o = __shfl_sync(0xffffffffu, mine, g);
      rank += (o > mine || (o == mine && g < lane)) ? 1 : 0;
    }
    // -inf if fewer than W groups have elements: then all are candidates
    thr = __shfl_sync(0xffffffffu, mine, __ffs(__ballot_sync(0xffffffffu, rank == a.W - 1)) - 1);
  }
  if (m >= thr && m > -INFINITY) s_hot[atomicAdd(&s_nhot, 1)] = tid;
  __syncthreads();
  const int nhot = s_nhot;
  for (int h = warp; h < nhot; h += kWarps) {
    // thread t's vectors: v0 + t + i * kRowThreads
    for (int v = v0 + s_hot[h] + lane * kRowThreads; v < v1; v += 32 * kRowThreads) {
      float x[kE];
      elements<T>(*reinterpret_cast<const uint4*>(src + size_t(v) * kE), v * kE, a.V, x);
#pragma unroll
      for (int k = 0; k < kE; ++k) {
        if (x[k] >= thr && x[k] > -INFINITY) {
          const int at = atomicAdd(&s_n, 1);
          if (at < kList) {
            s_v[at] = x[k];
            s_id[at] = v * kE + k;
          }
        }
      }
    }
  }
  __syncthreads();
  const size_t out = size_t(row) * a.S + sg;
  int n = s_n;
  if (n <= kList) {
    // the order in which candidates came does not matter: their ranks are by value and id
    for (int i = tid; i < n; i += kRowThreads) {
      const float v = s_v[i];
      const int id = s_id[i];
      int rank = 0;
      for (int j = 0; j < n; ++j) rank += ahead(s_v[j], s_id[j], v, id) ? 1 : 0;
      if (rank < a.W) {
        a.cand_v[out * a.W + rank] = v;
        a.cand_id[out * a.W + rank] = id;
      }
    }
  } else {
    // many logits tie at the bound: W rounds over the segment, each for the best behind the last one
    float lv = INFINITY;
    int li = -1;
    n = min(n, a.W);
    for (int k = 0; k < n; ++k) {
      float bv = -INFINITY;
      int bi = 0x7fffffff;
      for (int v = v0 + tid; v < v1; v += kRowThreads) {
        float x[kE];
        elements<T>(*reinterpret_cast<const uint4*>(src + size_t(v) * kE), v * kE, a.V, x);
#pragma unroll
        for (int e = 0; e < kE; ++e) {
          const int id = v * kE + e;
          if (ahead(lv, li, x[e], id) && ahead(x[e], id, bv, bi)) {
            bv = x[e];
            bi = id;
          }
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float ov = __shfl_xor_sync(0xffffffffu, bv, o);
        const int oi = __shfl_xor_sync(0xffffffffu, bi, o);
        if (ahead(ov, oi, bv, bi)) {
          bv = ov;
          bi = oi;
        }
      }
      __syncthreads();
      if (lane == 0) {
        s_bv[warp] = bv;
        s_bi[warp] = bi;
      }
      __syncthreads();
      lv = s_bv[0];
      li = s_bi[0];
#pragma unroll
      for (int w = 1; w < kWarps; ++w)
        if (ahead(s_bv[w], s_bi[w], lv, li)) {
          lv = s_bv[w];
          li = s_bi[w];
        }
      if (tid == 0) {
        a.cand_v[out * a.W + k] = lv;
        a.cand_id[out * a.W + k] = li;
      }
    }
  }
  if (warp == 0) {
    // fp64 runs at a sixteenth of fp32's rate and less here: the sums join as pairs of fp32 numbers
    const float r = lane < kWarps ? s_ref[lane] : kNoRef;
    const float mw = lane < kWarps ? s_max[lane] : -INFINITY;
    float top = warp_max(r), f = r == kNoRef ? 1.f : ex2(r - top);
    int coarse = 0;
    if (__any_sync(0xffffffffu, is_coarse(a, mw))) {
      const float best = warp_max(mw);
      if (is_coarse(a, mw) ? mw != best : is_coarse(a, best)) f = 0.f;
      if (is_coarse(a, best)) {
        top = best;
        coarse = kCoarseSeg;
      }
    }
    dfloat t = lane < kWarps ? s_sum[lane] : df_make(0.f);
    t = {t.hi * f, t.lo * f};
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) t = df_add(t, df_shfl_xor(t, o));
    if (lane == 0) {
      Seg g;
      g.sum = t;
      g.ref = top;
      g.count = min(n, a.W) + coarse;
      a.seg[out] = g;
    }
  }
}

// fp64 values in the order of signed whole numbers (no NaN); -0 as 0
__device__ __forceinline__ long long rank_key(double v) {
  const long long b = __double_as_longlong(v + 0.0);
  return b < 0 ? b ^ 0x7fffffffffffffffLL : b;
}

__global__ void __launch_bounds__(kPickThreads) beam_pick_kernel(SelectDev a) {
  constexpr int kHold = SPEC_MAX_BEAMS * kMaxSegLists / kPickThreads;
  __shared__ float s_v[SPEC_MAX_BEAMS * kMaxSegLists];      // beam's segment lists, id 0x7fffffff where short
  __shared__ int s_id[SPEC_MAX_BEAMS * kMaxSegLists];
  __shared__ double s_lse[SPEC_MAX_BEAMS], s_inv[SPEC_MAX_BEAMS];      // log2 of the row's sum; 1 / penalty
  __shared__ float s_base[SPEC_MAX_BEAMS];                             // what logits are taken from: 0, or a coarse maximum
  __shared__ dfloat s_sum[SPEC_MAX_BEAMS];
  __shared__ float s_top[SPEC_MAX_BEAMS];
  __shared__ float s_score[SPEC_MAX_BEAMS];
  __shared__ int s_len[SPEC_MAX_BEAMS], s_fin[SPEC_MAX_BEAMS], s_live[SPEC_MAX_BEAMS];
  __shared__ long long s_key[SPEC_MAX_BEAMS * SPEC_MAX_BEAMS];
  __shared__ double s_total[SPEC_MAX_BEAMS * SPEC_MAX_BEAMS];
  __shared__ int s_tok[SPEC_MAX_BEAMS * SPEC_MAX_BEAMS];
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, W = a.W, per = a.S * W;
  const int r0 = b * W;
  // all candidates on their way at once; what a beam that was not read left there is not used
  float cv[kHold];
  int ci[kHold];
#pragma unroll
  for (int k = 0; k < kHold; ++k) {
    const int i = tid + k * kPickThreads;
    if (i < W * per) {
      cv[k] = a.cand_v[size_t(r0) * per + i];
      ci[k] = a.cand_id[size_t(r0) * per + i];
      const int j = i / per, sg = (i - j * per) / W;
      if (i - j * per - sg * W >= (a.seg[size_t(r0 + j) * a.S + sg].count & (kCoarseSeg - 1))) ci[k] = 0x7fffffff;
    }
  }
  // sixteen lanes a beam: the sum over its segments
  {
    const int w = tid >> 4, sub = tid & 15;
    const bool mine = w < W;
    const int row = r0 + (mine ? w : 0);
    float ref = kNoRef, base = 0.f;
    bool coarse = false;
    dfloat sum = df_make(0.f);
    const float sc = a.scores[row];
    const int fin = a.finished[row] != 0, len = a.lengths[row];
    if (mine && sub < a.S && fin == 0 && sc > -INFINITY) {      // 16 segments at most; false for NaN
      const Seg g = a.seg[size_t(row) * a.S + sub];
      ref = g.ref;
      sum = g.sum;
      coarse = (g.count & kCoarseSeg) != 0;
    }
    // sixteen lanes join what they have; a warp has two beams
    if (__any_sync(0xffffffffu, coarse)) {
      float best = coarse ? ref : ref == kNoRef ? -INFINITY : 0.f;
      const float m = best;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
      if (coarse ? m != best : is_coarse(a, best)) sum = {sum.hi * 0.f, sum.lo * 0.f};      // (a NaN stays)
      if (coarse || is_coarse(a, best)) ref = kNoRef;
      base = is_coarse(a, best) ? best : 0.f;
    }
    float top = ref;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float f = ref == kNoRef ? 1.f : ex2(ref - top);     // a segment of -inf only has the sum 0, or NaN if it holds one
    sum = {sum.hi * f, sum.lo * f};
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) sum = df_add(sum, df_shfl_xor(sum, o));
    if (mine && sub == 0) {
      // a NaN or an infinity: the row is out
      const bool good = sum.hi > 0.f && sum.hi < INFINITY && base < INFINITY;
      s_sum[w] = good ? sum : df_make(1.f);
      s_top[w] = good && base == 0.f ? top : 0.f;
      s_base[w] = good ? base : 0.f;
      s_score[w] = sc;
      s_len[w] = len;
      s_fin[w] = fin;
      s_live[w] = sc > -INFINITY && (fin != 0 || good) ? 1 : 0;
    }
  }
  if (tid < W * W) {
    s_tok[tid] = -1;
    s_key[tid] = (long long)0x8000000000000000LL;      // behind every rank
  }
  __syncthreads();
  // the fp64 functions, of all beams at once in one warp each
  if (warp == 0 && lane < W) {
    s_lse[lane] = double(s_top[lane]) + log2_of(df_to_d(s_sum[lane]));
  } else if (warp == 1 && lane < W) {
    // penalties beyond fp64's range stay at its ends
    const double pen = (5 + s_len[lane] + (s_fin[lane] ? 0 : 1)) * (1.0 / 6.0);
    s_inv[lane] = a.alpha == 0.0 ? 1.0 : exp2_of(fmin(fmax(-a.alpha * log2_of(fmax(pen, 0.5)), -990.0), 990.0));
  }
#pragma unroll
  for (int k = 0; k < kHold; ++k) {
    const int i = tid + k * kPickThreads;
    if (i < W * per) {
      const int j = i / per;
      if (!s_live[j] || s_fin[j]) ci[k] = 0x7fffffff;
      s_v[i] = ci[k] == 0x7fffffff ? -INFINITY : cv[k];
      s_id[i] = ci[k];
    }
  }
  __syncthreads();
  // a beam's W best, in order
#pragma unroll
  for (int k = 0; k < kHold; ++k) {
    const int i = tid + k * kPickThreads;
    if (i >= W * per || ci[k] == 0x7fffffff) continue;
    const int j = i / per;
    int rank = 0;
#pragma unroll 8
    for (int q = j * per; q < (j + 1) * per; ++q) rank += ahead(s_v[q], s_id[q], cv[k], ci[k]) ? 1 : 0;
    if (rank < W) {
      const double total = double(s_score[j]) + (double(cv[k] - s_base[j]) * double(a.k2) - s_lse[j]) * 0.693147180559945309417;
      s_tok[j * W + rank] = ci[k];
      s_total[j * W + rank] = total;
      s_key[j * W + rank] = rank_key(total * s_inv[j]);
    }
  }
  if (tid < W && s_live[tid] && s_fin[tid]) {
    s_tok[tid * W] = a.eos >= 0 && a.eos < a.V ? a.eos : 0;
    s_total[tid * W] = double(s_score[tid]);
    s_key[tid * W] = rank_key(double(s_score[tid]) * s_inv[tid]);
  }
  __syncthreads();
  const int offered = __syncthreads_count(tid < W * W && s_tok[tid] >= 0);
  if (tid < W * W && s_tok[tid] >= 0) {
    const long long mine = s_key[tid];
    int rank = 0;
    // equal logits of a beam have equal ranks: the list's order, beam by beam, settles ties
#pragma unroll 8
    for (int k = 0; k < W * W; ++k) rank += s_key[k] > mine || (s_key[k] == mine && k < tid) ? 1 : 0;
    if (rank < W) {
      const int j = tid / W, at = r0 + rank;
      a.parent[at] = j;
      a.token[at] = s_tok[tid];
      a.out_score[at] = float(s_total[tid]);
      a.out_length[at] = s_len[j] + (s_fin[j] ? 0 : 1);
      a.out_finished[at] = (s_fin[j] || s_tok[tid] == a.eos) ? 1 : 0;
    }
  }
  if (tid >= offered && tid < W) {
    const int at = r0 + tid;
    a.parent[at] = tid;
    a.token[at] = 0;
    a.out_score[at] = -INFINITY;
    a.out_length[at] = s_len[tid];
    a.out_finished[at] = 0;
  }
}

// Segments of a row: enough CTAs for the GPU when there are few rows, none shorter than 4 KB, and
// segments x W within the pick's lists.
static int segments(const spec_beam_select_params* p) {
  const long long rows = (long long)p->B * p->W;
  const int es = p->dtype == SPEC_BF16 ? 2 : 4;
  const long long want = 4LL * sm_count_current_device();
  long long s = (want + rows - 1) / rows;
  const long long most = (long long)p->V * es / 4096;
  if (s > most) s = most;
  if (s > kMaxSegLists / p->W) s = kMaxSegLists / p->W;
  if (s > 16) s = 16;
  return s < 1 ? 1 : int(s);
}

struct SelectWs {
  size_t seg, v, id, total;
  int S;
};
static SelectWs select_ws(const spec_beam_select_params* p) {
  SelectWs w;
  w.S = segments(p);
  const size_t lists = size_t(p->B) * p->W * w.S;
  size_t off = 0;
  w.seg = off; off = align_up(off + sizeof(Seg) * lists, 256);
  w.v = off; off = align_up(off + sizeof(float) * lists * p->W, 256);
  w.id = off; off = align_up(off + sizeof(int32_t) * lists * p->W, 256);
  w.total = off;
  return w;
}

static spec_status_t check_select(const spec_beam_select_params* p) {
  if (!p) return SPEC_ERR_INVALID_ARG;
  if (p->dtype != SPEC_F32 && p->dtype != SPEC_BF16) return SPEC_ERR_INVALID_ARG;
  if (p->B < 1 || p->W < 1 || p->V < 1 || p->ld < p->V) return SPEC_ERR_INVALID_ARG;
  if (!(p->tau > 0.0) || isinf(p->tau) || !(p->alpha >= 0.0) || isinf(p->alpha)) return SPEC_ERR_INVALID_ARG;
  const double k2 = 1.4426950408889634 / p->tau;
  if (!(k2 < 3.0e38) || !(k2 > 1.2e-38)) return SPEC_ERR_INVALID_ARG;    // the scale has to be a normal fp32 number
  if (!p->logits || !aligned16(p->logits) || !p->scores || !p->lengths || !p->finished || !p->parent ||
      !p->token || !p->out_score || !p->out_length || !p->out_finished)
    return SPEC_ERR_INVALID_ARG;
  if ((p->ld * (p->dtype == SPEC_BF16 ? 2 : 4)) % 16) return SPEC_ERR_INVALID_ARG;
  if (p->W > SPEC_MAX_BEAMS || p->V > 0x7fffffff - 1024 || (long long)p->B * p->W > 65535) return SPEC_ERR_UNSUPPORTED;
  return SPEC_OK;
}

// ------------------------------------------------------------------------------ reorder
// beam_plan_kernel, one CTA per request: checks, which writing pages are copied where, and the tables (a
// thread moves whole columns, so in place is safe).  beam_copy_kernel, one CTA per (copy, layer): a head's
// live rows of a page are one run of bytes, 16 bytes a thread.  Sources are pages of beams with children,
// destinations pages of beams without, so no copy reads what another writes.  Two launches, because
// the tables change in place and every copy needs the pages that stood in them before.  Bound by the copied
// bytes when there are many layers, by the two launches' chains when there are few.
constexpr int kPlanThreads = 128;
constexpr int kCopyThreads = 256;
struct PlanRec {
  int n, rem;
  int from[SPEC_MAX_BEAMS], to[SPEC_MAX_BEAMS];
};

struct ReorderDev {
  char* k;
  char* v;
  float* ks;
  float* vs;
  int64_t layer_stride_bytes, scale_layer_stride;
  int32_t* block_table;
  const int32_t* kv_len;
  const int32_t* parent;
  int32_t* beam_status;
  PlanRec* plan;
  int32_t W, H_kv, row_bytes, bs, num_blocks, max_blocks;
};

__global__ void __launch_bounds__(kPlanThreads) beam_plan_kernel(ReorderDev a) {
  __shared__ int s_parent[SPEC_MAX_BEAMS], s_page[SPEC_MAX_BEAMS], s_new[SPEC_MAX_BEAMS];
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x, tid = threadIdx.x, W = a.W;
  int32_t* table = a.block_table + size_t(b) * W * a.max_blocks;
  const int L = a.kv_len[b], page = L / a.bs, rem = L - page * a.bs;
  int bad = 0;
  if (tid < W) {
    s_parent[tid] = a.parent[b * W + tid];
    if (s_parent[tid] < 0 || s_parent[tid] >= W) bad = SPEC_REQ_BAD_PARENT;
    s_page[tid] = -1;
    if (L >= 0 && page < a.max_blocks) s_page[tid] = table[size_t(tid) * a.max_blocks + page];
  }
  bad = __syncthreads_or(bad);
  if (!bad && (L < 0 || page >= a.max_blocks)) bad = SPEC_REQ_BAD_SIZE;
  int page_bad = 0;
  if (!bad && tid < W) {
    const int pb = s_page[tid];
    page_bad = pb < 0 || pb >= a.num_blocks;
    for (int j = 0; j < W; ++j) page_bad = page_bad || (j != tid && s_page[j] == pb);
  }
  if (__syncthreads_or(page_bad) && !bad) bad = SPEC_REQ_BAD_BLOCK;
  if (tid == 0) {
    a.beam_status[b] = bad;
    int n = 0;
    if (!bad) {
      unsigned used = 0, met = 0;
      for (int j = 0; j < W; ++j) used |= 1u << s_parent[j];
      int next = 0;
      for (int j = 0; j < W; ++j) {
        const int p = s_parent[j];
        if (!((met >> p) & 1u)) {
          met |= 1u << p;
          s_new[j] = s_page[p];
        } else {
          while ((used >> next) & 1u) ++next;    // as many beams without children as there are further ones
          s_new[j] = s_page[next];
          a.plan[b].from[n] = s_page[p];
          a.plan[b].to[n] = s_page[next];
          ++next;
          ++n;
        }
      }
    }
    a.plan[b].n = rem > 0 ? n : 0;
    a.plan[b].rem = rem;
  }
  __syncthreads();
  if (bad) return;
  if (tid < W) table[size_t(tid) * a.max_blocks + page] = s_new[tid];
  for (int i = tid; i < page; i += kPlanThreads) {
    int32_t old[SPEC_MAX_BEAMS];
#pragma unroll
    for (int j = 0; j < SPEC_MAX_BEAMS; ++j)
      if (j < W) old[j] = table[size_t(s_parent[j]) * a.max_blocks + i];
#pragma unroll
    for (int j = 0; j < SPEC_MAX_BEAMS; ++j)
      if (j < W) table[size_t(j) * a.max_blocks + i] = old[j];
  }
}

__global__ void __launch_bounds__(kCopyThreads) beam_copy_kernel(ReorderDev a) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x / (a.W - 1), c = blockIdx.x - b * (a.W - 1), layer = blockIdx.y, tid = threadIdx.x;
  const PlanRec& rec = a.plan[b];
  if (c >= rec.n) return;
  const int rem = rec.rem;
  const size_t head_bytes = size_t(a.bs) * a.row_bytes;
  const size_t from = size_t(rec.from[c]) * a.H_kv * head_bytes, to = size_t(rec.to[c]) * a.H_kv * head_bytes;
  const int run = rem * (a.row_bytes / 16);       // vectors of one head's live rows
  char* kb = a.k + layer * a.layer_stride_bytes;
  char* vb = a.v + layer * a.layer_stride_bytes;
  for (int i = tid; i < run * a.H_kv; i += kCopyThreads) {
    const int h = i / run;
    const size_t off = h * head_bytes + size_t(i - h * run) * 16;
    const uint4 x = *reinterpret_cast<const uint4*>(kb + from + off);
    const uint4 y = *reinterpret_cast<const uint4*>(vb + from + off);
    *reinterpret_cast<uint4*>(kb + to + off) = x;
    *reinterpret_cast<uint4*>(vb + to + off) = y;
  }
  if (a.ks) {
    float* ks = a.ks + layer * a.scale_layer_stride;
    float* vs = a.vs + layer * a.scale_layer_stride;
    for (int h = tid; h < a.H_kv; h += kCopyThreads) {
      ks[size_t(rec.to[c]) * a.H_kv + h] = ks[size_t(rec.from[c]) * a.H_kv + h];
      vs[size_t(rec.to[c]) * a.H_kv + h] = vs[size_t(rec.from[c]) * a.H_kv + h];
    }
  }
}

static spec_status_t check_reorder(const spec_beam_reorder_params* p) {
  if (!p) return SPEC_ERR_INVALID_ARG;
  if (p->dtype != SPEC_F32 && p->dtype != SPEC_BF16 && p->dtype != SPEC_E4M3) return SPEC_ERR_INVALID_ARG;
  if (p->B < 1 || p->W < 1 || p->H_kv < 1 || p->head_dim < 1 || p->block_size < 1 || p->num_blocks < 1 ||
      p->max_blocks_per_req < 1 || p->num_layers < 1 || p->layer_stride < 0 || p->scale_layer_stride < 0)
    return SPEC_ERR_INVALID_ARG;
  const int64_t es = p->dtype == SPEC_F32 ? 4 : p->dtype == SPEC_BF16 ? 2 : 1;
  const int64_t row_bytes = int64_t(p->head_dim) * es;
  if (row_bytes % 16 || (p->layer_stride * es) % 16) return SPEC_ERR_INVALID_ARG;
  if (!p->k_cache || !p->v_cache || !aligned16(p->k_cache) || !aligned16(p->v_cache) || !p->block_table ||
      !p->kv_len || !p->parent || !p->beam_status)
    return SPEC_ERR_INVALID_ARG;
  if (p->dtype == SPEC_E4M3 && (!p->k_scale || !p->v_scale)) return SPEC_ERR_INVALID_ARG;
  if (p->W > SPEC_MAX_BEAMS || p->num_layers > 65535 || (long long)p->B * p->W >= (1LL << 31))
    return SPEC_ERR_UNSUPPORTED;
  if (row_bytes / 16 * p->block_size * p->H_kv >= (1LL << 31)) return SPEC_ERR_UNSUPPORTED;
  return SPEC_OK;
}

}  // namespace beam
}  // namespace spec

extern "C" {

size_t spec_beam_select_workspace_size(const spec_beam_select_params* p) {
  if (spec::beam::check_select(p) != SPEC_OK) return 0;
  return spec::beam::select_ws(p).total;
}

spec_status_t spec_beam_select(const spec_beam_select_params* p, void* workspace, size_t ws_bytes,
                               spec_stream_t stream) {
  using namespace spec;
  using namespace spec::beam;
  const spec_status_t st = check_select(p);
  if (st != SPEC_OK) return st;
  const SelectWs w = select_ws(p);
  if (!workspace || ws_bytes < w.total || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return SPEC_ERR_INVALID_ARG;
  char* base = static_cast<char*>(workspace);
  const bool bf16 = p->dtype == SPEC_BF16;
  SelectDev d;
  d.logits = p->logits; d.scores = p->scores; d.lengths = p->lengths; d.finished = p->finished;
  d.parent = p->parent; d.token = p->token; d.out_score = p->out_score; d.out_length = p->out_length;
  d.out_finished = p->out_finished;
  d.seg = reinterpret_cast<Seg*>(base + w.seg);
  d.cand_v = reinterpret_cast<float*>(base + w.v);
  d.cand_id = reinterpret_cast<int32_t*>(base + w.id);
  d.ld = p->ld;
  d.W = p->W; d.V = p->V; d.S = w.S; d.eos = p->eos;
  const int per = bf16 ? 8 : 4, nvec = (p->V + per - 1) / per;
  d.seg_vecs = (nvec + w.S - 1) / w.S;
  d.k2 = float(1.4426950408889634 / p->tau);
  d.coarse = float(2147483648.0 / double(d.k2));
  d.alpha = p->alpha;
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = launch_pdl(bf16 ? beam_rows_kernel<__nv_bfloat16> : beam_rows_kernel<float>,
                             dim3(w.S, p->B * p->W), dim3(kRowThreads), 0, s, d);
  if (e == cudaSuccess) e = launch_pdl(beam_pick_kernel, dim3(p->B), dim3(kPickThreads), 0, s, d);
  return launch_result(e);
}

size_t spec_beam_reorder_workspace_size(const spec_beam_reorder_params* p) {
  if (spec::beam::check_reorder(p) != SPEC_OK) return 0;
  return spec::align_up(sizeof(spec::beam::PlanRec) * size_t(p->B), 256);
}

spec_status_t spec_beam_reorder(const spec_beam_reorder_params* p, void* workspace, size_t ws_bytes,
                                spec_stream_t stream) {
  using namespace spec;
  using namespace spec::beam;
  const spec_status_t st = check_reorder(p);
  if (st != SPEC_OK) return st;
  if (!workspace || ws_bytes < align_up(sizeof(PlanRec) * size_t(p->B), 256) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return SPEC_ERR_INVALID_ARG;
  const int64_t es = p->dtype == SPEC_F32 ? 4 : p->dtype == SPEC_BF16 ? 2 : 1;
  ReorderDev d;
  d.k = static_cast<char*>(p->k_cache);
  d.v = static_cast<char*>(p->v_cache);
  d.ks = p->dtype == SPEC_E4M3 ? p->k_scale : nullptr;
  d.vs = p->dtype == SPEC_E4M3 ? p->v_scale : nullptr;
  d.layer_stride_bytes = p->layer_stride * es;
  d.scale_layer_stride = p->scale_layer_stride;
  d.block_table = p->block_table; d.kv_len = p->kv_len; d.parent = p->parent; d.beam_status = p->beam_status;
  d.plan = static_cast<PlanRec*>(workspace);
  d.W = p->W; d.H_kv = p->H_kv; d.row_bytes = int(p->head_dim * es); d.bs = p->block_size;
  d.num_blocks = p->num_blocks; d.max_blocks = p->max_blocks_per_req;
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = launch_pdl(beam_plan_kernel, dim3(p->B), dim3(kPlanThreads), 0, s, d);
  if (e == cudaSuccess && p->W > 1)
    e = launch_pdl(beam_copy_kernel, dim3(p->B * (p->W - 1), p->num_layers), dim3(kCopyThreads), 0, s, d);
  return launch_result(e);
}

}  // extern "C"
