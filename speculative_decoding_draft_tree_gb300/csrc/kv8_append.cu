// spec_kv8_append: new K/V rows quantised into the 8-bit paged cache.
//
// Mathematics (include/spec_verify.h): per (block, head, cache) the largest finite |x| of the
// block's new rows gives a power-of-two scale; a block that already holds rows keeps the larger
// of its scale and that one, its rows requantised when it grows.  Bound by bytes: each x is read
// once and each code written once.
//
// A team of W warps owns one (block, head, cache): it keeps the block's new rows in registers
// (8 sixteen-byte vectors a thread: 16 rows of 128 bf16 values are one warp's) between the
// maximum and the conversion, so x is read once; W grows with the block's bytes, and vectors past
// the registers (very large blocks only) are read a second time.  The tokens are cut into
// windows of kWindow; a CTA handles the blocks whose first new row (the request's first token, or
// one at a block boundary) lies in its window, so nothing has to be counted or sorted first, and
// one launch serves single tokens, trees and prompts alike.
//
// Measured (bf16, head_dim 128, blocks of 16): prompts, 49,000 tokens of 32 KV heads (1.2 GB) 191
// us, 6.4 TB/s, 94% of the copy rate (fp32: 298 us, at the copy rate); 64 trees of 8 .. 56 tokens, 8 KV
// heads (12 MB) 8.2 us (fp32 10.6) and 64 single tokens 4 us, both bound by the launch and the chain offsets -> page -> scale -> codes.
#include "kv8.cuh"

namespace spec {

struct AppendDev {
  const char* k_new;
  const char* v_new;
  uint8_t* k_cache;
  uint8_t* v_cache;
  float* k_scale;
  float* v_scale;
  const int32_t* block_table;
  const int32_t* start;
  const int32_t* row_offset;
  int32_t* req_status;
  int64_t k_ld_bytes, v_ld_bytes;
  int32_t B, N, H_kv, d, bs, num_blocks, max_blocks, window;
  uint32_t columns;   // CTAs over the (head, cache) units
};

constexpr int kAppendThreads = 256;
constexpr int kHold = 8;   // vectors a thread keeps in registers
constexpr int kAppendCtas = 304;

// The codes of one 16-byte vector of x, and its largest magnitude: NaN is passed over, infinity is
// not (the kernel looks again, element by element, where one turns up).
template <typename T> struct Codes;
template <> struct Codes<__nv_bfloat16> {
  using type = uint2;
  __device__ __forceinline__ static uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  __device__ __forceinline__ static float top(float m, const uint4& v) {
    const uint32_t k = 0x7FFF7FFFu;
    const uint32_t a = max2(max2(v.x & k, v.y & k), max2(v.z & k, v.w & k));
    return fmaxf(m, fmaxf(bf16_lo(a), bf16_hi(a)));
  }
  __device__ __forceinline__ static type make(const float (&f)[8]) {
    return make_uint2(kv8::pack_e4m3x4(f[0], f[1], f[2], f[3]),
                      kv8::pack_e4m3x4(f[4], f[5], f[6], f[7]));
  }
};
template <> struct Codes<float> {
  using type = uint32_t;
  __device__ __forceinline__ static float top(float m, const uint4& v) {
    m = fmaxf(m, fmaxf(fabsf(__uint_as_float(v.x)), fabsf(__uint_as_float(v.y))));
    return fmaxf(m, fmaxf(fabsf(__uint_as_float(v.z)), fabsf(__uint_as_float(v.w))));
  }
  __device__ __forceinline__ static type make(const float (&f)[4]) {
    return kv8::pack_e4m3x4(f[0], f[1], f[2], f[3]);
  }
};

// Offsets [o, o1) and first slot p0 of a request that cannot be appended, and its report (a request
// that another call has flagged keeps its bits).
__device__ __forceinline__ bool bad_request(const AppendDev& a, int o, int o1, int p0) {
  return o < 0 || o1 < o || o1 > a.N || p0 < 0 || (long long)p0 + o1 - o > INT32_MAX;
}
__device__ __forceinline__ void report_bad(const AppendDev& a, int r) {
  if ((a.req_status[r] & ~SPEC_REQ_BAD_BLOCK) == 0) atomicOr(&a.req_status[r], SPEC_REQ_BAD_SIZE);
}

template <typename T, int W>
__global__ void __launch_bounds__(kAppendThreads, 3) kv8_append_kernel(AppendDev a) {
  constexpr int E = elem<T>::per16;
  constexpr int kTeam = 32 * W, kTeams = kAppendThreads / kTeam;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31;
  const int team = tid / kTeam, tt = tid % kTeam;
  // heads vary fastest over the CTAs: a token's heads are neighbours in x
  const int win = int(blockIdx.x / a.columns), column = int(blockIdx.x - uint32_t(win) * a.columns);
  const int n0 = win * a.window, n1 = min(a.N, n0 + a.window);
  // The request of token n0: as many requests end at or before it, where offsets only go up.  CTA 0
  // reports the requests that cannot be appended, whether or not they own a token.
  int r = 0;
  bool back = false;
  for (int i = 0; i < a.B; i += kAppendThreads) {
    const int q = i + tid;
    int o = 0, o1 = 0;
    if (q < a.B) {
      o = a.row_offset[q];
      o1 = a.row_offset[q + 1];
      if (blockIdx.x == 0 && bad_request(a, o, o1, a.start[q])) report_bad(a, q);
    }
    back = back || o1 < o;
    r += __syncthreads_count(q < a.B && o1 <= n0);
  }
  // Each warp's largest offset of the requests walked past (not in a register: the vectors in flight need
  // them all).  It decides only where some offsets go backwards, which takes the walk from the
  // first request on.
  __shared__ int s_top[kAppendThreads / 32];
  if (lane == 0) s_top[tid >> 5] = INT32_MIN;
  back = __syncthreads_or(back);
  if (back) {
    r = 0;
    if (blockIdx.x == 0 && tid == 0) {
      for (int q = 0, t = INT32_MIN; q < a.B; ++q) {
        const int o = a.row_offset[q];
        if (o < t) report_bad(a, q);
        t = max(t, max(o, a.row_offset[q + 1]));
      }
    }
  }
  const int unit = column * kTeams + team;          // (head, cache)
  const bool mine = unit < 2 * a.H_kv;
  const int h = unit >> 1;
  const bool is_v = unit & 1;
  const char* x = (is_v ? a.v_new : a.k_new) + size_t(mine ? h : 0) * a.d * sizeof(T);
  const int64_t ld = is_v ? a.v_ld_bytes : a.k_ld_bytes;
  uint8_t* cache = is_v ? a.v_cache : a.k_cache;
  float* scale = is_v ? a.v_scale : a.k_scale;
  const int vpr = a.d / E;                          // vectors per row
  // a thread's vectors are kTeam apart: the same column of every (kTeam / vpr)-th row where a row's
  // vectors divide the team
  const bool even = kTeam % vpr == 0;
  const int r0 = tt / vpr;
  const char* const x0 = x + int64_t(r0) * ld + (tt - r0 * vpr) * 16;
  const int64_t step = int64_t(kTeam / vpr) * ld;
  __shared__ float s_max[kAppendThreads / 32];
  int n = n0;
  while (n < n1 && r < a.B) {                       // uniform across the CTA
    const int o = a.row_offset[r], o1 = a.row_offset[r + 1], p0 = a.start[r];
    const bool bad = bad_request(a, o, o1, p0) || o < s_top[tid >> 5];
    if (bad || n >= o1) {
      __syncwarp();
      if (lane == 0) s_top[tid >> 5] = max(s_top[tid >> 5], max(o, o1));
      __syncwarp();
      ++r;
      continue;
    }
    if (o > n) {                                    // offsets that start late, or a bad request before
      n = o;
      continue;
    }
    if ((a.req_status[r] & ~SPEC_REQ_BAD_BLOCK) != 0) {
      n = o1;
      continue;
    }
    const int slot = p0 + (n - o), row = slot % a.bs;
    const int seg = min(a.bs - row, o1 - n);        // rows from n to the end of n's block
    if (n != o && row != 0) {                       // the block began in an earlier window
      n += seg;
      continue;
    }
    const int lb = slot / a.bs;
    const int pb = lb < a.max_blocks ? a.block_table[size_t(r) * a.max_blocks + lb] : -1;
    const int nv = mine ? seg * vpr : 0;            // this team's vectors
    const char* const xn = x0 + int64_t(n) * ld;
    auto load = [&](int q) -> uint4 {               // vector tt + q kTeam
      if (even) return ld_stream16(xn + q * step);
      const int i = tt + q * kTeam, rr = i / vpr;
      return ld_stream16(x + int64_t(n + rr) * ld + (i - rr * vpr) * 16);
    };
    uint4 v[kHold];
    float m = 0.f;
    // (the rows are on their way before the page id is looked at)
#pragma unroll
    for (int q = 0; q < kHold; ++q) {
      const int i = tt + q * kTeam;
      if (i < nv) v[q] = load(q);
    }
    // the next block's rows into L2
    if (mine) {
      const int lines = (int(a.d * sizeof(T)) + 127) / 128, rows = min(a.bs, n1 - (n + seg));
      for (int i = tt; i < rows * lines; i += kTeam) {
        const int rr = i / lines;
        asm volatile("prefetch.global.L2 [%0];" ::"l"(x + int64_t(n + seg + rr) * ld + (i - rr * lines) * 128));
      }
    }
    if (pb < 0 || pb >= a.num_blocks) {
      if (tid == 0) atomicOr(&a.req_status[r], SPEC_REQ_BAD_BLOCK);
      n += seg;
      continue;
    }
    const size_t sidx = size_t(pb) * a.H_kv + (mine ? h : 0);
    uint8_t* page = cache + sidx * size_t(a.bs) * a.d;
    const float old = row > 0 ? scale[sidx] : 0.f;
    // the team's maximum
    auto over_team = [&](float m) -> float {
      m = warp_max(m);
      if (W > 1) {
        __syncthreads();                            // s_max of the block before has been read
        if (lane == 0) s_max[tid >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < W; ++w) m = fmaxf(m, s_max[team * W + w]);
      }
      return m;
    };
#pragma unroll
    for (int q = 0; q < kHold; ++q)
      if (tt + q * kTeam < nv) m = Codes<T>::top(m, v[q]);
    for (int q = kHold; tt + q * kTeam < nv; ++q) m = Codes<T>::top(m, load(q));
    m = over_team(m);
    if (W > 1 ? __syncthreads_or(m > FLT_MAX) : m > FLT_MAX) {   // an infinity: finite values only
      m = 0.f;
#pragma unroll 1
      for (int q = 0; tt + q * kTeam < nv; ++q) {
        float f[E];
        elem<T>::unpack(load(q), f);
#pragma unroll
        for (int e = 0; e < E; ++e) m = fabsf(f[e]) <= FLT_MAX ? fmaxf(m, fabsf(f[e])) : m;
      }
      m = over_team(m);
    }
    const float s = fmaxf(old, kv8::need_scale(m));
    // a power of two's reciprocal is exact, and so is multiplying by it (scales another writer
    // left there need the division)
    const uint32_t sb = __float_as_uint(s);
    const bool pow2 = (sb & 0x807FFFFFu) == 0 && sb >= (uint32_t(kv8::kMinScaleExp) << 23) &&
                      sb <= (uint32_t(kv8::kMaxScaleExp) << 23);
    const float inv = pow2 ? __uint_as_float((254u << 23) - sb) : 0.f;
    // E codes a vector, the rows of a block next to each other
    auto* const to = reinterpret_cast<typename Codes<T>::type*>(page + size_t(row) * a.d) + tt;
    if (pow2) {
      auto put = [&](int q, const uint4& w) {
        float f[E];
        elem<T>::unpack(w, f);
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] *= inv;
        to[q * kTeam] = Codes<T>::make(f);
      };
#pragma unroll
      for (int q = 0; q < kHold; ++q)
        if (tt + q * kTeam < nv) put(q, v[q]);
      for (int q = kHold; tt + q * kTeam < nv; ++q) put(q, load(q));
    } else {
      // (apart from the loop above: with the division as a branch inside it, the whole kernel took
      // 1.7 times as long)
#pragma unroll 1
      for (int q = 0; tt + q * kTeam < nv; ++q) {
        float f[E];
        elem<T>::unpack(load(q), f);
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = __fdiv_rn(f[e], s);
        to[q * kTeam] = Codes<T>::make(f);
      }
    }
    if (mine && row > 0 && s > old) {
      const float ratio = __fdiv_rn(old, s);
      uint4* p = reinterpret_cast<uint4*>(page);
      for (int i = tt; i < row * (a.d / 16); i += kTeam) p[i] = kv8::rescale_e4m3x16(p[i], ratio);
    }
    if (W > 1) __syncthreads();                     // every warp has read the old scale
    else __syncwarp();
    if (mine && tt == 0) scale[sidx] = s;
    n += seg;
  }
}

template <typename T, int W>
static cudaError_t launch_append(const AppendDev& d, cudaStream_t s) {
  const long long ctas = (long long)d.columns * ((d.N + d.window - 1) / d.window);
  return launch_pdl(kv8_append_kernel<T, W>, dim3(unsigned(ctas)), dim3(kAppendThreads), 0, s, d);
}

template <typename T>
static cudaError_t launch_append_w(const AppendDev& d, cudaStream_t s) {
  // warps that hold a whole block in registers: 8 vectors of 16 bytes a lane
  const long long bytes = (long long)d.bs * d.d * sizeof(T);
  if (bytes <= 4096) return launch_append<T, 1>(d, s);
  if (bytes <= 8192) return launch_append<T, 2>(d, s);
  if (bytes <= 16384) return launch_append<T, 4>(d, s);
  return launch_append<T, 8>(d, s);
}

}  // namespace spec

extern "C" spec_status_t spec_kv8_append(const spec_kv8_append_params* p, spec_stream_t stream) {
  using namespace spec;
  if (!p) return SPEC_ERR_INVALID_ARG;
  if (p->dtype != SPEC_F32 && p->dtype != SPEC_BF16) return SPEC_ERR_INVALID_ARG;
  if (p->B < 1 || p->N < 0 || !p->start || !p->row_offset || !p->req_status)
    return SPEC_ERR_INVALID_ARG;
  const spec_status_t st =
      kv8::check_cache(p->H_kv, p->head_dim, p->block_size, p->num_blocks, p->max_blocks_per_req,
                       p->k_cache, p->v_cache, p->k_scale, p->v_scale, p->block_table);
  if (st != SPEC_OK) return st;
  const int64_t es = p->dtype == SPEC_BF16 ? 2 : 4;
  const int64_t row = int64_t(p->H_kv) * p->head_dim;
  if (p->N > 0 && (!p->k_new || !p->v_new || !aligned16(p->k_new) || !aligned16(p->v_new)))
    return SPEC_ERR_INVALID_ARG;
  if (p->k_ld < row || p->v_ld < row || (p->k_ld * es) % 16 || (p->v_ld * es) % 16)
    return SPEC_ERR_INVALID_ARG;
  if (p->N == 0) return SPEC_OK;
  AppendDev d;
  d.k_new = static_cast<const char*>(p->k_new);
  d.v_new = static_cast<const char*>(p->v_new);
  d.k_cache = static_cast<uint8_t*>(p->k_cache);
  d.v_cache = static_cast<uint8_t*>(p->v_cache);
  d.k_scale = p->k_scale;
  d.v_scale = p->v_scale;
  d.block_table = p->block_table;
  d.start = p->start;
  d.row_offset = p->row_offset;
  d.req_status = p->req_status;
  d.k_ld_bytes = p->k_ld * es;
  d.v_ld_bytes = p->v_ld * es;
  d.B = p->B; d.N = p->N; d.H_kv = p->H_kv; d.d = p->head_dim; d.bs = p->block_size;
  d.num_blocks = p->num_blocks; d.max_blocks = p->max_blocks_per_req;
  // Windows as long as they leave kAppendCtas CTAs: a CTA's first loads (which request, where it
  // starts) are a chain of their own, so long calls give a CTA several blocks.
  const int es4 = p->dtype == SPEC_BF16 ? 2 : 4;
  const long long block_bytes = (long long)p->block_size * p->head_dim * es4;
  const int teams = block_bytes <= 4096 ? 8 : block_bytes <= 8192 ? 4 : block_bytes <= 16384 ? 2 : 1;
  const long long columns = (2LL * p->H_kv + teams - 1) / teams;
  d.columns = uint32_t(columns);
  // (64 trees of 8 .. 56: 8.2 us; 10.3 with 152 CTAs, 9.5 with 608.  Prompts, windows of at most 8
  // blocks: 191 us; 229 with one block, 209 with 32.)
  d.window = 1;
  while (d.window < 8 * p->block_size && p->N * columns / (2 * d.window) >= kAppendCtas) d.window *= 2;
  if (columns * ((p->N + d.window - 1) / d.window) >= (1LL << 31)) return SPEC_ERR_UNSUPPORTED;
  const cudaStream_t s = (cudaStream_t)stream;
  return launch_result(p->dtype == SPEC_BF16 ? launch_append_w<__nv_bfloat16>(d, s)
                                             : launch_append_w<float>(d, s));
}
