// spec_tree_attention_kv8: tree attention over the 8-bit cache.  Argument checks, dispatch, and
// the CUDA-core kernel that serves what the tensor-core kernels do not: fp32 queries, head
// dimensions other than 128, unusual block sizes and head ratios.
//
// The CUDA-core kernel: one CTA per (node, four query heads of one KV head).  Each warp takes
// every eighth chunk of 32 keys, one key a lane: the lane reads its key's codes in 16-byte vectors
// and forms the four dot products (the block's scale multiplies the sum, not the elements); the
// chunk's weights then go lane by lane to the whole warp, which reads each visible key's V row
// together and accumulates it.  The warps' running maxima, sums and rows are joined at the end.
// Products and sums in fp32 (codes are exact in fp32); bound by its instructions, not by memory:
// 64 tokens over 8192 slots, 32 query heads on one KV head 1120 us, 0.1 TB/s of codes.
#include <math.h>

#include "attention_kv8.cuh"

namespace spec {

namespace kv8_simt {
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kHeads = 4;          // query heads of a CTA
constexpr int kMaxD = 256;
constexpr int kCols = kMaxD / 32;  // output columns of a lane
}  // namespace kv8_simt

template <typename T>
__global__ void __launch_bounds__(kv8_simt::kThreads) attn_kv8_simt_kernel(AttnKv8Dev a) {
  using namespace kv8_simt;
  __shared__ __align__(16) float sq[kHeads][kMaxD];
  __shared__ float s_o[kWarps][kHeads][kMaxD];
  __shared__ float s_m[kWarps][kHeads], s_l[kWarps][kHeads];
  pdl_wait();
  pdl_trigger();
  const int n = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int chunks = (a.G + kHeads - 1) / kHeads;
  const int h = blockIdx.y / chunks, g0 = (blockIdx.y % chunks) * kHeads;
  const int heads = min(kHeads, a.G - g0);
  int r = 0;
  for (int i = 0; i < a.B; i += kThreads)
    r += __syncthreads_count(i + tid < a.B && a.node_offset[i + tid + 1] <= n);
  if (r >= a.B) return;
  const int o = a.node_offset[r], T_r = a.node_offset[r + 1] - o, P = a.prefix_len[r];
  if (n < o) return;
  const Kv8Live live = kv8_live(a, r, T_r, P);
  if (live != Kv8Live::yes) {
    if (live == Kv8Live::beyond_table && tid == 0) atomicOr(&a.req_status[r], SPEC_REQ_BAD_BLOCK);
    return;
  }
  const T* q = static_cast<const T*>(a.q) + (size_t(n) * a.H_q + h * a.G + g0) * a.d;
  for (int i = tid; i < heads * a.d; i += kThreads)
    sq[i / a.d][i % a.d] = elem<T>::load1(q + i);
  __syncthreads();
  const uint32_t* anc = a.anc + size_t(n) * a.W;
  const int32_t* table = a.block_table + size_t(r) * a.max_blocks;
  const int len = P + T_r;
  float m[kHeads], l[kHeads], acc[kHeads][kCols];
#pragma unroll
  for (int g = 0; g < kHeads; ++g) {
    m[g] = -INFINITY;
    l[g] = 0.f;
#pragma unroll
    for (int c = 0; c < kCols; ++c) acc[g][c] = 0.f;
  }
  for (int k0 = warp * 32; k0 < len; k0 += kThreads) {
    const int key = k0 + lane;
    bool vis = key < P;
    if (key >= P && key < len) vis = (anc[(key - P) >> 5] >> ((key - P) & 31)) & 1u;
    int pb = 0;
    if (vis) {
      pb = table[key / a.bs];
      if (pb < 0 || pb >= a.num_blocks) {
        atomicOr(&a.req_status[r], SPEC_REQ_BAD_BLOCK);
        vis = false;
        pb = 0;
      }
    }
    const size_t sidx = size_t(pb) * a.H_kv + h;
    const size_t row = (sidx * a.bs + key % a.bs) * a.d;
    float x[kHeads] = {0.f, 0.f, 0.f, 0.f};
    if (vis) {
      for (int c = 0; c < a.d; c += 16) {
        const uint4 w = ld_stream16(a.k + row + c);
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float f[4];
          kv8::unpack_e4m3x4(ws[e], f);
#pragma unroll
          for (int g = 0; g < kHeads; ++g) {
            const float4 y = *reinterpret_cast<const float4*>(&sq[g][c + 4 * e]);
            x[g] = fmaf(f[0], y.x, fmaf(f[1], y.y, fmaf(f[2], y.z, fmaf(f[3], y.w, x[g]))));
          }
        }
      }
    }
    const float ks = vis ? a.k_scale[sidx] * a.scale_log2 : 0.f;
    const float vs = vis ? a.v_scale[sidx] : 0.f;
    float p[kHeads];
#pragma unroll
    for (int g = 0; g < kHeads; ++g) {
      x[g] = vis ? x[g] * ks : -INFINITY;
      const float mx = fmaxf(m[g], warp_max(x[g]));
      const float f = m[g] == -INFINITY ? 0.f : ex2(m[g] - mx);
      p[g] = vis ? ex2(x[g] - mx) : 0.f;
      l[g] = l[g] * f + p[g];                       // this lane's share of the sum
      p[g] *= vs;
      m[g] = mx;
      if (f != 1.f) {
#pragma unroll
        for (int c = 0; c < kCols; ++c) acc[g][c] *= f;
      }
    }
    uint32_t todo = __ballot_sync(0xffffffffu, vis);
    while (todo) {
      const int j = __ffs(todo) - 1;
      todo &= todo - 1;
      const size_t vrow = __shfl_sync(0xffffffffu, row, j);
      float pj[kHeads];
#pragma unroll
      for (int g = 0; g < kHeads; ++g) pj[g] = __shfl_sync(0xffffffffu, p[g], j);
#pragma unroll
      for (int c4 = 0; c4 < kCols / 4; ++c4) {
        const int col = c4 * 128 + lane * 4;
        if (col < a.d) {
          float f[4];
          kv8::unpack_e4m3x4(*reinterpret_cast<const uint32_t*>(a.v + vrow + col), f);
#pragma unroll
          for (int g = 0; g < kHeads; ++g)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              acc[g][c4 * 4 + e] = fmaf(pj[g], f[e], acc[g][c4 * 4 + e]);
        }
      }
    }
  }
#pragma unroll
  for (int g = 0; g < kHeads; ++g) {
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) l[g] += __shfl_xor_sync(0xffffffffu, l[g], s);
    if (lane == 0) {
      s_m[warp][g] = m[g];
      s_l[warp][g] = l[g];
    }
#pragma unroll
    for (int c4 = 0; c4 < kCols / 4; ++c4)
#pragma unroll
      for (int e = 0; e < 4; ++e) s_o[warp][g][c4 * 128 + lane * 4 + e] = acc[g][c4 * 4 + e];
  }
  __syncthreads();
  T* out = static_cast<T*>(a.o) + (size_t(n) * a.H_q + h * a.G + g0) * a.d;
  for (int i = tid; i < heads * a.d; i += kThreads) {
    const int g = i / a.d, c = i % a.d;
    float M = -INFINITY, sum = 0.f, v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][g]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = s_m[w][g] == -INFINITY ? 0.f : ex2(s_m[w][g] - M);
      sum += s_l[w][g] * f;
      v += s_o[w][g][c] * f;
    }
    const float y = sum == 0.f ? 0.f : v / sum;     // a row that sees nothing is 0
    if constexpr (sizeof(T) == 2) out[i] = __float2bfloat16_rn(y);
    else out[i] = y;
    if (c == 0 && a.lse)
      a.lse[size_t(n) * a.H_q + h * a.G + g0 + g] =
          sum == 0.f ? -INFINITY : (M + log2f(sum)) * 0.6931471805599453f;
  }
}

bool attn_kv8_tc_takes(const AttnKv8Dev& a, bool bf16);
size_t attn_kv8_tc_workspace(const AttnKv8Dev& a);
spec_status_t launch_attn_kv8_tc(const AttnKv8Dev& a, void* ws, size_t ws_bytes, cudaStream_t s);

static spec_status_t check_attn_kv8(const spec_attn_kv8_params* p) {
  if (!p) return SPEC_ERR_INVALID_ARG;
  if (p->dtype != SPEC_F32 && p->dtype != SPEC_BF16) return SPEC_ERR_INVALID_ARG;
  if (p->B < 1 || p->N < 0 || p->T_max < 1 || p->T_max > SPEC_MAX_TREE) return SPEC_ERR_INVALID_ARG;
  if (p->H_q < 1 || p->H_kv < 1 || p->H_q % p->H_kv) return SPEC_ERR_INVALID_ARG;
  if (!p->prefix_len || !p->node_offset || !p->req_status) return SPEC_ERR_INVALID_ARG;
  if (p->N > 0 && (!p->q || !p->o || !p->anc_mask || !aligned16(p->q) || !aligned16(p->o)))
    return SPEC_ERR_INVALID_ARG;
  return kv8::check_cache(p->H_kv, p->head_dim, p->block_size, p->num_blocks,
                          p->max_blocks_per_req, p->k_cache, p->v_cache, p->k_scale, p->v_scale,
                          p->block_table);
}

static AttnKv8Dev make_dev(const spec_attn_kv8_params* p) {
  AttnKv8Dev d;
  d.q = p->q;
  d.k = static_cast<const uint8_t*>(p->k_cache);
  d.v = static_cast<const uint8_t*>(p->v_cache);
  d.k_scale = p->k_scale;
  d.v_scale = p->v_scale;
  d.block_table = p->block_table;
  d.prefix_len = p->prefix_len;
  d.node_offset = p->node_offset;
  d.anc = p->anc_mask;
  d.o = p->o;
  d.lse = p->lse;
  d.req_status = p->req_status;
  d.B = p->B; d.N = p->N; d.H_q = p->H_q; d.H_kv = p->H_kv; d.G = p->H_q / p->H_kv;
  d.d = p->head_dim; d.bs = p->block_size; d.T_max = p->T_max; d.W = (p->T_max + 31) / 32;
  d.num_blocks = p->num_blocks; d.max_blocks = p->max_blocks_per_req;
  const float scale = p->scale > 0.f ? p->scale : 1.f / sqrtf(float(p->head_dim));
  d.scale_log2 = scale * 1.4426950408889634f;
  return d;
}

}  // namespace spec

extern "C" {

size_t spec_attention_kv8_workspace_size(const spec_attn_kv8_params* p) {
  if (spec::check_attn_kv8(p) != SPEC_OK) return 0;
  const spec::AttnKv8Dev d = spec::make_dev(p);
  return spec::attn_kv8_tc_takes(d, p->dtype == SPEC_BF16) ? spec::attn_kv8_tc_workspace(d) : 256;
}

spec_status_t spec_tree_attention_kv8(const spec_attn_kv8_params* p, void* workspace,
                                      size_t ws_bytes, spec_stream_t stream) {
  using namespace spec;
  const spec_status_t st = check_attn_kv8(p);
  if (st != SPEC_OK) return st;
  if (p->N == 0) return SPEC_OK;
  const AttnKv8Dev d = make_dev(p);
  const cudaStream_t s = (cudaStream_t)stream;
  if (attn_kv8_tc_takes(d, p->dtype == SPEC_BF16))
    return launch_attn_kv8_tc(d, workspace, ws_bytes, s);
  const int chunks = (d.G + kv8_simt::kHeads - 1) / kv8_simt::kHeads;
  const long long ys = (long long)d.H_kv * chunks;
  if (ys > 65535) return SPEC_ERR_UNSUPPORTED;
  const dim3 grid(p->N, unsigned(ys));
  return launch_result(
      p->dtype == SPEC_BF16
          ? launch_pdl(attn_kv8_simt_kernel<__nv_bfloat16>, grid, dim3(kv8_simt::kThreads), 0, s, d)
          : launch_pdl(attn_kv8_simt_kernel<float>, grid, dim3(kv8_simt::kThreads), 0, s, d));
}

}  // extern "C"
