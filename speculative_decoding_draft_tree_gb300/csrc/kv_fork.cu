// spec_kv_fork: child sequences share the parent's full pages and copy its partial one.
//
// One CTA per (fork, layer).  A head's live rows of the partial page are one contiguous run of
// bytes, so the copy is 16-byte vectors over (cache, head, run); bound by those bytes when there
// are many forks and layers, by the chain status -> length -> table -> rows when there are few.
// Every CTA of a fork checks it alike (no fork reads what another one of the call writes: a
// child that is also a parent, or named twice, is refused), and the layer-0 CTA writes the table
// row, the length and the status.
//
// Measured (8-bit cache, 8 KV heads, head_dim 128): 64 forks, blocks of 64, 32 layers (252 MB) 35.4
// us, 7.1 TB/s (a part of the pages is still in L2); 2 forks, one layer 4.1 us.
#include "common.cuh"

namespace spec {

struct ForkDev {
  char* k;
  char* v;
  float* ks;
  float* vs;
  int64_t layer_stride_bytes, scale_layer_stride;
  int32_t* block_table;
  int32_t* kv_len;
  const int32_t* src;
  const int32_t* dst;
  const int32_t* new_block;
  int32_t* fork_status;
  int32_t B, F, H_kv, row_bytes, bs, num_blocks, max_blocks;
};

constexpr int kForkThreads = 256;

__global__ void __launch_bounds__(kForkThreads) kv_fork_kernel(ForkDev a) {
  pdl_wait();
  pdl_trigger();
  const int f = blockIdx.x, layer = blockIdx.y, tid = threadIdx.x;
  const int src = a.src[f], dst = a.dst[f], nb = a.new_block[f];
  bool clash = src < 0 || src >= a.B || dst < 0 || dst >= a.B;
  for (int g = tid; g < a.F; g += kForkThreads) {
    clash = clash || a.src[g] == dst || (g != f && a.dst[g] == dst);
  }
  int bad = __syncthreads_or(clash) ? SPEC_REQ_BAD_PARENT : 0;
  int L = 0, full = 0, rem = 0;
  if (!bad) {
    L = a.kv_len[src];
    full = L / a.bs;
    rem = L - full * a.bs;
    if (L < 0 || full + (rem > 0) > a.max_blocks) bad = SPEC_REQ_BAD_SIZE;
  }
  const int32_t* prow = a.block_table + size_t(bad ? 0 : src) * a.max_blocks;
  const int pages = bad ? 0 : full + (rem > 0);
  bool page_bad = !bad && rem > 0 && (nb < 0 || nb >= a.num_blocks);
  for (int i = tid; i < pages; i += kForkThreads) {
    const int pb = prow[i];
    page_bad = page_bad || pb < 0 || pb >= a.num_blocks || (rem > 0 && pb == nb);
  }
  // a fresh page named by another fork that copies into it, too (no fork of the call changes the
  // length of a request that is a src)
  bool twice = false;
  for (int g = tid; !bad && rem > 0 && g < a.F; g += kForkThreads) {
    if (g == f || a.new_block[g] != nb) continue;
    const int sg = a.src[g];
    twice = twice || (sg >= 0 && sg < a.B && a.kv_len[sg] % a.bs != 0);
  }
  if (__syncthreads_or(twice)) bad = SPEC_REQ_BAD_PARENT;
  if (__syncthreads_or(page_bad) && !bad) bad = SPEC_REQ_BAD_BLOCK;
  if (layer == 0 && tid == 0) a.fork_status[f] = bad;
  if (bad) return;
  if (layer == 0) {
    int32_t* crow = a.block_table + size_t(dst) * a.max_blocks;
    for (int i = tid; i < full; i += kForkThreads) crow[i] = prow[i];
    if (tid == 0) {
      if (rem > 0) crow[full] = nb;
      a.kv_len[dst] = L;
    }
  }
  if (rem == 0) return;
  const int pb = prow[full];
  const size_t head_bytes = size_t(a.bs) * a.row_bytes;
  const int run = rem * (a.row_bytes / 16);         // vectors of one head's live rows
  const size_t from = size_t(pb) * a.H_kv * head_bytes, to = size_t(nb) * a.H_kv * head_bytes;
  char* kb = a.k + layer * a.layer_stride_bytes;
  char* vb = a.v + layer * a.layer_stride_bytes;
  for (int i = tid; i < run * a.H_kv; i += kForkThreads) {
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
    for (int h = tid; h < a.H_kv; h += kForkThreads) {
      ks[size_t(nb) * a.H_kv + h] = ks[size_t(pb) * a.H_kv + h];
      vs[size_t(nb) * a.H_kv + h] = vs[size_t(pb) * a.H_kv + h];
    }
  }
}

}  // namespace spec

extern "C" spec_status_t spec_kv_fork(const spec_fork_params* p, spec_stream_t stream) {
  using namespace spec;
  if (!p) return SPEC_ERR_INVALID_ARG;
  if (p->dtype != SPEC_F32 && p->dtype != SPEC_BF16 && p->dtype != SPEC_E4M3)
    return SPEC_ERR_INVALID_ARG;
  if (p->B < 1 || p->F < 0 || p->H_kv < 1 || p->head_dim < 1 || p->block_size < 1 ||
      p->num_blocks < 1 || p->max_blocks_per_req < 1 || p->num_layers < 1 || p->layer_stride < 0 ||
      p->scale_layer_stride < 0)
    return SPEC_ERR_INVALID_ARG;
  const int64_t es = p->dtype == SPEC_F32 ? 4 : p->dtype == SPEC_BF16 ? 2 : 1;
  const int64_t row_bytes = int64_t(p->head_dim) * es;
  if (row_bytes % 16 || (p->layer_stride * es) % 16) return SPEC_ERR_INVALID_ARG;
  if (!p->k_cache || !p->v_cache || !aligned16(p->k_cache) || !aligned16(p->v_cache) ||
      !p->block_table || !p->kv_len)
    return SPEC_ERR_INVALID_ARG;
  if (p->dtype == SPEC_E4M3 && (!p->k_scale || !p->v_scale)) return SPEC_ERR_INVALID_ARG;
  if (p->F > 0 && (!p->src || !p->dst || !p->new_block || !p->fork_status))
    return SPEC_ERR_INVALID_ARG;
  if (p->num_layers > 65535) return SPEC_ERR_UNSUPPORTED;
  if (row_bytes / 16 * p->block_size * p->H_kv >= (1LL << 31)) return SPEC_ERR_UNSUPPORTED;
  if (p->F == 0) return SPEC_OK;
  ForkDev d;
  d.k = static_cast<char*>(p->k_cache);
  d.v = static_cast<char*>(p->v_cache);
  d.ks = p->dtype == SPEC_E4M3 ? p->k_scale : nullptr;
  d.vs = p->dtype == SPEC_E4M3 ? p->v_scale : nullptr;
  d.layer_stride_bytes = p->layer_stride * es;
  d.scale_layer_stride = p->scale_layer_stride;
  d.block_table = p->block_table;
  d.kv_len = p->kv_len;
  d.src = p->src;
  d.dst = p->dst;
  d.new_block = p->new_block;
  d.fork_status = p->fork_status;
  d.B = p->B; d.F = p->F; d.H_kv = p->H_kv; d.row_bytes = int(row_bytes); d.bs = p->block_size;
  d.num_blocks = p->num_blocks; d.max_blocks = p->max_blocks_per_req;
  return launch_result(launch_pdl(kv_fork_kernel, dim3(p->F, p->num_layers), dim3(kForkThreads),
                                  0, (cudaStream_t)stream, d));
}
