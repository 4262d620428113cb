// spec_kv8_compact: the accepted path's rows committed to contiguous slots of an 8-bit cache.
//
// A row that moves into a block of another scale has to be requantised, and raising a block's
// scale requantises the rows that stay there, so the unit of work is a destination block: one
// warp per (request, layer, head, cache) takes the destination blocks of the accepted path in
// increasing order.  Because path[d] >= d, a block's rows come from itself or from later blocks,
// whose codes and scales the warp has not changed yet; within a block the rows move in increasing
// d, every load of a group before its stores, which gives gather semantics as if everything had
// been read first.  Warps share nothing, so one launch has B * layers * 2 H_kv independent
// chains; each is bound by the latency of its dependent loads (table entry, scale, row), the
// whole by the moved rows' bytes when there are many.
#include "kv8.cuh"

namespace spec {

struct Compact8Dev {
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  int64_t layer_stride, scale_layer_stride;
  const int32_t* block_table;
  const int32_t* prefix_len;
  const int32_t* path;
  const int32_t* n_acc;
  int32_t* req_status;
  int32_t* new_kv_len;
  int32_t* slot_map;
  int32_t* blocks_in_use;
  int32_t H_kv, d, bs, num_blocks, max_blocks, max_path;
};

constexpr int kCompact8Threads = 256;

__global__ void __launch_bounds__(kCompact8Threads) kv8_compact_kernel(Compact8Dev a) {
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.x, layer = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 31;
  const int P = a.prefix_len[r], na = a.n_acc[r];
  const int32_t* prow = a.path + size_t(r) * a.max_path;
  const int32_t* trow = a.block_table + size_t(r) * a.max_blocks;
  // every CTA of the request checks its path alike
  bool ok = a.req_status[r] == 0 && na >= 0 && na < a.max_path && P >= 0;
  int flags = 0;
  if (ok) {
    for (int d = tid; d <= na; d += kCompact8Threads) {
      const int pd = prow[d];
      const long long src = (long long)P + pd, dst = (long long)P + d;
      const bool good = (d == 0 ? pd == 0 : pd >= d) && src / a.bs < a.max_blocks;
      if (!good) {
        flags |= SPEC_REQ_BAD_PARENT;
      } else {
        const int sb = trow[src / a.bs], db = trow[dst / a.bs];
        if (sb < 0 || sb >= a.num_blocks || db < 0 || db >= a.num_blocks)
          flags |= SPEC_REQ_BAD_BLOCK;
      }
    }
  }
  const int bad_parent = __syncthreads_or(flags & SPEC_REQ_BAD_PARENT);
  const int bad_block = __syncthreads_or(flags & SPEC_REQ_BAD_BLOCK);
  const int bad = (bad_parent ? SPEC_REQ_BAD_PARENT : 0) | (bad_block ? SPEC_REQ_BAD_BLOCK : 0);
  const bool report = layer == 0 && blockIdx.z == 0;
  if (bad && report && tid == 0) atomicOr(&a.req_status[r], bad);
  ok = ok && !bad;
  if (report) {
    for (int d = tid; d < a.max_path; d += kCompact8Threads) {
      const bool in = ok && d <= na;
      a.slot_map[(size_t(r) * a.max_path + d) * 2] = in ? P + prow[d] : -1;
      a.slot_map[(size_t(r) * a.max_path + d) * 2 + 1] = in ? P + d : -1;
    }
    if (tid == 0) {
      const int len = ok ? P + na + 1 : P;
      a.new_kv_len[r] = len;
      a.blocks_in_use[r] = (len + a.bs - 1) / a.bs;
    }
  }
  if (!ok) return;
  const int unit = blockIdx.z * (kCompact8Threads / 32) + (tid >> 5);
  if (unit >= 2 * a.H_kv) return;
  const int h = unit >> 1;
  uint8_t* cache = ((unit & 1) ? a.v : a.k) + layer * a.layer_stride;
  float* scale = ((unit & 1) ? a.vs : a.ks) + layer * a.scale_layer_stride;
  const size_t page_bytes = size_t(a.bs) * a.d;
  auto page = [&](int pb) { return cache + (size_t(pb) * a.H_kv + h) * page_bytes; };
  const int vpr = a.d / 16;
  const int group = 128 / vpr;               // rows whose vectors a warp holds, four a lane
  for (int lb = P / a.bs; lb <= (P + na) / a.bs; ++lb) {
    const int d0 = max(0, lb * a.bs - P), d1 = min(na + 1, (lb + 1) * a.bs - P);
    const int kept = max(0, min(a.bs, P - lb * a.bs));
    const int pb = trow[lb];
    float* sp = scale + size_t(pb) * a.H_kv + h;
    const float own = *sp;
    float s = kept > 0 ? own : 0.f;
    bool moves = false;
    for (int d = d0 + lane; d < d1; d += 32) {
      const int pd = prow[d];
      moves = moves || pd != d;
      s = fmaxf(s, scale[size_t(trow[(P + pd) / a.bs]) * a.H_kv + h]);
    }
    if (!__any_sync(0xffffffffu, moves)) continue;
    s = warp_max(s);
    uint8_t* to = page(pb);
    if (kept > 0 && s != own) {
      const float ratio = __fdiv_rn(own, s);
      uint4* p = reinterpret_cast<uint4*>(to);
      for (int i = lane; i < kept * vpr; i += 32) p[i] = kv8::rescale_e4m3x16(p[i], ratio);
    }
    for (int g0 = d0; g0 < d1; g0 += group) {
      const int nv = min(group, d1 - g0) * vpr;
      uint4 v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int i = lane + 32 * q;
        if (i < nv) {
          const int rr = i / vpr, c = i - rr * vpr;
          const int src = P + prow[g0 + rr];
          const int sb = trow[src / a.bs];
          v[q] = *reinterpret_cast<const uint4*>(page(sb) + size_t(src % a.bs) * a.d + c * 16);
          const float ss = scale[size_t(sb) * a.H_kv + h];
          if (ss != s) v[q] = kv8::rescale_e4m3x16(v[q], __fdiv_rn(ss, s));
        }
      }
      __syncwarp();                          // the group is read before any of it is written
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int i = lane + 32 * q;
        if (i < nv) {
          const int rr = i / vpr, c = i - rr * vpr;
          *reinterpret_cast<uint4*>(to + size_t((P + g0 + rr) % a.bs) * a.d + c * 16) = v[q];
        }
      }
      __syncwarp();
    }
    if (lane == 0 && s != own) *sp = s;
    __syncwarp();
  }
}

}  // namespace spec

extern "C" spec_status_t spec_kv8_compact(const spec_kv8_compact_params* p, spec_stream_t stream) {
  using namespace spec;
  if (!p) return SPEC_ERR_INVALID_ARG;
  if (p->B < 1 || p->num_layers < 1 || p->max_path < 1 || p->layer_stride < 0 ||
      p->scale_layer_stride < 0)
    return SPEC_ERR_INVALID_ARG;
  const spec_status_t st =
      kv8::check_cache(p->H_kv, p->head_dim, p->block_size, p->num_blocks, p->max_blocks_per_req,
                       p->k_cache, p->v_cache, p->k_scale, p->v_scale, p->block_table);
  if (st != SPEC_OK) return st;
  if (p->layer_stride % 16) return SPEC_ERR_INVALID_ARG;
  if (!p->prefix_len || !p->path || !p->n_acc || !p->req_status || !p->new_kv_len ||
      !p->slot_map || !p->blocks_in_use)
    return SPEC_ERR_INVALID_ARG;
  const int zs = (2 * p->H_kv + kCompact8Threads / 32 - 1) / (kCompact8Threads / 32);
  if (p->num_layers > 65535 || zs > 65535) return SPEC_ERR_UNSUPPORTED;
  Compact8Dev d;
  d.k = static_cast<uint8_t*>(p->k_cache);
  d.v = static_cast<uint8_t*>(p->v_cache);
  d.ks = p->k_scale;
  d.vs = p->v_scale;
  d.layer_stride = p->layer_stride;
  d.scale_layer_stride = p->scale_layer_stride;
  d.block_table = p->block_table;
  d.prefix_len = p->prefix_len;
  d.path = p->path;
  d.n_acc = p->n_acc;
  d.req_status = p->req_status;
  d.new_kv_len = p->new_kv_len;
  d.slot_map = p->slot_map;
  d.blocks_in_use = p->blocks_in_use;
  d.H_kv = p->H_kv; d.d = p->head_dim; d.bs = p->block_size; d.num_blocks = p->num_blocks;
  d.max_blocks = p->max_blocks_per_req; d.max_path = p->max_path;
  return launch_result(launch_pdl(kv8_compact_kernel, dim3(p->B, p->num_layers, zs),
                                  dim3(kCompact8Threads), 0, (cudaStream_t)stream, d));
}
