// spec_kv8_compact: the accepted path's rows committed to contiguous slots of an 8-bit cache.
//
// A row that moves into a block of another scale has to be requantised, and raising a block's
// scale requantises the rows that stay there, so the unit of work is a destination block: one
// warp per (request, head, cache, group of layers) takes the destination blocks of the accepted
// path in increasing order.  Because path[d] >= d, a block's rows come from itself or from later
// blocks, whose codes and scales the warp has not changed yet; within a block the rows move in
// increasing d, every load of a group before its stores, which gives gather semantics as if
// everything had been read first.  Warps share nothing.  Bound by the latency of dependent loads:
// what does not depend on the layer (path, pages, row offsets) is looked up once for a CTA's
// layers, and then a layer's scales and rows are loaded together, kLayersInFlight layers at a time.
//
// Measured (8 KV heads, head_dim 128, blocks of 16): 64 requests, 5 accepted rows, 32 layers (42 MB)
// 21.4 us, 2.0 TB/s of rows that lie apart; 16 requests, 3 rows, one layer 4 us.
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
  int32_t H_kv, d, bs, num_blocks, max_blocks, max_path, num_layers, layers_per_cta;
};

constexpr int kCompact8Threads = 256;
constexpr int kLayersInFlight = 2;   // 64 x 5, 32 layers: 21.4 us; 24.2 with 1, 23.4 with 4 (spills)

__global__ void __launch_bounds__(kCompact8Threads) kv8_compact_kernel(Compact8Dev a) {
  // per step of a chunk of the path: source page, source row, whether it moves
  constexpr int kChunk = 256;
  __shared__ int s_page[kChunk], s_row[kChunk];
  __shared__ int s_moves;
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31;
  const int P = a.prefix_len[r], na = a.n_acc[r];
  const int32_t* prow = a.path + size_t(r) * a.max_path;
  const int32_t* trow = a.block_table + size_t(r) * a.max_blocks;
  // Every CTA of the request checks its path alike.  The reporting CTA's bits may appear in the status
  // while another one reads it, so a CTA takes one verdict of it for all its threads: threads apart
  // would check some steps of the path, skip others, and move rows by those that nobody checked.
  if (tid == 0) s_moves = 0;
  bool ok = __syncthreads_and(a.req_status[r] == 0) && na >= 0 && na < a.max_path && P >= 0;
  int flags = 0;
  bool any = false;
  if (ok) {
    for (int d = tid; d <= na; d += kCompact8Threads) {
      const int pd = prow[d];
      const long long src = (long long)P + pd, dst = (long long)P + d;
      const bool good = (d == 0 ? pd == 0 : pd >= d) && src / a.bs < a.max_blocks &&
                        src <= (long long)INT32_MAX - 1024;   // (slot numbers stay in 32 bits)
      if (!good) {
        flags |= SPEC_REQ_BAD_PARENT;
      } else {
        const int sb = trow[src / a.bs], db = trow[dst / a.bs];
        if (sb < 0 || sb >= a.num_blocks || db < 0 || db >= a.num_blocks)
          flags |= SPEC_REQ_BAD_BLOCK;
        any = any || pd != d;
        if (d < kChunk) {
          s_page[d] = sb;
          s_row[d] = int(src % a.bs);
        }
      }
    }
  }
  if (flags & SPEC_REQ_BAD_PARENT) atomicOr(&s_moves, 2);
  if (flags & SPEC_REQ_BAD_BLOCK) atomicOr(&s_moves, 4);
  if (any) atomicOr(&s_moves, 1);
  __syncthreads();
  const int seen = s_moves;
  const int bad = ((seen & 2) ? SPEC_REQ_BAD_PARENT : 0) | ((seen & 4) ? SPEC_REQ_BAD_BLOCK : 0);
  const bool report = blockIdx.y == 0 && blockIdx.z == 0;
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
  if (!ok || !(seen & 1)) return;
  const int unit = blockIdx.z * (kCompact8Threads / 32) + (tid >> 5);
  if (unit >= 2 * a.H_kv) return;
  const int h = unit >> 1;
  uint8_t* const cache = (unit & 1) ? a.v : a.k;
  float* const scale = (unit & 1) ? a.vs : a.ks;
  const size_t page_bytes = size_t(a.bs) * a.d;
  auto page_at = [&](int pb) { return (size_t(pb) * a.H_kv + h) * page_bytes; };
  auto src_page = [&](int d) { return d < kChunk ? s_page[d] : trow[(P + prow[d]) / a.bs]; };
  auto src_row = [&](int d) { return d < kChunk ? s_row[d] : (P + prow[d]) % a.bs; };
  const int vpr = a.d / 16;
  const int group = 64 / vpr;                // rows whose vectors a warp holds, two a lane
  const int l0 = blockIdx.y * a.layers_per_cta, l1 = min(a.num_layers, l0 + a.layers_per_cta);
  for (int lb = P / a.bs; lb <= (P + na) / a.bs; ++lb) {
    const int d0 = max(0, lb * a.bs - P), d1 = min(na + 1, (lb + 1) * a.bs - P);
    const int kept = max(0, min(a.bs, P - lb * a.bs));
    bool moves = false;
    for (int d = d0 + lane; d < d1; d += 32) moves = moves || prow[d] != d;
    if (!__any_sync(0xffffffffu, moves)) continue;
    const int pb = trow[lb];
    const size_t own_at = size_t(pb) * a.H_kv + h;
    uint8_t* const to = cache + page_at(pb);
    for (int g0 = d0; g0 < d1; g0 += group) {
      // this lane's vectors of the group: where from, with which scale, where to
      const int nv = min(group, d1 - g0) * vpr;
      const uint8_t* from[2];
      uint8_t* dest[2];
      const float* from_scale[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int i = lane + 32 * q, rr = i / vpr, c = i - rr * vpr;
        const int d = g0 + min(rr, d1 - 1 - g0), sb = src_page(d);
        from[q] = cache + page_at(sb) + size_t(src_row(d)) * a.d + c * 16;
        from_scale[q] = scale + size_t(sb) * a.H_kv + h;
        dest[q] = to + size_t(P + d - lb * a.bs) * a.d + c * 16;
      }
      // the pages that the block's rows come from, one a lane (the first 32 rows; the rest below)
      const float* of_row = scale + size_t(src_page(min(d0 + lane, d1 - 1))) * a.H_kv + h;
      for (int layer = l0; layer < l1; layer += kLayersInFlight) {
        float own[kLayersInFlight], s[kLayersInFlight], ss[kLayersInFlight][2];
        uint4 v[kLayersInFlight][2];
#pragma unroll
        for (int u = 0; u < kLayersInFlight; ++u) {
          if (layer + u >= l1) continue;
          const int64_t so = (layer + u) * a.scale_layer_stride, co = (layer + u) * a.layer_stride;
          own[u] = scale[so + own_at];
          s[u] = of_row[so];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            if (lane + 32 * q < nv) {
              v[u][q] = *reinterpret_cast<const uint4*>(from[q] + co);
              ss[u][q] = from_scale[q][so];
            }
          }
        }
#pragma unroll
        for (int u = 0; u < kLayersInFlight; ++u) {
          if (layer + u >= l1) continue;
          const int64_t so = (layer + u) * a.scale_layer_stride, co = (layer + u) * a.layer_stride;
          for (int d = d0 + lane + 32; d < d1; d += 32)
            s[u] = fmaxf(s[u], scale[so + size_t(src_page(d)) * a.H_kv + h]);
          s[u] = warp_max(s[u]);
          if (kept > 0) s[u] = fmaxf(s[u], own[u]);
          if (g0 == d0 && kept > 0 && s[u] != own[u]) {
            const float ratio = __fdiv_rn(own[u], s[u]);
            uint4* p = reinterpret_cast<uint4*>(to + co);
            for (int i = lane; i < kept * vpr; i += 32) p[i] = kv8::rescale_e4m3x16(p[i], ratio);
          }
          __syncwarp();                      // the group is read before any of it is written
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            if (lane + 32 * q < nv) {
              uint4 w = v[u][q];
              if (ss[u][q] != s[u]) w = kv8::rescale_e4m3x16(w, __fdiv_rn(ss[u][q], s[u]));
              *reinterpret_cast<uint4*>(dest[q] + co) = w;
            }
          }
          // (a block's own scale is read by each of its groups)
          if (lane == 0 && g0 + group >= d1 && s[u] != own[u]) scale[so + own_at] = s[u];
        }
        __syncwarp();
      }
    }
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
  d.num_layers = p->num_layers;
  // as many layers to a CTA as leave the device full (64 requests, 32 layers: 21.4 us; 37.1 with
  // one layer a CTA, 29.8 with half as many CTAs)
  const long long ctas = (long long)p->B * p->num_layers * zs;
  d.layers_per_cta = int(ctas / 512 < 1 ? 1 : ctas / 512 > 8 ? 8 : ctas / 512);
  const int ys = (p->num_layers + d.layers_per_cta - 1) / d.layers_per_cta;
  return launch_result(launch_pdl(kv8_compact_kernel, dim3(p->B, ys, zs),
                                  dim3(kCompact8Threads), 0, (cudaStream_t)stream, d));
}
