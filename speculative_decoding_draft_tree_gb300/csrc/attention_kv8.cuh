// Device arguments and request checks shared by the kernels of spec_tree_attention_kv8.
#pragma once

#include "kv8.cuh"

namespace spec {

struct AttnKv8Dev {
  const void* q;
  const uint8_t* k;
  const uint8_t* v;
  const float* k_scale;
  const float* v_scale;
  const int32_t* block_table;
  const int32_t* prefix_len;
  const int32_t* node_offset;
  const uint32_t* anc;
  void* o;
  float* lse;
  int32_t* req_status;
  int32_t B, N, H_q, H_kv, G, d, bs, T_max, W, num_blocks, max_blocks;
  float scale_log2;
};

enum class Kv8Live { yes, no, beyond_table };

// Whether request r has rows to compute.  The bits this call sets itself (BAD_BLOCK, TIMEOUT) are
// ignored, so that every CTA decides alike.
__device__ __forceinline__ Kv8Live kv8_live(const AttnKv8Dev& a, int r, int T, int P) {
  const int st = a.req_status[r] & ~(SPEC_REQ_BAD_BLOCK | SPEC_REQ_TIMEOUT);
  if (st != 0 || T < 1 || T > a.T_max || P < 0) return Kv8Live::no;
  // (slot numbers and a tile past them stay in 32 bits)
  const long long end = min((long long)a.max_blocks * a.bs, (long long)INT32_MAX - 1024);
  return (long long)P + T <= end ? Kv8Live::yes : Kv8Live::beyond_table;
}

}  // namespace spec
