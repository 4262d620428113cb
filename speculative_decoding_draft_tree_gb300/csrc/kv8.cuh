// The 8-bit K/V cache's number format: e4m3 conversions, a block's power-of-two scale and the
// requantisation of codes from one scale to another.  Shared by the kernels that write the
// cache (append, compaction) and the ones that read it (attention).
#pragma once

#include <float.h>

#include "common.cuh"

namespace spec {
namespace kv8 {

constexpr int kMinScaleExp = 27;    // biased exponent of 2^-100
constexpr int kMaxScaleExp = 246;   // of 2^119: 448 * 2^119 is below FLT_MAX

// Smallest power of two s with a <= 448 s, kept in [2^-100, 2^119] (a >= 0, finite).  448 =
// 1.75 * 2^8: the exponent of a moves up by one exactly when its mantissa field exceeds 1.75's
// (0x600000), which is the carry of the addition.  A power of two loses nothing against a / 448:
// e4m3 is a floating-point format, so its relative rounding error does not depend on the scale;
// at most one binade at the subnormal end goes unused.  In return a scale that grows requantises
// the rows already there exactly.
__device__ __forceinline__ float need_scale(float a) {
  int e = int((__float_as_uint(a) + 0x1FFFFFu) >> 23) - 8;
  e = e < kMinScaleExp ? kMinScaleExp : (e > kMaxScaleExp ? kMaxScaleExp : e);
  return __uint_as_float(uint32_t(e) << 23);
}

// two fp32 -> two e4m3 codes (a in the low byte), to nearest even, saturating at +-448
__device__ __forceinline__ uint32_t pack_e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  return pack_e4m3x2(a, b) | (pack_e4m3x2(c, d) << 16);
}
// two codes -> two halves (exact: every e4m3 value is an fp16 value)
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(uint16_t(v)));
  return r;
}
__device__ __forceinline__ float f16_lo(uint32_t v) {
  float f;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(f) : "r"(v));
  return f;
}
__device__ __forceinline__ float f16_hi(uint32_t v) {
  float f;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, h;\n\t}" : "=f"(f) : "r"(v));
  return f;
}
// four codes of a 32-bit word as fp32
__device__ __forceinline__ void unpack_e4m3x4(uint32_t w, float (&f)[4]) {
  const uint32_t lo = e4m3x2_to_f16x2(w & 0xFFFFu), hi = e4m3x2_to_f16x2(w >> 16);
  f[0] = f16_lo(lo);
  f[1] = f16_hi(lo);
  f[2] = f16_lo(hi);
  f[3] = f16_hi(hi);
}
// codes times a ratio of scales, rounded to e4m3 again
__device__ __forceinline__ uint32_t rescale_e4m3x4(uint32_t w, float ratio) {
  float f[4];
  unpack_e4m3x4(w, f);
  return pack_e4m3x4(f[0] * ratio, f[1] * ratio, f[2] * ratio, f[3] * ratio);
}
__device__ __forceinline__ uint4 rescale_e4m3x16(uint4 v, float ratio) {
  return make_uint4(rescale_e4m3x4(v.x, ratio), rescale_e4m3x4(v.y, ratio),
                    rescale_e4m3x4(v.z, ratio), rescale_e4m3x4(v.w, ratio));
}

// host: the shape checks that the entry points of the 8-bit cache share
inline spec_status_t check_cache(int H_kv, int head_dim, int block_size, int num_blocks,
                                 int max_blocks, const void* k, const void* v, const void* ks,
                                 const void* vs, const void* table) {
  if (H_kv < 1 || head_dim < 1 || block_size < 1 || num_blocks < 1 || max_blocks < 1)
    return SPEC_ERR_INVALID_ARG;
  if (!k || !v || !ks || !vs || !table || !aligned16(k) || !aligned16(v))
    return SPEC_ERR_INVALID_ARG;
  if (head_dim % 16 || head_dim > 256 || block_size > 1024) return SPEC_ERR_UNSUPPORTED;
  if ((long long)num_blocks * H_kv * block_size >= (1LL << 31)) return SPEC_ERR_UNSUPPORTED;
  if ((long long)max_blocks * block_size >= (1LL << 31)) return SPEC_ERR_UNSUPPORTED;
  return SPEC_OK;
}

}  // namespace kv8
}  // namespace spec
