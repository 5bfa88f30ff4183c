// The 8-bit cache block, shared by the kernels that write it and the ones that read it.
//
// A block is the 16 tokens x head_dim values of one (page, KV head).  It stands for
// e4m3 value x scale, with one fp32 scale
//     scale = 2^max(-126, ceil(log2(amax / 448))),
// amax over the block's finite values.  e4m3 keeps 4 significant bits whatever the
// scale, so a power of two costs no precision against amax / 448 and buys two things:
// quantising divides exactly, and a block that grows (an append into an open page) is
// moved to a larger scale by a shift, which is exact down to e4m3's subnormals instead
// of one more rounding of every value.  A value that is not finite is stored as NaN.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kvrp.h"

namespace kvrp {
namespace q8 {

constexpr int kPage = 16;   // tokens per page (and per block)
constexpr int kMostTokens = 0x7fffff00;   // of a sequence: a tile more stays an int

#ifdef __CUDACC__

__device__ __forceinline__ void flag(uint32_t* status, uint32_t bit) {
  if (status) atomicOr(status, bit);
}
// The rows and length of sequence s; false (and rows 0) where they are out of range.
// A sequence of length 0 is an idle place of the batch: no rows, and nothing wrong.
__device__ __forceinline__ bool sequence(const kvrp_seqs& q, int s, int& row0, int& rows, int& len) {
  row0 = q.row_start ? q.row_start[s] : s;
  const int end = q.row_start ? q.row_start[s + 1] : s + 1;
  len = q.seq_lens[s];
  rows = end - row0;
  const bool ok = row0 >= 0 && end >= row0 && end <= q.n_rows && len >= rows &&
                  len <= kMostTokens && (int64_t)len <= (int64_t)q.table_stride * kPage;
  if (!ok || len == 0) rows = 0;
  return ok || len == 0;
}

// The scale of a block whose largest finite magnitude is amax: the exponent of the
// least power of two s with amax <= 448 s = 1.75 * 2^8 s, read off amax's own bits.
__device__ __forceinline__ float scale_of(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return __uint_as_float((uint32_t)(max(e, -126) + 127) << 23);
}
// Four finite values to e4m3 bytes (x * inv, |x * inv| <= 448).
__device__ __forceinline__ uint32_t finite_to_e4m3x4(float a, float b, float c, float d, float inv) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(__fmul_rn(b, inv)), "f"(__fmul_rn(a, inv)));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(__fmul_rn(d, inv)), "f"(__fmul_rn(c, inv)));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}
// The same for any values; inf and NaN become NaN.
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d, float inv) {
  a = __fmaf_rn(a, 0.f, __fmul_rn(a, inv));   // + 0 for a finite value, NaN for inf and NaN
  b = __fmaf_rn(b, 0.f, __fmul_rn(b, inv));
  c = __fmaf_rn(c, 0.f, __fmul_rn(c, inv));
  d = __fmaf_rn(d, 0.f, __fmul_rn(d, inv));
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}
// Two e4m3 bytes to an f16 pair (exact: every e4m3 value is an f16 value).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
  return r;
}
// The NaN among four e4m3 bytes (0x7f, with any sign), as bits 0x80 of them.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t v) { return ((v & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

#endif  // __CUDACC__

}  // namespace q8

// Tensor map of an 8-bit pool [num_pages][16][row_bytes] whose box is one head of one page:
// head_dim bytes (128- or 64-byte swizzle) of its 16 slots.  Coordinates (head * head_dim, 0, page).
kvrp_status encode_q8_pool(CUtensorMap* map, const void* pool, int num_pages, int row_bytes, int head_dim);

// Host checks that the entry points over a ragged batch (kvrp_seqs) share.
kvrp_status check_seqs(const char* fn, const kvrp_seqs* s);
kvrp_status check_heads(const char* fn, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim);

}  // namespace kvrp
