// What the two attention kernels over the 8-bit cache share: few rows a sequence
// (kvrp_attend_q8.cu) and many (kvrp_attend_q8_prompt.cu).
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kvrp.h"
#include "kvrp_ptx.h"
#include "kvrp_ptx_math.h"
#include "kvrp_q8.h"

namespace kvrp {
namespace attend_q8 {

using namespace kvrp::ptx;
using q8::flag;
using q8::kPage;
using q8::sequence;

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kShift = 7.f;       // weights of the accumulator are exp2(. + 7)
constexpr float kLazy = 8.f;        // how far a score may pass the running maximum
constexpr float kLeastFactor = 1.17549435e-38f;   // 2^-126: what a score is multiplied with where some are masked
constexpr float kZeroBlock = 0x1p-126f;    // a zero block's scale, which a page outside the pool reads as
constexpr int kMaxCtasPerSm = 2, kMaxCtas = 1024;   // bounds of the grid
constexpr int kMaxCols = 16;        // rows x group of the decode kernel

struct Params {
  const uint16_t* q;
  int64_t q_stride;
  uint16_t* out;
  float* lse;
  const uint8_t *k_pool, *v_pool;
  const float *k_scale, *v_scale;
  kvrp_seqs seqs;
  uint32_t* status;
  float* partial;       // [n_cta][2][cols][D + 4]: O, then max, accumulator max, sum; of a unit begun
                        // before this CTA's share, and of one that goes on after it
  int4* meta;           // [n_cta] (few rows) or [n_cta][2]: the unit whose first, not last, part this CTA holds
  int Hq, Hkv, g, n_cta, max_rows;
  int cols;             // (head, row) columns of a part: heads of a group x max_rows x g, or kPromptRows
  int hg, n_grp;        // few rows: KV heads a CTA takes together, their groups,
  int streams, rounds;  // warps that share a head's pages, rounds that merge them
  int unit_pages;       // a unit's cost beside its pages
  uint64_t g_inverse;   // 2^32 / g, rounded up
  float scale;          // softmax_scale * log2(e)
  long long wait_cycles;   // many rows: limit of the pipeline's waits
};

// The kernel for many rows: its columns (rows a partial result holds) and its launch,
// p.n_cta blocks.
constexpr int kPromptRows = 256;
cudaError_t launch_prompt(const CUtensorMap& kmap, const CUtensorMap& vmap, const Params& p, int head_dim, cudaStream_t stream);

#ifdef __CUDACC__
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Assignments that the compiler keeps inside their branch.
__device__ __forceinline__ void make_minus_inf(float& x) { asm volatile("mov.b32 %0, 0xff800000;" : "=f"(x)); }
__device__ __forceinline__ void make_zero(uint32_t& x) { asm volatile("mov.b32 %0, 0;" : "=r"(x)); }

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Bounded wait that ignores the abort flag: lets this CTA's own copies land before it exits.
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity, uint32_t* status) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (clock64() - t0 > kTimeoutCycles) {
      if (status) atomicOr(status, KVRP_DEV_TIMEOUT);
      return;
    }
  }
}

// What an accumulator is multiplied with in the end, 2^(om - m - 7) / l, in two factors: one alone leaves fp32's range
// where value scales are near its ends.
__device__ __forceinline__ float2 result_factors(float m, float om, float l) {
  if (l == 0.f) return make_float2(0.f, 0.f);
  const float d = om - m - kShift, half = fmaxf(0.5f * d, -100.f);   // d is -inf where all scales are 0
  return make_float2(ex2(half), ex2(d - half) / l);
}

__device__ __forceinline__ void write_idle(const Params& p, int D) {
  // idle places of the batch (length 0): zeros, and no tokens' log-sum-exp
  for (int s = blockIdx.x; s < p.seqs.n_seqs; s += gridDim.x) {
    int row0, rows, len;
    if (!sequence(p.seqs, s, row0, rows, len) || len != 0) continue;
    const int end = p.seqs.row_start ? p.seqs.row_start[s + 1] : s + 1;
    if (row0 < 0 || end > p.seqs.n_rows) {
      if (threadIdx.x == 0) flag(p.status, KVRP_DEV_BAD_LENGTH);
      continue;
    }
    for (int64_t i = (int64_t)row0 * p.Hq * D + threadIdx.x * 8; i < (int64_t)end * p.Hq * D; i += blockDim.x * 8)
      *reinterpret_cast<uint4*>(p.out + i) = make_uint4(0, 0, 0, 0);
    if (p.lse)
      for (int64_t i = (int64_t)row0 * p.Hq + threadIdx.x; i < (int64_t)end * p.Hq; i += blockDim.x) p.lse[i] = -INFINITY;
  }
}

#endif  // __CUDACC__

}  // namespace attend_q8
}  // namespace kvrp
