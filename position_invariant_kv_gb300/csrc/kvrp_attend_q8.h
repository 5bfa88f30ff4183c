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
constexpr int kFewHeads = 8;        // KV heads that a CTA of it takes together, at most: its warps

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
  // kv_attend_shared_q8 only: the tokens that all sequences begin with, and its passes' results
  const int32_t *prefix_table, *prefix_length;
  int prefix_pages;
  int all_rows, chunks; // few rows: a sequence's rows in up to `chunks` runs of max_rows, all_rows in all
  bool behind;          // few rows: launched behind the shared tokens' pass, on which nothing here depends
  float* dense;         // [n_rows][Hq][D + 4]: like `partial`, of a unit that one CTA held
  int2* found;          // [n_rows][n_grp], few rows: by a sequence's first row the CTA that begins a unit, and its
                        // parts (0: it is dense)
};

// Which tokens a kernel's rows attend over: all of their sequence's (kv_attend_q8); the shared ones, for all rows
// of the batch as if they were one sequence's, each row seeing all; those behind the shared ones; or both, read by
// each sequence for itself.
enum Part { kAll, kShared, kRest, kEach };

// The kernel for many rows: its columns (rows a partial result holds) and its launch,
// p.n_cta blocks.
constexpr int kPromptRows = 256;
// Tokens of its tiles: what TMEM holds.
__host__ __device__ constexpr int prompt_tokens(int head_dim) { return head_dim == 128 ? 80 : 128; }
// Beginning and ending a unit (its queries, the first scores, the results) takes a CTA as long as some
// tiles do; the shares count that, or the CTAs of a batch's many short units finish last.
constexpr int kUnitTiles = 6;   // 4: 222 us for 6 questions of 37 to 900 rows, 6: 220 (215 with a later step)
// The fewest CTAs' worth of a batch: a share is at least a unit's tiles and two more.
__host__ __device__ constexpr int64_t prompt_ctas(int64_t total) { return (total + kUnitTiles + 1) / (kUnitTiles + 2); }
// The units of the shared tokens' pass, tiles of kPromptRows (row, query head) pairs for each KV head, all over the same
// tokens, and the CTAs that take them.  In general the costs of all units are cut into equal shares, of which some end
// inside one unit and go on in the next, beginning it as well.  Where the tokens are so few that such shares are
// mostly beginnings, every unit is cut into `parts`, one a CTA, of three tiles or more, on two thirds of the SMs at most:
// the others begin the own tokens' pass, and more parts take the join longer (5 sequences over 4000 shared
// tokens and 300 own, 8 heads: 21.8 us, with all SMs 25.0, in shares 23.9; 3 over 1008, 4 KV heads: 17.9, in shares 21.5).
// Where parts would not be a third shorter than shares, shares are faster (4 over 16000: 25.3 us, in parts 29.6).
struct EvenUnits {
  int n_kv;             // token tiles of a unit
  int parts;            // 0: shares
  int64_t units, cost, total;   // shares: a unit's cost, all units'
  int64_t n_cta;
  __host__ __device__ EvenUnits(int64_t pairs, int heads, int tokens, int head_dim, int most_cta) {
    const int n = prompt_tokens(head_dim);
    n_kv = (tokens + n - 1) / n;
    units = n_kv == 0 ? 0 : (pairs + kPromptRows - 1) / kPromptRows * heads;
    cost = n_kv + kUnitTiles;
    total = units * cost;
    parts = 0;
    n_cta = 0;
    if (units == 0) return;
    n_cta = prompt_ctas(total) < most_cta ? prompt_ctas(total) : most_cta;
    if (units <= most_cta && total <= 12 * n_cta) {   // 32 bits from here on
      const int places = most_cta * 2 / 3 / (int)units, three = (n_kv + 2) / 3, k = places < three ? places : three;
      if (k > 0 && 3 * ((n_kv + k - 1) / k) <= 2 * (((int)total + (int)n_cta - 1) / (int)n_cta)) {
        parts = k;
        n_cta = units * k;
      }
    }
  }
  __host__ __device__ static int64_t div(int64_t a, int64_t b) {   // of numbers that are not negative
    return (uint64_t)(a | b) < (1ull << 31) ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
  }
  __host__ __device__ int part_begin(int i) const { return (int)div((int64_t)n_kv * i, parts); }
  __host__ __device__ int64_t share(int i) const { return div(total * i, n_cta); }   // where CTA i's costs begin
  // The first CTA with tiles of a unit, and how many have some.
  __host__ __device__ void find(int64_t unit, int& first, int& n) const {
    if (parts) {
      first = (int)unit * parts;
      n = parts;
    } else {   // the CTA whose costs hold x is the largest c with total c / n_cta not above it
      first = (int)div((unit * cost + kUnitTiles + 1) * n_cta - 1, total);
      n = (int)div((unit + 1) * cost * n_cta - 1, total) - first + 1;
    }
  }
};
cudaError_t launch_prompt(const CUtensorMap& kmap, const CUtensorMap& vmap, const Params& p, int head_dim, cudaStream_t stream,
                          Part part = kAll);
// The kernel for few rows, p.n_cta blocks.
cudaError_t launch_few(const Params& p, int head_dim, cudaStream_t stream, Part part);
void set_few(Params& p, int sms, int head_dim);   // p's fields for it
// Merges what that kernel (kAll, kEach) left in parts.
cudaError_t launch_combine(const Params& p, int head_dim, int sms, cudaStream_t stream);
// The host checks of both calls, and what they fill in of the parameters.
kvrp_status check_call(const char* fn, const void* q, int64_t& q_stride, const kvrp_seqs* seqs, int32_t n_q_heads,
                       int32_t n_kv_heads, int32_t head_dim, float softmax_scale, const void* k_pool, const void* v_pool,
                       const float* k_scale, const float* v_scale, void* out, float* lse, uint32_t* d_status, Params& p);
kvrp_status check_rows(const char* fn, const Params& p);
size_t meta_bytes(int n_cta);
int head_group(int n_kv_heads);
int sm_count();

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

// The shared tokens of kv_attend_shared_q8, in whole pages, and the batch's rows; tokens -1: out of range.
struct View {
  int tokens, first, end;
};
__device__ __forceinline__ View load_view(const Params& p) {
  View v;
  v.first = p.seqs.row_start ? p.seqs.row_start[0] : 0;
  v.end = p.seqs.row_start ? p.seqs.row_start[p.seqs.n_seqs] : p.seqs.n_rows;
  const int length = *p.prefix_length;
  const bool ok = length >= 0 && length / kPage <= p.prefix_pages && v.first >= 0 && v.end >= v.first && v.end <= p.seqs.n_rows;
  v.tokens = ok ? length / kPage * kPage : -1;
  return v;
}
// sequence() for the tokens behind the shared ones (kRest) or for all (kEach).  A sequence that is not behind them, or
// whose rows are not among the batch's, is bad.
template <Part kPart>
__device__ __forceinline__ bool own_sequence(const Params& p, int s, int& row0, int& rows, int& len) {
  const View v = load_view(p);
  bool ok = sequence(p.seqs, s, row0, rows, len);
  if (ok && rows > 0) {
    ok = v.tokens >= 0 && len - rows >= v.tokens && row0 >= v.first && row0 + rows <= v.end && rows <= p.all_rows;
    if (!ok) rows = 0;
    else if (kPart == kRest) len -= v.tokens;
  }
  return ok;
}
// The sequence whose run of rows number s is.
__device__ __forceinline__ int place_sequence(const Params& p, int s) {
  return p.chunks == 1 ? s : (int)((uint32_t)s / (uint32_t)p.chunks);
}
// sequence() for a part: rows, and the tokens that they see at most of it.  A run of a sequence's rows is a sequence
// that ends with its last row.
template <Part kPart>
__device__ __forceinline__ bool part_sequence(const Params& p, int s, int& row0, int& rows, int& len) {
  if constexpr (kPart == kAll) return sequence(p.seqs, s, row0, rows, len);
  if constexpr (kPart == kShared) {
    const View v = load_view(p);
    row0 = v.first;
    rows = v.tokens > 0 ? v.end - v.first : 0;
    len = max(v.tokens, 0);
    return true;
  }
  if (p.chunks == 1) return own_sequence<kPart>(p, s, row0, rows, len);
  const int seq = place_sequence(p, s), before = (s - seq * p.chunks) * p.max_rows;
  const bool ok = own_sequence<kPart>(p, seq, row0, rows, len);
  const int after = max(rows - before - p.max_rows, 0);
  len -= rows > 0 ? after : 0;
  row0 += before;
  rows = max(rows - before - after, 0);
  return ok;
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
