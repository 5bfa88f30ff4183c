// New rows into the paged cache (kv_append, kv_append_q8) and bf16 pages into the
// 8-bit cache (kv_pack_q8).
//
// append_kernel.  Row x of a query or key head becomes
//     y = w * x * rsqrt(mean(x^2) + eps)          (where norm weights are given)
//     (y_i, y_{i+d/2}) -> (y_i cos a_i - y_{i+d/2} sin a_i, y_{i+d/2} cos a_i + y_i sin a_i),
// a_i = position * theta^(-2i/d), all in fp32 and rounded once at the store; values
// pass through.  What it costs is bytes: every row is read once and written once.
//   - The unit is a run: the new rows of one sequence inside one 16-token page, for one
//     head, held by one warp in registers as they came.  A run is exactly the part of an
//     8-bit block that the call writes, so the block's amax is a warp reduction and the rows
//     are rounded once, straight from fp32.
//   - A CTA takes one run and a share of its heads.  cos and sin of the run's rows are
//     formed once per CTA, in shared memory, while the first head's loads are in flight:
//     per head they would cost more issue slots than the rotation.
//   - The angle mod 2 pi comes from 64-bit integer arithmetic: the frequency as a
//     fraction of a turn in units of 2^-64, times the position, wraps by itself; fp64
//     (1/64 of the fp32 rate here) is not touched.
//   - 80 registers a thread, three CTAs an SM: what bounds a prompt is how many loads are in
//     flight.  The 8-bit form loads the next head's rows as it is done with this one's; in the
//     bf16 form that measured slower (40.7 against 35.6 us) and it loads a head at a time.
//   Measured: 8 sequences, 8719 rows of 28 + 2 x 4 heads x 128 with norms and M-RoPE, 160 MB, 35.6 us
//   (4.5 TB/s, 67% of a copy); 6790 rows of 32 + 2 x 32 heads into 8 bits, 278 MB, 58.1 us (71%);
//   one row of each of 16 sequences 3.0 us, of 64 into 8 bits 4.5 us (launch and latency).
//
// pack_kernel.  One warp a block: 16 rows of one head of one layer in registers, amax (two bf16
// magnitudes an instruction), scale, one rounding, 16 rows out.  63 registers keep 32 warps of loads
// in flight on an SM: 28 layers x 4096 tokens x 4 heads x 128, 352 MB, in 52.7 us, a copy's rate
// (72.4 us when the largest magnitude was taken in fp32: 106 registers, half the warps).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "kvrp.h"
#include "kvrp_plan.h"
#include "kvrp_ptx.h"
#include "kvrp_ptx_math.h"
#include "kvrp_q8.h"

namespace kvrp {
namespace append {

using namespace kvrp::ptx;
using q8::flag;
using q8::kPage;
using q8::sequence;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

struct Params {
  const uint16_t *q, *k, *v, *q_norm, *k_norm;
  int64_t q_stride, k_stride, v_stride;
  uint16_t* q_out;
  void *k_pool, *v_pool;
  float *k_scale, *v_scale;
  const int32_t* positions;
  kvrp_seqs seqs;
  uint32_t* status;
  int Hq, Hkv, h0;        // head slots [h0, Hq + 2 Hkv): queries, keys, values (h0 = Hq without q)
  int splits;             // CTAs that share a run's heads
  float eps;
  int sec1, sec2;         // first frequency pair of the second and third M-RoPE section
  int mrope;
  uint64_t turn[64];      // theta^(-2i/d) / (2 pi), in units of 2^-64 turns
};

// One run: rows [row0, row0 + n) are the tokens at positions pos0 .. of sequence seq.
struct Run {
  int seq, row0, n, pos0;
};

// Run number `want` of the batch.  With one row per sequence that is sequence `want`;
// else the CTA scans the sequences' run counts, 256 at a time.
__device__ __forceinline__ bool find_run(const Params& p, int want, Run* out, int* sh) {
  const kvrp_seqs& q = p.seqs;
  if (!q.row_start) {
    int row0, rows, len;
    if (!sequence(q, want, row0, rows, len) && threadIdx.x == 0) flag(p.status, KVRP_DEV_BAD_LENGTH);
    if (rows == 0) return false;
    *out = Run{want, row0, 1, len - 1};
    return true;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (want == 0)   // tells what is out of range past the first pass, which the scan below may leave before
    for (int s = kThreads + threadIdx.x; s < q.n_seqs; s += kThreads) {
      int row0, rows, len;
      if (!sequence(q, s, row0, rows, len)) flag(p.status, KVRP_DEV_BAD_LENGTH);
    }
  int before = 0;   // runs of the sequences scanned so far
  for (int s0 = 0; s0 < q.n_seqs; s0 += kThreads) {
    const int s = s0 + threadIdx.x;
    int row0 = 0, rows = 0, len = 0, runs = 0;
    if (s < q.n_seqs) {
      if (!sequence(q, s, row0, rows, len) && want == 0 && s0 == 0) flag(p.status, KVRP_DEV_BAD_LENGTH);
      if (rows > 0) runs = (len - 1) / kPage - (len - rows) / kPage + 1;
    }
    int sum = runs;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += t;
    }
    if (lane == 31) sh[warp] = sum;
    if (threadIdx.x == 0) sh[kWarps] = -1;
    __syncthreads();
    int all = 0, mine = before + sum - runs;   // runs of this pass, and before this sequence
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) mine += sh[w];
      all += sh[w];
    }
    if (want >= mine && want < mine + runs) {
      const int i = want - mine, first = len - rows;          // the sequence's i-th page of new rows
      const int a = i == 0 ? first : (first / kPage + i) * kPage;
      const int b = min((first / kPage + i + 1) * kPage, len);
      sh[kWarps] = s;
      sh[kWarps + 1] = row0 + a - first;
      sh[kWarps + 2] = b - a;
      sh[kWarps + 3] = a;
    }
    __syncthreads();
    const bool found = sh[kWarps] >= 0;
    if (found) *out = Run{sh[kWarps], sh[kWarps + 1], sh[kWarps + 2], sh[kWarps + 3]};
    __syncthreads();
    if (found) return true;
    before += all;
  }
  return false;
}

__device__ __forceinline__ void unpack8(const uint4& u, float* x) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
// The same as fp32 pairs, and back.
__device__ __forceinline__ void widen8(const uint4& u, uint64_t* x) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = pair2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ uint4 narrow8(const uint64_t* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = unpair2(x[i]);
    const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint32_t pairs_to_e4m3x4(uint64_t a, uint64_t b, float inv) {
  const float2 x = unpair2(a), y = unpair2(b);
  return q8::to_e4m3x4(x.x, x.y, y.x, y.y, inv);
}
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.f;   // false for NaN too
}

// cos and sin of an angle in units of 2^-64 turns.  The nearest quarter turn is taken off
// in integers, so the fp32 angle is at most 1/8 turn and its rounding 2^-25 of that.
__device__ __forceinline__ void turn_of(uint64_t turns, float* c, float* s) {
  const uint32_t quarter = (uint32_t)((turns + (1ull << 61)) >> 62);
  const int32_t rest = (int32_t)((int64_t)(turns - ((uint64_t)quarter << 62)) >> 30);   // units of 2^-34 turns
  float cs, sn;
  sincospif((float)rest * 0x1p-33f, &sn, &cs);
  const float a = quarter & 1 ? sn : cs, b = quarter & 1 ? cs : sn;
  *c = (quarter + 1) & 2 ? -a : a;
  *s = quarter & 2 ? -b : b;
}

// Moves the rows < n_old of a block to a larger scale.
template <int D>
__device__ __forceinline__ void rescale_block(uint8_t* block, int64_t row_stride, int n_old, float ratio) {
  for (int i = threadIdx.x & 31; i < n_old * (D / 4); i += 32) {
    uint32_t* at = reinterpret_cast<uint32_t*>(block + (int64_t)(i / (D / 4)) * row_stride + (i % (D / 4)) * 4);
    const uint32_t v = *at;
    const uint32_t lo = q8::e4m3x2_to_f16x2((uint16_t)v), hi = q8::e4m3x2_to_f16x2((uint16_t)(v >> 16));
    float f[4];
    asm("{.reg .f16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}" : "=f"(f[0]), "=f"(f[1]) : "r"(lo));
    asm("{.reg .f16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}" : "=f"(f[2]), "=f"(f[3]) : "r"(hi));
    *at = q8::to_e4m3x4(f[0], f[1], f[2], f[3], ratio);
  }
}

template <int D, bool kQ8>
__global__ void __launch_bounds__(kThreads, 3) append_kernel(const __grid_constant__ Params p) {
  constexpr int kLanes = D / 16;          // lanes of a row: 8 features and their 8 partners each
  constexpr int kStep = 32 / kLanes;      // rows a warp holds side by side
  constexpr int kSteps = kPage / kStep;
  __shared__ int sh[kWarps + 4];
  // cos and sin of pairs (2j, 2j + 1) of a lane's 8 features: [row][j][lane]
  __shared__ float4 table[kPage * 4 * kLanes];
  pdl_wait();
  pdl_launch_dependents();
  Run run;
  if (!find_run(p, blockIdx.x / p.splits, &run, sh)) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int sub = lane / kLanes, l = lane % kLanes;
  const int heads = p.Hq + 2 * p.Hkv, half = D / 2;
  const int first = p.h0 + (blockIdx.x % p.splits) * kWarps + warp, hop = p.splits * kWarps;

  // The rows of one head, as they came: a lane's 8 features and their partners, for each step of rows.
  uint4 raw[kSteps][2];
  auto load_step = [&](int h, int i) {
    const uint16_t* base;
    int64_t stride;
    if (h < p.Hq) base = p.q + (int64_t)h * D, stride = p.q_stride;
    else if (h < p.Hq + p.Hkv) base = p.k + (int64_t)(h - p.Hq) * D, stride = p.k_stride;
    else base = p.v + (int64_t)(h - p.Hq - p.Hkv) * D, stride = p.v_stride;
    const int r = i * kStep + sub;
    raw[i][0] = raw[i][1] = make_uint4(0, 0, 0, 0);
    if (r < run.n) {
      const uint16_t* at = base + (run.row0 + r) * stride + l * 8;
      raw[i][0] = *reinterpret_cast<const uint4*>(at);
      raw[i][1] = *reinterpret_cast<const uint4*>(at + half);
    }
  };
  if (first < heads) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) load_step(first, i);
  }

  const int page = p.seqs.block_tables[(int64_t)run.seq * p.seqs.table_stride + run.pos0 / kPage];
  const int slot0 = run.pos0 % kPage;
  const bool page_ok = page >= 0 && page < p.seqs.num_pages;
  if (!page_ok && tid == 0) flag(p.status, KVRP_DEV_BAD_PAGE);

  for (int i = tid; i < run.n * (half / 2); i += kThreads) {   // two pairs each
    const int r = i / (half / 2), pair = i % (half / 2) * 2;
    float4 cs;
    float* c = reinterpret_cast<float*>(&cs);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int f = pair + e;
      int64_t at = run.pos0 + r;
      if (p.positions) {
        const int sec = p.mrope ? (f >= p.sec1) + (f >= p.sec2) : 0;
        at = p.positions[(int64_t)sec * p.seqs.n_rows + run.row0 + r];
      }
      turn_of((uint64_t)at * p.turn[f], &c[e], &c[2 + e]);
    }
    table[(r * 4 + (pair / 2) % 4) * kLanes + pair / 8] = cs;
  }
  __syncthreads();

  // A step's rows of a query or key head, normed and turned: features in pairs, two an instruction.
  auto turn = [&](int i, const uint4 (&w)[2], bool normed, uint64_t (&x)[8]) {
    widen8(raw[i][0], x);
    widen8(raw[i][1], x + 4);
    if (normed) {
      uint64_t ss2 = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss2 = fma2(x[e], x[e], ss2);
      const float2 s2 = unpair2(ss2);
      float ss = s2.x + s2.y;
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float inv = rsqrtf(ss * (1.f / D) + p.eps);
      const uint64_t inv2 = pair2(inv, inv);
      uint64_t w2[8];
      widen8(w[0], w2);
      widen8(w[1], w2 + 4);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = mul2(x[e], mul2(w2[e], inv2));
    }
    const int r = i * kStep + sub;
    const uint64_t minus = pair2(-1.f, -1.f);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 cs = table[((r < run.n ? r : 0) * 4 + j) * kLanes + l];
      const uint64_t c = pair2(cs.x, cs.y), s = pair2(cs.z, cs.w);
      const uint64_t a = x[j], b = x[4 + j];
      x[j] = fma2(a, c, mul2(b, mul2(s, minus)));
      x[4 + j] = fma2(b, c, mul2(a, s));
    }
  };

  // One head; kLive of the run's steps have rows.  Without a way out between the steps they overlap.
  auto do_head = [&](int h, auto live_steps) {
    constexpr int kLive = decltype(live_steps)::value;
    const bool is_q = h < p.Hq, turned = h < p.Hq + p.Hkv;
    const int hk = h - p.Hq - (turned ? 0 : p.Hkv);   // the KV head of a key or value slot
    if (!kQ8 && h != first) {
#pragma unroll
      for (int i = 0; i < kLive; ++i) load_step(h, i);
    }
    uint4 w[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    const uint16_t* weights = is_q ? p.q_norm : p.k_norm;
    const bool normed = turned && weights != nullptr;
    if (normed) {
      w[0] = *reinterpret_cast<const uint4*>(weights + l * 8);
      w[1] = *reinterpret_cast<const uint4*>(weights + half + l * 8);
    }
    const int64_t row_values = (int64_t)p.Hkv * D;
    const int64_t block = (int64_t)page * kPage * row_values + (int64_t)hk * D;
    uint8_t* pool8 = static_cast<uint8_t*>(turned ? p.k_pool : p.v_pool) + block;
    float inv = 1.f;
    if (kQ8 && !is_q && page_ok) {
      // The block's scale comes first.  A key is turned once for it and once for the store: holding the
      // run's turned rows instead takes 64 registers a lane, and the warps that hide the loads.
      float* scale_at = (turned ? p.k_scale : p.v_scale) + (int64_t)page * p.Hkv + hk;
      const float old_scale = slot0 > 0 ? *scale_at : 0.f;   // a fresh block begins at 0
      float amax = 0.f;   // rows past the run are zeros
#pragma unroll
      for (int i = 0; i < kLive; ++i) {
        uint64_t x[8];
        if (turned) {
          turn(i, w, normed, x);
        } else {
          widen8(raw[i][0], x);
          widen8(raw[i][1], x + 4);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 v = unpair2(x[e]);
          amax = fmaxf(amax, fmaxf(finite_abs(v.x), finite_abs(v.y)));
        }
      }
      amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
      const float scale = fmaxf(q8::scale_of(amax), old_scale);
      if (slot0 > 0 && scale > old_scale) rescale_block<D>(pool8, row_values, slot0, old_scale / scale);
      if (lane == 0 && scale != old_scale) *scale_at = scale;
      inv = 1.f / scale;
    }
#pragma unroll
    for (int i = 0; i < kLive; ++i) {
      const int r = i * kStep + sub;
      const bool live = r < run.n;
      uint64_t x[8];
      if (turned) {
        turn(i, w, normed, x);
      } else if (kQ8) {
        widen8(raw[i][0], x);
        widen8(raw[i][1], x + 4);
      } else if (live && page_ok) {   // a bf16 value goes through as it came, a NaN's payload too
        uint16_t* at = static_cast<uint16_t*>(p.v_pool) + block + (slot0 + r) * row_values + l * 8;
        *reinterpret_cast<uint4*>(at) = raw[i][0];
        *reinterpret_cast<uint4*>(at + half) = raw[i][1];
      }
      if (kQ8 && h + hop < heads) load_step(h + hop, i);   // in flight while the later rows are turned
      if (is_q) {
        if (live) {
          uint16_t* at = p.q_out + ((int64_t)(run.row0 + r) * p.Hq + h) * D + l * 8;
          *reinterpret_cast<uint4*>(at) = narrow8(x);
          *reinterpret_cast<uint4*>(at + half) = narrow8(x + 4);
        }
      } else if (!kQ8) {
        if (turned && live && page_ok) {
          uint16_t* at = static_cast<uint16_t*>(p.k_pool) + block + (slot0 + r) * row_values + l * 8;
          *reinterpret_cast<uint4*>(at) = narrow8(x);
          *reinterpret_cast<uint4*>(at + half) = narrow8(x + 4);
        }
      } else if (live && page_ok) {
        uint8_t* at = pool8 + (slot0 + r) * row_values + l * 8;
        *reinterpret_cast<uint2*>(at) = make_uint2(pairs_to_e4m3x4(x[0], x[1], inv), pairs_to_e4m3x4(x[2], x[3], inv));
        *reinterpret_cast<uint2*>(at + half) = make_uint2(pairs_to_e4m3x4(x[4], x[5], inv), pairs_to_e4m3x4(x[6], x[7], inv));
      }
    }
  };
  if (run.n <= kStep) {
    for (int h = first; h < heads; h += hop) do_head(h, std::integral_constant<int, 1>());
  } else {
    for (int h = first; h < heads; h += hop) do_head(h, std::integral_constant<int, kSteps>());
  }
}

struct PackParams {
  const uint16_t *k_src, *v_src;
  int64_t src_layer_stride, pool_layer_stride, scale_layer_stride;
  const int32_t *src_table, *block_table;
  uint8_t *k_pool, *v_pool;
  float *k_scale, *v_scale;
  uint32_t* status;
  int64_t blocks;         // 2 * layers * pages * heads
  int src_pages, num_pages, n_tokens, pages, heads, layers;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 4) pack_kernel(const __grid_constant__ PackParams p) {
  constexpr int kLanes = D / 8;           // lanes of a row, 8 features each
  constexpr int kStep = 32 / kLanes;
  constexpr int kSteps = kPage / kStep;
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, sub = lane / kLanes, l = lane % kLanes;
  const int64_t b = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (b >= p.blocks) return;
  // heads innermost: a CTA's warps read neighbouring pieces of the same rows
  const int h = (int)(b % p.heads);
  int64_t rest = b / p.heads;
  const int i = (int)(rest % p.pages);
  rest /= p.pages;
  const int layer = (int)(rest % p.layers);
  const bool is_v = rest >= p.layers;
  const int src = p.src_table ? p.src_table[i] : i, dst = p.block_table ? p.block_table[i] : i;
  if ((p.src_table && (src < 0 || src >= p.src_pages)) || dst < 0 || dst >= p.num_pages) {
    if (lane == 0) flag(p.status, KVRP_DEV_BAD_PAGE);
    return;
  }
  const int64_t row_values = (int64_t)p.heads * D;
  const uint16_t* from = (is_v ? p.v_src : p.k_src) + layer * p.src_layer_stride + src * kPage * row_values + h * D + l * 8;
  const int n = min(kPage, p.n_tokens - i * kPage);
  uint4 raw[kSteps];
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int r = s * kStep + sub;
    raw[s] = r < n ? *reinterpret_cast<const uint4*>(from + r * row_values) : make_uint4(0, 0, 0, 0);
  }
  // the largest magnitude, as bf16 bits: two values an instruction
  uint32_t most = 0;
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    most = __vmaxu2(__vmaxu2(most, raw[s].x & 0x7fff7fffu), raw[s].y & 0x7fff7fffu);
    most = __vmaxu2(__vmaxu2(most, raw[s].z & 0x7fff7fffu), raw[s].w & 0x7fff7fffu);
  }
  uint32_t top = max(most & 0xffffu, most >> 16);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  const bool finite = top < 0x7f80u;
  float amax = __uint_as_float(top << 16);
  if (!finite) {   // some value is inf or NaN: the largest of the others
    amax = 0.f;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      float x[8];
      unpack8(raw[s], x);
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = fmaxf(amax, finite_abs(x[e]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  }
  const float scale = q8::scale_of(amax), inv = 1.f / scale;
  uint8_t* to = (is_v ? p.v_pool : p.k_pool) + layer * p.pool_layer_stride + dst * kPage * row_values + h * D + l * 8;
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    float x[8];
    unpack8(raw[s], x);
    uint2 v;
    if (finite) v = make_uint2(q8::finite_to_e4m3x4(x[0], x[1], x[2], x[3], inv), q8::finite_to_e4m3x4(x[4], x[5], x[6], x[7], inv));
    else v = make_uint2(q8::to_e4m3x4(x[0], x[1], x[2], x[3], inv), q8::to_e4m3x4(x[4], x[5], x[6], x[7], inv));
    *reinterpret_cast<uint2*>(to + (s * kStep + sub) * row_values) = v;
  }
  if (lane == 0) (is_v ? p.v_scale : p.k_scale)[layer * p.scale_layer_stride + (int64_t)dst * p.heads + h] = scale;
}

// theta^(-2i/d) / (2 pi) in units of 2^-64 turns.  1 / (2 pi) is carried as a double and
// its remainder, so the product keeps the frequency's own 53 bits.
uint64_t turn_fraction(double theta, int i, int d) {
  const double hi = 0.15915494309189535, lo = -9.839338337591243e-18;
  const double inv = std::pow(theta, -2.0 * i / d);
  double t = inv * hi;
  const double rest = std::fma(inv, hi, -t) + inv * lo;
  t -= std::floor(t);   // theta < 1 turns more than once a position
  return (uint64_t)std::ldexp(t, 64) + (uint64_t)(int64_t)std::llrint(std::ldexp(rest, 64));
}

// The frequencies of a model, kept from call to call: 64 powers cost more than a launch.
const uint64_t* turn_fractions(double theta, int d) {
  thread_local double kept_theta = 0.0;
  thread_local int kept_d = 0;
  thread_local uint64_t kept[64];
  if (theta != kept_theta || d != kept_d) {
    for (int i = 0; i < d / 2; ++i) kept[i] = turn_fraction(theta, i, d);
    kept_theta = theta;
    kept_d = d;
  }
  return kept;
}

kvrp_status run(const char* fn, bool q8, const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                int64_t v_stride, const kvrp_seqs* seqs, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                const void* q_norm, const void* k_norm, float norm_eps, double rope_theta, const int32_t* positions,
                const int32_t* mrope_section, void* q_out, void* k_pool, void* v_pool, float* k_scale, float* v_scale,
                uint32_t* d_status, kvrp_stream_t stream) {
  g_last_launches = 0;
  kvrp_status st = check_seqs(fn, seqs);
  if (st != KVRP_OK) return st;
  st = check_heads(fn, n_q_heads, n_kv_heads, head_dim);
  if (st != KVRP_OK) return st;
  if (!k || !v || !k_pool || !v_pool || (q8 && (!k_scale || !v_scale)))
    return fail(KVRP_ERR_INVALID_ARG, "%s: NULL argument", fn);
  if (!q != !q_out) return fail(KVRP_ERR_INVALID_ARG, "%s: q and q_out go together", fn);
  if (!q_norm != !k_norm) return fail(KVRP_ERR_INVALID_ARG, "%s: q_norm and k_norm go together", fn);
  if (!(rope_theta > 0.0) || !std::isfinite(rope_theta)) return fail(KVRP_ERR_INVALID_ARG, "%s: rope_theta must be > 0", fn);
  if (q_norm && (!(norm_eps >= 0.f) || !std::isfinite(norm_eps)))
    return fail(KVRP_ERR_INVALID_ARG, "%s: norm_eps must be >= 0", fn);
  if (mrope_section && (mrope_section[0] < 0 || mrope_section[1] < 0 || mrope_section[2] < 0 ||
                        (int64_t)mrope_section[0] + mrope_section[1] + mrope_section[2] != head_dim / 2))
    return fail(KVRP_ERR_INVALID_ARG, "%s: mrope_section must sum to head_dim / 2", fn);
  const int64_t q_row = (int64_t)n_q_heads * head_dim, kv_row = (int64_t)n_kv_heads * head_dim;
  q_stride = q_stride ? q_stride : q_row;
  k_stride = k_stride ? k_stride : kv_row;
  v_stride = v_stride ? v_stride : kv_row;
  if ((q && q_stride < q_row) || k_stride < kv_row || v_stride < kv_row)
    return fail(KVRP_ERR_INVALID_ARG, "%s: a row stride is shorter than the row", fn);
  if (q && q == q_out && q_stride != q_row) return fail(KVRP_ERR_INVALID_ARG, "%s: q_out == q needs dense q rows", fn);
  if (q_stride % 8 || k_stride % 8 || v_stride % 8 || !aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) ||
      !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(q_norm) || !aligned16(k_norm))
    return fail(KVRP_ERR_ALIGNMENT, "%s: pointers must be 16-byte aligned, strides multiples of 8", fn);
  for (const void* x : {(const void*)positions, (const void*)k_scale, (const void*)v_scale, (const void*)d_status})
    if (reinterpret_cast<uintptr_t>(x) % 4) return fail(KVRP_ERR_ALIGNMENT, "%s: a 4-byte array is not aligned", fn);
  if (seqs->n_rows == 0) return KVRP_OK;
  int sms = 0, smem = 0;
  st = current_device_sms(&sms, &smem);
  if (st != KVRP_OK) return st;

  Params p;
  std::memset(&p, 0, sizeof(p));
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.q_norm = static_cast<const uint16_t*>(q_norm);
  p.k_norm = static_cast<const uint16_t*>(k_norm);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_out = static_cast<uint16_t*>(q_out);
  p.k_pool = k_pool;
  p.v_pool = v_pool;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.positions = positions;
  p.seqs = *seqs;
  p.status = d_status;
  p.Hq = n_q_heads;
  p.Hkv = n_kv_heads;
  p.h0 = q ? 0 : n_q_heads;
  p.eps = norm_eps;
  p.mrope = mrope_section != nullptr;
  p.sec1 = mrope_section ? mrope_section[0] : head_dim;
  p.sec2 = mrope_section ? mrope_section[0] + mrope_section[1] : head_dim;
  std::memcpy(p.turn, turn_fractions(rope_theta, head_dim), sizeof(uint64_t) * (head_dim / 2));
  // A sequence of n rows has at most (n - 1) / 16 + 2 runs, and at most n.
  const int64_t runs = !seqs->row_start ? seqs->n_seqs
                                        : std::min<int64_t>(seqs->n_rows, seqs->n_rows / kPage + 2 * (int64_t)seqs->n_seqs);
  // A run's heads are shared out among CTAs while the GPU has room for more (three CTAs an SM): a
  // decode step is a few runs, and its time is one warp's chain of loads.  Above one filling a run takes
  // two CTAs where the last filling would be at most half full, and so ends half a filling earlier, one
  // elsewhere: the second table of angles costs more than an evener end gives.  Measured with one / two a
  // run, us (28 + 2 x 4 heads with norms, 32 + 2 x 32 without; 456 places; * is the rule's):
  //   runs / places        1.1         1.3         1.6         1.9         2.2         2.7         3.3         3.8
  //   bf16, 28 + 8    36.5/31.9*  37.8/35.4*  40.9*/42.3  44.4*/47.4  56.7/54.5*  62.3*/65.3  77.2/77.9*  83.8*/88.5
  //   bf16, 32 + 64   76.3/66.7*  77.2/74.1*  93.5*/91.6  110*/103    125/120*    147*/146    180/176*    207*/202
  //   8 bits, 28 + 8  46.3/40.6*  48.6/43.5*  51.8*/53.5  55.0*/59.1  72.5/68.5*  79.0*/82.7  99.7/98.5*  106*/112
  //   8 bits, 32 + 64 88.1/74.2*  94.7/81.0*  100*/102    113*/116    141/134*    164*/162    197/194*    220*/222
  const int64_t places = 3 * (int64_t)sms;
  const int rounds = (n_q_heads - p.h0 + 2 * n_kv_heads + kWarps - 1) / kWarps;
  // of a ragged batch, whose sequences mostly begin and end inside a page
  const int64_t likely = !seqs->row_start ? runs : std::min<int64_t>(runs, seqs->n_rows / kPage + seqs->n_seqs);
  const bool half = (2 * likely + places - 1) / places < 2 * ((likely + places - 1) / places);
  const int64_t wanted = likely <= places ? places / likely : half ? 2 : 1;
  p.splits = (int)std::max<int64_t>(1, std::min<int64_t>(rounds, wanted));
  if (runs * p.splits > INT32_MAX) return fail(KVRP_ERR_UNSUPPORTED, "%s: too many rows", fn);

  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(runs * p.splits));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto kernel = head_dim == 64 ? (q8 ? append_kernel<64, true> : append_kernel<64, false>)
                               : (q8 ? append_kernel<128, true> : append_kernel<128, false>);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  if (e != cudaSuccess) return fail(KVRP_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
  g_last_launches = 1;
  return KVRP_OK;
}

}  // namespace append

kvrp_status check_heads(const char* fn, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim) {
  if (head_dim != 64 && head_dim != 128) return fail(KVRP_ERR_UNSUPPORTED, "%s: head_dim must be 64 or 128", fn);
  if (n_kv_heads <= 0 || n_q_heads <= 0 || n_q_heads % n_kv_heads || n_q_heads / n_kv_heads > 16 || n_kv_heads > 4096)
    return fail(KVRP_ERR_UNSUPPORTED, "%s: n_q_heads must be a multiple of n_kv_heads (<= 4096), at most 16 x", fn);
  return KVRP_OK;
}

kvrp_status check_seqs(const char* fn, const kvrp_seqs* s) {
  if (!s || !s->seq_lens || !s->block_tables) return fail(KVRP_ERR_INVALID_ARG, "%s: NULL seqs, seq_lens or block_tables", fn);
  if (s->n_seqs <= 0 || s->n_seqs > 65535) return fail(KVRP_ERR_INVALID_ARG, "%s: 1 <= n_seqs <= 65535", fn);
  if (s->n_rows < 0 || s->max_rows < 0 || s->max_rows > s->n_rows)
    return fail(KVRP_ERR_INVALID_ARG, "%s: 0 <= max_rows <= n_rows", fn);
  if (!s->row_start && s->n_rows != s->n_seqs)
    return fail(KVRP_ERR_INVALID_ARG, "%s: without row_start there is one row per sequence", fn);
  if (s->table_stride <= 0 || s->num_pages <= 0 || s->num_pages > INT32_MAX / q8::kPage)
    return fail(KVRP_ERR_INVALID_ARG, "%s: table_stride and num_pages out of range", fn);
  for (const void* x : {(const void*)s->row_start, (const void*)s->seq_lens, (const void*)s->block_tables})
    if (reinterpret_cast<uintptr_t>(x) % 4) return fail(KVRP_ERR_ALIGNMENT, "%s: a 4-byte array of seqs is not aligned", fn);
  return KVRP_OK;
}

}  // namespace kvrp

using namespace kvrp;

extern "C" {

kvrp_status kv_append(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                      const kvrp_seqs* seqs, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim, const void* q_norm,
                      const void* k_norm, float norm_eps, double rope_theta, const int32_t* positions,
                      const int32_t* mrope_section, void* q_out, void* k_pool, void* v_pool, uint32_t* d_status,
                      kvrp_stream_t stream) {
  return append::run("kv_append", false, q, k, v, q_stride, k_stride, v_stride, seqs, n_q_heads, n_kv_heads, head_dim, q_norm,
                     k_norm, norm_eps, rope_theta, positions, mrope_section, q_out, k_pool, v_pool, nullptr, nullptr, d_status,
                     stream);
}

kvrp_status kv_append_q8(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                         const kvrp_seqs* seqs, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim, const void* q_norm,
                         const void* k_norm, float norm_eps, double rope_theta, const int32_t* positions,
                         const int32_t* mrope_section, void* q_out, void* k_pool, void* v_pool, float* k_scale,
                         float* v_scale, uint32_t* d_status, kvrp_stream_t stream) {
  return append::run("kv_append_q8", true, q, k, v, q_stride, k_stride, v_stride, seqs, n_q_heads, n_kv_heads, head_dim, q_norm,
                     k_norm, norm_eps, rope_theta, positions, mrope_section, q_out, k_pool, v_pool, k_scale, v_scale, d_status,
                     stream);
}

kvrp_status kv_pack_q8(const void* k_src, const void* v_src, int64_t src_layer_stride, const int32_t* src_table,
                       int32_t src_pages, int32_t n_layers, int32_t n_tokens, int32_t n_kv_heads, int32_t head_dim,
                       void* k_pool, void* v_pool, int64_t pool_layer_stride, float* k_scale, float* v_scale,
                       int64_t scale_layer_stride, const int32_t* block_table, int32_t num_pages, uint32_t* d_status,
                       kvrp_stream_t stream) {
  const char* fn = "kv_pack_q8";
  g_last_launches = 0;
  kvrp_status st = check_heads(fn, n_kv_heads, n_kv_heads, head_dim);
  if (st != KVRP_OK) return st;
  if (n_layers <= 0 || n_tokens < 0) return fail(KVRP_ERR_INVALID_ARG, "%s: n_layers > 0, n_tokens >= 0", fn);
  if (!k_src || !v_src || !k_pool || !v_pool || !k_scale || !v_scale) return fail(KVRP_ERR_INVALID_ARG, "%s: NULL argument", fn);
  const int pages = (int)(((int64_t)n_tokens + append::kPage - 1) / append::kPage);
  const int64_t D = (int64_t)n_kv_heads * head_dim;
  constexpr int kMostPages = INT32_MAX / append::kPage;
  if (num_pages <= 0 || num_pages > kMostPages || (src_table && (src_pages <= 0 || src_pages > kMostPages)) ||
      (!block_table && pages > num_pages))
    return fail(KVRP_ERR_INVALID_ARG, "%s: num_pages or src_pages out of range", fn);
  const int64_t src_need = src_table ? (int64_t)src_pages * append::kPage * D : (int64_t)n_tokens * D;
  src_layer_stride = src_layer_stride ? src_layer_stride : src_need;
  pool_layer_stride = pool_layer_stride ? pool_layer_stride : (int64_t)num_pages * append::kPage * D;
  scale_layer_stride = scale_layer_stride ? scale_layer_stride : (int64_t)num_pages * n_kv_heads;
  if (n_layers > 1 && (src_layer_stride < src_need || pool_layer_stride < (int64_t)num_pages * append::kPage * D ||
                       scale_layer_stride < (int64_t)num_pages * n_kv_heads))
    return fail(KVRP_ERR_INVALID_ARG, "%s: a layer stride is shorter than the layer", fn);
  if (src_layer_stride % 8 || pool_layer_stride % 16 || !aligned16(k_src) || !aligned16(v_src) || !aligned16(k_pool) ||
      !aligned16(v_pool))
    return fail(KVRP_ERR_ALIGNMENT, "%s: pointers and layer strides must be 16-byte aligned", fn);
  for (const void* x : {(const void*)src_table, (const void*)block_table, (const void*)k_scale, (const void*)v_scale,
                        (const void*)d_status})
    if (reinterpret_cast<uintptr_t>(x) % 4) return fail(KVRP_ERR_ALIGNMENT, "%s: a 4-byte array is not aligned", fn);
  if (n_tokens == 0) return KVRP_OK;
  int sms = 0, smem = 0;
  st = current_device_sms(&sms, &smem);
  if (st != KVRP_OK) return st;
  append::PackParams p;
  std::memset(&p, 0, sizeof(p));
  p.k_src = static_cast<const uint16_t*>(k_src);
  p.v_src = static_cast<const uint16_t*>(v_src);
  p.src_layer_stride = src_layer_stride;
  p.pool_layer_stride = pool_layer_stride;
  p.scale_layer_stride = scale_layer_stride;
  p.src_table = src_table;
  p.block_table = block_table;
  p.k_pool = static_cast<uint8_t*>(k_pool);
  p.v_pool = static_cast<uint8_t*>(v_pool);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.status = d_status;
  p.blocks = 2 * (int64_t)n_layers * pages * n_kv_heads;
  p.src_pages = src_pages;
  p.num_pages = num_pages;
  p.n_tokens = n_tokens;
  p.pages = pages;
  p.heads = n_kv_heads;
  p.layers = n_layers;
  const int64_t grid = (p.blocks + append::kWarps - 1) / append::kWarps;
  if (grid > INT32_MAX) return fail(KVRP_ERR_UNSUPPORTED, "%s: too many blocks", fn);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(append::kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, head_dim == 64 ? append::pack_kernel<64> : append::pack_kernel<128>, p);
  if (e != cudaSuccess) return fail(KVRP_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
  g_last_launches = 1;
  return KVRP_OK;
}

}  // extern "C"
