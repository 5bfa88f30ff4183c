// Attention over the 8-bit paged cache (kv_attend_q8).
//
//   out[r][j] = sum_t p_t v_t,   p = softmax_t(softmax_scale q[r][j] . k_t),   t up to r's own position,
//   k_t = ks[page(t)] K_t,  v_t = vs[page(t)] V_t  (K_t, V_t the stored e4m3 values, one scale
//   for each page of 16 tokens and KV head).
//
// The scales stay out of the inner products: ks multiplies the finished scores, and vs
// enters the softmax weights' exponent, so that K and V go to the tensor cores as stored
// (e4m3 values are f16 values exactly).
//
// decode_kernel: few rows a sequence (rows x group <= 16).  Bound by the bytes of K and V.
//   - Work is the list of (sequence, KV head, page); each CTA takes an equal contiguous
//     share, so every SM streams the same bytes whatever the lengths; a share's part of one
//     (sequence, head) is a segment.  The shares are computed on the device from the
//     lengths there: a captured graph keeps its balance as sequences grow.
//   - A warp is a pipeline of its own: it takes every 8th page of the segment through a
//     private ring of TMA boxes (16 x head_dim bytes of K and of V) on its own mbarriers,
//     which runs on across segments.  No warp waits for another inside a segment.
//   - mma.sync m16n8k16 with f16 operands and tokens as the product's rows: S = K Q^T, 16
//     tokens x 8 heads a tile, then O^T += V^T P^T with P^T transposed in registers.  A page
//     is exactly the 16 rows (and the 16-deep contraction of the second product), so its
//     two scales are uniform in a tile.  The contraction index may be permuted freely, so a
//     lane's K fragment is 32 consecutive bytes of a row and its V fragment 16 consecutive
//     bytes of four rows: wide, conflict-free shared loads, and no transposing load.
//   - q enters as one f16 number: a row is divided by the power of two of its largest
//     element, after which bf16's 8 significant bits are exact down to 2^-16 of the largest
//     and no element is off by more than 2^-25 of it.
//   - Two running maxima a row: of the scores x (for the sum of weights), and of x + log2 vs
//     (for the accumulator, whose weights are exp2(x + log2 vs - max)).  The second keeps
//     the f16 weights in range however far the pages' value scales lie apart.
//   - Maxima move only when a score passes them by 2^8 (one vote a page instead of six
//     shuffles); weights then stay below 2^15, inside f16.
// combine_kernel: merges the partial results of (sequence, head)s that more than one CTA shared.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "kvrp.h"
#include "kvrp_plan.h"
#include "kvrp_ptx.h"
#include "kvrp_q8.h"
#include "kvrp_attend_q8.h"

namespace kvrp {
namespace attend_q8 {


// ---- shares ---------------------------------------------------------------------------
struct Seq {
  int row0, rows, len, pages;
};
// Sequence s as the decode kernel sees it; pages 0 where it has no work.
__device__ __forceinline__ Seq seq_at(const Params& p, int s, int max_rows, bool tell = false) {
  Seq r;
  const bool ok = sequence(p.seqs, s, r.row0, r.rows, r.len) && r.rows <= max_rows;
  r.pages = ok && r.rows > 0 ? (r.len + kPage - 1) / kPage : 0;
  if (tell && !ok) flag(p.status, KVRP_DEV_BAD_LENGTH);
  return r;
}

// A position in the list of (sequence, head, page), and the pages left of the share.
struct Cursor {
  int s, h, page, end;    // the segment's next page and its end
  int64_t left;           // pages of the share from `page` on
};

__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t* sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  int64_t all = 0;
  for (int w = 0; w < (int)blockDim.x / 32; ++w) all += sh[w];
  return all;
}

// This CTA's share of the pages.  A share is at least one page a warp, so that a small
// batch is not cut into parts that cost more to merge than to read.
template <int kWarps>
__device__ __forceinline__ bool find_share(const Params& p, int max_rows, Cursor* out, int64_t* sh, int* found) {
  const int n = p.seqs.n_seqs, threads = 32 * kWarps;
  const int tid = threadIdx.x;
  int64_t mine = 0;
  for (int s = tid; s < n; s += threads) mine += (int64_t)seq_at(p, s, max_rows, blockIdx.x == 0).pages * p.Hkv;
  const int64_t total = block_sum(mine, sh);
  const int n_cta = (int)min((int64_t)p.n_cta, (total + kWarps - 1) / kWarps);
  if ((int)blockIdx.x >= n_cta) return false;
  const int64_t a = total * blockIdx.x / n_cta, b = total * (blockIdx.x + 1) / n_cta;
  // the sequence that holds page a: prefix sums, `threads` sequences at a time
  int64_t before = 0;
  for (int s0 = 0; s0 < n; s0 += threads) {
    const int s = s0 + tid;
    const int64_t c = s < n ? (int64_t)seq_at(p, s, max_rows).pages * p.Hkv : 0;
    int64_t sum = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t t = __shfl_up_sync(0xffffffffu, sum, o);
      if ((tid & 31) >= o) sum += t;
    }
    __syncthreads();
    if ((tid & 31) == 31) sh[tid >> 5] = sum;
    if (tid == 0) *found = -1;
    __syncthreads();
    int64_t at = before + sum - c;
    for (int w = 0; w < kWarps; ++w) {
      if (w < (tid >> 5)) at += sh[w];
      before += sh[w];
    }
    if (a >= at && a < at + c) {
      *found = s;
      sh[kWarps] = a - at;
    }
    __syncthreads();
    if (*found >= 0) break;
  }
  const Seq q = seq_at(p, *found, max_rows);
  out->s = *found;
  out->h = (int)(sh[kWarps] / q.pages);
  out->page = (int)(sh[kWarps] % q.pages);
  out->left = b - a;
  out->end = (int)min((int64_t)q.pages, out->page + out->left);
  return true;
}
// The next segment of the share; false at its end.
__device__ __forceinline__ bool next_segment(const Params& p, int max_rows, Cursor& c, int first, Seq& q) {
  c.left -= c.end - first;
  if (c.left <= 0) return false;
  if (++c.h == p.Hkv) {
    c.h = 0;
    do q = seq_at(p, ++c.s, max_rows);
    while (q.pages == 0);
  }
  c.page = 0;
  c.end = (int)min((int64_t)q.pages, c.left);
  return true;
}

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// ---- decode ----------------------------------------------------------------------------
constexpr int kWarps = 8;
template <int D, int NT>
struct Decode {
  static constexpr int kBox = kPage * D;                      // bytes of one head's K (or V) of a page
  // 8 to 12 KB a warp, 128 to 192 KB in flight on an SM; two CTAs fit beside their merge buffers
  static constexpr int kStages = D == 128 ? (NT == 1 ? 3 : 2) : (NT == 1 ? 6 : 5);
  static constexpr int kRing = kWarps * kStages * 2 * kBox;
  static constexpr int kMerge = 32 * (D / 16 * NT * 4 + NT * 6);   // words of one warp's accumulator and statistics
  static constexpr int kSmem = 1024 + kRing + kWarps / 2 * kMerge * 4;
};

template <int D, int NT>   // head_dim; tiles of 8 (row, head) columns
__global__ void __launch_bounds__(32 * kWarps, 2)
    decode_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                  const __grid_constant__ Params p) {
  constexpr int KT = D / 16;                 // 16-deep steps over the features; 16-feature tiles of O^T
  constexpr int kBox = Decode<D, NT>::kBox, kStages = Decode<D, NT>::kStages, kMerge = Decode<D, NT>::kMerge;
  constexpr int FPL = D / 8;                 // features of O a lane holds for a column
  extern __shared__ uint8_t raw_smem[];
  __shared__ __align__(8) uint64_t bars[kWarps * kStages];
  __shared__ float2 scales[kWarps * kStages];
  __shared__ int64_t sh[kWarps + 1];
  __shared__ int found, abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, tig = lane & 3;
  const uint32_t smem = (smem_u32(raw_smem) + 1023u) & ~1023u;
  const uint32_t ring = smem + (uint32_t)warp * kStages * 2 * kBox;
  float* merge = reinterpret_cast<float*>(raw_smem + (smem - smem_u32(raw_smem)) + Decode<D, NT>::kRing);
  const uint32_t bar0 = smem_u32(bars) + 8u * warp * kStages;
  float2* my_scales = scales + warp * kStages;
  if (tid == 0) {
    for (int i = 0; i < kWarps * kStages; ++i) mbar_init(smem_u32(bars) + 8u * i, 1);
    abort_flag = 0;
    mbar_init_fence();
  }
  volatile int* abort_p = &abort_flag;
  if (tid == 32) {
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
  }
  pdl_wait();
  pdl_launch_dependents();
  const int max_rows = p.max_rows;
  Cursor ic;
  if (!find_share<kWarps>(p, max_rows, &ic, sh, &found)) {
    if (tid == 0) p.meta[blockIdx.x] = make_int4(-1, 0, 0, 0);
    write_idle(p, D);
    return;
  }
  __syncthreads();   // the barriers are initialised
  Cursor cc = ic;    // the segment being computed
  Seq cq = seq_at(p, cc.s, max_rows), iq = cq;

  // ---- the issuing side: which page goes into the ring next --------------------------
  int issue_first = ic.page;   // the segment's first page
  int b_page = 0, b_at = 32;   // a batch of table entries and scales, one a lane
  float b_ks = 0.f, b_vs = 0.f;
  int n_issued = 0;
  bool more = true;
  auto refill = [&]() {
    const int pg = ic.page + lane * kWarps;
    b_page = p.seqs.num_pages;   // past the pool: the box reads zeros
    b_ks = b_vs = 0.f;
    if (pg < ic.end) {
      const int e = p.seqs.block_tables[(int64_t)ic.s * p.seqs.table_stride + pg];
      if (e >= 0 && e < p.seqs.num_pages) {
        b_page = e;
        b_ks = p.k_scale[(int64_t)e * p.Hkv + ic.h];
        b_vs = p.v_scale[(int64_t)e * p.Hkv + ic.h];
      } else {
        flag(p.status, KVRP_DEV_BAD_PAGE);
      }
    }
    b_at = 0;
  };
  auto settle = [&]() {   // move to the first segment that has a page for this warp
    while (more && ic.page >= ic.end) {
      more = next_segment(p, max_rows, ic, issue_first, iq);
      issue_first = 0;
      ic.page = warp;
      b_at = 32;
    }
  };
  ic.page += warp;
  settle();
  auto issue = [&]() {
    if (!more || __shfl_sync(0xffffffffu, *abort_p, 0)) return;
    if (b_at == 32) refill();
    const int st = n_issued % kStages;
    const int pg = __shfl_sync(0xffffffffu, b_page, b_at);
    const float ks = __shfl_sync(0xffffffffu, b_ks, b_at), vs = __shfl_sync(0xffffffffu, b_vs, b_at);
    if (lane == 0) {
      const uint32_t bar = bar0 + 8u * st, at = ring + (uint32_t)st * 2 * kBox;
      my_scales[st] = make_float2(ks, vs);
      mbar_expect_tx(bar, 2 * kBox);
      tma_load_3d(at, &kmap, bar, ic.h * D, 0, pg);
      tma_load_3d(at + kBox, &vmap, bar, ic.h * D, 0, pg);
    }
    ++b_at;
    ++n_issued;
    ic.page += kWarps;
    settle();
  };
  for (int i = 0; i < kStages; ++i) issue();

  int n_used = 0;
  int4 meta = make_int4(-1, 0, 0, 0);
  while (true) {
    // ---- a segment: the queries of its KV head ------------------------------------------
    const int first = cc.page, cols = cq.rows * p.g, ctx = cq.len - cq.rows;
    uint32_t qb[KT][NT][2];
    float fac[NT][2];
    int limit[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int c = nt * 8 + gid;
      uint32_t w[KT][2];
#pragma unroll
      for (int kk = 0; kk < KT; ++kk) w[kk][0] = w[kk][1] = 0u;
      if (c < cols) {
        const uint16_t* at = p.q + (cq.row0 + c / p.g) * p.q_stride + (int64_t)(cc.h * p.g + c % p.g) * D + tig * (D / 4);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const uint4 u = reinterpret_cast<const uint4*>(at)[i];
          w[2 * i][0] = u.x;
          w[2 * i][1] = u.y;
          w[2 * i + 1][0] = u.z;
          w[2 * i + 1][1] = u.w;
        }
      }
      uint32_t top = 0;   // the row's largest magnitude, as bf16 bits
#pragma unroll
      for (int kk = 0; kk < KT; ++kk)
#pragma unroll
        for (int e = 0; e < 2; ++e) top = max(top, max(w[kk][e] & 0x7fffu, (w[kk][e] >> 16) & 0x7fffu));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^e, e the largest element's exponent; an all-zero row, and one with inf or NaN, keeps 1
      int e = (int)(top >> 7) - 127;
      if (e == 128 || top == 0) e = 0;
      e = min(max(e, -125), 126);
      const float down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
      for (int kk = 0; kk < KT; ++kk)
#pragma unroll
        for (int b = 0; b < 2; ++b) qb[kk][nt][b] = pack_f16(bf_lo(w[kk][b]) * down, bf_hi(w[kk][b]) * down);
      const float up = p.scale * __uint_as_float((uint32_t)(e + 127) << 23);
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int cb = nt * 8 + 2 * tig + b;
        fac[nt][b] = __shfl_sync(0xffffffffu, up, (2 * tig + b) * 4);
        limit[nt][b] = cb < cols ? ctx + cb / p.g + 1 : 0;
      }
    }
    float o[KT][NT][4];
    float m[NT][2], om[NT][2], l[NT][2];   // running maxima of x and of x + log2 vs; sum of weights (this lane's tokens)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        m[nt][b] = om[nt][b] = -INFINITY;
        l[nt][b] = 0.f;
      }
#pragma unroll
      for (int mt = 0; mt < KT; ++mt) o[mt][nt][0] = o[mt][nt][1] = o[mt][nt][2] = o[mt][nt][3] = 0.f;
    }

    for (int pg = first + warp; pg < cc.end; pg += kWarps) {
      const int st = n_used % kStages;
      wait_phase(bar0 + 8u * st, (n_used / kStages) & 1, abort_p, p.status);
      __syncwarp();
      ++n_used;
      const uint32_t kat = ring + (uint32_t)st * 2 * kBox, vat = kat + kBox;
      const float2 sc = my_scales[st];
      // ---- S = K Q^T -----------------------------------------------------------------
      float c[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) c[nt][0] = c[nt][1] = c[nt][2] = c[nt][3] = 0.f;
      {
        uint32_t k0[KT], k1[KT];   // rows gid and gid + 8: features tig D/4 + 4 kk + {0..3}
#pragma unroll
        for (int i = 0; i < KT / 4; ++i) {
          const int chunk = tig * (KT / 4) + i;
          const uint32_t off = D == 128 ? (uint32_t)(gid * 128 + ((chunk ^ gid) << 4))
                                        : (uint32_t)(gid * 64 + ((chunk ^ (gid >> 1)) << 4));
          asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(k0[4 * i]), "=r"(k0[4 * i + 1]), "=r"(k0[4 * i + 2]), "=r"(k0[4 * i + 3]) : "r"(kat + off));
          asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(k1[4 * i]), "=r"(k1[4 * i + 1]), "=r"(k1[4 * i + 2]), "=r"(k1[4 * i + 3]) : "r"(kat + off + 8 * D));
        }
#pragma unroll
        for (int kk = 0; kk < KT; ++kk) {
          const uint32_t a[4] = {q8::e4m3x2_to_f16x2((uint16_t)k0[kk]), q8::e4m3x2_to_f16x2((uint16_t)k1[kk]),
                                 q8::e4m3x2_to_f16x2((uint16_t)(k0[kk] >> 16)), q8::e4m3x2_to_f16x2((uint16_t)(k1[kk] >> 16))};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816_f16(c[nt], a, qb[kk][nt][0], qb[kk][nt][1]);
        }
      }
      const float lvs = lg2(sc.y);   // exact for a power of two; -inf for a zero scale
      const bool tail = (pg + 1) * kPage > ctx + 1;
      bool grow = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = c[nt][e] * (sc.x * fac[nt][e & 1]);
          if (tail && pg * kPage + gid + (e >> 1) * 8 >= limit[nt][e & 1]) x = -INFINITY;
          c[nt][e] = x;
          grow |= x > m[nt][e & 1] + kLazy || x + lvs > om[nt][e & 1] + kLazy;
        }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            float t = fmaxf(c[nt][b], c[nt][2 + b]);
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
            const float nm = fmaxf(m[nt][b], t), no = fmaxf(om[nt][b], t + lvs);
            if (nm > m[nt][b]) l[nt][b] *= ex2(m[nt][b] - nm);     // a first maximum: 2^-inf = 0
            m[nt][b] = nm;
            const float r = no > om[nt][b] ? ex2(om[nt][b] - no) : 1.f;
            om[nt][b] = no;
#pragma unroll
            for (int mt = 0; mt < KT; ++mt) {
              o[mt][nt][b] *= r;
              o[mt][nt][2 + b] *= r;
            }
          }
      }
      uint32_t pb[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = c[nt][e], mm = m[nt][e & 1], oo = om[nt][e & 1];
          l[nt][e & 1] += ex2(x - (mm == -INFINITY ? 0.f : mm));
          w[e] = ex2(x + lvs - (oo == -INFINITY ? 0.f : oo) + kShift);
        }
        pb[nt][0] = movmatrix_trans(pack_f16(w[0], w[1]));
        pb[nt][1] = movmatrix_trans(pack_f16(w[2], w[3]));
      }
      // ---- O^T += V^T P^T --------------------------------------------------------------
      {
        uint32_t v[4][FPL / 4];   // tokens 2 tig, 2 tig + 1, 2 tig + 8, 2 tig + 9: features gid FPL ..
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = 2 * tig + (i & 1) + (i >> 1) * 8;
          if constexpr (D == 128) {
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(v[i][0]), "=r"(v[i][1]), "=r"(v[i][2]), "=r"(v[i][3])
                         : "r"(vat + (uint32_t)(t * 128 + ((gid ^ (t & 7)) << 4))));
          } else {
            asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];"
                         : "=r"(v[i][0]), "=r"(v[i][1])
                         : "r"(vat + (uint32_t)(t * 64 + (((gid >> 1) ^ ((t >> 1) & 3)) << 4) + (gid & 1) * 8)));
          }
          if (tail && pg * kPage + t >= cq.len) {   // a slot past the sequence may hold anything, NaN included
#pragma unroll
            for (int j = 0; j < FPL / 4; ++j) v[i][j] = 0u;
          }
        }
        __syncwarp();   // every lane has read the stage
#pragma unroll
        for (int j = 0; j < FPL / 4; ++j)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t sel = half ? 0x7362u : 0x5140u;
            const uint32_t x = __byte_perm(v[0][j], v[1][j], sel), y = __byte_perm(v[2][j], v[3][j], sel);
            const uint32_t a[4] = {q8::e4m3x2_to_f16x2((uint16_t)x), q8::e4m3x2_to_f16x2((uint16_t)(x >> 16)),
                                   q8::e4m3x2_to_f16x2((uint16_t)y), q8::e4m3x2_to_f16x2((uint16_t)(y >> 16))};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816_f16(o[2 * j + half][nt], a, pb[nt][0], pb[nt][1]);
          }
      }
      issue();
    }
    // ---- merge the warps: halves of the CTA into the other half, then quarters ------------
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        float t = l[nt][b];
        t += __shfl_xor_sync(0xffffffffu, t, 4);
        t += __shfl_xor_sync(0xffffffffu, t, 8);
        t += __shfl_xor_sync(0xffffffffu, t, 16);
        l[nt][b] = t;
      }
    const int live = min(kWarps, cc.end - first);   // warps that had a page
    for (int step = kWarps / 2; step > 0; step /= 2) {
      if (step >= live) continue;
      float* at = merge + (warp & (step - 1)) * kMerge + lane;
      if (warp >= step && warp < 2 * step && warp < live) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int mt = 0; mt < KT; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) at[32 * ((mt * NT + nt) * 4 + e)] = o[mt][nt][e];
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            at[32 * (KT * NT * 4 + nt * 6 + b)] = m[nt][b];
            at[32 * (KT * NT * 4 + nt * 6 + 2 + b)] = om[nt][b];
            at[32 * (KT * NT * 4 + nt * 6 + 4 + b)] = l[nt][b];
          }
        }
      }
      __syncthreads();
      if (warp < step && warp + step < live) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const float m2 = at[32 * (KT * NT * 4 + nt * 6 + b)], o2 = at[32 * (KT * NT * 4 + nt * 6 + 2 + b)];
            const float nm = fmaxf(m[nt][b], m2), no = fmaxf(om[nt][b], o2);
            const float ra = nm == -INFINITY ? 0.f : ex2(m[nt][b] - nm), rb = nm == -INFINITY ? 0.f : ex2(m2 - nm);
            l[nt][b] = l[nt][b] * ra + at[32 * (KT * NT * 4 + nt * 6 + 4 + b)] * rb;
            m[nt][b] = nm;
            const float sa = no == -INFINITY ? 0.f : ex2(om[nt][b] - no), sb = no == -INFINITY ? 0.f : ex2(o2 - no);
            om[nt][b] = no;
#pragma unroll
            for (int mt = 0; mt < KT; ++mt)
#pragma unroll
              for (int e = b; e < 4; e += 2) o[mt][nt][e] = o[mt][nt][e] * sa + at[32 * ((mt * NT + nt) * 4 + e)] * sb;
          }
      }
      __syncthreads();
    }
    // ---- the segment's result: a whole unit goes out, a part goes to the combine -----------
    const bool begins = first == 0, ends = cc.end == cq.pages;
    if (begins && !ends) meta.x = cc.s, meta.y = cc.h;
    if (!begins) meta.z = ends ? 2 : 1;
    if (warp == 0) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int c = nt * 8 + 2 * tig + b;
          if (c >= cols) continue;
          if (begins && ends) {
            const float r = l[nt][b] == 0.f ? 0.f : ex2(om[nt][b] - m[nt][b] - kShift) / l[nt][b];
            const int64_t row = (int64_t)(cq.row0 + c / p.g) * p.Hq + cc.h * p.g + c % p.g;
            uint32_t w[FPL / 2];
#pragma unroll
            for (int mt = 0; mt < KT; ++mt) {
              const __nv_bfloat162 v = __floats2bfloat162_rn(o[mt][nt][b] * r, o[mt][nt][2 + b] * r);
              w[mt] = *reinterpret_cast<const uint32_t*>(&v);
            }
            uint4* to = reinterpret_cast<uint4*>(p.out + row * D + gid * FPL);
#pragma unroll
            for (int i = 0; i < FPL / 8; ++i) to[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
            if (p.lse && gid == 0) p.lse[row] = (m[nt][b] + lg2(l[nt][b])) * kLn2;
          } else {
            float* to = p.partial + ((int64_t)(blockIdx.x * 2 + (begins ? 1 : 0)) * p.cols + c) * (D + 4);
            float4* of = reinterpret_cast<float4*>(to + gid * FPL);
#pragma unroll
            for (int i = 0; i < FPL / 4; ++i)
              of[i] = make_float4(o[2 * i][nt][b], o[2 * i][nt][2 + b], o[2 * i + 1][nt][b], o[2 * i + 1][nt][2 + b]);
            if (gid == 0) *reinterpret_cast<float4*>(to + D) = make_float4(m[nt][b], om[nt][b], l[nt][b], 0.f);
          }
        }
    }
    if (!next_segment(p, max_rows, cc, first, cq)) break;
  }
  if (tid == 0) p.meta[blockIdx.x] = meta;
  write_idle(p, D);
  if (*abort_p)   // let every copy land before the CTA exits
    for (int i = max(0, n_issued - kStages); i < n_issued; ++i) drain_wait(bar0 + 8u * (i % kStages), (i / kStages) & 1, p.status);
}

// ---- combine ---------------------------------------------------------------------------
// Block (i, c): column c of the unit that begins in CTA i and goes on in CTAs i + 1, ...
constexpr int kCombineThreads = 128;
template <int D>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const __grid_constant__ Params p) {
  constexpr int kLanes = D / 4, kGroups = kCombineThreads / kLanes;
  __shared__ int last;
  __shared__ float red[kCombineThreads / 32][3];
  __shared__ float4 part[kGroups][kLanes];
  pdl_wait();
  pdl_launch_dependents();
  const int i = blockIdx.x, c = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
  const int4 mt = p.meta[i];
  if (mt.x < 0) return;
  int row0, rows, len;
  sequence(p.seqs, mt.x, row0, rows, len);
  if (c >= rows * p.g) return;
  // the CTA that ends the unit
  if (tid == 0) last = 0x7fffffff;
  __syncthreads();
  for (int j0 = i + 1; j0 < p.n_cta; j0 += kCombineThreads) {
    const int j = j0 + tid;
    if (j < p.n_cta && p.meta[j].z == 2) atomicMin(&last, j);
    __syncthreads();
    if (last != 0x7fffffff) break;
    __syncthreads();
  }
  const int n = min(last, p.n_cta - 1) - i + 1;
  auto entry = [&](int k) { return p.partial + ((int64_t)((i + k) * 2 + (k == 0 ? 1 : 0)) * p.cols + c) * (D + 4); };
  float m = -INFINITY, om = -INFINITY;
  for (int k = tid; k < n; k += kCombineThreads) {
    const float4 s = *reinterpret_cast<const float4*>(entry(k) + D);
    m = fmaxf(m, s.x);
    om = fmaxf(om, s.y);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    om = fmaxf(om, __shfl_xor_sync(0xffffffffu, om, o));
  }
  if (lane == 0) red[tid >> 5][0] = m, red[tid >> 5][1] = om;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kCombineThreads / 32; ++w) {
    m = fmaxf(m, red[w][0]);
    om = fmaxf(om, red[w][1]);
  }
  const int f = tid % kLanes, grp = tid / kLanes;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
#pragma unroll 8
  for (int k = grp; k < n; k += kGroups) {
    const float* e = entry(k);
    const float4 s = *reinterpret_cast<const float4*>(e + D), v = reinterpret_cast<const float4*>(e)[f];
    const float w = om == -INFINITY ? 0.f : ex2(s.y - om);
    l += m == -INFINITY ? 0.f : s.z * ex2(s.x - m);
    acc.x = fmaf(v.x, w, acc.x);
    acc.y = fmaf(v.y, w, acc.y);
    acc.z = fmaf(v.z, w, acc.z);
    acc.w = fmaf(v.w, w, acc.w);
  }
  part[grp][f] = acc;
  __shared__ float lsum[kGroups];
  if (f == 0) lsum[grp] = l;
  __syncthreads();
  if (grp != 0) return;
  l = 0.f;
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int k = 0; k < kGroups; ++k) {
    l += lsum[k];
    acc.x += part[k][f].x;
    acc.y += part[k][f].y;
    acc.z += part[k][f].z;
    acc.w += part[k][f].w;
  }
  const float r = l == 0.f ? 0.f : ex2(om - m - kShift) / l;
  const int64_t row = (int64_t)(row0 + c / p.g) * p.Hq + mt.y * p.g + c % p.g;
  const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * r, acc.y * r), hi = __floats2bfloat162_rn(acc.z * r, acc.w * r);
  *reinterpret_cast<uint2*>(p.out + row * D + 4 * f) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  if (p.lse && f == 0) p.lse[row] = (m + lg2(l)) * kLn2;
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      n <= 0) {
    cudaGetLastError();
    n = 160;   // no device: a size for the checks of a host without one
  }
  return n;
}

size_t meta_bytes(int n_cta) { return ((size_t)n_cta * sizeof(int4) + 255) / 256 * 256; }
size_t workspace_bytes(int n_cta, int cols, int head_dim) {
  return 256 + meta_bytes(n_cta) + (size_t)n_cta * 2 * cols * (head_dim + 4) * sizeof(float);
}

}  // namespace attend_q8
}  // namespace kvrp

using namespace kvrp;

extern "C" {

size_t kv_attend_q8_workspace_size(int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim, int32_t max_rows) {
  if (check_heads("kv_attend_q8_workspace_size", n_q_heads, n_kv_heads, head_dim) != KVRP_OK || max_rows <= 0) return 0;
  const bool few = (int64_t)max_rows * (n_q_heads / n_kv_heads) <= attend_q8::kMaxCols;
  return few ? attend_q8::workspace_bytes(attend_q8::kMaxCtasPerSm * attend_q8::sm_count(), attend_q8::kMaxCols, head_dim)
             : attend_q8::workspace_bytes(attend_q8::sm_count(), attend_q8::kPromptRows, head_dim);
}

kvrp_status kv_attend_q8(const void* q, int64_t q_stride, const kvrp_seqs* seqs, int32_t n_q_heads, int32_t n_kv_heads,
                         int32_t head_dim, float softmax_scale, const void* k_pool, const void* v_pool, const float* k_scale,
                         const float* v_scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                         uint32_t* d_status, kvrp_stream_t stream) {
  const char* fn = "kv_attend_q8";
  g_last_launches = 0;
  kvrp_status st = check_seqs(fn, seqs);
  if (st != KVRP_OK) return st;
  st = check_heads(fn, n_q_heads, n_kv_heads, head_dim);
  if (st != KVRP_OK) return st;
  if (!q || !k_pool || !v_pool || !k_scale || !v_scale || !out) return fail(KVRP_ERR_INVALID_ARG, "%s: NULL argument", fn);
  if (!(softmax_scale > 0.f) || !std::isfinite(softmax_scale))
    return fail(KVRP_ERR_INVALID_ARG, "%s: softmax_scale must be > 0", fn);
  const int64_t q_row = (int64_t)n_q_heads * head_dim;
  q_stride = q_stride ? q_stride : q_row;
  if (q_stride < q_row) return fail(KVRP_ERR_INVALID_ARG, "%s: a row stride is shorter than the row", fn);
  if (q_stride % 8 || !aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out))
    return fail(KVRP_ERR_ALIGNMENT, "%s: pointers must be 16-byte aligned, strides multiples of 8", fn);
  for (const void* x : {(const void*)k_scale, (const void*)v_scale, (const void*)lse, (const void*)d_status})
    if (reinterpret_cast<uintptr_t>(x) % 4) return fail(KVRP_ERR_ALIGNMENT, "%s: a 4-byte array is not aligned", fn);
  if (seqs->n_rows == 0) return KVRP_OK;
  const int max_rows = !seqs->row_start ? 1 : seqs->max_rows ? seqs->max_rows : seqs->n_rows;
  const size_t need = kv_attend_q8_workspace_size(n_q_heads, n_kv_heads, head_dim, max_rows);
  if (!workspace || workspace_bytes < need) return fail(KVRP_ERR_WORKSPACE, "%s: workspace of %zu bytes needed", fn, need);
  const int g = n_q_heads / n_kv_heads;
  const bool few = (int64_t)max_rows * g <= attend_q8::kMaxCols;
  const int cols = few ? max_rows * g : attend_q8::kPromptRows;
  int sms = 0, smem_optin = 0;
  st = current_device_sms(&sms, &smem_optin);
  if (st != KVRP_OK) return st;

  attend_q8::Params p;
  std::memset(&p, 0, sizeof(p));
  p.q = static_cast<const uint16_t*>(q);
  p.q_stride = q_stride;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.seqs = *seqs;
  p.status = d_status;
  p.Hq = n_q_heads;
  p.Hkv = n_kv_heads;
  p.g = g;
  p.n_cta = few ? attend_q8::kMaxCtasPerSm * sms : sms;
  p.cols = few ? attend_q8::kMaxCols : attend_q8::kPromptRows;
  p.max_rows = max_rows;
  p.scale = softmax_scale * 1.4426950408889634f;
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(workspace) + 255) & ~uintptr_t(255));
  p.meta = reinterpret_cast<int4*>(base);
  p.partial = reinterpret_cast<float*>(base + attend_q8::meta_bytes(p.n_cta));
  CUtensorMap kmap, vmap;
  st = encode_q8_pool(&kmap, k_pool, seqs->num_pages, n_kv_heads * head_dim, head_dim);
  if (st == KVRP_OK) st = encode_q8_pool(&vmap, v_pool, seqs->num_pages, n_kv_heads * head_dim, head_dim);
  if (st != KVRP_OK) return st;

  if (!few) {
    const cudaError_t e = attend_q8::launch_prompt(kmap, vmap, p, head_dim, stream);
    if (e != cudaSuccess) return fail(KVRP_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
    g_last_launches = 2;
    return KVRP_OK;
  }
  const bool two = cols > 8;
  auto kernel = head_dim == 64 ? (two ? attend_q8::decode_kernel<64, 2> : attend_q8::decode_kernel<64, 1>)
                               : (two ? attend_q8::decode_kernel<128, 2> : attend_q8::decode_kernel<128, 1>);
  const int smem = head_dim == 64 ? (two ? attend_q8::Decode<64, 2>::kSmem : attend_q8::Decode<64, 1>::kSmem)
                                  : (two ? attend_q8::Decode<128, 2>::kSmem : attend_q8::Decode<128, 1>::kSmem);
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(p.n_cta);
  cfg.blockDim = dim3(32 * attend_q8::kWarps);
  cfg.dynamicSmemBytes = smem;
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, kernel, kmap, vmap, p);
  if (e == cudaSuccess) {
    cfg.gridDim = dim3(p.n_cta, cols);
    cfg.blockDim = dim3(attend_q8::kCombineThreads);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, head_dim == 64 ? attend_q8::combine_kernel<64> : attend_q8::combine_kernel<128>, p);
  }
  if (e != cudaSuccess) return fail(KVRP_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
  g_last_launches = 2;
  return KVRP_OK;
}

}  // extern "C"
