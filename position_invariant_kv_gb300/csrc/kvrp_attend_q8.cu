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
//   - Work is the list of (sequence, head group, page); each CTA takes a contiguous share of
//     equal cost, so every SM streams about the same bytes whatever the lengths; a share's part
//     of one (sequence, head group) is a segment.  The shares are computed on the device from
//     the lengths there: a captured graph keeps its balance as sequences grow.
//   - A head group is up to 8 KV heads, a warp each (or several warps, streams, a head where the
//     group is smaller).  A token's heads lie side by side, so the CTA's warps read whole
//     neighbouring pieces of the same rows at about the same time: 24 uneven sequences of 32 KV
//     heads took 253 us with a head a CTA and 109 with a head a warp.
//   - A warp is a pipeline of its own: it takes its stream's pages through a private ring of
//     16-byte asynchronous copies, swizzled on the way, which runs on across segments.  No warp
//     waits for another inside a segment.  (TMA boxes of a page and head took the same time.)
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
//   - Maxima move only when a score passes them by 2^8 (one vote a step instead of six
//     shuffles); weights then stay below 2^15, inside f16.  They are summed in fp32 before they are
//     rounded to it, 2^-11 of each at most: the output, rounded to bf16, is 1.7e-3 from the 64-bit
//     result with them as with fp32 weights, and a low part would double the second product.
// combine_kernel: merges the partial results of units that more than one CTA shared.
//
// Measured: 16 sequences x 16384 tokens, 28 / 4 heads x 128 (269 MB): 55.1 us, 4.9 TB/s, 73% of a
// copy.  From the first data to the last page the reads run at the memory's rate (about 34 us); 6 us
// go before them (the shares, the first table entries, the first pages), SMs end up to 5 us apart,
// merging and combining take 6.  24 uneven multi-head sequences (566 MB): 97 us, 87%.  4 rows x 4
// heads x 64 over 32 sequences (118 MB): 44.6 us, 40%: 8 warps an SM, each bound by the latency of its
// own chain of products and powers.  One sequence of 1000 tokens: 12 us, two launches and about ten
// dependent trips to memory.
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
#include "kvrp_q8.h"
#include "kvrp_attend_q8.h"

namespace kvrp {
namespace attend_q8 {


// ---- shares ---------------------------------------------------------------------------
constexpr int kWarps = 8, kThreads = 32 * kWarps;

struct Seq {
  int row0, rows, len, pages;   // pages 0: no work
};
// a / n and a b / n, by the 32-bit divider where they fit
__device__ __forceinline__ int64_t div64(int64_t a, int64_t b) {
  return (uint64_t)(a | b) < (1ull << 31) ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
__device__ __forceinline__ Seq seq_at(const Params& p, int s, bool* idle = nullptr, bool tell = false) {
  Seq r;
  const bool ok = sequence(p.seqs, s, r.row0, r.rows, r.len) && r.rows <= p.max_rows;
  r.pages = ok && r.rows > 0 ? (r.len + kPage - 1) / kPage : 0;
  if (tell && !ok) flag(p.status, KVRP_DEV_BAD_LENGTH);
  if (idle && r.len == 0) *idle = true;
  return r;
}

// A segment: pages [page, end) of (sequence, head group).  Shares are cut by cost: a page counts 1
// and a unit, (sequence, head group), p.unit_pages more for its queries and results, or the CTAs of a
// batch's short sequences finish last.
struct Cursor {
  int s, grp, page, end;
  int from, spent;      // the segment's costs [from, from + spent) of its unit
  int64_t left;         // cost of the share from here on
};
__device__ __forceinline__ void take(const Params& p, Cursor& c, int pages, int from) {
  const int to = (int)min((int64_t)pages + p.unit_pages, from + c.left);
  c.from = from;
  c.spent = to - from;
  c.page = max(0, from - p.unit_pages);
  c.end = max(0, to - p.unit_pages);
}
struct Plan {
  Cursor at;
  Seq seq;
  int64_t total, b;   // the cost in all, the share's end
  int n_cta;
  bool idle;          // some place of the batch is idle
};
struct PlanSmem {
  int64_t sum[kWarps];
  int64_t before;
  Seq seq;
  int found;
};

// This CTA's share of the list of (sequence, head group, page).  A share is at least kLeast
// pages a stream, so that a small batch is not cut into parts that cost more to join than to read.
constexpr int kLeast = 2;
__device__ __forceinline__ bool find_share(const Params& p, Plan* out, PlanSmem& sh) {
  const int n = p.seqs.n_seqs, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  bool idle = false;
  auto cost = [&](const Seq& q) { return q.pages > 0 ? q.pages + p.unit_pages : 0; };   // of one head group
  int64_t later = 0;   // the sequences past the first kThreads
  for (int s = kThreads + tid; s < n; s += kThreads) later += cost(seq_at(p, s, &idle, blockIdx.x == 0));
  if (n > kThreads) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) later += __shfl_xor_sync(0xffffffffu, later, o);
    if (lane == 0) sh.sum[warp] = later;
    __syncthreads();
    later = 0;
    for (int w = 0; w < kWarps; ++w) later += sh.sum[w];
    __syncthreads();
  }
  int64_t before = 0, a = 0;
  for (int s0 = 0; s0 < n; s0 += kThreads) {   // prefix sums, kThreads sequences at a time
    const int s = s0 + tid;
    Seq q = {0, 0, 0, 0};
    if (s < n) q = s0 == 0 ? seq_at(p, s, &idle, blockIdx.x == 0) : seq_at(p, s);
    const int mine = cost(q);
    int64_t sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t t = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += t;
    }
    if (lane == 31) sh.sum[warp] = sum;
    if (tid == 0) sh.found = -1;
    out->idle = __syncthreads_or(idle);
    int64_t lo = before + sum - mine;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) lo += sh.sum[w];
      before += sh.sum[w];
    }
    if (s0 == 0) {
      out->total = (before + later) * p.n_grp;
      out->n_cta = (int)min((int64_t)p.n_cta, div64(out->total + kLeast * p.streams - 1, kLeast * p.streams));
      if ((int)blockIdx.x >= out->n_cta) return false;
      a = div64(out->total * blockIdx.x, out->n_cta);
      out->b = div64(out->total * (blockIdx.x + 1), out->n_cta);
    }
    if (a >= lo * p.n_grp && a < (lo + mine) * p.n_grp) {
      sh.found = s;
      sh.before = lo * p.n_grp;
      sh.seq = q;
    }
    __syncthreads();
    if (sh.found >= 0) break;
    __syncthreads();
  }
  out->seq = sh.seq;
  out->at.s = sh.found;
  const int64_t at = a - sh.before;
  const int unit = out->seq.pages + p.unit_pages;
  out->at.grp = (int)div64(at, unit);
  out->at.left = out->b - a;
  take(p, out->at, out->seq.pages, (int)(at - (int64_t)out->at.grp * unit));
  return out->at.end > out->at.page;   // else the share ends before its unit's first page
}
// The next segment of the share; false at its end.
__device__ __forceinline__ bool next_segment(const Params& p, Cursor& c, Seq& q) {
  c.left -= c.spent;
  if (c.left <= 0) return false;
  if (++c.grp == p.n_grp) {
    c.grp = 0;
    do q = seq_at(p, ++c.s);
    while (q.pages == 0);
  }
  take(p, c, q.pages, 0);
  return c.end > 0;
}

// Asynchronous copies to shared memory (zeros past the first `bytes`), and their groups.
__device__ __forceinline__ void copy4(uint32_t to, const float* from, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t to, const uint8_t* from, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>   // until at most N of this thread's groups are in flight
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Where a box keeps 16-byte chunk `chunk` of row `row` (the row's D bytes, 16 rows): swizzled so that
// both the fragment loads of K (8 rows a chunk at a time) and of V (4 rows, every other one) and the
// copies themselves touch all banks.
template <int D>
__device__ __forceinline__ uint32_t box_offset(int row, int chunk) {
  if (D == 128) return (uint32_t)(row * 128 + ((chunk ^ (row & 7)) << 4));
  return (uint32_t)((row >> 1) * 128 + (((row ^ (row >> 1)) & 1) << 6) + ((chunk ^ ((row >> 1) & 2)) << 4));
}

// ---- decode ----------------------------------------------------------------------------
constexpr int kMergeSlots = 2;   // warps that hand over their results at a time
template <int D, int NT>
struct Decode {
  static constexpr int kPages = 128 / D;                      // pages of a step
  static constexpr int kBox = kPage * D;                      // bytes of one head's K (or V) of a page
  static constexpr int kStage = 2 * kPages * kBox;            // 4 KB
  // Two CTAs an SM, 12 KB in flight a warp; with two column tiles one CTA, 24 KB a warp: in 128
  // registers they spill (32 sequences of 4 rows x 4 x 64: 56.6 us with two CTAs, 44.8 with one).
  static constexpr int kCtas = NT == 2 ? 1 : 2;
  static constexpr int kStages = kCtas == 1 ? 6 : 3;
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kMerge = 32 * (D / 16 * NT * 4 + NT * 6);   // words of one warp's accumulator and statistics
  static constexpr int kSmem = kRing + kMergeSlots * kMerge * 4;
};

template <int D, int NT>   // head_dim; tiles of 8 (row, head) columns
__global__ void __launch_bounds__(kThreads, (Decode<D, NT>::kCtas)) decode_kernel(const __grid_constant__ Params p) {
  using C = Decode<D, NT>;
  constexpr int KT = D / 16;                 // 16-deep steps over the features; 16-feature tiles of O^T
  constexpr int PG = C::kPages, kBox = C::kBox, kStages = C::kStages, kMerge = C::kMerge;
  constexpr int FPL = D / 8;                 // features of O a lane holds for a column
  extern __shared__ __align__(128) uint8_t raw_smem[];
  __shared__ float2 scales[kWarps * kStages * PG];
  __shared__ PlanSmem plan_smem;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, tig = lane & 3;
  const uint32_t ring = smem_u32(raw_smem) + (uint32_t)warp * kStages * C::kStage;
  float* merge = reinterpret_cast<float*>(raw_smem + C::kRing);
  float2* my_scales = scales + warp * kStages * PG;
  pdl_wait();
  pdl_launch_dependents();
  Plan plan;
  if (!find_share(p, &plan, plan_smem)) {
    if (tid == 0) p.meta[blockIdx.x] = make_int4(0, 0, 0, 0);
    if (plan.idle) write_idle(p, D);
    return;
  }
  // this warp's head of the group, and its stream: pages stream, stream + streams, ... of a segment
  const int hd = warp & (p.hg - 1), stream = warp / p.hg;

  // ---- the issuing side: which pages go into the ring next ------------------------------
  // Steps that this stream has in pages [first, end).
  auto steps_of = [&](int first, int end) {
    const int blocks = (end - first + PG - 1) / PG;
    return blocks > stream ? (blocks - stream - 1) / p.streams + 1 : 0;
  };
  Cursor ic = plan.at;
  Seq iq = plan.seq;
  int i_first = ic.page;                             // the segment's first page
  int i_left = steps_of(ic.page, ic.end), i_q = 0;   // steps to issue in it, pages of the stream begun in it
  int b_page = -1, b_at = 32;                        // a batch of table entries, one a lane
  int i_st = 0;
  bool more = true;
  auto settle = [&]() {   // to the next segment that has a step for this stream
    while (i_left == 0 && (more = next_segment(p, ic, iq))) {
      i_first = i_q = 0;
      i_left = steps_of(0, ic.end);
      b_at = 32;
      // its queries, which the computing side reads some steps from now: a 128-byte line a lane
      const int lines = D / 64 * p.g, line = lane;   // of one row's heads
      for (int x = line; x < iq.rows * lines; x += 32)
        prefetch_l1(p.q + (iq.row0 + x / lines) * p.q_stride + (int64_t)((ic.grp * p.hg + hd) * p.g) * D + (x % lines) * 64);
    }
  };
  if (i_left == 0) settle();
  // A lane's 16 bytes of a box: row `brow` (and every kRows-th after it), chunk lane % (D / 16).
  constexpr int kRows = 512 / D;
  const int row_bytes = p.Hkv * D, page_bytes = row_bytes * kPage;
  const int brow = lane / (D / 16), bchunk = lane % (D / 16);
  const uint8_t* k_lane = p.k_pool + (int64_t)brow * row_bytes + bchunk * 16 + hd * D;
  const uint8_t* v_lane = p.v_pool + (int64_t)brow * row_bytes + bchunk * 16 + hd * D;
  const uint32_t to_lane = ring + box_offset<D>(brow, bchunk);
  auto issue = [&]() {
    if (more) {
      if (b_at == 32) {   // the next 32 pages of the stream
        const int q = i_q + lane, pg = i_first + (stream + q / PG * p.streams) * PG + q % PG;
        b_page = -1;      // none
        if (pg < ic.end) {
          b_page = p.seqs.block_tables[(int64_t)ic.s * p.seqs.table_stride + pg];
          if (b_page < 0 || b_page >= p.seqs.num_pages) {
            b_page = p.seqs.num_pages;   // read as zeros
            flag(p.status, KVRP_DEV_BAD_PAGE);
          }
        }
        b_at = 0;
      }
      const uint32_t at = to_lane + (uint32_t)(i_st * C::kStage);
#pragma unroll
      for (int w = 0; w < PG; ++w) {
        const int pg = __shfl_sync(0xffffffffu, b_page, b_at + w);
        if (PG > 1 && pg < 0) {   // past the segment: no weight, whatever the box holds
          if (lane == 0) my_scales[i_st * PG + w] = make_float2(0.f, 0.f);
          continue;
        }
        const uint32_t bytes = pg < p.seqs.num_pages ? 16 : 0;
        const int at_page = bytes ? pg : 0;
        const uint8_t* kf = k_lane + (int64_t)at_page * page_bytes + ic.grp * p.hg * D;
        const uint8_t* vf = v_lane + (int64_t)at_page * page_bytes + ic.grp * p.hg * D;
#pragma unroll
        for (int i = 0; i < kPage / kRows; ++i) {
          // 128: rows brow + 4 i, whose swizzle differs in bit 2 of the chunk for odd i; 64: rows brow + 8 i
          const uint32_t to = (at ^ (D == 128 && (i & 1) ? 64u : 0u)) + w * kBox + i * kRows * D;
          copy16(to, kf, bytes);
          copy16(to + PG * kBox, vf, bytes);
          kf += kRows * row_bytes;
          vf += kRows * row_bytes;
        }
        if (lane < 2)
          copy4(smem_u32(my_scales + i_st * PG + w) + 4 * lane,
                (lane ? p.v_scale : p.k_scale) + (int64_t)at_page * p.Hkv + ic.grp * p.hg + hd, bytes / 4);
      }
      i_st = i_st + 1 == kStages ? 0 : i_st + 1;
      b_at += PG;
      i_q += PG;
      if (--i_left == 0) settle();
    }
    copies_commit();   // an empty group past the share's end: the count of groups in flight stays the same
  };
#pragma unroll 1
  for (int i = 0; i < kStages; ++i) issue();

  // A lane's V fragment of a page: tokens 2 tig, 2 tig + 1, 2 tig + 8, 2 tig + 9, features gid FPL ..
  auto token_of = [&](int i) { return 2 * tig + (i & 1) + (i >> 1) * 8; };
  auto load_v = [&](uint32_t box, int i, uint32_t (&v)[FPL / 4]) {
    if constexpr (D == 128) {
      asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(box + box_offset<D>(token_of(i), gid)));
    } else {
      asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];"
                   : "=r"(v[0]), "=r"(v[1]) : "r"(box + box_offset<D>(token_of(i), gid >> 1) + (gid & 1) * 8));
    }
  };

  Cursor cc = plan.at;   // the segment being computed
  Seq cq = plan.seq;
  int c_st = 0;
  int4 meta = make_int4(0, 0, 0, 0);   // of a unit that begins here and goes on: rows, head group, parts, first row
  while (true) {
    // ---- a segment: the queries of this warp's KV head ------------------------------------
    const int first = cc.page, cols = cq.rows * p.g, ctx = cq.len - cq.rows, head = cc.grp * p.hg + hd;
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
        const uint16_t* at = p.q + (cq.row0 + c / p.g) * p.q_stride + (int64_t)(head * p.g + c % p.g) * D + tig * (D / 4);
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

    const int steps = steps_of(first, cc.end);
    int pg = first + stream * PG;
#pragma unroll 1
    for (int step = 0; step < steps; ++step, pg += p.streams * PG) {
      const int st = c_st;
      copies_wait<kStages - 1>();
      __syncwarp();   // every lane's copies of the stage have landed
      if (++c_st == kStages) c_st = 0;
      const uint32_t kat = ring + (uint32_t)st * C::kStage, vat = kat + PG * kBox;
      // the pages next to the end: a row sees its own position and before; the share's end cuts a step
      const bool tail = (pg + PG) * kPage > ctx + 1 || pg + PG > cc.end;
      // ---- S = K Q^T -----------------------------------------------------------------
      float c[PG][NT][4], f[PG][NT][2], lvs[PG];   // raw scores; x = c f; log2 of the value scales
      bool grow = false;
#pragma unroll
      for (int w = 0; w < PG; ++w) {
        const float2 sc = my_scales[st * PG + w];
        lvs[w] = lg2(sc.y);   // exact for a power of two; -inf for a zero scale
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) c[w][nt][0] = c[w][nt][1] = c[w][nt][2] = c[w][nt][3] = 0.f;
        uint32_t k0[KT], k1[KT];   // rows gid and gid + 8: features tig D/4 + 4 kk + {0..3}
#pragma unroll
        for (int i = 0; i < KT / 4; ++i) {
          const int chunk = tig * (KT / 4) + i;
          const uint32_t off = w * kBox + box_offset<D>(gid, chunk);
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
          for (int nt = 0; nt < NT; ++nt) mma16816_f16(c[w][nt], a, qb[kk][nt][0], qb[kk][nt][1]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int b = 0; b < 2; ++b) f[w][nt][b] = sc.x * fac[nt][b];
      }
      if (tail) {   // rare, and a branch: as selects it would cost every page a third of its instructions
#pragma unroll
        for (int w = 0; w < PG; ++w)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const int seen = pg + w < cc.end ? limit[nt][b] - (pg + w) * kPage : 0;
              // -inf times the factor has to stay -inf, also where the page has no say or the product underflows
              if (seen <= 0) f[w][nt][b] = 1.f;
              else if (f[w][nt][b] < kLeastFactor) f[w][nt][b] = kLeastFactor;
              if (gid >= seen) make_minus_inf(c[w][nt][b]);
              if (gid + 8 >= seen) make_minus_inf(c[w][nt][2 + b]);
            }
      }
#pragma unroll
      for (int w = 0; w < PG; ++w)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int b = 0; b < 2; ++b)
            grow |= fmaxf(c[w][nt][b], c[w][nt][2 + b]) * f[w][nt][b] > fminf(m[nt][b], om[nt][b] - lvs[w]) + kLazy;
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            float t = -INFINITY, u = -INFINITY;
#pragma unroll
            for (int w = 0; w < PG; ++w) {
              const float x = fmaxf(c[w][nt][b], c[w][nt][2 + b]) * f[w][nt][b];
              t = fmaxf(t, x);
              u = fmaxf(u, x + lvs[w]);
            }
#pragma unroll
            for (int d = 4; d < 32; d *= 2) {
              t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, d));
              u = fmaxf(u, __shfl_xor_sync(0xffffffffu, u, d));
            }
            const float nm = fmaxf(m[nt][b], t), no = fmaxf(om[nt][b], u);
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
      uint32_t pb[PG][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float mm[2], oo[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          mm[b] = m[nt][b] == -INFINITY ? 0.f : m[nt][b];
          oo[b] = (om[nt][b] == -INFINITY ? 0.f : om[nt][b]) - kShift;
        }
#pragma unroll
        for (int w = 0; w < PG; ++w) {
          float e4[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = c[w][nt][e], k = f[w][nt][e & 1];
            l[nt][e & 1] += ex2(fmaf(x, k, -mm[e & 1]));
            e4[e] = ex2(fmaf(x, k, lvs[w] - oo[e & 1]));
          }
          pb[w][nt][0] = movmatrix_trans(pack_f16(e4[0], e4[1]));
          pb[w][nt][1] = movmatrix_trans(pack_f16(e4[2], e4[3]));
        }
      }
      // ---- O^T += V^T P^T --------------------------------------------------------------
#pragma unroll
      for (int w = 0; w < PG; ++w) {
        uint32_t v[4][FPL / 4];
#pragma unroll
        for (int i = 0; i < 4; ++i) load_v(vat + w * kBox, i, v[i]);
        if (tail) {   // a slot past the sequence, or past the share, may hold anything, NaN included
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if ((pg + w) * kPage + token_of(i) >= cq.len || pg + w >= cc.end) {
#pragma unroll
              for (int j = 0; j < FPL / 4; ++j) make_zero(v[i][j]);
            }
          }
          // A NaN of a token that not all rows see: weight 0 would not keep it from the others.  It is taken out
          // of the stage, byte by byte and on few registers, and the accumulators of the rows that do see it
          // become NaN.  (Looking for it costs a sequence's last pages: 43.5 -> 44.5 us for 4 rows x 32 sequences.
          // One row a sequence has no such tokens: with one tile of columns leaving the vote out takes 11.5 us
          // instead of 11.8 for a short sequence; with two the other code that it leads to takes 45.2 instead of 44.5.)
          const int t0 = (pg + w) * kPage;
          bool odd = false;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t nan = 0;
#pragma unroll
            for (int j = 0; j < FPL / 4; ++j) nan |= q8::nan_bytes(v[i][j]);
            odd |= nan && t0 + token_of(i) > ctx;
          }
          if ((NT == 2 || cq.rows > 1) && __any_sync(0xffffffffu, odd)) {
            const int end = pg + w < cc.end ? cq.len : 0;
#pragma unroll
            for (int f = 0; f < FPL; ++f) {
              int at = INT32_MAX;   // the first such token with a NaN in this lane's feature f
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int t = t0 + token_of(i);
                const uint32_t byte = vat + w * kBox + box_offset<D>(token_of(i), gid * FPL / 16) + (gid * FPL + f) % 16;
                uint32_t x;
                asm volatile("ld.shared.u8 %0, [%1];" : "=r"(x) : "r"(byte));
                if (t > ctx && t < end && (x & 0x7f) == 0x7f) {
                  at = min(at, t);
                  asm volatile("st.shared.u8 [%0], %1;" ::"r"(byte), "r"(0) : "memory");
                }
              }
              at = min(at, __shfl_xor_sync(0xffffffffu, at, 1));
              at = min(at, __shfl_xor_sync(0xffffffffu, at, 2));
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int b = 0; b < 2; ++b)
                  if (at < limit[nt][b]) o[f / 2][nt][2 * (f % 2) + b] = __int_as_float(0x7fc00000);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              load_v(vat + w * kBox, i, v[i]);
              if (t0 + token_of(i) >= end)
#pragma unroll
                for (int j = 0; j < FPL / 4; ++j) make_zero(v[i][j]);
            }
          }
        }
#pragma unroll
        for (int j = 0; j < FPL / 4; ++j)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t sel = half ? 0x7362u : 0x5140u;
            const uint32_t x = __byte_perm(v[0][j], v[1][j], sel), y = __byte_perm(v[2][j], v[3][j], sel);
            const uint32_t a[4] = {q8::e4m3x2_to_f16x2((uint16_t)x), q8::e4m3x2_to_f16x2((uint16_t)(x >> 16)),
                                   q8::e4m3x2_to_f16x2((uint16_t)y), q8::e4m3x2_to_f16x2((uint16_t)(y >> 16))};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816_f16(o[2 * j + half][nt], a, pb[w][nt][0], pb[w][nt][1]);
          }
      }
      __syncwarp();   // every lane has read the stage
      issue();
    }
    // ---- merge the streams of a head ----------------------------------------------------------
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
    // Warps from, from + 1 into to, to + 1; with warp = stream * hg + head these are streams of
    // the same heads, and one, two or four heads a group need the first four, three or two rounds.
    const int live = min(p.streams, (cc.end - first + PG - 1) / PG) * p.hg;   // warps that had a page
    for (int round = 0; round < p.rounds; ++round) {
      const int from = round == 0 ? 6 : round == 1 ? 4 : round == 2 ? 2 : 1, to = round == 0 ? 2 : 0, count = round == 3 ? 1 : 2;
      if (from >= live) continue;
      const bool gives = warp >= from && warp < from + count && warp < live;
      const bool takes = warp >= to && warp < to + count && warp - to + from < live;
      float* at = merge + (warp - (gives ? from : to)) * kMerge + lane;
      if (gives) {
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
      if (takes) {
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
    if (begins && !ends) {
      // the CTA whose share holds the unit's last page: the largest j with total j / n_cta below the unit's end
      const int64_t last = plan.b - cc.left - cc.from + cq.pages + p.unit_pages;
      const int j = (int)div64(last * plan.n_cta - 1, plan.total);
      meta = make_int4(cq.rows, cc.grp, j - (int)blockIdx.x + 1, cq.row0);
    }
    if (stream == 0) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int c = nt * 8 + 2 * tig + b;
          if (c >= cols) continue;
          if (begins && ends) {
            const float2 r = result_factors(m[nt][b], om[nt][b], l[nt][b]);
            const int64_t row = (int64_t)(cq.row0 + c / p.g) * p.Hq + head * p.g + c % p.g;
            uint32_t w[FPL / 2];
#pragma unroll
            for (int mt = 0; mt < KT; ++mt) {
              const __nv_bfloat162 v = __floats2bfloat162_rn(o[mt][nt][b] * r.x * r.y, o[mt][nt][2 + b] * r.x * r.y);
              w[mt] = *reinterpret_cast<const uint32_t*>(&v);
            }
            uint4* to = reinterpret_cast<uint4*>(p.out + row * D + gid * FPL);
#pragma unroll
            for (int i = 0; i < FPL / 8; ++i) to[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
            if (p.lse && gid == 0) p.lse[row] = (m[nt][b] + lg2(l[nt][b])) * kLn2;
          } else {
            float* to = p.partial + ((int64_t)(blockIdx.x * 2 + (begins ? 1 : 0)) * p.cols + hd * p.max_rows * p.g + c) * (D + 4);
            float4* of = reinterpret_cast<float4*>(to + gid * FPL);
#pragma unroll
            for (int i = 0; i < FPL / 4; ++i)
              of[i] = make_float4(o[2 * i][nt][b], o[2 * i][nt][2 + b], o[2 * i + 1][nt][b], o[2 * i + 1][nt][2 + b]);
            if (gid == 0) *reinterpret_cast<float4*>(to + D) = make_float4(m[nt][b], om[nt][b], l[nt][b], 0.f);
          }
        }
    }
    if (!next_segment(p, cc, cq)) break;
  }
  if (tid == 0) p.meta[blockIdx.x] = meta;
  if (plan.idle) write_idle(p, D);
}

// ---- combine ---------------------------------------------------------------------------
// An item is one (head of the group, column) of a unit that begins in some CTA i and goes on in
// CTAs i + 1, ...; every block lists those units from the CTAs' records.  A group of threads
// holds an item's features, four each.  Where units have few parts each group takes an item of its
// own; else a block takes one, its groups every kGroups-th part.
constexpr int kCombineThreads = 128, kFewParts = 16;
template <int D>
__global__ void __launch_bounds__(kCombineThreads, 5) combine_kernel(const __grid_constant__ Params p) {
  constexpr int kLanes = D / 4, kGroups = kCombineThreads / kLanes, kWarpsHere = kCombineThreads / 32;
  __shared__ float4 part[kGroups][kLanes];
  __shared__ float stat[kGroups][3];
  __shared__ int4 unit[kMaxCtas];   // its record, with the CTA in x's high half
  __shared__ int count[kWarpsHere], total[kWarpsHere];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, f = tid % kLanes, grp = tid / kLanes;
  int units = 0, parts = 0;
  for (int j0 = 0; j0 < p.n_cta; j0 += kCombineThreads) {
    const int j = j0 + tid;
    int4 mt = j < p.n_cta ? p.meta[j] : make_int4(0, 0, 0, 0);
    const bool begins = mt.x > 0;
    const uint32_t vote = __ballot_sync(0xffffffffu, begins);
    const int sum = __reduce_add_sync(0xffffffffu, begins ? mt.z : 0);
    if ((tid & 31) == 0) count[tid >> 5] = __popc(vote), total[tid >> 5] = sum;
    __syncthreads();
    int at = units + __popc(vote & ((1u << (tid & 31)) - 1));
#pragma unroll
    for (int w = 0; w < kWarpsHere; ++w) {
      if (w < (tid >> 5)) at += count[w];
      units += count[w];
      parts += total[w];
    }
    mt.x |= j << 16;   // a record's rows are at most 16
    if (begins) unit[at] = mt;
    __syncthreads();
  }
  const int most = p.max_rows * p.g;
  const bool alone = parts <= kFewParts * units && units * p.cols > (int)gridDim.x;   // a group an item
  const int per = alone ? kGroups : 1, step = alone ? 1 : kGroups;
  for (int first = blockIdx.x * per; first < units * p.cols; first += gridDim.x * per) {
    const int item = first + (alone ? grp : 0);
    const int4 mt = unit[min(item, units * p.cols - 1) / p.cols];
    const int i = mt.x >> 16, y = item % p.cols, hd = y / most, c = y % most;
    const bool live = item < units * p.cols && c < (mt.x & 0xffff) * p.g;
    const int n = live ? min(mt.z, p.n_cta - i) : 0;
    float m = -INFINITY, om = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kBatch = 8;   // parts in flight
    for (int k0 = alone ? 0 : grp; k0 < n; k0 += kBatch * step) {
      float4 s[kBatch], v[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int k = k0 + b * step;
        s[b] = make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
        v[b] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k < n) {
          const float* e = p.partial + ((int64_t)((i + k) * 2 + (k == 0 ? 1 : 0)) * p.cols + y) * (D + 4);
          s[b] = *reinterpret_cast<const float4*>(e + D);
          v[b] = reinterpret_cast<const float4*>(e)[f];
        }
      }
      float nm = m, no = om;
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        nm = fmaxf(nm, s[b].x);
        no = fmaxf(no, s[b].y);
      }
      const float zm = nm == -INFINITY ? 0.f : nm, zo = no == -INFINITY ? 0.f : no;   // 2^-inf = 0, and no inf - inf
      l *= ex2(m - zm);
      const float r = ex2(om - zo);
      acc = make_float4(acc.x * r, acc.y * r, acc.z * r, acc.w * r);
      m = nm;
      om = no;
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        l = fmaf(s[b].z, ex2(s[b].x - zm), l);
        const float w = ex2(s[b].y - zo);
        acc.x = fmaf(v[b].x, w, acc.x);
        acc.y = fmaf(v[b].y, w, acc.y);
        acc.z = fmaf(v[b].z, w, acc.z);
        acc.w = fmaf(v[b].w, w, acc.w);
      }
    }
    if (!alone) {
      __syncthreads();   // the last item's have been read
      part[grp][f] = acc;
      if (f == 0) stat[grp][0] = m, stat[grp][1] = om, stat[grp][2] = l;
      __syncthreads();
      if (grp != 0) continue;
      m = om = -INFINITY;
      l = 0.f;
#pragma unroll
      for (int k = 0; k < kGroups; ++k) {
        m = fmaxf(m, stat[k][0]);
        om = fmaxf(om, stat[k][1]);
      }
      acc = make_float4(0.f, 0.f, 0.f, 0.f);
      const float zm = m == -INFINITY ? 0.f : m, zo = om == -INFINITY ? 0.f : om;
#pragma unroll
      for (int k = 0; k < kGroups; ++k) {
        l = fmaf(stat[k][2], ex2(stat[k][0] - zm), l);
        const float w = ex2(stat[k][1] - zo);
        acc.x = fmaf(part[k][f].x, w, acc.x);
        acc.y = fmaf(part[k][f].y, w, acc.y);
        acc.z = fmaf(part[k][f].z, w, acc.z);
        acc.w = fmaf(part[k][f].w, w, acc.w);
      }
    }
    if (!live) continue;
    const float2 r = result_factors(m, om, l);
    acc = make_float4(acc.x * r.x * r.y, acc.y * r.x * r.y, acc.z * r.x * r.y, acc.w * r.x * r.y);
    const int64_t row = (int64_t)(mt.w + c / p.g) * p.Hq + (mt.y * p.hg + hd) * p.g + c % p.g;
    const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x, acc.y), hi = __floats2bfloat162_rn(acc.z, acc.w);
    *reinterpret_cast<uint2*>(p.out + row * D + 4 * f) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    if (p.lse && f == 0) p.lse[row] = (m + lg2(l)) * kLn2;
  }
}

// KV heads that a CTA takes together: the largest power of two that divides them, at most its
// warps.  A token's heads lie side by side, so the warps of a CTA then read neighbouring bytes
// at about the same time, and there are fewer streams of a head to merge.
int head_group(int n_kv_heads) {
  int hg = 1;
  while (hg < kWarps && n_kv_heads % (2 * hg) == 0) hg *= 2;
  return hg;
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      n <= 0) {
    cudaGetLastError();
    n = 160;   // no device: a size for the checks of a host without one
  }
  return std::min(n, kMaxCtas / kMaxCtasPerSm);
}

size_t meta_bytes(int n_cta) { return ((size_t)n_cta * 2 * sizeof(int4) + 255) / 256 * 256; }
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
  return few ? attend_q8::workspace_bytes(attend_q8::kMaxCtasPerSm * attend_q8::sm_count(),
                                          attend_q8::head_group(n_kv_heads) * max_rows * (n_q_heads / n_kv_heads), head_dim)
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
  if ((int64_t)seqs->n_rows * n_q_heads >= 1ll << 32 || (int64_t)seqs->n_rows * g >= (1 << 28) - attend_q8::kPromptRows)
    return fail(KVRP_ERR_UNSUPPORTED, "%s: n_rows x n_q_heads must stay below 2^32, n_rows x group below 2^28", fn);
  const int hg = attend_q8::head_group(n_kv_heads);
  int sms = 0, smem_optin = 0;
  st = current_device_sms(&sms, &smem_optin);
  if (st != KVRP_OK) return st;

  attend_q8::Params p;
  std::memset(&p, 0, sizeof(p));
  p.q = static_cast<const uint16_t*>(q);
  p.q_stride = q_stride;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.k_pool = static_cast<const uint8_t*>(k_pool);
  p.v_pool = static_cast<const uint8_t*>(v_pool);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.seqs = *seqs;
  p.status = d_status;
  p.Hq = n_q_heads;
  p.Hkv = n_kv_heads;
  p.g = g;
  p.g_inverse = ((1ull << 32) + g - 1) / g;
  p.n_cta = std::min(attend_q8::kMaxCtas, few ? attend_q8::kMaxCtasPerSm * sms : sms);
  p.cols = few ? hg * max_rows * g : attend_q8::kPromptRows;
  p.max_rows = max_rows;
  p.hg = hg;
  p.n_grp = n_kv_heads / hg;
  p.streams = attend_q8::kWarps / hg;
  p.unit_pages = std::max(1, 2048 / (hg * head_dim));   // about 2 us of a CTA's share of the bandwidth
  p.rounds = hg == 1 ? 4 : hg == 2 ? 3 : hg == 4 ? 2 : 0;
  p.scale = softmax_scale * 1.4426950408889634f;
  p.wait_cycles = test_wait_limit() ? (long long)test_wait_limit() : ptx::kTimeoutCycles;
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(workspace) + 255) & ~uintptr_t(255));
  p.meta = reinterpret_cast<int4*>(base);
  p.partial = reinterpret_cast<float*>(base + attend_q8::meta_bytes(p.n_cta));
  if (!few) {
    CUtensorMap kmap, vmap;
    st = encode_q8_pool(&kmap, k_pool, seqs->num_pages, n_kv_heads * head_dim, head_dim);
    if (st == KVRP_OK) st = encode_q8_pool(&vmap, v_pool, seqs->num_pages, n_kv_heads * head_dim, head_dim);
    if (st != KVRP_OK) return st;
    const cudaError_t e = attend_q8::launch_prompt(kmap, vmap, p, head_dim, stream);
    if (e != cudaSuccess) return fail(KVRP_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
    g_last_launches = 2;
    return KVRP_OK;
  }
  const bool two = max_rows * g > 8;
  if (two) p.n_cta = std::min(p.n_cta, attend_q8::Decode<128, 2>::kCtas * sms);
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
  cfg.blockDim = dim3(attend_q8::kThreads);
  cfg.dynamicSmemBytes = smem;
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, kernel, p);
  if (e == cudaSuccess) {
    cfg.gridDim = dim3(5 * sms);
    cfg.blockDim = dim3(attend_q8::kCombineThreads);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, head_dim == 64 ? attend_q8::combine_kernel<64> : attend_q8::combine_kernel<128>, p);
  }
  if (e != cudaSuccess) return fail(KVRP_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
  g_last_launches = 2;
  return KVRP_OK;
}

}  // extern "C"
