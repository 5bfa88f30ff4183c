// Attention of many rows over the 8-bit paged cache (kv_attend_q8 on prompts).
//
//   out[r][j] = softmax(scale q[r][j] . K) V, causal; K_t = ks[page] K8_t, V_t = vs[page] V8_t.
//
// Bound by the tensor cores: 4 head_dim operations for each (row, head, visible token).
//   - A unit is 256 rows of one (sequence, KV head): the rows x group pairs (token, query
//     head) in order, so every row of the tile is used whatever the group, and K and V are
//     loaded once for all query heads that share them.  It runs over its visible tokens in
//     tiles of 128.  The list of (unit, token tile) is cut into equal contiguous shares, one
//     a CTA, on the device; a unit that several CTAs share goes through the combine.
//   - S = Q K^T by tcgen05 kind::f8f6f4: K goes from memory to the tensor cores as stored.
//     q is split into two e4m3 parts, high and low, after its row was divided by a power of
//     two: bf16's 8 significant bits are 4 + 4, so the parts are q exactly down to 2^-10 of
//     the row's largest element and off by at most 2^-18 of it below.  Two products at
//     twice the f16 rate cost what one would, without converting K.
//   - O += P V by kind::f16: P as f16 from TMEM (it takes the place of its scores), V as f16 in
//     shared memory, converted from e4m3 by four warps together with the page's scale
//     relative to a running reference (a power of two): exact for power-of-two scales
//     within 2^14 of each other.
//   - Warps: two groups of four hold 128 rows each, a thread a row, and turn scores into
//     weights while the tensor cores work on the other group's tile; four convert V; one
//     issues TMA boxes (a page and head each), one the MMAs.
#include <algorithm>

#include "kvrp_attend_q8.h"

namespace kvrp {
namespace attend_q8 {

namespace {

constexpr int kTile = 128;                 // tokens of a K, V tile; rows of a Q tile
constexpr int kPagesPerTile = kTile / kPage;
constexpr int kWarpsAll = 16, kThreadsAll = 32 * kWarpsAll;
constexpr int kScaleSlots = 8;             // tiles whose scales are kept: K runs at most kKst + 1 ahead of the softmax
constexpr float kVShift = 7.f;             // V enters as v * vs * 2^7 / vref: up to 448 * 128 in f16

template <int D>
struct Prompt {
  static constexpr int kQ = kTile * D;             // bytes of one e4m3 part of a Q tile
  static constexpr int kKV = kTile * D;            // bytes of a raw K or V tile
  static constexpr int kKst = 3, kVst = 2;         // stages of K, of raw V
  static constexpr int kVc = kTile * D * 2;        // bytes of a converted V tile (two buffers)
  static constexpr int kOffK = 4 * kQ, kOffV = kOffK + kKst * kKV, kOffVc = kOffV + kVst * kKV;
  static constexpr int kSmem = 1024 + kOffVc + 2 * kVc;
};

// ---- tensor-core pieces ------------------------------------------------------------------
// Shared-memory matrix descriptors.  K-major, rows of D bytes swizzled over D (128 or 64) bytes.
template <int D>
__device__ __forceinline__ uint64_t desc_rows(uint32_t addr) {
  uint64_t d = (uint64_t)((addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)1 << 16;
  d |= (uint64_t)(8 * D >> 4) << 32;                 // next 8 rows
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)(D == 128 ? 2 : 4) << 61;           // 128- or 64-byte swizzle
  return d;
}
// N-major (the transposed operand): 64 f16 columns = 128 swizzled bytes a token, 8 tokens an atom.
__device__ __forceinline__ uint64_t desc_cols(uint32_t addr) {
  uint64_t d = (uint64_t)((addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(kTile * 128 >> 4) << 16;           // next 64 columns
  d |= (uint64_t)(1024 >> 4) << 32;                  // next 8 tokens
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
// Two fp32 operations an instruction.
__device__ __forceinline__ uint64_t pair2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpair2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// Until this thread's TMEM loads have arrived; names the registers they fill, so that nothing that
// reads them can be moved ahead of the wait.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.wait::ld.sync.aligned;"
      : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), 
        "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), 
        "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), 
        "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
      :
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.wait::ld.sync.aligned;"
      : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), 
        "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
      :
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ---- units and shares ------------------------------------------------------------------------
// A unit's part inside this CTA's share: tiles [j0, j1) of its n_kv.
struct Unit {
  int s, rt, h;             // sequence, row tile, KV head
  int row0, rows, len;      // the sequence
  int n_rt, n_kv, j0, j1;
  int64_t left;             // tiles of the share from j0 on
};
__device__ __forceinline__ int tiles_of(int row0_col, int g, int rows, int len) {   // token tiles of a row tile
  const int last = min(rows - 1, (row0_col + kPromptRows - 1) / g);                 // its last token among the rows
  return (len - rows + last + kTile) / kTile;
}
__device__ __forceinline__ bool load_seq(const Params& p, int s, Unit& u, bool tell = false) {
  const bool ok = sequence(p.seqs, s, u.row0, u.rows, u.len) && u.rows <= p.max_rows;
  if (tell && !ok) flag(p.status, KVRP_DEV_BAD_LENGTH);
  u.n_rt = ok ? (int)(((int64_t)u.rows * p.g + kPromptRows - 1) / kPromptRows) : 0;
  return u.n_rt > 0;
}
// The tiles of sequence s over all its row tiles, by one warp (one head's worth).
__device__ __forceinline__ int64_t seq_cost(const Params& p, int s, bool tell) {
  Unit u;
  int64_t sum = 0;
  if (load_seq(p, s, u, tell && (threadIdx.x & 31) == 0))
    for (int rt = threadIdx.x & 31; rt < u.n_rt; rt += 32) sum += tiles_of(rt * kPromptRows, p.g, u.rows, u.len);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}
struct Shared {
  __align__(8) uint64_t bars[32];
  float ks[kScaleSlots][kPagesPerTile], vs[kScaleSlots][kPagesPerTile];
  int64_t cost[kWarpsAll];
  Unit first;
  int found;
  int abort_flag;
  uint32_t tmem;
};
__device__ __forceinline__ bool find_share(const Params& p, Shared& sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = p.seqs.n_seqs;
  int64_t mine = 0;
  for (int s = warp; s < n; s += kWarpsAll) mine += seq_cost(p, s, blockIdx.x == 0) * p.Hkv;
  if (lane == 0) sh.cost[warp] = mine;
  __syncthreads();
  int64_t total = 0;
  for (int w = 0; w < kWarpsAll; ++w) total += sh.cost[w];
  const int64_t n_cta = min((int64_t)p.n_cta, total);
  if ((int)blockIdx.x >= n_cta) return false;
  const int64_t a = total * blockIdx.x / n_cta, b = total * (blockIdx.x + 1) / n_cta;
  int64_t before = 0;
  int s = 0;
  for (int s0 = 0; s0 < n; s0 += kWarpsAll) {   // the sequence that holds tile a
    __syncthreads();
    const int64_t c = s0 + warp < n ? seq_cost(p, s0 + warp, false) * p.Hkv : 0;
    if (lane == 0) sh.cost[warp] = c;
    __syncthreads();
    bool here = false;
    for (int w = 0; w < kWarpsAll && !here; ++w) {
      here = a < before + sh.cost[w];
      if (here) s = s0 + w;
      else before += sh.cost[w];
    }
    if (here) break;
  }
  // the unit inside it, by warp 0: 32 row tiles at a time
  if (warp == 0) {
    Unit u;
    load_seq(p, s, u);
    int64_t at = a - before;   // tiles into the sequence
    for (int r0 = 0; r0 < u.n_rt; r0 += 32) {
      const int rt = r0 + lane;
      const int t = rt < u.n_rt ? tiles_of(rt * kPromptRows, p.g, u.rows, u.len) : 0;
      int64_t sum = (int64_t)t * p.Hkv;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
      }
      const int64_t lo = sum - (int64_t)t * p.Hkv;
      if (at >= lo && at < sum) {
        u.s = s;
        u.rt = rt;
        u.n_kv = t;
        u.h = (int)((at - lo) / t);
        u.j0 = (int)((at - lo) % t);
        u.left = b - a;
        u.j1 = (int)min((int64_t)t, u.j0 + u.left);
        sh.first = u;
      }
      at -= __shfl_sync(0xffffffffu, sum, 31);
      if (at < 0) break;
    }
  }
  __syncthreads();
  return true;
}
// The share's next unit; false at its end.
__device__ __forceinline__ bool next_unit(const Params& p, Unit& u) {
  u.left -= u.j1 - u.j0;
  if (u.left <= 0) return false;
  if (++u.h == p.Hkv) {
    u.h = 0;
    if (++u.rt == u.n_rt) {
      u.rt = 0;
      do ++u.s;
      while (!load_seq(p, u.s, u));
    }
    u.n_kv = tiles_of(u.rt * kPromptRows, p.g, u.rows, u.len);
  }
  u.j0 = 0;
  u.j1 = (int)min((int64_t)u.n_kv, u.left);
  return true;
}
__device__ __forceinline__ int active_tiles(const Params& p, const Unit& u) {   // Q tiles with rows in them
  return (int64_t)u.rows * p.g - (int64_t)u.rt * kPromptRows > kTile ? 2 : 1;
}
// The reference of the value scales after a tile: a power of two at least the largest scale,
// two octaves above it when it moves, so that it moves seldom.
__device__ __forceinline__ float next_vref(float vref, const float* vs) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < kPagesPerTile; ++i) top = fmaxf(top, vs[i]);
  if (!(top > vref)) return vref;
  const uint32_t e = (__float_as_uint(top) + 0x7fffffu) >> 23;   // 2^ceil(log2 top)
  return __uint_as_float(min(e + 2u, 254u) << 23);
}

template <int D>
__global__ void __launch_bounds__(kThreadsAll, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                  const __grid_constant__ Params p) {
  using L = Prompt<D>;
  extern __shared__ uint8_t raw_smem[];
  __shared__ Shared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t smem = (smem_u32(raw_smem) + 1023u) & ~1023u;
  const uint32_t bar0 = smem_u32(sh.bars);
  auto kfull = [&](int i) { return bar0 + 8u * i; };
  auto kempty = [&](int i) { return bar0 + 8u * (3 + i); };
  auto vfull = [&](int i) { return bar0 + 8u * (6 + i); };
  auto vempty = [&](int i) { return bar0 + 8u * (8 + i); };
  auto cfull = [&](int i) { return bar0 + 8u * (10 + i); };    // converted V
  auto cempty = [&](int i) { return bar0 + 8u * (12 + i); };
  auto qfull = [&](int t) { return bar0 + 8u * (14 + t); };
  auto sfull = [&](int t) { return bar0 + 8u * (16 + t); };    // scores in TMEM
  auto pfull = [&](int t, int half) { return bar0 + 8u * (18 + 2 * t + half); };   // weights in TMEM, accumulator corrected
  auto ofull = [&](int t) { return bar0 + 8u * (22 + t); };    // accumulator updated
  auto drained = [&](int t) { return bar0 + 8u * (24 + t); };
  if (tid == 0) {
    for (int i = 0; i < 3; ++i) mbar_init(kfull(i), 1), mbar_init(kempty(i), 2);   // both Q tiles
    for (int i = 0; i < 2; ++i) {
      mbar_init(vfull(i), 1);
      mbar_init(vempty(i), 128);
      mbar_init(cfull(i), 128);
      mbar_init(cempty(i), 2);
      mbar_init(qfull(i), 128);
      mbar_init(sfull(i), 1);
      mbar_init(pfull(i, 0), 128);
      mbar_init(pfull(i, 1), 128);
      mbar_init(ofull(i), 1);
      mbar_init(drained(i), 1);
    }
    sh.abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 13) tmem_alloc(smem_u32(&sh.tmem), 512);
  if (tid == 32) {
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
  }
  pdl_wait();
  pdl_launch_dependents();
  const bool any = find_share(p, sh);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  volatile int* abort_p = &sh.abort_flag;
  auto wait = [&](uint32_t bar, uint32_t parity) {   // the same answer in the whole warp
    const bool ok = wait_phase(bar, parity, abort_p, p.status);
    return __all_sync(0xffffffffu, ok) != 0;
  };
  Unit u = sh.first;

  if (!any) {
    if (tid == 0) p.meta[blockIdx.x] = make_int4(-1, 0, 0, 0);
  } else if (warp == 12) {
    // ---- TMA: a lane a page ---------------------------------------------------------------
    int n = 0, nk = 0, nv = 0;   // the tile, K and V tiles issued
    bool ok = true;
    do {
      const int pages = (u.len + kPage - 1) / kPage;
      for (int j = u.j0; j < u.j1 && ok; ++j, ++n) {
        const int ks = n % L::kKst, vs = n % L::kVst, slot = n % kScaleSlots;
        const int pg = j * kPagesPerTile + lane;
        const bool mine = lane < kPagesPerTile && pg < pages;
        int page = p.seqs.num_pages;   // past the pool: the box reads zeros
        float fk = 0.f, fv = 0.f;
        if (mine) {
          const int e = p.seqs.block_tables[(int64_t)u.s * p.seqs.table_stride + pg];
          if (e >= 0 && e < p.seqs.num_pages) {
            page = e;
            fk = p.k_scale[(int64_t)e * p.Hkv + u.h];
            fv = p.v_scale[(int64_t)e * p.Hkv + u.h];
          } else {
            flag(p.status, KVRP_DEV_BAD_PAGE);
          }
        }
        ok = wait(kempty(ks), ((n / L::kKst) & 1) ^ 1);   // the first pass finds the stage free
        if (!ok) break;
        // tile n - kScaleSlots has been turned into weights long ago: K runs at most kKst ahead
        if (lane < kPagesPerTile) {
          sh.ks[slot][lane] = fk;
          sh.vs[slot][lane] = fv;
        }
        const uint32_t bytes = (uint32_t)min(kPagesPerTile, pages - j * kPagesPerTile) * kPage * D;
        __syncwarp();
        if (lane == 0) mbar_expect_tx(kfull(ks), bytes);
        __syncwarp();
        if (mine) tma_load_3d(smem + L::kOffK + ks * L::kKV + lane * kPage * D, &kmap, kfull(ks), u.h * D, 0, page);
        ++nk;
        ok = wait(vempty(vs), ((n / L::kVst) & 1) ^ 1);
        if (!ok) break;
        if (lane == 0) mbar_expect_tx(vfull(vs), bytes);
        __syncwarp();
        if (mine) tma_load_3d(smem + L::kOffV + vs * L::kKV + lane * kPage * D, &vmap, vfull(vs), u.h * D, 0, page);
        ++nv;
      }
    } while (ok && next_unit(p, u));
    if (!ok && lane == 0) {   // every issued copy lands before the CTA exits
      for (int i = max(0, nk - L::kKst); i < nk; ++i) drain_wait(kfull(i % L::kKst), (i / L::kKst) & 1, p.status);
      for (int i = max(0, nv - L::kVst); i < nv; ++i) drain_wait(vfull(i % L::kVst), (i / L::kVst) & 1, p.status);
    }
  } else if (warp == 13 || warp == 14) {
    // ---- MMA: a warp a Q tile, so that one tile's waits leave the tensor cores to the other ----
    const int t = warp - 13;
    // descriptor: fp32 accumulator, M = 128; e4m3 (0) or f16 (0) operands; the second product's B is N-major
    const uint32_t id_qk = (1u << 4) | ((uint32_t)(kTile >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
    const uint32_t id_pv = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
    int n = 0;                   // tiles begun
    uint32_t nq = 0, np = 0;     // units begun and tiles weighted, of this Q tile
    bool ok = true;
    do {
      const int act = active_tiles(p, u);
      if (t >= act) {            // no rows: the stages pass by, every phase observed (a wait tests a parity only)
        for (int j = u.j0; j < u.j1 && ok; ++j, ++n) {
          ok = wait(kfull(n % L::kKst), (n / L::kKst) & 1);
          if (ok && lane == 0) mbar_arrive(kempty(n % L::kKst));
          ok = ok && wait(cfull(n & 1), (n >> 1) & 1);
          if (ok && lane == 0) mbar_arrive(cempty(n & 1));
          __syncwarp();
        }
        continue;
      }
      auto scores = [&](int tile) {   // S_t = (Q_hi + Q_lo) K^T
        if (lane == 0) {
          const uint32_t k = smem + L::kOffK + (tile % L::kKst) * L::kKV;
#pragma unroll
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
              mma_e4m3(tmem + t * kTile, desc_rows<D>(smem + (2 * t + part) * L::kQ + 32 * i), desc_rows<D>(k + 32 * i), id_qk,
                       (part | i) != 0);
          mma_commit(sfull(t));
          mma_commit(kempty(tile % L::kKst));
        }
        __syncwarp();
      };
      ok = wait(qfull(t), nq++ & 1) && wait(kfull(n % L::kKst), (n / L::kKst) & 1);
      if (!ok) break;
      tc_fence_after();
      scores(n);
      for (int j = u.j0; j < u.j1; ++j, ++n, ++np) {
        const int vb = n & 1;
        for (int half = 0; half < 2 && ok; ++half) {
          ok = wait(pfull(t, half), np & 1);
          if (ok && half == 0) ok = wait(cfull(vb), (n >> 1) & 1);
          if (!ok) break;
          tc_fence_after();
          if (lane == 0) {
            const uint32_t v = smem + L::kOffVc + vb * L::kVc;
#pragma unroll
            for (int i = 0; i < kTile / 32; ++i) {
              const int k = half * (kTile / 32) + i;
              mma_f16_ts(tmem + 2 * kTile + t * D, tmem + t * kTile + 8 * k, desc_cols(v + 2048 * k), id_pv, j > u.j0 || k > 0);
            }
          }
          __syncwarp();
        }
        if (!ok) break;
        if (lane == 0) {
          mma_commit(ofull(t));
          mma_commit(cempty(vb));
        }
        __syncwarp();
        if (j + 1 < u.j1) {   // the next scores take the place of these weights: wait until they have been read
          ok = wait(kfull((n + 1) % L::kKst), ((n + 1) / L::kKst) & 1) && wait(ofull(t), np & 1);
          if (!ok) break;
          tc_fence_after();
          scores(n + 1);
        }
      }
    } while (ok && next_unit(p, u));
    if (!ok && lane == 0) {   // let the tensor cores finish before TMEM is freed
      mma_commit(drained(t));
      drain_wait(drained(t), 0, p.status);
    }
    __syncwarp();
  } else if (warp >= 8 && warp < 12) {
    // ---- V: e4m3 to f16, a thread a token -----------------------------------------------------
    const int tok = tid - 256;
    int n = 0;
    bool ok = true;
    do {
      float vref = 0.f;
      for (int j = u.j0; j < u.j1 && ok; ++j, ++n) {
        const int vs = n % L::kVst, vb = n & 1;
        ok = wait(vfull(vs), (n / L::kVst) & 1);
        if (!ok) break;
        vref = next_vref(vref, sh.vs[n % kScaleSlots]);
        const float mine = sh.vs[n % kScaleSlots][tok / kPage];
        const float ratio = mine > 0.f ? mine / vref * 128.f : 0.f;
        const __half2 r2 = __float2half2_rn(ratio);
        const bool held = j * kTile + tok < u.len;   // a slot past the sequence may hold anything, NaN included
        const uint32_t from = smem + L::kOffV + vs * L::kKV + tok * D;
        uint32_t w[D / 4];
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          const uint32_t at = from + (D == 128 ? ((c ^ (tok & 7)) << 4) : ((c ^ ((tok >> 1) & 3)) << 4));
          asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(w[4 * c]), "=r"(w[4 * c + 1]), "=r"(w[4 * c + 2]), "=r"(w[4 * c + 3]) : "r"(at));
        }
        mbar_arrive(vempty(vs));
        ok = wait(cempty(vb), ((n >> 1) & 1) ^ 1);
        if (!ok) break;
        const uint32_t to = smem + L::kOffVc + vb * L::kVc + tok * 128;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {   // 8 features, 16 bytes
          uint32_t h[4];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t x = held ? w[2 * c + i] : 0u;
            const uint32_t a = q8::e4m3x2_to_f16x2((uint16_t)x), b = q8::e4m3x2_to_f16x2((uint16_t)(x >> 16));
            const __half2 fa = __hmul2(*reinterpret_cast<const __half2*>(&a), r2);
            const __half2 fb = __hmul2(*reinterpret_cast<const __half2*>(&b), r2);
            h[2 * i] = *reinterpret_cast<const uint32_t*>(&fa);
            h[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&fb);
          }
          const uint32_t at = to + (c / 8) * (kTile * 128) + (((c % 8) ^ (tok & 7)) << 4);
          asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]) : "memory");
        }
        fence_proxy_async_smem();
        mbar_arrive(cfull(vb));
      }
    } while (ok && next_unit(p, u));
  } else if (warp < 8) {
    // ---- softmax: a thread a row ----------------------------------------------------------------
    const int t = warp >> 2, row = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t S = tmem + lanes + t * kTile, O = tmem + lanes + 2 * kTile + t * D;
    int n = 0;                  // tiles of the share
    uint32_t ns = 0;            // of them, this Q tile's
    bool ok = true;
    int4 meta = make_int4(-1, 0, 0, 0);
    do {
      const bool begins = u.j0 == 0, ends = u.j1 == u.n_kv;
      if (begins && !ends) meta.x = u.s, meta.y = u.h, meta.w = u.rt;
      if (!begins) meta.z = ends ? 2 : 1;
      if (t >= active_tiles(p, u)) {
        n += u.j1 - u.j0;
        continue;
      }
      const int64_t col = (int64_t)u.rt * kPromptRows + t * kTile + row;   // (token, query head) pair
      const bool live = col < (int64_t)u.rows * p.g;
      const int tok = (int)(col / p.g);
      const int limit = live ? u.len - u.rows + tok + 1 : 0;               // tokens the row sees
      const int first_limit = u.len - u.rows + (int)(((int64_t)u.rt * kPromptRows + t * kTile) / p.g) + 1;
      const int64_t out_row = live ? (int64_t)(u.row0 + tok) * p.Hq + u.h * p.g + (int)(col % p.g) : 0;
      float c;   // scores times this are x, the exponent in base 2
      {
        // q / 2^(e - 7) = high + low, both e4m3; the scores of the unit before have all been computed
        const uint4* at = reinterpret_cast<const uint4*>(
            p.q + (live ? (u.row0 + tok) * p.q_stride + (int64_t)(u.h * p.g + (int)(col % p.g)) * D : 0));
        uint32_t top = 0;
        if (live)
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            const uint4 v = at[i];
            for (uint32_t x : {v.x, v.y, v.z, v.w}) top = max(top, max(x & 0x7fffu, (x >> 16) & 0x7fffu));
          }
        int e = (int)(top >> 7) - 127;
        if (e == 128 || top == 0) e = 0;
        e = min(max(e, -110), 126);
        const float down = __uint_as_float((uint32_t)(127 + 7 - e) << 23);
        c = p.scale * __uint_as_float((uint32_t)(127 - 7 + e) << 23);
        const uint32_t to = smem + 2 * t * L::kQ + row * D;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {   // 16 features
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint4 v = live ? at[2 * i + k] : make_uint4(0, 0, 0, 0);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              float f[4] = {bf_lo(w[2 * z]) * down, bf_hi(w[2 * z]) * down, bf_lo(w[2 * z + 1]) * down, bf_hi(w[2 * z + 1]) * down};
              const uint32_t h8 = q8::to_e4m3x4(f[0], f[1], f[2], f[3], 1.f);
              const uint32_t ha = q8::e4m3x2_to_f16x2((uint16_t)h8), hb = q8::e4m3x2_to_f16x2((uint16_t)(h8 >> 16));
              const float2 fa = __half22float2(*reinterpret_cast<const __half2*>(&ha));
              const float2 fb = __half22float2(*reinterpret_cast<const __half2*>(&hb));
              hi[2 * k + z] = h8;
              lo[2 * k + z] = q8::to_e4m3x4(f[0] - fa.x, f[1] - fa.y, f[2] - fb.x, f[3] - fb.y, 1.f);
            }
          }
          const uint32_t off = to + (D == 128 ? ((i ^ (row & 7)) << 4) : ((i ^ ((row >> 1) & 3)) << 4));
          asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(off), "r"(hi[0]), "r"(hi[1]), "r"(hi[2]), "r"(hi[3]) : "memory");
          asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(off + L::kQ), "r"(lo[0]), "r"(lo[1]), "r"(lo[2]), "r"(lo[3]) : "memory");
        }
        fence_proxy_async_smem();
        mbar_arrive(qfull(t));
      }
      float m = -INFINITY, l = 0.f, vref = 0.f;
      for (int j = u.j0; j < u.j1; ++j, ++n, ++ns) {
        ok = wait(sfull(t), ns & 1);
        if (!ok) break;
        tc_fence_after();
        const float* ks = sh.ks[n % kScaleSlots];
        const int seen = limit - j * kTile;   // columns below this are visible
        const bool masked = (j + 1) * kTile > first_limit;
        // Two passes over the row, 32 scores at a time, the next 32 on their way from TMEM meanwhile:
        // a row in registers would leave none for the rest.
        uint32_t r[2][32];
        auto fetch = [&](int b) { tmem_ld32(S + 32 * b, r[b & 1]); };
        auto hide = [&](int b) {
          if (masked) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (32 * b + i >= seen) asm volatile("mov.b32 %0, 0xff800000;" : "=r"(r[b & 1][i]));   // -inf
          }
        };
        float f[kPagesPerTile];
        float top = -INFINITY;
        fetch(0);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          tmem_wait_ld(r[b & 1]);
          fetch((b + 1) & 3);
          hide(b);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int q = 2 * b + h;
            f[q] = ks[q] * c;
            if (f[q] == 0.f) f[q] = 1.f;   // no scale: no page, or one of zeros; -inf stays -inf
            float a = __uint_as_float(r[b & 1][16 * h]);
#pragma unroll
            for (int i = 1; i < 16; ++i) a = fmaxf(a, __uint_as_float(r[b & 1][16 * h + i]));
            top = fmaxf(top, a * f[q]);
          }
        }
        const float nvref = next_vref(vref, sh.vs[n % kScaleSlots]);
        const bool grow = top > m + kLazy;
        float fix = 1.f;   // what the accumulator is multiplied with
        if (grow) {
          const float g = ex2(m - top);   // 0 at the first
          l *= g;
          fix = g;
          m = top;
        }
        if (nvref != vref) fix *= vref / nvref;
        vref = nvref;
        if (j > u.j0 && __any_sync(0xffffffffu, fix != 1.f)) {
          ok = wait(ofull(t), (ns - 1) & 1);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int b = 0; b < D / 16; ++b) {
            uint32_t o[16];
            tmem_ld16(O + 16 * b, o);
            tmem_wait_ld(o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * fix);
            tmem_st16(O + 16 * b, o);
          }
        }
        const float base = kShift - (m == -INFINITY ? 0.f : m);
        const uint64_t base2 = pair2(base, base);
        uint64_t sum2 = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          tmem_wait_ld(r[b & 1]);
          if (b < 3) fetch(b + 1);
          hide(b);
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float fq = f[2 * b + i / 8];
            const float2 x = unpair2(fma2(pair2(__uint_as_float(r[b & 1][2 * i]), __uint_as_float(r[b & 1][2 * i + 1])),
                                          pair2(fq, fq), base2));
            const float e0 = ex2(x.x), e1 = ex2(x.y);
            sum2 = add2(sum2, pair2(e0, e1));
            const __half2 h = __floats2half2_rn(e0, e1);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
          }
          tmem_st16(S + 16 * b, w);   // over scores that this thread has read
          if (b & 1) {
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(pfull(t, b / 2));
          }
        }
        const float2 sum = unpair2(sum2);
        l += sum.x + sum.y;
      }
      if (!ok) break;
      // ---- the part's result -----------------------------------------------------------------
      ok = wait(ofull(t), (ns - 1) & 1);
      if (!ok) break;
      tc_fence_after();
      l *= 0x1p-7f;   // 2^-kShift
      const float om = m + lg2(vref) - kVShift;   // the accumulator holds sums of 2^(x - om + 7) times v
      if (begins && ends) {
        const float f = l == 0.f ? 0.f : vref * 0x1p-14f / l;
#pragma unroll
        for (int b = 0; b < D / 32; ++b) {
          uint32_t r[32], w[16];
          tmem_ld32(O + 32 * b, r);
          tmem_wait_ld(r);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(r[2 * i]) * f, __uint_as_float(r[2 * i + 1]) * f);
            w[i] = *reinterpret_cast<const uint32_t*>(&v);
          }
          if (live)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              reinterpret_cast<uint4*>(p.out + out_row * D + 32 * b)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
        if (live && p.lse) p.lse[out_row] = (m + lg2(l)) * kLn2;
      } else {
        float* to = p.partial + ((int64_t)(blockIdx.x * 2 + (begins ? 1 : 0)) * p.cols + t * kTile + row) * (D + 4);
#pragma unroll
        for (int b = 0; b < D / 32; ++b) {
          uint32_t r[32];
          tmem_ld32(O + 32 * b, r);
          tmem_wait_ld(r);
          if (live)
#pragma unroll
            for (int i = 0; i < 8; ++i)
              reinterpret_cast<uint4*>(to + 32 * b)[i] = make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
        }
        if (live) *reinterpret_cast<float4*>(to + D) = make_float4(m, om, l, 0.f);
      }
      tc_fence_before();   // the accumulator is read before the next unit's first product
    } while (ok && next_unit(p, u));
    if (tid == 0) p.meta[blockIdx.x] = meta;
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 13) tmem_dealloc(tmem, 512);
  write_idle(p, D);
}

// A warp a row of a unit that more than one CTA held: block (i, y) takes rows y * 16 .. of the
// unit that begins in CTA i.
constexpr int kCombineWarps = 4, kCombineRows = 16;
template <int D>
__global__ void __launch_bounds__(32 * kCombineWarps) prompt_combine_kernel(const __grid_constant__ Params p) {
  constexpr int V = D / 32;   // values a lane
  __shared__ int last;
  pdl_wait();
  pdl_launch_dependents();
  const int i = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
  const int4 mt = p.meta[i];
  if (mt.x < 0) return;
  int row0, rows, len;
  sequence(p.seqs, mt.x, row0, rows, len);
  const int64_t col0 = (int64_t)mt.w * kPromptRows + blockIdx.y * kCombineRows, cols = (int64_t)rows * p.g;
  if (col0 >= cols) return;
  if (tid == 0) last = 0x7fffffff;
  __syncthreads();
  for (int j0 = i + 1; j0 < p.n_cta; j0 += 32 * kCombineWarps) {   // the CTA that ends the unit
    const int j = j0 + tid;
    if (j < p.n_cta && p.meta[j].z == 2) atomicMin(&last, j);
    __syncthreads();
    if (last != 0x7fffffff) break;
    __syncthreads();
  }
  const int n = min(last, p.n_cta - 1) - i + 1;
  for (int k = tid >> 5; k < kCombineRows; k += kCombineWarps) {
    const int64_t col = col0 + k;
    if (col >= cols) break;
    auto entry = [&](int x) {
      return p.partial + ((int64_t)((i + x) * 2 + (x == 0 ? 1 : 0)) * p.cols + blockIdx.y * kCombineRows + k) * (D + 4);
    };
    float m = -INFINITY, om = -INFINITY;
    for (int x = lane; x < n; x += 32) {
      const float4 s = *reinterpret_cast<const float4*>(entry(x) + D);
      m = fmaxf(m, s.x);
      om = fmaxf(om, s.y);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      om = fmaxf(om, __shfl_xor_sync(0xffffffffu, om, o));
    }
    float acc[V], l = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.f;
#pragma unroll 4
    for (int x = 0; x < n; ++x) {
      const float* e = entry(x);
      const float4 s = *reinterpret_cast<const float4*>(e + D);
      const float w = om == -INFINITY ? 0.f : ex2(s.y - om);
      l += m == -INFINITY ? 0.f : s.z * ex2(s.x - m);
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] = fmaf(e[lane * V + v], w, acc[v]);
    }
    const float r = l == 0.f ? 0.f : ex2(om - m - kShift) / l;
    const int64_t row = (row0 + col / p.g) * p.Hq + mt.y * p.g + col % p.g;
#pragma unroll
    for (int v = 0; v < V; v += 2) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(acc[v] * r, acc[v + 1] * r);
      *reinterpret_cast<uint32_t*>(p.out + row * D + lane * V + v) = *reinterpret_cast<const uint32_t*>(&b);
    }
    if (p.lse && lane == 0) p.lse[row] = (m + lg2(l)) * kLn2;
  }
}

template <int D>
cudaError_t launch(const CUtensorMap& kmap, const CUtensorMap& vmap, const Params& p, cudaStream_t stream) {
  cudaError_t e = cudaFuncSetAttribute(prompt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Prompt<D>::kSmem);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(p.n_cta);
  cfg.blockDim = dim3(kThreadsAll);
  cfg.dynamicSmemBytes = Prompt<D>::kSmem;
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, prompt_kernel<D>, kmap, vmap, p);
  cfg.gridDim = dim3(p.n_cta, kPromptRows / kCombineRows);
  cfg.blockDim = dim3(32 * kCombineWarps);
  cfg.dynamicSmemBytes = 0;
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, prompt_combine_kernel<D>, p);
  return e;
}

}  // namespace

cudaError_t launch_prompt(const CUtensorMap& kmap, const CUtensorMap& vmap, const Params& p, int head_dim, cudaStream_t stream) {
  return head_dim == 64 ? launch<64>(kmap, vmap, p, stream) : launch<128>(kmap, vmap, p, stream);
}

}  // namespace attend_q8
}  // namespace kvrp
