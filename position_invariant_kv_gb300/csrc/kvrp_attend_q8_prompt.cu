// Attention of many rows over the 8-bit paged cache (kv_attend_q8 on prompts).
//
//   out[r][j] = softmax(scale q[r][j] . K) V, causal; K_t = ks[page] K8_t, V_t = vs[page] V8_t.
//
// Bound by the tensor cores: 4 head_dim operations for each (row, head, visible token).
//   - A unit is 256 rows of one (sequence, KV head): the rows x group pairs (token, query
//     head) in order, so every row of the tile is used whatever the group, and K and V are
//     loaded once for all query heads that share them.  It runs over its visible tokens in
//     tiles of 80 (head_dim 128) or 128 (64).  The list of (unit, token tile) is cut into equal
//     contiguous shares, one a CTA, on the device; a unit that several CTAs share goes through
//     the combine.
//   - S = Q K^T by tcgen05 kind::f8f6f4: K goes from memory to the tensor cores as stored.
//     q is split into two e4m3 parts, high and low, after its row was divided by a power of
//     two: bf16's 8 significant bits are 4 + 4, so the parts are q exactly down to 2^-9 of
//     the row's largest element and off by at most 2^-17 of it below.  Two products at
//     twice the f16 rate cost what one would, without converting K.
//   - O += P V by kind::f16: P as f16 from TMEM, V as f16 in shared memory, converted from e4m3
//     by four warps together with the page's scale relative to a running reference (a power
//     of two), exact for powers of two within 2^12 of it.  From the first tile on whose scales lie
//     farther apart, a unit's part has V unscaled and the scales in the weights' exponent, with a
//     running maximum of x + log2 vs for the accumulator beside that of x for the sum.  The weights
//     are rounded to f16, 2^-11 of each at most, and summed before that in fp32: the output, rounded to
//     bf16, is 1.7e-3 from the 64-bit result with them as with fp32 weights, and a second, low part
//     would double the second product.
//   - Two 128-row Q tiles a CTA, each with its own softmax warps (a thread a row) and its own
//     MMA issuer.  TMEM holds for each the accumulator, the scores and, apart from them, the
//     weights: the next tile's scores are formed while this one's are being turned into
//     weights.  That is why a token tile is 80 at head_dim 128: 80 columns of scores + 40 of
//     weights + 128 of accumulator, twice, are what 512 columns hold.  (With 128 tokens and
//     the weights in the scores' place each tile waited for both products: 911 TFLOP/s on
//     4096 rows over 16441 tokens.)
//
// Measured: 4096 rows over 16441 tokens, 28 / 4 heads x 128: 688 us, 1229 TFLOP/s, 63% of the measured
// bf16 peak; 6 questions of 37 to 900 rows behind 500 to 12000 tokens: 215 us, 1038 TFLOP/s.  The same
// with 32 / 8 heads x 64: 667 and 215 us, 724 and 591 TFLOP/s.  With value scales spread over 2^30: 1626
// and 468 us (head_dim 128).  A tile takes about 2300 cycles, its products alone 1500: the softmax warps
// wait some 800 of them for products, which share the 128 bytes a cycle of shared memory with the
// conversion of V (two thirds busy).  What is in the way of the next scores costs at once: instructions
// between a tile's scores and their release, and in the warp that loads (70 more a tile: 60 us of 690).
// Beginning and ending a unit costs about 7 us.
#include <cudaTypedefs.h>

#include <algorithm>

#include "kvrp_attend_q8.h"
#include "kvrp_plan.h"

namespace kvrp {

kvrp_status encode_q8_pool(CUtensorMap* map, const void* pool, int num_pages, int row_bytes, int head_dim) {
  // found once: the driver's entry point does not change while the library is loaded
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    cudaDriverEntryPointQueryResult q;
    void* fn = nullptr;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
    return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn) : nullptr;
  }();
  if (!encode) return fail(KVRP_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const cuuint64_t dims[3] = {(cuuint64_t)row_bytes, 16, (cuuint64_t)num_pages};
  const cuuint64_t strides[2] = {(cuuint64_t)row_bytes, (cuuint64_t)row_bytes * 16};
  const cuuint32_t box[3] = {(cuuint32_t)head_dim, 16, 1}, estr[3] = {1, 1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(pool), dims, strides, box, estr,
                            CU_TENSOR_MAP_INTERLEAVE_NONE,
                            head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                            // a wider fetch would bring in the next head's rows, which another CTA reads
                            head_dim == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_64B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(KVRP_ERR_INVALID_ARG, "cuTensorMapEncodeTiled failed (%d) for an 8-bit pool", (int)r);
  return KVRP_OK;
}

namespace attend_q8 {

namespace {

constexpr int kRows = 128;                 // rows of a Q tile
constexpr int kWarpsAll = 16, kThreadsAll = 32 * kWarpsAll;
constexpr int kWarpsRows = 8, kMostFeatures = 128;   // the softmax warps; head_dim at most
constexpr int kScaleSlots = 8;             // tiles whose scales are kept
constexpr int kMostPages = 8;              // pages of a token tile
constexpr uint32_t kNoRow = 0xffffffffu;   // a row of the tile that no query fills
constexpr float kVShift = 7.f;             // V enters as v * vs * 2^7 / vref: up to 448 * 128 in f16
// With a reference, a value scale is at least kNear of it, so that its products with e4m3 values (multiples of 2^-9)
// and 2^7 are f16's normal numbers; and the part's first reference at least kReach of it.
constexpr float kNear = 0x1p-12f, kReach = 0x1p-48f;

template <int D>
struct Prompt {
  static constexpr int kN = D == 128 ? 80 : 128;   // tokens of a tile
  static constexpr int kP = kN / kPage;            // its pages
  static constexpr int kP0 = (kP + 1) / 2;         // the pages whose weights are handed over first
  static constexpr int kQ = kRows * D;             // bytes of one e4m3 part of a Q tile
  static constexpr int kKV = kN * D;               // bytes of a raw K or V tile
  static constexpr int kKst = 4, kVst = 3, kCst = 3;   // stages of K, of raw and of converted V
  static constexpr int kVc = kN * D * 2;           // bytes of a converted V tile
  // TMEM columns of Q tile t: scores, weights (two a column), accumulator
  static __host__ __device__ constexpr int tmem_s(int t) { return t * 128; }
  static __host__ __device__ constexpr int tmem_p(int t) { return D == 128 ? t * 128 + 80 : 256 + t * 64; }
  static __host__ __device__ constexpr int tmem_o(int t) { return D == 128 ? 256 + t * 128 : 384 + t * 64; }
  // Registers a thread of the softmax (which holds a row of scores), V and other warps: the
  // 4 x 128 that the warp groups were launched with, shared out anew.  head_dim 64, 128 scores a row:
  // 184 / 88 / 56 spill 600 bytes a thread and take 757 us for 4096 rows over 16441 tokens, 192 / 80 / 48
  // 704, 200 / 64 / 48 (384 bytes) 657, 200 / 56 / 56 662.
  static constexpr int kRegsRow = D == 128 ? 168 : 200, kRegsV = D == 128 ? 88 : 64, kRegsMisc = D == 128 ? 88 : 48;
  static_assert(2 * kRegsRow + kRegsV + kRegsMisc <= 4 * 128, "more registers than the block holds");
  static constexpr int kOffK = 4 * kQ, kOffV = kOffK + kKst * kKV, kOffVc = kOffV + kVst * kKV;
  static constexpr int kSmem = 1024 + kOffVc + kCst * kVc;
  static_assert(kSmem <= 227 * 1024 - 8192, "shared memory");
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
template <int N>
__device__ __forceinline__ uint64_t desc_cols(uint32_t addr) {
  uint64_t d = (uint64_t)((addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(N * 128 >> 4) << 16;               // next 64 columns
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
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
// Whether a phase has completed, without waiting.
__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}
// Two f16 values to e4m3 (NaN stays NaN; nothing here is above 448).
__device__ __forceinline__ uint16_t f16x2_to_e4m3x2(uint32_t v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(v));
  return r;
}
// A value that is the same in all lanes, and known to be.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }
// True in one lane, the same one each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{.reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p;}" : "=r"(r));
  return r != 0;
}
template <int N>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
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
// Beginning and ending a unit (its queries, the first scores, the results) takes a CTA as long as some
// tiles do; the shares count that, or the CTAs of a batch's many short units finish last.
constexpr int kUnitTiles = 6;   // 4: 222 us for the 6 questions above, 6: 220 (215 with a later step)

// A unit's part inside this CTA's share: tiles [j0, j1) of its n_kv.
struct Unit {
  int s, rt, h;             // sequence, row tile, KV head
  int row0, rows, len;      // the sequence
  int n_rt, n_kv, j0, j1;
  int from, spent;          // this part's costs [from, from + spent) of its unit
  int64_t left;             // cost of the share from here on
};
template <int N>
__device__ __forceinline__ int tiles_of(int row0_col, int g, int rows, int len) {   // token tiles of a row tile
  const int last = min(rows - 1, (row0_col + kPromptRows - 1) / g);                 // its last token among the rows
  return (len - rows + last + N) / N;
}
__device__ __forceinline__ bool load_seq(const Params& p, int s, Unit& u, bool tell = false) {
  const bool ok = sequence(p.seqs, s, u.row0, u.rows, u.len) && u.rows <= p.max_rows;
  if (tell && !ok) flag(p.status, KVRP_DEV_BAD_LENGTH);
  u.n_rt = ok ? (int)(((int64_t)u.rows * p.g + kPromptRows - 1) / kPromptRows) : 0;
  return u.n_rt > 0;
}
// The cost of sequence s over all its row tiles, by one warp (one head's worth).
template <int N>
__device__ __forceinline__ int64_t seq_cost(const Params& p, int s, bool tell) {
  Unit u;
  int64_t sum = 0;
  if (load_seq(p, s, u, tell && (threadIdx.x & 31) == 0))
    for (int rt = threadIdx.x & 31; rt < u.n_rt; rt += 32) sum += kUnitTiles + tiles_of<N>(rt * kPromptRows, p.g, u.rows, u.len);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}
// The unit's tiles among the costs [from, from + left): its first kUnitTiles stand for beginning and ending it.
__device__ __forceinline__ void take(Unit& u, int from) {
  const int to = (int)min((int64_t)u.n_kv + kUnitTiles, from + u.left);
  u.j0 = max(0, from - kUnitTiles);
  u.j1 = max(0, to - kUnitTiles);
  u.from = from;
  u.spent = to - from;
}
struct Shared {
  __align__(8) uint64_t bars[40];
  __align__(16) float ks[kScaleSlots][kMostPages];   // a tile's scales of K,
  float vs[kScaleSlots][kMostPages];                 // of V,
  float vref[kScaleSlots];                           // and the reference of V's, 0 from where they lie apart
  int64_t cost[kWarpsAll];
  int64_t total, end;     // the cost in all, and where this CTA's share ends
  int n_cta;
  Unit first;
  int found;
  int abort_flag;
  int later_nan;          // a value taken out of a product because not all rows of its unit see it was NaN
  int nan_at[kWarpsRows][kMostFeatures];   // then: the first token with one, by features, a softmax warp's unit
  uint32_t tmem;
};
template <int N>
__device__ __forceinline__ bool find_share(const Params& p, Shared& sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = p.seqs.n_seqs;
  int64_t mine = 0;
  for (int s = warp; s < n; s += kWarpsAll) mine += seq_cost<N>(p, s, blockIdx.x == 0) * p.Hkv;
  if (lane == 0) sh.cost[warp] = mine;
  __syncthreads();
  int64_t total = 0;
  for (int w = 0; w < kWarpsAll; ++w) total += sh.cost[w];
  const int64_t n_cta = min((int64_t)p.n_cta, (total + kUnitTiles + 1) / (kUnitTiles + 2));
  if ((int)blockIdx.x >= n_cta) return false;
  const int64_t a = total * blockIdx.x / n_cta, b = total * (blockIdx.x + 1) / n_cta;
  if (threadIdx.x == 0) {
    sh.total = total;
    sh.end = b;
    sh.n_cta = (int)n_cta;
  }
  int64_t before = 0;
  int s = 0;
  for (int s0 = 0; s0 < n; s0 += kWarpsAll) {   // the sequence that holds tile a
    __syncthreads();
    const int64_t c = s0 + warp < n ? seq_cost<N>(p, s0 + warp, false) * p.Hkv : 0;
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
      const int t = rt < u.n_rt ? tiles_of<N>(rt * kPromptRows, p.g, u.rows, u.len) : -kUnitTiles;
      const int cost = t + kUnitTiles;
      int64_t sum = (int64_t)cost * p.Hkv;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
      }
      const int64_t lo = sum - (int64_t)cost * p.Hkv;
      if (at >= lo && at < sum) {
        u.s = s;
        u.rt = rt;
        u.n_kv = t;
        u.h = (int)((at - lo) / cost);
        u.left = b - a;
        take(u, (int)((at - lo) % cost));
        sh.first = u;
      }
      at -= __shfl_sync(0xffffffffu, sum, 31);
      if (at < 0) break;
    }
  }
  __syncthreads();
  return sh.first.j1 > sh.first.j0 || sh.first.left > sh.first.spent;
}
// The share's next unit; false at its end.
template <int N>
__device__ __forceinline__ bool next_unit(const Params& p, Unit& u) {
  u.left -= u.spent;
  if (u.left <= 0) return false;
  if (++u.h == p.Hkv) {
    u.h = 0;
    if (++u.rt == u.n_rt) {
      u.rt = 0;
      do ++u.s;
      while (!load_seq(p, u.s, u));
    }
    u.n_kv = tiles_of<N>(u.rt * kPromptRows, p.g, u.rows, u.len);
  }
  take(u, 0);
  return u.j1 > 0;
}
__device__ __forceinline__ int active_tiles(const Params& p, const Unit& u) {   // Q tiles with rows in them
  return (int64_t)u.rows * p.g - (int64_t)u.rt * kPromptRows > kRows ? 2 : 1;
}
// x / g for 0 <= x < 2^28 (the host keeps rows x group below): by a product with 2^32 / g, rounded up.
__device__ __forceinline__ int over_group(const Params& p, int x) { return (int)((uint64_t)(uint32_t)x * p.g_inverse >> 32); }
// Tokens below this are seen by all rows of the unit.
__device__ __forceinline__ int seen_by_all(const Params& p, const Unit& u) {
  return u.len - u.rows + over_group(p, u.rt * kPromptRows) + 1;
}
// The reference of the value scales after a tile: a power of two at least the largest scale,
// two octaves above it when it moves, so that it moves seldom.
__device__ __forceinline__ float next_vref(float vref, float top) {
  if (!(top > vref)) return vref;
  const uint32_t e = (__float_as_uint(top) + 0x7fffffu) >> 23;   // 2^ceil(log2 top)
  return __uint_as_float(min(e + 2u, 254u) << 23);
}

// The first of the tokens [from, to) of sequence s whose value is NaN, for each feature of KV head h (INT32_MAX:
// none), by a warp.  Reads the values again; a cache without such values never comes here.
template <int D>
__device__ __noinline__ void find_later_nan(const Params& p, int s, int h, int from, int to, int* at) {
  constexpr int kEach = D / 32;
  const int lane = threadIdx.x & 31;
  int first[kEach];
#pragma unroll
  for (int e = 0; e < kEach; ++e) first[e] = INT32_MAX;
  for (int t = to - 1; t >= from; --t) {
    const int page = p.seqs.block_tables[(int64_t)s * p.seqs.table_stride + t / kPage];
    if (page < 0 || page >= p.seqs.num_pages) continue;
    const uint8_t* v = p.v_pool + (((int64_t)page * kPage + t % kPage) * p.Hkv + h) * D + lane * kEach;
#pragma unroll
    for (int e = 0; e < kEach; ++e)
      if ((v[e] & 0x7f) == 0x7f) first[e] = t;
  }
  __syncwarp();
#pragma unroll
  for (int e = 0; e < kEach; ++e) at[lane * kEach + e] = first[e];
  __syncwarp();
}

template <int D>
__global__ void __launch_bounds__(kThreadsAll, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                  const __grid_constant__ Params p) {
  using L = Prompt<D>;
  constexpr int N = L::kN;
  extern __shared__ uint8_t raw_smem[];
  __shared__ Shared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t smem = (smem_u32(raw_smem) + 1023u) & ~1023u;
  const uint32_t bar0 = smem_u32(sh.bars);
  auto kfull = [&](int i) { return bar0 + 8u * i; };
  auto kempty = [&](int i) { return bar0 + 8u * (4 + i); };
  auto vfull = [&](int i) { return bar0 + 8u * (8 + i); };
  auto vempty = [&](int i) { return bar0 + 8u * (11 + i); };
  auto cfull = [&](int i) { return bar0 + 8u * (14 + i); };    // converted V
  auto cempty = [&](int i) { return bar0 + 8u * (17 + i); };
  auto qfull = [&](int t) { return bar0 + 8u * (20 + t); };
  auto sfull = [&](int t) { return bar0 + 8u * (22 + t); };    // scores in TMEM
  auto sread = [&](int t) { return bar0 + 8u * (24 + t); };    // scores read, their place is free
  auto pfull = [&](int t, int half) { return bar0 + 8u * (26 + 2 * t + half); };   // weights in TMEM, accumulator corrected
  auto ofull = [&](int t) { return bar0 + 8u * (30 + t); };    // accumulator updated, the weights' place is free
  auto pread = [&](int t) { return bar0 + 8u * (32 + t); };    // the first part of the weights read
  auto drained = [&](int t) { return bar0 + 8u * (34 + t); };
  if (tid == 0) {
    for (int i = 0; i < L::kKst; ++i) mbar_init(kfull(i), 1), mbar_init(kempty(i), 2);   // both Q tiles
    for (int i = 0; i < L::kVst; ++i) mbar_init(vfull(i), 1), mbar_init(vempty(i), 128);
    for (int i = 0; i < L::kCst; ++i) mbar_init(cfull(i), 128), mbar_init(cempty(i), 2);
    for (int t = 0; t < 2; ++t) {
      mbar_init(qfull(t), 128);
      mbar_init(sfull(t), 1);
      mbar_init(sread(t), 128);
      mbar_init(pfull(t, 0), 128);
      mbar_init(pfull(t, 1), 128);
      mbar_init(ofull(t), 1);
      mbar_init(pread(t), 1);
      mbar_init(drained(t), 1);
    }
    sh.abort_flag = 0;
    sh.later_nan = 0;
    mbar_init_fence();
  }
  if (warp == 13) tmem_alloc(smem_u32(&sh.tmem), 512);
  if (tid == 32) {
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
  }
  pdl_wait();
  pdl_launch_dependents();
  const bool any = find_share<N>(p, sh);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  volatile int* abort_p = &sh.abort_flag;
  auto wait = [&](uint32_t bar, uint32_t parity) {   // bounded; the same answer in the whole warp
    bool ok = mbar_test_wait(bar, parity);
    if (!__all_sync(0xffffffffu, ok)) {
      const long long t0 = clock64();
      while (!ok && !*abort_p) {
        if (clock64() - t0 > p.wait_cycles) {
          *abort_p = 1;
          flag(p.status, KVRP_DEV_TIMEOUT);
          break;
        }
        ok = mbar_try_wait(bar, parity);
      }
    }
    return __all_sync(0xffffffffu, ok) != 0;
  };
  Unit u = sh.first;

  if (!any) {
    if (tid == 0) p.meta[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
  } else if (warp >= 12) {
    fewer_registers<L::kRegsMisc>();
    if (warp == 12) {
      // ---- TMA: a lane a page ---------------------------------------------------------------
      int n = 0, nk = 0, nv = 0;   // the tile, K and V tiles issued
      bool ok = true;
      do {
        const int pages = (u.len + kPage - 1) / kPage;
        // The reference of the value scales; none from a tile on whose scales lie too far apart for it, or from where
        // it is too far from the first one for the accumulator that began relative to that.
        float vref = 0.f, first_vref = 0.f;
        bool apart = false;
        for (int j = u.j0; j < u.j1 && ok; ++j, ++n) {
          const int ks = n % L::kKst, vs = n % L::kVst, slot = n % kScaleSlots;
          const int pg = j * L::kP + lane;
          const bool mine = lane < L::kP && pg < pages;
          int page = p.seqs.num_pages;   // past the pool: the box reads zeros
          float fk = 0.f, fv = mine ? kZeroBlock : 0.f;
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
          // Both issuers have done tile n - 4's scores, so both softmax groups have read tile n - 5's, and
          // V's warps are past tile n - 5: nobody needs slot n - 8 any more.
          if (lane < kMostPages) {
            sh.ks[slot][lane] = fk;
            sh.vs[slot][lane] = fv;
          }
          // positive numbers are in the order of their bits
          const uint32_t least = __reduce_min_sync(0xffffffffu, mine ? __float_as_uint(fv) : 0x7f7fffffu);
          const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(fv));
          const float next = next_vref(vref, __uint_as_float(most));
          if (j == u.j0) first_vref = next;
          apart |= __uint_as_float(least) < next * kNear || first_vref < next * kReach;
          vref = next;
          if (lane == 0) sh.vref[slot] = apart ? 0.f : next;
          const uint32_t bytes = (uint32_t)min(L::kP, pages - j * L::kP) * kPage * D;
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
      } while (ok && next_unit<N>(p, u));
      if (!ok && lane == 0) {   // every issued copy lands before the CTA exits
        for (int i = max(0, nk - L::kKst); i < nk; ++i) drain_wait(kfull(i % L::kKst), (i / L::kKst) & 1, p.status);
        for (int i = max(0, nv - L::kVst); i < nv; ++i) drain_wait(vfull(i % L::kVst), (i / L::kVst) & 1, p.status);
      }
    } else if (warp < 15) {
      // ---- MMA: a warp a Q tile, so that one tile's waits leave the tensor cores to the other ----
      // What the products take has to be the same in the whole warp, and to be seen to be.
      const int t = (int)uniform(warp - 13);
      const uint32_t s_tmem = uniform(tmem + L::tmem_s(t)), o_tmem = uniform(tmem + L::tmem_o(t)), p_tmem = uniform(tmem + L::tmem_p(t));
      const uint64_t qd = desc_rows<D>(uniform(smem + 2 * t * L::kQ));   // an address is its low bits, in units of 16 bytes
      // descriptor: fp32 accumulator, M = 128; e4m3 (0) or f16 (0) operands; the second product's B is N-major
      const uint32_t id_qk = (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
      const uint32_t id_pv = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
      int n = 0;                   // tiles begun
      uint32_t nq = 0, np = 0;     // units begun and tiles weighted, of this Q tile
      bool ok = true;
      auto scores = [&](int tile) {   // S_t = (Q_hi + Q_lo) K^T
        const uint64_t kd = desc_rows<D>(uniform(smem + L::kOffK + (tile % L::kKst) * L::kKV));
        if (elect_one()) {
#pragma unroll
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
              mma_e4m3(s_tmem, qd + (part * L::kQ + 32 * i) / 16, kd + 2 * i, id_qk, (part | i) != 0);
          mma_commit(sfull(t));
          mma_commit(kempty(tile % L::kKst));
        }
        __syncwarp();
      };
      auto values = [&](int tile, int from, int to, uint32_t more) {   // O_t += P_t V, pages [from, to) of the tile
        const uint64_t vd = desc_cols<N>(uniform(smem + L::kOffVc + (tile % L::kCst) * L::kVc));
        if (elect_one()) {
#pragma unroll
          for (int i = from; i < to; ++i) mma_f16_ts(o_tmem, p_tmem + 8 * i, vd + 128 * i, id_pv, i > 0 ? 1u : more);
          if (to == L::kP) {
            mma_commit(ofull(t));
            mma_commit(cempty(tile % L::kCst));
          } else {
            mma_commit(pread(t));
          }
        }
        __syncwarp();
      };
      do {
        if (t >= active_tiles(p, u)) {   // no rows: the stages pass by, every phase observed (a wait tests a parity only)
          for (int j = u.j0; j < u.j1 && ok; ++j, ++n) {
            ok = wait(kfull(n % L::kKst), (n / L::kKst) & 1);
            if (ok && lane == 0) mbar_arrive(kempty(n % L::kKst));
            ok = ok && wait(cfull(n % L::kCst), (n / L::kCst) & 1);
            if (ok && lane == 0) mbar_arrive(cempty(n % L::kCst));
            __syncwarp();
          }
          continue;
        }
        ok = wait(qfull(t), nq++ & 1) && wait(kfull(n % L::kKst), (n / L::kKst) & 1);
        if (!ok) break;
        tc_fence_after();
        scores(n);
        for (int j = u.j0; j < u.j1; ++j, ++n, ++np) {
          ok = wait(sread(t), np & 1);
          if (ok && j + 1 < u.j1) {   // the next scores, while these are being weighted
            ok = wait(kfull((n + 1) % L::kKst), ((n + 1) / L::kKst) & 1);
            if (!ok) break;
            tc_fence_after();
            scores(n + 1);
          }
          ok = ok && wait(pfull(t, 0), np & 1) && wait(cfull(n % L::kCst), (n / L::kCst) & 1);
          if (!ok) break;
          tc_fence_after();
          const uint32_t more = uniform(j > u.j0);
          values(n, 0, L::kP0, more);
          ok = wait(pfull(t, 1), np & 1);
          if (!ok) break;
          tc_fence_after();
          values(n, L::kP0, L::kP, 1);
        }
      } while (ok && next_unit<N>(p, u));
      if (!ok && elect_one()) {   // let the tensor cores finish before TMEM is freed
        mma_commit(drained(t));
        drain_wait(drained(t), 0, p.status);
      }
      __syncwarp();
    }
  } else if (warp >= 8) {
    fewer_registers<L::kRegsV>();
    // ---- V: e4m3 to f16, 16 features of a token at a time ---------------------------------------
    constexpr int kChunks = D / 16, kEach = N * kChunks / 128;
    // Thread x takes chunks x, x + 128, ...: four chunks of two tokens to 8 threads, whose stores (every
    // other 16-byte column of a token's row, swizzled by its lowest bits) then touch all banks.
    const int x0 = tid - 256;
    const int tok0 = D == 128 ? (x0 >> 4) * 2 + ((x0 >> 2) & 1) : x0 >> 2;
    const int c = D == 128 ? (x0 & 3) | ((x0 >> 1) & 4) : x0 & 3;
    constexpr int kHop = 128 / kChunks;   // tokens between a thread's chunks: a multiple of 16
    int n = 0;
    bool ok = true;
    do {
      const int seen_all = seen_by_all(p, u);
      for (int j = u.j0; j < u.j1 && ok; ++j, ++n) {
        const int vs = n % L::kVst, vb = n % L::kCst, slot = n % kScaleSlots;
        ok = wait(vfull(vs), (n / L::kVst) & 1);
        if (!ok) break;
        const float vref = sh.vref[slot];
        const int held = u.len - j * N;   // a slot past the sequence may hold anything, NaN included
        // A scale enters relative to vref before the 2^7 does: 2^7 / vref alone passes fp32's range where all
        // of a tile's blocks are zeros (scale 2^-126).
        const float inv = vref > 0.f ? 1.f / vref : 0.f;
        const uint32_t from = smem + L::kOffV + vs * L::kKV;
        uint4 w[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          const int tok = tok0 + kHop * i;
          const uint32_t at = from + tok * D + (D == 128 ? ((c ^ (tok & 7)) << 4) : ((c ^ ((tok >> 1) & 3)) << 4));
          asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w) : "r"(at));
          if (__builtin_expect(tok >= held, 0)) {
            make_zero(w[i].x);
            make_zero(w[i].y);
            make_zero(w[i].z);
            make_zero(w[i].w);
          }
        }
        const int from_tok = seen_all - j * N;
        if (__builtin_expect(from_tok < N, 0)) {
          // A NaN of a token that not all rows see: weight 0 would not keep it from the others' sums.  It is
          // taken out, and the softmax warps put it into the rows that do see the token.
          bool odd = false;
#pragma unroll
          for (int i = 0; i < kEach; ++i) {
            if (tok0 + kHop * i < from_tok) continue;
            uint32_t* const x[4] = {&w[i].x, &w[i].y, &w[i].z, &w[i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t nan = q8::nan_bytes(*x[e]);
              odd |= nan != 0;
              *x[e] &= ~((nan >> 7) * 0xffu);
            }
          }
          if (odd) *static_cast<volatile int*>(&sh.later_nan) = 1;
        }
        mbar_arrive(vempty(vs));
        ok = wait(cempty(vb), ((n / L::kCst) & 1) ^ 1);
        if (!ok) break;
        const uint32_t to = smem + L::kOffVc + vb * L::kVc;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          const int tok = tok0 + kHop * i;
          const __half2 r2 = __float2half2_rn(vref > 0.f ? sh.vs[slot][tok / kPage] * inv * 128.f : 128.f);
          const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
          const uint32_t row = to + (c / 4) * (N * 128) + tok * 128;   // of the 64-column block c / 4
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t h[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t v = x[2 * half + e];
              const uint32_t a = q8::e4m3x2_to_f16x2((uint16_t)v), b = q8::e4m3x2_to_f16x2((uint16_t)(v >> 16));
              const __half2 fa = __hmul2(*reinterpret_cast<const __half2*>(&a), r2);
              const __half2 fb = __hmul2(*reinterpret_cast<const __half2*>(&b), r2);
              h[2 * e] = *reinterpret_cast<const uint32_t*>(&fa);
              h[2 * e + 1] = *reinterpret_cast<const uint32_t*>(&fb);
            }
            const uint32_t at = row + (((2 * (c % 4) + half) ^ (tok & 7)) << 4);
            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]) : "memory");
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(cfull(vb));
      }
    } while (ok && next_unit<N>(p, u));
  } else {
    more_registers<L::kRegsRow>();
    // ---- softmax: a thread a row ----------------------------------------------------------------
    const int t = warp >> 2, row = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t S = tmem + lanes + L::tmem_s(t), O = tmem + lanes + L::tmem_o(t), P = tmem + lanes + L::tmem_p(t);
    int n = 0;                  // tiles of the share
    uint32_t ns = 0;            // of them, this Q tile's
    bool ok = true;
    int4 meta = make_int4(0, 0, 0, 0);   // of a unit that begins here and goes on: parts, KV head, row tile, first row
    int meta_cols = 0;                   // and (row, query head) pairs of its sequence
    // Where 16-byte chunk x of row r is in part 0 (high) or 1 (low) of this Q tile; between units the
    // two rows of a thread's row are where its results are laid out for whole-row stores.
    auto row_chunk = [&](int part, int r, int x) {
      return smem + (2 * t + part) * L::kQ + r * D + (D == 128 ? ((x ^ (r & 7)) << 4) : ((x ^ ((r >> 1) & 3)) << 4));
    };
    auto scale_accumulator = [&](float fix) {
#pragma unroll
      for (int b = 0; b < D / 16; ++b) {
        uint32_t o[16];
        tmem_ld16(O + 16 * b, o);
        tmem_wait_ld(o);
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * fix);
        tmem_st16(O + 16 * b, o);
      }
    };
    do {
      const bool begins = u.j0 == 0, ends = u.j1 == u.n_kv;
      if (begins && !ends && tid == 0) {
        // the CTA whose share holds the unit's last tile: the largest j with total j / n_cta below the unit's end
        const int64_t unit_end = sh.end - u.left - u.from + u.n_kv + kUnitTiles;
        meta = make_int4((int)((unit_end * sh.n_cta - 1) / sh.total) - (int)blockIdx.x + 1, u.h, u.rt, u.row0);
        meta_cols = u.rows * p.g;
      }
      if (t >= active_tiles(p, u)) {
        n += u.j1 - u.j0;
        continue;
      }
      const int col = u.rt * kPromptRows + t * kRows + row;   // (token, query head) pair: below 2^31, n_rows x group is
      const bool live = col < u.rows * p.g;
      const int tok = over_group(p, col);
      const int limit = live ? u.len - u.rows + tok + 1 : 0;               // tokens the row sees
      const int first_limit = u.len - u.rows + over_group(p, u.rt * kPromptRows + t * kRows) + 1;
      const uint32_t out_row = live ? (uint32_t)(u.row0 + tok) * p.Hq + u.h * p.g + (col - tok * p.g) : kNoRow;
      // ---- q / 2^(e - 7) = high + low, both e4m3 -------------------------------------------------
      // A warp its 32 rows, D / 16 lanes a row, so that a load takes whole rows (a row a thread took
      // 4 us of load instructions).  The scores of the unit before have all been computed.
      float c = 0.f;   // scores times this are x, the exponent in base 2
      {
        constexpr int kLanes = D / 16, kStep = 32 / kLanes, kSteps = 32 / kStep;
        const int first = u.rt * kPromptRows + t * kRows + (warp & 3) * 32, x = lane % kLanes;
        const int cols = u.rows * p.g;
        uint4 v[kSteps][2];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const int rc = first + i * kStep + lane / kLanes;
          v[i][0] = v[i][1] = make_uint4(0, 0, 0, 0);
          if (rc < cols) {
            const int tk = over_group(p, rc);
            const uint4* at = reinterpret_cast<const uint4*>(p.q + (u.row0 + tk) * p.q_stride + (u.h * p.g + rc - tk * p.g) * D) + 2 * x;
            v[i][0] = at[0];
            v[i][1] = at[1];
          }
        }
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const uint4 v0 = v[i][0], v1 = v[i][1];
          const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
          uint32_t most = 0;   // the row's largest magnitude, as bf16 bits
#pragma unroll
          for (int k = 0; k < 8; ++k) most = __vmaxu2(most, w[k] & 0x7fff7fffu);
          uint32_t top = max(most & 0xffffu, most >> 16);
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
          const int e = top == 0 ? 0 : min(max((int)(top >> 7) - 127, -110), 126);
          // a row with inf or NaN becomes NaN; |q| below 256 has 8 bits in f16 too, down to 2^-14
          const float down = top >= 0x7f80u ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)(127 + 7 - e) << 23);
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint16_t h8[2], l8[2];
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const uint32_t q2 = pack_f16(bf_lo(w[2 * k + z]) * down, bf_hi(w[2 * k + z]) * down);
              h8[z] = f16x2_to_e4m3x2(q2);
              const uint32_t back = q8::e4m3x2_to_f16x2(h8[z]);
              const __half2 rest = __hsub2(*reinterpret_cast<const __half2*>(&q2), *reinterpret_cast<const __half2*>(&back));
              l8[z] = f16x2_to_e4m3x2(*reinterpret_cast<const uint32_t*>(&rest));
            }
            hi[k] = (uint32_t)h8[0] | ((uint32_t)h8[1] << 16);
            lo[k] = (uint32_t)l8[0] | ((uint32_t)l8[1] << 16);
          }
          const uint32_t at = row_chunk(0, (warp & 3) * 32 + i * kStep + lane / kLanes, x);
          asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(hi[0]), "r"(hi[1]), "r"(hi[2]), "r"(hi[3]) : "memory");
          asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at + L::kQ), "r"(lo[0]), "r"(lo[1]), "r"(lo[2]), "r"(lo[3]) : "memory");
          const float mine = __shfl_sync(0xffffffffu, p.scale * __uint_as_float((uint32_t)(127 - 7 + e) << 23), (lane % kStep) * kLanes);
          if (i == lane / kStep) c = mine;
        }
        fence_proxy_async_smem();
        mbar_arrive(qfull(t));
      }
      float m = -INFINITY, l = 0.f, vref = 0.f;
      bool apart = false;
      int j = u.j0;
      for (; j < u.j1; ++j, ++n, ++ns) {
        ok = wait(sfull(t), ns & 1);
        if (!ok) break;
        tc_fence_after();
        uint32_t r[L::kP][16];   // the row's scores, by pages
#pragma unroll
        for (int q = 0; q < L::kP; ++q) tmem_ld16(S + 16 * q, r[q]);
        float f[L::kP];
#pragma unroll
        for (int q = 0; q < L::kP; ++q) f[q] = sh.ks[n % kScaleSlots][q] * c;
        const float nvref = sh.vref[n % kScaleSlots];
        apart = !(nvref > 0.f);
#pragma unroll
        for (int q = 0; q < L::kP; ++q) tmem_wait_ld(r[q]);
        if (__builtin_expect(apart, 0)) break;
        tc_fence_before();
        mbar_arrive(sread(t));
        if (__builtin_expect((j + 1) * N > first_limit, 0)) {
          const int seen = limit - j * N;   // columns below this are visible
#pragma unroll
          for (int q = 0; q < L::kP; ++q) {
            // A masked score is -inf times its page's factor, which has to be above 0.  A page of which the row
            // sees nothing, or which is not there, has no say; one that it sees at least fp32's smallest normal
            // number: with less its scores, products below 2^25, vanish either way.
            if (16 * q >= seen) f[q] = 1.f;
            else if (f[q] < kLeastFactor) f[q] = kLeastFactor;
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (16 * q + i >= seen) asm volatile("mov.b32 %0, 0xff800000;" : "=r"(r[q][i]));   // -inf
          }
        }
        float top = -INFINITY;
#pragma unroll
        for (int q = 0; q < L::kP; ++q) {
          float a = __uint_as_float(r[q][0]);
#pragma unroll
          for (int i = 1; i < 16; ++i) a = fmaxf(a, __uint_as_float(r[q][i]));
          top = fmaxf(top, a * f[q]);
        }
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
        const bool correct = __any_sync(0xffffffffu, fix != 1.f);
        if (j > u.j0) {
          ok = wait(pread(t), (ns - 1) & 1);   // the place of the first part of the weights is free
          if (ok && correct) {
            ok = wait(ofull(t), (ns - 1) & 1);
            if (!ok) break;
            tc_fence_after();
            scale_accumulator(fix);
          }
          if (!ok) break;
        }
        const float base = kShift - (m == -INFINITY ? 0.f : m);
        const uint64_t base2 = pair2(base, base);
        uint64_t sum2 = 0;
#pragma unroll
        for (int q = 0; q < L::kP; ++q) {
          uint32_t w[8];
          const uint64_t f2 = pair2(f[q], f[q]);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 x = unpair2(fma2(pair2(__uint_as_float(r[q][2 * i]), __uint_as_float(r[q][2 * i + 1])), f2, base2));
            const float e0 = ex2(x.x), e1 = ex2(x.y);
            sum2 = add2(sum2, pair2(e0, e1));
            w[i] = pack_f16(e0, e1);
          }
          if (q == L::kP0 && j > u.j0) {   // and the place of the second part
            ok = wait(ofull(t), (ns - 1) & 1);
            if (!ok) break;
          }
          tmem_st8(P + 8 * q, w);
          if (q == L::kP0 - 1 || q == L::kP - 1) {
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(pfull(t, q == L::kP - 1));
          }
        }
        if (!ok) break;
        const float2 sum = unpair2(sum2);
        l += sum.x + sum.y;
      }
      float om = m + lg2(vref);   // the accumulator holds sums of 2^(x - om + 14) times v
      if (__builtin_expect(apart, 0)) {
        // The part's remaining tiles, from one whose scales lie apart: the accumulator's weights are
        // 2^(x + log2 vs - om + 7).  Rare, so by pages, from TMEM as often as the scores are needed.
        if (m == -INFINITY) om = -INFINITY;
#pragma unroll 1
        while (ok) {
          const int slot = n % kScaleSlots, seen = limit - j * N;
          const auto scores = [&](int q, uint32_t (&x)[16]) {
            tmem_ld16(S + 16 * q, x);
            tmem_wait_ld(x);
            const float f = sh.ks[slot][q] * c;
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = 16 * q + i < seen ? __float_as_uint(__uint_as_float(x[i]) * f) : 0xff800000u;
          };
          float top = -INFINITY, high = -INFINITY;
#pragma unroll 1
          for (int q = 0; q < L::kP; ++q) {
            uint32_t x[16];
            scores(q, x);
            float a = __uint_as_float(x[0]);
#pragma unroll
            for (int i = 1; i < 16; ++i) a = fmaxf(a, __uint_as_float(x[i]));
            top = fmaxf(top, a);
            high = fmaxf(high, a + lg2(sh.vs[slot][q]));
          }
          if (top > m + kLazy) {
            l *= ex2(m - top);
            m = top;
          }
          float fix = 1.f;
          if (high > om + kLazy) {
            fix = ex2(om - high);
            om = high;
          }
          if (j > u.j0) {
            ok = wait(ofull(t), (ns - 1) & 1);   // the places of the weights are free, the accumulator is at rest
            if (!ok) break;
            tc_fence_after();
            if (__any_sync(0xffffffffu, fix != 1.f)) scale_accumulator(fix);
          }
          const float zm = m == -INFINITY ? 0.f : m, zo = om == -INFINITY ? 0.f : om;
#pragma unroll 1
          for (int q = 0; q < L::kP; ++q) {
            uint32_t x[16], w[8];
            scores(q, x);
            const float base = kShift + lg2(sh.vs[slot][q]) - zo;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float a = __uint_as_float(x[2 * i]), b = __uint_as_float(x[2 * i + 1]);
              l += ex2(a - zm + kShift) + ex2(b - zm + kShift);
              w[i] = pack_f16(ex2(a + base), ex2(b + base));
            }
            tmem_st8(P + 8 * q, w);
          }
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(sread(t));
          mbar_arrive(pfull(t, 0));
          mbar_arrive(pfull(t, 1));
          ++n, ++ns;
          if (++j == u.j1) break;
          ok = wait(sfull(t), ns & 1);
          tc_fence_after();
        }
      }
      if (!ok) break;
      // ---- the part's result -----------------------------------------------------------------
      ok = wait(ofull(t), (ns - 1) & 1);
      if (!ok) break;
      tc_fence_after();
      l *= 0x1p-7f;   // 2^-kShift
      om -= kVShift;
      // Rows are laid out in shared memory, in the Q tile that the finished unit no longer needs, and
      // leave by whole rows (32 rows' 16 bytes an instruction took 2 us a unit): kRowChunks chunks a pass.
      constexpr int kRowChunks = D / 8, kHalf = D / 16;   // 16-byte chunks of the two parts, of one
      const bool whole = begins && ends;
      const float2 f = result_factors(m, om, l);
      float* part = p.partial + ((int64_t)(blockIdx.x * 2 + (begins ? 1 : 0)) * p.cols + t * kRows) * (D + 4);
      const bool odd = uniform(*static_cast<volatile int*>(&sh.later_nan)) != 0;
      if (odd) find_later_nan<D>(p, u.s, u.h, max(seen_by_all(p, u), u.j0 * N), min(u.len, u.j1 * N), sh.nan_at[warp]);
      auto stage = [&](int x, uint32_t a, uint32_t b2, uint32_t c2, uint32_t d) {
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(row_chunk(x / kHalf, row, x % kHalf)), "r"(a), "r"(b2), "r"(c2), "r"(d) : "memory");
      };
#pragma unroll 1
      for (int pass = 0; pass < (whole ? 1 : 2); ++pass) {
        if (whole) {
#pragma unroll
          for (int b = 0; b < D / 32; ++b) {
            uint32_t r[32], w[16];
            tmem_ld32(O + 32 * b, r);
            tmem_wait_ld(r);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(r[2 * i]) * f.x * f.y, __uint_as_float(r[2 * i + 1]) * f.x * f.y);
              w[i] = *reinterpret_cast<const uint32_t*>(&v);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) stage(4 * b + i, w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
          }
        } else {
#pragma unroll
          for (int b = 0; b < D / 64; ++b) {
            uint32_t r[32];
            tmem_ld32(O + pass * (D / 2) + 32 * b, r);
            tmem_wait_ld(r);
#pragma unroll
            for (int i = 0; i < 8; ++i) stage(8 * b + i, r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
          }
        }
        __syncwarp();
        // kAtOnce rows an instruction; the rows' swizzle differs by constants, so an address is one xor away
        constexpr int kAtOnce = 32 / kRowChunks;
        const int x = lane % kRowChunks, sub = lane / kRowChunks;
        const uint32_t from = row_chunk(x / kHalf, (warp & 3) * 32 + sub, x % kHalf);
        uint8_t* to_out = reinterpret_cast<uint8_t*>(p.out) + 16 * x;
        uint8_t* to_part = reinterpret_cast<uint8_t*>(part + (int64_t)((warp & 3) * 32 + sub) * (D + 4) + pass * (D / 2)) + 16 * x;
#pragma unroll
        for (int i = 0; i < 32 / kAtOnce; ++i) {
          const uint32_t to_row = __shfl_sync(0xffffffffu, out_row, i * kAtOnce + sub);
          const uint32_t swizzle = (D == 128 ? (i * kAtOnce) & 6 : (i * kAtOnce / 2) & 2) << 4;
          uint4 v;
          asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                       : "r"((from ^ swizzle) + i * kAtOnce * D));
          if (odd) {   // rows that see a value that was taken out
            const int lim = __shfl_sync(0xffffffffu, limit, i * kAtOnce + sub);
            const int* at = sh.nan_at[warp] + (whole ? 8 * x : pass * (D / 2) + 4 * x);
            uint32_t* const word[4] = {&v.x, &v.y, &v.z, &v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (!whole && at[e] < lim) *word[e] = 0x7fc00000u;
              if (whole && at[2 * e] < lim) *word[e] |= 0x7fc0u;
              if (whole && at[2 * e + 1] < lim) *word[e] |= 0x7fc00000u;
            }
          }
          if (to_row != kNoRow) {
            if (whole) *reinterpret_cast<uint4*>(to_out + (int64_t)to_row * (2 * D)) = v;
            else *reinterpret_cast<uint4*>(to_part + i * kAtOnce * (D + 4) * 4) = v;
          }
        }
        __syncwarp();
      }
      if (live) {
        if (!whole) *reinterpret_cast<float4*>(part + (int64_t)row * (D + 4) + D) = make_float4(m, om, l, 0.f);
        else if (p.lse) p.lse[out_row] = (m + lg2(l)) * kLn2;
      }
      tc_fence_before();   // the accumulator is read before the next unit's first product
    } while (ok && next_unit<N>(p, u));
    if (tid == 0) {
      p.meta[2 * blockIdx.x] = meta;
      p.meta[2 * blockIdx.x + 1] = make_int4(meta_cols, 0, 0, 0);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 13) tmem_dealloc(tmem, 512);
  write_idle(p, D);
}

// A warp a row of a unit that more than one CTA held: block (i, y) takes rows y * kCombineRows .. of
// the unit that begins in CTA i, two rows a warp and two parts of each at a time. That CTA knows from its
// share where the unit ends and says so, so that nothing is searched here. Four parts at a time cost 5 us
// more of the 6 questions' 215: most units have two.
constexpr int kCombineWarps = 4, kCombineRows = 8;
template <int D>
__global__ void __launch_bounds__(32 * kCombineWarps) prompt_combine_kernel(const __grid_constant__ Params p) {
  constexpr int V = D / 32;   // values a lane
  constexpr int kEach = kCombineRows / kCombineWarps, kBatch = 2;   // rows a warp, parts in flight
  // No word to the dependents before the end: a prompt kernel that is let in while this one leaves gets its blocks
  // onto the SMs in the order in which they fall free, shares that lie side by side in the list no longer run side by
  // side, and call after call grows slower (4096 rows over 16441 tokens, 200 calls in a row: 719 us each against 688).
  pdl_wait();
  const int i = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int4 mt = p.meta[2 * i], mt2 = p.meta[2 * i + 1];
  const int col0 = mt.z * kPromptRows + blockIdx.y * kCombineRows, n = min(mt.x, p.n_cta - i);
  if (mt.x <= 0 || col0 >= mt2.x) return;
  float acc[kEach][V], m[kEach], om[kEach], l[kEach];
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    m[k] = om[k] = -INFINITY;
    l[k] = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) acc[k][v] = 0.f;
  }
  for (int x0 = 0; x0 < n; x0 += kBatch) {
    float4 st[kEach][kBatch];
    float val[kEach][kBatch][V];
#pragma unroll
    for (int k = 0; k < kEach; ++k)
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int x = x0 + b, row = warp + k * kCombineWarps;
        const bool held = x < n && col0 + row < mt2.x;
        const float* e = p.partial +
                         ((int64_t)((i + x) * 2 + (x == 0 ? 1 : 0)) * p.cols + blockIdx.y * kCombineRows + row) * (D + 4);
        st[k][b] = held ? *reinterpret_cast<const float4*>(e + D) : make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
#pragma unroll
        for (int v = 0; v < V; ++v) val[k][b][v] = held ? e[lane * V + v] : 0.f;
      }
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      float nm = m[k], no = om[k];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        nm = fmaxf(nm, st[k][b].x);
        no = fmaxf(no, st[k][b].y);
      }
      const float zm = nm == -INFINITY ? 0.f : nm, zo = no == -INFINITY ? 0.f : no;   // 2^-inf = 0, and no inf - inf
      l[k] *= ex2(m[k] - zm);
      const float r = ex2(om[k] - zo);
#pragma unroll
      for (int v = 0; v < V; ++v) acc[k][v] *= r;
      m[k] = nm;
      om[k] = no;
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        l[k] = fmaf(st[k][b].z, ex2(st[k][b].x - zm), l[k]);
        const float w = ex2(st[k][b].y - zo);
#pragma unroll
        for (int v = 0; v < V; ++v) acc[k][v] = fmaf(val[k][b][v], w, acc[k][v]);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int col = col0 + warp + k * kCombineWarps;
    if (col >= mt2.x) continue;
    const float2 r = result_factors(m[k], om[k], l[k]);
    const int tok = over_group(p, col);
    const int64_t row = (int64_t)(mt.w + tok) * p.Hq + mt.y * p.g + col - tok * p.g;
#pragma unroll
    for (int v = 0; v < V; v += 2) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(acc[k][v] * r.x * r.y, acc[k][v + 1] * r.x * r.y);
      *reinterpret_cast<uint32_t*>(p.out + row * D + lane * V + v) = *reinterpret_cast<const uint32_t*>(&b);
    }
    if (p.lse && lane == 0) p.lse[row] = (m[k] + lg2(l[k])) * kLn2;
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
