// Drafted tokens against the target's probabilities (kv_verify_drafts).
//
//   Draft d of a sequence stays while u_d q_d(t) < p_d(t); at the first row a that turns one down
//   (or has none) a token is drawn from max(0, p_a - q_a) (from p_a where none was turned down).
//
// Probabilities become whole numbers, floor(2^40 x), before they are subtracted and summed: sums
// are exact in 64 bits (vocab up to 2^22), so the drawn token depends on neither their order nor on
// how a row is split, and the result can be compared for equality.  A value below 2^-40 weighs
// nothing: 2^22 of them together are 4e-6.
//
// Bound by memory: one row of p and, where a draft was turned down, one of q.
//   - A cluster of CTAs takes a sequence.  Each CTA looks at the drafts by itself (a few gathered
//     values), streams its share of the row (16 bytes a load, 4 of p and 4 of q in flight a thread)
//     and keeps a sum for each warp, whose part of the row is contiguous; the CTAs' sums go to every
//     CTA of the cluster through shared memory.  One of them finds the draw inside its own part, reads
//     the part of the warp that holds it again (from L2), a vector a thread, and scans that.
//   - A row begins wherever its stride puts it: vectors are cut at 16-byte boundaries, the ends
//     are read by elements, and where p's and q's rows begin differently q is.
//
// Measured: 256 sequences x 262144 values (fp32, 424 MB) 77 us, 5.5 TB/s, 81% of a copy; 64 x 130003 (56 MB)
// 15.8 us, where finding the rows before and the token after streaming them takes 5; 37 x 50021 bf16 9.6 us; one
// sequence x 32000 5.1 us, a launch and five dependent trips to memory.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cstring>

#include "kvrp.h"
#include "kvrp_plan.h"
#include "kvrp_ptx.h"
#include "kvrp_q8.h"

namespace kvrp {
namespace verify {

using namespace kvrp::ptx;
using q8::flag;
using q8::sequence;

constexpr int kThreads = 512, kWarps = kThreads / 32, kMostCtas = 8;

struct Params {
  const void *target, *draft;
  int64_t target_stride, draft_stride;
  const int32_t* tokens;
  const float *u_accept, *u_sample;
  int32_t *out, *accepted, *kept;
  kvrp_seqs seqs;
  uint32_t* status;
  int vocab;
};

__device__ __forceinline__ float value(float x) { return x; }
__device__ __forceinline__ float value(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
// floor(2^40 x), x in [0, 1], as 2^20 high + low, both below 2^23 and so in the low bits of a sum with 2^23
// that is rounded down; `bits` are those sums' own, kBits above high and low.  Every step is exact.  (The
// conversion to 64 bits runs at a fraction of these four operations' rate: 256 rows of 262144 took 226 us.)
constexpr uint32_t kBits = 0x4b000000u;   // 2^23
struct Whole {
  uint32_t high, low;
  __device__ __forceinline__ explicit Whole(float x) {
    const float h = __fmaf_rd(x, 0x1p20f, 0x1p23f);
    const float rest = __fmaf_rn(x, 0x1p20f, 0x1p23f - h);
    high = __float_as_uint(h);
    low = __float_as_uint(__fmaf_rd(rest, 0x1p20f, 0x1p23f));
  }
};
__device__ __forceinline__ uint64_t whole(float x) {
  const Whole w(x);
  return ((uint64_t)(w.high - kBits) << 20) + (w.low - kBits);
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void store_to_cta(uint32_t local, uint32_t rank, uint64_t v) {
  uint32_t at;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(local), "r"(rank));
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(v) : "memory");
}

template <typename T>
__device__ __forceinline__ uint64_t warp_scan(T v) {   // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  return v;
}

// A row of probabilities, in vectors of kE that begin on 16 bytes: the row's element 0 is element
// `skip` of vector 0.
template <typename T>
struct Row {
  static constexpr int kE = 16 / sizeof(T);
  const T* at;
  int skip;
  __device__ __forceinline__ Row(const void* base, int64_t offset)
      : at(static_cast<const T*>(base) + offset), skip((int)(reinterpret_cast<uintptr_t>(at) / sizeof(T)) & (kE - 1)) {}
};
template <typename T>
__device__ __forceinline__ void load(const T* row, int first, int vocab, bool fits, T (&x)[16 / sizeof(T)]) {
  constexpr int kE = 16 / sizeof(T);
  if (fits && first >= 0 && first + kE <= vocab) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(row + first));
    memcpy(x, &v, 16);
  } else {
#pragma unroll
    for (int i = 0; i < kE; ++i) x[i] = first + i >= 0 && first + i < vocab ? __ldg(row + first + i) : T(0);
  }
}

enum Kind { kTarget, kPositivePart, kWithout };   // weights: p; max(0, p - q); p but for one token
template <typename T>
struct Weights {
  static constexpr int kE = Row<T>::kE;
  Row<T> p, q;
  int vocab, token;
  bool q_fits;
  template <Kind K>
  __device__ __forceinline__ void raw(int v, T (&a)[kE], T (&b)[kE]) const {
    const int first = v * kE - p.skip;
    load<T>(p.at, first, vocab, true, a);
    if (K == kPositivePart) load<T>(q.at, first, vocab, q_fits, b);
  }
  template <Kind K>
  __device__ __forceinline__ uint64_t weight(int v, int i, T a, T b) const {
    const float x = __saturatef(value(a));   // [0, 1], and 0 of NaN
    if (K == kWithout) return v * kE - p.skip + i == token ? 0 : whole(x);
    if (K == kTarget) return whole(x);
    return whole(x) - whole(fminf(x, __saturatef(value(b))));   // where q is not below p, p - p
  }
  // Of vectors [begin, end), this lane's share.  With K = kWithout the token counts: taken off once, below.
  template <Kind K>
  __device__ __forceinline__ uint64_t sum(int begin, int end) const {
    constexpr int kDepth = 4;
    const int lane = threadIdx.x & 31;
    uint64_t s = 0;
    const auto add = [&](const T (&a)[kE], const T (&b)[kE], uint32_t& high, uint32_t& low) {
#pragma unroll
      for (int i = 0; i < kE; ++i) {
        const float x = __saturatef(value(a[i]));
        const Whole w(x);
        if (K == kPositivePart) {
          const Whole less(fminf(x, __saturatef(value(b[i]))));
          high += w.high - less.high;
          low += w.low - less.low;
        } else {
          high += w.high - kBits;
          low += w.low - kBits;
        }
      }
    };
    // at most 32 values at a time: |high|, |low| stay below 2^25; low may be negative
    const auto flush = [&](uint32_t high, uint32_t low) { s += ((uint64_t)high << 20) + (uint64_t)(int64_t)(int32_t)low; };
    int v = begin + lane;
    for (; v + 32 * (kDepth - 1) < end; v += 32 * kDepth) {
      T a[kDepth][kE], b[kDepth][kE];
#pragma unroll
      for (int d = 0; d < kDepth; ++d) raw<K>(v + 32 * d, a[d], b[d]);
      uint32_t high = 0, low = 0;
#pragma unroll
      for (int d = 0; d < kDepth; ++d) add(a[d], b[d], high, low);
      flush(high, low);
    }
    for (; v < end; v += 32) {
      T a[kE], b[kE];
      raw<K>(v, a, b);
      uint32_t high = 0, low = 0;
      add(a, b, high, low);
      flush(high, low);
    }
    if (K == kWithout && token >= 0 && token < vocab) {
      const int at = (token + p.skip) / kE;
      if (at >= begin && at < end && (at - begin) % 32 == lane) s -= whole(__saturatef(value(p.at[token])));
    }
    return s;
  }
};

struct Smem {
  uint64_t cta[2][kMostCtas];   // the CTAs' sums, for each of the two tries
  uint64_t warp[kWarps];
  uint64_t scan[kWarps];
};

// The token whose running sum first passes t, among vectors [begin, end); whole CTA.
template <Kind K, typename T>
__device__ __forceinline__ void find(const Weights<T>& w, Smem& sh, int begin, int end, uint64_t t, int32_t* out) {
  constexpr int kE = Row<T>::kE;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint64_t before = 0;
  for (int v0 = begin; v0 < end; v0 += kThreads) {
    const int v = v0 + tid;
    T a[kE], b[kE];
    uint64_t x[kE], mine = 0;
    if (v < end) w.template raw<K>(v, a, b);
#pragma unroll
    for (int i = 0; i < kE; ++i) {
      x[i] = v < end ? w.template weight<K>(v, i, a[i], b[i]) : 0;
      mine += x[i];
    }
    const uint64_t upto = warp_scan(mine);
    if (lane == 31) sh.scan[warp] = upto;
    __syncthreads();
    uint64_t lo = before + upto - mine;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) lo += sh.scan[i];
      before += sh.scan[i];
    }
    if (t >= lo && t < lo + mine) {   // in one thread
      int i = 0;
#pragma unroll
      for (int j = 0; j < kE - 1; ++j) {
        if (i == j && t >= lo + x[j]) lo += x[j], i = j + 1;
      }
      *out = v * kE - w.p.skip + i;
    }
    if (before > t) return;   // the same in all threads
    __syncthreads();
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) verify_kernel(const __grid_constant__ Params p) {
  __shared__ Smem sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, s = blockIdx.y;
  const int rank = (int)cluster_rank(), ctas = (int)cluster_size();
  cluster_arrive();   // this CTA runs: the others may write to its shared memory
  pdl_wait();
  pdl_launch_dependents();
  int row0, rows, len;
  const bool ok = sequence(p.seqs, s, row0, rows, len);
  if (!ok || rows == 0) {
    cluster_wait();
    if (rank != 0) return;
    const int end = p.seqs.row_start ? p.seqs.row_start[s + 1] : s + 1;
    const bool inside = row0 >= 0 && end >= row0 && end <= p.seqs.n_rows;
    if (!ok || !inside) {
      if (tid == 0) flag(p.status, KVRP_DEV_BAD_LENGTH);
      return;
    }
    for (int r = row0 + tid; r < end; r += kThreads) p.out[r] = -1;   // an idle place's rows
    if (tid == 0) {
      if (p.accepted) p.accepted[s] = 0;
      if (p.kept && len > 0) p.kept[s] = len;
    }
    return;
  }
  // ---- the drafts that stay; every warp looks for itself ---------------------------------
  int a = rows - 1, token = -1;
  for (int d0 = 0; d0 < rows - 1; d0 += 32) {
    const int d = d0 + lane;
    int t = 0;
    bool stays = true;
    if (d < rows - 1) {
      t = p.tokens[row0 + d + 1];
      stays = false;
      if (t >= 0 && t < p.vocab) {
        const float u = p.u_accept[row0 + d];
        const float x = value(static_cast<const T*>(p.target)[(row0 + d) * p.target_stride + t]);
        const float y = p.draft ? value(static_cast<const T*>(p.draft)[(row0 + d) * p.draft_stride + t]) : 1.f;
        stays = (double)u * (double)y < (double)x;
      }
    }
    const uint32_t down = __ballot_sync(0xffffffffu, !stays);
    if (down) {
      const int at = __ffs(down) - 1;
      a = d0 + at;
      token = __shfl_sync(0xffffffffu, t, at);
      break;
    }
  }
  const bool turned_down = a < rows - 1, strange = turned_down && (token < 0 || token >= p.vocab);
  // ---- the weights' sums ------------------------------------------------------------------
  Weights<T> w = {Row<T>(p.target, (row0 + a) * p.target_stride),
                  Row<T>(p.draft ? p.draft : p.target, p.draft ? (row0 + a) * p.draft_stride : (row0 + a) * p.target_stride),
                  p.vocab, token, false};
  w.q_fits = w.q.skip == w.p.skip;
  Kind kind = !turned_down ? kTarget : p.draft ? kPositivePart : kWithout;
  const int vectors = (p.vocab + w.p.skip + Row<T>::kE - 1) / Row<T>::kE;
  const int each = ((vectors + ctas * kWarps - 1) / (ctas * kWarps) + 31) / 32 * 32;   // a warp's
  const int begin = min(vectors, (rank * kWarps + warp) * each), end = min(vectors, begin + each);
  const uint32_t r = __float2uint_rz(p.u_sample[s] * 0x1p32f);   // 0 of NaN and of less, 2^32 - 1 of 1 and more
  uint64_t total = 0, before = 0, own = 0;
#pragma unroll 1
  for (int attempt = 0; attempt < 2; ++attempt) {
    uint64_t sum = kind == kTarget ? w.template sum<kTarget>(begin, end)
                                   : kind == kWithout ? w.template sum<kWithout>(begin, end) : w.template sum<kPositivePart>(begin, end);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) sh.warp[warp] = sum;
    __syncthreads();
    own = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) own += sh.warp[i];
    if (attempt == 0) cluster_wait();
    if (tid < ctas) store_to_cta(smem_u32(&sh.cta[attempt][rank]), (uint32_t)tid, own);
    cluster_arrive();
    cluster_wait();
    total = before = 0;
    for (int i = 0; i < ctas; ++i) {
      if (i < rank) before += sh.cta[attempt][i];
      total += sh.cta[attempt][i];
    }
    if (total > 0 || kind == kTarget) break;
    kind = kTarget;   // no positive part
  }
  // ---- the draw ---------------------------------------------------------------------------
  if (total > 0) {
    uint64_t t = __umul64hi((uint64_t)r << 32, total);
    if (t >= before && t < before + own) {
      t -= before;
      int x = 0;   // the warp whose part holds it
      while (t >= sh.warp[x]) t -= sh.warp[x++];
      const int b = min(vectors, (rank * kWarps + x) * each), e = min(vectors, b + each);
      int32_t* out = p.out + row0 + a;
      if (kind == kTarget) find<kTarget>(w, sh, b, e, t, out);
      else if (kind == kWithout) find<kWithout>(w, sh, b, e, t, out);
      else find<kPositivePart>(w, sh, b, e, t, out);
    }
  }
  if (rank != 0) return;
  if (tid == 0) {
    if (total == 0) p.out[row0 + a] = -1;
    if (total == 0 || strange) flag(p.status, KVRP_DEV_BAD_TOKEN);
    if (p.accepted) p.accepted[s] = a;
    if (p.kept) p.kept[s] = len - (rows - 1 - a);
  }
  for (int i = tid; i < rows; i += kThreads)
    if (i != a) p.out[row0 + i] = i < a ? p.tokens[row0 + i + 1] : -1;
}

}  // namespace verify
}  // namespace kvrp

using namespace kvrp;

extern "C" kvrp_status kv_verify_drafts(const void* target, int64_t target_stride, const void* draft, int64_t draft_stride,
                                        int32_t prob_type, int32_t vocab, const kvrp_seqs* seqs, const int32_t* tokens,
                                        const float* u_accept, const float* u_sample, int32_t* out_tokens, int32_t* accepted,
                                        int32_t* kept_lens, uint32_t* d_status, kvrp_stream_t stream) {
  const char* fn = "kv_verify_drafts";
  g_last_launches = 0;
  kvrp_status st = check_seqs(fn, seqs);
  if (st != KVRP_OK) return st;
  if (!target || !tokens || !u_accept || !u_sample || !out_tokens) return fail(KVRP_ERR_INVALID_ARG, "%s: NULL argument", fn);
  if (prob_type != KVRP_F32 && prob_type != KVRP_BF16) return fail(KVRP_ERR_UNSUPPORTED, "%s: prob_type must be KVRP_F32 or KVRP_BF16", fn);
  if (vocab <= 0 || vocab > 1 << 22) return fail(KVRP_ERR_UNSUPPORTED, "%s: 1 <= vocab <= 2^22", fn);
  target_stride = target_stride ? target_stride : vocab;
  draft_stride = draft_stride ? draft_stride : vocab;
  if (target_stride < vocab || draft_stride < vocab) return fail(KVRP_ERR_INVALID_ARG, "%s: a row stride is shorter than the row", fn);
  if (out_tokens == tokens) return fail(KVRP_ERR_INVALID_ARG, "%s: out_tokens cannot be tokens", fn);
  const uintptr_t each = prob_type == KVRP_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(target) % each || reinterpret_cast<uintptr_t>(draft) % each)
    return fail(KVRP_ERR_ALIGNMENT, "%s: probabilities are not aligned", fn);
  for (const void* x : {(const void*)tokens, (const void*)u_accept, (const void*)u_sample, (const void*)out_tokens,
                        (const void*)accepted, (const void*)kept_lens, (const void*)d_status})
    if (reinterpret_cast<uintptr_t>(x) % 4) return fail(KVRP_ERR_ALIGNMENT, "%s: a 4-byte array is not aligned", fn);
  int sms = 0, smem_optin = 0;
  st = current_device_sms(&sms, &smem_optin);
  if (st != KVRP_OK) return st;

  verify::Params p;
  std::memset(&p, 0, sizeof(p));
  p.target = target;
  p.draft = draft;
  p.target_stride = target_stride;
  p.draft_stride = draft_stride;
  p.tokens = tokens;
  p.u_accept = u_accept;
  p.u_sample = u_sample;
  p.out = out_tokens;
  p.accepted = accepted;
  p.kept = kept_lens;
  p.seqs = *seqs;
  p.status = d_status;
  p.vocab = vocab;

  // CTAs a sequence, of at least 4096 values each: what one filling of the GPU holds, two an SM, or the
  // second filling costs as much as the first (64 sequences of 130003: 15.7 us with 4, 22.5 with 6,
  // 20.6 with 8); for more sequences than that two, whose uneven ends hide each other (256 of 262144:
  // 81.5 us with 1, 76.8 with 2, 85.9 with 8).
  const int ctas = std::max(1, std::min({verify::kMostCtas, std::max(2, 2 * sms / seqs->n_seqs), vocab / 4096}));
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas, (unsigned)seqs->n_seqs);
  cfg.blockDim = dim3(verify::kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = prob_type == KVRP_F32 ? cudaLaunchKernelEx(&cfg, verify::verify_kernel<float>, p)
                                              : cudaLaunchKernelEx(&cfg, verify::verify_kernel<uint16_t>, p);
  if (e != cudaSuccess) return fail(KVRP_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
  g_last_launches = 1;
  return KVRP_OK;
}
