// Attention over the 8-bit paged cache of a batch whose sequences begin with the same tokens
// (kv_attend_shared_q8).
//
//   out = (e^a O_a + e^b O_b) / (e^a + e^b):  O_a, a the attention and log-sum-exp over the shared tokens,
//   O_b, b over a sequence's own tokens behind them (causal).
//
// Where little is shared each sequence reads it (kEachBytes): the kernel for few rows over the prefix's pages and the
// sequence's own, one after the other.  Else three passes, none of which reads much twice:
//   - the shared tokens, for all rows of the batch as if they were one sequence's: the tensor-core kernel
//     for prompts (kvrp_attend_q8_prompt.cu) with every row seeing every token.  K and V of the shared pages are
//     read once for each 256 (row, query head) pairs of a KV head instead of once a sequence, and few rows
//     a sequence become full tiles.
//   - the sequences' own tokens, from the shared pages' end on: kv_attend_q8's kernel for few rows (see
//     Runs for more of them than it takes at once) or for many.
//   - join_kernel merges both passes' partial results, in fp32, and rounds once.  A unit of the first pass
//     that several CTAs shared is found by arithmetic (EvenUnits); one of the second by a record that the
//     CTA that begins it leaves.
// The second pass depends on nothing in the first: its blocks take the SMs that the first one's leave, one
// after another, and wait for it at their end alone; the join looks up what it needs before it waits.
//
// Measured, 28 / 4 heads x 128, beside kv_attend_q8, which reads the shared tokens for each sequence: 64 sequences,
// 16384 shared tokens, 30 to 1500 own 49.8 us (135.7); 96, 100000 and 100 to 3000: 173 us, 800 TFLOP/s (1092); 16 of 5
// rows, 65536 and 40 to 2000: 120 us (425).  32 / 32 heads, 24 sequences, 4144 and 20 to 700: 44.8 us (107).  32 / 8 heads
// x 64, 32 of 4 rows, 9008 and 10 to 900: 42.7 us (78.2).  Of the 49.8 us, by time stamps: 4 until the first pass knows its
// share, 5 until its queries are laid out, 14 for 11 token tiles a CTA, 3 for its results, 12 for the own tokens behind them
// (26 MB: latency), 6 for the join (20 MB of partial results from L2); the rest lies between the launches.  A token tile
// takes 1.2 us whatever the rows: 1850 of its 2300 cycles are the softmax warps', a thread a row, and the products and
// conversions beside them take as long in turn.
// Many rows a sequence: 8 sequences of 200 (900) rows over 16384 shared tokens 416 us (1735), where kv_attend_q8 takes 359
// (1394): its work is the same, and it writes no partial results of two passes.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <cstring>

#include "kvrp.h"
#include "kvrp_attend_q8.h"
#include "kvrp_plan.h"
#include "kvrp_q8.h"

namespace kvrp {
namespace attend_q8 {

namespace {

struct Join {
  Params p;                   // of the second pass
  const float *shared, *shared_dense;   // the first one's partial and dense results, its CTAs at most
  int shared_ctas;
  bool few;
};

constexpr int kJoinThreads = 128;

// A row and kItems of its query heads a block; D / 4 threads hold an item's features, four each.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ Join j) {
  constexpr int kLanes = D / 4, kItems = kJoinThreads / kLanes, N = prompt_tokens(D), kStep = D + 4;
  const Params& p = j.p;
  const int chunks = (p.Hq + kItems - 1) / kItems;
  const int row = blockIdx.x / chunks, head = blockIdx.x % chunks * kItems + threadIdx.x / kLanes, f = threadIdx.x % kLanes;
  // What is looked up first was there before this call: the passes' blocks had all waited for it, or were let in by
  // blocks that had, when they let this kernel's in.
  pdl_launch_dependents();
  const View view = load_view(p);
  int s = row;   // the row's sequence: the last whose first row is not behind it
  if (p.seqs.row_start && view.tokens >= 0) {
    int lo = 0, hi = p.seqs.n_seqs;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.seqs.row_start[mid] <= row) lo = mid;
      else hi = mid;
    }
    s = lo;
  }
  int row0 = 0, rows = 0, len = 0;
  const bool ok = view.tokens >= 0 && row >= view.first && row < view.end && own_sequence<kRest>(p, s, row0, rows, len);
  const int64_t at = (int64_t)row * p.Hq + head;
  const bool idle = ok && len == 0;
  const int h = head / p.g, jq = head - h * p.g;
  // the shared tokens' parts
  int first = 0, n_shared = 0;
  int64_t y = 0;
  if (ok && !idle && view.tokens > 0) {
    const int64_t col = (int64_t)(row - view.first) * p.g + jq;
    const EvenUnits e((int64_t)(view.end - view.first) * p.g, p.Hkv, view.tokens, D, j.shared_ctas);
    e.find(col / kPromptRows * p.Hkv + h, first, n_shared);
    y = col % kPromptRows;
  }
  pdl_wait();
  if (view.tokens < 0 && blockIdx.x == 0 && threadIdx.x == 0) flag(p.status, KVRP_DEV_BAD_LENGTH);
  if (!ok || head >= p.Hq) return;   // bad sequences are flagged by the own tokens' pass
  if (idle) {   // a place of the batch that is free
    const int end = p.seqs.row_start ? p.seqs.row_start[s + 1] : s + 1;
    if (row < row0 || row >= end) return;
    *reinterpret_cast<uint2*>(p.out + at * D + 4 * f) = make_uint2(0, 0);
    if (p.lse && f == 0) p.lse[at] = -INFINITY;
    return;
  }
  if (row < row0 || row >= row0 + rows) return;
  // the own tokens'
  int2 own = make_int2(0, 0);
  int64_t own_y = 0;
  if (j.few) {
    const int in_run = (row - row0) % p.max_rows;
    own = p.found[(int64_t)(row - in_run) * p.n_grp + h / p.hg];
    own_y = (h % p.hg) * p.max_rows * p.g + in_run * p.g + jq;
  }
  const int n = n_shared + max(own.y, 1);
  const auto entry = [&](int x) -> const float* {
    if (x < n_shared) return n_shared == 1 ? j.shared_dense + at * kStep
                                           : j.shared + ((int64_t)((first + x) * 2 + (x == 0 ? 1 : 0)) * kPromptRows + y) * kStep;
    x -= n_shared;
    return own.y == 0 ? p.dense + at * kStep : p.partial + ((int64_t)((own.x + x) * 2 + (x == 0 ? 1 : 0)) * p.cols + own_y) * kStep;
  };
  float m = -INFINITY, om = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kBatch = 16;   // parts in flight
  for (int x0 = 0; x0 < n; x0 += kBatch) {
    float4 st[kBatch], v[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      st[b] = make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
      v[b] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (x0 + b < n) {
        const float* e = entry(x0 + b);
        st[b] = *reinterpret_cast<const float4*>(e + D);
        v[b] = reinterpret_cast<const float4*>(e)[f];
      }
    }
    float nm = m, no = om;
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      nm = fmaxf(nm, st[b].x);
      no = fmaxf(no, st[b].y);
    }
    const float zm = nm == -INFINITY ? 0.f : nm, zo = no == -INFINITY ? 0.f : no;   // 2^-inf = 0, and no inf - inf
    l *= ex2(m - zm);
    const float r = ex2(om - zo);
    acc = make_float4(acc.x * r, acc.y * r, acc.z * r, acc.w * r);
    m = nm;
    om = no;
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      l = fmaf(st[b].z, ex2(st[b].x - zm), l);
      const float w = ex2(st[b].y - zo);
      acc.x = fmaf(v[b].x, w, acc.x);
      acc.y = fmaf(v[b].y, w, acc.y);
      acc.z = fmaf(v[b].z, w, acc.z);
      acc.w = fmaf(v[b].w, w, acc.w);
    }
  }
  const float2 r = result_factors(m, om, l);
  const __nv_bfloat162 a = __floats2bfloat162_rn(acc.x * r.x * r.y, acc.y * r.x * r.y),
                       b = __floats2bfloat162_rn(acc.z * r.x * r.y, acc.w * r.x * r.y);
  *reinterpret_cast<uint2*>(p.out + at * D + 4 * f) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  if (p.lse && f == 0) p.lse[at] = (m + lg2(l)) * kLn2;
}

// A sequence's rows go through the kernel for few rows in runs of as many as it takes, each reading the sequence's own
// tokens again (from L2), if there are few runs; else through the kernel for many.
// 28 / 4 heads x 128: 16 sequences of 5 rows over 16000 shared tokens and 60 to 600 own, three runs, 56.3 us against
// 67.8 the other way; 32 of 8 rows over 300 to 3000 own, four runs, 100.2 against 99.2.  The rule does not know how long the
// own contexts are, which each run reads again, from memory where they do not fit L2: behind 1024 shared tokens, 16384 own
// each, 16 sequences of 4 rows, two runs, take 111 us (kv_attend_q8 139), of 6, three, 157 (139), of 8, four, 205 (139); 32 of
// 4 rows 205 (267), of 8 401 (268).
constexpr int kMostRuns = 4;
struct Runs {
  int rows;        // of a run
  int64_t count;   // runs of max_rows rows
  bool few;
};
Runs runs(int64_t max_rows, int g) {
  const int rows = (int)std::min<int64_t>(max_rows, kMaxCols / g);
  const int64_t count = (max_rows + rows - 1) / rows;
  return {rows, count, count <= kMostRuns};
}

// Up to this many bytes of shared keys and values, counted for each run of each sequence, and for up to two runs
// in all, every sequence reads them for itself (again from L2): one pass and kv_attend_q8's combine instead of
// three launches.  28 / 4 heads x 128, read by each and once: 8 sequences over 4000 shared tokens (31 MB) 19.1 and 20.5 us,
// over 12000 (94 MB) 26.2 and 25.9, 16 over 8000 (125 MB) 29.9 and 23.5, 8 over 16000 30.3 and 26.6; 2 over 64000 (125 MB)
// 36.6 and 45.6, 1 over 160000 50.8 and 84.7, 4 over 160000 91.2 and 84.5.  More runs a sequence than above do so too, if all
// that its table can hold is counted: 2 sequences of 6 rows over 16, 64 / 4 heads, 42.8 us the other way.
constexpr int64_t kEachBytes = 96 << 20;
constexpr int kEachRuns = 2, kMostEachRuns = 16;
std::atomic<int64_t> each_bytes{kEachBytes};   // tests set it

// Where things are in the workspace, in bytes.
struct Layout {
  size_t meta, found, shared, shared_dense, partial, dense, end;
};
Layout layout(int Hq, int Hkv, int D, int64_t max_rows, int64_t n_rows, int sms) {
  const auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const int g = Hq / Hkv, hg = head_group(Hkv);
  const Runs r = runs(max_rows, g);
  const bool few = r.few;
  const size_t entry = (D + 4) * sizeof(float), rows = (size_t)n_rows * Hq * entry;
  Layout l;
  l.meta = 256;   // what aligning the caller's pointer takes
  l.found = l.meta + meta_bytes(kMaxCtasPerSm * sms);
  l.shared = l.found + (few ? up((size_t)n_rows * (Hkv / hg) * sizeof(int2)) : 0);
  l.shared_dense = l.shared + up((size_t)sms * 2 * kPromptRows * entry);
  l.partial = l.shared_dense + up(rows);
  l.dense = l.partial + (few ? up((size_t)kMaxCtasPerSm * sms * 2 * hg * r.rows * g * entry)
                             : up((size_t)sms * 2 * kPromptRows * entry));   // which holds the other's at most too
  static_assert(kPromptRows >= kMaxCtasPerSm * kFewHeads * kMaxCols, "the parts of the kernel for few rows");
  l.end = l.dense + up(rows);
  return l;
}

}  // namespace

}  // namespace attend_q8
}  // namespace kvrp

using namespace kvrp;

extern "C" {

void kvrp_test_set_each_limit(int64_t bytes) { attend_q8::each_bytes = bytes < 0 ? attend_q8::kEachBytes : bytes; }

int32_t kvrp_test_even_units(int64_t pairs, int32_t heads, int32_t tokens, int32_t head_dim, int32_t most_cta,
                             const int64_t* units, int32_t n_units, const int32_t* blocks, int32_t n_blocks, int64_t* out) {
  if (pairs < 0 || pairs >= 1 << 28 || heads <= 0 || heads > 4096 || tokens < 0 || tokens > q8::kMostTokens ||
      (head_dim != 64 && head_dim != 128) || most_cta <= 0 || most_cta > attend_q8::kMaxCtas || !out || n_units < 0 ||
      n_blocks < 0 || (n_units && !units) || (n_blocks && !blocks))
    return -1;
  const attend_q8::EvenUnits e(pairs, heads, tokens, head_dim, most_cta);
  const int64_t head[] = {e.n_kv, e.parts, e.units, e.cost, e.n_cta};
  out = std::copy(head, head + 5, out);
  for (int i = 0; i < n_units; ++i, out += 2) {
    if (units[i] < 0 || units[i] >= e.units) return -1;
    int first = 0, n = 0;
    e.find(units[i], first, n);
    out[0] = first;
    out[1] = n;
  }
  for (int i = 0; i < n_blocks; ++i, out += 2) {
    if (blocks[i] < 0 || blocks[i] >= e.n_cta) return -1;
    const int in_unit = e.parts ? blocks[i] % e.parts : 0;
    out[0] = e.parts ? e.part_begin(in_unit) : e.share(blocks[i]);
    out[1] = e.parts ? e.part_begin(in_unit + 1) : e.share(blocks[i] + 1);
  }
  return 0;
}

size_t kv_attend_shared_q8_workspace_size(int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim, int32_t max_rows,
                                          int32_t n_rows) {
  if (check_heads("kv_attend_shared_q8_workspace_size", n_q_heads, n_kv_heads, head_dim) != KVRP_OK || max_rows <= 0 ||
      n_rows < max_rows)
    return 0;
  return attend_q8::layout(n_q_heads, n_kv_heads, head_dim, max_rows, n_rows, attend_q8::sm_count()).end;
}

kvrp_status kv_attend_shared_q8(const void* q, int64_t q_stride, const kvrp_seqs* seqs, const kvrp_prefix* prefix,
                                int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim, float softmax_scale,
                                const void* k_pool, const void* v_pool, const float* k_scale, const float* v_scale, void* out,
                                float* lse, void* workspace, size_t workspace_bytes, uint32_t* d_status, kvrp_stream_t stream) {
  const char* fn = "kv_attend_shared_q8";
  g_last_launches = 0;
  attend_q8::Params p;
  kvrp_status st = attend_q8::check_call(fn, q, q_stride, seqs, n_q_heads, n_kv_heads, head_dim, softmax_scale, k_pool, v_pool,
                                         k_scale, v_scale, out, lse, d_status, p);
  if (st != KVRP_OK) return st;
  if (!prefix) return fail(KVRP_ERR_INVALID_ARG, "%s: NULL prefix", fn);
  st = check_prefix(fn, prefix);
  if (st != KVRP_OK) return st;
  if (seqs->n_rows == 0) return KVRP_OK;
  const size_t need = kv_attend_shared_q8_workspace_size(n_q_heads, n_kv_heads, head_dim, p.max_rows, seqs->n_rows);
  if (!workspace || workspace_bytes < need) return fail(KVRP_ERR_WORKSPACE, "%s: workspace of %zu bytes needed", fn, need);
  st = attend_q8::check_rows(fn, p);
  if (st != KVRP_OK) return st;
  int sms = 0, smem_optin = 0;
  st = current_device_sms(&sms, &smem_optin);
  if (st != KVRP_OK) return st;
  sms = attend_q8::sm_count();   // at most what the workspace is laid out for
  const attend_q8::Runs runs = attend_q8::runs(p.max_rows, p.g);
  const bool few = runs.few;
  const attend_q8::Layout at = attend_q8::layout(n_q_heads, n_kv_heads, head_dim, p.max_rows, seqs->n_rows, sms);
  p.all_rows = p.max_rows;
  p.chunks = 1;
  uint8_t* base = reinterpret_cast<uint8_t*>(reinterpret_cast<uintptr_t>(workspace) & ~uintptr_t(255));
  p.prefix_table = prefix->block_table;
  p.prefix_length = prefix->length;
  p.prefix_pages = prefix->n_pages;
  p.n_cta = sms;
  p.cols = attend_q8::kPromptRows;

  p.meta = reinterpret_cast<int4*>(base + at.meta);
  p.found = reinterpret_cast<int2*>(base + at.found);
  p.partial = reinterpret_cast<float*>(base + at.partial);
  p.dense = reinterpret_cast<float*>(base + at.dense);
  const int64_t all_runs = (int64_t)seqs->n_seqs * runs.count, limit = attend_q8::each_bytes;
  const double pages = few ? prefix->n_pages : std::max(prefix->n_pages, seqs->table_stride);
  const double each = (double)all_runs * pages * 2 * q8::kPage * n_kv_heads * head_dim;   // past 64 bits at the ends
  if (runs.count <= attend_q8::kMostEachRuns &&
      (each <= (double)limit || (few && all_runs <= attend_q8::kEachRuns && limit > 0))) {
    p.max_rows = runs.rows;
    p.chunks = (int)runs.count;
    attend_q8::set_few(p, sms, head_dim);
    cudaError_t e = attend_q8::launch_few(p, head_dim, stream, attend_q8::kEach);
    if (e == cudaSuccess) e = attend_q8::launch_combine(p, head_dim, sms, stream);
    if (e != cudaSuccess) return fail(KVRP_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
    g_last_launches = 2;
    return KVRP_OK;
  }

  CUtensorMap kmap, vmap;
  st = encode_q8_pool(&kmap, k_pool, seqs->num_pages, n_kv_heads * head_dim, head_dim);
  if (st == KVRP_OK) st = encode_q8_pool(&vmap, v_pool, seqs->num_pages, n_kv_heads * head_dim, head_dim);
  if (st != KVRP_OK) return st;
  attend_q8::Params shared = p;
  shared.partial = reinterpret_cast<float*>(base + at.shared);
  shared.dense = reinterpret_cast<float*>(base + at.shared_dense);
  cudaError_t e = cudaSuccess;
  int launches = 0;
  if (prefix->n_pages > 0) {
    e = attend_q8::launch_prompt(kmap, vmap, shared, head_dim, stream, attend_q8::kShared);
    ++launches;
  }
  p.behind = few && launches > 0;
  if (few) {
    p.max_rows = runs.rows;
    p.chunks = (int)runs.count;
    attend_q8::set_few(p, sms, head_dim);
  }
  if (e == cudaSuccess)
    e = few ? attend_q8::launch_few(p, head_dim, stream, attend_q8::kRest)
            : attend_q8::launch_prompt(kmap, vmap, p, head_dim, stream, attend_q8::kRest);
  launches += few ? 1 : 2;

  attend_q8::Join j;
  j.p = p;
  j.shared = shared.partial;
  j.shared_dense = shared.dense;
  j.shared_ctas = shared.n_cta;
  j.few = few;
  const int items = attend_q8::kJoinThreads / (head_dim / 4);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3((unsigned)((int64_t)seqs->n_rows * ((n_q_heads + items - 1) / items)));
  cfg.blockDim = dim3(attend_q8::kJoinThreads);
  if (e == cudaSuccess)
    e = cudaLaunchKernelEx(&cfg, head_dim == 64 ? attend_q8::join_kernel<64> : attend_q8::join_kernel<128>, j);
  if (e != cudaSuccess) return fail(KVRP_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
  g_last_launches = launches + 1;
  return KVRP_OK;
}

}  // extern "C"
