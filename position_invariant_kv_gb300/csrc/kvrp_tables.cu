// The batch of a step built on the device (kv_step_tables): row starts, lengths, block tables,
// positions and slots from each sequence's kept tokens and new rows.
//
//   need_s   = ceil((kept_s + new_s) / 16) pages, of which it holds held_s and the first
//              `shared` are the batch's common ones
//   takes_s  = max(0, need_s - max(held_s, shared))          from the ring of free pages
//   offset_s = sum of takes_j, j < s:    page i of them is ring[(head + offset_s + i) mod size]
//   gives_s  = max(0, held_s - max(need_s, shared))          to the ring, behind the free ones
//
// A sequence is served if the ring holds offset_s + takes_s pages, so whether one is depends on
// those before it alone and nothing is searched for.  All of it is whole numbers and prefix sums.
//
// Bound by latency: the inputs of 64 sequences are 1 KB.  A block takes 512 sequences at a time,
// one a thread, and scans them; rows and table entries are then flat lists that its threads share
// evenly however uneven the sequences are, each entry finding its sequence by bisection in shared
// memory.  Small calls are one block, which fills and then moves the state on.  Large ones (prompts)
// are two launches: blocks over the whole GPU, each scanning all sequences again (cheaper than a
// third launch), fill tables, positions, slots and the ring's end; the second launch, one block, moves
// lengths, pages held and the ring's state on, which the first still reads.
//
// Measured: 64 sequences of 5 rows 5.2 us, of which a launch is half and the rest three dependent trips to
// memory; 48 places, prompts of 37 to 6000 rows (47000) behind 1024 shared pages 8.2 us; 3000 sequences, half of them
// beginning behind 1024 shared pages, a third ending, 41 us: six rounds of 512 in each of two launches.  What comes back
// is not counted when the launches are chosen: in a step of few rows one block moves it all, a third of 500 sequences
// of 250 pages 46 us, of 3000 sequences 249 us (20 where none ends).
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cstring>

#include "kvrp.h"
#include "kvrp_plan.h"
#include "kvrp_ptx.h"
#include "kvrp_q8.h"

namespace kvrp {
namespace tables {

using namespace kvrp::ptx;
using q8::flag;
using q8::kPage;

constexpr int kThreads = 512, kWarps = kThreads / 32;

struct Params {
  const int32_t *kept, *fresh;          // tokens kept, rows new
  const int32_t* held;
  int32_t* held_out;
  int32_t *row_start, *seq_lens, *table;
  int32_t* ring;                        // read from head on, written behind the free ones: never the same places
  const int32_t* state;
  int32_t* state_out;
  const int32_t *prefix_table, *prefix_length;
  int32_t* positions;
  int64_t* slots;
  uint32_t* status;
  int n_seqs, n_rows, stride, num_pages, prefix_pages;
};

// What a sequence of the block's 512 has to do.
struct Counts {
  int kept, fresh, held;
};
struct Plan {
  int length, need, held;
  int take0;          // pages that the sequences before it take
  int from;           // its first page that is its own: max(held, shared)
};
struct Smem {
  int64_t rows[kWarps];
  int takes[kWarps], entries[kWarps], gives[kWarps], taken[kWarps];
  int row_end[kThreads];    // of the batch's rows, at most n_rows
  int entry_end[kThreads];  // of the block's new table entries,
  int give_end[kThreads];   // of the pages given back
  Plan plan[kThreads];
  uint8_t served[kThreads];
};

template <typename T>
__device__ __forceinline__ T warp_scan(T v) {   // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  return v;
}
// The first of the block's ascending ends that is above x (x is below the last).
__device__ __forceinline__ int above(const int* end, int x) {
  int at = 0;
#pragma unroll
  for (int step = kThreads / 2; step > 0; step >>= 1)
    if (end[at + step - 1] <= x) at += step;
  return at;
}
__device__ __forceinline__ int ring_at(int head, int i, int size) {   // head, i < size
  const int64_t at = (int64_t)head + i;
  return (int)(at < size ? at : at - size);
}

// kFill: table entries, positions, slots, pages into the ring.  kApply: row starts, lengths, pages held, the ring's state.
template <bool kFill, bool kApply>
__global__ void __launch_bounds__(kThreads) tables_kernel(const __grid_constant__ Params p) {
  __shared__ Smem sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, size = p.num_pages;
  const int worker = blockIdx.x * kThreads + tid, workers = gridDim.x * kThreads;
  if constexpr (kFill) {
    pdl_wait();
    pdl_launch_dependents();
  }
  // (Without kFill this is the second launch: what it reads here was there before the first one began.)
  int head = __ldcg(p.state), count = __ldcg(p.state + 1), shared = 0;
  bool usable = head >= 0 && head < size && count >= 0 && count <= size;
  if (!usable) head = count = 0;
  if (p.prefix_length) {
    const int length = __ldcg(p.prefix_length);
    shared = length >> 4;
    if (length < 0 || shared > p.prefix_pages) usable = false, shared = 0;
  }
  if (kApply && tid == 0 && !usable) flag(p.status, KVRP_DEV_BAD_LENGTH);
  if constexpr (!kFill) {
    pdl_wait();   // the first launch has read what changes from here on
    pdl_launch_dependents();
  }
  // A page of a sequence that it does not hold yet.
  const auto page_of = [&](int at, const Plan& q) {
    return at < shared ? p.prefix_table[at] : p.ring[ring_at(head, q.take0 + at - q.from, size)];
  };

  int64_t rows0 = 0;           // of the sequences before the block's
  int64_t asked0 = 0;          // pages asked for by them
  int64_t took = 0, gave = 0;  // pages taken and given back by them
  const auto counts = [&](int s) {
    return s < p.n_seqs ? Counts{__ldcg(p.kept + s), __ldcg(p.fresh + s), __ldcg(p.held + s)} : Counts{0, 0, 0};
  };
  Counts next = counts(tid);
  for (int s0 = 0; s0 < p.n_seqs; s0 += kThreads) {
    const int s = s0 + tid, kept = next.kept, fresh = next.fresh, held = next.held;
    next = counts(s + kThreads);   // those of the sequences after, meanwhile
    const int64_t rows = max(fresh, 0), length = (int64_t)kept + fresh;
    bool fine = usable && kept >= 0 && fresh >= 0 && held >= 0 && held <= p.stride && (held == 0 || held >= shared) &&
                length <= q8::kMostTokens && length <= (int64_t)p.stride * kPage;
    // tokens are kept in pages that are held or shared, and no row goes into a shared page
    if (fine && length > 0) fine = kept >= shared * kPage && kept <= (int64_t)max(held, shared) * kPage;
    const int need = fine ? (int)((length + kPage - 1) / kPage) : 0, from = max(held, shared);
    const int64_t row_sum = warp_scan(rows);
    if (lane == 31) sh.rows[warp] = row_sum;
    __syncthreads();
    const int64_t block_row = min(rows0, (int64_t)p.n_rows);   // the rows of these sequences
    int64_t row_end = rows0 + row_sum;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) row_end += sh.rows[w];
      rows0 += sh.rows[w];
    }
    const int64_t end_row = min(rows0, (int64_t)p.n_rows);
    if (row_end > p.n_rows) fine = false;
    const int takes = fine && need > from ? need - from : 0;
    const int entries = fine && need > held ? need - held : 0;
    const int take_sum = warp_scan(takes), entry_sum = warp_scan(entries);
    if (lane == 31) sh.takes[warp] = take_sum, sh.entries[warp] = entry_sum;
    __syncthreads();
    int64_t upto = asked0 + take_sum;
    int entry_end = entry_sum, entry_total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) upto += sh.takes[w], entry_end += sh.entries[w];
      asked0 += sh.takes[w];
      entry_total += sh.entries[w];
    }
    const bool served = fine && (takes == 0 || upto <= count);
    const int gives = served && held > max(need, shared) ? held - max(need, shared) : 0, taken = served ? takes : 0;
    const int give_sum = warp_scan(gives), taken_sum = warp_scan(taken);
    if (lane == 31) sh.gives[warp] = give_sum, sh.taken[warp] = taken_sum;
    sh.row_end[tid] = (int)min(row_end, (int64_t)p.n_rows);
    sh.entry_end[tid] = entry_end;
    sh.plan[tid] = {(int)length, need, held, (int)min(upto - takes, (int64_t)size), from};
    sh.served[tid] = served;
    __syncthreads();
    int give_end = give_sum, give_total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) give_end += sh.gives[w];
      give_total += sh.gives[w];
      took += sh.taken[w];
    }

    if constexpr (kFill) {
      for (int64_t e = worker; e < entry_total; e += workers) {   // new table entries
        const int x = above(sh.entry_end, (int)e);
        const Plan q = sh.plan[x];
        if (!sh.served[x]) continue;
        const int at = q.need - (sh.entry_end[x] - (int)e);
        const int page = page_of(at, q);
        if (page < 0 || page >= size) flag(p.status, KVRP_DEV_BAD_PAGE);
        p.table[(int64_t)(s0 + x) * p.stride + at] = page;
      }
      if (p.positions || p.slots) {
        for (int64_t r = block_row + worker; r < end_row; r += workers) {
          const int x = above(sh.row_end, (int)r);
          const Plan q = sh.plan[x];
          int at = 0;
          int64_t slot = -1;
          if (sh.served[x]) {
            at = q.length - (sh.row_end[x] - (int)r);
            const int page = at / kPage < q.held ? p.table[(int64_t)(s0 + x) * p.stride + at / kPage] : page_of(at / kPage, q);
            if (page < 0 || page >= size) flag(p.status, KVRP_DEV_BAD_PAGE);
            else slot = (int64_t)page * kPage + at % kPage;
          }
          if (p.positions) p.positions[r] = at;
          if (p.slots) p.slots[r] = slot;
        }
      }
      if (give_total > 0) {   // the ring's places behind the free pages: nobody reads them in this call
        sh.give_end[tid] = give_end;
        __syncthreads();
        for (int64_t e = worker; e < give_total; e += workers) {
          const int x = above(sh.give_end, (int)e);
          const Plan q = sh.plan[x];
          const int page = p.table[(int64_t)(s0 + x) * p.stride + q.held - (sh.give_end[x] - (int)e)];
          if (page < 0 || page >= size) flag(p.status, KVRP_DEV_BAD_PAGE);
          const int64_t place = gave + e;   // a ring that the pages would pass the end of loses them
          if (place < size - count) p.ring[ring_at(head, count + (int)place, size)] = page;
          else flag(p.status, KVRP_DEV_BAD_LENGTH);
        }
      }
    }
    gave += give_total;
    if constexpr (kApply) {
      if (s < p.n_seqs) {
        if (!fine) flag(p.status, KVRP_DEV_BAD_LENGTH);
        else if (!served) flag(p.status, KVRP_DEV_NO_PAGES);
        p.row_start[s + 1] = (int)min(row_end, (int64_t)p.n_rows);
        p.seq_lens[s] = served ? (int)length : 0;
        p.held_out[s] = served ? need : held;
      }
    }
    __syncthreads();
  }
  if constexpr (kFill) {   // rows behind the last sequence have no slot
    for (int64_t r = min(rows0, (int64_t)p.n_rows) + worker; r < p.n_rows; r += workers) {
      if (p.positions) p.positions[r] = 0;
      if (p.slots) p.slots[r] = -1;
    }
  }
  if (kApply && tid == 0) {
    p.row_start[0] = 0;
    if (usable) {
      p.state_out[0] = ring_at(head, (int)took, size);
      // Pages that the ring had no place for are lost: counted, they would stand for places whose pages have just been taken.
      p.state_out[1] = (int)(count - took + min(gave, (int64_t)size - count));
    } else {
      const int a = __ldcg(p.state), b = __ldcg(p.state + 1);
      p.state_out[0] = a;
      p.state_out[1] = b;
    }
  }
}

// Rows and likely table entries up to which one block does a call: beyond it two launches.
constexpr int64_t kOneBlock = 8192;

}  // namespace tables

kvrp_status check_prefix(const char* fn, const kvrp_prefix* x) {
  if (!x->length || (!x->block_table && x->n_pages)) return fail(KVRP_ERR_INVALID_ARG, "%s: NULL in prefix", fn);
  if (x->n_pages < 0 || x->n_pages > INT32_MAX / q8::kPage)
    return fail(KVRP_ERR_INVALID_ARG, "%s: prefix n_pages out of range", fn);
  if (reinterpret_cast<uintptr_t>(x->length) % 4 || reinterpret_cast<uintptr_t>(x->block_table) % 4)
    return fail(KVRP_ERR_ALIGNMENT, "%s: a 4-byte array of prefix is not aligned", fn);
  return KVRP_OK;
}

}  // namespace kvrp

using namespace kvrp;

extern "C" kvrp_status kv_step_tables(const int32_t* kept_lens, const int32_t* new_rows, const kvrp_seqs* seqs,
                                      const kvrp_prefix* prefix, const int32_t* held_pages, int32_t* held_out,
                                      int32_t* free_pages, const int32_t* free_state, int32_t* free_state_out,
                                      int32_t* positions, int64_t* slots, uint32_t* d_status, kvrp_stream_t stream) {
  const char* fn = "kv_step_tables";
  g_last_launches = 0;
  kvrp_status st = check_seqs(fn, seqs);
  if (st != KVRP_OK) return st;
  if (prefix) st = check_prefix(fn, prefix);
  if (st != KVRP_OK) return st;
  if (!seqs->row_start) return fail(KVRP_ERR_INVALID_ARG, "%s: row_start is written and cannot be NULL", fn);
  if (!kept_lens || !new_rows || !held_pages || !held_out || !free_pages || !free_state || !free_state_out)
    return fail(KVRP_ERR_INVALID_ARG, "%s: NULL argument", fn);
  for (const void* x : {(const void*)kept_lens, (const void*)new_rows, (const void*)held_pages, (const void*)held_out,
                        (const void*)free_pages, (const void*)free_state, (const void*)free_state_out, (const void*)positions,
                        (const void*)d_status})
    if (reinterpret_cast<uintptr_t>(x) % 4) return fail(KVRP_ERR_ALIGNMENT, "%s: a 4-byte array is not aligned", fn);
  if (reinterpret_cast<uintptr_t>(slots) % 8) return fail(KVRP_ERR_ALIGNMENT, "%s: slots is not 8-byte aligned", fn);
  if ((int64_t)seqs->n_seqs * seqs->table_stride > INT32_MAX)
    return fail(KVRP_ERR_UNSUPPORTED, "%s: n_seqs x table_stride must stay below 2^31", fn);
  int sms = 0, smem_optin = 0;
  st = current_device_sms(&sms, &smem_optin);
  if (st != KVRP_OK) return st;

  tables::Params p;
  std::memset(&p, 0, sizeof(p));
  p.kept = kept_lens;
  p.fresh = new_rows;
  p.held = held_pages;
  p.held_out = held_out;
  p.row_start = const_cast<int32_t*>(seqs->row_start);
  p.seq_lens = const_cast<int32_t*>(seqs->seq_lens);
  p.table = const_cast<int32_t*>(seqs->block_tables);
  p.ring = free_pages;
  p.state = free_state;
  p.state_out = free_state_out;
  if (prefix) {
    p.prefix_table = prefix->block_table;
    p.prefix_length = prefix->length;
    p.prefix_pages = prefix->n_pages;
  }
  p.positions = positions;
  p.slots = slots;
  p.status = d_status;
  p.n_seqs = seqs->n_seqs;
  p.n_rows = seqs->n_rows;
  p.stride = seqs->table_stride;
  p.num_pages = seqs->num_pages;

  // A sequence that begins copies the shared pages, 16 entries in the time of a row's bisection.
  const int64_t load = (int64_t)p.n_rows + (int64_t)p.n_seqs * p.prefix_pages / 16;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(tables::kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e;
  if (load <= tables::kOneBlock) {
    e = cudaLaunchKernelEx(&cfg, tables::tables_kernel<true, true>, p);
  } else {
    cfg.gridDim = dim3((unsigned)std::min<int64_t>(sms, (load + tables::kThreads - 1) / tables::kThreads));
    e = cudaLaunchKernelEx(&cfg, tables::tables_kernel<true, false>, p);
    cfg.gridDim = dim3(1);
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, tables::tables_kernel<false, true>, p);
  }
  if (e != cudaSuccess) return fail(KVRP_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
  g_last_launches = load <= tables::kOneBlock ? 1 : 2;
  return KVRP_OK;
}
