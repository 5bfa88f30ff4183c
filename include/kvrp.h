/*
 * kvrp.h -- C ABI of the GB300 KV relocation + rank-m patch library (libkvrp.so).
 *
 * The operator (Kamera, gist.science/pt/paper/2606.23581, section 2 "O Operador
 * Kamera"; the Korean summary gist.science/ko/paper/2606.23581 section 2 states
 * the same) reuses a chunk B that was cached on its own, KV(B|empty), at a new
 * position after a new antecedent A:
 *
 *     KV^(B|A) = R(delta) . KV(B|empty) + U_m V_m^T
 *
 *   R(delta)   exact RoPE re-rotation of the cached keys by the position shift
 *              delta (new position - old position), rotate-half convention:
 *              feature i of a rotated head pairs with feature i + d/2 and the
 *              pair turns by delta * theta^(-2i/d).  Values are not rotated
 *              (GQA/MHA); for MLA only the 64-dim k_rope is turned and c_KV is
 *              reused byte for byte (section 2, family bullets).
 *   U_m V_m^T  rank-m conditioning patch, added after the rotation, to K and
 *              to V (each tensor has its own factor pair), or to the whole
 *              576-wide MLA row (one pair).
 *
 * The result is rounded to bf16 and written straight into a paged KV cache:
 * token t of a chunk lands at position q = dst_start + t of its sequence,
 * physical page block_table[q / 16], slot q % 16.
 *
 * Conventions shared by every entry point
 *   - bf16 data is passed as raw pointers (uint16 bit patterns).  Rows are
 *     dense: a token row of one tensor is D contiguous bf16 values, with
 *     D = n_kv_heads * head_dim (GQA/MHA) or kv_lora_dim + rope_dim (MLA).
 *   - Canonical source of one tensor: [n_layers][n_tokens][D]; layer l starts
 *     at src + l * src_layer_stride (elements).
 *   - Patch factors of one tensor: U_m [n_layers][n_tokens][rank] (token-major)
 *     and V_m [n_layers][D][rank] (feature-major); layer strides in elements.
 *     Singular values are expected to be folded into U_m.
 *   - Destination pool of one tensor: layer l at base + l * layer_stride,
 *     laid out [num_pages][16][D].  A NULL block_table means a contiguous
 *     destination (identity table: position q is row q of the layer).
 *   - Every device pointer is owned by the caller, must be 16-byte aligned
 *     (block tables: 4-byte aligned) and must stay valid until the stream work
 *     is done.  Strides and dst_start are in elements; strides must be
 *     multiples of 8 elements.
 *   - rank must be 0 or a multiple of 8 up to 128 (the factor rows are then a
 *     multiple of 16 bytes, as the TMA copies need); head_dim must be 64 or
 *     128; MLA rope_dim must be 64 and kv_lora_dim a multiple of 64.
 *   - Calls are asynchronous on `stream` (NULL = the legacy default stream).
 *     Host-detected problems are returned as kvrp_status before anything is
 *     enqueued.  Problems only the device can see are OR-ed into *d_status
 *     (optional, device memory, read it after synchronising):
 *     KVRP_DEV_BAD_PAGE: a block-table entry was outside [0, num_pages); the
 *     rows of that page were skipped.  KVRP_DEV_TIMEOUT: an internal pipeline
 *     wait gave up (it is bounded); the output is incomplete.
 *   - Destination slots written by one call must not overlap (a bijective
 *     block table); overlapping slots give an unspecified winner.  Source and
 *     destination must not overlap.
 *   - Thread safety: calls may come from several host threads.
 */
#ifndef KVRP_H
#define KVRP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t. */
typedef struct CUstream_st* kvrp_stream_t;

typedef enum kvrp_status {
  KVRP_OK = 0,
  KVRP_ERR_INVALID_ARG = 1,   /* a NULL pointer, a size or stride out of range      */
  KVRP_ERR_ALIGNMENT = 2,     /* a pointer or stride breaks the 16-byte rule        */
  KVRP_ERR_UNSUPPORTED = 3,   /* head_dim / rank / rope_dim outside the kernel's set */
  KVRP_ERR_CUDA = 4,          /* a CUDA runtime or driver call failed               */
  KVRP_ERR_WORKSPACE = 5      /* the batch workspace is missing or too small        */
} kvrp_status;

#define KVRP_DEV_BAD_PAGE 0x1u
#define KVRP_DEV_TIMEOUT 0x2u
#define KVRP_DEV_BAD_LENGTH 0x4u   /* kvrp_seqs: a sequence's rows or length out of range */
#define KVRP_DEV_NO_PAGES 0x8u     /* kv_step_tables: too few free pages for a sequence */
#define KVRP_DEV_BAD_TOKEN 0x10u   /* kv_verify_drafts: a drafted token outside the vocabulary,
                                      or a row of probabilities without weight */

/* One destination pool (one tensor). */
typedef struct kvrp_dst {
  void* base;                 /* bf16 pool; layer l at base + l * layer_stride          */
  int64_t layer_stride;       /* elements between layers (>= num_pages * 16 * D)        */
  const int32_t* block_table; /* device int32, one entry per logical page of the
                                 sequence (>= ceil((dst_start + n_tokens) / 16)); NULL
                                 = contiguous                                            */
  int32_t num_pages;          /* physical pages per layer                               */
  int32_t page_size;          /* tokens per page; must be 16                            */
  int64_t dst_start;          /* sequence position of the chunk's first token (>= 0)    */
} kvrp_dst;

/*
 * kv_relocate_patch -- one GQA/MHA chunk, all layers, K and V, one launch.
 *   K gets R(delta) + U_K V_K^T; V gets V + U_V V_V^T (section 2, GQA bullet:
 *   relocate the full keys by re-applying RoPE, patch both K and V; the MHA
 *   bullet is the same with n_kv_heads = query heads).
 *   k_src, v_src  canonical K and V, [n_layers][n_tokens][D] at src_layer_stride.
 *   rank          m; 0 = relocation only (V is then copied byte for byte).
 *   uk, vk        U_m [L][T][m] and V_m [L][D][m] of the K patch (NULL iff rank 0).
 *   uv, vv        the same for the V patch.
 *   rope_theta    RoPE base (theta_i = rope_theta^(-2i/head_dim)).
 *   delta         position shift, new minus old.
 */
kvrp_status kv_relocate_patch(
    const void* k_src, const void* v_src, int64_t src_layer_stride,
    int32_t n_layers, int32_t n_tokens, int32_t n_kv_heads, int32_t head_dim,
    int64_t delta, double rope_theta, int32_t rank,
    const void* uk, const void* vk, const void* uv, const void* vv,
    int64_t u_layer_stride, int64_t v_layer_stride,
    const kvrp_dst* k_dst, const kvrp_dst* v_dst,
    uint32_t* d_status, kvrp_stream_t stream);

/*
 * kv_relocate_patch_mrope -- kv_relocate_patch under M-RoPE, the multimodal
 * RoPE of Qwen-VL-style models, which re-rotate image and video KV with it
 * (gist.science/pt/paper/2606.17107, section 4: transplanted image KV is
 * re-rotated with M-RoPE).  The head_dim / 2 frequency pairs form three
 * consecutive sections -- temporal, height, width -- of mrope_section[0..2]
 * pairs (Qwen2.5-VL with head_dim 128: {16, 24, 24}); pair i turns by
 * delta_thw[s] * theta^(-2i/head_dim), s being the section holding i.
 *   delta_thw      host array: the (temporal, height, width) position shift.
 *   mrope_section  host array: frequency pairs per section, summing to head_dim / 2.
 *   Everything else as kv_relocate_patch.  Equal shifts give plain RoPE.
 */
kvrp_status kv_relocate_patch_mrope(
    const void* k_src, const void* v_src, int64_t src_layer_stride,
    int32_t n_layers, int32_t n_tokens, int32_t n_kv_heads, int32_t head_dim,
    const int64_t delta_thw[3], const int32_t mrope_section[3],
    double rope_theta, int32_t rank,
    const void* uk, const void* vk, const void* uv, const void* vv,
    int64_t u_layer_stride, int64_t v_layer_stride,
    const kvrp_dst* k_dst, const kvrp_dst* v_dst,
    uint32_t* d_status, kvrp_stream_t stream);

/*
 * kv_relocate_patch_mla -- one MLA chunk, all layers, one launch (section 2,
 * MLA bullet: only the decoupled 64-dim k_rope is relocated, c_KV is reused
 * byte for byte, the patch goes to both channels).
 *   src   rows [n_layers][n_tokens][kv_lora_dim + rope_dim] = c_KV ++ k_rope.
 *   u, v  U_m [L][T][m] and V_m [L][kv_lora_dim + rope_dim][m] (NULL iff rank 0).
 *   With rank 0 the c_KV part of every row is copied bit for bit.
 */
kvrp_status kv_relocate_patch_mla(
    const void* src, int64_t src_layer_stride, int32_t n_layers, int32_t n_tokens,
    int32_t kv_lora_dim, int32_t rope_dim, int64_t delta, double rope_theta,
    int32_t rank, const void* u, const void* v,
    int64_t u_layer_stride, int64_t v_layer_stride,
    const kvrp_dst* dst, uint32_t* d_status, kvrp_stream_t stream);

/* One chunk of a batch: its own source, shift, patch and destination. */
typedef struct kvrp_chunk {
  const void* k_src;          /* [n_layers][n_tokens][D] at src_layer_stride            */
  const void* v_src;
  int64_t src_layer_stride;
  int32_t n_tokens;
  int32_t rank;               /* 0 = relocation only                                    */
  int64_t delta;
  const void* uk;             /* K patch U_m [L][T][m]; NULL iff rank 0                 */
  const void* vk;             /* K patch V_m [L][D][m]                                  */
  const void* uv;             /* V patch U_m                                            */
  const void* vv;             /* V patch V_m                                            */
  int64_t u_layer_stride;
  int64_t v_layer_stride;
  kvrp_dst k_dst;
  kvrp_dst v_dst;
} kvrp_chunk;

/*
 * kv_relocate_batch -- many GQA/MHA chunks, each with its own delta and patch,
 * in ONE relocation kernel launch (section 3, the three window operations:
 * reorder under an orbit patch, sliding-window survival with R(delta) alone,
 * recall of an evicted chunk with a fresh patch).
 *   chunks      host array of n_chunks descriptors (read before the call returns).
 *   workspace   device scratch of at least kv_relocate_batch_workspace_size(n_chunks)
 *               bytes, 256-byte aligned, owned by the caller.  The call writes the
 *               launch's descriptors there on `stream` (small copy kernels carry
 *               them in their parameters, ahead of the relocation kernel); do not
 *               reuse it for another purpose until the stream work is done.  Two
 *               batch calls may share one workspace only on the same stream.
 * The workspace size covers every batch call below (GQA/MHA, M-RoPE, MLA).
 */
size_t kv_relocate_batch_workspace_size(int32_t n_chunks);

kvrp_status kv_relocate_batch(
    const kvrp_chunk* chunks, int32_t n_chunks,
    int32_t n_layers, int32_t n_kv_heads, int32_t head_dim, double rope_theta,
    void* workspace, size_t workspace_bytes,
    uint32_t* d_status, kvrp_stream_t stream);

/*
 * kv_relocate_batch_mrope -- kv_relocate_batch under M-RoPE: a window of
 * image or video chunks of a Qwen-VL-style model, each moved by its own
 * (temporal, height, width) shift, in one launch (transplanted image KV is
 * re-rotated with M-RoPE: gist.science/pt/paper/2606.17107, section 4; the
 * window operations are those of Kamera, section 3).
 *   delta_thw      host array [n_chunks][3]: chunk i turns frequency pair p by
 *                  delta_thw[3i + s] * theta^(-2p/head_dim), s being the section
 *                  of p; the chunks' own .delta fields are not read.
 *   mrope_section  host array: frequency pairs per (t, h, w) section, summing to
 *                  head_dim / 2 (Qwen2.5-VL with head_dim 128: {16, 24, 24}).
 *   Everything else as kv_relocate_batch (same workspace size).
 */
kvrp_status kv_relocate_batch_mrope(
    const kvrp_chunk* chunks, const int64_t* delta_thw, int32_t n_chunks,
    int32_t n_layers, int32_t n_kv_heads, int32_t head_dim,
    const int32_t mrope_section[3], double rope_theta,
    void* workspace, size_t workspace_bytes,
    uint32_t* d_status, kvrp_stream_t stream);

/* One MLA chunk of a batch: its own source rows, shift, patch and destination. */
typedef struct kvrp_mla_chunk {
  const void* src;            /* rows [n_layers][n_tokens][kv_lora_dim + rope_dim] = c_KV ++ k_rope */
  int64_t src_layer_stride;
  int32_t n_tokens;
  int32_t rank;               /* 0 = relocation only (c_KV copied byte for byte)       */
  int64_t delta;
  const void* u;              /* U_m [L][T][m]; NULL iff rank 0                         */
  const void* v;              /* V_m [L][kv_lora_dim + rope_dim][m]                     */
  int64_t u_layer_stride;
  int64_t v_layer_stride;
  kvrp_dst dst;
} kvrp_mla_chunk;

/*
 * kv_relocate_batch_mla -- many MLA chunks, each with its own delta and patch,
 * in one launch: the window operations of Kamera section 3 (survival by
 * R(delta) alone, recall with a fresh patch) on a DeepSeek-style cache, where
 * only the k_rope tail of each row turns and c_KV is reused byte for byte
 * (section 2, MLA bullet: survival needs only R(delta) for GQA and MLA alike).
 *   Shapes and rules per chunk as kv_relocate_patch_mla; workspace as
 *   kv_relocate_batch (kv_relocate_batch_workspace_size(n_chunks) bytes).
 */
kvrp_status kv_relocate_batch_mla(
    const kvrp_mla_chunk* chunks, int32_t n_chunks, int32_t n_layers,
    int32_t kv_lora_dim, int32_t rope_dim, double rope_theta,
    void* workspace, size_t workspace_bytes,
    uint32_t* d_status, kvrp_stream_t stream);

/*
 * kv_relocate_batch_noalloc -- kv_relocate_batch for callers that cannot
 * allocate device memory.  The pages have no counterpart of this call; it
 * exists for integration.  Some callers own no device allocator at all: a
 * plugin inside a host engine that hands out only its own tensors, or a
 * serving process whose memory pool reserved all of the GPU up front, so that
 * an extra cudaMalloc either fails or breaks the pool's accounting; others
 * cannot afford the device-wide synchronisation an allocation may cause.
 * This call takes the same chunks and does the same work in the same single
 * kernel launch, but keeps the launch's descriptors in a fixed array inside
 * the library instead of a caller workspace (small copy kernels write them
 * there from their parameters).  It calls no cudaMalloc, cudaFree,
 * cudaHostAlloc or other allocating routine.
 *   Limits: at most KVRP_NOALLOC_MAX_CHUNKS chunks; more is rejected with
 *   KVRP_ERR_INVALID_ARG before any work.  The array (about 0.55 MB) lives on
 *   every GPU that loads the library, until the process exits.
 *   Set-up: the first call on a device looks up the array's device address
 *   with cudaGetSymbolAddress (the device must be current); make that first
 *   call before any stream capture.
 *   Sharing: every call on a device uses the same array, and each call
 *   rewrites the part its kernel reads.  Calls on one stream are ordered and
 *   safe; calls that can overlap on the GPU (different streams, or several
 *   host threads) race on the array and must not be issued.
 */
#define KVRP_NOALLOC_MAX_CHUNKS 256

kvrp_status kv_relocate_batch_noalloc(
    const kvrp_chunk* chunks, int32_t n_chunks,
    int32_t n_layers, int32_t n_kv_heads, int32_t head_dim, double rope_theta,
    uint32_t* d_status, kvrp_stream_t stream);

/*
 * Patch formation -- the rank-m factors of the conditioning deficit (Kamera,
 * section 2, patch bullet: computed once, at compile time or on first reuse,
 * from one conditioned pass over [A, B] followed by an SVD that keeps the
 * top-m factors).  The conditioned pass itself belongs to the model and is
 * the caller's: this call takes its output KV(B|A) together with the
 * canonical KV(B|empty) of the same tensor and forms
 *     Delta = KV(B|A) - R(delta) KV(B|empty)      (the destination frame)
 * per layer, then factors U_m [T][m] (singular values folded in) and
 * V_m [D][m] in bf16 such that U_m V_m^T approximates Delta, ready for
 * kv_relocate_patch / _mla / _batch.  The factorisation is a randomized range
 * finder with `power_iters` power iterations, Cholesky-QR orthonormalisation
 * and an fp32 Jacobi eigensolver on the small projected problem.
 *   conditioned, canonical  device bf16 [n_layers][n_tokens][row_width], rows
 *               dense; layer l at base + l * *_layer_stride elements (0: dense
 *               layers).  Only read.
 *   rope_kind   KVRP_ROPE_HEADS: every head of rot_dim features turns (keys;
 *               row_width a multiple of rot_dim);
 *               KVRP_ROPE_NONE: nothing turns (values; rot_dim, delta, theta unused);
 *               KVRP_ROPE_MLA_TAIL: the last rot_dim features turn (MLA k_rope).
 *               rot_dim: a multiple of 4, at most 128.  row_width: a multiple of 4.
 *   delta, rope_theta  the position shift and the RoPE base, as in kv_relocate_patch.
 *   rank, oversample  m >= 1 and the range finder's extra columns p >= 0;
 *               m + p <= 96, m <= min(n_tokens, row_width).
 *   power_iters 0..8 subspace iterations (1-2 suffice for decaying spectra).
 *   omega       device fp32 [row_width][m + p], row-major: the caller's Gaussian
 *               test matrix (N(0, 1) entries), shared by all layers; only read.
 *   u_out, v_out  device bf16 U_m [L][T][m] and V_m [L][row_width][m],
 *               row-major, layer strides u/v_layer_stride elements (0: dense);
 *               V_m has orthonormal columns, U_m = Delta V_m.
 *   workspace   device scratch of at least kv_patch_form_workspace_size(...)
 *               bytes, owned by the caller, busy until the call's work on
 *               `stream` completes (no two overlapping calls may share it).
 *               Calls with their own workspaces may run concurrently on
 *               different streams (K and V of one chunk, say): the k x k
 *               solves occupy one CTA per layer, so a second call's passes
 *               fill the rest of the GPU meanwhile.
 *   d_status    optional device word; KVRP_DEV_TIMEOUT is OR-ed in if a
 *               pipeline wait of the tensor-core passes gave up (results invalid).
 * Base pointers must be 16-byte aligned.  Precision: Delta is stored in bf16
 * (rows and transposed rows), the passes over it are bf16 x bf16 tensor-core
 * products accumulated in fp32; Gram matrices, the k x k solves (shifted
 * Cholesky QR, Jacobi) and the small products run in fp32; factors are rounded
 * once to bf16.
 * Errors: INVALID_ARG, ALIGNMENT, UNSUPPORTED (sizes beyond the limits above)
 * and WORKSPACE are returned before any CUDA work is queued; CUDA if a launch
 * fails.  Asynchronous on `stream`; the result is an approximation of the
 * truncated SVD whose quality grows with p and power_iters.
 */
#define KVRP_ROPE_NONE 0
#define KVRP_ROPE_HEADS 1
#define KVRP_ROPE_MLA_TAIL 2

size_t kv_patch_form_workspace_size(int32_t n_layers, int32_t n_tokens, int32_t row_width,
                                    int32_t rank, int32_t oversample);

kvrp_status kv_patch_form(
    const void* conditioned, const void* canonical,
    int64_t cond_layer_stride, int64_t canon_layer_stride,
    int32_t n_layers, int32_t n_tokens, int32_t row_width,
    int32_t rope_kind, int32_t rot_dim, int64_t delta, double rope_theta,
    int32_t rank, int32_t oversample, int32_t power_iters, const float* omega,
    void* u_out, void* v_out, int64_t u_layer_stride, int64_t v_layer_stride,
    void* workspace, size_t workspace_bytes, uint32_t* d_status, kvrp_stream_t stream);

/*
 * Orbit patch (Kamera, section 3, reordering bullet: one patch, averaged over
 * the orderings of a cached set, serves every ordering).  Same as
 * kv_patch_form, with n_orbit conditioned caches KV(B|A_pi), each in its own
 * destination frame delta_pi, and the deficit averaged before the factorisation:
 *     Delta = (1/n) sum_pi [KV(B|A_pi) - R(delta_pi) KV(B|empty)].
 *   conditioned  host array of n_orbit device pointers (bf16, layout and
 *                layer stride as `conditioned` of kv_patch_form), only read.
 *   deltas       host array of the n_orbit position shifts.
 *   n_orbit      1..64 (UNSUPPORTED beyond).  n_orbit = 1 is kv_patch_form.
 * Other arguments, errors and precision as kv_patch_form.
 */
kvrp_status kv_patch_form_orbit(
    const void* const* conditioned, const int64_t* deltas, int32_t n_orbit,
    const void* canonical, int64_t cond_layer_stride, int64_t canon_layer_stride,
    int32_t n_layers, int32_t n_tokens, int32_t row_width,
    int32_t rope_kind, int32_t rot_dim, double rope_theta,
    int32_t rank, int32_t oversample, int32_t power_iters, const float* omega,
    void* u_out, void* v_out, int64_t u_layer_stride, int64_t v_layer_stride,
    void* workspace, size_t workspace_bytes, uint32_t* d_status, kvrp_stream_t stream);

/*
 * Decode attention over relocated, patched chunks, without writing the
 * relocated cache (the fused read-side use of the operator of Kamera, section 2:
 * a chunk cached as KV(B|empty) is read as K^ = R(delta) K + U_k V_k^T and
 * V^ = V + U_v V_v^T).  For one new query token per sequence,
 *     out[s][j] = softmax(softmax_scale * q[s][j] . K^_s) V^_s
 * over the concatenated chunks of sequence s, query head j reading KV head
 * j / (n_q_heads / n_kv_heads).  The query is rotated by R(-delta) once per
 * chunk and the key patch enters as (V_k^T q) . u_k,t, so a token costs its
 * canonical k_t, v_t and the rank-m rows u_k,t, u_v,t.
 *   q           device bf16 [n_seqs][n_q_heads][head_dim].
 *   chunks      host array of n_chunks (1..KVRP_ATTN_MAX_CHUNKS) kvrp_attn_chunk,
 *               ordered by sequence: sequence s owns chunks
 *               [seq_chunks[s], seq_chunks[s + 1]) (host array of n_seqs + 1,
 *               from 0 to n_chunks, non-decreasing).
 *   kvrp_attn_chunk.k, .v   device bf16 [n_tokens][n_kv_heads * head_dim] rows
 *               of one layer, or, with .block_table, pools [num_pages][16][row]
 *               in which token t of the chunk sits at page block_table[t / 16],
 *               slot t % 16 (a paged cache; an entry outside [0, num_pages)
 *               sets KVRP_DEV_BAD_PAGE and reads page 0 instead, the output then
 *               being undefined); .rank 0 or a multiple of 16 up to 128; .uk, .uv
 *               [n_tokens][rank], .vk, .vv [n_kv_heads * head_dim][rank] bf16
 *               (all four, or none when rank is 0); .delta the shift.
 *   head_dim    64 or 128; n_q_heads a multiple of n_kv_heads, at most 16x.
 *   out         device bf16 [n_seqs][n_q_heads][head_dim]; a sequence with no
 *               tokens gets zeros.
 *   workspace   device scratch of kv_attend_relocated_workspace_size(...) bytes
 *               (fp32 partial results and which blocks hold them); its contents
 *               need not survive between calls.  The size depends on the current
 *               device's SM count, and the call returns WORKSPACE if it is smaller
 *               than the size for the device it runs on.
 *   d_status    optional device word; KVRP_DEV_TIMEOUT is OR-ed in if an internal
 *               pipeline wait gave up (the output is then undefined).
 * Pointers 16-byte aligned.  Arithmetic fp32 on the bf16 inputs (rotation
 * angles in fp64; q, V_k^T q and the softmax weights enter the tensor-core
 * products as high + low bf16 parts), output rounded once to bf16.  Errors
 * (INVALID_ARG, ALIGNMENT, UNSUPPORTED -- also beyond 2^31 - 1 tokens in one
 * call -- and WORKSPACE) are returned before any CUDA work; CUDA on a launch
 * failure.  Asynchronous on `stream`.
 */
#define KVRP_ATTN_MAX_CHUNKS 256

typedef struct {
  const void* k;
  const void* v;
  int32_t n_tokens;
  int32_t rank;
  int64_t delta;
  const void* uk;
  const void* vk;
  const void* uv;
  const void* vv;
  const int32_t* block_table;  /* device; NULL => k, v are contiguous [n_tokens][row] */
  int32_t num_pages;           /* pages of the pool k, v point to (when block_table != NULL) */
} kvrp_attn_chunk;

size_t kv_attend_relocated_workspace_size(int32_t n_chunks, const int32_t* chunk_tokens, int32_t n_q_heads,
                                          int32_t n_kv_heads, int32_t head_dim);

kvrp_status kv_attend_relocated(
    const void* q, const kvrp_attn_chunk* chunks, int32_t n_chunks, const int32_t* seq_chunks,
    int32_t n_seqs, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
    double rope_theta, float softmax_scale, void* out,
    void* workspace, size_t workspace_bytes, uint32_t* d_status, kvrp_stream_t stream);

/*
 * Serving rows behind reused chunks.  After the chunks of a window were
 * relocated into the paged cache (Kamera, section 3), the model goes on over
 * that cache: new rows (a question, then one token at a time) are normed,
 * rotated and appended, and attend over everything before them.  kv_append
 * writes the bf16 pools of the relocation calls (one layer); kv_append_q8,
 * kv_pack_q8 and kv_attend_q8 keep the cache in 8 bits, half the bytes that a
 * decode step has to read.
 *
 * The 8-bit cache of one tensor (K or V) of one layer:
 *   data    e4m3 (float8 e4m3fn) [num_pages][16][n_kv_heads * head_dim]: the
 *           layout of the bf16 pools, one byte a value.
 *   scale   fp32 [num_pages][n_kv_heads]: one for each block, the 16 tokens x
 *           head_dim values of a (page, head).  A block stands for value * scale.
 * The calls here write scale = 2^max(-126, ceil(log2(amax / 448))), amax over
 * the block's finite values (a power of two: see kv_append_q8 on blocks that
 * grow); kv_attend_q8 reads any finite scale > 0.  Values that are not finite
 * are stored as NaN.
 *
 * kvrp_seqs -- a ragged batch of sequences over one paged cache.  The arrays
 * are on the device, so a captured graph can be replayed while they change;
 * the same kvrp_seqs serves the append and the attention of a step.
 *   row_start     int32 [n_seqs + 1], non-decreasing from >= 0 to <= n_rows:
 *                 sequence s owns the rows [row_start[s], row_start[s + 1]) of
 *                 q, k, v, out.  NULL: one row per sequence (n_rows == n_seqs).
 *   seq_lens      int32 [n_seqs]: tokens of the cache, the new rows included;
 *                 row i of sequence s is the token at position
 *                 seq_lens[s] - (rows of s) + i.  0 marks an idle place of the
 *                 batch: its rows are not appended, and attention gives zeros.
 *   block_tables  int32 [n_seqs][table_stride]: physical page of each 16
 *                 tokens; entries past ceil(seq_lens[s] / 16) are not read.
 *   max_rows      host bound on the rows of one sequence (0: n_rows); it only
 *                 chooses the kernel, see kv_attend_q8.
 * What only the device can see is OR-ed into *d_status: KVRP_DEV_BAD_LENGTH
 * (rows out of order or range, a negative length, fewer tokens than rows, more
 * tokens than the table has pages for): the sequence is skipped, its rows of
 * the outputs stay as they were; KVRP_DEV_BAD_PAGE (a table entry outside
 * [0, num_pages)): see each call.
 */
typedef struct kvrp_seqs {
  const int32_t* row_start;
  const int32_t* seq_lens;
  const int32_t* block_tables;
  int32_t n_seqs;
  int32_t n_rows;
  int32_t table_stride;
  int32_t num_pages;
  int32_t max_rows;
} kvrp_seqs;

/*
 * kv_append -- the new rows of one layer into the paged bf16 cache, in one
 * launch: per head an RMS norm of q and k (optional), the position rotation,
 * q returned, k and v written into their slots.
 *     q', k' = R(position) (w * x / sqrt(mean(x^2) + norm_eps)),  v' = v
 * in fp32, rounded once to bf16.  R is rotate-half RoPE or, with mrope_section,
 * M-RoPE; the angle position * theta^(-2i/head_dim) is formed mod 2 pi in
 * 64-bit fixed point, from a frequency of a double's precision: off by at most
 * 2^-56 turns a position, 2^-25 turns at the ends of the int32 range (theta >= 1).
 *   q, k, v      device bf16, row r at base + r * stride elements, heads
 *                contiguous [n_heads][head_dim] inside a row (so a fused
 *                projection [q | k | v] passes three pointers and one stride).
 *                Strides 0: dense rows.  q may be NULL with q_out NULL.
 *   q_norm, k_norm   device bf16 [head_dim] weights, both or neither.
 *   positions    device int32 [n_rows], or [3][n_rows] (t, h, w) with
 *                mrope_section; NULL: the cache positions (all three sections).
 *   mrope_section  host array of 3 frequency-pair counts summing to
 *                head_dim / 2, or NULL (plain RoPE).
 *   q_out        device bf16 [n_rows][n_q_heads][head_dim], dense.  May be q
 *                itself when q is dense.
 *   k_pool, v_pool   bf16 pools [num_pages][16][n_kv_heads * head_dim] of the layer.
 * A row whose page is bad (KVRP_DEV_BAD_PAGE) is left out of the pools; its q
 * row is written.  n_q_heads a multiple of n_kv_heads, at most 16 x; head_dim
 * 64 or 128.  Two sequences must not append into one page.  Pointers and row
 * strides as everywhere: 16 bytes, multiples of 8 elements.  Asynchronous on
 * `stream`; may be captured into a graph.
 */
kvrp_status kv_append(
    const void* q, const void* k, const void* v,
    int64_t q_stride, int64_t k_stride, int64_t v_stride, const kvrp_seqs* seqs,
    int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
    const void* q_norm, const void* k_norm, float norm_eps,
    double rope_theta, const int32_t* positions, const int32_t* mrope_section,
    void* q_out, void* k_pool, void* v_pool,
    uint32_t* d_status, kvrp_stream_t stream);

/*
 * kv_append_q8 -- kv_append into the 8-bit cache: k', v' are rounded once, from
 * fp32 to e4m3 under their block's scale.  A block whose first slot is among
 * the new rows starts afresh.  One that holds earlier tokens keeps the larger
 * of its scale and the new rows'; where it grows, its earlier values are
 * rounded again to the new scale (a shift by a power of two: exact but for
 * values that fall among e4m3's subnormals).  Slots past the new rows keep
 * their bytes.  Calling again with the same rows gives the same cache.
 */
kvrp_status kv_append_q8(
    const void* q, const void* k, const void* v,
    int64_t q_stride, int64_t k_stride, int64_t v_stride, const kvrp_seqs* seqs,
    int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
    const void* q_norm, const void* k_norm, float norm_eps,
    double rope_theta, const int32_t* positions, const int32_t* mrope_section,
    void* q_out, void* k_pool, void* v_pool, float* k_scale, float* v_scale,
    uint32_t* d_status, kvrp_stream_t stream);

/*
 * kv_pack_q8 -- bf16 tokens of all layers (a chunk that a relocation call just
 * wrote, or canonical rows) into the 8-bit cache, K and V in one launch.
 * Logical page i (tokens 16 i ..) goes to page block_table[i]; slots of the
 * last page past n_tokens become zero and do not count for its scale.
 *   k_src, v_src   bf16; layer l at base + l * src_layer_stride elements (0:
 *                  dense), as rows [n_tokens][D], or with src_table as pools
 *                  [src_pages][16][D] read through it (D = n_kv_heads * head_dim).
 *   k_pool, v_pool e4m3 pools, layer l at base + l * pool_layer_stride elements
 *                  (0: num_pages * 16 * D; a multiple of 16).
 *   k_scale, v_scale   layer l at base + l * scale_layer_stride (0: num_pages *
 *                  n_kv_heads).
 *   block_table    device int32 [ceil(n_tokens / 16)]; NULL: page i.
 * A bad entry of either table sets KVRP_DEV_BAD_PAGE and skips the page.
 */
kvrp_status kv_pack_q8(
    const void* k_src, const void* v_src, int64_t src_layer_stride,
    const int32_t* src_table, int32_t src_pages,
    int32_t n_layers, int32_t n_tokens, int32_t n_kv_heads, int32_t head_dim,
    void* k_pool, void* v_pool, int64_t pool_layer_stride,
    float* k_scale, float* v_scale, int64_t scale_layer_stride,
    const int32_t* block_table, int32_t num_pages,
    uint32_t* d_status, kvrp_stream_t stream);

/*
 * kv_attend_q8 -- attention of the new rows over the 8-bit cache of one layer:
 *     out[r][j] = softmax(softmax_scale * q[r][j] . K) V
 * over the tokens 0 .. position of row r (causal: the rows of a sequence are
 * its last tokens, appended before this call), query head j reading KV head
 * j / (n_q_heads / n_kv_heads).  One row a sequence is a decode step, a few are
 * a draft's verification, many a prompt behind reused chunks.
 *   q            device bf16, row r at q + r * q_stride elements (0: dense),
 *                [n_q_heads][head_dim] inside a row, rotated (kv_append_q8's q_out).
 *   k_pool, v_pool, k_scale, v_scale   the cache; only read.
 *   out          device bf16 [n_rows][n_q_heads][head_dim], dense.
 *   lse          optional device fp32 [n_rows][n_q_heads]: the natural log of the
 *                sum of exp(score), with which partial results over disjoint
 *                token sets are merged.
 *   workspace    device scratch of kv_attend_q8_workspace_size(...) bytes; its
 *                contents need not survive between calls; calls that can overlap
 *                need one each.  max_rows is kvrp_seqs.max_rows (1 without row_start,
 *                n_rows where that is 0); few and many rows need different sizes,
 *                neither always the larger.
 * An idle sequence (length 0) gets zeros and a log-sum-exp of -inf.  A sequence
 * with a bad length, or more rows than max_rows, is flagged and its rows are left as
 * they were.  A bad table entry sets KVRP_DEV_BAD_PAGE and reads as a page of
 * zeros.  Slots past a sequence's length are never used, whatever they hold; a
 * value that is NaN reaches the rows that see its token and no others.
 * rows x group up to 16 take a kernel for few rows, more one that fills tensor-core
 * tiles with rows; n_rows x n_q_heads must stay below 2^32, n_rows x group below 2^28
 * (UNSUPPORTED).  KVRP_DEV_TIMEOUT is OR-ed in if an internal pipeline wait gave up
 * (the output is then undefined).  The same call gives the same bits.  How the work is
 * split over the GPU's SMs moves the output by rounding alone: of the softmax weights to
 * f16 (2^-11 of each at most) and of sums in fp32.  With many rows, value scales more than
 * 2^12 apart cost time (about 2.3 times that of others).  Asynchronous on `stream`; may be
 * captured into a graph and replayed as lengths and tables change.
 */
size_t kv_attend_q8_workspace_size(int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim, int32_t max_rows);

kvrp_status kv_attend_q8(
    const void* q, int64_t q_stride, const kvrp_seqs* seqs,
    int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim, float softmax_scale,
    const void* k_pool, const void* v_pool, const float* k_scale, const float* v_scale,
    void* out, float* lse, void* workspace, size_t workspace_bytes,
    uint32_t* d_status, kvrp_stream_t stream);

/*
 * A context that all sequences of a batch begin with (reused chunks, a system
 * prompt), held once in the pages of the pools: token t at page
 * block_table[t / 16], slot t % 16.  Both arrays are on the device.
 *   block_table   int32 [n_pages].
 *   length        int32 [1]: its tokens, rounded down to whole pages (the rest of
 *                 an open page belongs to each sequence alone); at most 16 n_pages.
 */
typedef struct kvrp_prefix {
  const int32_t* block_table;
  const int32_t* length;
  int32_t n_pages;
} kvrp_prefix;

/*
 * kv_attend_shared_q8 -- kv_attend_q8 for a batch whose sequences all begin with
 * the prefix's tokens: those are read once for the whole batch instead of once a
 * sequence (or by each, where they are so few that this is faster).  The same result up
 * to rounding, the same arguments, and
 *   prefix       the shared tokens, in pages of the same pools.  Table entries of
 *                the sequences for these pages are not read.
 *   workspace    kv_attend_shared_q8_workspace_size(...) bytes, max_rows and n_rows
 *                those of the call (see kv_attend_q8 on max_rows).
 * The first row of a sequence has to lie behind the prefix: one that does not, or a
 * prefix longer than its table, or row_start out of order, is KVRP_DEV_BAD_LENGTH, and
 * the rows concerned stay as they were.  A prefix of no tokens, and batches of one
 * sequence, are fine.  Several prefixes: one call each, over the sequences of seqs'
 * arrays that share it (row_start may begin above 0).  Everything else, NaN, bad pages,
 * idle sequences and lse among it, is as in kv_attend_q8.  The workspace holds partial
 * results of both passes in fp32, 2 x (head_dim + 4) x 4 bytes for each (row, query
 * head) beside a fixed part: for long prompts kv_attend_q8, whose work is the same there,
 * needs less and is faster (28 / 4 heads x 128, 8 sequences of 200 rows over 16384 shared
 * tokens: 359 us, this call 416).  So it is where sequences have more than 2 x floor(16 / group)
 * rows each and long contexts of their own, which this call reads up to four times (32
 * sequences of 8 rows, 1024 shared tokens, 16384 own: 268 us, this call 401).  Rows that two
 * sequences of a row_start out of order both claim hold no meaning.
 */
size_t kv_attend_shared_q8_workspace_size(int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim, int32_t max_rows,
                                          int32_t n_rows);

kvrp_status kv_attend_shared_q8(
    const void* q, int64_t q_stride, const kvrp_seqs* seqs, const kvrp_prefix* prefix,
    int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim, float softmax_scale,
    const void* k_pool, const void* v_pool, const float* k_scale, const float* v_scale,
    void* out, float* lse, void* workspace, size_t workspace_bytes,
    uint32_t* d_status, kvrp_stream_t stream);

/*
 * kv_step_tables -- the batch of a step, built on the device: writes the arrays
 * that `seqs` points to (row_start, seq_lens, block_tables; row_start may not be
 * NULL here) from each sequence's tokens and rows, so that a captured step goes
 * on by itself while lengths, accepted drafts and sequences come and go.
 *   kept_lens    int32 [n_seqs]: tokens of the cache that stay (kv_verify_drafts'
 *                kept_lens; 0 for a place that falls free).  May be seqs->seq_lens (a
 *                sequence that cannot be served then loses its length).
 *   new_rows     int32 [n_seqs]: rows to append behind them.
 *   prefix       optional: the first pages of every sequence, owned by none.  Its
 *                length may change only while no sequence holds pages.
 *   held_pages   int32 [n_seqs]: pages that the sequence's table holds, the
 *                prefix's included; 0 for one that begins (its table then starts
 *                with the prefix's pages).  held_out: the same after the call.
 *   free_pages   int32 [num_pages]: a ring of free pages, of which
 *   free_state   int32 [2] = {head, count} says free_pages[(head + i) mod num_pages],
 *                i < count, are free.  free_state_out: the same after the call.
 *   positions    optional int32 [n_rows]: the position of each row.
 *   slots        optional int64 [n_rows]: page * 16 + slot of each row.
 * held_out and free_state_out may be their inputs; the other arrays are distinct.
 * A sequence needs ceil((kept + new) / 16) pages.  In the order of the batch,
 * sequences take what they lack from the ring's head on; what one has too much
 * goes back behind the free ones and can be taken from the next call on.  Table
 * entries past those needed keep what they held.
 *   row_start    the running sum of new_rows (at most n_rows).
 *   seq_lens     kept + new; 0 (an idle place, whose rows the other calls leave out)
 *                for a sequence that cannot be served.  It keeps its pages and table
 *                (and, kv_verify_drafts' kept_lens being an array of its own, its place);
 *                its rows get position 0 and slot -1, as do the rows behind the last
 *                sequence.
 * *d_status: KVRP_DEV_NO_PAGES, if a sequence and those before it ask for more
 * pages than are free (all those behind it that ask for any are left out too);
 * KVRP_DEV_BAD_LENGTH, for a sequence with a negative count, kept tokens that it
 * has no pages for, fewer kept tokens than the prefix, rows past n_rows, or more
 * tokens than its table has entries for, for all sequences where free_state or the
 * prefix's length is out of range, and where more pages come back than the ring
 * has places for (those past its end are lost and not counted); KVRP_DEV_BAD_PAGE, where a page written or given back is
 * outside [0, num_pages) (it goes where it belongs all the same; a row on it gets
 * slot -1).  n_seqs x table_stride must stay below 2^31 (UNSUPPORTED).
 * Asynchronous on `stream`; may be captured into a graph.
 */
kvrp_status kv_step_tables(
    const int32_t* kept_lens, const int32_t* new_rows, const kvrp_seqs* seqs, const kvrp_prefix* prefix,
    const int32_t* held_pages, int32_t* held_out,
    int32_t* free_pages, const int32_t* free_state, int32_t* free_state_out,
    int32_t* positions, int64_t* slots, uint32_t* d_status, kvrp_stream_t stream);

/*
 * kv_verify_drafts -- which drafted tokens of a step stay, and the token after
 * the last one that does.  Sequence s owns the rows of kvrp_seqs: its first row is
 * its last token, each row after that a draft; row r of `target` (and `draft`) holds
 * the probabilities of the token that follows row r's.  The drafts are taken in turn:
 *   draft tokens[r + 1] stays while   u_accept[r] * draft[r][token] < target[r][token]
 * and at the first row a whose draft does not, or that has none, a token is drawn:
 *   weight of i = the positive part of w(target[a][i]) - w(draft[a][i]) where a draft
 *                 was turned down, and w(target[a][i]) where there was none or no
 *                 positive part is left;   w(x) = floor(2^40 x), x in [0, 1]
 *   token       = the first i at which the weights' running sum passes
 *                 floor(floor(2^32 u_sample[s]) * (their sum) / 2^32)
 * so that with independent uniform numbers the tokens are distributed as the target's
 * own.  Weights and sums are whole numbers: the token does not depend on how the sum
 * is split up.  The comparison is exact too (64-bit products of the 32-bit values).
 *   target, draft   device, row r at base + r * stride elements (0: vocab), of
 *                 prob_type KVRP_F32 or KVRP_BF16.  Values below 0 and NaN weigh
 *                 nothing, values above 1 as 1.  A sequence's last row of `draft` is not
 *                 read.  draft NULL: the drafts are certain (looked up, not drawn), that
 *                 is draft[r][i] = 1 at the drafted token and 0 elsewhere.
 *   tokens        device int32 [n_rows]; u_accept, u_sample   device fp32 [n_rows],
 *                 [n_seqs], in [0, 1).
 *   out_tokens    device int32 [n_rows], apart from all other arrays: from each sequence's first row on the drafts that
 *                 stay, the drawn token, then -1.
 *   accepted      optional device int32 [n_seqs]: how many drafts stay.
 *   kept_lens     optional device int32 [n_seqs]: seq_lens without the rows turned down
 *                 (the cache then holds all tokens but the drawn one).  May be
 *                 seqs->seq_lens.
 * An idle sequence (length 0) gets -1 in its rows and 0 accepted, and its kept_lens stays
 * as it was: one that kv_step_tables had no pages for goes on where it stood once there
 * are some.  One without rows gets 0, and its length.  A sequence with a bad length is flagged (KVRP_DEV_BAD_LENGTH) and its
 * outputs stay as they were.  KVRP_DEV_BAD_TOKEN: a drafted token outside [0, vocab)
 * (it is turned down), or a row without weight (the token is -1).  block_tables and
 * num_pages of `seqs` are not used beyond its checks.  vocab up to 2^22.  Pointers 4-byte
 * aligned (bf16 probabilities 2); rows that begin on 16 bytes are read fastest.
 * Asynchronous on `stream`; may be captured into a graph.
 */
#define KVRP_F32 0
#define KVRP_BF16 1

kvrp_status kv_verify_drafts(
    const void* target, int64_t target_stride, const void* draft, int64_t draft_stride, int32_t prob_type,
    int32_t vocab, const kvrp_seqs* seqs, const int32_t* tokens, const float* u_accept, const float* u_sample,
    int32_t* out_tokens, int32_t* accepted, int32_t* kept_lens, uint32_t* d_status, kvrp_stream_t stream);

/*
 * kvrp_test_set_wait_limit -- for tests of the failure path only.  Sets the
 * limit, in SM clock cycles, of the relocation kernel's pipeline waits in the
 * plans built from now on by any thread, and of kv_attend_q8's kernel for many
 * rows (and kv_attend_shared_q8's) in the calls from now on (0 restores the default
 * of about one second).  With a limit of a few hundred cycles the waits give up almost
 * at once: the launch then ORs KVRP_DEV_TIMEOUT into *d_status, lets its copies
 * and tensor-core work drain, frees its TMEM and returns, leaving the output
 * incomplete.  It never hangs the GPU, whatever the limit.
 */
void kvrp_test_set_wait_limit(uint32_t cycles);

/*
 * kvrp_test_set_each_limit -- for tests only.  Sets how many bytes of shared keys and
 * values (counted once a sequence) kv_attend_shared_q8 lets each sequence read for
 * itself, in the calls from now on by any thread: 0 none (nor any alone), so that the
 * small cases of a test take the shared pass too; below 0 restores the library's own.
 */
void kvrp_test_set_each_limit(int64_t bytes);

/*
 * kvrp_test_even_units -- for tests of the host-side planning only; no CUDA call.  How
 * kv_attend_shared_q8's pass over `tokens` shared tokens divides itself among at most
 * most_cta blocks, for `pairs` (row, query head) pairs of each of `heads` KV heads:
 *   out[0..4]  token tiles of a unit, parts of a unit (0: shares), units, a unit's cost, blocks;
 * then for each of the n_units numbers in `units` the first block with tiles of that unit
 * and how many have some; then for each of the n_blocks numbers in `blocks` where that block's
 * share begins and ends, in the costs of all units, or, where units are cut into parts, the first
 * tile of its part and the one behind the last.  out holds 5 + 2 n_units + 2 n_blocks numbers.
 * Returns 0, or -1 on invalid arguments (numbers out of range among them).
 */
int32_t kvrp_test_even_units(int64_t pairs, int32_t heads, int32_t tokens, int32_t head_dim, int32_t most_cta,
                             const int64_t* units, int32_t n_units, const int32_t* blocks, int32_t n_blocks, int64_t* out);

/*
 * kvrp_test_attend_split -- for tests of the host-side planning only; no CUDA
 * call.  The work split kv_attend_relocated gives n_cta blocks for chunks of
 * these token counts and ranks (host arrays of n_chunks): the stage sequence
 * (head group, chunk, stage) cut into contiguous shares of about equal bytes,
 * counting each stage's K, V and factor rows and each segment's V_k, query and
 * V_v slots.  Writes the boundaries share0[0 .. count] (share0 holds n_cta + 1
 * entries) and returns count (<= n_cta, every share non-empty), 0 when no chunk
 * has tokens, -1 on an invalid argument.  The other arguments are those of
 * kv_attend_relocated.
 */
int32_t kvrp_test_attend_split(const int32_t* chunk_tokens, const int32_t* chunk_ranks, int32_t n_chunks,
                               int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim, int32_t n_cta,
                               int32_t* share0);

/* Human-readable name of a status code (static string). */
const char* kvrp_status_string(kvrp_status status);

/* Text of the last error seen by this host thread (static per thread). */
const char* kvrp_last_error(void);

/* Kernel launches that this host thread's last relocation call (kv_relocate_*),
 * attention call (kv_attend_*), append, pack, step tables or verification enqueued.  Relocation: the relocation
 * kernel, plus for a batch the small copy launches that carry its launch plan to
 * the device (31 KB of plan each).  Attention: the block and combine kernels (2;
 * the combine alone when no chunk has tokens); kv_attend_shared_q8 2 where little is
 * shared, else 3, with more than 4 x floor(16 / group) rows a sequence 4 (3 where the
 * prefix has no pages).  Append, pack and draft verification: 1.
 * Step tables: 1, or 2 for many rows.  0 when the
 * call returned an error or had nothing to move. */
int32_t kvrp_last_launch_count(void);

/* Library version, major * 10000 + minor * 100 + patch. */
int32_t kvrp_version(void);

#ifdef __cplusplus
}
#endif

#endif /* KVRP_H */
