/*
 * mla_decode.h — C ABI of the GB300 (sm_103a) MLA decode library.
 *
 * Multi-head Latent Attention decoding over a paged latent KV cache.  Every
 * query head attends to one shared latent KV head: a cached row of
 * d = 576 bf16 values (512 latent + 64 decoupled-RoPE dims) serves as the key,
 * and its first dv = 512 dims as the value.  Pages hold 64 tokens and are
 * addressed through a per-sequence block table.
 *
 * Sources for the operations declared here:
 *  - "Novita AI, H100 및 H200에서 FlashMLA 평가", section "MLA란 무엇인가요?",
 *    table "MHA vs MQA vs GQA vs MLA": all heads share a compressed latent KV
 *    vector per token, with RoPE decoupled.
 *  - "FlashMLA란 무엇인가?" (topnet.top article 5338), section "FlashMLA의 주요
 *    특성": bf16 and a paged KV cache with block size 64.
 *  - same page, section "FlashMLA 설치 및 사용":
 *      step 2 "MLA 메타데이터 가져오기": get_mla_metadata(cache_seqlens,
 *        s_q * h_q // h_kv, h_kv) -> (tile_scheduler_metadata, num_splits),
 *        computed once and reused by every layer;
 *      step 3 "MLA 디코딩 실행": flash_mla_with_kvcache(q, kvcache, block_table,
 *        cache_seqlens, dv, tile_scheduler_metadata, num_splits, causal)
 *        -> (o, lse).
 *  - same page, section "FlashMLA의 기술 구현" ("병렬 디코딩"): several query
 *    tokens per step, read here as s_q > 1 with a causal mask: query i of a
 *    sequence of length T sees cached positions < T - s_q + i + 1.
 *
 * Conventions for every call:
 *  - Pointers marked "device" are CUDA device pointers on the current device;
 *    the caller allocates, owns and frees them.  The library never allocates,
 *    frees or retains caller memory and keeps no per-call state.
 *  - `stream` is a CUDA stream (cudaStream_t / CUstream; NULL = legacy default).
 *    Calls that launch work enqueue it on `stream` and return without waiting.
 *  - Return value: MLA_OK (0) or a negative MLA_ERR_* code.  Arguments are
 *    validated on the host before anything is launched; on an argument error
 *    nothing is launched and no output is touched.
 *  - bf16 tensors are raw IEEE bfloat16 bit patterns (2 bytes per element),
 *    row-major and densely packed in the shapes given.
 *  - The library looks up the device addresses of its own device arrays (the
 *    status word, the scratch of mla_decode_kvcache_noalloc) once per device
 *    and keeps them for the life of the process.  cudaDeviceReset invalidates
 *    them: do not call the library on a device after resetting it in the same
 *    process.
 *
 * Supported on the GPU path: d = 576 or 512 (bf16 cache) or 576 (packed
 * e4m3 cache, mla_decode_kvcache_fp8), dv = 512, page size 64,
 * h_kv = 1, any batch >= 1, any s_q >= 1 and h_q >= 1 with
 * s_q * h_q <= 65536.  d = 512 is the d_qk = 512 variant that the
 * "[FlashInfer] ... SM120 sparse MLA" page names for DSv4, read as a
 * 512-dim cached row that is both key and value (no separate RoPE part).
 * Other shapes return MLA_ERR_UNSUPPORTED.
 */
#ifndef MLA_DECODE_H
#define MLA_DECODE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st;

#if defined(__GNUC__)
#define MLA_API __attribute__((visibility("default")))
#else
#define MLA_API
#endif

/* status codes */
#define MLA_OK 0
#define MLA_ERR_INVALID_ARG (-1)   /* null pointer, negative size, inconsistent shapes */
#define MLA_ERR_UNSUPPORTED (-2)   /* shape or device outside what the GPU path implements */
#define MLA_ERR_WORKSPACE (-3)     /* workspace smaller than mla_workspace_bytes() */
#define MLA_ERR_CUDA (-4)          /* a CUDA runtime call or kernel launch failed */
#define MLA_ERR_DEVICE (-5)        /* a kernel reported an error (see mla_device_status) */

/* fixed shape constants of the GPU path */
#define MLA_PAGE_SIZE 64
#define MLA_HEAD_DIM 576
#define MLA_V_DIM 512
#define MLA_METADATA_INTS 8
#define MLA_TILE_ROWS 128  /* query rows of one tensor-core tile */
#define MLA_PREFILL_HEAD_DIM 128  /* dims of a prompt's heads, RoPE dims apart */
/* fixed cost of one split-KV segment, in pages, used by the work partition */
#define MLA_SCHED_FIXED_COST_PAGES 8
/* cost, in pages, that the partition charges for needing the combine pass */
#define MLA_SCHED_COMBINE_COST_PAGES 4
/* the same two costs for the sparse decode, in 64-entry list chunks: a list
   chunk's row gathers take about four times a dense page, so the per-segment
   costs come to a quarter or less (measured on GB300: topk 2048 over b = 64
   sequences, split + combine 170 us with the dense costs, 156 us with a
   fixed cost of 2 chunks, 153 us with 1) */
#define MLA_SCHED_SPARSE_FIXED_COST_CHUNKS 1
#define MLA_SCHED_SPARSE_COMBINE_COST_CHUNKS 1
/* largest cost mla_get_metadata_costs accepts */
#define MLA_SCHED_MAX_COST (1 << 20)

/* device-side error bits reported through mla_device_status() */
#define MLA_DEVERR_TIMEOUT 0x1     /* a bounded wait inside a kernel gave up */
#define MLA_DEVERR_BLOCK_ID 0x2    /* a block_table entry was outside [0, num_blocks) */
#define MLA_DEVERR_SEQLEN 0x4      /* a cache_seqlens entry was negative or beyond the table */
#define MLA_DEVERR_SCALE 0x8       /* an e4m3 page held a scale with |c| >= 255 (or NaN) for a token
                                      inside its sequence (mla_decode_kvcache_fp8) */

/*
 * mla_num_sm_parts — number of split-KV work parts for one decode call.
 *
 * Host-only query.  The caller uses it to size tile_scheduler_metadata
 * ([num_parts * MLA_METADATA_INTS] int32) before mla_get_metadata.
 *   device      CUDA device ordinal the decode will run on
 *   num_q_rows  query rows per KV head: s_q * h_q / h_kv (the pages' second
 *               argument of get_mla_metadata)
 *   h_kv        KV heads (must be 1)
 *   num_parts   out: number of parts (>= 1)
 * Errors: MLA_ERR_INVALID_ARG (null out pointer, num_q_rows < 1),
 *         MLA_ERR_UNSUPPORTED (h_kv != 1), MLA_ERR_CUDA (device query failed).
 */
MLA_API int mla_num_sm_parts(int device, int num_q_rows, int h_kv, int *num_parts);

/*
 * mla_get_metadata — split-KV work partition ("MLA 메타데이터 가져오기").
 *
 * Launches the tile-scheduler kernel on `stream`.  It reads the sequence
 * lengths and cuts the (sequence, page) range into `num_parts` contiguous
 * parts of near-equal cost (pages plus MLA_SCHED_FIXED_COST_PAGES per
 * segment); a sequence may be cut across several parts (split-KV).  When
 * the batch is smaller than num_parts and one part per sequence is
 * estimated to finish sooner (no sequence cut, so no combine, charged
 * MLA_SCHED_COMBINE_COST_PAGES), only `batch` parts get work and the
 * others are empty.
 *   cache_seqlens            device int32 [batch]; entries >= 0
 *   batch                    number of sequences (>= 1)
 *   num_q_rows, h_kv         as for mla_num_sm_parts
 *   num_parts                parts to produce (>= 1; normally mla_num_sm_parts)
 *   tile_scheduler_metadata  device int32 [num_parts][MLA_METADATA_INTS], out:
 *                            per part {begin_seq, begin_page, end_seq,
 *                            end_page, begin_split, 0, 0, 0}; the part covers
 *                            the (sequence, page) cursor range [begin, end)
 *   num_splits               device int32 [batch + 1], out: prefix sum over
 *                            sequences of the number of parts touching each
 * The outputs stay valid for every decode call with the same cache_seqlens
 * values, num_q_rows and num_parts (one computation serves all layers).
 * A negative length sets MLA_DEVERR_SEQLEN in the device status word.
 * Errors: MLA_ERR_INVALID_ARG, MLA_ERR_UNSUPPORTED (h_kv != 1), MLA_ERR_CUDA.
 */
MLA_API int mla_get_metadata(const int32_t *cache_seqlens, int batch, int num_q_rows, int h_kv,
                     int num_parts, int32_t *tile_scheduler_metadata, int32_t *num_splits,
                     struct CUstream_st *stream);

/*
 * mla_get_metadata_costs — the same partition with the two costs given.
 *
 * mla_get_metadata is this call with fixed_cost = MLA_SCHED_FIXED_COST_PAGES
 * and combine_cost = MLA_SCHED_COMBINE_COST_PAGES.  The costs are in units
 * of one page of the lengths the partition is computed on (for the sparse
 * decode: one 64-entry list chunk; MLA_SCHED_SPARSE_*_CHUNKS are its
 * measured values).  They change only how the work is cut, never what a
 * decode computes.
 *   fixed_cost    cost of one segment (>= 1, <= MLA_SCHED_MAX_COST)
 *   combine_cost  cost charged for needing the combine (>= 0, <= MLA_SCHED_MAX_COST)
 * Other arguments, outputs and errors: as mla_get_metadata.
 */
MLA_API int mla_get_metadata_costs(const int32_t *cache_seqlens, int batch, int num_q_rows, int h_kv,
                           int num_parts, int fixed_cost, int combine_cost, int32_t *tile_scheduler_metadata,
                           int32_t *num_splits, struct CUstream_st *stream);

/*
 * mla_workspace_bytes — device scratch that mla_decode_kvcache needs for the
 * partial results of split sequences: fp32 partial outputs and their LSE for
 * at most (batch + num_parts) splits.  Returns 0 on invalid arguments.
 */
MLA_API size_t mla_workspace_bytes(int batch, int s_q, int h_q, int h_kv, int dv, int num_parts);

/*
 * mla_decode_kvcache — MLA decode over the paged latent cache ("MLA 디코딩 실행").
 *
 * For batch b, query token i, head h (all heads share KV head 0):
 *   T    = cache_seqlens[b]                 (causal == 0, or s_q == 1)
 *   T    = cache_seqlens[b] - s_q + i + 1   (causal != 0)
 *   k_j  = kcache[block_table[b][j / 64]][j % 64][0][0..d),     j < T
 *   s_j  = softmax_scale * <q[b][i][h], k_j>
 *   lse  = ln sum_j exp(s_j)
 *   o    = sum_j exp(s_j - lse) * k_j[0..512)
 * Rows with T <= 0 get o = 0 and lse = -inf.
 *
 *   q              device bf16 [batch][s_q][h_q][d]
 *   kcache         device bf16 [num_blocks][64][h_kv][d]; 16-byte aligned.
 *                  Rows past a sequence's end may hold any bits (NaN too).
 *   num_blocks     physical pages in kcache
 *   block_table    device int32 [batch][max_blocks_per_seq]; the first
 *                  ceil(T_b / 64) entries of row b must lie in [0, num_blocks)
 *   cache_seqlens  device int32 [batch]; 0 <= T_b <= 64 * max_blocks_per_seq
 *   d, dv          576 (or 512) and 512
 *   tile_scheduler_metadata, num_splits, num_parts
 *                  from mla_get_metadata with the same cache_seqlens
 *   softmax_scale  multiplies q.k before the softmax (e.g. 1/sqrt(576))
 *   causal         nonzero: the causal rule above (only matters for s_q > 1)
 *   o              device bf16 [batch][s_q][h_q][dv], out
 *   lse            device fp32 [batch][s_q][h_q], out (natural log)
 *   workspace      device scratch of at least mla_workspace_bytes(...) bytes,
 *                  256-byte aligned; its contents on entry do not matter
 * Out-of-range block ids or lengths found on the device are skipped and set
 * bits in the device status word (mla_device_status); they never fault.
 * Stream order: two kernels are enqueued on `stream` (split-KV, then the
 * combine), both as programmatic dependent launches.  Each may be scheduled
 * while the kernel before it is finishing, but reads and writes no global
 * memory until that kernel has completed, so the call observes every earlier
 * write on the stream exactly as an ordinary launch would.  The launches can
 * be captured in a CUDA graph once the first call on a device has set the
 * kernel attributes.
 * Errors: MLA_ERR_INVALID_ARG, MLA_ERR_UNSUPPORTED, MLA_ERR_WORKSPACE,
 *         MLA_ERR_CUDA (launch failure).
 */
MLA_API int mla_decode_kvcache(const void *q, const void *kcache, int64_t num_blocks,
                       const int32_t *block_table, int max_blocks_per_seq,
                       const int32_t *cache_seqlens, int batch, int s_q, int h_q, int h_kv,
                       int d, int dv, const int32_t *tile_scheduler_metadata,
                       const int32_t *num_splits, int num_parts, float softmax_scale,
                       int causal, void *o, float *lse, void *workspace,
                       size_t workspace_bytes, struct CUstream_st *stream);

/*
 * mla_decode_kvcache_fp8 — the same decode over a cache of packed e4m3 pages
 * with per-token scales.
 *
 * The page "[flashinfer] FlashInfer, SM120 GPU를 위한 희소 MLA 커널 추가로 LLM
 * 추론 속도 향상" (item 5, flashinfer/mla/trtllm.py) says that the MLA decode
 * API takes a `kv_scale_format` for a packed KV cache with scales, and the page
 * "[vllm] Blackwell을 위한 새로운 MLA 백엔드: TOKENSPEED_MLA 분석" (section
 * "들어가며") runs the Blackwell decode on an FP8 KV cache; neither gives the
 * layout.  This library's reading: a page of the cache is one packed
 * record of MLA_FP8_PAGE_BYTES(d) bytes,
 *   bytes [0, 64 d)          64 rows of d OCP e4m3 codes (row j, dim c at j d + c)
 *   bytes [64 d, 64 d + 256) 64 fp32 per-token scales c_j (little endian)
 * and cached row j dequantizes to k_j[c] = c_j * e4m3(code[j][c]).  The call
 * then computes exactly what mla_decode_kvcache computes on the dequantized
 * rows (V = their first 512 dims).
 *
 *   kv_pages       device bytes [num_blocks][MLA_FP8_PAGE_BYTES(d)]; 16-byte
 *                  aligned.  Codes and scales of rows past a sequence's end
 *                  may hold any bits.
 *   d              576 only (other values: MLA_ERR_UNSUPPORTED)
 *   everything else as for mla_decode_kvcache (q, o and lse stay bf16/fp32).
 * Precision: the kernel computes in f16 on the tensor cores.  The e4m3 codes
 * widen to f16 exactly; q is rounded to f16 (exact for |q| in [2^-17, 65504]);
 * the softmax weights times c_j are rounded to f16, so |c_j| must stay below
 * 255 for every token inside a sequence (a larger one can overflow f16).  A
 * scale with |c_j| >= 255, or a NaN scale, of a token inside its sequence
 * sets MLA_DEVERR_SCALE in the device status word, and the outputs of that
 * sequence are then undefined.  Scales of rows past a sequence's end are
 * never read.
 * Stream order, graph capture and errors: as for mla_decode_kvcache.
 */
#define MLA_FP8_PAGE_BYTES(d) (MLA_PAGE_SIZE * (d) + MLA_PAGE_SIZE * 4)
MLA_API int mla_decode_kvcache_fp8(const void *q, const void *kv_pages, int64_t num_blocks,
                                   const int32_t *block_table, int max_blocks_per_seq,
                                   const int32_t *cache_seqlens, int batch, int s_q, int h_q, int h_kv,
                                   int d, int dv, const int32_t *tile_scheduler_metadata,
                                   const int32_t *num_splits, int num_parts, float softmax_scale,
                                   int causal, void *o, float *lse, void *workspace,
                                   size_t workspace_bytes, struct CUstream_st *stream);

/*
 * mla_decode_kvcache_sparse — sparse top-k decode: each query token attends
 * only to the cached tokens its index list names.
 *
 * The page "[flashinfer] FlashInfer, SM120 GPU를 위한 희소 MLA 커널 추가로 LLM
 * 추론 속도 향상" (section "왜 이게 좋은가?", item 2) describes sparse MLA as
 * attention over only the top-k selected tokens of a paged cache; it gives no
 * interface.  This library's reading: query token i of sequence b carries
 * indices[b][i][0 .. topk) (token positions, shared by all its heads); an
 * entry is ignored when it is outside [0, cache_seqlens[b]) (-1 pads short
 * lists) or at or past list_lens[b]; every other entry is one term of the
 * softmax (a position listed twice counts twice); no causal mask applies:
 *   s_t = softmax_scale * <q, k_{indices[t]}>,  lse = ln sum_t exp(s_t),
 *   o   = sum_t exp(s_t - lse) * k_{indices[t]}[0..512)   over valid entries t.
 * A row with no valid entry gets o = 0 and lse = -inf.
 *
 *   kcache, block_table, cache_seqlens, q, o, lse, workspace
 *                  as for mla_decode_kvcache (bf16 cache, d = 576 only)
 *   indices        device int32 [batch][s_q][topk]
 *   topk           entries per list, >= 1
 *   list_lens      device int32 [batch]: the lengths the work partition was
 *                  computed on (tile_scheduler_metadata and num_splits come
 *                  from mla_get_metadata_costs on this array with
 *                  MLA_SCHED_SPARSE_FIXED_COST_CHUNKS and
 *                  MLA_SCHED_SPARSE_COMBINE_COST_CHUNKS, or from
 *                  mla_get_metadata; normally topk for every sequence)
 * A 128-row tile holds one query token's heads: s_q must be 1, or h_q 128
 * (MLA_ERR_UNSUPPORTED otherwise).  Rows are gathered one by one from the
 * cache (TMA gathers over the cache viewed as num_blocks * 64 rows, which
 * must stay below 2^31: MLA_ERR_UNSUPPORTED otherwise), so any positions may
 * be listed.
 * Stream order, graph capture and errors: as for mla_decode_kvcache.
 */
MLA_API int mla_decode_kvcache_sparse(const void *q, const void *kcache, int64_t num_blocks,
                                      const int32_t *block_table, int max_blocks_per_seq,
                                      const int32_t *cache_seqlens, const int32_t *indices, int topk,
                                      const int32_t *list_lens, int batch, int s_q, int h_q, int h_kv,
                                      int d, int dv, const int32_t *tile_scheduler_metadata,
                                      const int32_t *num_splits, int num_parts, float softmax_scale,
                                      void *o, float *lse, void *workspace, size_t workspace_bytes,
                                      struct CUstream_st *stream);

/*
 * mla_decode_kvcache_noalloc — mla_decode_kvcache for callers that cannot
 * allocate device memory.
 *
 * The pages have no counterpart of this call; it exists for callers that may
 * not allocate at decode time: runtimes that plan every byte of device memory
 * up front in their own arena, plugin interfaces that pass a call its inputs
 * and outputs but no workspace, and hot loops that must avoid an
 * allocation's implicit synchronisation.  The arguments and results are those
 * of mla_decode_kvcache without `workspace` / `workspace_bytes`: the split-KV
 * scratch comes from one fixed device array of MLA_NOALLOC_SCRATCH_BYTES
 * inside the library, which every GPU that loads the library keeps until the
 * process exits.  No call allocates (no cudaMalloc, cudaFree or allocating
 * library routine).
 *  - The first call on a device looks up the array's device address with that
 *    device current (a one-time set-up per device); make that first call
 *    before any stream capture.
 *  - Every call shares the array and it keeps the previous call's contents;
 *    nothing in it needs to start at zero.  Calls whose kernels overlap on the
 *    GPU (e.g. on two streams) race on it: order them on one stream.
 * Errors: those of mla_decode_kvcache, and MLA_ERR_WORKSPACE when
 * mla_workspace_bytes() for the shape exceeds MLA_NOALLOC_SCRATCH_BYTES
 * (nothing is launched then).
 */
#define MLA_NOALLOC_SCRATCH_BYTES (64u * 1024u * 1024u)
MLA_API int mla_decode_kvcache_noalloc(const void *q, const void *kcache, int64_t num_blocks,
                                       const int32_t *block_table, int max_blocks_per_seq,
                                       const int32_t *cache_seqlens, int batch, int s_q, int h_q, int h_kv,
                                       int d, int dv, const int32_t *tile_scheduler_metadata,
                                       const int32_t *num_splits, int num_parts, float softmax_scale,
                                       int causal, void *o, float *lse, struct CUstream_st *stream);

/* largest |scale| of an e4m3 token that the decode accepts (exclusive) */
#define MLA_FP8_SCALE_LIMIT 255

/*
 * mla_cache_write — write the rows of new tokens into the paged bf16 cache.
 *
 * Input row r is the latent part latent[r][0..512) followed, for d = 576, by
 * the RoPE part k_rope[r][0..64).  It belongs to sequence b with
 * cu_rows[b] <= r < cu_rows[b + 1] and becomes the cached row at position
 * starts[b] + r - cu_rows[b] of that sequence.  Rows at or behind
 * cu_rows[batch] (a padded input buffer) and rows before cu_rows[0] are ignored.
 *   latent, k_rope   device bf16, rows latent_stride / k_rope_stride elements
 *                    apart (multiples of 8; 0 repeats one row); 16-byte aligned.
 *                    d = 512: k_rope is not read and may be NULL
 *   num_rows         rows of the input, >= 0 (0: nothing is launched)
 *   cu_rows          device int32 [batch + 1], non-decreasing, or NULL: every
 *                    sequence has num_rows / batch rows (batch divides num_rows)
 *   starts           device int32 [batch]: position of the sequence's first row
 *   kcache           device bf16 [num_blocks][64][1][d], in/out; 16-byte aligned
 *   block_table      device int32 [batch][max_blocks_per_seq]
 *   d                576 or 512
 * Nothing but the named rows is touched.  A position outside
 * [0, 64 * max_blocks_per_seq) sets MLA_DEVERR_SEQLEN and a block id outside
 * [0, num_blocks) MLA_DEVERR_BLOCK_ID; the row is then skipped.  Two rows that
 * name the same place in one call leave either row's values, piece by piece.
 * One kernel is enqueued as a programmatic dependent launch; it can be captured
 * in a CUDA graph once any call of the library has run on the device.
 * Errors: MLA_ERR_INVALID_ARG, MLA_ERR_UNSUPPORTED, MLA_ERR_CUDA.
 */
MLA_API int mla_cache_write(const void *latent, int64_t latent_stride, const void *k_rope, int64_t k_rope_stride,
                            int64_t num_rows, const int32_t *cu_rows, const int32_t *starts, int batch, void *kcache,
                            int64_t num_blocks, const int32_t *block_table, int max_blocks_per_seq, int d,
                            struct CUstream_st *stream);

/*
 * mla_cache_write_fp8 — the same into packed e4m3 pages, quantised per token
 * (d = 576 only; the page layout of mla_decode_kvcache_fp8):
 *   c_j = max |x| / 448 over the row (1 for a row of zeros), code = e4m3(x / c_j)
 * with both quotients in fp32 (IEEE) and round to nearest even; a zero's code is
 * +0.  A row whose
 * scale reaches MLA_FP8_SCALE_LIMIT, or that holds a NaN or an infinity (its
 * scale becomes NaN), sets MLA_DEVERR_SCALE: the decode would report it too.
 */
MLA_API int mla_cache_write_fp8(const void *latent, int64_t latent_stride, const void *k_rope, int64_t k_rope_stride,
                                int64_t num_rows, const int32_t *cu_rows, const int32_t *starts, int batch,
                                void *kv_pages, int64_t num_blocks, const int32_t *block_table, int max_blocks_per_seq,
                                int d, struct CUstream_st *stream);

/*
 * mla_cache_read — read a range of each sequence's cached rows back into
 * contiguous rows (what the prompt path up-projects): output row r of sequence
 * b (cu_rows as for mla_cache_write) is the cached row at position
 * starts[b] + r - cu_rows[b], its first 512 dims into latent[r] and, for
 * d = 576, its last 64 into k_rope[r].
 *   latent, k_rope   device bf16, out; strides as for mla_cache_write, but at
 *                    least 512 / 64 (rows must not overlap)
 * Output rows of no sequence, and rows that are skipped as in mla_cache_write,
 * are left as they were.  The rest as for mla_cache_write.
 */
MLA_API int mla_cache_read(const void *kcache, int64_t num_blocks, const int32_t *block_table, int max_blocks_per_seq,
                           const int32_t *starts, const int32_t *cu_rows, int batch, int64_t num_rows, void *latent,
                           int64_t latent_stride, void *k_rope, int64_t k_rope_stride, int d,
                           struct CUstream_st *stream);

/*
 * mla_cache_read_fp8 — the same from packed e4m3 pages (d = 576): every value is
 * c_j * e4m3(code) in fp32, rounded to bf16 (nearest even).
 */
MLA_API int mla_cache_read_fp8(const void *kv_pages, int64_t num_blocks, const int32_t *block_table,
                               int max_blocks_per_seq, const int32_t *starts, const int32_t *cu_rows, int batch,
                               int64_t num_rows, void *latent, int64_t latent_stride, void *k_rope,
                               int64_t k_rope_stride, int d, struct CUstream_st *stream);

/*
 * mla_update_page_keys — recompute the page keys that mla_decode_kvcache_blocks
 * scores, for every page that the positions [starts[b], cache_seqlens[b]) of
 * some sequence touch (the whole page is summarised, from its first row to the
 * sequence's end).  For a page with n rows inside its sequence:
 *   mean  = (sum of its n rows) / n   in fp32, summed as a balanced tree over the
 *           64 rows (neighbours first, absent rows 0)
 *   scale = max |mean| / 127 (1 for a mean of zeros),  key = rint(mean / scale)
 * (IEEE fp32 quotients; a subnormal scale is at least 2^-149, and a key that it
 * would round past 127 is 127).  A mean that is not finite gives key 0 and scale NaN.
 *   cache_seqlens  device int32 [batch], as for mla_decode_kvcache
 *   starts         device int32 [batch] (e.g. the lengths before the last write),
 *                  or NULL: every page of every sequence
 *   page_keys      device int8 [num_blocks][d], in/out; 16-byte aligned
 *   page_scales    device fp32 [num_blocks], in/out
 * Entries of other pages are left as they were.  A page shared by two sequences
 * must have the same rows in both.  Lengths outside [0, 64 *
 * max_blocks_per_seq] and bad block ids set status bits, as for the decode.
 * Launches, capture and errors: as for mla_cache_write.
 */
MLA_API int mla_update_page_keys(const void *kcache, int64_t num_blocks, const int32_t *block_table,
                                 int max_blocks_per_seq, const int32_t *cache_seqlens, const int32_t *starts, int batch,
                                 int d, int8_t *page_keys, float *page_scales, struct CUstream_st *stream);
/* the same over packed e4m3 pages (d = 576): the rows c_j * e4m3(code) in fp32 */
MLA_API int mla_update_page_keys_fp8(const void *kv_pages, int64_t num_blocks, const int32_t *block_table,
                                     int max_blocks_per_seq, const int32_t *cache_seqlens, const int32_t *starts,
                                     int batch, int d, int8_t *page_keys, float *page_scales,
                                     struct CUstream_st *stream);

/*
 * mla_blocks_workspace_bytes — device scratch of mla_decode_kvcache_blocks
 * (num_parts from mla_num_sm_parts(device, 1, 1)).  0 on invalid arguments.
 */
MLA_API size_t mla_blocks_workspace_bytes(int batch, int s_q, int h_q, int h_kv, int dv, int max_blocks_per_seq,
                                          int topk_pages, int num_parts);

/*
 * mla_decode_kvcache_blocks — sparse decode over whole pages: each query token
 * attends to topk_pages pages that a score against the page keys selects for it.
 *
 * Query token i of sequence b sees positions < L (L = T_b, or the causal
 * T_b - s_q + i + 1), on ceil(L / 64) pages.  With at most topk_pages of them it
 * takes all; otherwise the first sink_pages, the last local_pages, and of the
 * rest those with the highest scores, ties to the lowest page:
 *   u_h   = max |q_h| / 127 (1 for a head of zeros),  qi_h = rint(q_h / u_h)
 *   score = page_scales[blk] * max_h (u_h * <qi_h, page_keys[blk]>)
 * The integer product is exact and each of the two fp32 products is rounded
 * once, so the selection does not depend on how it is computed.  A NaN score
 * (a query or a mean that is not finite) ranks highest.  o and lse are then
 * those of mla_decode_kvcache over the rows of the selected pages that lie
 * before L; a token with L <= 0 gets o = 0, lse = -inf and no pages.
 *   q, kcache, block_table, cache_seqlens, o, lse
 *                  as for mla_decode_kvcache (d = 576 or 512; batch * s_q <= 65535,
 *                  h_q <= 16384)
 *   page_keys, page_scales
 *                  from mla_update_page_keys; 16-byte aligned keys
 *   topk_pages     pages per query token, >= sink_pages + local_pages
 *   sink_pages, local_pages
 *                  >= 0 and >= 1 (the last visible page, which may be partial, is
 *                  always taken)
 *   num_parts      split-KV parts of the decode: mla_num_sm_parts(device, 1, 1), one
 *                  per CTA pair
 *   softmax_scale  > 0
 *   causal         nonzero: the causal rule above
 *   pages          device int32 [batch][s_q][topk_pages], out: the selected
 *                  pages of each token (logical, ascending), -1 behind them
 *   workspace      device scratch of at least mla_blocks_workspace_bytes(...)
 *                  bytes, 256-byte aligned
 * Five kernels are enqueued on `stream` (query codes, scores, selection with the
 * partition, split-KV, combine).  Stream order, graph capture, status bits and errors: as for
 * mla_decode_kvcache.
 */
MLA_API int mla_decode_kvcache_blocks(const void *q, const void *kcache, int64_t num_blocks,
                                      const int32_t *block_table, int max_blocks_per_seq,
                                      const int32_t *cache_seqlens, const int8_t *page_keys, const float *page_scales,
                                      int topk_pages, int sink_pages, int local_pages, int batch, int s_q, int h_q,
                                      int h_kv, int d, int dv, int num_parts, float softmax_scale, int causal, void *o,
                                      float *lse, int32_t *pages, void *workspace, size_t workspace_bytes,
                                      struct CUstream_st *stream);
/* the same over packed e4m3 pages (d = 576; precision as for mla_decode_kvcache_tree_fp8) */
MLA_API int mla_decode_kvcache_blocks_fp8(const void *q, const void *kv_pages, int64_t num_blocks,
                                          const int32_t *block_table, int max_blocks_per_seq,
                                          const int32_t *cache_seqlens, const int8_t *page_keys,
                                          const float *page_scales, int topk_pages, int sink_pages, int local_pages,
                                          int batch, int s_q, int h_q, int h_kv, int d, int dv, int num_parts,
                                          float softmax_scale, int causal, void *o, float *lse, int32_t *pages,
                                          void *workspace, size_t workspace_bytes, struct CUstream_st *stream);

/*
 * mla_tree_mask — the masks of draft trees from their parent lists.
 *
 *   parents    device int32 [batch][s_q]: the parent of each node, a node before
 *              it, or -1 (a root).  Any other value sets MLA_DEVERR_SEQLEN and
 *              counts as -1
 *   tree_mask  device int32 [batch][s_q][ceil(s_q / 32)], out: bit j % 32 of word
 *              j / 32 of row i is set when j is node i or an ancestor of it
 * Errors: MLA_ERR_INVALID_ARG, MLA_ERR_UNSUPPORTED (s_q > 65536), MLA_ERR_CUDA.
 */
MLA_API int mla_tree_mask(const int32_t *parents, int batch, int s_q, int32_t *tree_mask, struct CUstream_st *stream);

/*
 * mla_get_metadata_tree — split-KV work partition of a draft-tree decode.
 *
 * As mla_get_metadata, over the 128-row tiles of every sequence (tile t holds
 * rows 128 t .. of its s_q * h_q rows; tiles = ceil(s_q * h_q / 128)) instead of
 * over whole sequences, so that every CTA pair gets its share whatever the
 * number of tiles, and a tile that holds only rows behind its tree costs
 * nothing.  Computed once per step, used by every layer.
 *   tree_lens   as for mla_decode_kvcache_tree (the same values), or NULL
 *   num_parts   mla_num_sm_parts(device, 1, 1): one part per CTA pair
 *   tile_scheduler_metadata  device int32 [num_parts][MLA_METADATA_INTS], out
 *   num_splits  device int32 [batch * tiles + 1], out
 * Errors: as mla_get_metadata; batch * tiles above 2^24: MLA_ERR_UNSUPPORTED.
 */
MLA_API int mla_get_metadata_tree(const int32_t *cache_seqlens, const int32_t *tree_lens, int batch, int s_q, int h_q,
                                  int h_kv, int num_parts, int32_t *tile_scheduler_metadata, int32_t *num_splits,
                                  struct CUstream_st *stream);
/* device scratch of mla_decode_kvcache_tree; 0 on invalid arguments */
MLA_API size_t mla_tree_workspace_bytes(int batch, int s_q, int h_q, int h_kv, int dv, int num_parts);

/*
 * mla_decode_kvcache_tree — decode of a tree of drafted tokens.
 *
 * The last n_b = tree_lens[b] of the T_b cached rows of sequence b are drafted
 * nodes (written before the call), and query token i < n_b is node i.  It sees
 * every position before the nodes, and node j (position T_b - n_b + j) exactly
 * where bit j % 32 of word j / 32 of tree_mask[b][i] is set; its own bit too is
 * the mask's to set.  A row that sees nothing, and every row of a token
 * i >= n_b (a padded batch), gets o = 0 and lse = -inf.
 *   tree_mask  device int32 [batch][s_q][ceil(s_q / 32)] (mla_tree_mask, or any bits)
 *   tree_lens  device int32 [batch], 0 <= n_b <= s_q, or NULL: s_q everywhere.
 *              A value outside sets MLA_DEVERR_SEQLEN and is clamped
 *   tile_scheduler_metadata, num_splits, num_parts
 *              from mla_get_metadata_tree with the same lengths and tree lengths;
 *              both NULL: computed by this call, in the workspace, for num_parts
 *              parts
 *   workspace  at least mla_tree_workspace_bytes(...) bytes, 256-byte aligned
 *   everything else as for mla_decode_kvcache (d = 576 or 512; no causal
 *   argument: a chain's mask is the causal one).  T_b < n_b drops the nodes that
 *   would lie before the sequence.
 * A cached row that some query token of its sequence sees must be finite (a
 * non-finite one makes that token's o and lse NaN, and may make those of the tokens
 * of the same 128-row tile); a node's row that no token sees may hold any bits.
 * A query row that is not finite and sees something gets o = lse = NaN, and leaves
 * the other rows as they are.
 */
MLA_API int mla_decode_kvcache_tree(const void *q, const void *kcache, int64_t num_blocks, const int32_t *block_table,
                                    int max_blocks_per_seq, const int32_t *cache_seqlens, const int32_t *tree_mask,
                                    const int32_t *tree_lens, int batch, int s_q, int h_q, int h_kv, int d, int dv,
                                    const int32_t *tile_scheduler_metadata, const int32_t *num_splits, int num_parts,
                                    float softmax_scale, void *o, float *lse, void *workspace, size_t workspace_bytes,
                                    struct CUstream_st *stream);
/*
 * mla_decode_kvcache_tree_fp8 — the same over packed e4m3 pages (d = 576).
 *
 * Scales as for mla_decode_kvcache_fp8 (that of a node that no token sees may be
 * anything, like its row).  Precision: both products run on the fp8
 * tensor cores.  q is held exactly, but for elements below 2^-11 of their row's
 * largest (to 2^-19 of it).  A softmax weight times its token's scale, w, is held to
 * 2^-8 of itself; what weights too small for that lose is kept below 2^-9 of the
 * row's sum of w, whatever their number (a heavy key before thousands of light ones).
 */
MLA_API int mla_decode_kvcache_tree_fp8(const void *q, const void *kv_pages, int64_t num_blocks,
                                        const int32_t *block_table, int max_blocks_per_seq,
                                        const int32_t *cache_seqlens, const int32_t *tree_mask,
                                        const int32_t *tree_lens, int batch, int s_q, int h_q, int h_kv, int d, int dv,
                                        const int32_t *tile_scheduler_metadata, const int32_t *num_splits,
                                        int num_parts, float softmax_scale, void *o, float *lse, void *workspace,
                                        size_t workspace_bytes, struct CUstream_st *stream);

/*
 * mla_assign_pages — block tables, positions and slots of a step's new rows,
 * pages taken from a free list on the device.
 *
 * Sequence b holds len_b = cache_seqlens[b] rows and gets n_b = cu_rows[b + 1] -
 * cu_rows[b] more (one of a decoding step, a whole prompt), so it needs
 * need_b = ceil((len_b + n_b) / 64) - ceil(len_b / 64) new pages.  The free
 * list is a stack: of num_free pages, page k of the call is
 * free_pages[num_free - 1 - k].  Sequences are taken in order; b is served when
 * need_b = 0 or need_0 + .. + need_b <= num_free (the needs of all before it,
 * served or not, so that nobody overtakes), and then
 *   block_table[b][ceil(len_b / 64) ..]   its new pages, in order
 *   new_seqlens[b]   len_b + n_b
 *   positions[r]     len_b + r - cu_rows[b] for its rows r
 *   slots[r]         64 * page + position % 64
 * A sequence that is not served keeps its entries, new_seqlens[b] = len_b, and
 * its rows get position 0 and slot -1 (as rows of no sequence do), which
 * mla_norm_rope_cache_write skips.
 *   cache_seqlens  device int32 [batch]
 *   cu_rows        device int32 [batch + 1], ascending, at most num_rows
 *   num_rows       rows of positions and slots, >= cu_rows[batch]
 *   block_table    device int32 [batch][max_blocks_per_seq], in/out
 *   free_pages     device int32 [max_free]; num_free  device int32 [1]
 *   num_free_out   device int32 [1], out; may be num_free (the step is taken) or
 *                  another word (the step is planned: free_pages is only read)
 *   new_seqlens    device int32 [batch], out; may be cache_seqlens
 *   positions, slots  device int32 / int64 [num_rows], out, or NULL
 * A sequence whose bounds or lengths make no sense (bounds that descend, leave the rows
 * or begin before the end of an earlier sequence), or that would pass its table,
 * is not served and needs nothing, and sets MLA_DEVERR_SEQLEN; a table entry that is
 * no page where a row lands gives slot -1 and sets MLA_DEVERR_BLOCK_ID.
 * One kernel, no workspace.  Errors: MLA_ERR_INVALID_ARG, MLA_ERR_UNSUPPORTED
 * (2^31 rows or pages), MLA_ERR_CUDA.
 */
MLA_API int mla_assign_pages(const int32_t *cache_seqlens, const int32_t *cu_rows, int batch, int64_t num_rows,
                             int32_t *block_table, int max_blocks_per_seq, const int32_t *free_pages, int64_t max_free,
                             const int32_t *num_free, int32_t *num_free_out, int32_t *new_seqlens, int32_t *positions,
                             int64_t *slots, struct CUstream_st *stream);

/*
 * mla_release_pages — the pages of finished sequences back onto the free list.
 *
 * For every b with finished[b] != 0, in order: its ceil(cache_seqlens[b] / 64)
 * table entries are pushed in order and set to -1, and its length becomes 0.
 *   cache_seqlens  device int32 [batch], in/out;  finished  device int32 [batch]
 *   num_blocks     pages of the pool
 *   free_pages, max_free, num_free   as for mla_assign_pages, all in/out
 * An entry outside [0, num_blocks) is not pushed (MLA_DEVERR_BLOCK_ID); pages past
 * max_free are dropped (MLA_DEVERR_SEQLEN).  Uses of a page are not counted: one that
 * several finished sequences name is pushed by each.  Errors: as mla_assign_pages.
 */
MLA_API int mla_release_pages(int32_t *cache_seqlens, const int32_t *finished, int batch, int32_t *block_table,
                              int max_blocks_per_seq, int64_t num_blocks, int32_t *free_pages, int64_t max_free,
                              int32_t *num_free, struct CUstream_st *stream);

/*
 * mla_rope_turns — rotation frequencies as turns per position, in units of 2^-64
 * (host memory in, host memory out; the calls below take a device copy).
 *
 *   f_i = base^(-2 i / rope_dim) radians per position, i < rope_dim / 2
 * For contexts `factor` times longer: f_i / factor, or, with original_positions
 * > 0, f_i (1 - r_i) + f_i / factor * r_i, where the ramp r goes from 0 at the pair
 * that makes fast_turns turns in original_positions to 1 at the one that makes
 * slow_turns:
 *   pair(t) = rope_dim ln(original_positions / (2 pi t)) / (2 ln base)
 *   lo = max(0, floor(pair(fast_turns))), hi = min(rope_dim - 1, ceil(pair(slow_turns)))
 *   r_i = clamp((i - lo) / max(hi - lo, 0.001), 0, 1)
 *   rope_dim  even, > 0;  base > 1;  factor >= 1;  turns  int64 [rope_dim / 2], out
 * Returns MLA_OK or MLA_ERR_INVALID_ARG.
 */
MLA_API int mla_rope_turns(int rope_dim, double base, double factor, int original_positions, double fast_turns,
                           double slow_turns, int64_t *turns);

/*
 * mla_norm_rope — norm of every head and rotation of its last rope_dim values,
 * in one pass, fp32 inside, rounded to bf16 once.
 *
 *   y = x / sqrt(mean(x^2) + eps) * weight          (weight NULL: y = x)
 *   (a, b) = (a cos t - b sin t, b cos t + a sin t) * rope_scale
 * for the pairs of the last rope_dim values, t = positions[token] * turns[i] (whole
 * turns drop out exactly, at any position): pair i is (i, i + rope_dim / 2) of
 * them, or (2 i, 2 i + 1) with `interleaved`.
 *   x       device bf16 [num_tokens][heads][d], read with the two strides (elements,
 *           multiples of 8); 16-byte aligned
 *   d       a multiple of 8, at most 576
 *   weight  device bf16 [d], 16-byte aligned, or NULL
 *   positions  device int32 [num_tokens];  turns  device int64 [rope_dim / 2]
 *   rope_dim   a multiple of 16, at most min(d, 256); 0: no rotation
 *   out     device bf16, as x with its own strides, heads not overlapping; x
 *           itself (same strides) for a call in place, which without a weight
 *           touches the rotated values only.  No other overlap with x
 * Errors: MLA_ERR_INVALID_ARG, MLA_ERR_UNSUPPORTED, MLA_ERR_CUDA.
 */
MLA_API int mla_norm_rope(const void *x, int64_t x_token_stride, int64_t x_head_stride, int64_t num_tokens, int heads,
                          int d, const void *weight, float eps, const int32_t *positions, const int64_t *turns,
                          int rope_dim, int interleaved, float rope_scale, void *out, int64_t out_token_stride,
                          int64_t out_head_stride, struct CUstream_st *stream);

/*
 * mla_norm_rope_cache_write — new rows from a projection's output into the cache
 * in one pass: the 512 latent dims normalised, the 64 RoPE dims rotated (as
 * mla_norm_rope), and the row stored at slots[r] = 64 * block + row of the page.
 *   latent, k_rope  as for mla_cache_write (slices of one buffer, strides in
 *                   elements, multiples of 8); k_rope, positions and turns are
 *                   not read for d = 512
 *   weight      device bf16 [512], 16-byte aligned, or NULL: latent as it is
 *   positions   device int32 [num_rows];  turns  device int64 [32]
 *   slots       device int64 [num_rows] (mla_assign_pages); negative: the row goes
 *               nowhere; past the pool: the same, and MLA_DEVERR_BLOCK_ID
 *   latent_out, k_rope_out   device bf16, out, or NULL: the rows as bf16 as well
 *               (what the prompt path up-projects), for every row, slot or not
 * Two rows of one call must not have the same slot.
 * Errors: MLA_ERR_INVALID_ARG, MLA_ERR_UNSUPPORTED (row width), MLA_ERR_CUDA.
 */
MLA_API int mla_norm_rope_cache_write(const void *latent, int64_t latent_stride, const void *k_rope, int64_t k_rope_stride,
                                      int64_t num_rows, const void *weight, float eps, const int32_t *positions,
                                      const int64_t *turns, int interleaved, float rope_scale, const int64_t *slots,
                                      void *kcache, int64_t num_blocks, int d, void *latent_out, int64_t latent_out_stride,
                                      void *k_rope_out, int64_t k_rope_out_stride, struct CUstream_st *stream);

/*
 * mla_norm_rope_cache_write_fp8 — the same into packed e4m3 pages (d = 576): a
 * row's scale is max |y| / 448 (1 for zeros) of its fp32 values y, its codes
 * e4m3(y / scale), rounded once.  A row that is not finite, or whose scale reaches
 * the limit of the e4m3 decode, sets MLA_DEVERR_SCALE as in mla_cache_write_fp8.
 */
MLA_API int mla_norm_rope_cache_write_fp8(const void *latent, int64_t latent_stride, const void *k_rope,
                                          int64_t k_rope_stride, int64_t num_rows, const void *weight, float eps,
                                          const int32_t *positions, const int64_t *turns, int interleaved, float rope_scale,
                                          const int64_t *slots, void *kv_pages, int64_t num_blocks, int d, void *latent_out,
                                          int64_t latent_out_stride, void *k_rope_out, int64_t k_rope_out_stride,
                                          struct CUstream_st *stream);

/*
 * mla_prefill_metadata_ints, mla_prefill_workspace_bytes — int32 words of the work
 * partition, and device scratch, of a prompt attention on the current device.  0 on
 * invalid arguments.
 */
MLA_API int64_t mla_prefill_metadata_ints(int batch, int64_t num_q, int h_q, int h_kv);
MLA_API size_t mla_prefill_workspace_bytes(int batch, int64_t num_q, int h_q, int h_kv);

/*
 * mla_get_metadata_prefill — work partition of a prompt attention: blocks of query
 * tokens, the longest first, cut along their keys where that fills the GPU.
 *
 * It depends on the bounds and shapes only: one call serves every layer.
 *   cu_q, cu_k, batch, num_q, num_k, h_q, h_kv, causal   as for mla_prefill
 *   metadata   device int32 [mla_prefill_metadata_ints(...)], out
 * Errors: MLA_ERR_INVALID_ARG, MLA_ERR_UNSUPPORTED, MLA_ERR_CUDA.
 */
MLA_API int mla_get_metadata_prefill(const int32_t *cu_q, const int32_t *cu_k, int batch, int64_t num_q, int64_t num_k,
                                     int h_q, int h_kv, int causal, int32_t *metadata, struct CUstream_st *stream);

/*
 * mla_prefill — attention of packed prompts, or of chunks of new tokens behind a
 * context that was read back (mla_cache_read) and up-projected.
 *
 * Query rows cu_q[b] .. cu_q[b + 1] attend to key rows cu_k[b] .. cu_k[b + 1] of the
 * same sequence; query head h uses key head h / (h_q / h_kv).  With `causal`, row
 * i of n_q sees the first n_k - n_q + i + 1 of the n_k keys (the last row sees all of
 * them).  A row that sees nothing gets o = 0 and lse = -inf.
 *   q        device bf16 [num_q][h_q][d_qk], d_qk = 128, or 192 with k_rope
 *   k        device bf16 [num_k][h_kv][128]: the dims of a key without RoPE
 *   v        device bf16 [num_k][h_kv][128] (d_v = 128)
 *   k_rope   device bf16 [num_k][64], the RoPE dims of a key, shared by all heads
 *            (the last 64 of d_qk), or NULL
 *            each with strides in elements, multiples of 8, 16-byte aligned,
 *            heads not overlapping (slices of wider rows)
 *   cu_q, cu_k   device int32 [batch + 1], ascending, at most num_q / num_k.
 *            Sequences whose bounds make no sense are skipped, with
 *            MLA_DEVERR_SEQLEN
 *   h_q      a multiple of h_kv, at most 128 h_kv
 *   softmax_scale  > 0
 *   metadata from mla_get_metadata_prefill with the same bounds, shapes and mask, or NULL:
 *            computed by this call, in the workspace.  One that was made for another mask or
 *            other heads, or whose cut blocks a call of this num_q and num_k would not join,
 *            does nothing but set MLA_DEVERR_SEQLEN
 *   out      device bf16 [num_q][h_q][128], out, 32-byte aligned;  lse  device fp32
 *            [num_q][h_q], out:
 *            natural log of the sum of exp(softmax_scale q . k), for joining with other
 *            keys' results.  Rows of no sequence are left as they were
 *   workspace  at least mla_prefill_workspace_bytes(...) bytes, 256-byte aligned; calls
 *            that may overlap need workspaces of their own
 * Keys and values that some row of their sequence sees must be finite (one that is not
 * makes the rows that see it NaN, and may make those of the same 128-row tile); other
 * rows of k, k_rope and v may hold any bits.  A query row that is not finite leaves the
 * other rows as they are.  Weights are summed against a reference that the largest may pass
 * by 2^20, so values beyond 2^100 may overflow where the exact o would not.
 * Up to three kernels are enqueued (partition, attention, combine of cut blocks).  Stream
 * order and graph capture: as for mla_decode_kvcache.  Errors: MLA_ERR_INVALID_ARG,
 * MLA_ERR_UNSUPPORTED (widths, 2^30 rows), MLA_ERR_WORKSPACE, MLA_ERR_CUDA.
 */
MLA_API int mla_prefill(const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *k, int64_t k_token_stride,
                        int64_t k_head_stride, const void *v, int64_t v_token_stride, int64_t v_head_stride,
                        const void *k_rope, int64_t k_rope_token_stride, const int32_t *cu_q, const int32_t *cu_k, int batch,
                        int64_t num_q, int64_t num_k, int h_q, int h_kv, int d_qk, int d_v, float softmax_scale, int causal,
                        const int32_t *metadata, void *out, float *lse, void *workspace, size_t workspace_bytes,
                        struct CUstream_st *stream);

/*
 * mla_device_status — read the device status word of the current device.
 *
 * Synchronizes the device, stores the OR of the MLA_DEVERR_* bits raised by
 * kernels since the last clear into *status, and clears the word if `clear`
 * is nonzero.  Returns MLA_OK, MLA_ERR_INVALID_ARG or MLA_ERR_CUDA.
 */
MLA_API int mla_device_status(int *status, int clear);

/*
 * mla_set_timing_events — profiling aid: time the split-KV kernel alone.
 *
 * While set, every mla_decode_kvcache call records `split_begin` on its
 * stream just before the split-KV kernel and `split_end` just after it, so
 * that cudaEventElapsedTime gives that kernel's duration (the combine kernel
 * is outside the pair).  Both are cudaEvent_t handles created by the caller
 * on the device the decode runs on; pass NULL, NULL to stop.  The setting is
 * process-wide.  Returns MLA_OK, or MLA_ERR_INVALID_ARG if only one is NULL.
 */
MLA_API int mla_set_timing_events(void *split_begin, void *split_end);

/*
 * mla_set_cluster_multicast — how mla_decode_kvcache_sparse gathers rows.
 *
 * With 1 (the default) the two CTAs of a cluster split each list chunk's row
 * gathers between them and write every gathered row into both CTAs with a
 * TMA cluster multicast (within this GPU's own memory).  With 0 each CTA
 * gathers every row chunk it uses itself and nothing is multicast; the
 * results are bit-identical, the decode about 1.3x slower.  A process that
 * runs one job across several GPUs sets 0 before its first call.  The
 * setting is process-wide.  Returns MLA_OK, or MLA_ERR_INVALID_ARG unless
 * `enabled` is 0 or 1.
 */
MLA_API int mla_set_cluster_multicast(int enabled);

/* mla_status_string — static description of a status code (never NULL). */
MLA_API const char *mla_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* MLA_DECODE_H */
