/*
 * oasr_attn.h - C ABI of the paged-KV chunk attention library for GB300 (sm_103a).
 *
 * One hot path of a streaming ASR encoder (OASR documentation pages):
 *
 *   - ASR Engine page, section 4.3 "Batched paged forward": a lockstep cohort of B
 *     streams shares one stacked block_table (B, blocks_per_seq) and one
 *     cache_seqlens (B,) across every layer's paged K/V cache; each step writes the
 *     new chunk into the pool through the block table and the caller commits the
 *     cache length afterwards.
 *   - Scheduler page, section 4.3 "Heterogeneous-offset batching": the attention
 *     over the paged pool masks each stream by its cache_seqlens and adds the
 *     Transformer-XL position term matrix_bd / sqrt(d_k) to the content score.
 *   - Model Layer page, table "Three optional encoder declarations", row
 *     fixed_attention_window: with a uniform cache length one relative-position
 *     table serves the whole cohort, its distances being cache + i - j.
 *   - Model Layer page, Nemotron ASR section: Transformer-XL relative position with
 *     rel_shift.
 *   - ASR Engine page, section 4.1: with sequence packing an offline micro-batch is
 *     one gapless varlen-attention row.
 *
 * Layouts (row-major, innermost last; every pointer is DEVICE memory owned by the
 * caller; the library keeps no pointer after a call returns):
 *   q, k_new, v_new, out (streaming) : [B, T, H, D]
 *   k_pool, v_pool                   : [num_blocks, block_size, H, D]
 *   block_table                      : int32 [B, max_blocks_per_seq]
 *   cache_seqlens                    : int32 [B]  (frames cached BEFORE this chunk)
 *   pos_bias_u, pos_bias_v           : [H, D]
 *   rel                              : [R, H, D]
 *   q, k, v, out (packed)            : [total, H, D]
 *   cu_seqlens                       : int32 [num_seqs + 1], cu[0] = 0, non-decreasing,
 *                                      cu[num_seqs] = total
 * All float tensors of one call share the dtype `dt`.  Base pointers must be 16-byte
 * aligned (the tensor-core path reads them with TMA).
 *
 * The score of query i against key j, for one head, is
 *     s_ij = scale * ( (q_i + u) . k_j + (q_i + v) . rel[rho] )
 * followed by a softmax over j and a weighted sum of the value rows.  The rel row is
 * rho = z - dist in rel_shift order (row 0 holds the largest distance):
 *     streaming: dist = C + i - j, z = R - T, keys j in [0, C + T) (the whole cache
 *                and the whole chunk; no mask inside the chunk), R >= C + 2T - 1;
 *     packed:    dist = i - j within one segment, z = (R - 1) / 2, R >= 2 Lmax - 1.
 *
 * Execution: every call is asynchronous and stream-ordered on `stream`; none
 * synchronises, none allocates device memory.  Host-side argument checks return
 * OASR_ERR_INVALID_ARG / OASR_ERR_UNSUPPORTED before anything is enqueued.  Device
 * data (block ids, cache_seqlens, cu_seqlens) is not read on the host: an entry that
 * points outside its table makes the kernel skip or clamp that access and set a bit of
 * the device status word (oasr_device_status), never read or write out of bounds.
 */
#ifndef OASR_ATTN_H
#define OASR_ATTN_H

#include <stdint.h>

#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    OASR_OK = 0,
    OASR_ERR_INVALID_ARG = 1, /* null pointer, non-positive size, misaligned pointer   */
    OASR_ERR_UNSUPPORTED = 2, /* a size or dtype this build has no kernel for         */
    OASR_ERR_CUDA = 3,        /* a CUDA runtime call or a kernel launch failed         */
    OASR_ERR_BOUNDS = 4,      /* (oasr_device_status) a device index was out of range  */
    OASR_ERR_TIMEOUT = 5      /* (oasr_device_status) a kernel wait ran out of time    */
} oasr_status;

typedef enum { OASR_F32 = 0, OASR_BF16 = 1 } oasr_dtype;

/*
 * Paged append (ASR Engine page, section 4.3, step 1: the chunk's rows go into each
 * stream's pool blocks through its block_table).
 *
 * For b < B, t < T, h < H: logical position p = cache_seqlens[b] + t is written to
 * block block_table[b][p / block_size], slot p % block_size:
 *     k_pool[blk][slot][h][:] = k_new[b][t][h][:],  v_pool likewise.
 * A pure copy (bit-exact).  cache_seqlens is read, never advanced: the caller commits
 * the chunk afterwards.  Rows whose position lies past max_blocks_per_seq pages, or whose
 * block id is outside [0, num_blocks), are skipped (status bit OASR_ERR_BOUNDS).
 * D * sizeof(dtype) must be a multiple of 16 bytes and 2 * B * T at most 2^26 (else
 * OASR_ERR_UNSUPPORTED).
 */
oasr_status oasr_paged_append(const void* k_new, const void* v_new, void* k_pool, void* v_pool,
                              int num_blocks, int block_size, const int32_t* block_table,
                              int max_blocks_per_seq, const int32_t* cache_seqlens, int B,
                              int T, int H, int D, oasr_dtype dt, cudaStream_t stream);

/*
 * Streaming chunk attention over the paged pool (Scheduler page, section 4.3; Model
 * Layer page, fixed_attention_window row; Nemotron ASR section).
 *
 * For every stream b, head h and chunk row i < T, attends over the C_b + T keys that
 * the pool holds for stream b (C_b = cache_seqlens[b]: the cached frames followed by
 * this chunk, which oasr_paged_append must already have written on the same stream)
 * and writes out[b][i][h][:].  Requirements: D = 64; 1 <= T <= 64; block_size a power of
 * two in [8, 256]; R >= max_b C_b + 2T - 1; C_b + T <= max_blocks_per_seq * block_size.
 * A stream that breaks either raises the status bit OASR_ERR_BOUNDS and its row is then
 * unspecified: the bf16 path drops its keys past min(max_blocks_per_seq * block_size,
 * R - T + 1) (the keys the host can bound, for which it sizes its shared memory, so an
 * engine-sized block table costs nothing), the f32 path drops keys past the table's pages
 * and reads zero rows for the distances the rel table lacks.  scale is normally 1/sqrt(D).
 * bf16: bf16 inputs, fp32 accumulation and softmax, bf16 output rounded once; chunks of
 * 33 to 64 frames with an even H run on the 5th-generation tensor cores (two heads of a
 * stream per 128-row tile), other shapes on the legacy mma.sync path.
 * f32: fp32 throughout (no TF32).
 */
oasr_status oasr_chunk_relattn_paged(const void* q, const void* k_pool, const void* v_pool,
                                     int num_blocks, int block_size,
                                     const int32_t* block_table, int max_blocks_per_seq,
                                     const int32_t* cache_seqlens, const void* pos_bias_u,
                                     const void* pos_bias_v, const void* rel, int R, void* out,
                                     int B, int T, int H, int D, float scale, oasr_dtype dt,
                                     cudaStream_t stream);

/*
 * One fused streaming step: oasr_paged_append followed by oasr_chunk_relattn_paged, in
 * one launch.  Each (stream, head) program writes its head's slice of the chunk into
 * the pool and then attends over cache + chunk, so the chunk is never re-read from
 * HBM (when every page the chunk lands in is a valid block, the attention reads the
 * chunk's keys straight from k_new / v_new).  For bf16 chunks of 33 to 64 frames with an
 * even H the step is instead the two calls in sequence on `stream` (the append, then the
 * tensor-core attention over the pool).  Results equal the two calls in sequence up to
 * floating-point summation order; the pool afterwards is bit-identical.  The same
 * requirements apply.  Block ids of different streams must not alias a block that this
 * step writes.
 */
oasr_status oasr_chunk_step_paged(const void* q, const void* k_new, const void* v_new,
                                  void* k_pool, void* v_pool, int num_blocks, int block_size,
                                  const int32_t* block_table, int max_blocks_per_seq,
                                  const int32_t* cache_seqlens, const void* pos_bias_u,
                                  const void* pos_bias_v, const void* rel, int R, void* out,
                                  int B, int T, int H, int D, float scale, oasr_dtype dt,
                                  cudaStream_t stream);

/*
 * Packed varlen bidirectional attention (ASR Engine page, section 4.1; Model Layer
 * page, engine-facing surface table, forward_offline_packed).
 *
 * Segment s owns rows [cu_seqlens[s], cu_seqlens[s+1]); each of its queries attends to
 * every key of the same segment, with distance i - j (local indices) and rel row
 * z - (i - j), z = (R - 1) / 2.  Requirements: D = 64; 1 <= num_seqs <= 1024;
 * max_seqlen >= every segment length; R >= 2 * max_seqlen - 1; bf16: (total / 128 +
 * num_seqs) * H < 2^31 (else OASR_ERR_UNSUPPORTED).  Rows of a segment that would cross
 * `total` are clamped (status bit OASR_ERR_BOUNDS).
 */
oasr_status oasr_packed_relattn_varlen(const void* q, const void* k, const void* v,
                                       const int32_t* cu_seqlens, int num_seqs, int max_seqlen,
                                       int total, const void* pos_bias_u,
                                       const void* pos_bias_v, const void* rel, int R, void* out,
                                       int H, int D, float scale, oasr_dtype dt,
                                       cudaStream_t stream);

/*
 * Chunked-limited packed attention: the Nemotron offline mask (Model Layer page, Nemotron
 * ASR section: the chunked_limited mask applies offline too; a query sees its own chunk of
 * num_lookahead_tokens + 1 frames plus (sliding_window - 1) // chunk earlier chunks, and
 * the offline pass scores each query block against its own frames plus that history).
 *
 * As oasr_packed_relattn_varlen, but query i of a segment attends to key j only when
 * i / chunk_size - left_chunks <= j / chunk_size <= i / chunk_size (positions local to the
 * segment, integer division): chunk_size = num_lookahead_tokens + 1, left_chunks =
 * (sliding_window - 1) / chunk_size.  The work done grows with the segment length, not its
 * square.  Requirements as for oasr_packed_relattn_varlen, plus chunk_size >= 1 and
 * left_chunks >= 0 (else OASR_ERR_INVALID_ARG).  A chunk_size of at least every segment
 * length gives the bidirectional attention, up to summation order: in bf16 with an even head
 * count and at most 511 segments the call runs a tensor-core kernel of its own (64 queries
 * of a segment for a pair of heads per tile), otherwise the one-head packed kernel.
 */
oasr_status oasr_packed_relattn_chunked(const void* q, const void* k, const void* v,
                                        const int32_t* cu_seqlens, int num_seqs, int max_seqlen,
                                        int total, const void* pos_bias_u,
                                        const void* pos_bias_v, const void* rel, int R, void* out,
                                        int H, int D, float scale, int chunk_size,
                                        int left_chunks, oasr_dtype dt, cudaStream_t stream);

/*
 * Commit a streaming step with fixed-window history eviction (ASR Engine page, KV-pool sizing
 * paragraphs: an encoder with a trained attention window pages by chunk and retains
 * ceil(window / chunk) + 1 pages per stream; with eviction the cached length is held at the
 * window; section 4.3: the caller commits the cache length after the step).
 *
 * For every stream b, after a chunk of T frames was appended at cache_seqlens[b], the stream
 * holds n = cache_seqlens[b] + T frames in its first P = ceil(n / block_size) pages.  If
 * n > window_frames, the oldest d = min(ceil((n - window_frames) / block_size),
 * floor(n / block_size)) pages are dropped (whole pages only: a partly written newest page
 * stays, so with a window shorter than a page the cached length may exceed the window by
 * less than a page and is never negative): block_table[b][0 .. P) is rotated left by d, so
 * the dropped blocks become the next pages to be written, and cache_seqlens[b] becomes
 * n - d * block_size; otherwise cache_seqlens[b] becomes n.  Entries past the first P are
 * untouched.  Both arrays are device memory and are
 * updated in place on `stream`, so a captured step stays replayable.
 *
 * Requirements: B >= 1; 1 <= max_blocks_per_seq <= 512 (else OASR_ERR_UNSUPPORTED);
 * block_size >= 1; T >= 0; window_frames >= 0.  A negative cache length or a row that would
 * run past the table raises OASR_ERR_BOUNDS in the device status word and is clamped.
 */
oasr_status oasr_window_commit(int32_t* block_table, int32_t* cache_seqlens, int B,
                               int max_blocks_per_seq, int block_size, int T, int window_frames,
                               cudaStream_t stream);

/*
 * The projections that feed the path, in one launch (Model Layer page, fixed_attention_window
 * row: one positional projection per step serves the cohort; the Conformer rel-pos attention's
 * linear_q / linear_k / linear_v carry a bias, linear_pos does not):
 *
 *   q | k | v = x . w_qkv^T + b_qkv     x [M, d_model], w_qkv [3 d_model, d_model] (q rows,
 *                                       then k, then v), b_qkv [3 d_model]; q, k, v written as
 *                                       [M, H, 64] (M = B * T frames: the [B, T, H, 64] inputs of
 *                                       the attention calls)
 *   rel       = pos_emb . w_pos^T        pos_emb [R, d_model], w_pos [d_model, d_model]; rel
 *                                       written as [R, H, 64]
 *
 * bf16 in and out, fp32 accumulation, one rounding per output.  Requirements: d_model = 64 H
 * and a multiple of 128 (else OASR_ERR_UNSUPPORTED); every pointer 16-byte aligned.
 */
oasr_status oasr_project_qkv_pos(const void* x, const void* w_qkv, const void* b_qkv,
                                 const void* pos_emb, const void* w_pos, void* q, void* k, void* v,
                                 void* rel, int M, int R, int d_model, int H, oasr_dtype dt,
                                 cudaStream_t stream);

/*
 * The 8-bit cache: K and V pools whose rows (one head of one frame, 64 values) are e4m3 with one
 * power-of-two scale each, half the bytes of bf16 pools (64 + 1 instead of 128 per row).
 *
 *   k_pool, v_pool : [num_blocks, H, block_size, 64] e4m3 bytes
 *   kv_scale       : [num_blocks, H, 2, block_size] bytes (index 0 of the third axis: K, 1: V)
 *
 * A row r stands for q * 2^e, with e = max(-100, the least e for which max|r| <= 448 * 2^e), the
 * stored scale byte e + 127 and q = r * 2^-e rounded to e4m3 (nearest, ties to even).  A row with a
 * NaN or an infinity has the scale byte 255 and stands for NaN in every element.  q * 2^e is exact in
 * bf16 and fp32, so a row read back and written again keeps its bytes.  Block ids, block_table and
 * cache_seqlens mean what they mean for the other pools (oasr_window_commit serves both).  Every
 * pointer, kv_scale included, must be 16-byte aligned.
 *
 * oasr_paged_append_e4m3: as oasr_paged_append, the rows of k_new, v_new ([B, T, H, 64], `dt`)
 * quantised as they are written.  D = 64; 2 * H * T < 2^30.  Rows whose position lies past the table,
 * or whose block id is outside [0, num_blocks), are skipped (status bit OASR_ERR_BOUNDS).
 */
oasr_status oasr_paged_append_e4m3(const void* k_new, const void* v_new, void* k_pool, void* v_pool,
                                   void* kv_scale, int num_blocks, int block_size,
                                   const int32_t* block_table, int max_blocks_per_seq,
                                   const int32_t* cache_seqlens, int B, int T, int H, int D,
                                   oasr_dtype dt, cudaStream_t stream);

/*
 * Read cached rows back: k[b][i][h][:] and v[b][i][h][:] ([B, L, H, 64], `dt`) become the values of
 * stream b's position start[b] + i (start may be null: 0), for i < L.  Positions at or past
 * cache_seqlens[b] give zeros; negative positions, positions past the table's pages and invalid block
 * ids give zeros and raise OASR_ERR_BOUNDS.  D = 64; H * L < 2^30.
 */
oasr_status oasr_paged_read_e4m3(const void* k_pool, const void* v_pool, const void* kv_scale,
                                 int num_blocks, int block_size, const int32_t* block_table,
                                 int max_blocks_per_seq, const int32_t* cache_seqlens,
                                 const int32_t* start, void* k, void* v, int B, int L, int H, int D,
                                 oasr_dtype dt, cudaStream_t stream);

/*
 * oasr_chunk_relattn_paged over the 8-bit cache: the attention of that call on the values the pools
 * stand for.  D = 64; 1 <= T <= 64; block_size a power of two in [8, 256]; max_blocks_per_seq <= 512;
 * num_blocks * H * block_size < 2^31.  A stream with C_b + T > max_blocks_per_seq * block_size has the
 * keys past the table dropped; distances the rel table lacks (R < C_b + 2T - 1) count as zero rows; an
 * invalid block id reads as zero rows; a stream of negative C_b has output rows that are unspecified; each
 * raises OASR_ERR_BOUNDS.
 * bf16: the chunk, biases, rel and out are bf16; q + v and the position term are rounded to bf16, q + u
 * and the weights to fp16 (a weight with its key's V scale, relative to the row's largest such), everything
 * else is fp32.  The products are taken with q + u and q + v brought near one by a power of two for each row, so
 * K rows above 2^110 and rel rows above 2^90 may overflow whatever the query.  f32: fp32 throughout.
 */
oasr_status oasr_chunk_relattn_paged_e4m3(const void* q, const void* k_pool, const void* v_pool,
                                          const void* kv_scale, int num_blocks, int block_size,
                                          const int32_t* block_table, int max_blocks_per_seq,
                                          const int32_t* cache_seqlens, const void* pos_bias_u,
                                          const void* pos_bias_v, const void* rel, int R, void* out,
                                          int B, int T, int H, int D, float scale, oasr_dtype dt,
                                          cudaStream_t stream);

/*
 * One fused streaming step over the 8-bit cache: oasr_paged_append_e4m3 followed by
 * oasr_chunk_relattn_paged_e4m3 (in one launch for bf16 and T <= 16, else in two).  The chunk's own keys are
 * attended to as quantised, so the result is that of the two calls up to summation order, and the
 * pools afterwards are bit-identical (rows that the append drops, at negative positions too, are dropped here).
 * The requirements of both apply.  Block ids of different streams
 * must not alias a block that this step writes.
 */
oasr_status oasr_chunk_step_paged_e4m3(const void* q, const void* k_new, const void* v_new,
                                       void* k_pool, void* v_pool, void* kv_scale, int num_blocks,
                                       int block_size, const int32_t* block_table,
                                       int max_blocks_per_seq, const int32_t* cache_seqlens,
                                       const void* pos_bias_u, const void* pos_bias_v,
                                       const void* rel, int R, void* out, int B, int T, int H,
                                       int D, float scale, oasr_dtype dt, cudaStream_t stream);

/*
 * Quantise the rows of x ([M, K], `dt`) to 8-bit integers with one scale each: with
 * m = max(max|x_row|, 2^-100) in fp32, x8 = rint(x * (127 * (1 / m))) ([M, K] int8, ties to even; each
 * of the three operations rounded to fp32) and scale = m / 127 ([M] fp32), so x is about x8 * scale.  A row with a
 * NaN or an infinity gets zeros and a NaN scale, so that every result it enters is NaN.  Tokens are
 * rows of activations, output channels rows of a weight [N, K].  K must be a multiple of 16.
 */
oasr_status oasr_quantize_rows(const void* x, void* x8, float* scale, int M, int K, oasr_dtype dt,
                               cudaStream_t stream);

/*
 * Product of 8-bit integers with a scale per token and per output channel:
 *
 *   out[i][n] = (sum_k x8[i][k] * w8[n][k]) * x_scale[i] * w_scale[n] + bias[n]
 *
 * x8 [M, K] and w8 [N, K] int8, x_scale [M] and w_scale [N] fp32, bias [N] (null: none) and out [M, N]
 * of `dt`.  The sum is exact for K <= 1024.  For longer K it is the integer sum rounded once to fp32 for M <= 8,
 * and for M <= 128 where the library finds integer dot products faster than matrix tiles (its choice depends on
 * M, N, K and the GPU alone), else an fp32 accumulation: the same row can then differ in its last bits with the
 * batch that it is in.  The scales and the bias are applied in that order in fp32, and the result is rounded once.
 * K a multiple of 16, at most 65536; M and N at most 2^31 - 256; every pointer 16-byte aligned.
 */
oasr_status oasr_linear_w8a8(const void* x8, const float* x_scale, const void* w8, const float* w_scale,
                             const void* bias, void* out, int M, int N, int K, oasr_dtype dt,
                             cudaStream_t stream);

/*
 * oasr_project_qkv_pos with 8-bit integer products (one launch): q | k | v from x8 [M, d_model] and
 * w_qkv8 [3 d_model, d_model] with bias b_qkv [3 d_model], each written as [M, H, 64], and rel
 * [R, H, 64] from pos8 [R, d_model] and w_pos8 [d_model, d_model], without bias.  Scales and rounding
 * are those of oasr_linear_w8a8; the sums are exact for d_model <= 1024 and accumulated in fp32 otherwise.
 * d_model = 64 H, at most 16384; M and R at most 2^31 - 256; outputs and bias of `dt`.
 */
oasr_status oasr_project_qkv_pos_w8a8(const void* x8, const float* x_scale, const void* w_qkv8,
                                      const float* w_qkv_scale, const void* b_qkv, const void* pos8,
                                      const float* pos_scale, const void* w_pos8,
                                      const float* w_pos_scale, void* q, void* k, void* v, void* rel,
                                      int M, int R, int d_model, int H, oasr_dtype dt,
                                      cudaStream_t stream);

/* Human-readable name of a status code (static string). */
const char* oasr_status_string(oasr_status status);

/*
 * Device status word of the current device: an OR of OASR_ERR_BOUNDS (bit 0) and
 * OASR_ERR_TIMEOUT (bit 1) flags raised by kernels since the last clear.  Synchronises
 * the current device first.  *flags receives the raw bits (1 = bounds, 2 = timeout); if
 * clear is non-zero the word is reset to 0.  Returns OASR_ERR_CUDA if the read fails.
 */
oasr_status oasr_device_status(unsigned* flags, int clear);

/*
 * Diagnostic (the pages have no counterpart): run the library's bounded pipeline wait on a
 * barrier that nothing ever signals, with a limit of limit_us microseconds (1 .. 2000000),
 * on `stream`.  One CTA of one warp; when the wait runs out it raises the timeout bit of the
 * device status word and returns, as a kernel of the library does when a copy it waits for
 * never lands.  The context stays usable.  Returns OASR_ERR_INVALID_ARG for a limit outside
 * the range (nothing is launched), OASR_ERR_CUDA if the launch fails.
 */
oasr_status oasr_selftest_wait(unsigned limit_us, cudaStream_t stream);

/* Library version: major * 10000 + minor * 100 + patch. */
int oasr_version(void);

#ifdef __cplusplus
}
#endif

#endif /* OASR_ATTN_H */
