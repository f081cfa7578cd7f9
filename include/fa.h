/*
 * fa.h — C ABI of the GB300 (sm_103a) tiled online-softmax attention library
 * (libfa_gb300.so).
 *
 * What it computes.  Exact scaled-dot-product attention
 *     O = softmax(scale * Q K^T) V,   row-wise softmax,
 * with Q n×d, K m×d, V m×dv and O n×dv per (batch, head)
 * ("手搓 Attention：从三行循环到看懂 FlashAttention", §1).  The kernels never
 * form the n×m score matrix in memory: they stream K/V tiles and keep, per
 * query row, a running maximum m, a running sum l and an accumulator acc that
 * are rescaled by alpha = exp(m_old - m_new) whenever the maximum grows
 * (same page, §7 version 4; "S12 FlashAttention", 解法).  The log-sum-exp
 * LSE = m + ln(l) (natural log, over the SCALED scores) is returned beside O.
 *
 * Conventions shared by every entry point.
 *   - Pointers are DEVICE pointers owned by the caller, unless a parameter
 *     says otherwise.  The library never allocates device memory for a call;
 *     decode takes its split scratch from a caller-provided workspace.
 *   - Every call is asynchronous on `stream` (a cudaStream_t; NULL is the
 *     legacy default stream) and returns as soon as its launches are queued.
 *   - Arguments are validated before anything is launched; on a bad argument
 *     the call returns a non-zero fa_status and launches nothing.  The text of
 *     the last failure on the calling thread is returned by fa_last_error().
 *   - Problems that only the device can see (a block-table id out of range,
 *     a pipeline wait that exceeded its time limit) set a device status word
 *     instead of faulting; the affected outputs are left unspecified.
 *     fa_get_device_status() synchronises the stream and reads and clears it.
 *   - Layouts are dense row-major.  "BSHD" means [batch][token][head][dim].
 *   - Grouped heads: query head h reads kv head h / (H / Hkv); H % Hkv == 0.
 *   - bf16 values are IEEE bfloat16 bit patterns (uint16 storage); outputs O
 *     are rounded to bf16 with round-to-nearest-even; LSE is float32.
 *   - A query row that sees no key gets O = 0 and LSE = -inf.
 *   - Causal: key j is visible to query i iff j <= i + (m - n) (0-based):
 *     the n queries are the last n of the m key positions.  For n == m this
 *     is "query i sees the keys up to i"; for n > m the first n - m queries
 *     see no key (O = 0, LSE = -inf).  Varlen applies it per sequence.
 */
#ifndef FA_GB300_H
#define FA_GB300_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FA_OK = 0,
    FA_ERR_INVALID_ARG = 1,   /* null pointer, negative size, H % Hkv != 0, misaligned pointer */
    FA_ERR_UNSUPPORTED = 2,   /* valid but not implemented: d/dv/page_size outside the supported set,
                                 no sm_103a device */
    FA_ERR_WORKSPACE = 3,     /* workspace pointer null or smaller than the size query returns */
    FA_ERR_CUDA = 4,          /* a CUDA runtime call or launch failed; fa_last_error() has the text */
    FA_ERR_TIMEOUT = 5,       /* device status: a pipeline wait exceeded its limit */
    FA_ERR_BAD_BLOCK_TABLE = 6, /* device status: a block-table id outside [0, num_pages) */
    FA_ERR_DEBUG_CHECK = 7    /* device status, debug build (libfa_gb300_debug.so) only: a
                                 kernel's output index left the buffer it was given; the store
                                 was skipped.  Never set by the normal build. */
} fa_status;

/*
 * fa_forward — bf16 attention forward, dense batch.
 * Passage: "手搓 Attention" §1 (shapes and scale) and §7 version 4 (the
 * recurrence); "S12 FlashAttention", 解法; whole causal tiles above the
 * diagonal are skipped ("手搓 Attention" §6 and §7).
 *
 *   q    bf16 [B][n][H][d]       (BSHD)
 *   k    bf16 [B][m][Hkv][d]
 *   v    bf16 [B][m][Hkv][dv]
 *   o    bf16 [B][n][H][dv]      written
 *   lse  fp32 [B][H][n]          written (may be NULL: not written)
 *   scale  multiplies Q K^T; must be positive and finite (pass 1/sqrt(d)
 *          for the usual attention)
 *   causal 0 or 1
 * Non-finite inputs stay in their own batch element: the last K/V tile of an
 * element whose m is not a multiple of the tile reads zeros past its last row
 * (never the next element's rows, whose inf or NaN would otherwise turn the
 * masked keys' zero weights into NaN: 0 * inf = NaN).
 * Supported: d == dv, d in {64, 128}; pointers 16-byte aligned; n, m >= 0;
 * B*n, B*m and H*n below 2^31 (token rows and the LSE stride are 32-bit).
 * Computes S = Q K^T and P V on the tcgen05 tensor cores (bf16 operands,
 * fp32 accumulation in tensor memory); P is rounded to bf16 before P V.
 */
fa_status fa_forward(const void* q, const void* k, const void* v, void* o, float* lse,
                     int B, int H, int Hkv, int n, int m, int d, int dv,
                     float scale, int causal, void* stream);

/*
 * fa_forward_fp8 — attention forward with e4m3 (FP8) operands and per-tensor
 * descale factors: the values are q[i] * q_descale, k[j] * k_descale,
 * v[j] * v_descale.  Same shapes, layouts and semantics as fa_forward; o is
 * bf16, lse fp32 (of the descaled scores).  The pages name FP8 only as a
 * later FlashAttention feature ("S12 FlashAttention", 生产实践); the
 * recurrence is unchanged: S = Q K^T and P V run on the tcgen05 tensor cores
 * in kind::f8f6f4 with fp32 accumulation, and P is rounded to e4m3 (it lies
 * in [0, 256] under the lazy rescale, inside e4m3's range) before P V.
 *   q, k, v   e4m3 bytes [B][n][H][d], [B][m][Hkv][d], [B][m][Hkv][dv]
 *   descales  positive finite fp32
 * Supported: d == dv == 128; B*n, B*m and H*n below 2^31.
 */
fa_status fa_forward_fp8(const void* q, const void* k, const void* v, void* o, float* lse,
                         int B, int H, int Hkv, int n, int m, int d, int dv, float scale,
                         float q_descale, float k_descale, float v_descale, int causal,
                         void* stream);

/*
 * fa_forward_f32 — fp32 attention forward, dense batch; same shapes, layouts
 * and semantics as fa_forward with every tensor in float32.
 * Passage: "手搓 Attention" §1 (shapes and scale), §4 version 2 (subtract the
 * row maximum before exp; in fp32 that keeps hot scores of several hundred
 * finite and within a few 1e-6 of float64) and §7 version 4 (the recurrence).
 * Arithmetic is IEEE fp32 on the CUDA cores (no TF32); each score is carried
 * as a compensated (hi, lo) pair so that exp(s - m) keeps fp32 relative
 * accuracy when the scores are in the hundreds.
 *   scale  must be positive and finite, as for fa_forward (the row maximum is
 *          taken on the unscaled scores, which is the scaled maximum only for
 *          a positive scale); anything else returns FA_ERR_INVALID_ARG
 * Supported: d, dv in {64, 128}; pointers 16-byte aligned; H, B <= 65535.
 */
fa_status fa_forward_f32(const float* q, const float* k, const float* v, float* o, float* lse,
                         int B, int H, int Hkv, int n, int m, int d, int dv,
                         float scale, int causal, void* stream);

/*
 * fa_forward_varlen — bf16 attention forward over packed sequences of
 * different lengths.  Sequence s owns query tokens [cu_seqlens_q[s],
 * cu_seqlens_q[s+1]) and key tokens [cu_seqlens_k[s], cu_seqlens_k[s+1]).
 * Passage: each sequence is its own attention problem ("手搓 Attention" §1),
 * computed by the same recurrence (§7 version 4; "S12 FlashAttention", 解法)
 * over that sequence's K/V tiles only; a sequence whose length is not a
 * multiple of the tile ends on a partly masked tile, and rows whose first
 * tiles are fully masked take the guard of "S12 FlashAttention", 实现.
 *
 *   q    bf16 [total_q][H][d],  k bf16 [total_k][Hkv][d],  v bf16 [total_k][Hkv][dv]
 *   o    bf16 [total_q][H][dv]  written
 *   lse  fp32 [H][total_q] written (may be NULL)
 *   cu_seqlens_q, cu_seqlens_k  int32 [num_seqs + 1], DEVICE pointers,
 *        non-decreasing, starting at 0, ending at total_q / total_k
 *   total_q, total_k  rows of the packed q (and o) and k/v buffers; the
 *        kernels never read or write a row outside them (a sequence whose
 *        offsets exceed them is skipped and sets FA_ERR_INVALID_ARG in the
 *        device status word)
 *   max_seqlen_q, max_seqlen_k  upper bounds of the per-sequence lengths
 *        (sizes the launch grid; a larger value only launches idle blocks)
 * Supported as fa_forward; causal uses each sequence's own q and k lengths.
 * Non-finite values stay in their own sequence: the V rows past a sequence's
 * end in its last K/V tile (the next sequence's rows) are zeroed in shared
 * memory before P V, as the paged paths do with the rows past a sequence's
 * end in its last page.
 */
fa_status fa_forward_varlen(const void* q, const void* k, const void* v, void* o, float* lse,
                            const int* cu_seqlens_q, const int* cu_seqlens_k, int num_seqs,
                            int total_q, int total_k, int max_seqlen_q, int max_seqlen_k,
                            int H, int Hkv, int d, int dv, float scale, int causal, void* stream);

/*
 * fa_forward_window, fa_forward_varlen_window — bf16 attention forward under
 * a sliding window with a few first tokens that stay visible (sinks).
 * Passage: the pages name no window; the recurrence ("手搓 Attention" §7
 * version 4) runs over the tiles that hold a visible key only, as it does for
 * the causal mask (§6).
 *
 * Arguments, layouts and device status as fa_forward and fa_forward_varlen,
 * always causal (bottom-right): the query at position p = i + (m - n) sees key
 * j iff j <= p and (window == 0, or j > p - window, or j < sinks).
 *   window  0: no window; w > 0: the last w keys, the query's own among them
 *   sinks   keys from the start that stay visible under a window (ignored
 *           without one)
 * K/V tiles between the sinks and the window are never loaded, so the work is
 * linear in n for a fixed window.
 * A row whose visible scores hold a NaN gets O = LSE = NaN (never the LSE = -inf
 * of a row that sees no key).  A NaN in K reaches only the rows that see its key;
 * an inf or NaN in V may reach other rows of its batch element or sequence, as
 * under fa_forward's causal mask (a hidden key's weight is 0, and 0 * inf is NaN).
 * Supported: d == dv in {64, 128}; pointers 16-byte aligned; dense: B*n, B*m
 * and H*n below 2^31; packed: H*total_q below 2^31; both: fewer than 2^30 work
 * units (a batch element or sequence, empty ones among them; 2^a query heads of
 * one kv head, the largest power of two that divides H / Hkv, 128 at most;
 * 256 / 2^a query tokens, counted up to n or max_seqlen_q).
 */
fa_status fa_forward_window(const void* q, const void* k, const void* v, void* o, float* lse,
                            int B, int H, int Hkv, int n, int m, int d, int dv, float scale,
                            int window, int sinks, void* stream);

fa_status fa_forward_varlen_window(const void* q, const void* k, const void* v, void* o,
                                   float* lse, const int* cu_seqlens_q, const int* cu_seqlens_k,
                                   int num_seqs, int total_q, int total_k, int max_seqlen_q,
                                   int max_seqlen_k, int H, int Hkv, int d, int dv, float scale,
                                   int window, int sinks, void* stream);

/*
 * fa_paged_prefill — bf16 attention for several new query tokens per
 * sequence against that sequence's paged keys (chunked prefill).
 * Passage: "S12 FlashAttention", 它还解锁了什么 (the tiles the recurrence walks
 * need not be contiguous: each can be fetched through a block table) and 实现
 * (logical page p holds min(page_size, seq_len - p*page_size) valid tokens).
 *
 *   q            bf16 [total_q][H][d], sequence s owns rows
 *                [cu_seqlens_q[s], cu_seqlens_q[s+1])
 *   k_cache      bf16 [num_pages][Hkv][page_size][d]
 *   v_cache      bf16 [num_pages][Hkv][page_size][dv]
 *   block_table  int32 [num_seqs][max_blocks_per_seq]: logical -> physical page
 *   seq_lens     int32 [num_seqs]: keys of sequence s (its cached context and
 *                its new tokens), 0 <= seq_lens[s] <= max_blocks_per_seq*page_size
 *   cu_seqlens_q int32 [num_seqs + 1], non-decreasing from 0 to total_q
 *   o            bf16 [total_q][H][dv] written
 *   lse          fp32 [H][total_q]     written (may be NULL)
 *   max_seqlen_q upper bound of the per-sequence query counts
 *   causal       0 or 1: with 1 the n_s queries of sequence s are the last n_s
 *                of its seq_lens[s] positions (query i sees keys j <= i +
 *                seq_lens[s] - n_s)
 * All of K/V is read through TMA a page at a time on the tcgen05 path of
 * fa_forward.  Cache contents past seq_lens[s] in the last page are never
 * used, NaN included.  Page ids are range-checked on the device (an id
 * outside [0, num_pages) reads page 0 and sets FA_ERR_BAD_BLOCK_TABLE);
 * sequences whose query offsets fall outside total_q, or whose seq_lens[s]
 * falls outside [0, max_blocks_per_seq*page_size], are skipped (none of their
 * rows is written) and set FA_ERR_INVALID_ARG.
 * Supported: d == dv in {64, 128}, page_size == 16.
 */
fa_status fa_paged_prefill(const void* q, const void* k_cache, const void* v_cache,
                           const int* block_table, const int* seq_lens, const int* cu_seqlens_q,
                           void* o, float* lse, int num_seqs, int total_q, int max_seqlen_q,
                           int H, int Hkv, int d, int dv, int page_size, int num_pages,
                           int max_blocks_per_seq, float scale, int causal, void* stream);

/*
 * fa_paged_decode_workspace_size — bytes of workspace fa_paged_decode and
 * fa_paged_decode_fused need: the fused form's ticket words first (int32
 * [num_seqs][H], at the same offset for every split count), then the
 * per-split partial triples (m, l: fp32 [num_seqs][H][num_splits] each; o:
 * fp32 [num_seqs][H][num_splits][dv]), each array 256-byte aligned.
 * Passage: "S12 FlashAttention", 它还解锁了什么 and 练习 1 (flash-decoding:
 * each split of the keys leaves one (m, l, o) triple per query head, and the
 * merge reads them all).
 * Returns 0 on invalid sizes.
 */
size_t fa_paged_decode_workspace_size(int num_seqs, int H, int dv, int num_splits);

/*
 * fa_paged_decode — one query token per sequence against a paged KV cache,
 * split-KV ("flash-decoding"), grouped heads.
 * Passage: "S12 FlashAttention", 实现 (walk the block table; logical page p
 * holds min(page_size, seq_len - p*page_size) valid tokens), 组合 (block
 * table + grouped-head sharing + (m, l, o) in one loop), 它还解锁了什么 and
 * 练习 1 (split the keys across blocks, merge the (m, l, o) triples).
 *
 *   q            bf16 [num_seqs][H][d]
 *   k_cache      bf16 [num_pages][Hkv][page_size][d]
 *   v_cache      bf16 [num_pages][Hkv][page_size][dv]
 *   block_table  int32 [num_seqs][max_blocks_per_seq]: logical -> physical page
 *   seq_lens     int32 [num_seqs], 0 <= seq_lens[s] <= max_blocks_per_seq*page_size
 *   o            bf16 [num_seqs][H][dv]  written
 *   lse          fp32 [num_seqs][H]      written (may be NULL)
 *   num_splits   1..64: split x of a sequence with P pages covers logical
 *                pages [ceil(x*P/X), ceil((x+1)*P/X)); empty splits are allowed
 *   scale        positive and finite (else FA_ERR_INVALID_ARG)
 *   workspace    device scratch of at least fa_paged_decode_workspace_size()
 *                bytes, 256-byte aligned; the call writes the partials there
 *                and then merges them (fa_split_combine) on the same stream.
 * Tokens past seq_len in the last page are never used (their cache contents
 * may be anything, NaN included).  Page ids are range-checked on the device:
 * an id outside [0, num_pages) is skipped and sets FA_ERR_BAD_BLOCK_TABLE.  A
 * seq_lens[s] outside [0, max_blocks_per_seq*page_size] is treated as an
 * empty sequence (O = 0, LSE = -inf) and sets FA_ERR_INVALID_ARG.
 * Supported: d == dv == 128, page_size == 16, H / Hkv <= 16; num_pages*Hkv*16
 * and num_seqs*H*num_splits below 2^31.
 */
fa_status fa_paged_decode(const void* q, const void* k_cache, const void* v_cache,
                          const int* block_table, const int* seq_lens, void* o, float* lse,
                          int num_seqs, int H, int Hkv, int d, int dv, int page_size,
                          int num_pages, int max_blocks_per_seq, int num_splits, float scale,
                          void* workspace, size_t workspace_bytes, void* stream);

/*
 * fa_paged_decode_fused — fa_paged_decode in one launch.
 * Passage: "S12 FlashAttention", 接下来 (fuse the small-batch decode) and
 * 练习 1 (the split triples merge with the recurrence's rescale).
 *
 * Same arguments, layouts, supported sizes and device status as
 * fa_paged_decode, and the same O and LSE bits.  The merge runs inside the
 * decode launch: each (sequence, kv head, split) unit writes its triple,
 * then takes an atomic ticket of its (sequence, kv head); the unit that takes
 * the last ticket merges the triples of the group's query heads.  No unit
 * waits for another.
 *   workspace  as fa_paged_decode (the same size query).  Its ticket words
 *              must be zero before the first call that uses this workspace
 *              (cudaMemset the whole workspace to 0 once after allocating
 *              it); every call, also one that ends with FA_ERR_TIMEOUT,
 *              leaves them zero again.  Calls on one workspace must not
 *              overlap on the GPU.  (fa_paged_decode ignores the ticket
 *              words, so one workspace may serve both entries.)
 * After FA_ERR_TIMEOUT, O and LSE are undefined, as for fa_paged_decode.
 */
fa_status fa_paged_decode_fused(const void* q, const void* k_cache, const void* v_cache,
                                const int* block_table, const int* seq_lens, void* o, float* lse,
                                int num_seqs, int H, int Hkv, int d, int dv, int page_size,
                                int num_pages, int max_blocks_per_seq, int num_splits, float scale,
                                void* workspace, size_t workspace_bytes, void* stream);

/*
 * fa_paged_decode_noalloc — fa_paged_decode for callers that cannot allocate.
 * The pages have no counterpart for this call: it exists for library users.
 *
 * Some callers may not call cudaMalloc themselves: a plugin inside a host
 * framework that owns all device memory through its own allocator, or a
 * serving loop that must not allocate once it runs (cudaMalloc can
 * synchronise the device).  This entry point computes exactly what
 * fa_paged_decode computes (same kernels, same arguments minus the
 * workspace) and keeps its split partials in one fixed device array of
 * FA_NOALLOC_SCRATCH_BYTES that the library itself declares.  It allocates
 * nothing; the caller still owns and passes every input and output.
 *   - Every GPU that loads the library holds that array until the process ends.
 *   - The first call on a device looks up the array's device address
 *     (cudaGetSymbolAddress, with that device current) and keeps it; make
 *     that first call before any stream capture.  The address is kept per
 *     CUDA context: after cudaDeviceReset the next call is again a first
 *     call (it looks the new address up), so make it outside a capture too.
 *   - A problem whose partials (fa_paged_decode_workspace_size) exceed the
 *     array is rejected with FA_ERR_WORKSPACE before anything is launched.
 *   - All calls share the array, which keeps the last call's contents.  A
 *     call that ends with the device status clear has rewritten every partial
 *     its merge read, so nothing needs clearing.  After FA_ERR_TIMEOUT some
 *     partials were not rewritten and the merge read the previous call's:
 *     that call's O and LSE are undefined.  Calls that overlap on the GPU
 *     (other streams, other threads) race on the array and corrupt each
 *     other: serialise them.
 * Arguments, layouts, supported sizes and device status as fa_paged_decode.
 */
#define FA_NOALLOC_SCRATCH_BYTES (16u << 20)
fa_status fa_paged_decode_noalloc(const void* q, const void* k_cache, const void* v_cache,
                                  const int* block_table, const int* seq_lens, void* o,
                                  float* lse, int num_seqs, int H, int Hkv, int d, int dv,
                                  int page_size, int num_pages, int max_blocks_per_seq,
                                  int num_splits, float scale, void* stream);

/*
 * fa_paged_gather — checking tool for the block-table walk of fa_paged_decode.
 * Passage: "S12 FlashAttention", 实现 (logical page p of sequence s is
 * physical page block_table[s][p] and holds min(page_size, seq_len -
 * p*page_size) valid tokens).
 *
 * Runs the decode's units (sequence, kv head, split) with the decode's split
 * page ranges, page lookups, tensor copies and shared-memory page layout, and
 * copies the K and V rows it gathers out to dense buffers instead of scoring
 * them, so a test can compare them bit for bit with a host gather.
 *   k_cache, v_cache, block_table, seq_lens, num_pages, max_blocks_per_seq,
 *   num_splits   as fa_paged_decode
 *   k_out, v_out bf16 [num_seqs][max_blocks_per_seq*page_size][Hkv][d],
 *                caller-owned: token t of sequence s is written to row
 *                s*max_blocks_per_seq*page_size + t for t < seq_lens[s]; other
 *                rows are not written.
 * Device status as fa_paged_decode (bad page ids, out-of-range seq_lens).
 * Supported: d == 128, page_size == 16; num_pages*Hkv*16 and
 * num_seqs*Hkv*num_splits below 2^31.
 */
fa_status fa_paged_gather(const void* k_cache, const void* v_cache, const int* block_table,
                          const int* seq_lens, void* k_out, void* v_out, int num_seqs, int Hkv,
                          int d, int page_size, int num_pages, int max_blocks_per_seq,
                          int num_splits, void* stream);

/*
 * The e4m3 paged cache — half the bytes of the bf16 one.
 *
 *   k_cache, v_cache  e4m3 codes [num_pages][Hkv][page_size][d]
 *   k_scale, v_scale  one byte per row, [num_pages][Hkv][page_size]: the row
 *                     (a token of a kv head) stands for code * 2^(byte - 127)
 * The exponent byte - 127 of a written row is the smallest integer >= -127
 * with max|x| <= 448 * 2^(byte - 127) over the row's finite values (448 is
 * e4m3's largest value; a row of zeros gets byte 0), each code is x *
 * 2^-(byte - 127) rounded to nearest, ties to even; inf and NaN become e4m3's
 * NaN.  Caches written by other means may use any byte from 0 to 254.
 * Caches and scales are 16-byte aligned.
 * Supported: d in {64, 128}, page_size == 16; num_pages*Hkv*16 and rows*Hkv
 * below 2^31, max_blocks_per_seq below 2^26.
 * The block table, seq_lens and (where taken) cu_seqlens are as for
 * fa_paged_prefill: sequence s owns rows [cu_seqlens[s], cu_seqlens[s+1]) of
 * the packed tensors, and those n_s rows are the last n_s of its seq_lens[s]
 * tokens.  So one cu_seqlens writes a step's new tokens, then attends from them.
 */

/*
 * fa_paged_kv_write_e4m3 — quantise new K and V rows into the paged cache.
 * The pages have no counterpart for this call: "S12 FlashAttention", 生产实践,
 * names FP8 only as a later feature.
 *   k, v         bf16 rows [total][Hkv][d]; k_stride and v_stride are the
 *                elements from one token to the next (multiples of 8, at least
 *                Hkv*d; the heads of a token are dense), so K and V may be
 *                parts of one projection's output
 * Row cu_seqlens[s] + i is written to the slot of token seq_lens[s] - n_s + i.
 * Other slots, and the slots of rows no sequence owns, keep their contents.
 * Two rows of one call that name the same slot leave an unspecified mix there.
 * A sequence whose offsets leave the rows, with n_s > seq_lens[s] or with
 * seq_lens[s] outside [0, max_blocks_per_seq*page_size] is skipped and sets
 * FA_ERR_INVALID_ARG; a token whose page id is out of range is skipped and
 * sets FA_ERR_BAD_BLOCK_TABLE.
 */
fa_status fa_paged_kv_write_e4m3(const void* k, const void* v, void* k_cache, void* v_cache,
                                 void* k_scale, void* v_scale, const int* block_table,
                                 const int* seq_lens, const int* cu_seqlens, int num_seqs,
                                 int total, int Hkv, int d, long long k_stride, long long v_stride,
                                 int page_size, int num_pages, int max_blocks_per_seq,
                                 void* stream);

/*
 * fa_paged_kv_read_e4m3 — read cached rows back as bf16, the inverse of
 * fa_paged_kv_write_e4m3 (same arguments, same rows, same device status).
 *   k, v         bf16 [total][Hkv][d] written: code * 2^(byte - 127), rounded
 *                to bf16 (exact for every value in bf16's normal range).  Rows
 *                of skipped tokens are not written.
 */
fa_status fa_paged_kv_read_e4m3(const void* k_cache, const void* v_cache, const void* k_scale,
                                const void* v_scale, const int* block_table, const int* seq_lens,
                                const int* cu_seqlens, void* k, void* v, int num_seqs, int total,
                                int Hkv, int d, int page_size, int num_pages,
                                int max_blocks_per_seq, void* stream);

/*
 * fa_paged_e4m3_workspace_size — bytes of the optional workspace of
 * fa_paged_decode_e4m3 (max_seqlen_q 1) and fa_paged_prefill_e4m3: partials of
 * a few long sequences whose keys are split over the GPU.  Enough for every
 * table width and window of these sizes (for batches whose sequences are too
 * many to be split, too, although no call of theirs uses it); 0 where the form
 * that takes them has no partials, or for invalid sizes.  (A prefill of fewer
 * rows than the bound may run without the workspace it was sized for.)
 *
 * fa_paged_e4m3_workspace_used — the same bytes where a call with these
 * arguments splits its keys when it is given them, 0 where it runs without:
 * enough work as it is, or contexts (max_blocks_per_seq, or the window and
 * sinks) too short.  max_seqlen_q counts up to the call's total_q.
 */
size_t fa_paged_e4m3_workspace_size(int num_seqs, int max_seqlen_q, int H, int Hkv, int d);
size_t fa_paged_e4m3_workspace_used(int num_seqs, int max_seqlen_q, int H, int Hkv, int d,
                                    int max_blocks_per_seq, int causal, int window, int sinks);

/*
 * fa_paged_decode_e4m3 — one query token per sequence against the e4m3 paged
 * cache, grouped heads, split-KV.
 * Passage: as fa_paged_decode ("S12 FlashAttention", 实现, 组合, 它还解锁了什么
 * and 练习 1).
 *   q       bf16 [num_seqs][H][d]
 *   o       bf16 [num_seqs][H][d] written
 *   lse     fp32 [num_seqs][H]    written (may be NULL)
 *   window  0: every key; w > 0: the query (the last of its L keys) sees the
 *           last w keys, itself among them, and the first `sinks` keys
 *   sinks   keys from the start that stay visible under a window (ignored
 *           without one)
 *   workspace  device scratch of at least fa_paged_e4m3_workspace_size() bytes,
 *           256-byte aligned, or NULL; of any size where num_seqs * Hkv is
 *           above 38: no such call uses it.  A call normally runs in one launch,
 *           a thread-block cluster per (sequence, kv head) that splits the keys
 *           and merges; with a workspace, a few long sequences are instead cut
 *           into equal shares for every warp of the GPU, with a merge launch
 *           behind.  The workspace needs no initialisation; calls on one
 *           workspace must not overlap on the GPU.
 * Only pages that hold a visible key are looked up in the block table: ids of
 * the others may be anything.  Cache contents of keys no query sees are never
 * used, NaN included.  Device status as fa_paged_decode (bad page ids are
 * skipped; a bad seq_lens[s] is treated as an empty sequence).
 * K, V and the softmax weights enter the tensor cores in f16: codes exactly;
 * weights, each times its V row's 2^(byte - 127), rounded to 11 bits, fewer
 * below 2^-21 of the row's largest such product, and to zero below 2^-32 of it.
 * (So a V row whose scale is far above what its codes need, which this library
 * does not write, hides the others' share when its key has weight.)
 * Accumulation is fp32.
 * Supported: H / Hkv <= 32; num_seqs*H below 2^28.
 */
fa_status fa_paged_decode_e4m3(const void* q, const void* k_cache, const void* v_cache,
                               const void* k_scale, const void* v_scale, const int* block_table,
                               const int* seq_lens, void* o, float* lse, int num_seqs, int H,
                               int Hkv, int d, int page_size, int num_pages,
                               int max_blocks_per_seq, float scale, int window, int sinks,
                               void* workspace, size_t workspace_bytes, void* stream);

/*
 * fa_paged_prefill_e4m3 — several new query tokens per sequence against the
 * e4m3 paged cache (chunked prefill, draft tokens).
 * Passage: as fa_paged_prefill.
 *   q, cu_seqlens_q, max_seqlen_q, o, lse, causal   as fa_paged_prefill
 *   window, sinks  as fa_paged_decode_e4m3, for each query from its own
 *                  position p: keys j <= p with j > p - window or j < sinks;
 *                  a window needs causal = 1
 *   workspace      as fa_paged_decode_e4m3 (of any size only for the chunks that
 *                  run as it does)
 * A sequence with bad offsets, more than max_seqlen_q queries or a bad
 * seq_lens[s] is skipped (its rows are not written) and sets
 * FA_ERR_INVALID_ARG.  Bad page ids set FA_ERR_BAD_BLOCK_TABLE; the sequence's
 * output is then unspecified.
 * Cache contents of keys that none of a sequence's queries sees are never
 * used; a NaN in a key that one query sees may reach others of its sequence.
 * A row whose visible scores hold a NaN gets O = LSE = NaN, with a workspace or
 * without, as in fa_paged_decode_e4m3.
 * Chunks of at most 16 rows (max_seqlen_q * H / Hkv; 32 at d = 64 and where
 * H / Hkv is no power of two) run as
 * fa_paged_decode_e4m3 does; larger ones on the tcgen05 path of fa_forward,
 * their K/V tiles widened to bf16 (exactly) on the way to the tensor cores.
 * Supported: H / Hkv <= 32; num_seqs*max_seqlen_q*H below 2^28.
 */
fa_status fa_paged_prefill_e4m3(const void* q, const void* k_cache, const void* v_cache,
                                const void* k_scale, const void* v_scale, const int* block_table,
                                const int* seq_lens, const int* cu_seqlens_q, void* o, float* lse,
                                int num_seqs, int total_q, int max_seqlen_q, int H, int Hkv, int d,
                                int page_size, int num_pages, int max_blocks_per_seq, float scale,
                                int causal, int window, int sinks, void* workspace,
                                size_t workspace_bytes, void* stream);

/*
 * Drafted token trees over a paged cache.
 *
 * A serving loop that drafts a tree of tokens for each sequence appends them to
 * its cache as they are listed (a node behind its parent) and checks them in one
 * pass: fa_tree_layout turns the parents into ancestor bits and rotary positions,
 * fa_paged_qkv_write puts the nodes' K and V into the cache, each node attends to
 * the context and its ancestors (fa_paged_tree_attention), and
 * fa_paged_kv_accept moves the rows of the accepted path behind the context.
 * fa_paged_copy_pages gives a forked sequence pages of its own.
 * The pages of the passage have no counterpart for these calls; the attention is
 * the recurrence of fa_paged_prefill under another mask.
 *
 * Conventions.  seq_lens, cu_seqlens and the block table are as for
 * fa_paged_prefill: the n_s nodes of sequence s are rows [cu_seqlens[s],
 * cu_seqlens[s+1]) of the packed tensors and the last n_s of its seq_lens[s]
 * cached tokens; node t is token seq_lens[s] - n_s + t.  Packed rows that no
 * sequence owns are left as they are.  A sequence whose offsets leave the packed
 * rows, or with n_s > seq_lens[s], or seq_lens[s] beyond its table, is skipped
 * and sets FA_ERR_INVALID_ARG in the device status word.
 */

/*
 * fa_tree_layout — ancestor bits and positions of the nodes.
 *   parents    int32 [total]: the node's parent, an earlier node of its sequence
 *              (0 <= parent < t), or -1 for a child of the context.  Anything
 *              else counts as -1 and sets FA_ERR_INVALID_ARG.
 *   mask       int32 [total][mask_words] written: bit t % 32 of word t / 32 of
 *              row i says that node i sees node t, itself or an ancestor
 *   positions  int32 [total] written (may be NULL): seq_lens[s] - n_s + depth,
 *              depth 0 for a child of the context
 * A sequence of more than 32*mask_words nodes is skipped and sets
 * FA_ERR_INVALID_ARG.
 * Time grows with the depth of the deepest tree times mask_words (a chain of 256 nodes
 * 20 us, of 1024 938; trees of 1024 nodes with random parents 30).
 * Supported: 1 <= mask_words <= 32; total*mask_words below 2^31.
 */
fa_status fa_tree_layout(const int* parents, const int* seq_lens, const int* cu_seqlens, int* mask,
                         int* positions, int num_seqs, int total, int mask_words, void* stream);

/*
 * fa_qk_norm_rope — q and k of each head normalised and rotated in one pass.
 *   q, k       bf16 rows [total][H][d] and [total][Hkv][d]; q_stride and k_stride
 *              are the elements from one token to the next (multiples of 8, at
 *              least H*d and Hkv*d; the heads of a token are dense), so they may
 *              be parts of one projection's output
 *   q_weight, k_weight  bf16 [d], or NULL: that tensor is not normalised.  With
 *              them y = x / sqrt(mean(x^2) + eps) * weight over the head's d
 *              values.
 *   rot_dim    the first rot_dim values of a head are rotated: pair p is values
 *              (p, p + rot_dim/2), or (2p, 2p + 1) with interleaved = 1, and
 *              (a, b) becomes (a c - b s, b c + a s) with (c, s) = cos_sin[x][p],
 *              x the token's position on the pair's axis
 *   cos_sin    fp32 [max_positions][rot_dim/2][2]; any scaling of the angles or
 *              of the rotation is the table's (NULL with rot_dim 0)
 *   positions  int32 [num_axes][total] (NULL with rot_dim 0)
 *   sections   HOST int [num_axes]: rotary pairs of each axis, in order (time,
 *              height, width for images and video); their sum is rot_dim/2.
 *              NULL with one axis.
 *   q_out, k_out  bf16 [total][H][d], [total][Hkv][d] written; q itself where
 *              q_stride is H*d, and so for k (no other overlap)
 * The arithmetic is fp32, rounded once to bf16.  A token with a position outside
 * [0, max_positions) is skipped (its rows are not written) and sets
 * FA_ERR_INVALID_ARG in the device status word.
 * A head whose squares leave fp32's range is normed all the same (it is scaled by a power
 * of two first).  With eps 0 a head of zeros becomes NaN (0 / 0).
 * Supported: d in {64, 128}; rot_dim a multiple of 8 up to d; 1 <= num_axes <= 4;
 * pointers 16-byte aligned; H, Hkv <= 65536; total*(H + 2*Hkv) below 2^31.
 */
fa_status fa_qk_norm_rope(const void* q, const void* k, const void* q_weight, const void* k_weight,
                          const float* cos_sin, const int* positions, void* q_out, void* k_out,
                          int total, int H, int Hkv, int d, long long q_stride, long long k_stride,
                          int rot_dim, int interleaved, int num_axes, const int* sections,
                          int max_positions, float eps, void* stream);

/*
 * fa_paged_qkv_write — fa_qk_norm_rope with K and V going into the bf16 paged
 * cache of fa_paged_prefill.
 *   v, v_stride   bf16 rows [total][Hkv][d], as k; copied as they are
 *   k_cache, v_cache  bf16 [num_pages][Hkv][page_size][d]: row cu_seqlens[s] + i is
 *                 written to the slot of token seq_lens[s] - n_s + i, other slots
 *                 keep their contents.  Two rows of one call that name the same
 *                 slot leave an unspecified mix there.
 * The other arguments are as for fa_qk_norm_rope.  A token whose page id is out
 * of range is skipped and sets FA_ERR_BAD_BLOCK_TABLE.
 * Supported: as fa_qk_norm_rope; page_size == 16; num_pages*Hkv*16 below 2^31,
 * max_blocks_per_seq below 2^26.
 */
fa_status fa_paged_qkv_write(const void* q, const void* k, const void* v, const void* q_weight,
                             const void* k_weight, const float* cos_sin, const int* positions,
                             void* q_out, void* k_cache, void* v_cache, const int* block_table,
                             const int* seq_lens, const int* cu_seqlens, int num_seqs, int total,
                             int H, int Hkv, int d, long long q_stride, long long k_stride,
                             long long v_stride, int rot_dim, int interleaved, int num_axes,
                             const int* sections, int max_positions, float eps, int page_size,
                             int num_pages, int max_blocks_per_seq, void* stream);

/*
 * fa_paged_tree_workspace_size — bytes of workspace fa_paged_tree_attention and
 * fa_paged_tree_attention_e4m3 need (0 on invalid sizes): partials of the units
 * whose keys are split.
 */
size_t fa_paged_tree_workspace_size(int num_seqs, int max_seqlen_q, int H, int Hkv, int d);

/*
 * fa_paged_tree_attention — attention of drafted nodes over the bf16 paged cache
 * (fa_paged_qkv_write fills it).
 * Passage: as fa_paged_prefill.
 *   q, k_cache, v_cache, block_table, seq_lens, cu_seqlens_q, o, lse
 *                 as fa_paged_prefill
 *   mask          int32 [total_q][mask_words] as fa_tree_layout writes it, or any
 *                 other bits: node i sees every token of the context (the first
 *                 seq_lens[s] - n_s) and node t where bit t of its row is set.
 *                 Bits from n_s on are ignored.  A row that sees no key gets O = 0
 *                 and LSE = -inf.
 *   max_seqlen_q  upper bound of the per-sequence node counts.  With 0 the call does
 *                 nothing: it looks at no sequence, and o and lse stay as they are
 *                 (the binding's helpers, whose outputs are new, look at them all).
 *                 A bound beyond floor(128 / (H/Hkv)) selects the form for units of
 *                 two query tiles, which takes longer where every tree is smaller
 *                 (16 nodes of 64 sequences, H/Hkv = 4: bounds to 32 200 us, above 208)
 *   workspace     device scratch of at least fa_paged_tree_workspace_size() bytes,
 *                 256-byte aligned; it needs no initialisation, and calls on one
 *                 workspace must not overlap on the GPU
 * Cache contents of keys that no node of a sequence sees (past its end, or of
 * nodes whose bit nobody has) are never used, NaN included; a NaN in a key that
 * one node sees, or an infinite value in its V, may reach others of its sequence.
 * A row whose visible scores hold a NaN gets O = LSE = NaN.
 * O is summed in fp32 before it is divided, with weights of up to 2^8: finite values
 * of V give a finite O while the largest times the keys of a row stays below 2^119.
 * A sequence of more than max_seqlen_q or 32*mask_words nodes is skipped and sets
 * FA_ERR_INVALID_ARG.  Page ids outside [0, num_pages) set
 * FA_ERR_BAD_BLOCK_TABLE; the sequence's output is then unspecified.
 * Supported: d in {64, 128}, page_size == 16, H / Hkv <= 128; scale positive and
 * finite; 1 <= mask_words; num_seqs <= 4096; total_q*H and total_q*mask_words below
 * 2^31; num_pages*Hkv*16 below 2^31; units * (4*ceil(max_blocks_per_seq / 8) + 9)
 * below 2^31, where units = num_seqs * Hkv * ceil(max_seqlen_q / (2*floor(128 /
 * (H / Hkv)))).
 */
fa_status fa_paged_tree_attention(const void* q, const void* k_cache, const void* v_cache,
                                  const int* block_table, const int* seq_lens,
                                  const int* cu_seqlens_q, const int* mask, void* o, float* lse,
                                  int num_seqs, int total_q, int max_seqlen_q, int mask_words, int H,
                                  int Hkv, int d, int page_size, int num_pages,
                                  int max_blocks_per_seq, float scale, void* workspace,
                                  size_t workspace_bytes, void* stream);

/*
 * fa_paged_tree_attention_e4m3 — the same over the e4m3 paged cache
 * (fa_paged_kv_write_e4m3 fills it): K and V are the values that
 * fa_paged_kv_read_e4m3 returns.
 *   k_cache, v_cache, k_scale, v_scale  as fa_paged_prefill_e4m3
 * The other arguments, the conventions and the limits are as for
 * fa_paged_tree_attention.  (fa_qk_norm_rope and fa_paged_kv_write_e4m3 together
 * do for this cache what fa_paged_qkv_write does for the bf16 one.)
 */
fa_status fa_paged_tree_attention_e4m3(const void* q, const void* k_cache, const void* v_cache,
                                       const void* k_scale, const void* v_scale,
                                       const int* block_table, const int* seq_lens,
                                       const int* cu_seqlens_q, const int* mask, void* o, float* lse,
                                       int num_seqs, int total_q, int max_seqlen_q, int mask_words,
                                       int H, int Hkv, int d, int page_size, int num_pages,
                                       int max_blocks_per_seq, float scale, void* workspace,
                                       size_t workspace_bytes, void* stream);

/*
 * fa_paged_kv_accept — the accepted path's rows moved behind the context.
 *   k_cache, v_cache  [num_layers][num_pages][Hkv][page_size][d], bf16, or e4m3
 *                 with scale bytes k_scale, v_scale [num_layers][num_pages][Hkv]
 *                 [page_size] (both NULL for bf16); the layers share the table
 *   path          int32 [num_seqs][max_path]: the accepted nodes of sequence s,
 *                 in increasing order, path_lens[s] of them (0 <= path_lens[s] <=
 *                 max_path); the entries behind them may be anything
 *   new_seq_lens  int32 [num_seqs] written: seq_lens[s] - n_s + path_lens[s] (an
 *                 array of its own, not seq_lens itself).  With num_layers 0 the call
 *                 does nothing and leaves it as it is (the binding's helper refuses that)
 * The rows of node path[s][a] are copied to the slot of node a, for every a in
 * turn; the slots behind keep their contents.  A sequence whose path is longer
 * than max_path or n_s, leaves [0, n_s) or does not increase is skipped, its new
 * length is seq_lens[s], and FA_ERR_INVALID_ARG is set.  A node that moves and whose
 * page id is out of range, its own or its destination's, is skipped and sets
 * FA_ERR_BAD_BLOCK_TABLE.  The pages that hold a sequence's nodes must be its
 * own: two sequences that move rows within one page leave an unspecified mix.
 * Supported: d in {64, 128}, page_size == 16, max_path <= 1024, Hkv <= 65536,
 * num_layers <= 65535; num_pages*Hkv*16 below 2^31, max_blocks_per_seq below 2^26,
 * num_seqs * num_layers below 2^31.
 */
fa_status fa_paged_kv_accept(void* k_cache, void* v_cache, void* k_scale, void* v_scale,
                             const int* block_table, const int* seq_lens, const int* cu_seqlens,
                             const int* path, const int* path_lens, int* new_seq_lens, int num_seqs,
                             int total, int max_path, int num_layers, int Hkv, int d, int page_size,
                             int num_pages, int max_blocks_per_seq, void* stream);

/*
 * fa_paged_copy_pages — whole pages copied within a cache, in every layer.
 *   caches, scales, num_layers   as fa_paged_kv_accept
 *   pairs         int32 [num_pairs][2]: source page, destination page.  A pair
 *                 with an id out of range is skipped and sets
 *                 FA_ERR_BAD_BLOCK_TABLE.  A source may appear in several pairs; a
 *                 page that is the destination of two pairs, or of one and the
 *                 source of another, is left with an unspecified mix (and the
 *                 other's destination too).
 * Supported: as fa_paged_kv_accept; num_pairs * num_layers * Hkv below 2^27.
 */
fa_status fa_paged_copy_pages(void* k_cache, void* v_cache, void* k_scale, void* v_scale,
                              const int* pairs, int num_pairs, int num_layers, int Hkv, int d,
                              int page_size, int num_pages, void* stream);

/*
 * fa_split_combine — merge per-split partial triples with the recurrence's
 * rescale rule ("S12 FlashAttention", 练习 1): for each (s, h)
 *     M = max_x m_x,  w_x = exp(m_x - M)  (w_x = 0 when m_x = -inf),
 *     l = sum_x w_x l_x,  O = sum_x w_x o_x / l,  LSE = M + ln l.
 *
 *   part_m, part_l  fp32 [num_seqs][H][num_splits]: m_x is the split's maximum
 *                   scaled score (natural units), l_x = sum exp(s_j - m_x)
 *   part_o          fp32 [num_seqs][H][num_splits][dv]: sum exp(s_j - m_x) V[j]
 *   o               bf16 [num_seqs][H][dv] written
 *   lse             fp32 [num_seqs][H] written (may be NULL)
 * An (s, h) whose splits are all empty gets O = 0 and LSE = -inf.
 * Supported: dv % 4 == 0, dv <= 256, 1 <= num_splits <= 64; num_seqs*H below 2^31.
 */
fa_status fa_split_combine(const float* part_m, const float* part_l, const float* part_o,
                           void* o, float* lse, int num_seqs, int H, int num_splits, int dv,
                           void* stream);

/*
 * fa_last_error — NUL-terminated description of the last non-OK status
 * returned on the calling thread ("" if none).  Owned by the library; valid
 * until the thread's next failing call.
 */
const char* fa_last_error(void);

/*
 * fa_get_device_status — synchronise `stream`, then read and clear the
 * device status word of the current device (FA_OK, FA_ERR_TIMEOUT,
 * FA_ERR_BAD_BLOCK_TABLE, or FA_ERR_INVALID_ARG for varlen offsets outside
 * the buffers) into *status.  Returns FA_ERR_CUDA if the
 * synchronisation itself failed.
 */
fa_status fa_get_device_status(void* stream, int* status);

#ifdef __cplusplus
}
#endif

#endif /* FA_GB300_H */
