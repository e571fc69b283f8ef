/*
 * mla_lowbit.h -- C ABI of the low-bit MLA decode library (one GB300, sm_103a).
 *
 * What it computes follows "QuantMLA: Function-Aligned Dual-Path Quantization
 * for Low-Bit MLA KV Caching":
 *   - Abstract: the content latent (c_kv, 512 channels) is cached at INT4 or
 *     INT2 and the decoupled RoPE key (64 channels) at INT4; a native low-bit
 *     MLA attention kernel unpacks and dequantises inside attention;
 *   - Figure 3 caption: the backend stores packed cache representations and
 *     serves protected sink and recent tokens from bf16 buffers;
 *   - Figure 8 caption: a fused writer packs every incoming token and keeps the
 *     bf16 values of protected tokens; attention uses the bf16 values for
 *     protected tokens and dequantised values otherwise; the reconstructed
 *     content tile serves both matching (QK) and latent aggregation (PV); all
 *     valid tokens share one softmax normalisation;
 *   - Figure 5 / Table 9 captions: the protection policy is sink 4 / local 128.
 * The pages leave the quantiser open; this library fixes it as per-token
 * asymmetric quantisation over 64-channel groups with an fp16 scale and an fp16
 * min per group and round-half-to-even codes (details at mla_lowbit_write).
 *
 * Conventions for every call:
 *   - All tensors are device pointers unless marked "host".  The caller owns
 *     all memory; the library never allocates or frees device memory.
 *   - Calls are asynchronous on the caller's stream (`stream` is a
 *     cudaStream_t; NULL means the legacy default stream).
 *   - Return value: MLA_LOWBIT_OK or a negative MLA_LOWBIT_E* status for errors
 *     found on the host (bad layout, NULL pointer, misalignment, size, small
 *     workspace, launch failure).  Nothing is launched when a call fails.
 *   - Errors that only the device can see (a page id outside the pool, a
 *     position outside the block table, a sequence length out of range) are
 *     OR-ed into the int32 `err_word` (device memory, MLA_LOWBIT_DEV_* bits);
 *     the offending work is skipped, never trapped.  Read it with
 *     mla_lowbit_read_error.
 *   - Pointers to the page pool, bf16 buffers, queries, outputs and the
 *     workspace must be 16-byte aligned.
 */
#ifndef MLA_LOWBIT_H
#define MLA_LOWBIT_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Cache layout.  Supported (content_bits, rope_bits): (4,4) "C4R4", (2,4)
 * "C2R4", (16,16) unquantised bf16 pages.  The other fields must hold the
 * values shown (they are checked, so a caller states its assumptions). */
typedef struct mla_lowbit_layout {
  int content_bits; /* 4, 2, or 16 (bf16 pages) */
  int rope_bits;    /* 4, or 16 with bf16 pages */
  int group;        /* 64: channels per quantisation group */
  int sink;         /* 4: leading tokens kept in bf16 */
  int local;        /* 128: trailing tokens kept in bf16 */
  int page_tokens;  /* 64: tokens per page */
  int latent;       /* 512: content latent width (kv_lora_rank) */
  int rope;         /* 64: RoPE key width (qk_rope_head_dim) */
  int rotate;       /* 0, or 1 (packed layouts): online Hadamard rotation of the content
                       latent -- the writer replaces each 64-channel content group x by
                       R x, R = H_64 / 8 (orthonormal Sylvester-Hadamard; float32
                       butterfly stages h = 1, 2, .., 32, element i (bit h clear) and
                       i + h becoming (a + b, a - b), then x 1/8), rounded to bf16, for the
                       packed codes and the bf16 copies alike; decode rotates the
                       queries' content channels by R and rotates outputs back, so the
                       result is attention over R^T of the stored keys.  RoPE keys are
                       not rotated.  (QuantMLA, Table 1: QuaRot as an MLA-adapted
                       baseline; the pages' own transforms are fused offline -- this is
                       the un-fused variant.) */
} mla_lowbit_layout;

enum {
  MLA_LOWBIT_OK = 0,
  MLA_LOWBIT_EINVAL = -1,     /* bad layout or argument value */
  MLA_LOWBIT_ENULL = -2,      /* required pointer is NULL */
  MLA_LOWBIT_EALIGN = -3,     /* pointer not 16-byte aligned */
  MLA_LOWBIT_ESIZE = -4,      /* size outside the supported range */
  MLA_LOWBIT_EWORKSPACE = -5, /* workspace smaller than the plan needs */
  MLA_LOWBIT_ECUDA = -6       /* a CUDA runtime call or launch failed */
};

/* Bits OR-ed into the device error word. */
enum {
  MLA_LOWBIT_DEV_BAD_SEQ = 1,   /* writer: sequence index outside [0, num_seqs) */
  MLA_LOWBIT_DEV_BAD_POS = 2,   /* position < 0 or >= max_pages * 64 */
  MLA_LOWBIT_DEV_BAD_PAGE = 4,  /* block-table entry outside [0, num_pages) */
  MLA_LOWBIT_DEV_BAD_LEN = 8,   /* decode: seq_len < 0 or > max_pages * 64 */
  MLA_LOWBIT_DEV_PLAN = 16,     /* decode: device lengths disagree with seq_lens_host */
  MLA_LOWBIT_DEV_PIPELINE = 32, /* decode: an internal pipeline step failed -- a bounded wait gave up
                                  or shared memory was misaligned (the output is invalid) */
  MLA_LOWBIT_DEV_NO_ROOM = 64   /* assign: too few free pages or token slots (nothing was assigned) */
};

/* Element types of the calls that take more than one. */
enum { MLA_LOWBIT_BF16 = 0, MLA_LOWBIT_FP16 = 1, MLA_LOWBIT_FP32 = 2 };

/* OR-ed to mla_lowbit_read's out_dtype: the rows of skipped tokens become zeros. */
enum { MLA_LOWBIT_CLEAR_SKIPPED = 0x100 };

/* Scaling of the rotation's frequencies for contexts longer than the trained one. */
enum {
  MLA_LOWBIT_ROPE_NONE = 0,
  MLA_LOWBIT_ROPE_LINEAR = 1,
  MLA_LOWBIT_ROPE_NTK = 2,
  MLA_LOWBIT_ROPE_YARN = 3
};

/* Bytes of one 64-token page: 20736 (C4R4), 12544 (C2R4), 73728 (bf16).
 * Page layout (every region starts on a 128-byte boundary):
 *   packed: content codes [64][latent*content_bits/8] u8, then RoPE codes
 *           [64][rope*rope_bits/8] u8, then metadata [64][9] x {fp16 scale,
 *           fp16 min} (groups 0..7 content, 8 RoPE);
 *           INT4: channel 2i -> low nibble of byte i, 2i+1 -> high nibble;
 *           INT2: channel 4i+j -> bits 2j..2j+1 of byte i;
 *   bf16:   [64][576] bf16 (content then RoPE), no metadata.
 * Returns 0 for an unsupported layout. */
size_t mla_lowbit_page_bytes(const mla_lowbit_layout* layout);

/* Packed bytes per cached token: 324 (C4R4), 196 (C2R4), 1152 (bf16). */
size_t mla_lowbit_bytes_per_token(const mla_lowbit_layout* layout);

/* Fused cache writer (Figure 8 caption: each arriving token is packed, and the
 * bf16 values of protected tokens are kept in their own buffers).
 *
 * Token i (0 <= i < n_tokens) has content latent ckv[i][512] and RoPE key
 * krope[i][64] (bf16, already rotated), sequence seq_idx[i] (or i when seq_idx
 * is NULL) and position pos[i].  It is stored in page block_table[s][pos/64],
 * row pos%64.  For packed layouts each of its 9 groups of 64 channels is
 * quantised with bits b (content_bits for groups 0..7, rope_bits for group 8):
 *   mn, mx = min, max of the group (float32);
 *   s16 = fp16_rn(min((mx - mn) / (2^b - 1), 65504)), m16 = fp16_rn(mn clamped
 *   to +-65504), both float32 operations rounded to nearest;
 *   code = clamp(round_half_even((x - m16) / s16), 0, 2^b - 1) with float32
 *   subtraction and true division; every code is 0 when s16 == 0.
 * A packed copy is written for every token, protected or not.  In addition
 * (packed layouts only) a token with pos < 4 is copied to sink_buf[s][pos] and
 * a token with pos >= seq_lens_after[s] - 128 to recent_buf[s][pos % 128]
 * (seq_lens_after == NULL means pos[i] + 1, the one-token decode step).  Within
 * one call the positions of a sequence must be distinct.
 *
 *   ckv            [n_tokens][512] bf16        krope   [n_tokens][64] bf16
 *   seq_idx        [n_tokens] int32 or NULL    pos     [n_tokens] int32
 *   seq_lens_after [num_seqs] int32 or NULL
 *   block_table    [num_seqs][max_pages] int32 (physical page ids)
 *   page_pool      [num_pages][page_bytes] u8
 *   sink_buf       [num_seqs][4][576] bf16, recent_buf [num_seqs][128][576]
 *                  bf16 (may be NULL for bf16 pages)
 *   err_word       int32 (device), OR-ed MLA_LOWBIT_DEV_* bits
 */
int mla_lowbit_write(const mla_lowbit_layout* layout, int n_tokens, const void* ckv,
                     const void* krope, const int32_t* seq_idx, const int32_t* pos,
                     const int32_t* seq_lens_after, int num_seqs, const int32_t* block_table,
                     int max_pages, void* page_pool, int64_t num_pages, void* sink_buf,
                     void* recent_buf, int32_t* err_word, void* stream);

/* Split-KV plan of one decode call.  The work of a sequence is a list of
 * units: one per 64-token page that holds a packed-served token (bf16 pages:
 * every page), then, for packed layouts, its protected bf16 tokens (sink and
 * recent) in 64-token tiles of 3 units each.  The list is cut into splits of
 * `chunk_pages` units, chosen from the total work and the SM count: the
 * fewest waves of CTAs (one per SM) that the cap allows, or one or two more
 * waves of smaller chunks when the estimated time, waves x (chunk + 3), drops
 * by at least 5 %; the smallest chunk whose splits fit the waves.  The cap is
 * 128 units for the 128-row cluster kernel (query rows a multiple of 128,
 * no rotation) and 64 for the 16-row kernel; it bounds the tokens one split
 * accumulates in fp32 tensor-core outputs.  A bf16 tile belongs to the split
 * that holds its first unit.  Writes the number of splits and the workspace
 * bytes the call needs.  num_sms == 0 asks the current CUDA device. */
int mla_lowbit_decode_plan(const mla_lowbit_layout* layout, int num_seqs, int heads,
                           const int32_t* seq_lens_host, int num_sms, int* total_splits,
                           int* chunk_pages, size_t* workspace_bytes);

/* Low-bit MLA decode attention in absorbed form (Abstract: unpacking and
 * dequantisation inside attention; Figure 8 caption: bf16 values for
 * protected tokens, one global softmax, the content tile used for QK and PV).
 *
 * For sequence s with L = seq_lens[s] cached tokens and head h:
 *   key_t  = bf16 value of token t if t < 4 or t >= L - 128 (sink/recent
 *            buffers), else s16*code + m16 from its packed page (bf16 pages:
 *            always the page value);
 *   z_t    = softmax_scale * dot(q[s][h][0:576], key_t[0:576]);
 *   out[s][h][c] = sum_t softmax(z)_t * key_t[c],  c < 512 (value = latent);
 *   lse[s][h]    = log(sum_t exp(z_t)) (natural log; -inf and out = 0 when L = 0).
 * heads must be a multiple of 16, at most 128 (mla_lowbit_decode_plan takes
 * the rows of a sequence: heads, or n * heads for mla_lowbit_decode_multi,
 * at most 2048).  On packed layouts queries and protected values take part as
 * fp16: magnitudes from 65,536 on are infinite there, and what is below 2^-24 is lost.
 *
 *   q             [num_seqs][heads][576] bf16
 *   page_pool     [num_pages][page_bytes] u8 (as written by mla_lowbit_write)
 *   block_table   [num_seqs][max_pages] int32
 *   seq_lens      [num_seqs] int32 (device) and seq_lens_host (host, same
 *                 values; used to plan the split grid)
 *   sink_buf, recent_buf as for the writer (ignored for bf16 pages)
 *   out           [num_seqs][heads][512] float32
 *   lse           [num_seqs][heads] float32, or NULL
 *   workspace     at least the bytes mla_lowbit_decode_plan reports
 *   err_word      int32 (device), OR-ed MLA_LOWBIT_DEV_* bits
 * Launches the split kernel and the log-sum-exp combine kernel on `stream`.
 * The split kernel is fixed by the layout and the row count: packed,
 * unrotated layouts with a multiple of 128 rows per sequence run on tcgen05
 * tensor cores as 2-CTA clusters; every other call runs on mma.sync
 * tensor-core instructions in 16-row chunks. */
int mla_lowbit_decode(const mla_lowbit_layout* layout, int num_seqs, int heads,
                      float softmax_scale, const void* q, const void* page_pool,
                      int64_t num_pages, const int32_t* block_table, int max_pages,
                      const int32_t* seq_lens, const int32_t* seq_lens_host,
                      const void* sink_buf, const void* recent_buf, float* out, float* lse,
                      void* workspace, size_t workspace_bytes, int32_t* err_word,
                      void* stream);

/* One decode step with its append (QuantMLA, Figure 8 caption: the writer packs
 * every incoming token and attention runs over the packed cache and the bf16
 * buffers): writes the token at position seq_lens[s] - 1 of every sequence
 * exactly as mla_lowbit_write does with pos = seq_lens[s] - 1 and
 * seq_lens_after = seq_lens, then decodes exactly as mla_lowbit_decode over
 * seq_lens[s] tokens.  Results (pool bytes, bf16 buffers, out, lse) are
 * identical to that pair of calls.  For packed layouts on the default split
 * kernel both happen in the decode launch (the new token is inside the recent
 * window, so no packed split reads the bytes being written, and the bf16
 * split reads the new values from ckv_new/krope_new, rotating the content
 * latent itself on a rotated layout); otherwise the writer kernel runs first
 * on `stream`.
 *
 *   ckv_new    [num_seqs][512] bf16, krope_new [num_seqs][64] bf16 (16-byte aligned)
 *   seq_lens   device, every entry >= 1 (seq_lens_host the same values)
 *   page_pool, sink_buf, recent_buf are written (as by mla_lowbit_write)
 * Other arguments, errors and the workspace as for mla_lowbit_decode;
 * seq_lens_host entries < 1 return MLA_LOWBIT_EINVAL. */
int mla_lowbit_write_decode(const mla_lowbit_layout* layout, int num_seqs, int heads,
                            float softmax_scale, const void* q, const void* ckv_new,
                            const void* krope_new, void* page_pool, int64_t num_pages,
                            const int32_t* block_table, int max_pages, const int32_t* seq_lens,
                            const int32_t* seq_lens_host, void* sink_buf, void* recent_buf,
                            float* out, float* lse, void* workspace, size_t workspace_bytes,
                            int32_t* err_word, void* stream);

/* Multi-token query decode (several new tokens per sequence at once, as for
 * multi-token prediction or speculative verification): queries_per_seq = n
 * queries per sequence at positions L - n .. L - 1 (L = seq_lens[s], all n
 * tokens already written), each attending causally: query i sees tokens
 * 0 .. L - n + i.  Same arithmetic, tolerance and errors as mla_lowbit_decode
 * otherwise; the n queries run as n blocks of `heads` rows over one pass of the
 * cache (the masked tokens are all inside the recent window, 1 <= n <= 16).
 * On the 128-row kernel (n * heads a multiple of 128) a value of these n tokens that
 * is not finite reaches the queries before it too.
 *
 *   q      [num_seqs][n][heads][576] bf16
 *   out    [num_seqs][n][heads][512] float32; lse [num_seqs][n][heads] or NULL
 *   seq_lens_host entries >= n
 *   workspace  mla_lowbit_decode_plan with heads = n * heads
 * The split kernel is chosen as for mla_lowbit_decode from the row count
 * n * heads (so 128-row blocks run on tcgen05). */
int mla_lowbit_decode_multi(const mla_lowbit_layout* layout, int num_seqs, int queries_per_seq,
                            int heads, float softmax_scale, const void* q, const void* page_pool,
                            int64_t num_pages, const int32_t* block_table, int max_pages,
                            const int32_t* seq_lens, const int32_t* seq_lens_host,
                            const void* sink_buf, const void* recent_buf, float* out, float* lse,
                            void* workspace, size_t workspace_bytes, int32_t* err_word,
                            void* stream);

/* mla_lowbit_decode for callers that cannot allocate device memory.  The
 * pages have no counterpart to this entry point: it exists because some hosts
 * give a kernel only its inputs and outputs -- a serving engine that has
 * already reserved almost all of HBM for its own cache pool, a plug-in
 * interface without a workspace argument, or a loop that cannot afford the
 * device-wide synchronisation of cudaMalloc.
 *
 * Same arguments, results and error handling as mla_lowbit_decode, minus the
 * workspace: the split partials live in a fixed 32 MiB device array owned by
 * the library (every GPU that loads the library holds it until the process
 * exits).  Calls whose plan needs more than 32 MiB (see
 * mla_lowbit_decode_plan) return MLA_LOWBIT_ESIZE and launch nothing.  The
 * call allocates and frees nothing.
 *
 * The first call on a device looks up that device's address of the array
 * (cudaGetSymbolAddress, with that device current); make that first call
 * before any stream capture.  All calls share the one array and it keeps the
 * last call's contents (nothing in it needs to start at zero: each call writes
 * every byte it reads).  Calls that overlap on the GPU -- on different streams,
 * or from different threads without ordering -- race on the array; issue them
 * on one stream or order them yourself. */
int mla_lowbit_decode_noalloc(const mla_lowbit_layout* layout, int num_seqs, int heads,
                              float softmax_scale, const void* q, const void* page_pool,
                              int64_t num_pages, const int32_t* block_table, int max_pages,
                              const int32_t* seq_lens, const int32_t* seq_lens_host,
                              const void* sink_buf, const void* recent_buf, float* out,
                              float* lse, int32_t* err_word, void* stream);

/* ---------------------------------------------------------------------------
 * The rest of a serving step: slots for arriving tokens, the norm and the
 * rotation between projections and cache, the append from a projection's
 * output, cached tokens back as values, and attention over a sliding window.
 * Every length that these calls use lives on the device, so a captured graph of
 * a step stays valid while sequences grow, end and begin.
 * ------------------------------------------------------------------------- */

/* Block tables and slot maps of one step, from the requests' lengths.
 *
 * Sequence s holds seq_lens[s] tokens in the pages block_table[s][0 ..
 * ceil(seq_lens[s] / 64) - 1].  It first gives them all back when release[s] is
 * not 0 (release may be NULL: none does), then gets room for new_lens[s] >= 0
 * tokens.  The free pages are a stack: free_pages[0 .. free_count - 1].
 *   - The pages of released sequences are pushed on it, sequence after
 *     sequence, each one's pages in order: the first is free_pages[free_count].
 *   - New pages are popped from its top, sequence after sequence, page after
 *     page: a page that was pushed in this call can be taken in it.  The new
 *     pages' ids are written to block_table; its other entries stay.
 *   - Nothing is erased: popped entries of free_pages and the rows of released
 *     sequences in block_table keep their last values.
 * Outputs:
 *   seq_lens_after   [num_seqs] tokens held after the step (may be seq_lens)
 *   free_count_after [1] (may be free_count)
 *   token_start      [num_seqs + 1] first flattened token of each sequence, and
 *                    the total, or NULL
 *   seq_idx, pos     [max_tokens] sequence and position of every new token, in
 *                    the order of sequences and positions: the arguments of
 *                    mla_lowbit_write and mla_lowbit_norm_rope_write
 *   slots            [max_tokens] int64 page * 64 + row, or NULL
 * Entries of seq_idx, pos and slots behind the last token are set to -1.
 *
 * All or nothing: when a length is out of range (DEV_BAD_LEN: seq_lens[s] or
 * the length after the step outside [0, max_pages * 64], or new_lens[s] < 0), or
 * pages or slots are too few or the stack would overflow (DEV_NO_ROOM),
 * nothing is assigned or released: lengths and count are copied, token_start is
 * 0 and every slot -1.  A page id outside [0, num_pages) that is met on the
 * stack or in a released row sets DEV_BAD_PAGE and is passed on as it is (its
 * tokens' slots are -1).  A page belongs to one sequence.
 * num_seqs <= 8192, num_seqs * max_pages <= INT32_MAX; num_pages is the length
 * of free_pages.  seq_idx, pos and slots are 16-byte aligned.  Two calls on the
 * same state must be ordered by the caller. */
int mla_lowbit_assign(int num_seqs, int max_pages, int num_pages, int max_tokens,
                      const int32_t* new_lens, const int32_t* release, const int32_t* seq_lens,
                      const int32_t* free_count, int32_t* block_table, int32_t* free_pages,
                      int32_t* seq_lens_after, int32_t* free_count_after, int32_t* token_start,
                      int32_t* seq_idx, int32_t* pos, int64_t* slots, int32_t* err_word,
                      void* stream);

/* Frequencies of a rotation of `rot` channels (host): phase[i], i < rot / 2, is
 * the turn of pair i per position in units of 2^-64 turns, so that
 * pos * phase[i] mod 2^64 is the angle of any int32 position without loss.
 *   f_i = theta^(-2i/rot) radians a position;
 *   LINEAR: f_i / factor;
 *   NTK:    theta is theta * factor^(rot/(rot-2)) (rot > 2);
 *   YARN:   f_i (1 - r_i) + (f_i / factor) r_i, r_i = clamp((i - low) /
 *           max(high - low, 0.001), 0, 1), low = max(floor(c(beta_fast)), 0),
 *           high = min(ceil(c(beta_slow)), rot - 1), c(b) = rot ln(original_len
 *           / (2 pi b)) / (2 ln theta); *mscale = 0.1 ln(factor) + 1.
 * *mscale is 1 for the others.  (YaRN's factor for heads that are rotated whole.
 * Checkpoints whose key is rotated in a part give mscale and mscale_all_dim: with
 * t(m) = 0.1 m ln(factor) + 1 the calls' mscale is t(mscale) / t(mscale_all_dim),
 * and softmax_scale is multiplied by t(mscale_all_dim)^2.)  rot even, 2..2048; theta > 1; factor >= 1;
 * YARN: original_len >= 1, beta_fast >= beta_slow > 0. */
int mla_lowbit_rope_table(int rot, double theta, int scaling, double factor, int original_len,
                          double beta_fast, double beta_slow, uint64_t* phase_host,
                          float* mscale_host);

/* Norm of heads and rotation of a part of them, in one pass.
 *
 * Row (i, h), i < n_tokens, h < heads, has `dim` channels from
 * x + i * x_token_stride + h * x_head_stride (strides in elements, the channels
 * contiguous; strides of 0 share rows):
 *   norm:     v = x * w / sqrt(mean(x^2) + eps) (w = weight[dim], 1 when NULL);
 *             norm == 0: v = x;
 *   rotation: channels offset .. offset + rot - 1 of v, in pairs (2i, 2i + 1)
 *             when interleaved, else (i, i + rot/2), are turned by the angle of
 *             pos[i] (any int32) and multiplied by mscale; rot == 0: none.
 * Computed in float32 and rounded once.  y has strides of its own, which must
 * not make its rows overlap; y may be x itself (same pointer and strides), and
 * must not overlap it otherwise.  Arrays between whose ends the other one begins are
 * taken where they show to be apart: with the same strides as other columns of the
 * rows, with the same token stride as other columns of the tokens (the heads'
 * strides may differ), with the same head stride as other columns of the heads.
 *   x, y, weight   of type dtype (MLA_LOWBIT_BF16, _FP16, _FP32), aligned to it
 *   phase          [rot / 2] device copy of mla_lowbit_rope_table's
 *   pos            [n_tokens] int32
 * dim 1..2048, rot even, offset + rot <= dim, heads >= 1, n_tokens * heads <=
 * 2^31 - 1025. */
int mla_lowbit_norm_rope(int dtype, int n_tokens, int heads, int dim, const void* x,
                         int64_t x_token_stride, int64_t x_head_stride, void* y,
                         int64_t y_token_stride, int64_t y_head_stride, int norm,
                         const void* weight, float eps, int rot, int offset, int interleaved,
                         const uint64_t* phase, float mscale, const int32_t* pos, void* stream);

/* mla_lowbit_write from a projection's output: row i of kv (bf16, kv_stride
 * elements a row) holds the raw latent kv[i][0:512] and the raw key
 * kv[i][512:576].  What is written is, each rounded once to bf16 (to nearest
 * even from more than 32 bits, so that the packed codes are those of exact
 * arithmetic; where the sum of squares or a product leaves float32's normal
 * range, from float32 as it is),
 *   ckv   = latent * w / sqrt(mean(latent^2) + eps), w = weight[512] bf16 or
 *           NULL (1);
 *   krope = the key rotated at pos[i] as by mla_lowbit_norm_rope (rot 64);
 * and then exactly as mla_lowbit_write writes (ckv, krope), an online rotation
 * (layout field `rotate`) included.  Tokens with seq_idx[i] < 0 are padding and
 * are skipped without an error.  ckv_out [n][512] and krope_out [n][64] (bf16,
 * 16-byte aligned, or NULL) receive ckv and krope (before an online rotation;
 * rows of padding and of tokens with an error stay as they were).
 * kv is aligned to 2 bytes, weight and phase to 16. */
int mla_lowbit_norm_rope_write(const mla_lowbit_layout* layout, int n_tokens, const void* kv,
                               int64_t kv_stride, const void* weight, float eps, int interleaved,
                               const uint64_t* phase, float mscale, const int32_t* seq_idx,
                               const int32_t* pos, const int32_t* seq_lens_after, int num_seqs,
                               const int32_t* block_table, int max_pages, void* page_pool,
                               int64_t num_pages, void* sink_buf, void* recent_buf, void* ckv_out,
                               void* krope_out, int32_t* err_word, void* stream);

/* Cached tokens as values: out[i][0:576] is the key of token (seq_idx[i],
 * pos[i]) as decode uses it for a sequence of seq_lens[s] tokens: the bf16 value
 * of a protected token (pos < 4 or pos >= seq_lens[s] - 128), else
 * s16 * code + m16 (float32, one rounding).  seq_lens == NULL: the packed copy
 * of every token (sink_buf and recent_buf may then be NULL).  On a rotated cache
 * the content groups are rotated back (R, float32).  out is of type out_dtype
 * (MLA_LOWBIT_BF16, to nearest even, or MLA_LOWBIT_FP32), 16-byte aligned.
 * Tokens may come in any order and more than once; seq_idx[i] < 0 is skipped
 * without an error.  A sequence index or position out of range (with seq_lens:
 * pos >= seq_lens[s] too) or a bad page sets its error bit and the token is
 * skipped.  The rows of skipped tokens stay as they were, or become zeros (out_dtype
 * | MLA_LOWBIT_CLEAR_SKIPPED). */
int mla_lowbit_read(const mla_lowbit_layout* layout, int n_tokens, const int32_t* seq_idx,
                    const int32_t* pos, int num_seqs, const int32_t* seq_lens,
                    const int32_t* block_table, int max_pages, const void* page_pool,
                    int64_t num_pages, const void* sink_buf, const void* recent_buf, int out_dtype,
                    void* out, int32_t* err_word, void* stream);

/* Splits and workspace of mla_lowbit_decode_window: from the sizes alone, never
 * from the lengths, so it holds for every step of a cache.  num_sms == 0 asks
 * the current CUDA device.  Every sequence gets the same number of splits and
 * cuts its own units (a page with a visible token, or a tile of 64 protected
 * tokens) into that many chunks, equal ones or with a shorter last one. */
int mla_lowbit_window_plan(const mla_lowbit_layout* layout, int num_seqs, int heads,
                           int queries_per_seq, int window, int sinks, int max_pages, int num_sms,
                           int* splits_per_seq, size_t* workspace_bytes);

/* mla_lowbit_decode_multi over a sliding window and the first tokens: query i
 * of sequence s, at position p = seq_lens[s] - n + i (1 <= n <= 16), sees the
 * tokens t <= p with t < sinks or t > p - window.  window >= 1; sinks >= 0; both
 * may exceed the sequence (window >= its length: plain causal attention).  A
 * query with p < 0 (a sequence of fewer than n tokens, 0 for an idle row of the
 * batch) sees nothing: its output is 0 and its lse -inf.  The pages of tokens
 * that no query sees are not touched, and their block_table entries not read; a
 * token whose values are not finite reaches the queries that see it and no other.
 * seq_lens is read on the device only.
 *   q    [num_seqs][n][heads][576] bf16
 *   out  [num_seqs][n][heads][512] float32 or bf16 (out_dtype)
 *   lse  [num_seqs][n][heads] float32 or NULL
 *   workspace  mla_lowbit_window_plan's bytes (of this device)
 * Two calls that may overlap need workspaces of their own, and so do graphs
 * that may.  Everything else as mla_lowbit_decode_multi.
 *
 * Accuracy: mla_lowbit_decode's, max-abs 2e-3, rel-L2 1e-3 of exact attention over
 * the cached values.  The sizes choose between the two split kernels, so a sequence's
 * last bits, and its accuracy, change with the size of its batch.  The 16-row kernel
 * came out at 5e-7 of the result's norm (8 x 1,024 tokens) and 1e-4 at most in the lse;
 * the cluster kernel at 2.5e-5 (32 x 4,096 tokens, 128 heads, INT4), its logits being
 * sums in tensor memory that cut instead of rounding, and on packed pages its lse can
 * be off by slightly more than 1e-4 where a 64-channel group holds outliers.  A result
 * repeats bit for bit with the same arguments. */
int mla_lowbit_decode_window(const mla_lowbit_layout* layout, int num_seqs, int queries_per_seq,
                             int heads, float softmax_scale, int window, int sinks, const void* q,
                             const void* page_pool, int64_t num_pages, const int32_t* block_table,
                             int max_pages, const int32_t* seq_lens, const void* sink_buf,
                             const void* recent_buf, int out_dtype, void* out, float* lse,
                             void* workspace, size_t workspace_bytes, int32_t* err_word,
                             void* stream);

/* Self-test of the failure path of the tcgen05 decode kernels (the pages have
 * no counterpart to it; it checks this library's own error handling).  Those
 * kernels hand work between warp roles through mbarriers, and every wait on
 * one is bounded: when it runs out the CTA sets MLA_LOWBIT_DEV_PIPELINE in the
 * error word, its warps leave their loops together, the tensor-core work
 * already issued drains, tensor memory is freed and the kernel returns (no
 * trap, the context stays usable; the call's output is invalid).
 *
 * This sets, for every later decode call of the process (all threads):
 *   mode        0: normal operation; 1: the 128-row (tcgen05) decode kernel's
 *               unpack warps withhold their first hand-off, so that the waits
 *               behind it run out -- a fault made on purpose, for tests only;
 *   wait_cycles the wait limit in SM clock cycles; 0 restores the default
 *               (about one second).
 * Returns MLA_LOWBIT_EINVAL for a mode other than 0 or 1 or a negative limit.
 * The mma.sync kernel has no such waits and ignores both settings. */
int mla_lowbit_set_fault_injection(int mode, int64_t wait_cycles);

/* Synchronously copies the device error word to *code_out (a blocking
 * cudaMemcpy: it waits for prior work on the legacy default stream). */
int mla_lowbit_read_error(const int32_t* err_word, int32_t* code_out);

/* Human-readable text for a status code; never NULL. */
const char* mla_lowbit_strerror(int status);

/* Library version, major*10000 + minor*100 + patch. */
int mla_lowbit_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MLA_LOWBIT_H */
