/*
 * exact_attention.h -- C ABI of libexattn.so, the fused exact-attention forward for sm_103a.
 *
 * The operation (problem statement of "FlashAttention · InkStack", opening of "FlashAttention 1:
 * Data Movement", and the stored statistic of its section 2.1 "优化 Online Softmax"):
 *
 *     O   = softmax(scale * Q K^T + mask) V
 *     LSE = log sum_j exp(scale * q_i . k_j)     (natural log, over the keys row i may see)
 *
 * computed in one kernel launch without writing the N x N scores or probabilities anywhere:
 * Q is tiled into 128-row blocks, K/V are streamed in 128-row blocks, and each row keeps the
 * online-softmax state (running max m, running sum l, unnormalised output) on chip, merged with
 * the rescale factor alpha = e^(m_old - m_new) ("FlashAttention · InkStack", section 1.1.2).
 * The causal mask is lower-triangular with the diagonal included (key j visible to query i iff
 * j <= i); fully masked key blocks are skipped.
 *
 * Layout (all row-major, head dimension fastest, no padding between rows):
 *   q, k, v : [B, H, N, d], bf16 or fp8 e4m3fn (all three the same dtype)
 *   o       : [B, H, N, d], bf16 for both operand dtypes
 *   lse     : [B, H, N], fp32
 *
 * Ownership: every pointer is caller-owned device memory.  The library allocates no device
 * memory, frees nothing and keeps no pointer after the call returns.  The kernel runs
 * asynchronously on `stream` (a cudaStream_t, NULL = legacy default stream); the caller keeps
 * the buffers alive until the stream has passed the launch.  No call synchronises the stream.
 *
 * Errors: arguments are checked on the host before anything is launched; a failed check returns
 * a status code and launches nothing.  A launch failure returns FA_ERR_CUDA.  Inside the kernel
 * every wait is bounded in time; a wait that runs out makes the kernel stop early, free its
 * tensor memory and record FA_ERR_DEVICE_TIMEOUT in the device status word (see
 * fa_device_status / fa_fwd_opts.dev_status).  No exception crosses this interface.
 */
#ifndef EXACT_ATTENTION_H
#define EXACT_ATTENTION_H

#include <stddef.h>

#if defined(__GNUC__)
#define FA_API __attribute__((visibility("default")))
#else
#define FA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FA_DTYPE_BF16 = 0,          /* q, k, v are bf16 */
  FA_DTYPE_FP8_E4M3 = 1,      /* q, k, v are fp8 e4m3fn with fp32 descales; both products are
                                 fp8 ("FlashAttention · InkStack", section 3.3): P is rounded to
                                 e4m3, up to 2^-4 relative per probability, so a row whose mass
                                 sits on a few keys carries that error on O.  With the causal
                                 mask the first 256 query rows of every head (which see at most
                                 256 keys) take the f16 P V product of FP8_E4M3_PV16, in a
                                 second, small launch on the same stream */
  FA_DTYPE_FP8_E4M3_PV16 = 2  /* as FP8_E4M3, but the P V product is f16: P rounded to f16, V
                                 widened exactly from e4m3 in shared memory (slower; S = Q K^T
                                 stays an fp8 product) */
} fa_dtype;

typedef enum {
  FA_OK = 0,
  FA_ERR_INVALID_ARG = 1,    /* null pointer, non-positive size, bad scale or dtype */
  FA_ERR_UNSUPPORTED = 2,    /* head dim not in {64, 128}, or sizes beyond the kernel's limits */
  FA_ERR_MISALIGNED = 3,     /* a pointer is not 16-byte aligned */
  FA_ERR_CUDA = 4,           /* a CUDA runtime or driver call failed (no device, launch error) */
  FA_ERR_DEVICE_TIMEOUT = 5  /* a bounded wait inside the kernel ran out; outputs are invalid */
} fa_status;

/*
 * Attention forward.
 *   q, k, v : device pointers, [B, H, N, d] of `dtype` (16-byte aligned)
 *   o       : device pointer, [B, H, N, d] bf16 (16-byte aligned)
 *   lse     : device pointer, [B, H, N] fp32 (4-byte aligned)
 *   B, H, N : >= 1, with B * H <= 65535 and N < 2^31 - 512 (causal: N <= 65535 * 256)
 *   d       : head dimension, 64 or 128
 *   scale   : softmax scale applied to q . k, finite and >= 0 (usually 1/sqrt(d))
 *   causal  : 0 = no mask, nonzero = lower-triangular mask (diagonal included)
 *   dtype   : an fa_dtype; FP8_E4M3 uses descales of 1.0 here (see fa_fwd_ex)
 *   stream  : a cudaStream_t
 * Returns an fa_status.
 */
FA_API int fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int N,
           int d, float scale, int causal, int dtype, void* stream);

/*
 * Options of fa_fwd_ex.  For fp8 operands the stored values are code * descale: the scores are
 * scale * descale_q * descale_k * (q . k) and the output is descale_v * (P V) (per-tensor
 * scaling of "FlashAttention · InkStack", section 3.3.3 "Scaling").  The descales must be
 * finite and > 0; they are ignored for bf16.  `dev_status`, if not NULL, is a device int the
 * kernel sets to FA_ERR_DEVICE_TIMEOUT when a wait runs out (it never writes FA_OK: clear it
 * before the call); if NULL the library's own per-device status word is used instead.
 */
typedef struct {
  float descale_q;
  float descale_k;
  float descale_v;
  int* dev_status;
} fa_fwd_opts;

/* fa_fwd with options; `opts` may be NULL (descales 1.0, library status word). */
FA_API int fa_fwd_ex(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
              int N, int d, float scale, int causal, int dtype, const fa_fwd_opts* opts,
              void* stream);

/*
 * Key-split ("split-KV") variant of fa_fwd_ex.  The key blocks each query tile visits are
 * divided into `num_splits` contiguous ranges processed by separate CTAs (more parallelism when
 * B * H * ceil(N / 256) is small next to the GPU's SM count); each range leaves its normalised
 * output and log-sum-exp in `workspace`, and a second kernel merges the ranges with the
 * associative log-sum-exp merge ("FlashAttention · InkStack", section 2.2: independent key
 * blocks merged by an associative operation; the (m, l, U) recurrence of section 1.1.2).
 *   num_splits      : 1..16 (1 = fa_fwd_ex; workspace may then be NULL)
 *   workspace       : caller-owned device scratch, 16-byte aligned, at least
 *                     fa_fwd_split_workspace_bytes(B, H, N, d, num_splits) bytes; its contents
 *                     on entry do not matter and are undefined on return
 * Other arguments, layouts and errors as fa_fwd_ex; too small a workspace is
 * FA_ERR_INVALID_ARG.  The result equals fa_fwd_ex's up to fp32 rounding.
 */
FA_API int fa_fwd_split(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                        int H, int N, int d, float scale, int causal, int dtype, int num_splits,
                        void* workspace, size_t workspace_bytes, const fa_fwd_opts* opts,
                        void* stream);

/* Workspace bytes fa_fwd_split needs: num_splits * B * H * N * (d + 1) * 4, rounded up to 256;
 * 0 for invalid arguments. */
FA_API size_t fa_fwd_split_workspace_bytes(int B, int H, int N, int d, int num_splits);

/*
 * fa_fwd_split without any allocation, for callers that cannot allocate device memory when they
 * call: a plug-in whose host owns all of the GPU's memory and forbids libraries from allocating,
 * or a serving loop that must not stall or fail on an allocation mid-request.  The paper has no
 * counterpart of this entry point; it is an interface convenience of this library.
 *
 * Instead of a caller workspace, the split partials live in a fixed 64 MiB scratch array inside
 * the library's device image (every GPU that loads the library holds it until the process
 * exits).  The caller still passes inputs and outputs.  No call allocates or frees memory.
 *   - The first call on a device looks up the scratch's device address (cudaGetSymbolAddress,
 *     with that device current); make that first call before any stream capture.
 *   - Problems whose partials need more than 64 MiB, i.e.
 *     fa_fwd_split_workspace_bytes(B, H, N, d, num_splits) > 64 MiB, return FA_ERR_UNSUPPORTED
 *     and launch nothing.  num_splits == 1 needs no scratch and behaves as fa_fwd_ex.
 *   - Every call on a device shares the one array and leaves its last contents there; nothing in
 *     it needs to start at zero (every partial is written before it is read).  Calls whose
 *     kernels overlap on the GPU (concurrent streams on the same device) race on the array and
 *     give undefined results: serialise them.
 * Other arguments, layouts and errors as fa_fwd_split.
 */
FA_API int fa_fwd_split_noalloc(const void* q, const void* k, const void* v, void* o,
                                float* lse, int B, int H, int N, int d, float scale, int causal,
                                int dtype, int num_splits, const fa_fwd_opts* opts,
                                void* stream);

/*
 * fp8 forward with block scaling ("FlashAttention · InkStack", section 3.3.1 "Block
 * Quantization"; "FlashAttention 完全拆解（三）", section on block quantisation): every block of
 * 128 consecutive rows of one head of Q, K and V carries its own descale, so the stored value of
 * row i of head (b, h) is code * descale_X_blk[(b * H + h) * nblk + i / 128], nblk = ceil(N / 128).
 * Score block (i, j) is then scale * dq_i * dk_j * (q . k) and the output sum_j P_ij dv_j V_j.
 *   q, k, v           : device pointers, [B, H, N, d] e4m3fn codes (16-byte aligned)
 *   dtype             : FA_DTYPE_FP8_E4M3 or FA_DTYPE_FP8_E4M3_PV16 (precision of P V)
 *   descale_*_blk     : device pointers, [B, H, nblk] fp32 (4-byte aligned); every descale must
 *                       be finite and > 0 (fa_quantize_e4m3 writes such arrays), otherwise the
 *                       output is undefined (the kernel still runs to completion).  The value
 *                       descales enter P as dv_j / max_j dv_j: exact for powers of two, else
 *                       rounded with P (see FA_QUANT_POW2_DESCALE)
 *   num_splits, workspace, workspace_bytes : as fa_fwd_split (1 and NULL, 0 for no key split)
 *   dev_status        : as fa_fwd_opts.dev_status (NULL = the library's status word)
 * Other arguments, layouts and errors as fa_fwd_split.
 */
FA_API int fa_fwd_fp8_blockscaled(const void* q, const void* k, const void* v, void* o,
                                  float* lse, int B, int H, int N, int d, float scale,
                                  int causal, int dtype, const float* descale_q_blk,
                                  const float* descale_k_blk, const float* descale_v_blk,
                                  int num_splits, void* workspace, size_t workspace_bytes,
                                  int* dev_status, void* stream);

/* fa_quantize_e4m3 flag: round every descale up to a power of two (recommended for V). */
#define FA_QUANT_POW2_DESCALE 1

/*
 * Block quantiser to fp8 e4m3fn, with optional incoherent processing ("FlashAttention ·
 * InkStack", sections 3.3.1 "Block Quantization", 3.3.2 "Incoherent Processing" and 3.3.3
 * "Scaling").  For every block of 128 consecutive rows of each head:
 *     X'        = X diag(signs) Had / sqrt(d)   if signs != NULL (fast Walsh-Hadamard transform;
 *                 Had is the Sylvester-Hadamard matrix), else X' = X
 *     descale   = max |X'_blk| / 448            (1 if the block is all zero); with
 *                 FA_QUANT_POW2_DESCALE, the smallest power of two >= that quotient
 *     scale     = 448 / max |X'_blk|            (1 / descale with FA_QUANT_POW2_DESCALE)
 *     code      = e4m3(X' * scale)              (round to nearest even, saturate at 448)
 * Apply the same `signs` to Q and K (QK^T is unchanged) and none to V.  Power-of-two value
 * descales let fa_fwd_fp8_blockscaled fold them into P exactly; other value descales add one
 * more e4m3 rounding of relative size up to 2^-4 to each probability.
 *   x        : device pointer, [B, H, N, d] bf16 (16-byte aligned)
 *   codes    : device pointer, [B, H, N, d] e4m3fn output (16-byte aligned)
 *   descales : device pointer, [B, H, ceil(N / 128)] fp32 output (4-byte aligned)
 *   signs    : device pointer to d fp32 values, each +1 or -1 (16-byte aligned), or NULL
 *   d        : 64 or 128; B * H <= 65535
 *   flags    : 0 or FA_QUANT_POW2_DESCALE (other bits: FA_ERR_INVALID_ARG)
 * Arithmetic is fp32 (descale and scale correctly rounded once per block).  Returns an
 * fa_status; asynchronous on `stream` like fa_fwd.
 */
FA_API int fa_quantize_e4m3(const void* x, void* codes, float* descales, int B, int H, int N,
                            int d, const float* signs, int flags, void* stream);

/*
 * Attention backward for bf16 operands ("FlashAttention · InkStack", section 1.2: dV = P^T dO,
 * dP = dO V^T, dS = P * (dP - D) with D_i = rowsum(dO_i * O_i), dQ = scale dS K,
 * dK = scale dS^T Q; P recomputed from the forward's LSE as in section 1.2.2).  Three kernel
 * launches on `stream`: D, then dK/dV, then dQ.
 *   q, k, v, o, dout : device pointers, [B, H, N, d] bf16 (16-byte aligned); o and lse are the
 *                      forward outputs for q, k, v (same scale and mask)
 *   lse              : device pointer, [B, H, N] fp32 (4-byte aligned), natural log
 *   dq, dk, dv       : device pointers, [B, H, N, d] bf16 outputs (16-byte aligned)
 *   workspace        : caller-owned device scratch of fa_bwd_workspace_bytes(B, H, N) bytes
 *                      (16-byte aligned), holds D; contents on entry do not matter
 *   dev_status       : as fa_fwd_opts.dev_status (NULL = the library's status word)
 * Sizes, scale, mask and errors as fa_fwd (d in {64, 128}); too small a workspace is
 * FA_ERR_INVALID_ARG.
 */
FA_API int fa_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse,
                  const void* dout, void* dq, void* dk, void* dv, int B, int H, int N, int d,
                  float scale, int causal, void* workspace, size_t workspace_bytes,
                  int* dev_status, void* stream);

/* Workspace bytes fa_bwd needs: B * H * N * 4, rounded up to 256; 0 for invalid arguments. */
FA_API size_t fa_bwd_workspace_bytes(int B, int H, int N);

/* fa_rope flags */
#define FA_ROPE_INTERLEAVED 1  /* pairs (2i, 2i + 1); without it (i, i + rotary_dim / 2) */
#define FA_ROPE_INVERSE 2      /* turn by the negative angle: the gradient of the forward map */

/*
 * Rotary positions of one or two tensors (queries and keys) in one launch.  Pair i of the first
 * `rotary_dim` values of each head vector at position p is turned by p * f_i:
 *     y_a = mscale (a cos - b sin),  y_b = mscale (b cos + a sin)
 * the other d - rotary_dim values are copied.  The map is mscale times a rotation, so the gradient
 * dL/dx of a loss is the same call on dL/dy with FA_ROPE_INVERSE and the same mscale.
 *   q, k            : device pointers, bf16 (16-byte aligned), last dimension contiguous;
 *                     *_strides = {batch, head, row} strides in elements, multiples of 8, >= 0.
 *                     [B, H, N, d] and packed tokens [T, H, d] (B = 1, N = T) are both such
 *   q_out, k_out    : outputs, likewise; an output may be its own input (same pointer and
 *                     strides), any other overlap gives undefined results
 *   Hq, Hk          : heads of each; Hk = 0: no second tensor (k, k_out and strides unused)
 *   positions       : device int32, [N] with positions_batch_stride = 0 (shared by the batch) or
 *                     [B, N]; any int32 value
 *   turns           : device int64, [rotary_dim / 2]: f_i / (2 pi) in units of 2^-64 turn.  The
 *                     product with a position wraps to the exact fraction of a turn, so angles of
 *                     far positions keep fp32 accuracy.  Scalings for long contexts are made in
 *                     this table (and in mscale)
 *   B, N            : >= 1;  d : 64 or 128;  rotary_dim : a multiple of 16, <= d
 * Arithmetic is fp32 with one rounding to bf16.  Returns an fa_status; asynchronous like fa_fwd.
 */
FA_API int fa_rope(const void* q, const long long* q_strides, void* q_out,
                   const long long* q_out_strides, int Hq, const void* k,
                   const long long* k_strides, void* k_out, const long long* k_out_strides, int Hk,
                   int B, int N, int d, const int* positions, long long positions_batch_stride,
                   const long long* turns, int rotary_dim, int flags, float mscale, void* stream);

/*
 * Rotary positions with several axes (time, height and width of image and video tokens): as fa_rope, but each
 * token has a position on each of num_axes axes and pair i turns by position[axes[i]] * f_i.
 *   positions : device int32; the position of row n of batch b on axis x lies at
 *               x * positions_axis_stride + b * positions_batch_stride + n (strides >= 0; 0: shared)
 *   num_axes  : 1 to 4
 *   axes      : device uint8 [rotary_dim / 2] (8-byte aligned), the axis of each pair; an axis >= num_axes
 *               counts as axis 0
 * The rest, the gradient (FA_ROPE_INVERSE) included, as fa_rope.
 */
FA_API int fa_rope_axes(const void* q, const long long* q_strides, void* q_out,
                        const long long* q_out_strides, int Hq, const void* k,
                        const long long* k_strides, void* k_out, const long long* k_out_strides,
                        int Hk, int B, int N, int d, const int* positions, int num_axes,
                        long long positions_axis_stride, long long positions_batch_stride,
                        const unsigned char* axes, const long long* turns, int rotary_dim, int flags,
                        float mscale, void* stream);

/*
 * One step of a paged cache's bookkeeping, on the device: which request gets which pages, and
 * where each new token goes.  Request b holds lens[b] tokens in the pages table[b, 0 ..
 * ceil(lens[b] / page_size)); it brings new_lens[b] tokens, or, with new_lens[b] < 0, it has ended
 * and its pages return to the free ones.
 *   queue, queue_state : ring of `queue_size` free page ids; queue_state = {head, count}: the free
 *                        pages are queue[(head + i) % queue_size], i < count.  The ring should have
 *                        room for every page there is: of the pages that a step gets back it keeps
 *                        the first queue_size - count (count as the step found it), the rest are lost
 * Requests take pages from the front in their order.  A request is refused (keeps its length and
 * pages, gets no slots) when its table row is too narrow, or when it needs pages and the sum of
 * all needs up to and with its own exceeds count.  Pages of ended requests become free behind the
 * others, for the next step.
 *   table           : [B, table_width], new entries written, others left as they are
 *   lens_out        : [B] lengths after the step (0 for ended requests)
 *   q_offsets       : [B + 1] first token of each request in the packed batch, and their number
 *   positions, slots: [num_tokens] position and cache slot (page * page_size + row) of each token;
 *                     slot -1 for tokens of refused requests and on page ids that no cache has
 *                     (negative, or page_size * id >= 2^31); position 0 and slot -1 past the last
 *                     token.  num_tokens = 0: neither is written (they may be NULL)
 *   queue_state_out : {head, count} after the step
 *   num_tokens      : size of the packed batch, the refused requests' tokens included; tokens past
 *                     it get no place, although their requests' lengths grow
 *   page_size       : 16, 32, 64 or 128;  1 <= B <= 16384;  table_width * page_size <= 2^30;
 *                     B * table_width < 2^31;  the tokens of a step number < 2^31
 * All arrays are device int32.  No output may overlap an input or another output (lens_out and
 * queue_state_out are refused when they are the inputs; the table and the ring are both).  One launch,
 * integers only: results do not depend on scheduling.
 */
FA_API int fa_page_plan(const int* lens, const int* new_lens, int* table, int table_width,
                        int* queue, int queue_size, const int* queue_state, int B, int page_size,
                        int num_tokens, int* lens_out, int* q_offsets, int* positions, int* slots,
                        int* queue_state_out, void* stream);

/*
 * The 4-bit key/value cache: [num_pages, Hkv, 2 (keys, values), page_size * 9 d / 16] bytes.  Each
 * block holds page_size rows of d / 2 bytes of e2m1 codes (value 2i in the low half of byte i),
 * then page_size rows of d / 16 e4m3 scales, one for 16 neighbouring values:
 *     scale = e4m3(max |x / descale| / 6),  code = e2m1(x / descale / scale),
 *     value = code * scale * descale              (both roundings to nearest even, saturating)
 * descale is one power of two per tensor, the same in every call on the cache.  A head vector that
 * holds a NaN or an infinity reads back as NaN.  Slot s is row s % page_size of page s / page_size.
 * The bytes do not tell (d 64, page_size 2 p) from (d 128, page_size p): all calls on a cache take those
 * that it was made for.  Bytes of such a cache; 0 for invalid arguments.
 */
FA_API size_t fa_kv4_cache_bytes(int num_pages, int Hkv, int page_size, int d);

/*
 * Write keys and values into the cache.
 *   k, v      : device pointers, [T, Hkv, d] bf16 (16-byte aligned), last dimension contiguous, row
 *               and head strides in elements (multiples of 8, >= 0)
 *   cache     : device pointer (16-byte aligned)
 *   slots     : device int32 [T]; tokens whose slot lies outside the cache (-1) are skipped.  What
 *               a slot holds that several tokens of the call have is undefined, group by group
 *   T >= 1;  d 64 or 128;  page_size 16, 32, 64 or 128;  num_pages * page_size < 2^31;  descales powers of
 *   two in [2^-61, 2^59]
 */
FA_API int fa_kv4_append(const void* k, long long k_row_stride, long long k_head_stride,
                         const void* v, long long v_row_stride, long long v_head_stride,
                         void* cache, int num_pages, int page_size, const int* slots, int T,
                         int Hkv, int d, float k_descale, float v_descale, void* stream);

/* Read cached rows back as bf16 (exact): k, v are outputs [T, Hkv, d], contiguous, 16-byte
 * aligned, not the same; rows whose slot lies outside the cache are zeros.  Other arguments as fa_kv4_append. */
FA_API int fa_kv4_read(const void* cache, int num_pages, int page_size, const int* slots, void* k,
                       void* v, int T, int Hkv, int d, float k_descale, float v_descale,
                       void* stream);

/*
 * Attention of packed query tokens over the paged 4-bit cache.  Request b's queries are rows
 * q_offsets[b] .. q_offsets[b + 1) of q; its keys are the first lens[b] tokens of the pages
 * table[b, :].  Query head h reads key head h / (Hq / Hkv).  Causal: the queries are the last
 * tokens of the cache, so query i of n sees keys j <= lens[b] - n + i; otherwise all lens[b].
 * A row that sees no key gets O = 0 and LSE = -inf.
 *   q           : device pointer, [T, Hq, d] bf16 (16-byte aligned), last dimension contiguous, row
 *                 and head strides in elements (multiples of 8, >= 0)
 *   table, lens : device int32, [B, table_width] and [B].  Lengths outside [0, table_width *
 *                 page_size] are clamped; keys on a page id outside [0, num_pages) are not seen
 *   q_offsets   : device int32 [B + 1], not decreasing, or NULL: T / B queries each (T % B == 0).
 *                 Rows of q past q_offsets[B] are not read, their outputs left as they were.  Offsets
 *                 past T: the rows that there are, each at its place among all n queries
 *   o, lse      : outputs [T, Hq, d] bf16 (16-byte aligned) and [T, Hq] fp32; they overlap no input
 *                 (o = q is refused)
 *   max_q       : about the most queries of a request; any value >= 1 is correct, it picks the
 *                 kernel: how many query rows share a pass over the cache
 *   scale       : softmax scale, finite and >= 0
 *   workspace   : device scratch of fa_kv4_fwd_workspace_bytes(...) bytes, 16-byte aligned (NULL
 *                 when that is 0), contents on entry do not matter; calls that may run at the same
 *                 time need one each
 *   dev_status  : as fa_fwd_opts.dev_status (NULL = the library's status word)
 *   sizes       : T and B >= 1, Hq a multiple of Hkv, T * Hq < 2^30, table_width * page_size <= 2^30; d,
 *                 page_size and descales as fa_kv4_append
 * Queries enter the products as f16 scaled by a power of two per row: values below 2^-17 of a row's largest
 * lose bits, below 2^-26 they count as zero.  Probabilities are rounded to f16; sums are fp32.  A row whose
 * token has no slot (a request that fa_page_plan refused) means nothing: its key is not in the cache.
 * A key or value vector that is NaN makes the rows that see it NaN (O and LSE); rows that do not
 * see it, and whatever lies in the pages past a request's length, have no effect.  Partial sums
 * are merged in a fixed order: the same call gives the same bits.
 */
FA_API int fa_kv4_fwd(const void* q, long long q_row_stride, long long q_head_stride,
                      const void* cache, int num_pages, int page_size, const int* table,
                      int table_width, const int* lens, const int* q_offsets, void* o, float* lse,
                      int T, int B, int Hq, int Hkv, int d, int max_q, float scale, int causal,
                      float k_descale, float v_descale, void* workspace, size_t workspace_bytes,
                      int* dev_status, void* stream);

/* Workspace bytes fa_kv4_fwd needs for tables of `table_width` pages; 0 when it needs none (short
 * tables: no key head's work is split), and for invalid arguments. */
FA_API size_t fa_kv4_fwd_workspace_bytes(int Hq, int Hkv, int d, int max_q, int page_size,
                                         int table_width);

/*
 * Trees of drafted tokens.  A request's new tokens are the nodes 0 .. n - 1 of a tree behind its lens[b] cached
 * ones: node i hangs on node parents[i] < i of the same request, or (any other value, such as -1) on the last
 * cached token.  Positions are lens[b] + depth (0 for a node on the last cached token).  In `seen`, bit j % 32 of
 * word j / 32 of node i's row is set iff j is i or lies on i's way up.
 *   parents   : device int32 [T], packed by request
 *   q_offsets : device int32 [B + 1], not decreasing: first node of each request (rows past T do not count)
 *   words     : 1 to 8, words of a row of `seen`.  Nodes from 32 * words on have no bit: they are seen by none,
 *               and their rows hold the bits of the nodes above them that have one
 *   positions : output [T];  seen : output [T, words].  Rows past q_offsets[B]: position 0 and no bits
 *   sizes     : 1 <= B <= 16384, T >= 1, T * words < 2^31
 * No output may overlap an input.  One launch, integers only.
 */
FA_API int fa_tree_plan(const int* parents, const int* q_offsets, const int* lens, int B, int T,
                        int words, int* positions, unsigned* seen, void* stream);

/*
 * Attention of the nodes of such trees over the paged 4-bit cache, which holds them already: request b's nodes are
 * rows q_offsets[b] .. q_offsets[b + 1) of q and the last tokens of its lens[b] cached ones, in their order.  A node
 * sees the cached tokens before its tree (j < lens[b] - n) and node m (token lens[b] - n + m) iff bit m % 32 of
 * word m / 32 of its row of `seen` is set.  Nodes from 32 * words on are not seen.  Any mask of bits will do; a row
 * that sees nothing gets O = 0 and LSE = -inf.
 *   seen      : device [T, words] (4-byte aligned), words from 1 to 8
 *   q_offsets : as fa_kv4_fwd, not NULL
 *   workspace : fa_kv4_tree_fwd_workspace_bytes(...) bytes, as fa_kv4_fwd's
 * Everything else as fa_kv4_fwd.
 */
FA_API int fa_kv4_tree_fwd(const void* q, long long q_row_stride, long long q_head_stride,
                           const void* cache, int num_pages, int page_size, const int* table,
                           int table_width, const int* lens, const int* q_offsets,
                           const unsigned* seen, int words, void* o, float* lse, int T, int B, int Hq,
                           int Hkv, int d, int max_q, float scale, float k_descale, float v_descale,
                           void* workspace, size_t workspace_bytes, int* dev_status, void* stream);
FA_API size_t fa_kv4_tree_fwd_workspace_bytes(int Hq, int Hkv, int d, int max_q, int page_size,
                                              int table_width);

/*
 * What a step accepts of its trees.  choices[t] is the token that the model chose behind node t.  Node 0 of a
 * request is accepted (its token was chosen before), and every child of an accepted node whose token equals its
 * parent's choice (of several such children the one with the lowest number): a path down the tree.
 *   parents, seen, words, q_offsets : as for and from fa_tree_plan (`seen` that belongs to other parents gives
 *                   meaningless rows, but no access outside the buffers).  Nodes without a bit are not accepted
 *   tokens, choices : device int32 [T]
 *   lens, new_lens  : device int32 [B]: lengths before the step, and with all nodes (0 for ended requests).  A request
 *                   whose length did not grow (refused, ended, no nodes) accepts nothing
 *   slots         : device int32 [T]: the nodes' slots
 *   table, queue, queue_size, queue_state, page_size : as fa_page_plan, after it.  Pages that new_lens needs and
 *                   the accepted length does not go back to the ring, behind the free ones, in the requests' order
 *   lens_out      : [B] min(lens, new_lens) + accepted nodes;  counts : [B] accepted nodes
 *   path          : [T] a request's accepted nodes in their order in its first rows, -1 in the others
 *   next_tokens   : [B] choice of the last accepted node, -1 where none is
 *   sources       : [T] slots of the nodes of `path`, -1 in the other rows
 *   queue_state_out : {head, count} after the step
 *   sizes         : as fa_tree_plan; T = 0 is a step without nodes (arrays of T entries may be NULL)
 * All arrays are device int32.  No output may overlap an input or another output (lens_out and queue_state_out
 * are refused when they are the inputs; the ring is both).  One launch for up to 64 requests, else two; integers only.
 */
FA_API int fa_tree_accept(const int* parents, const unsigned* seen, int words, const int* tokens,
                          const int* choices, const int* lens, const int* new_lens,
                          const int* q_offsets, const int* slots, const int* table, int table_width,
                          int* queue, int queue_size, const int* queue_state, int B, int page_size,
                          int T, int* lens_out, int* counts, int* path, int* next_tokens,
                          int* sources, int* queue_state_out, void* stream);

/*
 * Move rows of paged 4-bit caches: for request b and i < counts[b], the keys and values of all heads at slot
 * sources[q_offsets[b] + i] to slot slots[q_offsets[b] + i], in each of num_caches caches (one a layer).
 *   caches  : HOST array of num_caches (1 to 256) device pointers to different caches of one shape
 *   sources, slots : device int32 [T]; rows with one outside the cache are skipped
 *   q_offsets, counts : device int32 [B + 1] and [B]
 * No source may be the slot of an earlier row of its request, or of any row of another: what is moved then is
 * undefined (fa_tree_accept's never are).  18 * Hkv * B < 2^31 - 128; the rest as fa_kv4_append.  One launch.
 */
FA_API int fa_kv4_move(void* const* caches, int num_caches, int num_pages, int page_size, int Hkv,
                       int d, const int* sources, const int* slots, const int* q_offsets,
                       const int* counts, int T, int B, void* stream);

/*
 * Read, and if `clear` is nonzero reset to FA_OK, the library's status word on the current
 * device.  Synchronises the device first.  Writes FA_OK or FA_ERR_DEVICE_TIMEOUT to *out.
 * Returns an fa_status for the call itself.
 */
FA_API int fa_device_status(int clear, int* out);

/* A static, human-readable name for a status code. */
FA_API const char* fa_status_string(int status);

/* Library version: major * 10000 + minor * 100 + patch. */
FA_API int fa_version(void);

/*
 * Diagnostic: evaluate the kernel's own 2^x routines on n inputs, for testing them against
 * exact exp2.  mode 0 = hardware approximation (MUFU ex2), mode 1 = the FMA polynomial
 * emulation the softmax uses for part of its columns ("FlashAttention4 精读", section 3.1.3
 * "Emulation of the exponential function").  x, y are device float arrays of n elements.
 */
FA_API int fa_debug_exp2(const float* x, float* y, long long n, int mode, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* EXACT_ATTENTION_H */
