/*
 * kinv.h -- C ABI of libkinv, a batch-invariant LLM forward step for NVIDIA
 * GB300 (sm_103a).
 *
 * What "batch-invariant" means here ("Deterministic and bit-exact inference",
 * trustbutveri.fyi record M-0002, *technical* and *How it works*): every
 * kernel fixes the reduction order of each output element whatever the batch
 * size, so the bits of row i (request b) depend only on row i's own inputs --
 * not on how many rows share the call, which rows they are, where row i sits
 * in the batch, or how a prompt was chunked.  The three reductions the pages
 * name are RMSNorm, matrix multiplication and attention; attention splits the
 * key/value dimension by a FIXED SPLIT SIZE, not a fixed number of splits.
 * The promise holds within one device class and one build (Kinetic
 * "Receipts", *What a receipt proves*: bits are promised only within one class
 * and one build); kinv_device_class() and kinv_build_id() name both.
 *
 * Conventions for every call below:
 *  - Pointers marked "device" are CUDA device pointers owned by the caller.
 *    The library never allocates, frees or synchronises on these paths; each
 *    call enqueues its kernels on `stream` (NULL = the legacy default stream)
 *    and returns.  Scratch space is passed in by the caller (`workspace`,
 *    sized by the matching *_workspace() query).
 *  - bf16 tensors are IEEE bfloat16 bit patterns, row-major, with the leading
 *    dimension (`ld*`, in elements) given.  fp32 accumulation throughout.
 *  - Errors are returned, never thrown, and nothing is launched when a call
 *    returns an error.  Shape, alignment and workspace checks happen on the
 *    host before any launch.  Launch failures return KINV_ERR_CUDA.  A device
 *    wait that runs out of time (every spin in the kernels is bounded) records
 *    a code in a device status word that kinv_last_device_status() reports.
 *  - Calls are thread-safe; the only global state is a lock-guarded cache,
 *    per CUDA context, of device attributes, of the device address of the
 *    status word and of kernel shared-memory limits.
 */
#ifndef KINV_H
#define KINV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* kinv_stream; /* same type as cudaStream_t */

typedef enum {
  KINV_OK = 0,
  KINV_ERR_INVALID_ARG = -1, /* null pointer, negative size, bad enum */
  KINV_ERR_UNSUPPORTED = -2, /* a shape or setting outside the supported set */
  KINV_ERR_ALIGNMENT = -3,   /* base or leading dimension not 16-byte aligned */
  KINV_ERR_WORKSPACE = -4,   /* workspace missing or smaller than the query */
  KINV_ERR_CUDA = -5,        /* a CUDA runtime/driver call failed */
  KINV_ERR_TIMEOUT = -6      /* a bounded device-side wait gave up */
} kinv_status;

typedef enum { KINV_BF16 = 0, KINV_F32 = 1, KINV_E4M3 = 2, KINV_I8 = 3 } kinv_dtype;

/* Human-readable name of a status code (static string). */
const char* kinv_status_string(int status);

/* Device class whose bits this build promises: "cuda-sm103a". */
const char* kinv_device_class(void);

/* Build id: 16 hex digits identifying this build of the kernels (a hash of
 * the sources and compile flags, fixed at build time).  Kinetic "Receipts",
 * *Making a receipt*: the receipt's build field pins every compiled kernel. */
const char* kinv_build_id(void);

/* Synchronises `stream`, then returns and clears the device status word of the
 * current device: KINV_OK, or the last code recorded since the previous call --
 * KINV_ERR_TIMEOUT (a bounded wait gave up), KINV_ERR_INVALID_ARG (an
 * attention or 8-bit cache call met a device-side length or place outside its
 * stated bounds, a call on drafted trees a broken tree, kinv_logprobs an id
 * beyond the vocabulary) or
 * KINV_ERR_UNSUPPORTED (a sampler row outside the supported settings).
 * Returns KINV_ERR_CUDA if the synchronisation itself fails. */
int kinv_last_device_status(kinv_stream stream);

/* Self-test of the bounded device waits (no counterpart on the pages; the
 * failure-detection rule every kernel here follows): launches one thread
 * block that waits on a shared-memory barrier nothing ever completes, for at
 * most limit_ns nanoseconds (1000 <= limit_ns <= 100000000), with the same
 * bounded-wait code the GEMM's pipeline waits use.  The wait gives up, records
 * KINV_ERR_TIMEOUT in the status word and the block exits, so the next
 * kinv_last_device_status() returns KINV_ERR_TIMEOUT and the context stays
 * usable.  Errors: KINV_ERR_INVALID_ARG for a limit outside the range. */
kinv_status kinv_test_bounded_wait(int64_t limit_ns, kinv_stream stream);

/* ------------------------------------------------------------------ GEMM
 * C[M][N] = A[M][K] . W[N][K]^T   ("Deterministic and bit-exact inference",
 * *technical*: batch-invariant matrix multiplication).
 *
 * A, W: device bf16, row-major, leading dimensions lda, ldw (elements).
 * C: device, bf16 (c_dtype = KINV_BF16) or fp32 (KINV_F32), leading dim ldc.
 * Arithmetic: bf16 products, fp32 accumulation on the tensor cores, one
 * rounding at the store.  The tile shape, the K order (ascending blocks of 64)
 * and the constant split of K (summed in fixed rank order) are chosen from
 * (N, K) alone, never from M: row i's bits are the same for every M.
 * Requirements: K % 64 == 0, N % 16 == 0, M >= 0; A, W, C 16-byte aligned;
 * lda, ldw multiples of 8; ldc a multiple of 8 (bf16) or 4 (fp32).
 * Errors: KINV_ERR_UNSUPPORTED / KINV_ERR_ALIGNMENT / KINV_ERR_INVALID_ARG.
 * M == 0 returns KINV_OK and launches nothing. */
kinv_status kinv_gemm(const void* A, int64_t lda, const void* W, int64_t ldw,
                      void* C, int64_t ldc, kinv_dtype c_dtype,
                      int M, int N, int K, kinv_stream stream);

/* RMSNorm folded into the projections around it ("Deterministic and
 * bit-exact inference", *technical*: batch-invariant RMSNorm and matmul).
 * The RMSNorm of a residual-stream row x, h = x / rms(x) * g, feeds only a
 * projection h . W^T, which equals (x . (W * g)^T) / rms(x) with the gain g
 * folded into W's columns once.  So:
 *  - a producing projection (`resid`) adds its bf16 output to the residual
 *    stream in its epilogue, resid[m][n] = bf16(resid[m][n] + out) with out
 *    the fp32 product (one rounding: the projection's output is not stored),
 *    and leaves the new row's sum of squares over each 128-column tile in
 *    ss_out[m][n / 128] (no other output; C may be NULL);
 *  - a consuming projection (`row_ss`) multiplies its fp32 result row m by
 *    1 / sqrt((row_ss[m][0] + row_ss[m][1] + ...) / norm_dim + eps), the
 *    tiles added in ascending order, before its rounding or epilogue;
 * so h is never rounded or stored.  Each partial and each row's total is
 * formed in a fixed order, so the bits do not depend on the batch.
 * row_ss: device fp32 [M][row_ss_tiles]; resid: device bf16 [M][N] (ld_resid,
 * a multiple of 8, N % 128 == 0); ss_out: device fp32 [M][N / 128]. */
typedef struct {
  const float* row_ss;
  int row_ss_tiles;
  int norm_dim;
  float eps;
  void* resid;
  int64_t ld_resid;
  float* ss_out;
} kinv_gemm_fusion;

/* kinv_gemm with the folded-RMSNorm options above (fusion nullable: plain
 * kinv_gemm).  Same tile, K order and split as kinv_gemm. */
kinv_status kinv_gemm_fused(const void* A, int64_t lda, const void* W, int64_t ldw,
                            void* C, int64_t ldc, kinv_dtype c_dtype, int M, int N, int K,
                            const kinv_gemm_fusion* fusion, kinv_stream stream);

/* Partial sums of squares of bf16 rows for a consuming projection's folded
 * RMSNorm (the first layer, whose input comes from the embedding):
 * ss_out[r][t] = sum over the 128 columns c of tile t of x[r][c]^2, in column
 * order.  x: device bf16 [rows][dim] (ldx); dim % 128 == 0. */
kinv_status kinv_row_sumsq(const void* x, int64_t ldx, int rows, int dim, float* ss_out,
                           kinv_stream stream);

/* QKV projection with kinv_rope_append in the epilogue: the product
 * qkv = A . W_qkv^T is formed with the same tile, K order and split as
 * kinv_gemm (N = (Hq + 2 Hkv) D), rounded to bf16 as kinv_gemm would store it,
 * and then, without going through memory, handled exactly as kinv_rope_append
 * handles its qkv rows (the same per-head arithmetic): q heads -> q_out, k heads
 * (RoPE, optional QK-norm) and v heads -> the caches at (seq[m], pos[m]).  The
 * result is bit-identical to kinv_gemm followed by kinv_rope_append
 * ("Deterministic and bit-exact inference", *technical*: the matmul is one of
 * the batch-invariant kernels; RoPE and the append reduce nothing across rows).
 * A bf16 [M][K] (lda), W_qkv bf16 [N][K] (ldw); q_out bf16 [M][Hq][D]; caches,
 * strides, seq, pos, norms, eps and rope_base as in kinv_rope_append.
 * fusion (nullable): the folded input RMSNorm (row_ss) of kinv_gemm_fused;
 * `resid` is not allowed here.
 * Requirements: D in {64, 128}, N % 128 == 0, K % 64 == 0, 16-byte alignment. */
kinv_status kinv_gemm_qkv_rope(const void* A, int64_t lda, const void* W_qkv, int64_t ldw,
                               void* q_out, void* k_cache, void* v_cache, int64_t seq_stride,
                               int64_t tok_stride, const int32_t* seq, const int32_t* pos,
                               const void* q_norm, const void* k_norm, float eps, int M, int Hq,
                               int Hkv, int D, int K, float rope_base,
                               const kinv_gemm_fusion* fusion, kinv_stream stream);

/* Gate/up projection with the SwiGLU applied in the epilogue:
 *   act[m][f] = bf16(silu(g) * u),  silu(g) = g / (1 + e^-g),
 *   g = A[m] . Wgate[f],  u = A[m] . Wup[f]  (fp32 accumulators, never rounded)
 * with the same tile, K order and split as kinv_gemm for N = 2F (so a row's
 * bits do not depend on M).  W_gu holds the 2F weight rows interleaved in
 * blocks of 64: rows 128j .. 128j+63 are gate rows 64j .. 64j+63 and rows
 * 128j+64 .. 128j+127 are up rows 64j .. 64j+63.  act: bf16 [M][F], leading
 * dimension ld_act (a multiple of 8).  fusion (nullable): the folded input
 * RMSNorm (row_ss) of kinv_gemm_fused, applied to g and u; `resid` is not
 * allowed here.  Requirements: F % 64 == 0, K % 64 == 0, alignment as for
 * kinv_gemm. */
kinv_status kinv_gemm_swiglu(const void* A, int64_t lda, const void* W_gu, int64_t ldw,
                             void* act, int64_t ld_act, int M, int F, int K,
                             const kinv_gemm_fusion* fusion, kinv_stream stream);

/* --------------------------------------------------------------- RMSNorm
 * y[r][i] = x[r][i] / sqrt(mean_j x[r][j]^2 + eps) * w[i]
 * ("Deterministic and bit-exact inference", *technical*: batch-invariant
 * RMSNorm).  One thread block per row, its size a function of `dim`; each
 * thread sums the squares of its chunks in a fixed order, a fixed xor
 * butterfly adds the lanes of a warp, and the warp sums are added in
 * ascending order, so a row's bits do not depend on `rows`.
 * residual (nullable): when given, s = bf16(x + residual) is formed first,
 * written back into `x` (the new residual stream), and y = RMSNorm(s).
 * x, residual, y: device bf16 [rows][dim] with leading dims ldx, ldx, ldy.
 * w: device bf16 [dim].  Requirements: dim % 8 == 0, 8 <= dim <= 16384,
 * 16-byte aligned bases, ldx and ldy multiples of 8.  `x` may be const when
 * residual is NULL (it is not written). */
kinv_status kinv_rmsnorm(void* x, int64_t ldx, const void* residual,
                         const void* w, void* y, int64_t ldy,
                         int rows, int dim, float eps, kinv_stream stream);

/* ------------------------------------------------------ decode attention
 * out[b][h] = sum_{j < L_b} softmax_j(scale * q[b][h] . k[b][j][g]) v[b][j][g],
 * g = h / (Hq / Hkv)  ("Deterministic and bit-exact inference", *technical*:
 * attention is batch-invariant when the keys are cut into splits of one fixed
 * length, whatever their number).
 *
 * Keys of sequence b are cut into splits of `split_len` keys at absolute
 * offsets 0, split_len, 2 split_len, ...; each split yields an fp32 partial
 * (max, sum of exponentials, unnormalised output) and the partials are folded
 * in ascending split order.  The cut depends only on L_b, so a sequence's bits
 * do not depend on its batch-mates or their lengths.  L_b == 0 gives zeros.
 * Within a split the softmax is taken in base 2: with r = q . k (fp32) and
 * c = fp32(scale * log2 e), m = fp32(max r * c) and the weights
 * e = 2^fma(r, c, -m) (the hardware's approximate exp2) are formed in fp32,
 * summed in fp32, and enter the tensor cores as the bf16 pair hi = bf16(e),
 * lo = bf16(e - hi), so they keep about 16 significant bits; P.V is one fp32
 * chain over 16-key steps, each adding its hi . V, then its lo . V.
 *
 * q, out: device bf16 [B][Hq][D] (contiguous).  k_cache, v_cache: device bf16;
 *   element (b, j, g, d) is at b*seq_stride + j*tok_stride + g*D + d
 *   (elements); e.g. a contiguous [B][Lmax][Hkv][D] cache has
 *   seq_stride = Lmax*Hkv*D, tok_stride = Hkv*D.
 * kv_len: device int32 [B], each in [0, Lmax]; a sequence whose kv_len lies
 *   outside gets zeros, and the status word records KINV_ERR_INVALID_ARG
 *   (no key beyond Lmax is read).
 * workspace: device, at least kinv_attn_decode_workspace(B, Hq, D, Lmax,
 *   split_len) bytes, 16-byte aligned.
 * Requirements: D in {64, 128}; Hq % Hkv == 0; Hq / Hkv in {1, 2, 4, 8};
 * split_len == 256; strides multiples of 8.  A scale that is not a positive
 * finite number means 1/sqrt(D). */
size_t kinv_attn_decode_workspace(int B, int Hq, int D, int Lmax, int split_len);
kinv_status kinv_attn_decode(const void* q, const void* k_cache, const void* v_cache,
                             int64_t seq_stride, int64_t tok_stride,
                             const int32_t* kv_len, void* out,
                             int B, int Hq, int Hkv, int D, int Lmax, int split_len,
                             float scale, void* workspace, size_t workspace_bytes,
                             kinv_stream stream);

/* --------------------------------------- decode attention, no allocation
 * The pages have no counterpart to this call: it exists for callers that
 * cannot allocate device memory.  Some code cannot call cudaMalloc -- a plug-in
 * whose host program owns every byte of device memory through its own pool, a
 * real-time loop that must not take the allocator's implicit device-wide
 * synchronisation, or a binding with no device allocator at all -- and so
 * cannot provide the scratch that kinv_attn_decode takes as `workspace`.
 *
 * Same arguments, arithmetic and output bits as kinv_attn_decode, minus the
 * workspace: the split partials live in a scratch array compiled into the
 * library (KINV_NOALLOC_SCRATCH_BYTES bytes on every GPU that loads it, held
 * until the process exits).  Nothing is allocated or freed.
 *  - A call whose partials need more than KINV_NOALLOC_SCRATCH_BYTES (that is,
 *    kinv_attn_decode_workspace(B, Hq, D, Lmax, split_len) is larger) returns
 *    KINV_ERR_WORKSPACE and launches nothing.
 *  - The first call in each CUDA context (normally once per device) looks up
 *    the array's device address with that device current, checks the lookup
 *    and caches the address for that context; make that first call before any
 *    stream capture.
 *  - Every call on a device shares the one array, which keeps whatever the
 *    last call left in it (each call writes every partial it later reads, so
 *    nothing needs clearing).  Calls that overlap on the GPU -- on two streams,
 *    or from two threads -- race on it: serialise them. */
#define KINV_NOALLOC_SCRATCH_BYTES (64u * 1024u * 1024u)
kinv_status kinv_attn_decode_noalloc(const void* q, const void* k_cache, const void* v_cache,
                                     int64_t seq_stride, int64_t tok_stride,
                                     const int32_t* kv_len, void* out,
                                     int B, int Hq, int Hkv, int D, int Lmax, int split_len,
                                     float scale, kinv_stream stream);

/* ----------------------------------------------------- prefill attention
 * Causal attention for chunks of new query rows against the cache (which
 * must already hold their keys).  Sequence b contributes q_len[b] rows,
 * stored at rows q_offset[b] .. q_offset[b] + q_len[b] - 1 of q/out, at
 * absolute positions q_start[b] .. q_start[b] + q_len[b] - 1; the row at
 * position p attends to keys 0..p of sequence b.
 * Each row is computed with exactly the arithmetic of kinv_attn_decode for a
 * sequence of length p + 1 (same splits at absolute offsets, same fold), so a
 * row's bits do not depend on the chunking, on p0, on the other rows, and a
 * decode step equals a one-row prefill bit for bit.
 * The rows run on the tcgen05 tensor cores, 128 (row, head) pairs of one
 * sequence and kv head per thread block, which folds the sequence's splits
 * one after another in registers: kinv_attn_prefill_workspace() is 0 and
 * `workspace` may be NULL.
 * q, out: device bf16 [total_rows][Hq][D].  q_start, q_len, q_offset: device
 * int32 [B].  Caches and strides as for decode, the cache holding at least
 * max_kv keys of each of the B sequences (seq_stride > 0 when B > 1).  max_q_len bounds q_len[b],
 * max_kv bounds q_start[b] + q_len[b] (both used to size the grid and the
 * workspace), and q_offset[b] + q_len[b] <= total_rows; a sequence whose
 * device-side values break one of these bounds (or is negative) is left out
 * -- its rows of `out` are not written -- and the status word records
 * KINV_ERR_INVALID_ARG.  Requirements as for decode. */
size_t kinv_attn_prefill_workspace(int total_rows, int Hq, int D, int max_kv, int split_len);
kinv_status kinv_attn_prefill(const void* q, const void* k_cache, const void* v_cache,
                              int64_t seq_stride, int64_t tok_stride,
                              const int32_t* q_start, const int32_t* q_len,
                              const int32_t* q_offset, void* out,
                              int B, int total_rows, int max_q_len, int max_kv,
                              int Hq, int Hkv, int D, int split_len, float scale,
                              void* workspace, size_t workspace_bytes,
                              kinv_stream stream);

/* ------------------------------------------- sliding window with sinks
 * Attention whose rows see the last `window` keys, their own among them, and
 * the first `sinks` keys of the sequence: the row at position p sees key j <= p
 * if j > p - window or j < sinks (the pages have no counterpart).  window = 0
 * means every key j <= p; where nothing is hidden a row has the bits of
 * kinv_attn_decode.  The splits stay at
 * their absolute offsets, splits without a visible key are left out, and hidden
 * keys in the others have weight 0 and are not read (decode) or do not count
 * (prefill), so the invariances hold as above: a row's bits depend on its own
 * sequence alone, and a decode step equals a one-row prefill.
 * What a hidden slot holds does not matter to decode, nor to prefill where it is
 * hidden from every row of the call.  Where a value that is an infinity or NaN
 * is visible to one row of a prompt chunk, other rows of the chunk near it may
 * get NaN as well, as in kinv_attn_prefill.
 * Arguments, requirements and errors as above; window < 0 or sinks < 0:
 * KINV_ERR_INVALID_ARG.  The decode call's workspace grows with the window and
 * the sinks instead of Lmax (Lmax = 0: none, and zeros).  The prefill call needs none (NULL); with as many bytes as
 * its query says (0 where it would not help) it spreads short chunks over long contexts
 * over the whole GPU, with the same bits. */
size_t kinv_attn_decode_window_workspace(int B, int Hq, int D, int Lmax, int split_len, int window, int sinks);
kinv_status kinv_attn_decode_window(const void* q, const void* k_cache, const void* v_cache,
                                    int64_t seq_stride, int64_t tok_stride,
                                    const int32_t* kv_len, void* out,
                                    int B, int Hq, int Hkv, int D, int Lmax, int split_len,
                                    int window, int sinks, float scale, void* workspace,
                                    size_t workspace_bytes, kinv_stream stream);
size_t kinv_attn_prefill_window_workspace(int B, int max_q_len, int Hq, int Hkv, int D, int max_kv,
                                          int split_len, int window, int sinks);
kinv_status kinv_attn_prefill_window(const void* q, const void* k_cache, const void* v_cache,
                                     int64_t seq_stride, int64_t tok_stride,
                                     const int32_t* q_start, const int32_t* q_len,
                                     const int32_t* q_offset, void* out,
                                     int B, int total_rows, int max_q_len, int max_kv,
                                     int Hq, int Hkv, int D, int split_len, int window, int sinks,
                                     float scale, void* workspace, size_t workspace_bytes,
                                     kinv_stream stream);

/* ------------------------------------------------ 8-bit key/value cache
 * Keys and values as 8-bit codes with a scale for every (token, kv head), keys
 * and values apart (the pages have no counterpart).  A value is code * 2^E.
 * With amax the largest magnitude among a vector's D bf16 values,
 *   KINV_E4M3  E = the smallest e with amax <= 448 * 2^e, -100 <= E <= 119
 *   KINV_I8    E = the smallest e with amax <= 127 * 2^e, -100 <= E <= 121
 *   code = x * 2^-E rounded to the nearest code (ties to even, saturating)
 * and E = -128 marks a vector that held an infinity or NaN; all of it reads back
 * as NaN (its codes are 0).  code * 2^E is a bf16 number, so nothing is lost
 * after the one rounding to a code: at most half a step, 2^-4 of the value
 * (e4m3, 2^-10 * 2^E where that is more) or 2^E / 2 (int8).  A code depends on
 * its own token alone, never on its neighbours in the cache, so the cache is the
 * same for every chunking of a prompt.
 *
 * Element (b, slot, g, d) of k and v is the byte at b*seq_stride +
 * slot*tok_stride + g*D + d; the exponents of (b, slot, g) are at
 * b*exp_seq_stride + g*exp_head_stride + slot.  B sequences of `slots` slots.
 * k, v 16-byte aligned, seq_stride and tok_stride multiples of 16, tok_stride >=
 * Hkv*D, exp_head_stride >= slots; D in {64, 128}.  The struct is read on the
 * host before a call returns.  Codes 0x7F and 0xFF of e4m3 and exponents outside
 * [-126, 121] but for -128 are never written and must not be given. */
typedef struct {
  void* k;
  void* v;
  int8_t* k_exp;
  int8_t* v_exp;
  int64_t seq_stride;
  int64_t tok_stride;
  int64_t exp_seq_stride;
  int64_t exp_head_stride;
  int B;
  int slots;
  kinv_dtype dtype; /* KINV_E4M3 or KINV_I8 */
} kinv_cache8;

/* kinv_rope_append with the key and value heads in 8 bits: the codes of the
 * rotated keys, rounded to bf16, and of the values.  The angles are carried a
 * little further than there, so a query or key may differ by a bf16 step where
 * it lies next to a rounding border.  Arguments, requirements and errors as
 * there, and gains 16-byte aligned; no two rows of a call may name the same place.  A row whose sequence or position lies
 * outside the cache is left out -- its row of q_out too -- and the status word
 * records KINV_ERR_INVALID_ARG. */
kinv_status kinv_rope_append8(const void* qkv, int64_t ld_qkv, void* q_out, const kinv_cache8* cache,
                              const int32_t* seq, const int32_t* pos, const void* q_norm,
                              const void* k_norm, float eps, int rows, int Hq, int Hkv, int D,
                              float rope_base, kinv_stream stream);

/* Keys and values between bf16 and the 8-bit cache: token i < len[b] of sequence
 * b, at b*seq_stride + i*tok_stride + g*D + d of the bf16 k and v (elements),
 * goes into (write) or comes from (read) slot start[b] + i.  start, len: device
 * int32 [B], B at most the cache's; max_len bounds len[b].  A sequence whose
 * numbers break a bound (0 <= len[b] <= max_len, 0 <= start[b], start[b] + len[b]
 * <= slots) is left out and the status word records KINV_ERR_INVALID_ARG.
 * Everything else in either cache stays as it was.  Strides multiples of 8,
 * 16-byte aligned bases, Hkv <= 1024.  The sequences' slots and tokens must not
 * overlap where they are written: a stride of 0 between sequences is refused
 * there (as in kinv_rope_append8) when B > 1. */
kinv_status kinv_cache8_write(const void* k, const void* v, int64_t seq_stride, int64_t tok_stride,
                              const kinv_cache8* cache, const int32_t* start, const int32_t* len,
                              int B, int max_len, int Hkv, int D, kinv_stream stream);
kinv_status kinv_cache8_read(const kinv_cache8* cache, const int32_t* start, const int32_t* len,
                             void* k, void* v, int64_t seq_stride, int64_t tok_stride, int B,
                             int max_len, int Hkv, int D, kinv_stream stream);

/* kinv_attn_decode and kinv_attn_prefill over the 8-bit cache, with a sliding
 * window and sinks as above (window = 0: every key).  A row gets the bits that
 * kinv_attn_decode_window and kinv_attn_prefill_window give on the cache read
 * back, wherever no score, product or sum on the way leaves the normal range of
 * fp32, in decode no value of q other than 0 lies below 2^-31 of the row and
 * head's largest, and with e4m3 no weight that counts below 2^-100 times the
 * largest scale among its 256 keys; so all their invariances hold.  Hidden slots
 * and those behind a sequence's last key may hold anything.
 * kv_len[b] in [0, slots], else zeros and KINV_ERR_INVALID_ARG in the status
 * word (a cache of no slots gives zeros, without a workspace); B at most the cache's,
 * max_kv at most its slots; seq_stride > 0 in decode when B > 1; other arguments,
 * requirements and errors as there.  workspace: device, 16-byte aligned, as many
 * bytes as the query says; calls that may run at the same time need one each.
 * The decode call's holds the split partials; the prefill call's holds the keys
 * and values that its rows see, read back, B max_kv Hkv D 4 bytes, without which it
 * refuses, and behind them, where the chunk is short, what kinv_attn_prefill_window may
 * use.  kinv_attn_prefill8_workspace() is enough for every window and every chunk of up
 * to total_rows; for a call of one max_q_len (no larger than its rows), window and sinks
 * those B max_kv Hkv D 4 bytes and kinv_attn_prefill_window_workspace() of them are. */
size_t kinv_attn_decode8_workspace(int B, int Hq, int D, int slots, int window, int sinks, int split_len);
kinv_status kinv_attn_decode8(const void* q, const kinv_cache8* cache, const int32_t* kv_len, void* out,
                              int B, int Hq, int Hkv, int D, int split_len, int window, int sinks,
                              float scale, void* workspace, size_t workspace_bytes, kinv_stream stream);
size_t kinv_attn_prefill8_workspace(int B, int total_rows, int Hq, int Hkv, int D, int max_kv, int split_len);
kinv_status kinv_attn_prefill8(const void* q, const kinv_cache8* cache, const int32_t* q_start,
                               const int32_t* q_len, const int32_t* q_offset, void* out, int B,
                               int total_rows, int max_q_len, int max_kv, int Hq, int Hkv, int D,
                               int split_len, int window, int sinks, float scale, void* workspace,
                               size_t workspace_bytes, kinv_stream stream);

/* --------------------------------------------------------------- sampler
 * Seeded sampler with the settings a Kinetic receipt records (Kinetic
 * "Receipts", *Making a receipt*, the `sampling` object).  Per row b, in this
 * order: the logit bias (each entry (id, bias) of the row's list adds bias to
 * logit id in fp32, in list order; ids outside [0, V) are ignored); the
 * penalties over the distinct ids among the last repeat_last_n
 * history tokens (n < 0: all, n == 0: none), first the repeat penalty
 * (z/r if z > 0 else z*r), then, when presence_penalty or frequency_penalty is
 * not 0, z - (c * frequency_penalty + presence_penalty) with c the id's count
 * in that window (each operation rounded to fp32);
 * temperature <= 0 -> greedy argmax (lowest id on ties); otherwise the top_k
 * candidates ordered by (z desc, id asc); s = z / temperature;
 * e_i = exp(s_i - s_0); typical-p (when 0 < typical_p < 1) keeps, with
 * p_i = e_i / sum(e) and H = -sum p_i log p_i, the shortest set of candidates
 * taken by |-log p_i - H| ascending (then candidate order) whose p reaches
 * typical_p, and the steps below see only that set, in candidate order;
 * top-p keeps the shortest prefix whose sum of e reaches top_p * sum(e)
 * (skipped when top_p >= 1); min-p keeps e_i >= min_p * e_first, e_first the
 * first kept candidate's e (skipped when min_p <= 0); then u = (Philox4x32-10(counter = (step lo, step hi, 0, 0),
 * key = (seed lo, seed hi)).word0 >> 8) * 2^-24 picks the first kept candidate
 * whose running sum of e exceeds u * (sum of kept e).  The counter is the
 * request's own step, never its batch slot: the drawn token depends only on
 * the row's logits, history, settings and step.  A cluster of up to eight
 * thread blocks shares a row (the count follows the batch size; the token
 * does not depend on it); ranking and thresholds are compare-only on fp32
 * values; sums in fixed order.
 * top_k <= 0 (or >= V) means the whole vocabulary: e is then summed over all
 * V ids (per 128-id block, blocks in order) and the top-p / min-p cut must
 * fall within the 1024 most likely ids.
 *
 * logits: device fp32 [B][ld]; params: device kinv_sampling_params [B];
 * history: device int32 [B][hist_ld], row b holding hist_len[b] ids, oldest
 * first; step: device int64 [B]; out_tokens: device int32 [B].
 * Requirements: 1 <= V; ld >= V; top_k in [1, 1024] or the whole vocabulary
 * (V <= 262144, and top_p < 1 or min_p > 0 cutting within the 1024 most
 * likely ids, typical-p off) unless temperature <= 0; hist_len[b] <= hist_ld <= 1024
 * (else KINV_ERR_UNSUPPORTED before launch); at most 1024 logit-bias entries
 * per row (further entries are ignored).  Rows whose
 * settings or logits fall outside this set get token -1 and the device status
 * word records KINV_ERR_UNSUPPORTED. */
typedef struct {
  int32_t id;
  float bias;
} kinv_logit_bias;

typedef struct {
  float temperature;
  float top_p;
  float min_p;
  float repeat_penalty;
  int32_t top_k;
  int32_t repeat_last_n;
  uint64_t seed;
  float presence_penalty;   /* 0: off */
  float frequency_penalty;  /* 0: off */
  const kinv_logit_bias* logit_bias;  /* device, n_logit_bias entries; NULL: none */
  int32_t n_logit_bias;               /* at most 1024 */
  float typical_p;                    /* on when 0 < typical_p < 1 */
} kinv_sampling_params;

size_t kinv_sample_workspace(int B, int V);
kinv_status kinv_sample(const float* logits, int64_t ld, int B, int V,
                        const kinv_sampling_params* params,
                        const int32_t* history, int hist_ld, const int32_t* hist_len,
                        const int64_t* step, int32_t* out_tokens,
                        void* workspace, size_t workspace_bytes, kinv_stream stream);

/* ------------------------------------------------------------ layer glue
 * Element-wise steps of the decoder block.  None of them sums across
 * elements, so each is batch-invariant by construction. */

/* out[r] = table[ids[r]] for r < rows; table bf16 [vocab][dim] (ld = dim),
 * ids device int32 [rows] (ids outside [0, vocab) give zeros), dim % 8 == 0. */
kinv_status kinv_embed(const void* table, int vocab, int dim, const int32_t* ids,
                       void* out, int rows, kinv_stream stream);

/* out[n][k] = bf16(w[n][k] * g[k]) (fp32 product): an RMSNorm gain g moved
 * into the input columns of the projection it feeds, once, when the weights are
 * loaded ("Deterministic and bit-exact inference", *technical*: RMSNorm and
 * matmul; see kinv_gemm_fusion).  w, out: device bf16 [N][K] (ldw, ldo
 * multiples of 8; out may equal w); g: device bf16 [K]; K % 8 == 0,
 * N <= 262140, 16-byte aligned bases. */
kinv_status kinv_scale_columns(const void* w, int64_t ldw, const void* g, void* out, int64_t ldo,
                               int N, int K, kinv_stream stream);

/* out = bf16(x + y), n elements, bf16, n % 8 == 0, 16-byte aligned. */
kinv_status kinv_add(const void* x, const void* y, void* out, int64_t n, kinv_stream stream);

/* out[r][i] = bf16(silu(gu[r][i]) * gu[r][F + i]), silu(g) = g / (1 + e^-g);
 * gu bf16 [rows][2F] (ld_gu), out bf16 [rows][F] (ld_out); F % 8 == 0. */
kinv_status kinv_swiglu(const void* gu, int64_t ld_gu, void* out, int64_t ld_out,
                        int rows, int F, kinv_stream stream);

/* Rotary embedding (rotate-half pairs (i, i + D/2), theta_i = p * base^(-2i/D))
 * with optional per-head RMSNorm first (q_norm / k_norm nullable, gains [D]),
 * then the key/value append: for row r of sequence seq[r] at absolute position
 * pos[r]:
 *   q_out[r][h]                = bf16(RoPE(norm(q)))        h < Hq
 *   k_cache[seq][pos][g]       = bf16(RoPE(norm(k)))        g < Hkv
 *   v_cache[seq][pos][g]       = v                           (copied bits)
 * qkv: device bf16 [rows][(Hq + 2 Hkv) D] (ld_qkv), q, k, v heads in that
 * order.  q_out: bf16 [rows][Hq][D].  seq, pos: device int32 [rows].
 * Requirements: D in {64, 128}; strides multiples of 8; 16-byte alignment. */
kinv_status kinv_rope_append(const void* qkv, int64_t ld_qkv, void* q_out,
                             void* k_cache, void* v_cache, int64_t seq_stride,
                             int64_t tok_stride, const int32_t* seq, const int32_t* pos,
                             const void* q_norm, const void* k_norm, float eps,
                             int rows, int Hq, int Hkv, int D, float rope_base,
                             kinv_stream stream);

/* One decode iteration's bookkeeping, per request b < B: append
 * tokens[b] to history row b (shifting out the oldest id once hist_len ==
 * hist_ld), hist_len[b] = min(hist_len[b] + 1, hist_ld), step[b] += 1, and
 * pos[b] += 1, kv_len[b] += 1 for whichever of pos / kv_len is not NULL.
 * All device pointers. */
kinv_status kinv_decode_advance(const int32_t* tokens, int32_t* history, int hist_ld,
                                int32_t* hist_len, int64_t* step, int32_t* pos,
                                int32_t* kv_len, int B, kinv_stream stream);

/* -------------------------------------------------- trees of drafted tokens
 * A batch of trees of drafted tokens to be verified in one step (the pages
 * have no counterpart: drafting changes only how many rows a step carries,
 * and a step whose rows do not depend on one another gives a drafted token
 * the bits it would have as a decode step of its own).
 *
 * Sequence b has ctx_len[b] keys in its cache (slots 0 .. ctx_len[b] - 1) and
 * n_nodes[b] drafted nodes, rows row_offset[b] .. row_offset[b] + n_nodes[b]
 * - 1 of the row tensors.  parent[row] is the index (within the sequence) of
 * the node's parent, below the node's own index, or -1: the node follows the
 * context itself.  With t ancestors a node has depth t: it is the token at
 * position ctx_len[b] + t, and its keys and values sit in cache slot
 * ctx_len[b] + (its index).
 *
 * All arrays: device int32; ctx_len, n_nodes, row_offset [B]; parent
 * [total_rows].  max_nodes (<= KINV_TREE_MAX_NODES) bounds n_nodes[b], max_kv
 * bounds ctx_len[b] + n_nodes[b] (the cache's slots per sequence), and
 * row_offset[b] + n_nodes[b] <= total_rows.  The rows of different sequences
 * must not overlap.  A sequence whose device-side numbers break a bound, or
 * that holds a parent outside [-1, own index), is left out of every call below
 * -- nothing of it is written, but for what kinv_tree_accept_marked is asked to
 * mark -- and the status word records KINV_ERR_INVALID_ARG.  Rows that belong to no sequence are left as they
 * were.  The struct itself is read on the host before a call returns; with B,
 * total_rows or max_nodes 0 no sequence has a node, and the arrays are not
 * read. */
#define KINV_TREE_MAX_NODES 64
typedef struct {
  const int32_t* ctx_len;
  const int32_t* n_nodes;
  const int32_t* row_offset;
  const int32_t* parent;
  int B;
  int total_rows;
  int max_nodes;
  int max_kv;
} kinv_tree;

/* kinv_rope_append for the rows of drafted trees: the same per-head arithmetic
 * (optional RMSNorm, then the rotation by the node's position ctx_len[b] +
 * depth), the keys and values written to the node's slot ctx_len[b] + index.
 * A drafted token's q, k and v therefore have the bits that kinv_rope_append
 * gives the same row at the same position.
 * qkv: device bf16 [total_rows][(Hq + 2 Hkv) D] (ld_qkv); q_out: bf16
 * [total_rows][Hq][D]; caches and strides as in kinv_rope_append (element
 * (b, slot, g, d) at b*seq_stride + slot*tok_stride + g*D + d); requirements
 * and errors as there, and KINV_ERR_UNSUPPORTED for max_nodes >
 * KINV_TREE_MAX_NODES or B > 65535. */
kinv_status kinv_rope_append_tree(const void* qkv, int64_t ld_qkv, void* q_out, void* k_cache,
                                  void* v_cache, int64_t seq_stride, int64_t tok_stride,
                                  const kinv_tree* tree, const void* q_norm, const void* k_norm,
                                  float eps, int Hq, int Hkv, int D, float rope_base,
                                  kinv_stream stream);

/* Attention of drafted nodes: node i of sequence b attends to the context
 * (slots 0 .. ctx_len[b] - 1), to its ancestors and to itself (slots ctx_len[b]
 * + ancestor index), which the cache must already hold.
 * Each row is computed with exactly the arithmetic of kinv_attn_decode for a
 * sequence of length ctx_len[b] + depth + 1 whose cache holds the context and
 * then the node's path in order (splits at absolute positions, the key of the
 * ancestor at depth t in the place of position ctx_len[b] + t), so a drafted
 * token's bits are those of the decode step that would follow its path, and
 * do not depend on the other nodes, the tree's shape or the batch.
 * q, out: device bf16 [total_rows][Hq][D] (contiguous).  Caches and strides as
 * for kinv_attn_decode.  workspace: device, 16-byte aligned, at least
 * kinv_attn_tree_workspace(B, total_rows, max_nodes, Hq, Hkv, D, max_kv,
 * split_len) bytes; two calls that may run at the same time need one each.
 * It has room for an fp32 partial of every (node, head) that max_nodes allows in
 * every split that max_kv allows, about B max_nodes Hq (D + 2) 4 ceil(max_kv /
 * split_len) bytes: with Hq 32 and D 128, 17 MB for 4 trees of 16 nodes in 4,096
 * slots, 8.7 GB for 64 of 64 in 32,768.  max_nodes and max_kv also decide which
 * kernels a call launches (never a bit of the result), so both pay for being
 * close: one tree of 8 nodes behind 500 keys takes 10.8 us with max_kv 576 and
 * 12.7 with 32,768.
 * Requirements as for kinv_attn_decode. */
size_t kinv_attn_tree_workspace(int B, int total_rows, int max_nodes, int Hq, int Hkv, int D,
                                int max_kv, int split_len);
kinv_status kinv_attn_tree(const void* q, const void* k_cache, const void* v_cache,
                           int64_t seq_stride, int64_t tok_stride, const kinv_tree* tree,
                           void* out, int Hq, int Hkv, int D, int split_len, float scale,
                           void* workspace, size_t workspace_bytes, kinv_stream stream);

/* The drafted tokens that the model agrees with, and their place in the cache.
 * tokens[row]: the node's token; next_tokens[row]: the model's own token after
 * the node (e.g. sampled from the row's logits).  Node 0 of a sequence is a
 * token that was already decided, so it is always taken; the path goes on to
 * the lowest-indexed child of its last node whose token equals next_tokens of
 * that node, and ends where there is none.  For each sequence with n_nodes[b]
 * > 0, with the path's node j_t at depth t < n_accepted[b]:
 *   path[b][t]       = j_t
 *   out_tokens[b][t] = next_tokens of j_t (the tokens this step decides: the
 *                      drafted ones it confirms, then one more)
 *   cache slot ctx_len[b] + t = the bits of slot ctx_len[b] + j_t,
 * in every one of n_layers layers of both caches, so that the slots 0 ..
 * ctx_len[b] + n_accepted[b] - 1 then hold what decoding those tokens one by
 * one would have put there; the slots behind them are left as they were.
 * path and out_tokens beyond n_accepted[b] are -1; n_accepted[b] = 0 for a
 * sequence without nodes.
 * n_accepted: device int32 [B]; path, out_tokens: device int32
 * [B][max_nodes].  None of them may overlap the tree's arrays, tokens or
 * next_tokens.  Element (layer, b, slot, g, d) of a cache is at
 * layer*layer_stride + b*seq_stride + slot*tok_stride + g*D + d.  n_layers = 0
 * moves nothing (k_cache and v_cache may then be NULL).
 * Requirements: D % 8 == 0, strides multiples of 8, 16-byte aligned caches,
 * n_layers <= 65535. */
kinv_status kinv_tree_accept(const kinv_tree* tree, const int32_t* tokens,
                             const int32_t* next_tokens, void* k_cache, void* v_cache,
                             int n_layers, int64_t layer_stride, int64_t seq_stride,
                             int64_t tok_stride, int Hkv, int D, int32_t* n_accepted,
                             int32_t* path, int32_t* out_tokens, kinv_stream stream);

/* The same with results also for a sequence that is left out for its broken
 * tree, in the outputs that `mark` names: n_accepted[b] = 0, path[b] and
 * out_tokens[b] all -1 (for outputs whose memory held something else before).
 * mark: KINV_TREE_MARK_* or'ed; other bits are KINV_ERR_INVALID_ARG.  0 is
 * kinv_tree_accept. */
#define KINV_TREE_MARK_COUNT 1
#define KINV_TREE_MARK_PATH 2
#define KINV_TREE_MARK_TOKENS 4
kinv_status kinv_tree_accept_marked(const kinv_tree* tree, const int32_t* tokens,
                                    const int32_t* next_tokens, void* k_cache, void* v_cache,
                                    int n_layers, int64_t layer_stride, int64_t seq_stride,
                                    int64_t tok_stride, int Hkv, int D, int32_t* n_accepted,
                                    int32_t* path, int32_t* out_tokens, int mark, kinv_stream stream);

/* ------------------------------------------------------ log probabilities
 * Per row r of logits x (V of them), with m = max x and S = sum e^(x - m):
 *   logprob[r][j]    = x[ids[r][j]] - m - ln S         (j < n_ids)
 *   entropy[r]       = ln S - (sum e^(x - m) (x - m)) / S       (nats)
 *   top_ids[r][j], top_logprobs[r][j]: the j-th likeliest id and its log
 *                      probability, by (x descending, id ascending), j < top_k.
 * The row is cut into units of 1024 ids; a warp takes a unit's maximum and sums
 * in one fixed order and the units are folded in one fixed order, all in fp32,
 * so a row's bits do not depend on the other rows.
 * NaN logits count as -infinity (as in kinv_sample).  -infinity has probability
 * 0 (logprob -infinity).  In a row that holds +infinity those ids share the
 * whole probability equally.  In a row of -infinity only, every logprob is
 * -infinity and the entropy 0.  An id below 0 is padding: its logprob is 0.
 * An id >= V gives NaN and the status word records KINV_ERR_INVALID_ARG.
 *
 * logits: device fp32 or bf16 [rows][ld] (16-byte loads where the base and ld
 * allow, any alignment works); ids: device int32 [rows][n_ids]; logprob fp32
 * [rows][n_ids]; entropy (nullable) fp32 [rows]; top_ids int32, top_logprobs
 * fp32 [rows][top_k].  ids and logprob may be NULL when n_ids = 0, the top
 * arrays when top_k = 0.
 * Requirements: 1 <= V <= 1048576, ld >= V, 0 <= top_k <= 32, top_k <= V. */
kinv_status kinv_logprobs(const void* logits, kinv_dtype dtype, int64_t ld, int rows, int V,
                          const int32_t* ids, int n_ids, float* logprob, float* entropy,
                          int top_k, int32_t* top_ids, float* top_logprobs, kinv_stream stream);

#ifdef __cplusplus
}
#endif
#endif /* KINV_H */
