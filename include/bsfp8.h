/*
 * bsfp8 -- block-scaled fp8 weight GEMM for small row counts on AMD MI355X (gfx950).
 *
 * The operation (page "recipes/docker-images/mia-tp4/adapter/wo_a_w8.py", module docstring and
 * kernels _wo_a_partial_w8 / _wo_a_mid_kernel): a weight is stored as e4m3 ("float8_e4m3fn")
 * codes q[g][n][k] plus one exponent byte b per 32x32 block; the weight value is
 * bf16(e4m3(q) * 2^(b-127)), rebuilt exactly in registers. For bf16 activations X the library
 * computes, per group g,
 *
 *     Y[m][g][n] = sum_k X[m][g*K + k] * W[g][n][k]
 *
 * with fp32 accumulation and a fixed summation order, and stores Y as bf16 (RNE) or fp32.
 *
 * Conventions for every entry point:
 *   - Pointers are DEVICE pointers unless stated "host". bf16 values are passed as their 16-bit
 *     patterns (uint16_t). The caller owns every buffer; the library allocates nothing in the
 *     per-call functions and keeps no state between calls, apart from the static scratch array
 *     of bsfp8_gemm_no_alloc (and its address, looked up once per device).
 *   - `stream` is a hipStream_t passed as void* (NULL = the default stream). Per-call functions
 *     only enqueue work: they never synchronise or allocate, so they can be captured in a HIP
 *     graph. The "prepare" functions are synchronous: they enqueue, wait for the stream and
 *     return a verdict.
 *   - Every shape, stride, alignment or scale-layout mismatch is reported as a negative status
 *     before anything is enqueued; nothing is silently degraded (page
 *     "recipes/docker-images/mia-tp4/adapter/shared_pad_k.py", module docstring, last paragraph).
 *   - Sizes are int64_t; an empty problem (M == 0) is a valid no-op.
 */
#ifndef BSFP8_H
#define BSFP8_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define BSFP8_ABI_VERSION 1

/* Symbols of the shared library; everything else in it is hidden. */
#if defined(__GNUC__) || defined(__clang__)
#define BSFP8_API __attribute__((visibility("default")))
#else
#define BSFP8_API
#endif

typedef enum bsfp8_status {
  BSFP8_OK = 0,
  BSFP8_NOT_EXACT = 1,      /* make_twin verdict: the twin does not rebuild the weight (not an error) */
  BSFP8_EINVAL = -1,        /* null pointer where one is required, bad enum value, or an output
                               buffer overlapping an input, the workspace or another output */
  BSFP8_ESHAPE = -2,        /* sizes out of range or not multiples of the 32x32 block */
  BSFP8_ESCALE = -3,        /* a block scale is not a positive finite power of two */
  BSFP8_ESTRIDE = -4,       /* leading dimension too small or misaligned, pointer not 16-byte aligned */
  BSFP8_EWORKSPACE = -5,    /* workspace missing or smaller than bsfp8_workspace_bytes() */
  BSFP8_EHIP = -6           /* a HIP runtime call failed */
} bsfp8_status;

typedef enum bsfp8_out {
  BSFP8_OUT_BF16 = 0,       /* y is uint16_t bf16 patterns, round-half-to-even from fp32 */
  BSFP8_OUT_F32 = 1         /* y is float (the LM-head logits of page
                               "recipes/docker-images/mia-tp4/docs/tp4-adapters.md", row draft_head_fp8) */
} bsfp8_out;

/* Human-readable name of a status code (static string, never NULL). */
BSFP8_API const char* bsfp8_strerror(int status);

/* BSFP8_ABI_VERSION of the built library. */
BSFP8_API int bsfp8_abi_version(void);

/* ------------------------------------------------------------------------------------------
 * Prepare (load time; synchronous)
 * ------------------------------------------------------------------------------------------ */

/* fp32 block scales -> exponent bytes.
 * Page "shared_pad_k.py", function _pad_weight: a block-fp8 weight [N,K] carries fp32 scales
 * [N/32, K/32] that must be positive powers of two (zero fraction bits and > 0).
 *   scales   : float [rows][cols], row-major, contiguous (device).
 *   exp_out  : uint8_t [rows][cols] (device); byte = fp32 exponent field (2^(b-127) == scale).
 *   n_bad_out: host, nullable; receives the number of refused scales.
 * Refused: fraction bits set, zero, negative, subnormal, +inf, NaN. Returns BSFP8_ESCALE if any
 * scale is refused (exp_out then holds 0 at those positions), BSFP8_ESHAPE if rows or cols < 0. */
BSFP8_API int bsfp8_scales_from_f32(const float* scales, int64_t rows, int64_t cols, uint8_t* exp_out,
                          int64_t* n_bad_out, void* stream);

/* bf16 weight -> e4m3 twin, accepted only when it rebuilds the weight bit for bit.
 * Page "wo_a_w8.py", function make_twin. Per 32x32 block: amax = max|w|; the block exponent e is
 * the least integer with max(amax, 2^-126) <= 448 * 2^e, clamped to [-127, 127]; q = e4m3 RNE of
 * w * 2^-e; the block is exact when bf16(e4m3(q) * 2^e) equals w in every bit.
 *   w        : uint16_t bf16 [G][R][D] (device), R and D multiples of 32.
 *   q_out    : uint8_t [G][R][D] (device).
 *   e_out    : uint8_t [G][R/32][D/32] (device), byte = e + 127.
 *   block_ok : uint8_t [G][R/32][D/32] (device, nullable): 1 exact, 0 not.
 *   n_bad_out: host, nullable: number of blocks that are not exact.
 * A block holding inf or NaN is never exact; it gets exponent byte 255 and codes 0x7F (e4m3 NaN).
 * Returns BSFP8_OK when every block is exact, BSFP8_NOT_EXACT otherwise (the page then keeps the
 * bf16 weight); outputs are written in both cases. */
BSFP8_API int bsfp8_make_twin(const uint16_t* w, int64_t G, int64_t R, int64_t D, uint8_t* q_out,
                    uint8_t* e_out, uint8_t* block_ok, int64_t* n_bad_out, void* stream);

/* bsfp8_make_twin without the synchronisation, for loading many layers: the encoder is enqueued
 * on `stream` and the call returns at once; the verdict stays on the device. Same rule, outputs
 * and page as bsfp8_make_twin.
 *   n_bad_dev: device int64_t, 8-byte aligned: the number of blocks that are not exact is ADDED to
 *              it (the caller zeroes it first; one counter may gather several layers). The twin
 *              is exact iff the count it received is 0.
 * Allocates nothing and does not wait, so it may be captured in a graph (zero the counter with a
 * kernel, not a memset node, before each replay that should count from zero). Returns BSFP8_OK once
 * enqueued, BSFP8_ESHAPE / ESTRIDE / EINVAL as bsfp8_make_twin (EINVAL also for a missing or
 * misaligned n_bad_dev, or one that overlaps w or an output), BSFP8_EHIP on a launch failure. */
BSFP8_API int bsfp8_make_twin_async(const uint16_t* w, int64_t G, int64_t R, int64_t D, uint8_t* q_out,
                                    uint8_t* e_out, uint8_t* block_ok, int64_t* n_bad_dev, void* stream);

/* bf16 weight -> e4m3 twin with one exponent per row and 32 columns, accepted only when it rebuilds
 * the weight bit for bit. Page "recipes/docker-images/mia-tp4/docs/tp4-adapters.md", row
 * draft_main_proj: each rank keeps its output columns as e4m3 with per-(row, 32-column)
 * power-of-two scales, checked to reproduce the weight exactly. The per-block rule is the one of
 * bsfp8_make_twin, applied to 1x32 blocks.
 *   w        : uint16_t bf16 [G][N][K] (device, 16-byte aligned), K a multiple of 32.
 *   q_out    : uint8_t [G][N][K] (device, 16-byte aligned).
 *   e_out    : uint8_t [G][N][K/32] (device), byte = e + 127 (255 for a block holding inf or NaN).
 *   block_ok : uint8_t [G][N][K/32] (device, nullable): 1 exact, 0 not.
 *   n_bad_out: host, nullable: number of blocks that are not exact.
 * Returns BSFP8_OK when every block is exact, BSFP8_NOT_EXACT otherwise; outputs are written in
 * both cases. */
BSFP8_API int bsfp8_make_twin_row32(const uint16_t* w, int64_t G, int64_t N, int64_t K, uint8_t* q_out,
                                    uint8_t* e_out, uint8_t* block_ok, int64_t* n_bad_out, void* stream);

/* Pad the contraction dimension of a twin: codes [G][N][K] -> [G][N][K_pad] with zero codes,
 * exponents [G][N/32][K/32] -> [G][N/32][K_pad/32] with byte 127 (factor 1.0).
 * Page "shared_pad_k.py", module docstring (WHAT THE PATCH DOES, item 1) and _pad_weight: the
 * weight is padded with zeros and its scales with ones. K, K_pad multiples of 32, K_pad >= K.
 * Asynchronous (no verdict). */
BSFP8_API int bsfp8_pad_k_weight(const uint8_t* q, const uint8_t* e, int64_t G, int64_t N, int64_t K,
                       int64_t K_pad, uint8_t* q_pad, uint8_t* e_pad, void* stream);

/* Standalone dequantisation of a twin to bf16 (page "wo_a_w8.py", _dequant_kernel and
 * dequant_into_scratch): w_out[g][n][k] = bf16(e4m3(q) * 2^(b-127)), exact.
 *   q: [G][N][K], e: [G][N/32][K/32], w_out: uint16_t [G][N][K] (all device, caller-owned);
 *   N and K multiples of 32, K <= 2^24; q and w_out 16-byte aligned. Asynchronous.
 * Returns BSFP8_ESHAPE (N or K not a multiple of 32, negative sizes, K > 2^24), BSFP8_EINVAL
 * (a missing pointer, w_out overlapping q or e), BSFP8_ESTRIDE (misaligned q or w_out), BSFP8_EHIP
 * on a launch failure; nothing to do (a zero size) is BSFP8_OK. */
BSFP8_API int bsfp8_dequant(const uint8_t* q, const uint8_t* e, int64_t G, int64_t N, int64_t K,
                  uint16_t* w_out, void* stream);

/* ------------------------------------------------------------------------------------------
 * Per call (asynchronous, graph-capturable, no allocation, no synchronisation)
 * ------------------------------------------------------------------------------------------ */

/* Pad activations: x [M][ldx] with group g at columns [g*K, (g+1)*K) -> x_pad [M][G*K_pad]
 * (contiguous), group g at [g*K_pad, g*K_pad + K) and zeros in [g*K_pad + K, (g+1)*K_pad).
 * Page "shared_pad_k.py", _pad_input (its tail stays zero). ldx >= G*K. */
BSFP8_API int bsfp8_pad_k_input(const uint16_t* x, int64_t ldx, int64_t M, int64_t G, int64_t K,
                      int64_t K_pad, uint16_t* x_pad, void* stream);

/* Workspace bytes the GEMM entry points need for this shape (0 when no split of K across
 * workgroups is used). split_k as in the GEMM calls (0 = built-in table). The workspace holds,
 * for the one-pass kernels, one 64-bit exchange slot per output (rows rounded up to 16) and node
 * of the pairwise-combine tree over the splits, and for the tile kernel the fp32 partials
 * [splits][M][G][N] its reduce kernel sums. It must be ZERO-FILLED once after allocation; every
 * call leaves the exchange slots at zero again (the second partner of each node clears its slot).
 * One workspace must not be used by two calls that can run at the same time (e.g. on two
 * streams). */
BSFP8_API size_t bsfp8_workspace_bytes(int64_t M, int64_t G, int64_t N, int64_t K, int split_k);

/* The GEMM. Page "wo_a_w8.py": _wo_a_partial_w8 (2..8 rows) and _wo_a_mid_kernel (9..192 rows).
 *   x       : uint16_t bf16 [M][ldx] (device, 16-byte aligned), group g at columns [g*K,(g+1)*K);
 *             ldx >= G*K and ldx % 8 == 0.
 *   q, e    : twin codes [G][N][K] and exponent bytes [G][N/32][K/32] (device; q 16-byte, e 4-byte aligned);
 *             N and K multiples of 32. Exponent byte 255 and e4m3 NaN codes give NaN outputs.
 *             The kernels read e in aligned 4-byte words: when its size is not a multiple of 4,
 *             up to 3 bytes past its end are read (within the same word, hence the same page);
 *             they never reach a result.
 *   split_k : number of workgroups that share one output tile's K range (fixed-order reduction);
 *             0 = the built-in table for this shape; otherwise 1..64.
 *   ws      : workspace of ws_bytes >= bsfp8_workspace_bytes(M,G,N,K,split_k) (may be NULL when
 *             that is 0).
 *   y       : [M][G][N] contiguous, bf16 (uint16_t) or float per out_dtype (device, 16-byte
 *             aligned); must not overlap x, q, e or ws (BSFP8_EINVAL).
 * Summation order: each output is an fp32 sum over 128-wide K chunks in a fixed order that
 * depends only on (M, G, N, split_k) and on K rounded up to a multiple of 128, so results are
 * bitwise reproducible run to run, and K zero-padded within the same multiple of 128 (e.g.
 * 576 -> 640) gives bitwise the same Y (page "shared_pad_k.py", LOSSLESS).
 * bsfp8_gemm_small takes 1 <= M <= 16, bsfp8_gemm_mid 1 <= M <= 256; bsfp8_gemm picks small for
 * M <= 8 and mid above (page "wo_a_w8.py", module docstring: 2..8 rows vs 9..192 rows). */
BSFP8_API int bsfp8_gemm_small(const uint16_t* x, int64_t ldx, int64_t M, int64_t G, int64_t N, int64_t K,
                     const uint8_t* q, const uint8_t* e, int split_k, void* ws, size_t ws_bytes,
                     void* y, int out_dtype, void* stream);
BSFP8_API int bsfp8_gemm_mid(const uint16_t* x, int64_t ldx, int64_t M, int64_t G, int64_t N, int64_t K,
                   const uint8_t* q, const uint8_t* e, int split_k, void* ws, size_t ws_bytes,
                   void* y, int out_dtype, void* stream);
BSFP8_API int bsfp8_gemm(const uint16_t* x, int64_t ldx, int64_t M, int64_t G, int64_t N, int64_t K,
               const uint8_t* q, const uint8_t* e, int split_k, void* ws, size_t ws_bytes,
               void* y, int out_dtype, void* stream);

/* bsfp8_gemm without a workspace argument, for callers that cannot allocate device memory (code
 * under HIP graph capture, tight serving loops, harnesses that forbid hipMalloc). Arguments,
 * plans, kernels, summation order and results are those of bsfp8_gemm with the same split_k
 * (bitwise the same Y). A plan that needs a workspace uses a fixed array in the library's own
 * device memory instead: BSFP8_NO_ALLOC_SCRATCH_BYTES bytes, of which each GPU the library runs
 * on holds its own copy until the process ends. The call allocates nothing; it enqueues a small zero-fill
 * kernel before a plan whose exchange slots must start at zero. Errors as bsfp8_gemm, plus
 * BSFP8_EWORKSPACE (nothing enqueued) when the plan's workspace (bsfp8_workspace_bytes) exceeds
 * BSFP8_NO_ALLOC_SCRATCH_BYTES, and BSFP8_EHIP when the array's address cannot be looked up.
 * Every call on one GPU shares that GPU's array: calls that can overlap on one GPU (two streams,
 * two threads) race and must not be made; calls ordered on one stream are safe. */
#define BSFP8_NO_ALLOC_SCRATCH_BYTES (16u << 20)
BSFP8_API int bsfp8_gemm_no_alloc(const uint16_t* x, int64_t ldx, int64_t M, int64_t G, int64_t N, int64_t K,
                                  const uint8_t* q, const uint8_t* e, int split_k, void* y, int out_dtype,
                                  void* stream);

/* The GEMM on a twin with one exponent per row and 32 columns (bsfp8_make_twin_row32): the GEMV
 * of page "recipes/docker-images/mia-tp4/docs/tp4-adapters.md", row draft_main_proj, for up to
 * 16 rows. W[g][n][k] = bf16(e4m3(q[g][n][k]) * 2^(e[g][n][k/32] - 127)); otherwise arguments,
 * layouts, summation order and errors as bsfp8_gemm, with 1 <= M <= 16 (0 is a no-op) and
 * K % 128 == 0. The workspace (exchange slots when K is split over workgroups) is sized by
 * bsfp8_workspace_bytes_row32 and must be zero-filled once after allocation. */
BSFP8_API size_t bsfp8_workspace_bytes_row32(int64_t M, int64_t G, int64_t N, int64_t K, int split_k);
BSFP8_API int bsfp8_gemm_row32(const uint16_t* x, int64_t ldx, int64_t M, int64_t G, int64_t N, int64_t K,
                               const uint8_t* q, const uint8_t* e, int split_k, void* ws, size_t ws_bytes,
                               void* y, int out_dtype, void* stream);

/* ------------------------------------------------------------------------------------------
 * MXFP8 activations and the fp8 x fp8 GEMM (W8A8; per call, asynchronous, no allocation)
 *
 * Page "recipes/docker-images/mia-tp4/adapter/shared_pad_k.py" (module docstring, DIAGNOSIS and
 * LOSSLESS): the pages' MXFP8 linear quantizes its bf16 input itself into e4m3 values with one
 * power-of-two (E8M0) scale per 32 consecutive values of a row and multiplies that with the
 * block-fp8 weight. The pages do not print the quantizer; the rule here is OCP Microscaling (MX)
 * v1.0 for MXFP8: per 32-value block, s = floor(log2(max |v|)) - 8 clamped to [-127, 127]
 * (an all-zero block gets -127), each element e4m3(v * 2^-s) rounded to nearest even and
 * saturated at +-448; a block holding inf or NaN gets scale byte 255 and e4m3 NaN codes
 * (0x7F, or 0xFF for a negative sign). Unlike the bf16 path this is lossy: it is the pages'
 * comparison path, not the exact twin GEMM.
 * ------------------------------------------------------------------------------------------ */

/* bf16 activations -> MXFP8 codes and scale bytes.
 *   x  : uint16_t bf16 [M][ldx] (device, 16-byte aligned), ldx >= L, ldx % 8 == 0.
 *   xq : uint8_t e4m3 codes [M][L] (device, contiguous, 16-byte aligned).
 *   xs : uint8_t scale bytes [M][L/32] (device, contiguous), byte = s + 127 (2^(byte-127)).
 * L % 32 == 0. Deterministic and exact (every decision is an integer one). */
BSFP8_API int bsfp8_quantize_mx(const uint16_t* x, int64_t ldx, int64_t M, int64_t L, uint8_t* xq,
                                uint8_t* xs, void* stream);

/* Y[m][g][n] = sum_k Xmx[m][g*K + k] * W[g][n][k], with Xmx = e4m3(xq) * 2^(xs - 127) per
 * 32-value row block and W = e4m3(q) * 2^(e - 127) per 32x32 weight block (the weight's block
 * exponent serves as the MX scale of each row's 32-value piece).
 *   xq, xs : codes [M][ldq] (16-byte aligned) and scale bytes [M][ldq/32] (4-byte aligned), group g
 *            at columns [g*K, (g+1)*K) (e.g. the output of bsfp8_quantize_mx with L = G*K);
 *            ldq >= G*K and ldq % 128 == 0.
 *   q, e   : the weight twin as for bsfp8_gemm (q 16-byte aligned, e 4-byte aligned).
 *   y      : [M][G][N] bf16 (RNE) or fp32 per out_dtype (16-byte aligned).
 * 1 <= M <= 256 (M == 0 is a no-op), N % 32 == 0, K % 128 == 0 and K <= 8192. The products run
 * on the block-scaled fp8 MFMA with fp32 accumulation across 128-wide chunks; the hardware sums
 * each group of eight adjacent products inside the instruction with a precision of about 2^-14
 * of the group's largest product (measured), so results are not those of an exact sum rounded
 * once. The summation order is fixed by the built-in configuration: bitwise reproducible. */
BSFP8_API int bsfp8_gemm_mx(const uint8_t* xq, const uint8_t* xs, int64_t ldq, int64_t M, int64_t G,
                            int64_t N, int64_t K, const uint8_t* q, const uint8_t* e, void* y,
                            int out_dtype, void* stream);

/* ------------------------------------------------------------------------------------------
 * MXFP8 output epilogue (per call, asynchronous, no allocation)
 *
 * Page "recipes/docker-images/mia-tp4/adapter/wo_a_w8.py": its module docstring reports the
 * MXFP8-epilogue path (what production runs), and in `install` the dropped-weight path and
 * small_mx hand the fp32 split partials [S][M][G][N] of _partial_w8 to a kernel that sums them
 * and quantises the sum to MXFP8 in one pass, where the plain path sums them with _wo_a_reduce and
 * rounds to bf16. Neither the quantiser nor the order of that sum is printed. Here:
 *   - the partials are added in fp32 in a fixed order (bsfp8_sum_order);
 *   - the sum, viewed as [M][L] (L = G*N for the GEMM), is quantised per 32 consecutive values of
 *     a row with the rule of bsfp8_quantize_mx (OCP MX v1.0: s = floor(log2 amax) - 8 clamped to
 *     [-127, 127], e4m3 RNE with saturation at 448, scale byte s + 127; byte 255 and e4m3 NaN
 *     codes for a block holding inf or NaN);
 *   - codes are [M][L] and scale bytes [M][L/32], both row-major (the pages' consumer wants its
 *     scales in a swizzled layout of its own, which is not reproduced).
 * ------------------------------------------------------------------------------------------ */

typedef enum bsfp8_sum_order {
  BSFP8_SUM_ASCENDING = 0,  /* ((p0 + p1) + p2) + ... : the order of the page's _wo_a_reduce */
  BSFP8_SUM_PAIRWISE = 1    /* pairwise tree over the split index: p2i + p2i+1, an unpaired last
                               partial carried up unchanged, repeated until one value is left */
} bsfp8_sum_order;

/* Fixed-order sum of S fp32 partials and MXFP8 quantisation of the sum.
 *   part  : float [S][M][L] (device, contiguous, 16-byte aligned).
 *   S     : 1..64 partials (S = 1 quantises part itself).
 *   order : a bsfp8_sum_order.
 *   yq    : uint8_t e4m3 codes [M][L] (device, contiguous, 16-byte aligned).
 *   ys    : uint8_t scale bytes [M][L/32] (device, contiguous).
 * L % 32 == 0 and L >= 32; M == 0 is a no-op. Every addition is an IEEE fp32 addition and every
 * quantisation decision an integer one, so the result is bit-exact and deterministic. */
BSFP8_API int bsfp8_reduce_quantize_mx(const float* part, int64_t S, int64_t M, int64_t L, int order,
                                       uint8_t* yq, uint8_t* ys, void* stream);

/* Workspace bytes of bsfp8_gemm_mxfp8 for this shape and split_k (never 0 for a valid shape:
 * the fp32 results, one copy per split, may pass through it). Nothing in it needs clearing; one
 * workspace must not be used by two calls that can run at the same time. */
BSFP8_API size_t bsfp8_workspace_bytes_mxfp8(int64_t M, int64_t G, int64_t N, int64_t K, int split_k);

/* The GEMM of bsfp8_gemm with the MXFP8 epilogue: the fp32 results of the plan that
 * bsfp8_plan_info(..., path 3) reports for (M, G, N, K, split_k) - the sum itself with one split,
 * else each split's partial - go to ws, and the epilogue adds the partials in the order of that
 * plan's own combine (pairwise for the one-pass kernels, ascending for the tile kernel), so the
 * quantised values are exactly the fp32 outputs of bsfp8_gemm_config with that configuration and
 * chunks per split (out_dtype = BSFP8_OUT_F32). That is bsfp8_gemm's own plan, except on the
 * decode shapes where bsfp8_gemm takes the paired kernel: its 8-row tiles hold a quarter of an MX
 * block, so this call keeps the 16-row decode plan, whose fused form quantises whole blocks.
 *   x, ldx, M, G, N, K, q, e, split_k : as bsfp8_gemm (1 <= M <= 256).
 *   ws    : >= bsfp8_workspace_bytes_mxfp8(M, G, N, K, split_k) bytes (device, 16-byte aligned).
 *   yq    : uint8_t e4m3 codes [M][G*N] (device, contiguous, 16-byte aligned).
 *   ys    : uint8_t scale bytes [M][G*N/32] (device, contiguous).
 * For a decode plan with one split (up to 16 rows, K a multiple of 128, at most 32 chunks) one
 * fused kernel computes and quantises 32 output columns per workgroup; otherwise two kernels run
 * on `stream`, the GEMM (writing the fp32 results into ws) and the epilogue. Both forms give the
 * same bits. */
BSFP8_API int bsfp8_gemm_mxfp8(const uint16_t* x, int64_t ldx, int64_t M, int64_t G, int64_t N, int64_t K,
                               const uint8_t* q, const uint8_t* e, int split_k, void* ws, size_t ws_bytes,
                               uint8_t* yq, uint8_t* ys, void* stream);

/* ------------------------------------------------------------------------------------------
 * The verify step of speculative decoding (per call, asynchronous, no allocation): the paged
 * MXFP8 key/value cache, attention of drafted tokens over it, and verification of the drafts.
 *
 * The decode and verify projections above run on a root token and a handful of drafted tokens
 * per sequence; these calls are what such a step does between them.
 * ------------------------------------------------------------------------------------------ */

/* A paged key/value cache in MXFP8 (the format of bsfp8_quantize_mx along the head dimension):
 *   kq, vq : uint8_t e4m3 codes [pages][heads][page][dim] (device, 16-byte aligned);
 *   ks, vs : uint8_t scale bytes [pages][heads][page][dim/32] (device, 16-byte aligned), 2^(byte-127).
 * dim is 64, 128, 192 or 256; page (tokens per page) a multiple of 16; heads >= 1; pages >= 0 and
 * pages * page < 2^31, pages * page * heads < 2^35 (offsets inside the cache are 64-bit). Slot s is token s % page of page
 * s / page. Every call below returns BSFP8_ESHAPE for sizes outside these, BSFP8_EINVAL for a
 * missing pointer, BSFP8_ESTRIDE for a misaligned one. */
typedef struct bsfp8_kv_cache {
  uint8_t* kq;
  uint8_t* ks;
  uint8_t* vq;
  uint8_t* vs;
  int64_t pages, heads, page, dim;
} bsfp8_kv_cache;

/* Write R tokens into the cache, with the norms of queries and keys and the position rotation in
 * the same pass. Per token r, in fp32 from the bf16 inputs:
 *   queries and keys: y = x * 1/sqrt(mean(x^2) + eps) * weight over the head's dim values (skipped
 *   where the weight is NULL), then the first `rot` values of the head are rotated by the angle of
 *   positions[r]: (a, b) -> (a cos - b sin, b cos + a sin) for the pairs (i, i + rot/2), or
 *   (2i, 2i + 1) when `interleaved` (skipped when rot is 0);
 *   queries are rounded to bf16 into q_out; keys and values are quantised to MXFP8 (the rule of
 *   bsfp8_quantize_mx, on the fp32 value: keys are not rounded to bf16 in between) into slots[r].
 *   slots     : int64_t [R] (device). A slot outside [0, pages * page) (e.g. -1 for a padding row)
 *               stores no key and value; its query is written all the same. Two rows of one call
 *               must not have the same slot: they would leave a mixture of both rows' bytes there.
 *   k, v      : bf16 [R][ldk], [R][ldv], head h at columns [h*dim, (h+1)*dim) (16-byte aligned; row
 *               strides >= heads*dim, multiples of 8: slices of a fused projection).
 *   q, q_out  : bf16 [R][ldq] with hq heads, and [R][hq][dim] contiguous; NULL with hq = 0.
 *   q_weight, k_weight : bf16 [dim] (16-byte aligned), nullable. eps >= 0 and finite.
 *   cos_sin   : float [n_positions][rot] (16-byte aligned): rot/2 cosines, then rot/2 sines.
 *   rot       : 0 or a multiple of 16 up to dim (cos_sin and positions are not read when 0).
 *   positions : int64_t [R] (device). A position outside [0, n_positions) gives NaN in the rotated
 *               values (and so a NaN block, scale byte 255, in the cache).
 * R < 2^24. q_out must not overlap an input or the cache, and the cache no input (BSFP8_EINVAL). */
BSFP8_API int bsfp8_cache_write(const bsfp8_kv_cache* cache, const int64_t* slots, int64_t R,
                                const uint16_t* k, int64_t ldk, const uint16_t* v, int64_t ldv,
                                const uint16_t* q, int64_t ldq, int64_t hq, uint16_t* q_out,
                                const uint16_t* q_weight, const uint16_t* k_weight, float eps,
                                const float* cos_sin, int64_t n_positions, int64_t rot,
                                const int64_t* positions, int interleaved, void* stream);

/* Rows of the cache as bf16: k_out, v_out [R][heads][dim] (contiguous, 16-byte aligned), each value
 * e4m3(code) * 2^(byte-127) rounded once to bf16 (exact unless it falls below the bf16 normals;
 * scale byte 255 and NaN codes give NaN). A slot outside the cache gives zeros. R * heads < 2^31 and
 * R * heads * dim <= 2^36 - 4096. */
BSFP8_API int bsfp8_cache_read(const bsfp8_kv_cache* cache, const int64_t* slots, int64_t R,
                               uint16_t* k_out, uint16_t* v_out, void* stream);

/* Workspace bytes of bsfp8_tree_attention for these sizes (0 for sizes it refuses; never more for a smaller B, T or
 * max_len of the same heads and dim: the largest call's workspace serves them all). The contents need no clearing; one
 * workspace must not be used by two calls that can run at the same time. */
BSFP8_API size_t bsfp8_attention_workspace_bytes(int64_t B, int64_t T, int64_t hq, int64_t hkv, int64_t dim,
                                                 int64_t max_len);

/* Attention of T drafted tokens (nodes) per sequence over the cache, which already holds them:
 *   out[b][t][h] = sum_j softmax_j(scale * q[b][t][h] . K[b][j][h / (hq/hkv)]) V[b][j][h / (hq/hkv)]
 * over the positions j that node t of sequence b sees. Sequence b holds lens[b] tokens, position j in
 * slot (pages[b][j / page], j % page); its last nodes[b] tokens are the nodes (node i at position
 * lens[b] - nodes[b] + i), the ones before them its prefix, which every node sees. Without a mask
 * node t sees nodes 0..t (a chain; T = 1 is plain decoding); with one it sees node i where bit i
 * of mask[b][t] is set (a tree: a node's ancestors and itself).
 *   q     : bf16 [B*T][ldq], head h at columns [h*dim, (h+1)*dim) (16-byte aligned, ldq % 8 == 0).
 *   pages : int32_t [B][ld_pages] (device). A page outside [0, cache->pages) holds no tokens: its
 *           positions are seen by no node.
 *   lens  : int32_t [B] (device), the nodes included; cut to [0, min(max_len, ld_pages * page)].
 *   nodes : int32_t [B] (device), cut to [0, T]; NULL: T everywhere. Rows t >= nodes[b] are zeros.
 *   mask  : int64_t [B][T] (device) or NULL; with a mask T <= 64.
 *   max_len : 0 to 2^31 - 2^14, a bound of lens.
 *   scale : finite (BSFP8_EINVAL).
 *   out   : bf16 [B][T][hq][dim] (contiguous, 16-byte aligned). A node that sees nothing gets zeros.
 * Values of positions that a node does not see never reach it, also when they are NaN or infinite
 * (a rejected draft's leftovers, a page never written); those that it sees have the effect they have in the formula,
 * values whose code times scale passes bf16 counting as infinite. (In fp32, that is: a weight below 2^-126 of the
 * row's largest is 0, and may make an infinity or NaN of an infinite value; a row whose scores are all -inf gets
 * zeros.) hq is a multiple of cache->heads, at most
 * 64 times it; T >= 1; B * T * hq < 2^31, and fewer than 2^24 blocks of 16 rows (B times the key/value
 * heads times T * hq / heads / 16, rounded up). Scores and sums are fp32; the weights of one tile are
 * rounded to bf16 for the product with V (rebuilt exactly from its codes, as K is). The split of
 * the positions over workgroups depends on lens and the sizes only: results repeat bit for bit. */
BSFP8_API int bsfp8_tree_attention(const uint16_t* q, int64_t ldq, int64_t B, int64_t T, int64_t hq,
                                   const bsfp8_kv_cache* cache, const int32_t* pages, int64_t ld_pages,
                                   const int32_t* lens, const int32_t* nodes, const int64_t* mask, float scale,
                                   int64_t max_len, void* ws, size_t ws_bytes, uint16_t* out, void* stream);

/* Type of the logits handed to the verification calls. */
typedef enum bsfp8_logits {
  BSFP8_LOGITS_BF16 = 0,
  BSFP8_LOGITS_F32 = 1
} bsfp8_logits;

/* Workspace bytes of the verification calls (0 for sizes they refuse; never more for smaller sizes). The
 * contents need no clearing: calls of any sizes may use it one after another. Not for two calls that can
 * run at the same time. */
BSFP8_API size_t bsfp8_verify_workspace_bytes(int64_t B, int64_t T, int64_t V);

/* Verification of a chain of T - 1 drafted tokens per sequence. With p_i = softmax(logits[b][i] / t)
 * and q_i = softmax(draft[b][i] / t), t = temperature[b]: draft token x_i = tokens[b][i] is accepted
 * while u[b][i] * q_i(x_i) < p_i(x_i). n = the number accepted before the first refusal. The next
 * token is the first index whose running sum of the weights passes u_sample[b] times their total,
 * the weights being max(p_n - q_n, 0) after a refusal (p_n where that is zero everywhere) and
 * p_{T-1} when all were accepted. With t = 0 (greedy; also t < 0 or NaN) x_i is accepted if it is
 * the lowest index of the largest logit of row i, and the next token is that of row n. An infinite t gives
 * every logit but -inf and NaN the same probability.
 *   logits : [B][T][V], draft : [B][T-1][V], of `dtype` (bsfp8_logits), contiguous, 16-byte aligned.
 *   tokens : int32_t [B][T-1]; one outside [0, V) is refused. temperature: float [B]; u: float
 *            [B][T-1]; u_sample: float [B], uniform in [0, 1) (all device; the draft arrays may be NULL
 *            when T = 1).
 *   out_tokens : int32_t [B][T]: the n accepted tokens, the next one, then -1. n_accepted: int32_t [B].
 * A sequence of fewer drafts than T - 1 fills up with tokens -1 and draft rows of -inf: the first of them is refused, and
 * since its draft row has no probability the next token comes from p_n. (A refused token with any other draft row draws from
 * max(p_n - q_n, 0).) What lies behind the first refusal takes no part.
 * 1 <= T <= 64, 1 <= V <= 2^24, B * (2 T - 1) < 2^24. Probabilities and running sums are 64-bit, so that neighbouring
 * sums are told apart. -inf logits have probability 0; a NaN logit counts as -inf; +inf ones share
 * the row. A row of nothing but -inf or NaN gives index 0. */
BSFP8_API int bsfp8_verify_chain(const void* logits, const void* draft, int dtype, int64_t B, int64_t T, int64_t V,
                                 const int32_t* tokens, const float* temperature, const float* u,
                                 const float* u_sample, void* ws, size_t ws_bytes, int32_t* out_tokens,
                                 int32_t* n_accepted, void* stream);

/* Verification of a tree of drafted tokens: node 0 is the root, node i carries tokens[b][i] and hangs
 * from node parents[b][i] < i. Every node samples its next token from softmax(logits[b][i] / t) with
 * u[b][i] (the rule above; the lowest index of the largest logit when t = 0); from the root, the walk
 * goes on to the child that carries the sampled token (the lowest-numbered one of equals) until there
 * is none.
 *   tokens, parents : int32_t [B][T] (device; the root's entries are not read). A parent outside [0, i) cuts the node off.
 *   out_tokens : int32_t [B][T]: the sampled token of each node of the path (the accepted drafts, then
 *                the next token), then -1. path: int32_t [B][T]: the path's nodes from the root, then -1.
 *   n_accepted : int32_t [B]: the drafts accepted (the path's length less one).
 * Other arguments and limits as bsfp8_verify_chain. */
BSFP8_API int bsfp8_verify_tree(const void* logits, int dtype, int64_t B, int64_t T, int64_t V, const int32_t* tokens,
                                const int32_t* parents, const float* temperature, const float* u, void* ws,
                                size_t ws_bytes, int32_t* out_tokens, int32_t* path, int32_t* n_accepted,
                                void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BSFP8_H */
