/*
 * mmq.h -- C ABI of libmmq: the k-quant "MMQ" prefill GEMM on GB300 (sm_103a)
 *
 *     Y[T x O] = X[T x K] . W[O x K]^T
 *
 * with W stored in a k-quant format (q4_K, q6_K, q5_K) or q8_0 and X quantised per
 * 32-element block to q8_1.  The method is the one described on the
 * "minfer" CUDA optimisation pages for the q4_K MMQ line:
 *   - "31 . r28 -- Direction-A raw-nibble NB kernel, 2 blocks/SM", section
 *     2.3 "The numerics contract": the integer dot of unsigned 4-bit weights
 *     with int8 activations over each 32-weight sub-block, followed by the
 *     f32 two-term fold  sum += dx*(d*sc)*C + (dx*ssum)*(-(dmin*m)),
 *     stored f32 with no f16 between the dot and the store;
 *   - "19 . r14 -- B fragments via ldmatrix + widened scale reads", 3.2(d):
 *     the q8_1 activation scale pair (f16 d | int16 block sum);
 *   - "43 . r40 -- __launch_bounds__(256,3) third resident block", 5:
 *     q6_K, w = d*sc*(q-32) on 16-weight sub-blocks.
 *
 * Which call for which job
 * ------------------------
 *   prefill, T >= ~256 ....... mmq_gemm_q4K / mmq_gemm_q5K / mmq_gemm_q6K
 *                              (whole-super-block accumulation on the tensor
 *                              core; Y to the f32 tolerance, the sub-block
 *                              dots are never formed as numbers)
 *   FFN gate + up + SwiGLU ... mmq_gemm_q4K_swiglu (writes the down
 *                              projection's q8_1 operands)
 *   few output tiles ......... mmq_gemm_q4K_splitk (caller scratch) or
 *                              mmq_gemm_q4K_splitk_static (no allocation)
 *   17 <= T <= 64 ............ mmq_gemm_q4K_small
 *   T <= 4 (decode), f32 in .. mmq_gemv_q4K_f32 / mmq_gemv_q6K_f32 (q8_1
 *                              quantisation built in; per-sub-block integer
 *                              dots on the SIMT cores)
 *   T <= 16 (decode) ......... mmq_gemv_q4K / mmq_gemv_q6K (per-sub-block
 *                              integer dots, exact); mmq_gemm_q4K_small_imma
 *                              takes qs + ds as the pages' q8_1 does, at the
 *                              int8 warp-MMA rate
 *   the pages' literal form .. mmq_gemm_q4K_subblock / _q5K_subblock /
 *                              _q6K_subblock / mmq_gemm_q8_0 (one exact
 *                              integer dot per sub-block, folded in f32 per
 *                              sub-block); slower, kept as the reference form
 *                              on the GPU and for q8_0
 *   positions + cache append . mmq_rope_append (rotary q and k, k and v into the
 *                              paged cache)
 *   attention, new tokens .... mmq_attn_decode (1..16 new tokens per sequence
 *                              over the paged cache)
 *   attention, prompts ....... mmq_attn_prefill (any number of new tokens; capped
 *                              scores, distance bias, window, prefix, documents)
 *   norms + positions + append mmq_norm_rope_append (normed q and k heads, positions
 *                              with several axes)
 *   trees of drafts .......... mmq_attn_tree, then mmq_kv_keep for the accepted path
 *   bounded cache ............ mmq_kv_evict (by accumulated attention weight)
 *   drafted tokens ........... mmq_spec_verify (speculative sampling's test and
 *                              resampling)
 *   diagnostics .............. mmq_debug_subdots_* (the int32 dots themselves),
 *                              mmq_probe_tensor_peak, mmq_debug_fault_inject
 *                              (test-only)
 *
 * Conventions for every call
 * --------------------------
 *   - All array arguments are DEVICE pointers allocated and owned by the
 *     caller (for example PyTorch tensors).  The library allocates no
 *     device memory per call, keeps no pointer after the call returns and
 *     writes only the output arrays named below.
 *   - Work is enqueued asynchronously on `stream` (a cudaStream_t; NULL is
 *     the legacy default stream) on the current device.  A return value of
 *     MMQ_OK means the work was validated and launched, not that it has
 *     finished.  Kernel-side failures (a pipeline wait that exceeded its
 *     time limit) are reported by mmq_check_status().
 *   - Every pointer must be 16-byte aligned.  Inputs must be finite; the
 *     result for NaN or Inf inputs is unspecified.
 *   - The device must be compute capability 10.3 (GB300).
 *   - Return value: MMQ_OK (0) or a negative MMQ_ERR_* code; on error
 *     nothing is launched and no output is written.
 *
 * Storage formats (little-endian, rows contiguous)
 * ------------------------------------------------
 *   q4_K super-block, 144 bytes per 256 weights of one row: f16 d (bytes
 *     0-1), f16 dmin (2-3), 12 bytes of packed 6-bit sub-block scales and
 *     mins (4-15, GGUF k-quant packing), 128 bytes of 4-bit quants (16-143);
 *     sub-block j (weights 32j..32j+31) is the low nibble (j even) or high
 *     nibble (j odd) of quant bytes 32*(j/2) .. 32*(j/2)+31.
 *     w = d*sc_j*q - dmin*m_j.
 *   q6_K super-block, 210 bytes: ql[128], qh[64], int8 scales[16], f16 d
 *     (GGUF order); w = d*sc_(e/16)*(q-32), q in 0..63.
 *   W: [O][K/256] super-blocks, O*(K/256)*bytes_per_block bytes in total.
 *   q8_1 activations, split-plane form of the pages' 40-byte block:
 *     qs  int8     [T][K]     quantised values, -127..127;
 *     xh  uint16   [T][K]     the same values as IEEE f16 (exact integers):
 *                             the operand of the per-sub-block kernels;
 *     xa  uint16   [2][T][K]  the dequantised value v = f32(d)*q as two f16
 *                             planes, hi = f16(v) then lo = f16(v - hi); both
 *                             are exact and hi + lo == v (v is a multiple of
 *                             2^-24 with at most 18 significant bits) as long
 *                             as |v| <= 65504, the f16 range (activations of
 *                             larger magnitude overflow the hi plane): the
 *                             operand of the production GEMMs;
 *     ds  uint32   [T][K/32]  low 16 bits: f16 d of the 32-block,
 *                             high 16 bits: int16 sum of its 32 values.
 *   Y: f32 [T][O], row-major, overwritten.
 */
#ifndef MMQ_H
#define MMQ_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st;
typedef struct CUstream_st *mmq_stream_t;   /* == cudaStream_t */

enum {
    MMQ_OK = 0,
    MMQ_ERR_SHAPE = -1,     /* a size is out of range (see each call)              */
    MMQ_ERR_ALIGN = -2,     /* a pointer or leading dimension is misaligned        */
    MMQ_ERR_ARCH = -3,      /* current device is not compute capability 10.3      */
    MMQ_ERR_LAUNCH = -4,    /* the CUDA runtime refused the launch                 */
    MMQ_ERR_TIMEOUT = -5,   /* (mmq_check_status) a kernel pipeline wait timed out */
    MMQ_ERR_NULL = -6,      /* a required pointer is NULL                          */
    MMQ_ERR_DRIVER = -7,    /* the driver could not build a TMA tensor map         */
    MMQ_ERR_CUDA = -8,      /* (mmq_check_status) a CUDA error is pending          */
    MMQ_ERR_SCRATCH = -9,   /* the call needs more than the library's static scratch */
    MMQ_ERR_DEVICE = -10,   /* current device index >= 64 (the library's per-device tables) */
    MMQ_ERR_INDEX = -11     /* (mmq_check_status) a page id, length, count or token that a
                               kernel read from device memory was out of range          */
};

/* Library ABI version; bumped on any change of a signature or format (not when calls are added). */
int mmq_version(void);

/* Human-readable name of a status code (static string, never NULL). */
const char *mmq_status_str(int status);

/*
 * q8_1 quantisation of activations ("31 . r28", 3.2: the q8_1 blocks
 * carrying int8 values and the (f16 d | int16 ssum) pair).
 * For every token t and 32-block b of x[t][0..K):
 *   amax = max |x|;  d32 = amax/127 (IEEE f32 division);
 *   q = clamp(round_half_away_from_zero(x/d32), -127, 127) (IEEE division);
 *   ssum = sum of the 32 q;  stored d = f16(d32), round to nearest even.
 *   An all-zero block stores d = 0, q = 0, ssum = 0.
 * x:   f32, T rows of leading dimension ldx elements (ldx >= K, ldx % 4 == 0).
 * qs:  int8 [T][K] or NULL.   xh: f16 bits [T][K] or NULL.
 * xa:  f16 bits [2][T][K] or NULL.   (at least one of qs, xh, xa)
 * ds:  uint32 [T][K/32], required.
 * T >= 0 (T == 0 is a no-op), 32 <= K <= 2^20, K % 32 == 0.
 */
int mmq_quantize_q8_1(const float *x, int64_t ldx, int T, int K,
                      int8_t *qs, uint32_t *ds, uint16_t *xh, uint16_t *xa, mmq_stream_t stream);

/*
 * q4_K x q8_1 GEMM ("31 . r28", 2.3):  y[t][o] = sum over 32-weight
 * sub-blocks b of  dx_b*(d*sc_b)*C_b + (dx_b*ssum_b)*(-(dmin*m_b)),
 * C_b the exact integer dot of the 32 unsigned quants with the 32 int8
 * activations, i.e. sum_k dequant(W)[o][k]*dequant(X)[t][k]; accumulation
 * in f32 (rounding order unspecified).
 * Production form: the tensor core accumulates each 256-weight super-block
 * from the exact operands v = f32(d)*q (xa, hi + lo) and sc*q; d and the
 * dmin*m term are applied per super-block.
 * w: O*(K/256)*144 bytes.  xa, ds: as written by mmq_quantize_q8_1.
 * y: f32 [T][O], overwritten.
 * T >= 0, O >= 1, 256 <= K <= 2^20, K % 256 == 0.
 */
int mmq_gemm_q4K(const void *w, const uint16_t *xa, const uint32_t *ds,
                 float *y, int T, int O, int K, mmq_stream_t stream);

/*
 * Split-K form of mmq_gemm_q4K for outputs with few 128 x 128 tiles (small T):
 * the super-blocks of each row are divided among up to `ksplit` CTAs per
 * output tile (ceil(K/256 / ksplit) each).  Every CTA writes its partial sums
 * to `part` [splits][T][O] f32; the last CTA of a tile to finish (counted in
 * counters[tile], tile = (t/128) * ceil(O/128) + o/128) adds the splits in
 * split order and writes y, so the result is the same on every call.  The
 * sum is the same mathematical Y as mmq_gemm_q4K's; only the f32 summation
 * order differs.
 * part, counters: caller-owned device scratch; mmq_splitk_sizes gives their
 * sizes.  counters (int32, 4-byte aligned) must be all zero before the first
 * call and are left all zero by every call whose kernel ran, one that timed
 * out included; after a call whose mmq_check_status is not MMQ_OK, y from that
 * call is undefined.  Two calls that use
 * the same part/counters at the same time (different streams) race.
 * ksplit == 1 is mmq_gemm_q4K (part and counters unused, may be NULL).
 * Limits as mmq_gemm_q4K; ksplit >= 1; part 16-byte aligned.
 */
int mmq_splitk_sizes(int T, int O, int K, int ksplit, int64_t *part_floats, int64_t *counters);
int mmq_gemm_q4K_splitk(const void *w, const uint16_t *xa, const uint32_t *ds, float *y,
                        int T, int O, int K, int ksplit, float *part, int *counters, mmq_stream_t stream);

/*
 * The 7B FFN's first half as one launch, chained into the down projection
 * (the pages' workload is whole-model prefill, "31 . r28", 5 "Results"; the
 * FFN activation is not printed there, so this follows the LLaMA-family
 * SwiGLU: h = silu(g) * u, silu(g) = g / (1 + e^-g)).
 *   g = X . W_gate^T and u = X . W_up^T are computed as mmq_gemm_q4K computes
 *   y; the epilogue then evaluates h in f32, one rounding per operation
 *   (expf, add, divide, multiply), and quantises h to q8_1 exactly as
 *   mmq_quantize_q8_1 quantises x: the outputs are the down projection's
 *   operands, ready for mmq_gemm_q4K with K = F.
 * w_gu: 2F q4_K rows, gate and up interleaved in groups of 64 rows: rows
 *   128j .. 128j+63 are gate rows 64j .. 64j+63 and rows 128j+64 .. 128j+127
 *   the up rows of the same features (O*(K/256)*144 bytes with O = 2F).
 * xa, ds: the input's planes as written by mmq_quantize_q8_1 (K columns).
 * h_xa: f16 bits [2][T][F] (hi, lo planes), h_ds: uint32 [T][F/32] (4-byte
 *   aligned), h_qs: int8 [T][F] or NULL; all written.
 * T >= 0, 64 <= F <= 2^20, F % 64 == 0, K as mmq_gemm_q4K.  Deterministic.
 */
int mmq_gemm_q4K_swiglu(const void *w_gu, const uint16_t *xa, const uint32_t *ds,
                        uint16_t *h_xa, uint32_t *h_ds, int8_t *h_qs,
                        int T, int F, int K, mmq_stream_t stream);

/*
 * q4_K GEMM for few tokens (1 <= T <= 64), where the GEMM is bound by
 * streaming W from HBM.  Same operands and result as mmq_gemm_q4K (xa, ds
 * from mmq_quantize_q8_1; y [T][O] f32, overwritten), computed with the
 * weight rows on the tensor core's 128-row side fed from tensor memory and
 * the (at most 64) tokens on the other; the per-super-block fold of
 * "31 . r28" (2.3), as in mmq_gemm_q4K.  Each 128-row tile is handled by a
 * cluster of up to 8 CTAs that split its super-blocks and add their partial
 * sums in a fixed order through distributed shared memory, so the result is
 * the same on every call.  Allocates nothing; no scratch.
 * T <= 64 (MMQ_ERR_SHAPE above), other limits as mmq_gemm_q4K.
 */
int mmq_gemm_q4K_small(const void *w, const uint16_t *xa, const uint32_t *ds, float *y,
                       int T, int O, int K, mmq_stream_t stream);

/*
 * q4_K GEMM for few tokens (1 <= T <= 16) on the int8 warp MMA: the pages'
 * per-sub-block form ("31 . r28", 2.3) with mma.sync m16n8k32 s8 (one
 * instruction per 32-weight sub-block, the nibbles used as int8 operands),
 * the exact integer dots C_b folded in f32 per sub-block.  qs: the int8 q8_1
 * values [T][K] and ds the scale words, both as written by
 * mmq_quantize_q8_1.  Result as mmq_gemm_q4K up to f32 summation order;
 * deterministic.  Allocates nothing.  Kept beside mmq_gemm_q4K_small as the
 * per-sub-block integer form of the same product.
 * T <= 16 (MMQ_ERR_SHAPE above), other limits as mmq_gemm_q4K.
 */
int mmq_gemm_q4K_small_imma(const void *w, const int8_t *qs, const uint32_t *ds, float *y,
                            int T, int O, int K, mmq_stream_t stream);

/*
 * Decode-shaped q4_K product for 1 <= T <= 16 tokens, where the whole cost is
 * reading W from HBM once.  The pages' per-sub-block form ("31 . r28", 2.3):
 * for every 32-weight sub-block the exact integer dot C_b of the 4-bit
 * quants with the int8 activations, folded in f32 as
 * (dx*(d*sc))*C_b + (dx*ssum)*(-(dmin*m)).  The dots run on the f16 warp MMA
 * with exact integer operands (every product and partial sum is an integer
 * below 2^24); one CTA per 16 weight rows streams the rows' super-blocks
 * through a shared-memory ring.
 * xh: the int8 q8_1 values as f16 [T][K] and ds the scale words [T][K/32],
 * both as written by mmq_quantize_q8_1.  y: f32 [T][O], overwritten.  Result
 * as mmq_gemm_q4K up to f32 summation order; the same on every call.
 * Allocates nothing.
 * Launched with programmatic stream serialisation: the kernel may start
 * while the previous kernel on `stream` is still running and reads the first
 * super-blocks of W before that kernel has completed (xh, ds and y are
 * touched only after it has).  So W must not be written by the kernel
 * launched immediately before on the same stream (weights written by a copy,
 * or by any earlier kernel, are fine).  The same holds for mmq_gemv_q6K.
 * T <= 16 (MMQ_ERR_SHAPE above), other limits as mmq_gemm_q4K.
 */
int mmq_gemv_q4K(const void *w, const uint16_t *xh, const uint32_t *ds, float *y,
                 int T, int O, int K, mmq_stream_t stream);

/*
 * Decode-shaped q4_K product for 1 <= T <= 4 tokens with the q8_1
 * quantisation of the f32 tokens built in: y = mmq_gemm_q4K applied to
 * mmq_quantize_q8_1(x), without the separate quantise launch.  Every CTA
 * quantises the tokens into shared memory with the same arithmetic as
 * mmq_quantize_q8_1 (bit-identical codes, scales and sums), then forms the
 * pages' per-sub-block exact integer dots ("31 . r28", 2.3) with __dp4a on
 * the SIMT cores and folds them in f32 as (dx*(d*sc))*C_b + (dx*ssum)*
 * (-(dmin*m)); one warp per weight row, the rows dealt over the CTAs so that
 * every SM streams the same share of W.  Result as mmq_gemm_q4K up to f32
 * summation order; the same on every call.  Allocates nothing.
 * x: f32 [T][ldx] (ldx >= K, ldx % 4 == 0), finite.  w: as mmq_gemm_q4K.
 * y: f32 [T][O], overwritten.  T <= 4, 256 <= K <= 32768, K % 256 == 0
 * (MMQ_ERR_SHAPE otherwise), O >= 1.
 * Launched with programmatic stream serialisation like mmq_gemv_q4K: W must
 * not be written by the kernel launched immediately before on the same
 * stream; x and y are touched only after that kernel has completed.
 */
int mmq_gemv_q4K_f32(const void *w, const float *x, int64_t ldx, float *y, int T, int O, int K,
                     mmq_stream_t stream);

/*
 * The same for q6_K ("43 . r40", 5: w = d*sc_u*(q-32) on 16-weight
 * sub-blocks; the pages' per-16 fold y += (dx*(d*sc_u))*C16_u with C16_u the
 * exact integer dot of (q - 32) with the int8 activations, __dp4a).  The
 * 210-byte blocks are only 2-byte aligned: every chunk is copied as the
 * 16-byte-aligned window around it, and the bytes of a window past the end
 * of W are read one by one, never beyond it.  w: O*(K/256)*210 bytes; other
 * arguments, limits and launch behaviour as mmq_gemv_q4K_f32.
 */
int mmq_gemv_q6K_f32(const void *w, const float *x, int64_t ldx, float *y, int T, int O, int K,
                     mmq_stream_t stream);

/*
 * Decode-shaped q6_K product for 1 <= T <= 16 tokens ("43 . r40", 5:
 * w = d*sc_u*(q-32) on 16-weight sub-blocks u with signed 8-bit scales): for
 * every sub-block the exact integer dot C16_u of (q-32) with the int8
 * activations, folded in f32 as (dx_b*(d*sc_u))*C16_u, b = u/2 the q8_1
 * block.  The dots run on the f16 warp MMA with exact integer operands; the
 * 210-byte blocks are staged through 16-byte-aligned windows.
 * w: O*(K/256)*210 bytes.  xh, ds: as for mmq_gemv_q4K.  y: f32 [T][O],
 * overwritten.  Result as mmq_gemm_q6K up to f32 summation order; the same on
 * every call.  Allocates nothing.
 * T <= 16 (MMQ_ERR_SHAPE above), other limits as mmq_gemm_q6K.
 */
int mmq_gemv_q6K(const void *w, const uint16_t *xh, const uint32_t *ds, float *y,
                 int T, int O, int K, mmq_stream_t stream);

/*
 * mmq_gemm_q4K_splitk without caller scratch: this entry point allocates
 * nothing.  The partial sums and tile counters live in the library's own
 * statically allocated device arrays, 4 Mi f32 (16 MiB) of partial sums and
 * 8192 tile counters per device.  (The pages have no counterpart: their
 * kernel never splits K.)
 *   - The scratch address is obtained once per device, with that device
 *     current, on the first call for that device that needs scratch (under a
 *     lock: first calls from several host threads are safe).  Make that
 *     first call before any stream capture.  The address belongs to the
 *     device's CUDA context of that moment: after cudaDeviceReset of the
 *     device, do not call this entry point again in the same process.
 *   - Calls with one split (ksplit == 1, or K == 256) need no scratch and
 *     run as mmq_gemm_q4K whatever their size.  Calls whose
 *     mmq_splitk_sizes exceed the scratch return MMQ_ERR_SCRATCH and
 *     launch nothing.
 *   - What must start at zero: the tile counters.  They are zero when the
 *     library is loaded, and every call that launched leaves them at zero
 *     when its kernel ends (a kernel that timed out included).  After a call
 *     whose mmq_check_status is not MMQ_OK, y from that call is undefined
 *     (an aborted split may have skipped its partial sums); the counters
 *     are still valid for the next call.
 *   - The scratch is shared by every call on the device: calls that may
 *     overlap in time (different streams, no ordering between them) race
 *     and give wrong results.  Order them on one stream.
 * Arguments, limits and result as mmq_gemm_q4K_splitk.
 */
int mmq_gemm_q4K_splitk_static(const void *w, const uint16_t *xa, const uint32_t *ds, float *y,
                               int T, int O, int K, int ksplit, mmq_stream_t stream);

/*
 * The same q4_K GEMM in the pages' per-sub-block form: the tensor core forms
 * every 32-weight sub-block's exact integer dot (times its 6-bit scale) in
 * its own TMEM accumulator and the f32 fold dx_b*C'_b runs per sub-block
 * ("31 . r28", 2.3 and 3.2).  xh: the int8 values as f16 (mmq_quantize_q8_1).
 * Same limits and result (up to f32 summation order) as mmq_gemm_q4K.
 */
int mmq_gemm_q4K_subblock(const void *w, const uint16_t *xh, const uint32_t *ds,
                          float *y, int T, int O, int K, mmq_stream_t stream);

/*
 * q6_K x q8_1 GEMM ("43 . r40", 5: w = d*sc_u*(q-32) on 16-weight
 * sub-blocks u):  y[t][o] = sum_k dequant(W)[o][k]*dequant(X)[t][k], i.e.
 * the pages' per-16 fold sum_u dx_(u/2)*(d*sc_u)*C16_u with C16_u the exact
 * integer dot of (q-32) with the int8 activations; accumulation in f32
 * (rounding order unspecified).
 * Production form: the tensor core accumulates each 256-weight super-block
 * from the exact activation planes xa (hi + lo) and the weight values
 * sc*(q-32) as exact f16 hi + lo planes (two MMAs per 16-k step, weight hi
 * and weight lo against both activation planes: every product exact in f32);
 * d is applied per super-block.
 * w: O*(K/256)*210 bytes.  xa: as written by mmq_quantize_q8_1.  ds: not
 * read (q6_K has no min term; may be NULL).  y: f32 [T][O], overwritten.
 * T >= 0, O >= 1, 256 <= K <= 2^20, K % 256 == 0.
 */
int mmq_gemm_q6K(const void *w, const uint16_t *xa, const uint32_t *ds,
                 float *y, int T, int O, int K, mmq_stream_t stream);

/*
 * The same q6_K GEMM in the pages' per-sub-block form: the tensor core forms
 * every 16-weight half's exact integer dot C16_u = sum (q-32)*a (operand xh,
 * the int8 values as f16) in its own TMEM accumulator and the f32 fold
 * dx*(d*sc_u)*C16_u runs per 16-weight half.  Same limits and result (up to
 * f32 summation order) as mmq_gemm_q6K.
 */
int mmq_gemm_q6K_subblock(const void *w, const uint16_t *xh, const uint32_t *ds,
                          float *y, int T, int O, int K, mmq_stream_t stream);

/*
 * q5_K x q8_1 GEMM, the sibling of q4_K in the same k-quant family (the pages
 * run the "q4_K line" and "q6_K line" of one skeleton, "43 . r40", 6; the
 * q5_K bytes are the GGUF layout, a reading): 176-byte super-blocks of 256
 * weights, d and dmin (f16) and the 12 scale/min bytes exactly as q4_K,
 * qh[32] at bytes 16-47, qs[128] at 48-175; weight 32j+i of a super-block
 * has q = (q4_K's nibble of qs for element 32j+i) + 16 * (bit j of qh[i]),
 * 0..31, and w = d*sc_j*q - dmin*m_j.
 * The q4_K fold and the production form of mmq_gemm_q4K (sc*q <= 1953 is
 * exact in f16).  w: O*(K/256)*176 bytes; xa, ds, y, limits as mmq_gemm_q4K.
 * mmq_gemm_q5K_subblock: the pages' per-sub-block form (exact integer dots
 * C_b, f32 fold per 32-weight sub-block) from xh, as mmq_gemm_q4K_subblock.
 */
int mmq_gemm_q5K(const void *w, const uint16_t *xa, const uint32_t *ds,
                 float *y, int T, int O, int K, mmq_stream_t stream);
int mmq_gemm_q5K_subblock(const void *w, const uint16_t *xh, const uint32_t *ds,
                          float *y, int T, int O, int K, mmq_stream_t stream);

/*
 * q8_0 x q8_1 GEMM: 34-byte blocks of 32 weights (f16 d, then 32 int8 values,
 * w = d*q; GGUF's q8_0, a reading), rows of K/32 blocks.  The pages' fold
 * with the weight block's scale in place of d*sc and no min term:
 * y[t][o] = sum_b (dx_b*d_b)*C_b, C_b the exact integer dot of the 32 int8
 * weights with the 32 int8 activations, formed by the tensor core (exact f16
 * operands) per block and folded in f32.  xh, ds: as written by
 * mmq_quantize_q8_1.  w: O*(K/32)*34 bytes, K % 256 == 0; other limits as
 * mmq_gemm_q4K.
 */
int mmq_gemm_q8_0(const void *w, const uint16_t *xh, const uint32_t *ds,
                  float *y, int T, int O, int K, mmq_stream_t stream);

/*
 * Diagnostic: the per-sub-block exact integer dots the GEMMs fold, through
 * the same tensor-core pipeline.  out: int32 [T][O][K/32] for q4_K
 * (C_b = sum q*a over 32 weights) or [T][O][K/16] for q6_K
 * (C16_u = sum (q-32)*a over 16 weights).  Same shape limits as the GEMMs.
 * Meant for small shapes (the output is K/32 or K/16 times larger than y).
 */
int mmq_debug_subdots_q4K(const void *w, const uint16_t *xh, int32_t *out,
                          int T, int O, int K, mmq_stream_t stream);
int mmq_debug_subdots_q6K(const void *w, const uint16_t *xh, int32_t *out,
                          int T, int O, int K, mmq_stream_t stream);
/* The same for q5_K and q8_0: int32 [T][O][K/32]. */
int mmq_debug_subdots_q5K(const void *w, const uint16_t *xh, int32_t *out,
                          int T, int O, int K, mmq_stream_t stream);
int mmq_debug_subdots_q8_0(const void *w, const uint16_t *xh, int32_t *out,
                           int T, int O, int K, mmq_stream_t stream);

/*
 * Paged key-value cache of one layer
 * ----------------------------------
 * Entry `slot` (0-based, in order of arrival) of sequence b lies in page
 * table[b*cols + slot / page_size] at offset slot % page_size:
 *     k element d of head h:  k[page*k_page + h*k_head + offset*k_slot + d]
 * and v likewise with its own strides (in elements; multiples of 8, so that
 * every row of `dim` values starts on 16 bytes).  Pages may be in any order
 * and table entries past a sequence's length may hold anything.  `weight` and
 * `pos` are per entry and head, [pages][heads][page_size], through the same
 * table: the attention weight the entry has received so far, and its
 * position; either may be NULL where the call does not need it.  len[b] is
 * the sequence's number of entries, the new tokens of the running step
 * included: the caller raises it once per step, before the step's first
 * layer, and lowers it after mmq_kv_evict or a rejected draft.
 * A page id outside 0..pages-1 is never followed: nothing is written there,
 * and results that depend on it are unspecified.  A len outside
 * 0..cols*page_size is taken as 0: the sequence's table row is not followed.
 * mmq_check_status reports either as MMQ_ERR_INDEX.
 */
enum { MMQ_F16 = 0, MMQ_BF16 = 1, MMQ_F32 = 2 };

typedef struct mmq_kv_cache {
    void *k, *v;                      /* f16 or bf16 pools                              */
    float *weight;                    /* [pages][heads][page_size] or NULL              */
    int32_t *pos;                     /* [pages][heads][page_size] or NULL              */
    const int32_t *table;             /* [seqs][cols] page ids                          */
    const int32_t *len;               /* [seqs] entries                                 */
    int64_t k_page, k_head, k_slot;   /* strides of k in elements                       */
    int64_t v_page, v_head, v_slot;   /* strides of v in elements                       */
    int64_t pages;                    /* pages in each pool, 1 .. 2^31-1                */
    int dtype;                        /* MMQ_F16 or MMQ_BF16 (k and v)                  */
    int heads;                        /* key-value heads                                */
    int dim;                          /* values per head: a multiple of 8, 8 .. 256     */
    int page_size;                    /* entries per page, >= 1                         */
    int seqs;                         /* sequences, 0 .. 65535                          */
    int cols;                         /* pages per table row; cols*page_size <= 2^30    */
} mmq_kv_cache;

/*
 * Rotary positions, and the append of the new tokens' keys and values.
 * Rows i = b*new_tokens + t, t < new_tokens, of q [.][q_heads][dim], k and v
 * [.][heads][dim] are f32, ldq/ldk/ldv floats apart (multiples of 4), as the
 * projections leave them.  Of every q and k head the first `rot` values (even,
 * 2..dim) are rotated in rot/2 pairs, the rest passes through; pair i is
 * (i, i + rot/2), or (2i, 2i+1) with interleaved != 0:
 *     (a, b) -> magnitude * (a cos - b sin, a sin + b cos),
 *     angle of pair i at position x = 2 pi frac(x * freq[i] / 2^64).
 * freq [rot/2] holds turns per position as 64-bit fractions: the product
 * wraps exactly, so the angle is as good at position 2^30 as at 0, and a
 * scaling for long contexts is a change of the table (ops.rope_table).
 * pos [seqs*new_tokens] int32.  q_out [.][q_heads][dim], rows ldo floats
 * apart, may be q itself (ldo == ldq).  new_len [seqs] (NULL: new_tokens
 * each) says how many of a sequence's rows are there: row t < new_len[b] goes
 * to slot len[b] - new_len[b] + t of every head, rounded to the cache's type
 * (nearest even); a row past it gets q_out = 0 and is not stored.  Where the
 * cache has them, `weight` of a new entry is set to 0 and `pos` to the row's
 * position.  Slots must not repeat within a call.  A new_len outside
 * 0..new_tokens is limited to it, here and in mmq_attn_decode, and a row whose
 * slot would be negative is not stored; both report MMQ_ERR_INDEX.
 */
int mmq_rope_append(const mmq_kv_cache *cache, const int64_t *freq, int rot, float magnitude,
                    int interleaved, const float *q, int64_t ldq, const float *k, int64_t ldk,
                    const float *v, int64_t ldv, const int32_t *pos, const int32_t *new_len,
                    float *q_out, int64_t ldo, int q_heads, int new_tokens, mmq_stream_t stream);

/*
 * Attention of the newest tokens over the cache (decode, or drafted tokens
 * scored together).  q rows as above (rotated), q head j reads key-value head
 * j / (q_heads/heads); row t < new_len[b] (NULL: new_tokens) of sequence b
 * sees the slots below len[b] - new_len[b] + t + 1:
 *     s = scale * q.k,  p = exp(s - max) / sum,  out = sum p v
 * out [seqs*new_tokens][q_heads][dim] f32, contiguous, not q.  A row that sees no
 * slot, or with t >= new_len[b], gets 0.  What a row does not see has no
 * influence on it, whatever it holds (stale NaN or Inf included).  Statistics
 * and sums are f32.  q and p enter the tensor core as sums of two f16 parts (22
 * bits of the row's largest |q|, and of the row's largest p) or three bf16 parts
 * (24 bits); against 64 bits the output is off by 3e-7 to 1e-6 of its norm, as
 * an f32 computation is.  Results do not depend on timing: they repeat bit for bit.
 * accumulate != 0 adds to cache->weight, for every entry a sequence has, the
 * sum of p over its rows and the query heads of the key-value head.  Rows of
 * drafted tokens add theirs like any other, and a shorter len does not take
 * that back: attend drafts without accumulating, and once it is known how many
 * stay, call again with the same q, len lowered, new_len = the rows that stay,
 * and accumulate.  What rows that are not finite add is unspecified.  Sequences
 * may share pages (a common beginning), but not then: two of them would add to
 * the same weight at the same time.  An entry that is not finite makes the
 * rows that see it not finite.
 * 1 <= new_tokens <= 16, q_heads a multiple (1 .. 128) of heads, scale finite.
 * Refused too (MMQ_ERR_SHAPE, by both calls) are caches of more than 2^31-1
 * tiles (32 to 128 entries of a sequence's cols*page_size, for each head), and
 * more than 2^31-1 of seqs * heads * (rows per key-value head, plus one per
 * 1024 of cols*page_size if weights are accumulated).
 * `work` holds the floats that mmq_attn_sizes says: the parts of split rows (a
 * few MB whatever the lengths), and with accumulate a score for each of seqs *
 * q_heads * new_tokens rows and cols*page_size slots besides.  Calls that share
 * it must be ordered (one stream).
 */
int mmq_attn_sizes(const mmq_kv_cache *cache, int q_heads, int new_tokens, int accumulate,
                   int64_t *work_floats);
int mmq_attn_decode(const mmq_kv_cache *cache, const float *q, int64_t ldq, const int32_t *new_len,
                    float *out, int q_heads, int new_tokens, float scale, int accumulate,
                    float *work, mmq_stream_t stream);

/*
 * mmq_rope_append with a norm of every q and k head before the rotation, and
 * positions with several axes:
 *     y = x * rsqrt(mean of x^2 over the head + eps) * w,
 * w = q_norm or k_norm, f32 [dim] (NULL: that side is rotated as it is; a
 * model that keeps w - 1 adds the 1).  Pair i turns by the row's position on
 * axis[i] (int32 [rot/2], 0..axes-1; NULL with one axis): pos int32
 * [axes][seqs*new_tokens], of which axis 0 goes to the cache's `pos`.  An axis
 * outside 0..axes-1 counts as 0 and is reported as MMQ_ERR_INDEX.  The
 * squares are added in f32: a head whose values pass 10^18 may become 0.
 * q_out is f32 or the cache's type (q_dtype), rounded once, rows ldo values
 * apart (multiples of 4, or of 8); it may be q itself where it is f32 and
 * ldo == ldq.  Everything else, ragged counts and reported errors among it, is
 * as in mmq_rope_append.  1 <= axes <= 8, eps >= 0.
 */
int mmq_norm_rope_append(const mmq_kv_cache *cache, const int64_t *freq, const int32_t *axis, int rot, float magnitude,
                         int interleaved, const float *q_norm, const float *k_norm, float eps, const float *q, int64_t ldq,
                         const float *k, int64_t ldk, const float *v, int64_t ldv, const int32_t *pos, int axes,
                         const int32_t *new_len, void *q_out, int64_t ldo, int q_dtype, int q_heads, int new_tokens,
                         mmq_stream_t stream);

/*
 * Attention of any number of new tokens over the cache: prompts, chunks of
 * them, and single tokens of models whose scores are capped or biased.  q is
 * of the cache's type, rows [seqs*new_tokens][q_heads][dim], ldq values apart
 * (a multiple of 8); q head j reads key-value head j / (q_heads/heads).  Row t
 * < new_len[b] (NULL: new_tokens) of sequence b stands at slot i = len[b] -
 * new_len[b] + t and sees the slots lo <= j < hi,
 *     hi = i + 1, or prefix[b] where that is more (limited to len[b]): the
 *          first prefix[b] slots see one another whole (NULL: none do);
 *     lo = max(0, i - window + 1) (window 0: 0), or first[row] where that is
 *          more (int32 [seqs*new_tokens]: where the row's document begins;
 *          NULL: 0):
 *     s = scale q.k;  cap > 0: s = cap tanh(s / cap);
 *     slopes (f32 [q_heads], or NULL): s += slopes[head] (j - i);
 *     p = exp(s - max) / sum,  out = sum p v
 * out [seqs*new_tokens][q_heads][dim], contiguous, not q, is f32 or of the
 * cache's type.  A row that sees nothing, or with t >= new_len[b], gets 0.  What
 * a row does not see has no influence on it, whatever it holds (NaN or Inf
 * included); a row that sees a V entry which is not finite, or a score that is
 * NaN or +Inf, is not finite.  Scores, maxima and sums are f32; p enters the
 * tensor core rounded to the cache's type (11 or 8 bits), and an f32 `out` is
 * not rounded besides.  Sums of p v are not divided before their end, with p up
 * to 2^8 (bf16) or 2^15 (f16): bf16 values past 2^119 over the number of entries
 * may overflow f32.  Results do not depend on timing.  Nothing is added to
 * cache->weight (mmq_attn_decode can): a prompt's entries keep the weight 0 that
 * their append gave them, and mmq_kv_evict ranks them by that.
 * new_tokens >= 1, q_heads a multiple (1 .. 128) of heads, scale * log2(e)
 * finite, 0 <= cap <= 1024, window >= 0.  A len outside 0..cols*page_size counts as 0, a
 * new_len outside 0..new_tokens is limited to it, one above len counts as 0;
 * all are reported as MMQ_ERR_INDEX.  Sequences may share pages.  Refused too
 * (MMQ_ERR_SHAPE, by both calls) are more than 2^31-1 tiles: cols*page_size /
 * 128 (64 for heads above 128) for each key-value head and 128 rows of it.
 * `work` holds the floats that mmq_prefill_sizes says (at most some 80 MB).
 * Calls that share it must be ordered (one stream).
 */
int mmq_prefill_sizes(const mmq_kv_cache *cache, int q_heads, int new_tokens, int64_t *work_floats);
int mmq_attn_prefill(const mmq_kv_cache *cache, const void *q, int64_t ldq, const int32_t *new_len, const int32_t *prefix,
                     const int32_t *first, const float *slopes, void *out, int out_dtype, int q_heads, int new_tokens,
                     float scale, float cap, int window, float *work, mmq_stream_t stream);

/*
 * Attention of a tree of drafted tokens.  The new_len[b] (NULL: new_tokens)
 * last entries of a sequence are the tree's nodes; row t sees every slot
 * before them from first[row] on (NULL: all), and of the nodes those whose bit
 * is set in tree[b*new_tokens + t] (bit j: node j; its own bit too, if it is
 * to see itself) and that lie at or after first[row].  Bits past the sequence's
 * nodes are ignored.  Everything else is as in mmq_attn_prefill, `work` among
 * it (mmq_prefill_sizes).  new_tokens <= 64.
 */
int mmq_attn_tree(const mmq_kv_cache *cache, const void *q, int64_t ldq, const uint64_t *tree, const int32_t *new_len,
                  const int32_t *first, void *out, int out_dtype, int q_heads, int new_tokens, float scale, float cap,
                  float *work, mmq_stream_t stream);

/*
 * What stays of a tree: of the last n = new_len[b] (NULL: nodes) entries of
 * sequence b, entry keep[b*width + i] moves to place i of them, for i <
 * count[b] (NULL: width), in every head, with its weight and position where
 * the cache has them.  keep is ascending; an index that is not, or not below n,
 * leaves its place as it was and is reported as MMQ_ERR_INDEX, as are a count
 * outside 0..width and a new_len outside 0..nodes, which are limited to that.
 * cache->len is not changed: the caller lowers it by n - count[b] once all
 * layers are done.  A sequence of fewer than n entries is left as it is and
 * reported.  The pages of the last n entries must not be shared.
 * 0 <= width <= nodes <= 64; keep int32 [seqs][width].
 */
int mmq_kv_keep(const mmq_kv_cache *cache, const int32_t *keep, const int32_t *count, const int32_t *new_len, int width,
                int nodes, mmq_stream_t stream);

/*
 * Eviction: every sequence with more than `budget` entries is cut down to
 * `budget` for each head by itself.  Entries with pos >= keep_from[b] rank
 * first, the others by `weight`; the first `budget` stay, ties going to the
 * lower slot.  Those that stay in a slot past the budget move, in order of
 * their slots, into the slots below it that became free, in order: nothing
 * else moves, and the order of slots is not the order of positions any more
 * (the attention does not need it: keys carry their rotation).  k and v move
 * in place; the bookkeeping of slots 0 .. min(len, budget)-1 is written to
 * weight_out and pos_out (the layout of weight and pos, no overlap with
 * them), which the caller uses from then on, so that a call leaves `weight`
 * and `pos` as they were.  Slots past that keep what they held.  Weights must
 * not be NaN.  cache->len is not changed: the caller lowers it to the budget
 * once all layers are done.  The pages of a sequence's first `budget` slots
 * must not be shared with another.
 * cols*page_size <= 262144, seqs*heads <= 268435455.  `work` holds
 * mmq_evict_sizes' count of ints.
 */
int mmq_evict_sizes(const mmq_kv_cache *cache, int budget, int64_t *work_ints);
int mmq_kv_evict(const mmq_kv_cache *cache, int budget, const int32_t *keep_from, float *weight_out,
                 int32_t *pos_out, int32_t *work, mmq_stream_t stream);

/*
 * Verification of drafted tokens (speculative sampling).  target
 * [seqs][drafts+1][vocab] and draft [seqs][drafts][vocab] are probabilities
 * of one type (MMQ_F16, MMQ_BF16 or MMQ_F32), contiguous; draft NULL means
 * drafts that were not sampled (probability 1 for the drafted token).
 * tokens [seqs][drafts]; uniform [seqs][drafts+1] in [0, 1); count [seqs]
 * (NULL: drafts each) the number of tokens drafted.  Draft i is accepted
 * while  uniform[i] * draft_i(x) < target_i(x)  (f32, rounded once).  At the
 * first draft a that is not, the token a is drawn from max(target_a -
 * draft_a, 0); with all accepted, from target_count.  The drawing is exact in
 * whole numbers, so it does not depend on the order of any sum: with
 * w_j = round(2^40 max(p_j - q_j, 0)) (nearest even; the difference in f32,
 * limited to 1), W their sum and u = floor(2^24 uniform[drafts]), the token is
 * the lowest j with w_0 + ... + w_j > floor(W u / 2^24).  If W = 0 (the two
 * agree), the target alone is drawn from; if that is 0 too, the token is 0.
 * out [seqs][drafts+1] gets the accepted tokens, the drawn one, then -1;
 * accepted [seqs] how many drafts were accepted.  A drafted token outside
 * 0..vocab-1 is not accepted, and then the target alone is drawn from; a
 * count outside 0..drafts is limited to it; both report MMQ_ERR_INDEX.
 * 0 <= seqs <= 65535, 1 <= drafts <= 64, 1 <= vocab <= 2^20.
 */
int mmq_spec_verify(const void *target, const void *draft, int dtype, const int32_t *tokens,
                    const float *uniform, const int32_t *count, int32_t *out, int32_t *accepted,
                    int seqs, int drafts, int vocab, mmq_stream_t stream);

/*
 * Diagnostic: measured warp-level tensor throughput of the current device,
 * in TMAC/s (10^12 multiply-accumulates per second), for kind 0 = int8
 * (mma.sync m16n8k32 s8*s8->s32, the only int8 tensor path on sm_103a) or
 * kind 1 = f16 (mma.sync m16n8k16, f32 accumulate).  Synchronous: runs a
 * few hundred microseconds of probe kernels on `stream` and waits for them.
 * The reported figure is the denominator of "fraction of int8 peak".
 */
int mmq_probe_tensor_peak(int kind, double *tmacs, mmq_stream_t stream);

/*
 * Waits for `stream`, then reports and clears a device status word of the
 * library for the current device: MMQ_OK, MMQ_ERR_TIMEOUT (a kernel's pipeline
 * wait ran past its limit; the kernel stopped early and its output is
 * invalid), MMQ_ERR_INDEX (an operator around the cache read an index that is
 * out of range) or MMQ_ERR_CUDA (the stream reported a CUDA error).  If
 * `detail` is non-NULL it receives 4 ints: code, kernel id, site (a wait, or
 * for MMQ_ERR_INDEX 1 = length, 2 = page id, 3 = count, 4 = token, 5 = axis,
 * 6 = node), linear block index of the first failure.
 * The products, the decode-side operators, and those for prompts and trees have
 * a word each, and a call reports one, in this order: where several hold an
 * error, the next call reports the next, so call until MMQ_OK to have all.
 */
int mmq_check_status(mmq_stream_t stream, int *detail);

/*
 * Test-only: exercises the bounded pipeline waits (the pages' launcher never
 * runs over its limits silently, "31 . r28", 3.3 Pitfalls; the waits and
 * this knob are the library's own).  Sets, for the current device, the time a
 * kernel's pipeline wait may take before it gives up (wait_limit_us > 0; <= 0
 * restores the default of 2 s) and a mode: 0 = off; 1 = the production q4_K
 * kernels (mmq_gemm_q4K, mmq_gemm_q4K_splitk*, mmq_gemm_q5K) withhold the raw
 * weight copy of their second super-block (K >= 512), and prompt and tree
 * attention (mmq_attn_prefill, mmq_attn_tree) the last tile of K of every run
 * of tiles that a CTA takes, so the waits for it run
 * out: the kernel records MMQ_ERR_TIMEOUT (see mmq_check_status), stops every
 * role, drains the work it issued, frees its tensor memory and returns; its
 * output is undefined.  (Captured launches of the two attentions keep the mode
 * they were captured under.)  Synchronous with respect to the host.  Returns MMQ_OK,
 * MMQ_ERR_SHAPE (unknown mode) or MMQ_ERR_CUDA.  Leave it at mode 0 outside
 * tests.
 */
int mmq_debug_fault_inject(int mode, int wait_limit_us);

/*
 * More detail on the last failure that mmq_check_status reported (no
 * counterpart on the pages; a diagnostic of the library's own bounded waits): info
 * receives 4 ints: the time the failed wait had waited (microseconds), its
 * poll count, the phase parity it waited for and the waited barrier's
 * shared-memory address.  All zero if no failure was reported yet.  Returns
 * MMQ_OK, or MMQ_ERR_NULL for a NULL `info`.
 */
int mmq_last_failure_info(int *info);

#ifdef __cplusplus
}
#endif

#endif /* MMQ_H */
