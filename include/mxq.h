/*
 * mxq.h -- C ABI of the mxq block-quantization library for AMD Instinct MI355X
 * (gfx950).
 *
 * These entry points quantize BF16 activations on the GPU:
 *   mxq_quant_fp8_1x128        FP8 E4M3 with one FP32 scale per 1x128 group
 *   mxq_quant_fp8_blockwise    the same row-wise and/or 128x1 column-wise on the
 *                              transpose, optionally with UE8M0 (power-of-two) scales
 *   mxq_hadamard_quant_fp8_ex  the DSA rotate + FP8 with UE8M0 and scale layouts
 *   mxq_swiglu_quant_fp8       FP32 SiLU(gate) * up -> FP8 1x128 (no BF16 round)
 *   mxq_hadamard_quant_fp8     cat[qk_pe, qk_nope] -> normalized 128-point
 *                              Walsh-Hadamard rotation -> FP8 1x128
 *   mxq_hadamard_quant_nvfp4   the same rotation -> NVFP4 row-wise (1x16 blocks,
 *                              one FP32 tensor scale, measured or supplied)
 *   mxq_group_rht_quant_nvfp4  grouped (MoE split sections) NVFP4, row-wise and
 *                              column-wise after a 16-point random-sign Hadamard
 *                              transform, optionally with an FP8 1x128 row-wise
 *                              output in the same call
 * and serve attention from a KV cache held in NVFP4:
 *   mxq_add_rmsnorm_quant_fp8  residual addition + RMS norm -> FP8 1x128 (the
 *                              quantized input of a projection)
 *   mxq_rope_append_nvfp4      rotary positions on Q and K, then K and V into a paged
 *                              NVFP4 cache
 *   mxq_attention_nvfp4        causal attention of ragged queries over that cache
 *   mxq_attention_prefix_nvfp4 the same where groups of sequences share long prefixes
 *   mxq_page_keys_nvfp4        the mean key of every page that an append has filled
 *   mxq_select_pages_nvfp4     the pages each query attends, by the scores of their mean keys
 *   mxq_attention_pages_nvfp4  causal attention over listed pages alone
 *
 * Conventions shared by every entry point
 *  - Pointers named *_bf16 / codes / scales / workspace are DEVICE pointers; the
 *    caller owns every buffer.  split_sections, mxq_sr and its offset arrays are
 *    HOST memory, read during the call only (their values are baked into the
 *    kernel arguments, so under stream capture the capture-time values are used).
 *  - `stream` is a hipStream_t (NULL = the default stream).  Calls are
 *    asynchronous: MXQ_OK means the work was enqueued.
 *  - The library never allocates, frees, memsets, synchronizes or reads the
 *    environment; it keeps no global state (the per-device scratch array of
 *    mxq_group_rht_quant_nvfp4_noalloc aside) and is re-entrant.  Calls in flight
 *    at the same time need distinct workspaces.
 *  - All argument checks run on the host before anything is enqueued; on an error
 *    nothing is launched and no output is touched.  A failed launch returns
 *    MXQ_ERR_HIP (outputs are then undefined).  There is no fallback path: an
 *    unsupported request is an error, never a slower substitute.
 *  - Arithmetic is IEEE binary32 with one rounding per operation in the order
 *    stated below; every output is bit-exact with respect to that definition, but
 *    for those of the mxq_attention_* calls, whose roundings are stated with
 *    mxq_attention_nvfp4.
 *
 * Sources of the operations (page, then section):
 *  - onnxruntime PR #33644, QMoE dynamic FP8 activation quantization,
 *    Description: K128 groups; scale = max(amax, 1e-10) * float32(1/448); FP32
 *    normalization by division; saturating nearest-even E4M3FN.
 *  - TensorRT-LLM PR #15158, "Add rotate_activation to DSA fused_cat_fp8 path",
 *    Summary: cat[qk_pe, qk_nope] -> rotate_activation -> fp8_quantize_1x128;
 *    the discussion's (Hq).(Hk) = q.k for the orthonormal rotation.
 *  - TransformerEngine PR #2564, "[NVFP4][MOE] Bug Fix for NVFP4 Grouped Quant",
 *    Greptile summary and sequence diagram: grouped row-wise + column-wise
 *    (RHT) NVFP4 cast with a caller-provided workspace, no allocation per call;
 *    review thread: a workspace-size query.
 *  - TransformerEngine PR #2555, review comments on cast.cpp and quantizer.cpp:
 *    split_section % 128 == 0; RHT on the column-wise (transposed) operand only;
 *    row-wise-only requests skip the RHT work; a separate column-wise RNG state;
 *    deterministic RNG offsets rather than sequential generator advancement.
 */
#ifndef MXQ_H
#define MXQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MXQ_OK = 0,
    MXQ_ERR_INVALID_ARGUMENT = 1,    /* NULL pointer, negative size, bad flags ...   */
    MXQ_ERR_MISALIGNED = 2,          /* k or a section not a multiple of 128, or a  */
                                     /* pointer / stride not 16-byte aligned        */
    MXQ_ERR_WORKSPACE_TOO_SMALL = 3, /* workspace_bytes < the size query's value    */
    MXQ_ERR_UNSUPPORTED = 4,         /* outside the supported profile (limits)      */
    MXQ_ERR_HIP = 5                  /* a HIP launch failed                          */
} mxq_status;

/* Static string naming the status; never NULL. */
const char* mxq_status_string(mxq_status s);

/* Library version string, e.g. "mxq 0.1.0 gfx950". */
const char* mxq_version(void);

/* Limits of the supported profile. */
#define MXQ_ROW_ALIGN 128          /* rows per section and k: multiples of this   */
#define MXQ_MAX_SECTIONS 256       /* split sections per grouped call             */
/* Every array a call addresses spans fewer than MXQ_MAX_EXTENT elements: rows of
 * length n at stride ld span (rows - 1) * ld + n, and a scale array addressed as
 * r * s_r + c * s_c reaches index (rows - 1) * s_r + (cols - 1) * s_c.  Larger
 * extents give MXQ_ERR_UNSUPPORTED before anything is enqueued. */
#define MXQ_MAX_EXTENT (1LL << 40)

/* ---------------------------------------------------------------------------
 * FP8 E4M3 (OCP E4M3FN), one FP32 scale per 1x128 group along k.
 * onnxruntime PR #33644, Description: the QMoE dynamic activation quantizer's
 * K128 groups, its scale max(amax, 1e-10) * float32(1/448), the FP32 division of
 * each element by its group's scale and the saturating nearest-even E4M3FN encode;
 * the one-ulp differences at E4M3 midpoints it reports are why the division is
 * exact IEEE here, never a reciprocal multiply.
 *
 *   x_bf16   [m][ldx] BF16 bit patterns, row-major, ldx >= k
 *   q_e4m3   [m][ldq] E4M3 codes, ldq >= k
 *   scales   scales[r * scale_stride_row + g * scale_stride_group] for group g of
 *            row r; ({k/128, 1} is [m][k/128]; {1, m} is the transposed [k/128][m])
 *
 * For each group G of 128 consecutive elements of a row:
 *   a = max |x| over G (NaN ignored; 0 if none),  s = fl(max(a, F(1e-10)) * F(1/448)),
 *   q_i = E4M3(fl(x_i / s))   (IEEE division, nearest-even, saturating at 448;
 *                               a NaN element gives 0x7F).
 * Requirements: k % 128 == 0; ldx, ldq multiples of 8 and 16; x, q 16-byte
 * aligned; scales 4-byte aligned.  m == 0 is a successful no-op.
 * ------------------------------------------------------------------------- */
mxq_status mxq_quant_fp8_1x128(const uint16_t* x_bf16, int64_t m, int64_t k, int64_t ldx,
                               uint8_t* q_e4m3, int64_t ldq,
                               float* scales, int64_t scale_stride_row, int64_t scale_stride_group,
                               void* stream);

/* ---------------------------------------------------------------------------
 * FP8 block variants (consumer-facing layouts of the same recipe).
 * TensorRT-LLM PR #15158, review of the DSA scale normalization: a use_ue8m0 option
 * of fp8_quantize_1x128_sf_transpose, and the 1-D scale tensor padded, reshaped and
 * transposed for its consumer.  The recipe is mxq_quant_fp8_1x128's.
 *
 * MXQ_FP8_UE8M0: every scale s = fl(max(a, F(1e-10)) * F(1/448)) is rounded up to
 * the nearest power of two (stored as that FP32 power of two: its UE8M0 byte is the
 * FP32 exponent field, bits >> 23); the codes are E4M3(x / s), exact divisions, and
 * |x| / s stays <= 448.
 * ------------------------------------------------------------------------- */
enum { MXQ_FP8_UE8M0 = 1u };

typedef struct {
    uint8_t* codes;             /* row-wise: [m][ld];  column-wise: [k][ld], row c = column c of x */
    int64_t  ld;
    float*   scales;            /* row-wise: (row r, group g) at r * scale_stride_a + g * scale_stride_b;
                                   column-wise: (column c, row block b) at c * scale_stride_a + b * scale_stride_b */
    int64_t  scale_stride_a;
    int64_t  scale_stride_b;
} mxq_fp8_block_out;

/* Row-wise 1x128 groups and/or column-wise 128x1 blocks (rows 128b .. min(128b+128,
 * m)-1 of column c, a ragged last block when m % 128 != 0; its codes go to row c of the
 * transposed output), from one read of x.  rowwise / columnwise may be NULL (not both).
 * Requirements: k % 128 == 0; ldx % 8 == 0; ld >= k (row-wise) or >= m (column-wise),
 * a multiple of 16; x and codes 16-byte aligned, scales 4-byte aligned; options in
 * {0, MXQ_FP8_UE8M0}.  m == 0 is a successful no-op. */
mxq_status mxq_quant_fp8_blockwise(const uint16_t* x_bf16, int64_t m, int64_t k, int64_t ldx, uint32_t options,
                                   const mxq_fp8_block_out* rowwise, const mxq_fp8_block_out* columnwise,
                                   void* stream);

/* mxq_hadamard_quant_fp8 with options and a (token, head) scale layout: row r is
 * token r / heads, head r % heads (heads >= 1), and its scale goes to
 * scales[token * scale_stride_token + head * scale_stride_head]: {heads, 1} is the
 * plain [tokens][heads] order, {1, T} the transposed [heads][T] one with T >= tokens
 * (rows T past the tokens are padding the call leaves untouched). */
mxq_status mxq_hadamard_quant_fp8_ex(const uint16_t* pe, int64_t ld_pe, int32_t d_pe,
                                     const uint16_t* nope, int64_t ld_nope, int64_t m, uint32_t options,
                                     int64_t heads, uint8_t* q_e4m3, float* scales,
                                     int64_t scale_stride_token, int64_t scale_stride_head, void* stream);

/* ---------------------------------------------------------------------------
 * SwiGLU -> FP8 1x128: the second dynamic quantizer of a W8A8 MoE, directly after
 * the FP32 SiLU/SwiGLU of the gate and up projections (onnxruntime PR #33644,
 * Description: no round to the input type between SwiGLU and the quantizer; the
 * same FP8 recipe as mxq_quant_fp8_1x128).  For each element:
 *   h = fl(SILU(gate) * up),  SILU(g) = fl(g / fl(1 + EXP(-g)))   (all FP32)
 * and then, per group G of 128 consecutive h of a row, exactly as
 * mxq_quant_fp8_1x128 (a = max |h| without NaNs, s = fl(max(a, F(1e-10)) * F(1/448)),
 * q = E4M3(fl(h / s)), 0x7F for a NaN).  EXP(x) is e^x by a stated binary32
 * algorithm (the pages do not fix one): NaN kept; x clamped to [-128, 128];
 * k = rint(fl(x * F(log2 e))); r = fma(-k, 0.693145751953125, x);
 * r = fma(-k, F(ln 2 - 0.693145751953125), r); p = the degree-7 Taylor polynomial of
 * e^r with coefficients F(1/n!) by Horner's rule with fma; EXP = fl(fl(p * 2^k1) * 2^k2),
 * k1 = floor(k/2), k2 = k - k1.  Inputs whose product overflows FP32 are out of
 * contract (as are infinite inputs).
 *
 *   gate_bf16 [m][ld_gate], up_bf16 [m][ld_up] BF16 (separate buffers, or the two
 *             halves of one [m][2n] buffer with up = gate + n)
 *   q_e4m3    [m][ldq] E4M3 codes; scales as mxq_quant_fp8_1x128 (row / group strides)
 * Requirements: n % 128 == 0; ld_gate, ld_up multiples of 8, ldq of 16; gate, up,
 * q 16-byte aligned; scales 4-byte aligned.  m == 0 is a successful no-op.
 * ------------------------------------------------------------------------- */
mxq_status mxq_swiglu_quant_fp8(const uint16_t* gate_bf16, int64_t ld_gate, const uint16_t* up_bf16, int64_t ld_up,
                                int64_t m, int64_t n, uint8_t* q_e4m3, int64_t ldq,
                                float* scales, int64_t scale_stride_row, int64_t scale_stride_group, void* stream);

/* ---------------------------------------------------------------------------
 * DSA-indexer rotate + quantize.  TensorRT-LLM PR #15158, Summary: the indexer
 * concatenates qk_pe and qk_nope, applies rotate_activation (the normalized
 * 128-point Hadamard transform) and then fp8_quantize_1x128; the discussion's
 * (Hq).(Hk) = q.k is why the rotation changes no attention score.  For each row r:
 *   v = cat(pe[r][0:d_pe], nope[r][0:128-d_pe])           (qk_pe first)
 *   y = BF16(fl(WHT_128(v) * F(1/sqrt(128))))            (Sylvester order, butterfly
 *        stages h = 1, 2, 4, ..., 64; (v_i, v_i+h) <- (v_i + v_i+h, v_i - v_i+h))
 *   q[r][:], scales[r] = FP8 1x128 of y (as mxq_quant_fp8_1x128).
 *
 *   pe    [m][ld_pe]   BF16, d_pe in {0, 8, 16, ..., 128}; may be NULL if d_pe == 0
 *   nope  [m][ld_nope] BF16; may be NULL if d_pe == 128
 *   q     [m][128] E4M3 codes;  scales [m] FP32
 * Requirements: ld_pe, ld_nope multiples of 8; pointers 16-byte aligned.
 * ------------------------------------------------------------------------- */
mxq_status mxq_hadamard_quant_fp8(const uint16_t* pe, int64_t ld_pe, int32_t d_pe,
                                  const uint16_t* nope, int64_t ld_nope, int64_t m,
                                  uint8_t* q_e4m3, float* scales, void* stream);

/* ---------------------------------------------------------------------------
 * DSA-indexer rotate + NVFP4 (row-wise 1x16).  The FP4 counterpart of the call
 * above: TensorRT-LLM PR #15158 (Summary) names the FP4 path's missing rotation and
 * its need for a standalone FP4 quantize-only kernel.  For each row r:
 *   y = BF16(fl(WHT_128(cat(pe[r][0:d_pe], nope[r][0:128-d_pe])) * F(1/sqrt(128))))
 *   (as mxq_hadamard_quant_fp8), then the row-wise NVFP4 encode of
 *   mxq_group_rht_quant_nvfp4 with ONE tensor scale for the whole call:
 *   g = fl(max(A, F(1e-10)) * F(1/2688)), A = max |y| over every row (NaN ignored)
 *   or *amax_in; per 1x16 block t = fl(fl(a * F(1/6)) / g), sc = E4M3(t),
 *   d = fl(E4M3(sc) * g), codes E2M1(fl(y / d)) (nearest-even, saturating); a block
 *   of a row holding a NaN gets scale 0x7F and zero codes.
 *
 *   pe, nope, d_pe, ld_pe, ld_nope: as mxq_hadamard_quant_fp8
 *   amax_in       device float[1], or NULL: measure A (two passes over the input)
 *   amax_out      device float[1], or NULL: the measured A of this call (0 for m = 0)
 *   codes         device [m][64]: codes of y[r][2i] (low nibble) and y[r][2i+1]
 *   block_scales  device [m][8] E4M3
 *   global_scale  device float[1]: g (also written for m = 0: the floor scale, or
 *                 the scale of *amax_in)
 *   workspace     device memory of mxq_hadamard_quant_nvfp4_workspace_size(m)
 *                 bytes (2 KB of scale table and 4 bytes per 64 rows, rounded up
 *                 to 256), 256-byte aligned; any contents (the call's kernels meet
 *                 through it in stream order and keep nothing in it between
 *                 calls).  Calls that share it must be ordered.  May be NULL when
 *                 m = 0.
 * Requirements: as mxq_hadamard_quant_fp8; codes and block_scales 16-byte aligned,
 * global_scale, amax_in, amax_out 4-byte aligned; m <= 2^31 - 128.  Errors are
 * returned before anything is enqueued.
 * ------------------------------------------------------------------------- */
size_t mxq_hadamard_quant_nvfp4_workspace_size(int64_t m);

mxq_status mxq_hadamard_quant_nvfp4(const uint16_t* pe, int64_t ld_pe, int32_t d_pe,
                                    const uint16_t* nope, int64_t ld_nope, int64_t m,
                                    const float* amax_in, float* amax_out,
                                    uint8_t* codes, uint8_t* block_scales, float* global_scale,
                                    void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Grouped NVFP4 quantization with a 16-point random Hadamard transform (RHT) on
 * the column-wise operand.  TransformerEngine PR #2564, Greptile summary and
 * sequence diagram: the grouped row-wise + column-wise RHT cast over MoE split
 * sections with a caller-provided workspace and no allocation per call (review
 * thread: the workspace-size query); PR #2555, review comments on cast.cpp and
 * quantizer.cpp: split sections in multiples of 128, the RHT on the column-wise
 * (transposed) operand only, its BF16 intermediate, and a separate column-wise RNG
 * with deterministic per-call offsets for stochastic rounding.
 *
 * x_bf16 is [total_rows][k] BF16 (row stride k), total_rows = sum(split_sections).
 * Section s covers rows [R_s, R_s + m_s), m_s = split_sections[s] (m_s may be 0).
 *
 * flags (any non-empty combination):
 *   MXQ_ROWWISE      NVFP4 of x along k:
 *                      codes  [total_rows][k/2]   (2 E2M1 codes per byte, even
 *                                                  element in the low nibble)
 *                      block_scales [total_rows][k/16] E4M3
 *                      global_scales[num_sections] FP32
 *   MXQ_COLUMNWISE   NVFP4 of the transposed, rotated operand: for each 16-row block
 *                    b of a section and each column c the values
 *                      Y[c][16b + t] = BF16(fl(0.25 * (H16 D x[16b + 0..15][c]))_t)
 *                    (D = diag of signs from rht_sign_mask, bit t set = negate row
 *                    16b + t; H16 Sylvester; butterfly stages h = 1, 2, 4, 8).
 *                    Section s's outputs: codes at byte offset k*R_s/2 as [k][m_s/2],
 *                    block_scales at byte offset k*R_s/16 as [k][m_s/16];
 *                    global_scales[num_sections] FP32.
 *   MXQ_FP8_ROWWISE  FP8 1x128 of x (as mxq_quant_fp8_1x128): codes [total_rows][k],
 *                    scales [total_rows][k/128].
 *
 * NVFP4 encoding of one direction of section s (values v = x or Y):
 *   A = max |v| over the section (NaN ignored);  g = fl(max(A, F(1e-10)) * F(1/2688))
 *   (stored in global_scales; an empty section stores fl(F(1e-10) * F(1/2688))).
 *   Per 1x16 block: if it holds a NaN, scale 0x7F and codes 0; else
 *   a = max |v|, t = fl(fl(a * F(1/6)) / g), sc = E4M3(t); if sc == 0, codes 0;
 *   else d = fl(E4M3value(sc) * g) and code_i = E2M1(fl(v_i / d)) (nearest-even,
 *   saturating at 6) or, with stochastic rounding, the grid neighbour above with
 *   probability floor(256 f)/256 via 8 Philox bits per element.
 *   Dequantization: E2M1value(code) * E4M3value(sc) * g.
 *
 * sr: NULL, or {seed, row_offsets, col_offsets} with host arrays of num_sections
 *   Philox4x32-10 offsets (NULL = nearest-even in that direction).  Each 1x16 block
 *   draws one Philox call with key (lo32(seed), hi32(seed)) and counter
 *   (lo32(off_s), hi32(off_s), lo32(beta), hi32(beta)); beta = r*(k/16) + kb for
 *   row r (section-local) and block kb, beta = c*(m_s/16) + b for column c and
 *   block b; element t uses byte t&3 of output word t>>2.
 *
 * workspace: device memory of at least
 *   mxq_group_rht_quant_nvfp4_workspace_size(total_rows, k, num_sections, flags)
 *   bytes (0 when only MXQ_FP8_ROWWISE is requested; otherwise 135,680 bytes plus
 *   8 bytes per 16 rows per started 1024 columns of x, rounded up to 256), 256-byte
 *   aligned,
 *   ZERO-FILLED BEFORE ITS FIRST USE.  It holds partial maxima and per-section
 *   scale tables through which the kernels of a call meet in stream order, and the
 *   single-read form's partial words and error word, which must start at zero;
 *   every call leaves them at zero again, so a workspace is zeroed once and then
 *   reused.  Calls that share a workspace must be ordered (same stream, or
 *   synchronized).
 *
 * Requirements: k % 128 == 0, every m_s % 128 == 0 (else MXQ_ERR_MISALIGNED, with
 * no unfused fallback); 1 <= num_sections <= MXQ_MAX_SECTIONS; k <= 2^26,
 * total_rows <= 2^31 - 128 and total_rows * k < 2^40 (else MXQ_ERR_UNSUPPORTED);
 * the requested outputs non-NULL and 16-byte aligned
 * (global scales 4-byte aligned); outputs of directions not requested may be NULL.
 * ------------------------------------------------------------------------- */
enum { MXQ_ROWWISE = 1u, MXQ_COLUMNWISE = 2u, MXQ_FP8_ROWWISE = 4u };

typedef struct {
    uint8_t* codes;
    uint8_t* block_scales;
    float*   global_scales;
} mxq_nvfp4_out;

typedef struct {
    uint8_t* codes;
    float*   scales;
} mxq_fp8_out;

typedef struct {
    uint64_t        seed;
    const uint64_t* row_offsets;   /* host [num_sections], or NULL: nearest-even row-wise */
    const uint64_t* col_offsets;   /* host [num_sections], or NULL: nearest-even column-wise */
} mxq_sr;

/* Bytes of workspace the grouped call needs (0 when none is needed). */
size_t mxq_group_rht_quant_nvfp4_workspace_size(int64_t total_rows, int64_t k,
                                                int64_t num_sections, uint32_t flags);

mxq_status mxq_group_rht_quant_nvfp4(const uint16_t* x_bf16, int64_t k,
                                     const int64_t* split_sections, int64_t num_sections,
                                     uint16_t rht_sign_mask, uint32_t flags, const mxq_sr* sr,
                                     const mxq_nvfp4_out* rowwise,
                                     const mxq_nvfp4_out* columnwise,
                                     const mxq_fp8_out* fp8_rowwise,
                                     void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * The grouped call with caller-supplied section maxima (a single pass over x) and
 * the measured maxima out, for scaling the next step by this step's maxima.
 *
 * amax (may be NULL: as mxq_group_rht_quant_nvfp4):
 *   row_in, col_in    device float[num_sections]: the A of the tensor scales,
 *                     g = fl(max(A, F(1e-10)) * F(1/2688)), instead of the measured
 *                     maxima; given for every requested NVFP4 direction or for none
 *                     (else MXQ_ERR_INVALID_ARGUMENT).  Blocks above the supplied A
 *                     saturate (scale 0x7E, codes at +-6).
 *   row_out, col_out  device float[num_sections] or NULL: the measured maxima of this
 *                     call (max |x| without NaNs; max |BF16(H16 D x / 4)| without NaNs),
 *                     written for the requested directions; an empty section gives 0.
 * With supplied maxima the amax pass is skipped: the workspace only carries the scale
 * tables, and the maxima out are gathered with atomic maxima while quantizing.
 * Reading of TransformerEngine PR #2564 (the workspace / size-query pattern) for a
 * delayed-scaling variant of the same cast; everything else as above.
 * ------------------------------------------------------------------------- */
typedef struct {
    const float* row_in;
    const float* col_in;
    float*       row_out;
    float*       col_out;
} mxq_amax;

mxq_status mxq_group_rht_quant_nvfp4_with_amax(const uint16_t* x_bf16, int64_t k,
                                               const int64_t* split_sections, int64_t num_sections,
                                               uint16_t rht_sign_mask, uint32_t flags, const mxq_sr* sr,
                                               const mxq_nvfp4_out* rowwise,
                                               const mxq_nvfp4_out* columnwise,
                                               const mxq_fp8_out* fp8_rowwise, const mxq_amax* amax,
                                               void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * The grouped call for callers that cannot allocate: code under stream capture,
 * tight serving loops, harnesses that forbid allocation.  Arguments, outputs,
 * checks and results are those of mxq_group_rht_quant_nvfp4 without the workspace:
 * the library's own device array of MXQ_NOALLOC_SCRATCH_BYTES bytes stands in for it
 * (one per GPU, held until the process ends; its device address is looked up once
 * per device, on the first call with that device current, and the words the call
 * needs at zero are cleared then by a fill kernel on that call's stream).  A call
 * whose workspace would exceed the array (mxq_group_rht_quant_nvfp4_workspace_size
 * above MXQ_NOALLOC_SCRATCH_BYTES: more than 114,112 bands of 16 rows x 1024 columns,
 * e.g. more than 456,448 rows at k = 4096) gives
 * MXQ_ERR_UNSUPPORTED before anything is enqueued.  The call itself allocates
 * nothing (no hipMalloc, no allocating library routine).  The stream must belong to
 * the current device.  Every call on one GPU uses that GPU's array: calls that
 * overlap on one GPU (other streams, or other host threads without ordering) race.
 * ------------------------------------------------------------------------- */
#define MXQ_NOALLOC_SCRATCH_BYTES (1u << 20)

mxq_status mxq_group_rht_quant_nvfp4_noalloc(const uint16_t* x_bf16, int64_t k,
                                             const int64_t* split_sections, int64_t num_sections,
                                             uint16_t rht_sign_mask, uint32_t flags, const mxq_sr* sr,
                                             const mxq_nvfp4_out* rowwise,
                                             const mxq_nvfp4_out* columnwise,
                                             const mxq_fp8_out* fp8_rowwise, void* stream);

/* ---------------------------------------------------------------------------
 * Residual addition + RMS norm -> FP8 1x128: the quantizer in front of a W8A8
 * projection, with the norm that feeds it in the same pass.  For each row:
 *   z_i = BF16(x_i + res_i)  (nearest-even; z_i = x_i without a residual)
 *   r   = F(1 / sqrt(sum_i z_i^2 / n + eps)), the sum and everything inside in
 *         binary64, rounded once to binary32
 *   y_i = fl(fl(z_i * r) * w_i)                       (FP32; no round to BF16)
 * and then, per group of 128 consecutive y, exactly as mxq_quant_fp8_1x128
 * (a = max |y| without NaNs, s = fl(max(a, F(1e-10)) * F(1/448)), rounded up to a
 * power of two with MXQ_FP8_UE8M0, q = E4M3(fl(y / s)), 0x7F for a NaN).  The squares
 * are exact and n <= 32768 of them are summed in 53 bits, so the order of the sum can
 * change r only where the exact value lies within 2^-37 (relative) of a binary32
 * rounding border.
 *
 *   x_bf16        [m][ldx] BF16;  residual [m][ld_res] BF16, or NULL
 *   residual_out  [m][ld_res_out] BF16: z.  Required with a residual, NULL without;
 *                 may be the residual or x itself (same pointer and stride), and
 *                 must not overlap an input in any other way
 *   weight_bf16   [n] BF16;  eps >= 0, finite
 *   y_bf16        [m][ld_y] BF16(y) as well (a router's input), or NULL
 *   q_e4m3, ldq, scales, scale strides: as mxq_quant_fp8_1x128
 * Requirements: n % 128 == 0, n <= MXQ_RMSNORM_MAX_N and m < 2^22 (else
 * MXQ_ERR_UNSUPPORTED); BF16 strides multiples of 8, ldq of 16; pointers 16-byte
 * aligned, scales 4-byte aligned; options in {0, MXQ_FP8_UE8M0}.  m == 0 is a successful no-op.
 * ------------------------------------------------------------------------- */
#define MXQ_RMSNORM_MAX_N 32768
mxq_status mxq_add_rmsnorm_quant_fp8(const uint16_t* x_bf16, int64_t ldx, const uint16_t* residual, int64_t ld_res,
                                     uint16_t* residual_out, int64_t ld_res_out, const uint16_t* weight_bf16,
                                     float eps, int64_t m, int64_t n, uint32_t options,
                                     uint16_t* y_bf16, int64_t ld_y, uint8_t* q_e4m3, int64_t ldq,
                                     float* scales, int64_t scale_stride_row, int64_t scale_stride_group,
                                     void* stream);

/* ---------------------------------------------------------------------------
 * A paged KV cache in NVFP4.  Token t of a sequence lives in page block_table[t /
 * page_size] of the sequence, at row t % page_size; the row of K (or V) of one head
 * is head_dim/2 bytes of E2M1 codes (element 2i in the low nibble of byte i) and
 * head_dim/16 E4M3 block scales, and its values are
 *   E2M1value(code) * E4M3value(scale) * global[head]
 * with one FP32 tensor scale per head (caller-supplied, fixed while rows written
 * with it are in use; positive, finite and normal).  A row's codes start at
 *   codes + page * code_stride_page + head * code_stride_head + row * code_stride_token
 * (bytes), its scales likewise with the scale strides; K and V share the strides, so
 * [page][head][row] and [page][row][head] orders and caches interleaved with other
 * arrays are all expressed by them.
 * Requirements: head_dim 64 or 128; page_size a power of two, 16 .. 2^20 (else
 * MXQ_ERR_UNSUPPORTED); strides >= 0, code strides multiples of 16, scale strides of
 * head_dim/16 (else MXQ_ERR_MISALIGNED), token strides at most 2^24 (else
 * MXQ_ERR_UNSUPPORTED); codes 16-byte, scales 8-byte, globals 4-byte aligned; rows of
 * different (page, head, row) do not overlap.
 * ------------------------------------------------------------------------- */
typedef struct {
    uint8_t* k_codes;
    uint8_t* k_scales;
    uint8_t* v_codes;
    uint8_t* v_scales;
    const float* k_global;           /* device [kv_heads] */
    const float* v_global;           /* device [kv_heads] */
    int64_t num_pages;
    int32_t page_size;
    int32_t kv_heads;
    int32_t head_dim;
    int64_t code_stride_page;
    int64_t code_stride_head;
    int64_t code_stride_token;
    int64_t scale_stride_page;
    int64_t scale_stride_head;
    int64_t scale_stride_token;
} mxq_nvfp4_kv;

/* Rotary positions.  Pair i (0 <= i < rot_dim/2) of a head turns by the angle
 *   theta = fl64(position * inv_freq[i]),
 * so a table of inverse frequencies in binary64 expresses every scaling of them for
 * long contexts; cos and sin are formed in binary64 (error below 2^-50 for |theta| < 2^45,
 * which any position keeps to under frequencies below 2^14; NaN past it) and
 *   c = F(factor * cos(theta)),  s = F(factor * sin(theta))   (one round to binary32).
 * Pair i is elements (i, i + rot_dim/2) of the head, or (2i, 2i + 1) with
 * MXQ_ROPE_INTERLEAVED; with (a, b) its BF16 values the rotated pair is
 *   BF16(fl(fl(a c) - fl(b s))),  BF16(fl(fl(b c) + fl(a s))).
 * Elements from rot_dim on stay as they are.  rot_dim: a multiple of 16, at most
 * head_dim; 0 rotates nothing (inv_freq may then be NULL). */
enum { MXQ_ROPE_INTERLEAVED = 1u };
typedef struct {
    const double* inv_freq;          /* device [rot_dim / 2] */
    int32_t  rot_dim;
    uint32_t flags;                  /* 0 or MXQ_ROPE_INTERLEAVED */
    double   factor;                 /* on cos and sin (1 for plain frequencies) */
} mxq_rope;

/* ---------------------------------------------------------------------------
 * Rotary positions on Q and K, then K (rotated) and V appended to the cache.
 * For every token t: q_out[t] = rope(q[t]) and, unless slots[t] is negative or not
 * below num_pages * page_size (such a token is padding: nothing of the cache is
 * written for it), row slots[t] % page_size of page slots[t] / page_size gets the
 * row-wise NVFP4 encode of mxq_group_rht_quant_nvfp4 with the tensor scale g =
 * global[head]: per 1x16 block a = max |y|, t = fl(fl(a * F(1/6)) / g),
 * sc = E4M3(min(t, 448)); d = fl(E4M3(sc) * g), codes E2M1(fl(y / d)); a block with a
 * NaN gets scale 0x7F and zero codes, one with sc == 0 zero codes.
 *
 *   q        [tokens][ld_q] BF16, head h of a token at h * head_dim; q_out the same
 *            with ld_q_out (q_out = q with the same stride works in place; no other
 *            overlap).  q_heads may be 0 (q, q_out then NULL)
 *   k, v     [tokens][ld_k] / [ld_v] BF16, kv_heads heads of head_dim
 *   positions  device int32[tokens];  slots  device int64[tokens], distinct where
 *            they are not padding
 *   k_values, v_values  [tokens][kv_heads][head_dim] BF16(E2M1 * E4M3 * global), the
 *            values the cache stands for (products of the first two exact, one FP32
 *            round by global, one to BF16), written for every token, padding
 *            included; or NULL
 * Requirements: strides multiples of 8 and at least heads * head_dim; BF16 pointers
 * 16-byte aligned, positions 4-, slots and inv_freq 8-byte aligned; at least one cached
 * head; tokens * (q_heads + 2 kv_heads) * head_dim / 8, the product of the last three
 * rounded up to 256, below 2^32 (else MXQ_ERR_UNSUPPORTED).  tokens == 0 is a
 * successful no-op.
 * ------------------------------------------------------------------------- */
mxq_status mxq_rope_append_nvfp4(const uint16_t* q, int64_t ld_q, int32_t q_heads, uint16_t* q_out, int64_t ld_q_out,
                                 const uint16_t* k, int64_t ld_k, const uint16_t* v, int64_t ld_v, int64_t tokens,
                                 const int32_t* positions, const int64_t* slots, const mxq_rope* rope,
                                 const mxq_nvfp4_kv* cache, uint16_t* k_values, uint16_t* v_values, void* stream);

/* ---------------------------------------------------------------------------
 * Causal attention of ragged queries over the paged NVFP4 cache.  Sequence b has
 * seq_lens[b] cached tokens (its new ones included: append first) and the queries
 * q[q_starts[b]] .. q[q_starts[b + 1] - 1], the last of them at position
 * seq_lens[b] - 1; one query per sequence is a decoding step, more are a draft, a
 * chunk or a whole prompt.  Query head h reads cached head h / (q_heads / kv_heads).
 * The query at position p sees token t iff
 *   t <= p  and  (window == 0 or t > p - window or t < sinks)
 * and out = softmax(softmax_scale * q . k) . v over the tokens it sees; 0 (and lse =
 * -inf) where it sees none.  Both products run on FP16 operands with FP32 accumulators;
 * scores, maxima and sums are FP32.  K and V without their tensor scales are exact in
 * FP16.  Q is taken times a power of two per row: elements down to 2^-31 of their row's
 * largest are exact, smaller ones off by at most 2^-39 of it (of 2^-100 in a row whose
 * largest is below that).  The softmax weights are rounded to FP16 (nearest-even) for
 * the product with V, and not for their sum: each is off by at most 2^-11 of itself, or
 * by 2^-34 of its row's largest weight where that is more.  out is rounded to BF16 once.
 * The order of the sums depends on the lengths and on max_seq_len, not on what the
 * arrays hold, and a call repeats bit for bit.
 * What a query does not see changes no bit of its output, whatever it holds (NaN scales
 * included).  A NaN K row it sees makes its output NaN; a NaN V block it sees makes
 * at least that block's 16 elements NaN.
 *
 *   q        [total_q][ld_q] BF16, head h at h * head_dim; out alike with ld_out;
 *            must not overlap
 *   lse      [total_q][q_heads] FP32: the natural logarithm of the sum of exponentials
 *            (to join parts of a softmax), or NULL
 *   block_table  device int32 [batch][ld_table], table_pages entries of each row;
 *   seq_lens device int32[batch]; q_starts device int32[batch + 1], ascending
 *   max_q_len    at least the longest query run: later queries of a longer one are
 *                left unwritten.  max_seq_len: an estimate of the longest cached
 *                length, which sizes the split over the cache (longer sequences are
 *                still right, only slower)
 * Values read on the device are bounded there: a length above table_pages * page_size
 * is read as that and a negative one as 0; rows outside [0, total_q) are not touched;
 * a page number outside [0, num_pages) gives no access, and queries that see one of its
 * tokens come out NaN.  Rows of q that belong to no sequence leave out and lse as they
 * were.
 *
 * workspace: device memory of mxq_attention_nvfp4_workspace_size(...) bytes for the
 * same shape (0: none needed, may be NULL), 256-byte aligned, any contents: the call's
 * kernels meet through it in stream order and keep nothing in it between calls.  Calls
 * that share it must be ordered.
 * Requirements: q_heads a multiple of kv_heads; 1 <= batch <= 65535; ld_q, ld_out
 * multiples of 8 and at least q_heads * head_dim; q, out 16-byte aligned, the others
 * 4-byte; softmax_scale > 0 and finite; window, sinks >= 0; total_q * q_heads < 2^31;
 * batch * kv_heads * ceil(max_q_len * q_heads / kv_heads / 128) < 2^24 (else
 * MXQ_ERR_UNSUPPORTED).
 * total_q == 0 or max_q_len == 0 is a successful no-op.
 * ------------------------------------------------------------------------- */
size_t mxq_attention_nvfp4_workspace_size(int32_t q_heads, int32_t kv_heads, int32_t head_dim, int64_t batch,
                                          int64_t total_q, int64_t max_q_len, int64_t max_seq_len,
                                          int32_t window, int32_t sinks);

mxq_status mxq_attention_nvfp4(const uint16_t* q, int64_t ld_q, int32_t q_heads, int64_t total_q,
                               uint16_t* out, int64_t ld_out, float* lse, const mxq_nvfp4_kv* cache,
                               const int32_t* block_table, int64_t ld_table, int64_t table_pages,
                               const int32_t* seq_lens, const int32_t* q_starts, int64_t batch,
                               int64_t max_q_len, int64_t max_seq_len, float softmax_scale,
                               int32_t window, int32_t sinks, void* workspace, size_t workspace_bytes,
                               void* stream);

/* ---------------------------------------------------------------------------
 * The same attention (without a window) where groups of sequences share long prefixes: a
 * system prompt, a document.  Each prefix is attended once for all queries of its group,
 * so its tokens are read and dequantized once, not once per sequence.  Group g is the
 * sequences group_starts[g] .. group_starts[g + 1] - 1; the first prefix_lens[b] tokens of
 * sequence b are read through the pages of its group's first sequence (that row of
 * block_table), the others through its own:
 *   out = softmax(softmax_scale * q . k) . v over all tokens t <= p,
 * 0 (and lse = -inf) where there are none.  The sequences of a group may share prefixes of
 * different lengths, 0 among them; a prefix may end anywhere in a page, may be longer
 * than the sequence's own seq_lens[b] (the query at position p then sees its first p + 1
 * tokens), and what a sequence's own row of block_table says of shared tokens is not read.
 * Arithmetic, roundings, NaN scales, unreadable pages and the other arguments as in
 * mxq_attention_nvfp4.  A row's work is cut into parts, over the prefix and its own tokens,
 * which are held and joined in FP32; the order of the sums depends on the lengths, the
 * groups and the estimates.
 * The split is planned for groups of about as many queries each, and for sequences of about
 * as many tokens of their own; others are right, but wait for the largest.  Sequences that
 * share nothing belong in one group with prefix_lens 0, or in another's, not in groups of
 * one.  A sequence with far more tokens of its own than the rest is better off in a call of
 * its own.
 *   group_starts device int32[groups + 1], ascending; the first counts as 0 and the last
 *                as batch
 *   prefix_lens  device int32[batch]; held to [0, table_pages * page_size]
 *   max_prefix_len, max_own_len  estimates of the longest prefix and the most tokens
 *                behind one, which size the split (longer ones are still right)
 * workspace: device memory of mxq_attention_prefix_nvfp4_workspace_size(...) bytes, as
 * there (never 0 but for calls that do nothing or are refused).
 * Requirements: as there; 1 <= groups <= 4096; total_q * q_heads <= 2^26 - 4 and in total
 * fewer than 2^24 work-groups (the pieces of all rows; else MXQ_ERR_UNSUPPORTED).
 * total_q == 0 or max_q_len == 0 is a successful no-op.
 * ------------------------------------------------------------------------- */
size_t mxq_attention_prefix_nvfp4_workspace_size(int32_t q_heads, int32_t kv_heads, int32_t head_dim, int64_t batch,
                                                 int64_t groups, int64_t total_q, int64_t max_q_len,
                                                 int64_t max_prefix_len, int64_t max_own_len);

mxq_status mxq_attention_prefix_nvfp4(const uint16_t* q, int64_t ld_q, int32_t q_heads, int64_t total_q,
                                      uint16_t* out, int64_t ld_out, float* lse, const mxq_nvfp4_kv* cache,
                                      const int32_t* block_table, int64_t ld_table, int64_t table_pages,
                                      const int32_t* seq_lens, const int32_t* q_starts, int64_t batch,
                                      const int32_t* group_starts, const int32_t* prefix_lens, int64_t groups,
                                      int64_t max_q_len, int64_t max_prefix_len, int64_t max_own_len,
                                      float softmax_scale, void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Mean keys of full pages, for the selection below: kept beside a cache, one per
 * page and cached head, as 8-bit integers with an FP32 scale.
 *   codes    device int8  [num_pages][kv_heads][head_dim], 16-byte aligned
 *   scales   device FP32  [num_pages][kv_heads], 4-byte aligned
 * The mean key is codes * scales.  Requirements: head_dim 64 or 128; page_size a
 * power of two, 16 .. 512 (else MXQ_ERR_UNSUPPORTED).
 * ------------------------------------------------------------------------- */
typedef struct {
    int8_t* codes;
    float* scales;
    int64_t num_pages;
    int32_t page_size;
    int32_t kv_heads;
    int32_t head_dim;
} mxq_page_keys;

/* The mean keys of the pages whose last row is among `slots`: with the slots of an
 * append, called after it, every page that it filled (rows of a sequence arrive in
 * order, so a page is full when its last row is written).  Slots that are negative or not
 * below num_pages * page_size are padding, other rows change nothing.  For one page and
 * head, over its page_size rows of K, with g = k_global[head]:
 *   S[d]   = sum of 1024 * E2M1value(code) * E4M3value(scale)      (whole numbers, exact)
 *   a      = max |S[d]|
 *   codes[d] = the whole number nearest to 127 S[d] / a, the even one of two; 0 if a == 0
 *   scales = F(fl64(fl64(a g) fl64(1 / (130048 page_size))))       (130048 = 127 * 1024)
 * A page with a NaN block scale gets codes 0 and a NaN scale.
 *   slots    device int64[tokens], 8-byte aligned
 * The cache's and keys' num_pages, page_size, kv_heads and head_dim are the same (else
 * MXQ_ERR_INVALID_ARGUMENT).  tokens == 0 is a successful no-op. */
mxq_status mxq_page_keys_nvfp4(const mxq_nvfp4_kv* cache, const int64_t* slots, int64_t tokens,
                               const mxq_page_keys* keys, void* stream);

/* ---------------------------------------------------------------------------
 * The pages that each query attends, for each cached head (its q_heads / kv_heads query
 * heads share them).  Sequences, queries and positions as in mxq_attention_nvfp4: the
 * query at position p sees pages 0 .. c = p / page_size of its sequence (counted along
 * its row of block_table).  pages[query][head] holds them all, ascending, where
 * c < top; else `top` of them, ascending: the first `first`, the last `last` (c among
 * them) and of the others those with the highest scores, lower ones before higher ones
 * where scores are equal.  Unused entries are -1.  The score of a page with mean key
 * (codes, scale) for the group's query heads h:
 *   s_h   = fl(max |q_h| * F(1/127));  i_h[d] = the whole number nearest to
 *           fl(q_h[d] / s_h), the even one of two, held to [-127, 127]
 *           (a row of zeros, or with an infinity or NaN: s_h = 0, i_h = 0)
 *   score = fl(max over h of fl((sum of i_h[d] codes[d]) * s_h) * scale)
 * (the sums are exact).  A NaN score, and that of a page number outside [0, num_pages),
 * is below all others.  Only pages that are full are scored: `last` is at least 1.
 *
 *   q        [total_q][ld_q] BF16, head h at h * head_dim
 *   pages    device int32 [total_q][kv_heads][top], 4-byte aligned; rows of queries
 *            that belong to no sequence are left as they were
 *   max_seq_len  an estimate of the longest cached length, which sizes what is held
 *            of the scores (longer sequences are still right, only slower)
 * block_table, table_pages, seq_lens and q_starts as in mxq_attention_nvfp4.
 * workspace: device memory of mxq_select_pages_nvfp4_workspace_size(...) bytes for the
 * same shape (0: none needed, may be NULL), 256-byte aligned, any contents, as there.
 * Requirements: q_heads a multiple of kv_heads; 1 <= batch <= 65535; ld_q a multiple of
 * 8 and at least q_heads * head_dim; q 16-byte aligned; first >= 0, last >= 1,
 * first + last <= top; top <= 65536; total_q * q_heads < 2^31 and total_q * kv_heads
 * below 2^24 (else MXQ_ERR_UNSUPPORTED).  total_q == 0 is a successful no-op.
 * ------------------------------------------------------------------------- */
size_t mxq_select_pages_nvfp4_workspace_size(int32_t q_heads, int32_t kv_heads, int32_t page_size, int64_t batch,
                                             int64_t total_q, int64_t max_seq_len);

mxq_status mxq_select_pages_nvfp4(const uint16_t* q, int64_t ld_q, int32_t q_heads, int64_t total_q,
                                  const mxq_page_keys* keys, const int32_t* block_table, int64_t ld_table,
                                  int64_t table_pages, const int32_t* seq_lens, const int32_t* q_starts,
                                  int64_t batch, int64_t max_seq_len, int32_t top, int32_t first, int32_t last,
                                  int32_t* pages, void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Causal attention over listed pages (without a window): the query at position p and the
 * query heads of cached head k attend the tokens t <= p of the pages pages[query][k][0 ..
 * top - 1] of their sequence (counted along its row of block_table, as
 * mxq_select_pages_nvfp4 writes them); out = 0 and lse = -inf where there is none.  Entries
 * that are negative or above p / page_size add nothing, in any place; a page that is listed
 * twice counts twice.  The arithmetic, its roundings, what NaN scales and unreadable pages
 * do, and the other arguments are those of mxq_attention_nvfp4 (few queries' lists are cut
 * into parts, held and joined in FP32).  Lists are read to their end by every work-group
 * before its first page; entries after the last that counts load nothing of the cache.
 *   pages    device int32 [total_q][kv_heads][top], 4-byte aligned
 * workspace: device memory of mxq_attention_pages_nvfp4_workspace_size(...) bytes, as there.
 * Requirements: those of mxq_attention_nvfp4 on q, out, the cache, the sequences and the
 * scale; 1 <= top <= 65536, top * page_size <= 2^30 and total_q * kv_heads *
 * ceil(q_heads / kv_heads / 32) below 2^24 (else MXQ_ERR_UNSUPPORTED).  total_q == 0 is a
 * successful no-op.
 * ------------------------------------------------------------------------- */
size_t mxq_attention_pages_nvfp4_workspace_size(int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                                int32_t page_size, int64_t total_q, int32_t top);

mxq_status mxq_attention_pages_nvfp4(const uint16_t* q, int64_t ld_q, int32_t q_heads, int64_t total_q,
                                     uint16_t* out, int64_t ld_out, float* lse, const mxq_nvfp4_kv* cache,
                                     const int32_t* block_table, int64_t ld_table, int64_t table_pages,
                                     const int32_t* seq_lens, const int32_t* q_starts, int64_t batch,
                                     const int32_t* pages, int32_t top, float softmax_scale, void* workspace,
                                     size_t workspace_bytes, void* stream);


#ifdef __cplusplus
}
#endif
#endif /* MXQ_H */
