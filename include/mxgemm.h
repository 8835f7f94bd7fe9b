/*
 * mxgemm.h -- C ABI of the block-scaled FP8 GEMM with a fused global-amax
 * epilogue, for AMD Instinct MI355X (gfx950).
 *
 * Operation ("GEMM + Amax (SM100)", section "Equations"):
 *
 *   A_hat[m,k,l] = dec(A[m,k,l]) * 2^(SFA(m, k/sf, l) - 127)
 *   B_hat[n,k,l] = dec(B[n,k,l]) * 2^(SFB(n, k/sf, l) - 127)
 *   C[m,n,l]     = sum_k A_hat[m,k,l] * B_hat[n,k,l]      (FP32 accumulation)
 *   Amax         = max_{m,n,l} |C[m,n,l]|
 *
 * with sf = sf_vec_size in {16, 32} consecutive K elements per E8M0 scale.
 *
 * Memory layout (section "Parameters", input/output tensors; all buffers are
 * device memory owned by the caller, contiguous, byte offsets 64-bit):
 *   A    : (L, M, K) element codes, one byte each ("k-major" A, strides
 *          (K, 1, M*K) in the page's (M, K, L) notation).
 *   B    : (L, N, K) element codes ("k-major" B).
 *   SFA  : E8M0 scale bytes in the physical atom layout
 *          (L, ceil(M/128), ceil(K/(4*sf)), 32, 4, 4) -- the C-contiguous
 *          allocation whose permutation (3,4,1,5,2,0) is the logical
 *          (32, 4, ceil(M/128), 4, ceil(K/(4*sf)), L) of section "Shapes"
 *          (section "Using JAX arrays").  Row mn = i0 + 32*i1 + 128*i2 and
 *          K-block kb = i3 + 4*i4 of logical index (i0,i1,i2,i3,i4,l), i.e.
 *          byte 16*(mn%32) + 4*((mn/32)%4) + kb%4 of 512-byte atom
 *          (l*ceil(M/128) + mn/128)*ceil(K/(4*sf)) + kb/4.
 *          Padding bytes (rows >= M, K-blocks >= ceil(K/sf)) are never used
 *          and may hold anything.
 *   SFB  : the same for B with N in place of M.
 *   C    : (L, M, N) float32 ("n-major" C, the page's default c_major="n").
 *   Amax : one float32 (the page's (1,1,1) tensor).
 *
 * Element formats: MXG_FMT_E4M3 (float8_e4m3fn) and MXG_FMT_E5M2
 * (float8_e5m2).  A and B may use different formats and FP8 may be used
 * with sf = 16; both go beyond the page's support list (section "Support
 * surface and constraints", Dtypes) and follow the format-agnostic equations.
 *
 * Errors: every entry point returns MXG_OK (0) or a negative status, and an
 * invalid argument is reported before any work is queued on the stream
 * (the error convention of "Grouped GEMM (SM100 BF16)", section
 * "Scheduling, caching, and errors").  MXG_ERR_LAUNCH reports a HIP error
 * from the launch itself.
 *
 * Streams: `stream` is a hipStream_t passed as void*; NULL is the null
 * stream (the page's eager default, section "Using JAX arrays").  Calls are
 * asynchronous; inputs must stay alive and unmodified, and outputs unread,
 * until the stream has reached the call.
 *
 * The library allocates no device memory (inputs, outputs and the stream
 * are the caller's) and keeps no pointer after a call returns.
 */
#ifndef MXGEMM_H
#define MXGEMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* element formats of A and B */
enum {
  MXG_FMT_E4M3 = 0, /* float8_e4m3fn: bias 7, no inf, NaN = 0x7F/0xFF, max 448 */
  MXG_FMT_E5M2 = 1, /* float8_e5m2:   bias 15, inf = 0x7C/0xFC, max 57344      */
  MXG_FMT_E2M1 = 2  /* float4_e2m1fn_x2: packed FP4, two elements per byte,
                       element 2k in the low nibble; bias 1, no inf/NaN, max 6.
                       A is then (L, M, K/2) bytes and B (L, N, K/2).  Both
                       operands must be E2M1, K % 32 == 0, and the default
                       (bf16) datapath; sf_vec_size 32 or 16 (the pages
                       exclude 16 only for 8-bit A/B, "Support surface and
                       constraints", dtypes); at 16 the kernel runs 128x128
                       tiles (the scale atoms of a 256x256 tile's step do
                       not fit beside it in LDS), and MXG_FLAG_TILE_256 is
                       MXG_ERR_FLAGS.  The pages list the packed container
                       ("Parameters", A dtype) but not which nibble comes
                       first: low first is the reading. */
};

/* status codes */
enum {
  MXG_OK = 0,
  MXG_ERR_NULL = -1,   /* a required pointer is NULL                          */
  MXG_ERR_SHAPE = -2,  /* a negative size, or a size whose offsets overflow   */
  MXG_ERR_ALIGN = -3,  /* A/B/C/Amax not 16-byte aligned, K % 16, N % 4       */
  MXG_ERR_SFVEC = -4,  /* sf_vec_size not 16 or 32                            */
  MXG_ERR_FMT = -5,    /* element format unknown, or E2M1 on one operand only */
  MXG_ERR_DEVICE = -6, /* current device is not gfx950, or a pointer is not
                          device memory of the current device                 */
  MXG_ERR_LAUNCH = -7, /* HIP reported an error when launching                */
  MXG_ERR_FLAGS = -8,  /* unknown bit in `flags`                              */
  MXG_ERR_SCRATCH = -9 /* the problem needs more scratch than the library's
                          fixed scratch array holds (the _noalloc entry)      */
};

/* flags of mxgemm_amax_ex */
enum {
  /* Do not clear Amax first: Amax := max(Amax, max|C|).  The caller keeps
     Amax a non-negative float (or NaN); lets several GEMMs share one Amax. */
  MXG_FLAG_AMAX_ACCUMULATE = 1u,
  /* Feed the FP8 codes straight to gfx950's scaled FP8 MFMA (twice the
     matrix rate of the default path).  That instruction keeps only the top
     ~13 bits, relative to the largest product, of each 8-element partial
     dot product, so small products next to large ones are truncated and
     the result can miss a 1e-5 * sum|A_hat*B_hat| error bound on
     heavy-tailed data.  The default path dequantises each element exactly
     to bf16 (scale folded in) and accumulates in fp32 on the bf16 MFMA. */
  MXG_FLAG_FP8_MFMA = 2u,
  /* Force the tile size instead of the automatic choice (for tests and
     tuning).  TILE_128: 128x128 tiles; TILE_256: 256x256 tiles; one
     workgroup per CU either way, of 4 computing waves (128x128 tiles on the
     default path, FP4 at sf = 16 aside: and 4 more that only stream the
     operands into LDS).  Both sizes compute every output the same way, so
     results agree bit for bit.  Ignored when K == 0.  Setting both is an
     error. */
  MXG_FLAG_TILE_128 = 4u,
  MXG_FLAG_TILE_256 = 8u,
  /* A 16-bit C ("GEMM + Amax (SM100)", section "Parameters": the C tensor
     may be float16 or bfloat16 as well as float32): C then holds (L, M, N)
     bfloat16 (C_BF16) or float16 (C_F16) elements, each the float32
     accumulator rounded to nearest even (float16 overflows to +-inf).  Amax
     is still taken over the float32 accumulators (the pages do not say which;
     the fused epilogue sees those).  The C pointer keeps its float* type in
     the signature and must still be 16-byte aligned.  Not with
     MXG_FLAG_FP8_MFMA; setting both C flags is an error. */
  MXG_FLAG_C_BF16 = 32u,
  MXG_FLAG_C_F16 = 64u,
  /* m-major C ("GEMM + Amax (SM100)", section "Parameters": C of shape
     (M, N, L) with strides (1, M, M*N), the wrapper's c_major="m"): C then
     holds (L, N, M) float32 elements, M contiguous.  The contiguous dimension
     must be 16-byte aligned, so M % 4 == 0 as well (MXG_ERR_ALIGN otherwise).
     The default datapath with a float32 C only: not with MXG_FLAG_FP8_MFMA
     or MXG_FLAG_C_BF16 / _F16 (MXG_ERR_FLAGS). */
  MXG_FLAG_C_MMAJOR = 128u,
  /* m-major A and n-major B ("GEMM + Amax (SM100)", section "Parameters":
     A of shape (M, K, L) with strides (1, M, M*K), B (N, K, L) with strides
     (1, N, N*K)): A then holds (L, K, M) codes, M contiguous (A_MMAJOR), B
     (L, K, N) codes, N contiguous (B_NMAJOR); either or both.  The kernel
     stages such a tile as K rows in LDS and reads it with gfx950's
     transposing LDS load, so no copy is made; results are bitwise those of
     the k-major operands.  8-bit formats, the default datapath and a
     float32 n-major C only (MXG_ERR_FLAGS otherwise); the contiguous
     dimension must be a multiple of 16 (MXG_ERR_ALIGN) and one batch of the
     operand (M*K or N*K bytes) below 2^31 (MXG_ERR_SHAPE). */
  MXG_FLAG_A_MMAJOR = 256u,
  MXG_FLAG_B_NMAJOR = 512u
};

/*
 * mxgemm_amax -- C = A_hat . B_hat^T per batch and Amax = max |C|.
 *
 *   A, B       device pointers to the element codes (layouts above).
 *   SFA, SFB   device pointers to the physical SF atom buffers,
 *              mxgemm_sf_bytes(M or N, K, L, sf_vec_size) bytes each.
 *   C          device pointer, L*M*N float32, fully overwritten.
 *   Amax       device pointer to one float32; set to max|C| (0 when
 *              M*N*L == 0; NaN if any C is NaN).
 *   M, N, K, L sizes, each >= 0.  K == 0 gives C == 0.
 *   sf_vec_size 16 or 32.
 *   a_fmt, b_fmt MXG_FMT_E4M3, MXG_FMT_E5M2, or MXG_FMT_E2M1 for both.
 *   stream     hipStream_t (NULL = null stream).
 *
 * Requirements: A, B, C, Amax, SFA, SFB 16-byte aligned; K % 16 == 0 (16-byte
 * rows of A/B) and K <= 2^23; N % 4 == 0 (16-byte rows of C) and N < 2^22 -- the page's "16-byte aligned along
 * the contiguous dimension" (section "Support surface and constraints",
 * Layouts and strides).  Current device must be gfx950 and own every pointer.
 *
 * Queues a one-wave kernel that clears Amax, then the GEMM kernel.
 */
int mxgemm_amax(const void* A, const void* B, const uint8_t* SFA, const uint8_t* SFB,
                float* C, float* Amax, int64_t M, int64_t N, int64_t K, int64_t L,
                int sf_vec_size, int a_fmt, int b_fmt, void* stream);

/*
 * mxgemm_amax_ex -- mxgemm_amax with flags.  flags == 0 is exactly
 * mxgemm_amax; MXG_FLAG_AMAX_ACCUMULATE skips the clearing kernel and
 * max-reduces into the existing Amax (queues the GEMM kernel only);
 * MXG_FLAG_FP8_MFMA selects the reduced-precision FP8 matrix path;
 * MXG_FLAG_TILE_128 / _256 force a tile configuration; MXG_FLAG_C_BF16 /
 * _F16 store a 16-bit C; MXG_FLAG_C_MMAJOR stores C m-major, (L, N, M)
 * float32 with M contiguous, which needs M % 4 == 0 (MXG_ERR_ALIGN) and
 * M < 2^22 (MXG_ERR_SHAPE; M takes N's place in the per-tile offsets).
 * Returns MXG_ERR_FLAGS for unknown bits, more than one tile flag, both C
 * flags, a C flag with MXG_FLAG_FP8_MFMA, or MXG_FLAG_C_MMAJOR with a flag it
 * excludes.
 *
 * Accuracy of the default path.  Every dequantised element is exact when its
 * value fits bf16: for every code when the scale byte lies in 3..246 (E4M3)
 * or 10..239 (E5M2); outside those bytes, codes whose value still fits bf16
 * stay exact and the others round to bf16.  Products are exact; the K sum is
 * an fp32 accumulation, one rounded add per 16 K, so its error grows with K:
 * at most about (K/16 + 1) * 2^-24 * S, S = sum_k |A_hat||B_hat|, reached
 * only when all products share a sign; mixed signs grow like sqrt(K).  The
 * bound is within 1e-5 * S for K <= 2048 whatever the data; beyond that,
 * same-sign data can exceed it (measured ratios are in the GPU tests).
 */
int mxgemm_amax_ex(const void* A, const void* B, const uint8_t* SFA, const uint8_t* SFB,
                   float* C, float* Amax, int64_t M, int64_t N, int64_t K, int64_t L,
                   int sf_vec_size, int a_fmt, int b_fmt, unsigned flags, void* stream);

/*
 * mxgemm_amax_reset -- queue the one-wave kernel that sets *Amax = 0.0f.
 * mxgemm_amax == mxgemm_amax_reset + mxgemm_amax_ex(MXG_FLAG_AMAX_ACCUMULATE).
 */
int mxgemm_amax_reset(float* Amax, void* stream);

/*
 * mxgemm_check_support -- host-only check of a problem description, the
 * counterpart of the page's check_support() (section "API Usage", class
 * API).  Returns MXG_OK or the status mxgemm_amax would return for these
 * sizes/formats (pointers and device are not checked).  No HIP call.
 */
int mxgemm_check_support(int64_t M, int64_t N, int64_t K, int64_t L, int sf_vec_size,
                         int a_fmt, int b_fmt);

/*
 * mxgemm_sf_bytes -- size of one physical SF buffer:
 * 512 * L * ceil(MN/128) * ceil(K/(4*sf_vec_size)); 0 for invalid input.
 * No HIP call.
 */
size_t mxgemm_sf_bytes(int64_t MN, int64_t K, int64_t L, int sf_vec_size);

/*
 * mxgemm_launch_config -- the tile shape and grid the GEMM kernel would use
 * for this problem with 8-bit operands (for reporting and tests; packed FP4
 * at sf_vec_size 16 always runs 128x128 tiles).  Writes tile_m, tile_n and
 * the number of workgroups (the tile count when the tiles fit the compute
 * units; otherwise the tiles of one of the rounds a full grid would need,
 * rounded up to a multiple of 8 and capped at the compute units, so every
 * workgroup runs the same number of tiles give or take one); any output
 * pointer may be NULL.  Returns a
 * status like mxgemm_check_support.  Queries the current device's compute
 * unit count (HIP call) only when `grid` is requested.
 */
int mxgemm_launch_config(int64_t M, int64_t N, int64_t K, int64_t L, int sf_vec_size,
                         int* tile_m, int* tile_n, int64_t* grid);

/*
 * Plans ("GEMM + Amax (SM100)", sections on the class API: check_support,
 * compile, then execute per call, and its note on per-launch CPU cost).
 * mxgemm_plan_init validates sizes, formats and flags once (the checks of
 * mxgemm_check_support plus the flag rules of mxgemm_amax_ex), queries the
 * current device and fixes the tile configuration.  mxgemm_plan_execute then
 * runs mxgemm_amax_ex with those sizes and flags on the given buffers,
 * checking only null pointers, 16-byte alignment and that the current device
 * is the plan's; it does not ask HIP where each pointer lives, so the caller
 * guarantees the buffers are device memory of that device (as the pages'
 * execute takes tensors already placed for the compiled kernel).
 *
 * mxgemm_plan is plain caller-owned memory (no allocation, nothing to free);
 * a plan may be copied and used from several threads and streams.  Results
 * are identical to mxgemm_amax_ex with the same arguments.  Errors:
 * init returns mxgemm_amax_ex's validation statuses (and MXG_ERR_DEVICE
 * without a gfx950 device); execute returns MXG_ERR_NULL (also for a plan
 * never initialised), MXG_ERR_ALIGN, MXG_ERR_DEVICE (another current
 * device) or MXG_ERR_LAUNCH.
 */
typedef struct mxgemm_plan {
  uint64_t opaque[32];
} mxgemm_plan;

int mxgemm_plan_init(mxgemm_plan* plan, int64_t M, int64_t N, int64_t K, int64_t L, int sf_vec_size,
                     int a_fmt, int b_fmt, unsigned flags);
int mxgemm_plan_execute(const mxgemm_plan* plan, const void* A, const void* B, const uint8_t* SFA,
                        const uint8_t* SFB, float* C, float* Amax, void* stream);

/*
 * mxgemm_mx_quantize -- MX block quantisation of float32 data into the
 * GEMM's input form: element codes plus E8M0 block scales in the physical
 * atom layout ("GEMM + RoPE + MXFP8 Projection (SM100)", section
 * "Equations": MXFP8 quantisation with an E8M0 scale per block of 32 and
 * E4M3 data; E5M2 and blocks of 16 follow the same rule).
 *
 *   X   : (L, MN, K) float32, K contiguous (an A or B operand before
 *         quantisation).
 *   Q   : (L, MN, K) element codes, one byte each (the layout of A / B).
 *   SF  : mxgemm_sf_bytes(MN, K, L, sf_vec_size) bytes, the physical atom
 *         layout described above for SFA / SFB.  Every byte is written:
 *         padding entries (rows >= MN, K-blocks >= ceil(K/sf)) get 127.
 *   fmt : MXG_FMT_E4M3 (FMAX = 448) or MXG_FMT_E5M2 (FMAX = 57344).
 *
 * Per row and block of sf_vec_size consecutive K elements (the last block
 * may be partial): bm = max |x|; e = the smallest integer with
 * FMAX * 2^e >= bm, clamped to [-127, 127], and e = 0 when bm = 0; scale
 * byte = e + 127; code = x * 2^-e rounded to the nearest code, ties to even
 * (nothing saturates: |x * 2^-e| <= FMAX).  The pages give no formula for
 * the scale; this rule is the one the GEMM's test inputs are made with (a
 * scale of 2^ceil(log2(blockmax / FMAX))).  Results for non-finite inputs
 * are unspecified.
 *
 * Errors (before any work): MXG_ERR_SHAPE (a negative size, K >= 2^23 or
 * too many atoms), MXG_ERR_SFVEC, MXG_ERR_FMT, MXG_ERR_ALIGN (K % 16 or a
 * pointer not 16-byte aligned), MXG_ERR_NULL, MXG_ERR_DEVICE.  MN, K or
 * L == 0 queues nothing and returns MXG_OK.  Q and SF must not overlap X.
 */
int mxgemm_mx_quantize(const float* X, void* Q, uint8_t* SF, int64_t MN, int64_t K, int64_t L,
                       int sf_vec_size, int fmt, void* stream);

/*
 * mxgemm_sf_rowwise_to_atoms -- row-wise E8M0 block scales into the
 * physical atom layout that mxgemm_amax reads (for operands quantised with
 * row-wise scales: "GEMM + RoPE + MXFP8 Projection (SM100)", section
 * "Shapes", x_scale (tokens, Q_LORA/32) and w_scale (rows, Q_LORA/32)).
 *
 *   rowwise : (L, MN, ceil(K/sf)) bytes, contiguous; byte (l, row, kb) is
 *             the scale of row `row`, K elements [kb*sf, (kb+1)*sf).
 *   SF      : mxgemm_sf_bytes(MN, K, L, sf_vec_size) bytes, 16-byte aligned;
 *             every byte is written, padding entries (rows >= MN, K-blocks
 *             >= ceil(K/sf)) get 127.
 *
 * Errors (before any work): MXG_ERR_SHAPE, MXG_ERR_SFVEC, MXG_ERR_NULL,
 * MXG_ERR_ALIGN (SF), MXG_ERR_DEVICE.  MN, K or L == 0 queues nothing.
 */
int mxgemm_sf_rowwise_to_atoms(const uint8_t* rowwise, uint8_t* SF, int64_t MN, int64_t K, int64_t L,
                               int sf_vec_size, void* stream);

/*
 * mxgemm_gemm_rope_mxfp8 -- the projection of "GEMM + RoPE + MXFP8
 * Projection (SM100)" (sections "Overview", "Shapes", "Equations") in one
 * kernel: Y = A B^T as in mxgemm_amax (L = 1; A (tokens, K) and B (N, K)
 * codes, N = num_heads * head_dim, SF atoms as there), and in place of
 * storing Y, per head: RoPE on the trailing qk_rope features (the rule of
 * mxgemm_proj_rope_mxfp8 below) and E4M3 codes with E8M0 scales in both
 * block directions, exactly what mxgemm_proj_rope_mxfp8 makes of the
 * float32 Y that mxgemm_amax (with 256x256 tiles) computes for these
 * operands.  No Y and no Amax is written.
 *   cos_bf16, sin_bf16 : (tokens, qk_rope) bf16 bits.
 *   row_codes (tokens, N) bytes, row_scales (tokens, N / 32),
 *   col_codes (tokens, N), col_scales (tokens / 32, N): caller-owned outputs.
 * Requirements: K > 0 and the GEMM's rules on K; tokens % 32 == 0
 * (MXG_ERR_ALIGN); head_dim a multiple of 32, at least 128; qk_rope a
 * multiple of 16, at most 64; N % 128 == 0; no head's rotary features
 * crossing a multiple of 128 columns (else MXG_ERR_SHAPE); a_fmt, b_fmt
 * E4M3 or E5M2; sf_vec_size 16 or 32; every pointer 16-byte aligned.
 * Asynchronous on `stream`; errors before any work; tokens or num_heads == 0
 * queues nothing.
 */
int mxgemm_gemm_rope_mxfp8(const void* A, const void* B, const uint8_t* SFA, const uint8_t* SFB,
                           const uint16_t* cos_bf16, const uint16_t* sin_bf16, uint8_t* row_codes,
                           uint8_t* row_scales, uint8_t* col_codes, uint8_t* col_scales, int64_t tokens,
                           int64_t num_heads, int64_t head_dim, int64_t qk_rope, int64_t K, int sf_vec_size, int a_fmt,
                           int b_fmt, void* stream);

/*
 * mxgemm_projection_workspace_bytes -- bytes of workspace that
 * mxgemm_projection_mxfp8 needs: the atom-layout scales of x and w
 * (mxgemm_sf_bytes of each, the first rounded up to 256).
 */
size_t mxgemm_projection_workspace_bytes(int64_t tokens, int64_t num_heads, int64_t head_dim, int64_t K);

/*
 * mxgemm_projection_mxfp8 -- the projection page's MXFP8-input path as the
 * page passes it: x (tokens, K) and w (num_heads * head_dim, K) E4M3 codes
 * with row-wise E8M0 scales x_scale (tokens, ceil(K/32)) and w_scale
 * (num_heads * head_dim, ceil(K/32)) ("Shapes": blocks of 32 along Q_LORA).
 * The scales are rewritten into the atom layout in `workspace` (device
 * memory of at least mxgemm_projection_workspace_bytes, 256-byte aligned,
 * caller-owned, overwritten), then mxgemm_gemm_rope_mxfp8 runs with
 * sf_vec_size 32.  Rules, outputs and errors as there; a short workspace is
 * MXG_ERR_SHAPE.  Three kernels on `stream`.
 */
int mxgemm_projection_mxfp8(const void* x, const void* w, const uint8_t* x_scale, const uint8_t* w_scale,
                            const uint16_t* cos_bf16, const uint16_t* sin_bf16, uint8_t* row_codes,
                            uint8_t* row_scales, uint8_t* col_codes, uint8_t* col_scales, int64_t tokens,
                            int64_t num_heads, int64_t head_dim, int64_t qk_rope, int64_t K, void* workspace,
                            size_t workspace_bytes, void* stream);

/*
 * mxgemm_projection_mxfp8_noalloc -- mxgemm_projection_mxfp8 for callers that
 * cannot allocate device memory (code under graph capture, tight serving
 * loops, harnesses that forbid it): the same operation, arguments and
 * results, with the workspace taken from a fixed array inside the library
 * (MXGEMM_NOALLOC_SCRATCH_BYTES per device, reserved when the library is
 * loaded and held until the process ends) instead of a caller buffer.  It
 * calls no allocator.  A problem whose workspace
 * (mxgemm_projection_workspace_bytes) exceeds the array is rejected with
 * MXG_ERR_SCRATCH before any work.  Every call on one device shares that
 * device's array: calls that may overlap on one device (other streams,
 * other threads) race and must be serialised by the caller.  The array's
 * contents are overwritten in full by each call before they are read.
 */
#define MXGEMM_NOALLOC_SCRATCH_BYTES (8u << 20)
int mxgemm_projection_mxfp8_noalloc(const void* x, const void* w, const uint8_t* x_scale, const uint8_t* w_scale,
                                    const uint16_t* cos_bf16, const uint16_t* sin_bf16, uint8_t* row_codes,
                                    uint8_t* row_scales, uint8_t* col_codes, uint8_t* col_scales, int64_t tokens,
                                    int64_t num_heads, int64_t head_dim, int64_t qk_rope, int64_t K, void* stream);

/*
 * mxgemm_codes_to_kmajor -- m-major (or n-major) 8-bit element codes into the
 * k-major rows mxgemm_amax reads ("GEMM + Amax (SM100)", section
 * "Parameters": A of shape (M, K, L) may have strides (1, M, M*K), B of shape
 * (N, K, L) strides (1, N, N*K); packed FP4 operands must be k-major).
 *
 *   src : (L, K, MN) bytes, MN contiguous -- byte (mn, k, l) at
 *         mn + MN*k + MN*K*l; 16-byte aligned.
 *   dst : (L, MN, K) bytes, K contiguous -- the A or B argument of
 *         mxgemm_amax; 16-byte aligned, caller-owned, not overlapping src.
 *   MN  : M for A, N for B.
 *
 * Asynchronous on `stream`; the library allocates nothing.  Errors (before
 * any work): MXG_ERR_SHAPE, MXG_ERR_ALIGN (MN % 16 or K % 16 -- the 16-byte
 * alignment of both contiguous dimensions -- or a pointer), MXG_ERR_NULL,
 * MXG_ERR_DEVICE.  MN, K or L == 0 queues nothing and returns MXG_OK.
 */
int mxgemm_codes_to_kmajor(const void* src, void* dst, int64_t MN, int64_t K, int64_t L, void* stream);

/*
 * mxgemm_proj_rope_mxfp8 -- the projection's per-head RoPE and dual-direction
 * MXFP8 quantisation ("GEMM + RoPE + MXFP8 Projection (SM100)", sections
 * "Overview", "Shapes" and "Equations"), applied to the float32 output Y of
 * mxgemm_amax (M = tokens, N = num_heads * head_dim).
 *
 *   Y          : (tokens, num_heads * head_dim) float32, 16-byte aligned.
 *   cos_bf16,
 *   sin_bf16   : (tokens, qk_rope) bfloat16 bit patterns, 16-byte aligned.
 *   row_codes  : (tokens, num_heads, head_dim) E4M3 codes, blocks of 32 along
 *                head_dim; row_scales: (tokens, num_heads, head_dim / 32)
 *                E8M0 bytes.
 *   col_codes  : (tokens, num_heads, head_dim) E4M3 codes, blocks of 32 along
 *                tokens; col_scales: (tokens / 32, num_heads, head_dim) E8M0.
 *
 * RoPE acts on the last qk_rope features of each head, interleaved in and
 * halves out: with (a_i, b_i) = (y[2i], y[2i+1]) of that part and
 * R = qk_rope / 2, out[i] = a_i cos[i] - b_i sin[i] and
 * out[R+i] = b_i cos[R+i] + a_i sin[R+i], in float32 with each product and
 * the sum rounded on its own.  Block scale 2^e with e the smallest integer
 * giving 448 * 2^e >= the block's largest magnitude (0 for an all-zero
 * block), codes rounded to nearest, ties to even (the rule of
 * mxgemm_mx_quantize).
 *
 * Asynchronous on `stream`; all buffers caller-owned device memory, outputs
 * not overlapping the inputs.  Errors (before any work): MXG_ERR_SHAPE
 * (head_dim not a multiple of 32 or above 256, qk_rope odd or above
 * head_dim or 128, sizes too large), MXG_ERR_ALIGN (tokens % 32, or Y, the
 * code buffers, cos or sin not 16-byte aligned), MXG_ERR_NULL,
 * MXG_ERR_DEVICE.  tokens or
 * num_heads == 0 queues nothing and returns MXG_OK.
 */
int mxgemm_proj_rope_mxfp8(const float* Y, const uint16_t* cos_bf16, const uint16_t* sin_bf16, uint8_t* row_codes,
                           uint8_t* row_scales, uint8_t* col_codes, uint8_t* col_scales, int64_t tokens,
                           int64_t num_heads, int64_t head_dim, int64_t qk_rope, void* stream);

/* ---------------------------------------------------------------------------
 * Projection operators on float32 scales per block of 128, rotary positions and
 * per-head norms.  Data types of plain (unquantised) tensors: */
enum {
  MXG_DT_F32 = 0,  /* float32  */
  MXG_DT_BF16 = 1, /* bfloat16 */
  MXG_DT_F16 = 2   /* float16  */
};

/* a flag of all of them */
enum {
  /* The caller vouches that every buffer is memory of the current device: the
     library does not ask HIP where each one lives (as a plan's execute does not;
     0.25 us of host time per buffer). */
  MXG_TRUSTED_POINTERS = 1073741824 /* 2^30 */
};

/* flags of mxgemm_block128_quantize */
enum {
  MXG_QUANT_SQUARE = 1u, /* blocks of 128x128 instead of 1x128 / 128x1        */
  MXG_QUANT_POW2 = 2u    /* scales are powers of two                          */
};

/*
 * mxgemm_block128_quantize -- 8-bit codes with one float32 scale per block of
 * 128, the operands of mxgemm_block128.  For every block with largest
 * magnitude a (taken as 448 * 2^-100 if it is smaller):
 *
 *   scale = a / FMAX,  code = rne(x FMAX / a)             FMAX 448 or 57344
 *
 * with the scale rounded to float32 and the code nearest to the exact quotient,
 * or, with MXG_QUANT_POW2, scale = 2^e with e the smallest integer giving
 * FMAX * 2^e >= a and code = rne(x * 2^-e).
 *
 *   X  : (L, M, K) of x_dtype, K contiguous, rows ldx >= K elements apart,
 *        batches M * ldx apart.
 *   Q  : (L, M, K16) codes in blocks of 1 x 128 along K, K16 = K rounded up to
 *        16; codes past K are zero.  S: (L, ceil(K/128), M) scales.
 *   QT : (L, K, M16) codes of the transpose in blocks of 128 along M, codes past
 *        M zero: the operand of a product that contracts over M.
 *        ST: (L, ceil(M/128), K) scales.
 *   MXG_QUANT_SQUARE: one scale per 128 x 128 block; S is (L, ceil(M/128),
 *        ceil(K/128)), ST its transpose (L, ceil(K/128), ceil(M/128)), and QT
 *        the transpose of Q's codes.
 * Q and S, or QT and ST, may both be NULL (not wanted); X is read once either
 * way.  A block that holds a NaN or an infinity gets a scale that is not
 * finite and NaN codes (those past K and M in it too), so everything it touches
 * in the product is NaN.
 *
 * Asynchronous on `stream`, allocates nothing; outputs must not overlap X.
 * Errors (before any work): MXG_ERR_SHAPE (negative or too large sizes, ldx <
 * K), MXG_ERR_FMT (x_dtype, or fmt not E4M3 / E5M2), MXG_ERR_FLAGS,
 * MXG_ERR_NULL (X, no output at all, or codes without scales), MXG_ERR_ALIGN
 * (Q or QT not 16-byte aligned, X or scales not aligned to their elements),
 * MXG_ERR_DEVICE, MXG_ERR_LAUNCH.  M, K or L == 0 queues nothing.
 */
int mxgemm_block128_quantize(const void* X, int64_t ldx, void* Q, float* S, void* QT, float* ST, int64_t M, int64_t K,
                             int64_t L, int x_dtype, int fmt, unsigned flags, void* stream);

/* flags of mxgemm_block128 */
enum {
  MXG_B128_B_ROWS = 1u,    /* B in blocks of 1 x 128 (SB as SA) instead of 128 x 128 */
  MXG_B128_ACCUMULATE = 2u /* C += product; float32 C                               */
};

/*
 * mxgemm_block128 -- the product of two operands of mxgemm_block128_quantize:
 *
 *   C[m,n] = sum_j SA[j,m] SB(j,n) sum_{k in block j} dec(A[m,k]) dec(B[n,k])
 *
 * over the blocks j of 128 consecutive K elements.
 *   A  : (L, M, K) codes, B: (L, N, K) codes, contiguous, K % 16 == 0.
 *   SA : (L, ceil(K/128), M) float32.
 *   SB : (L, ceil(N/128), ceil(K/128)) float32, or with MXG_B128_B_ROWS
 *        (L, ceil(K/128), N).
 *   C  : (L, M, N) of c_dtype, rows ldc >= N elements apart, batches M * ldc
 *        apart.
 * A layer's forward product, its input gradient (B the transposed weight codes
 * with the transposed scales) and its weight gradient (both operands in blocks
 * along the tokens, float32 C) are all of this form.
 *
 * Accuracy.  A float32 C takes exact products: codes are widened to bfloat16
 * (exact) and the sums are float32.  A 16-bit C takes the matrix cores' 8-bit
 * products, whose sums inside a group of 8 K elements drop what lies 2^-13
 * below the largest: 1.4e-5 of the result in 2-norm on normal data (measured),
 * against 1.6e-3 and 2e-4 that the rounding to bfloat16 / float16 costs, but in
 * the worst case 2^-10 of sum |A||B|, which where terms cancel is more than
 * that rounding.  Where this matters, take a float32 C and round it.  Sums
 * across groups and blocks are float32.  SA SB is rounded to float32 before it
 * multiplies a block's sum, so it should lie in float32's normal range.
 *
 * Workspace: device memory of at least mxgemm_block128_workspace_bytes, 16-byte
 * aligned, overwritten; NULL where that is 0.
 *
 * Asynchronous on `stream`, allocates nothing.  Errors (before any work):
 * MXG_ERR_SHAPE (negative or too large sizes, ldc < N, a short workspace),
 * MXG_ERR_FMT (formats or c_dtype), MXG_ERR_FLAGS (unknown, or ACCUMULATE
 * without a float32 C), MXG_ERR_ALIGN (K % 16, A or B not 16-byte aligned, C
 * or scales not aligned to their elements, workspace), MXG_ERR_NULL,
 * MXG_ERR_DEVICE, MXG_ERR_LAUNCH.  K == 0 gives C = 0 (C unchanged with
 * ACCUMULATE); M, N or L == 0 queues nothing.
 */
int mxgemm_block128(const void* A, const float* SA, const void* B, const float* SB, void* C, int64_t ldc, int64_t M,
                    int64_t N, int64_t K, int64_t L, int a_fmt, int b_fmt, int c_dtype, unsigned flags, void* workspace,
                    size_t workspace_bytes, void* stream);
size_t mxgemm_block128_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t L, int c_dtype);

/* activations */
enum {
  MXG_ACT_NONE = 0,
  MXG_ACT_RELU = 1,      /* max(z, 0)                                          */
  MXG_ACT_SILU = 2,      /* z s(z), s(u) = 1 / (1 + e^-u)                      */
  MXG_ACT_GELU = 3,      /* z P(z), P the normal distribution                  */
  MXG_ACT_GELU_TANH = 4  /* z s(2 sqrt(2/pi) (z + 0.044715 z^3))               */
};

/*
 * What follows a product: with p its value at (m, n),
 *
 *   z = p + bias[n],   y = act(z) * gate[m,n] + residual[m,n]
 *
 * in float32, y and z rounded once each.  Every tensor may be NULL (not there):
 *   bias     : (N), of C's type, or float32 with bias_dtype = MXG_DT_F32.
 *   gate, residual : (M, N) of C's type, rows ldgate / ldresidual >= N elements
 *              apart.  Either may be C itself with C's row distance.
 *   preact   : (M, N) of C's type, rows ldpreact >= N apart: receives z, from
 *              which mxgemm_activation_backward makes the gradients.
 * No row distance exceeds 2^21.  Other overlaps of C and preact with each other
 * or with what the call reads are refused (MXG_ERR_SHAPE).
 */
typedef struct {
  const void* bias;
  const void* gate;
  const void* residual;
  void* preact;
  int64_t ldgate, ldresidual, ldpreact;
  int activation, bias_dtype;
} mxgemm_ends_t;

/*
 * mxgemm_block128_linear -- C = y of the product of mxgemm_block128 (one batch,
 * B in blocks of 128 x 128) and what follows it, in one pass where K is not
 * divided.  Arguments, accuracy of the product and errors as there; ends must
 * not be NULL; flags: none of mxgemm_block128's.  Workspace:
 * mxgemm_block128_workspace_bytes(M, N, K, 1, c_dtype).  Errors besides:
 * MXG_ERR_FMT (activation, bias_dtype), MXG_ERR_SHAPE (a row distance),
 * MXG_ERR_ALIGN (a tensor not aligned to its elements).  K == 0 takes p = 0.
 */
int mxgemm_block128_linear(const void* A, const float* SA, const void* B, const float* SB, void* C, int64_t ldc, int64_t M,
                           int64_t N, int64_t K, int a_fmt, int b_fmt, int c_dtype, const mxgemm_ends_t* ends, unsigned flags,
                           void* workspace, size_t workspace_bytes, void* stream);

/*
 * mxgemm_activation_backward -- the gradients of y = act(z) gate + residual,
 * z = p + bias, from that of y: with act' the activation's derivative (relu's 0
 * at 0),
 *
 *   dz = dy * gate * act'(z),  dgate = dy * act(z),  dbias[n] = sum_m dz[m,n]
 *
 * in float32, dz and dgate rounded once, dbias from dz before its rounding.
 * (dp is dz, and the residual's gradient is dy.)
 *   DY, Z, GATE, DZ, DGATE : (M, N) of `dtype`, rows strides[0..4] >= N elements
 *            apart.  GATE and DGATE may both be NULL (no gate).  DZ and DGATE may each
 *            be one of DY, Z, GATE with the same row distance; other overlaps
 *            of what is written are refused (MXG_ERR_SHAPE).
 *   DBIAS : (N) float32, overwritten, or NULL.  Summed in a fixed order: equal
 *            calls give equal bits.
 *   workspace : device memory of at least
 *            mxgemm_activation_backward_workspace_bytes(M, N), 16-byte aligned,
 *            overwritten; needed for DBIAS only, NULL where that is 0.
 * Asynchronous, allocates nothing.  Errors (before any work): MXG_ERR_SHAPE
 * (sizes, a row distance, a short workspace), MXG_ERR_FMT (activation, dtype),
 * MXG_ERR_FLAGS, MXG_ERR_NULL, MXG_ERR_ALIGN, MXG_ERR_DEVICE, MXG_ERR_LAUNCH.
 * M == 0 makes DBIAS zero; N == 0 queues nothing.
 */
int mxgemm_activation_backward(const void* DY, const void* Z, const void* GATE, void* DZ, void* DGATE, float* DBIAS,
                               const int64_t* strides, int64_t M, int64_t N, int activation, int dtype, unsigned flags,
                               void* workspace, size_t workspace_bytes, void* stream);
size_t mxgemm_activation_backward_workspace_bytes(int64_t M, int64_t N);

/* flags of the entry points on rows in groups */
enum {
  MXG_GROUP_OFFSETS64 = 256u,  /* offsets are int64 instead of int32                */
  MXG_GROUP_ZERO_REST = 512u,  /* mxgemm_block128_grouped: zeros in C's rows of no group */
  MXG_GROUP_ZERO_PREACT = 1024u /* the same in preact                               */
};

/*
 * Rows in groups.  T rows lie in order of the E groups (experts) they belong
 * to: group e holds rows offsets[e] <= t < offsets[e + 1].  offsets (E + 1), int32 or
 * int64 (MXG_GROUP_OFFSETS64), is device memory that the kernels read: no size is known to the
 * host.  A group may have no rows; rows before offsets[0] and behind offsets[E]
 * belong to none.  Offsets must not decrease and lie within 0 .. T; others give
 * wrong results, not accesses out of bounds.  E <= 1024, T <= 2^24.
 *
 * Along the rows each group has blocks of 128 of its own, the last one filled
 * up with zeros.  mxgemm_group_blocks(T, E) is the number of blocks that E groups
 * of T rows in all can have, (T + 127 min(T, E)) / 128 rounded down (0 for E = 0): group
 * e's blocks follow those of the groups before it, and what is behind the last
 * group's is zero.
 */
int64_t mxgemm_group_blocks(int64_t T, int64_t E);

/*
 * mxgemm_block128_quantize_grouped -- mxgemm_block128_quantize with blocks along
 * the rows that start at each group's first row.
 *   X  : (T, K) of x_dtype, rows ldx apart.
 *   Q, S : codes (T, K16) and scales (ceil(K/128), T) in blocks of 1 x 128, of all
 *        rows; both may be NULL (not wanted).
 *   QT : (K, 128 G) codes of the transpose, G = mxgemm_group_blocks(T, E); ST: (G, K)
 *        scales.  Codes and scales of blocks that no group has are zero.
 * flags: MXG_QUANT_POW2, MXG_GROUP_OFFSETS64.  Errors as there, and
 * MXG_ERR_SHAPE for E or T past their limits, MXG_ERR_NULL without offsets, or QT
 * or ST where G > 0.  T or K == 0 queues nothing.
 */
int mxgemm_block128_quantize_grouped(const void* X, int64_t ldx, const void* offsets, void* Q, float* S, void* QT, float* ST,
                                     int64_t T, int64_t E, int64_t K, int x_dtype, int fmt, unsigned flags, void* stream);

/*
 * mxgemm_block128_grouped -- the product of every group's rows with the group's
 * own B, and what follows it: for rows t of group e
 *
 *   p[t,n] = sum_j SA[j,t] SB[e,n/128,j] sum_{k in block j} dec(A[t,k]) dec(B[e,n,k])
 *
 *   A  : (T, K) codes, SA: (ceil(K/128), T); B: (E, N, K) codes, SB: (E,
 *        ceil(N/128), ceil(K/128)); contiguous, K % 16 == 0, K > 0.
 *   C  : (T, N) of c_dtype, rows ldc >= N apart.  Rows of no group are left as
 *        they were, or made zero with MXG_GROUP_ZERO_REST (in preact with
 *        MXG_GROUP_ZERO_PREACT).
 *   ends : NULL, or activation, gate and preact (bias and residual must be
 *        NULL: MXG_ERR_FLAGS).
 * Accuracy as of mxgemm_block128.  Needs no workspace.  flags: MXG_GROUP_*.
 * Errors as of mxgemm_block128_linear, and MXG_ERR_SHAPE for E or T past their
 * limits and for K == 0.  T or N == 0 queues nothing.
 */
int mxgemm_block128_grouped(const void* A, const float* SA, const void* B, const float* SB, const void* offsets, void* C,
                            int64_t ldc, int64_t T, int64_t E, int64_t N, int64_t K, int a_fmt, int b_fmt, int c_dtype,
                            const mxgemm_ends_t* ends, unsigned flags, void* stream);

/*
 * mxgemm_block128_grouped_weight_gradient -- one product over the rows of each
 * group, of two operands that mxgemm_block128_quantize_grouped has made along
 * the rows with the same offsets:
 *
 *   C[e,m,n] = sum over e's blocks j of SA[j,m] SB[j,n] sum_{t in block j} dec(A[m,t]) dec(B[n,t])
 *
 *   A  : (M, 128 blocks) codes (QT), SA: (blocks, M) (ST); B: (N, 128 blocks), SB:
 *        (blocks, N); blocks = mxgemm_group_blocks(T, E) < 2^16.
 *   C  : (E, M, N) float32, rows ldc >= N apart, groups M * ldc apart; zero for
 *        a group without rows.  MXG_B128_ACCUMULATE: C += product.  It must not
 *        lie on what the call reads (MXG_ERR_SHAPE).
 * Products and sums as in a float32 C of mxgemm_block128.
 *   workspace : device memory of at least
 *        mxgemm_block128_grouped_weight_gradient_workspace_bytes, 16-byte aligned,
 *        overwritten; NULL where that is 0.
 * flags: MXG_GROUP_OFFSETS64, MXG_B128_ACCUMULATE.  Errors as there.  E, M or N
 * == 0 queues nothing; blocks == 0 makes C zero (leaves it with ACCUMULATE).
 */
int mxgemm_block128_grouped_weight_gradient(const void* A, const float* SA, const void* B, const float* SB, const void* offsets,
                                            float* C, int64_t ldc, int64_t blocks, int64_t E, int64_t M, int64_t N,
                                            int a_fmt, int b_fmt, unsigned flags, void* workspace, size_t workspace_bytes,
                                            void* stream);
size_t mxgemm_block128_grouped_weight_gradient_workspace_bytes(int64_t blocks, int64_t E, int64_t M, int64_t N);

/* layouts of the rotary features inside a head */
enum {
  MXG_ROPE_HALF = 0,                /* pairs (i, i + rot/2)                          */
  MXG_ROPE_INTERLEAVED = 1,         /* pairs (2i, 2i + 1)                            */
  MXG_ROPE_INTERLEAVED_TO_HALF = 2  /* pairs (2i, 2i + 1) in, (i, i + rot/2) out     */
};
/* flags of mxgemm_rope, mxgemm_qk_norm_rope and its backward */
enum {
  MXG_ROPE_TRANSPOSE = 1u, /* mxgemm_rope: the transposed map (the gradient)       */
  MXG_ROPE_POS64 = 2u      /* positions are int64 instead of int32                 */
};

/*
 * mxgemm_rope -- rotary positions on the heads of one tensor.  With (a_i, b_i)
 * the i-th pair of a head's rotary features [rot_offset, rot_offset + rot),
 * i < rot / 2, and p the token's position:
 *
 *   a'_i = a_i cos[p,i] - b_i sin[p,i],   b'_i = b_i cos[p,i] + a_i sin[p,i]
 *
 * in float32, rounded once; the other features are copied.
 * MXG_ROPE_TRANSPOSE applies the transposed map: of a gradient of Y it makes
 * the gradient of X (with INTERLEAVED_TO_HALF the halves go in and the
 * interleaved pairs come out).
 *
 *   X, Y      : (T, H, D) of `dtype`, features contiguous, element strides
 *               strides[0..3] = X token, X head, Y token, Y head.  Y may be X
 *               with the same strides; otherwise they must not overlap, and
 *               rows of Y must not overlap each other.
 *   cos, sin  : (table_rows, rot / 2) float32, contiguous.
 *   positions : (T) int32 (int64 with MXG_ROPE_POS64), rows of the tables, or
 *               NULL for token t at position t (then T <= table_rows).  The
 *               rotary features of a token whose position lies outside the
 *               tables become NaN.
 * Errors (before any work): MXG_ERR_SHAPE (negative sizes, D not 1..1024, rot
 * odd or rot_offset + rot > D, sizes or strides too large, rows of Y nearer to
 * each other than D or tokens as far apart as heads, T > table_rows without
 * positions), MXG_ERR_FMT (dtype, layout), MXG_ERR_FLAGS,
 * MXG_ERR_NULL, MXG_ERR_ALIGN (a pointer not aligned to its elements),
 * MXG_ERR_DEVICE, MXG_ERR_LAUNCH.  T or H == 0 queues nothing.  Asynchronous,
 * allocates nothing.
 */
int mxgemm_rope(const void* X, void* Y, const float* cos, const float* sin, const void* positions,
                const int64_t* strides, int64_t T, int64_t H, int64_t D, int64_t rot, int64_t rot_offset,
                int64_t table_rows, int layout, int dtype, unsigned flags, void* stream);

/*
 * mxgemm_qk_norm_rope -- the per-head norm of queries and keys and their rotary
 * positions in one pass: with x a head of Q or K and w its weight WQ or WK,
 *
 *   y = R_p( x * r * w ),   r = 1 / sqrt(mean(x^2) + eps)
 *
 * in float32, rounded once; R_p as in mxgemm_rope (rot may be 0: the norm
 * alone).
 *   Q (T, Hq, D), K (T, Hk, D), YQ, YK alike, of `dtype`; strides[0..7] = token
 *   and head strides of Q, K, YQ, YK.  YQ / YK may be Q / K with the same
 *   strides; no other overlap.  Hk == 0 leaves K, YK and WK out.
 *   WQ, WK : (D) of `dtype`, or float32 with w_dtype = MXG_DT_F32.
 * cos, sin, positions, errors as in mxgemm_rope (MXG_ERR_FMT also for w_dtype).
 */
int mxgemm_qk_norm_rope(const void* Q, const void* K, void* YQ, void* YK, const void* WQ, const void* WK,
                        const float* cos, const float* sin, const void* positions, const int64_t* strides, int64_t T,
                        int64_t Hq, int64_t Hk, int64_t D, int64_t rot, int64_t rot_offset, int64_t table_rows,
                        float eps, int layout, int dtype, int w_dtype, unsigned flags, void* stream);

/*
 * mxgemm_qk_norm_rope_backward -- the gradients of mxgemm_qk_norm_rope: with
 * g the gradient of y, n = x r and u = R_p^T g (the transposed rotation),
 *
 *   dw = sum over tokens and heads of u n,
 *   dx = r (u w - n mean(u w n))
 *
 *   GQ, GK : gradients of YQ, YK; DQ, DK: gradients of Q, K, of `dtype`;
 *            strides[0..11] = token and head strides of GQ, GK, Q, K, DQ, DK.
 *            DQ / DK may be GQ / GK or Q / K with the same strides.
 *   DWQ, DWK : (D) float32, overwritten.  Summed in a fixed order: equal
 *            calls give equal bits.
 *   workspace : device memory of at least
 *            mxgemm_qk_norm_rope_backward_workspace_bytes(T, D), 16-byte
 *            aligned, overwritten.
 * r is recomputed from Q and K, so nothing is kept from the forward pass.
 * Errors as in mxgemm_qk_norm_rope; a short workspace is MXG_ERR_SHAPE.  With
 * T == 0 (or Hq == 0) the weight gradients are zero.
 */
int mxgemm_qk_norm_rope_backward(const void* GQ, const void* GK, const void* Q, const void* K, void* DQ, void* DK,
                                 float* DWQ, float* DWK, const void* WQ, const void* WK, const float* cos,
                                 const float* sin, const void* positions, const int64_t* strides, int64_t T,
                                 int64_t Hq, int64_t Hk, int64_t D, int64_t rot, int64_t rot_offset,
                                 int64_t table_rows, float eps, int layout, int dtype, int w_dtype, unsigned flags,
                                 void* workspace, size_t workspace_bytes, void* stream);
size_t mxgemm_qk_norm_rope_backward_workspace_bytes(int64_t T, int64_t D);

/* mxgemm_strerror -- static text for a status code. No HIP call. */
const char* mxgemm_strerror(int status);

#ifdef __cplusplus
}
#endif

#endif /* MXGEMM_H */
