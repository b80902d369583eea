/*
 * w4a16.h -- C ABI of the GB300 (sm_103a) weight-only INT4 GEMM library (libw4a16.so).
 *
 * The operation (ferrum-kernels 0.8.5 src/backend/cuda/marlin.rs, doc of `marlin_gemm`):
 *     C[M, N] = A[M, K] (fp16) x dequant(B)[K, N],   fp32 accumulation, fp16 output,
 * where B holds 4-bit codes q with one fp16 scale s per group of `group_size` rows of K:
 *     u4b8:  w = (q - 8) * s                  (ferrum-kernels 0.8.4 vllm_marlin.rs, scalar U4B8)
 *     u4:    w = (q - z) * s, z an fp16 zero  (same page, scalar U4; marlin.rs Marlin-MoE `has_zp`)
 * with an optional act-order permutation (marlin.rs, `MarlinWeight::perm`: rows of B are
 * permuted by argsort(g_idx) at load time and the columns of A are gathered by the same
 * permutation at run time).
 *
 * Conventions shared by every entry point
 *   - Pointers named "device" must be CUDA device (or managed) memory; "host" ones host memory.
 *   - fp16 buffers are IEEE binary16, passed as `void*`.
 *   - All matrices are row-major.  The caller owns every allocation and keeps it alive until
 *     the work enqueued on `stream` has finished (marlin.rs, Marlin-MoE raw launch arguments).
 *   - Calls are asynchronous on `stream` and never synchronise, allocate, or fall back to the
 *     CPU.  The stream may be a capturing stream (CUDA graphs).
 *   - Return value: 0 on success, else a staged status `(stage << 16) | detail`, after the
 *     convention of marlin.rs (`marlin_moe_ffi_status`):
 *       stage 1  invalid argument      detail = W4A16_ARG_*
 *       stage 2  unsupported shape     detail = W4A16_ARG_*
 *       stage 3  device query/resource detail = cudaError_t
 *       stage 6  kernel launch         detail = cudaError_t
 *       stage 7  device-side error     detail = W4A16_DEV_* bits (read with w4a16_status)
 *     Argument checks run before any CUDA call, so they work on a machine without a GPU.
 */
#ifndef W4A16_H
#define W4A16_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define W4A16_ABI_VERSION 1

/* Weight types: the scalar ids of ferrum-kernels 0.8.4 vllm_marlin.rs (FERRUM_MARLIN_SCALAR_*). */
#define W4A16_TYPE_U4 4   /* codes with an explicit fp16 zero point per (group, column) */
#define W4A16_TYPE_U4B8 5 /* symmetric codes, zero point 8                              */
#define W4A16_TYPE_FE4M3 8 /* 8-bit FP8 E4M3 ("fn") weights, W8A16: w = e4m3(code) * s,
                              no zero points (scalar FERRUM_MARLIN_SCALAR_FE4M3FN)      */

/* Flags.  Bits 1..3 keep the positions of the page's FERRUM_MARLIN_HAS_ACT_ORDER,
 * FERRUM_MARLIN_IS_K_FULL and FERRUM_MARLIN_HAS_ZERO_POINTS (vllm_marlin.rs). */
#define W4A16_FLAG_ACT_ORDER (1u << 1)  /* g_idx and perm given; A is gathered by perm       */
#define W4A16_FLAG_IS_K_FULL (1u << 2)  /* this call sees the whole K (always true here)     */
#define W4A16_FLAG_HAS_ZP (1u << 3)     /* zeros given; required exactly for W4A16_TYPE_U4   */
#define W4A16_FLAG_FORCE_SIMT (1u << 8) /* run the CUDA-core reference kernel (diagnostics)  */
#define W4A16_FLAG_A_SMEM (1u << 9)     /* stage dequantised weights in shared memory instead
                                           of tensor memory (diagnostics / comparison)       */
#define W4A16_FLAG_FORCE_TC (1u << 10)  /* always use the tcgen05 kernel (diagnostics)      */
#define W4A16_FLAG_FORCE_MMA (1u << 11) /* always use the small-M split-K register-fragment
                                           kernel; M above 64 is then rejected
                                           (unsupported-shape)                               */
#define W4A16_FLAG_STATIC_WEIGHTS (1u << 12) /* b_packed, scales and zeros are not written by the
                                           work that precedes this call on its stream, so the
                                           kernel may start reading them before that work has
                                           finished (it still waits before reading A or
                                           writing C or the workspace).  Without the flag
                                           weights are only prefetched into L2 early.        */
#define W4A16_FLAG_FORCE_SLICE (1u << 13) /* always use the small-M column-slice kernel (each
                                           CTA owns 16-column slices over all of K, no
                                           split-K); M above 32 or a group size that is not
                                           -1 or a multiple of 64 is then rejected
                                           (unsupported-shape)                               */

#define W4A16_FLAG_SWIGLU (1u << 14) /* gated FFN epilogue: the weight's 2I columns are gate
                                           and up projections interleaved by
                                           w4_gate_up_interleave, and C receives
                                           H[M][I] = silu(A Wg) * (A Wu) (ldc >= I) instead of
                                           the product (tcgen05 kernel only: _FORCE_SIMT,
                                           _FORCE_MMA and _FORCE_SLICE are rejected)        */
#define W4A16_FLAG_GEGLU (1u << 15)  /* the same with gelu_tanh(x) = x/2 (1 + tanh(sqrt(2/pi)
                                           (x + 0.044715 x^3))) in place of silu; exclusive
                                           with W4A16_FLAG_SWIGLU.  Both activations are
                                           evaluated in fp32 as x sigmoid(y) (y = x for silu,
                                           2 sqrt(2/pi) (x + 0.044715 x^3) for gelu_tanh)
                                           with a fast exponential: within the gated
                                           tolerance, not correctly rounded               */
#define W4A16_FLAG_BF16 (1u << 16)   /* a, scales, zeros and c are bfloat16 instead of fp16
                                           (marlin.rs declares bf16 A and C for its
                                           `ferrum_vllm_marlin_moe_mxfp4_bf16` entry point;
                                           here with the 4-bit codes).  4-bit weight types
                                           only (not W4A16_TYPE_FE4M3); the tcgen05 kernel and,
                                           for group_size -1 or a multiple of 64, the small-M
                                           kernels (_FORCE_SIMT is rejected, _FORCE_MMA with
                                           other groups is unsupported-shape; the default choice
                                           sends those groups to the tcgen05 kernel).  (q - z)
                                           is exact in bf16 for integer
                                           zero points, the product with the scale is rounded
                                           once to bf16 (8 significant bits), products sum in
                                           fp32 and C is rounded once to bf16               */

#define W4A16_FLAG_ROPE_ADJACENT (1u << 17) /* rotary appends: a pair is values 2i and 2i + 1 of the
                                           rotated part, not i and rot_dim / 2 + i          */
#define W4A16_FLAG_MOE_RENORM (1u << 18) /* w4a16_moe_layer: the chosen experts' probabilities are
                                           divided by their sum                             */

/* Detail codes of stage-1/2 statuses. */
#define W4A16_ARG_NULL 1        /* a required pointer is NULL                                  */
#define W4A16_ARG_ALIGN 2       /* a pointer or leading dimension breaks its alignment rule    */
#define W4A16_ARG_SHAPE 3       /* a size is negative, or K % 128 / N % 256 is violated        */
#define W4A16_ARG_FLAGS 4       /* flags disagree with the pointers or the weight type         */
#define W4A16_ARG_OVERFLOW 5    /* an extent does not fit the index types                      */
#define W4A16_ARG_WORKSPACE 6   /* workspace missing or smaller than w4a16_*_workspace_size    */
#define W4A16_ARG_GROUP 7       /* group_size not -1 or a positive multiple of 16 dividing K  */
#define W4A16_ARG_TYPE 8        /* unknown weight type                                         */
#define W4A16_ARG_SCHEDULE 9    /* grouped schedule sizes out of range                         */
#define W4A16_ARG_SCRATCH 10    /* w4a16_gemm_noalloc: the call needs more scratch than it has */
#define W4A16_ARG_QZERO 11      /* a packed GPTQ zero code of 15 (its zero point would be 16)  */

/* Device-side error bits (stage 7), accumulated in the workspace status word. */
#define W4A16_DEV_TIMEOUT 1     /* a bounded wait inside a kernel ran out; the workspace's
                                   split-tile counters may then be left non-zero, so zero-fill
                                   the whole workspace again before its next use             */
#define W4A16_DEV_PERM 2        /* a perm entry was outside [0, K)                             */
#define W4A16_DEV_GIDX 4        /* g_idx[perm[i]] != i / group_size (groups not equal-sized)   */
#define W4A16_DEV_SCHEDULE 8    /* a CSR entry was outside its range                           */
#define W4A16_DEV_ZERO 16       /* w4a16_zero_points_check: a zero point is not an integer in
                                   [0, 15]                                                   */
#define W4A16_DEV_POSITION 32   /* rotary appends: a position outside [0, max_pos)             */
#define W4A16_DEV_SLOT 64       /* rotary appends: a slot past the cache                       */
#define W4A16_DEV_LENGTH 128    /* paged attentions: a length outside [0, max_pages x page]    */
#define W4A16_DEV_PAGE 256      /* paged attentions: a page number outside [0, n_pages)        */
#define W4A16_DEV_SETTING 512   /* w4a16_sample: a row's settings outside their ranges         */

/* ------------------------------------------------------------------------------------------
 * Packed tile layout (this library's own; the pages only say the kernel layout is a
 * permutation of the GPTQ words with the same byte count: marlin.rs module doc,
 * vllm_marlin.rs `ferrum_vllm_gptq_marlin_repack` doc).
 *
 * Input ("GPTQ") layout: int32 [K/8][N]; word (r, n) holds the codes of rows 8r..8r+7 of
 * column n, row 8r+i at bits 4i..4i+3 (low nibble first).
 *
 * Tile layout: K*N/8 int32 words.  "Sorted row" r is logical row perm[r] when a permutation
 * is given, else r.  Tile (nt, kb) covers sorted rows kb*64 .. kb*64+63 and columns
 * nt*128 .. nt*128+127 and occupies the 1024 words starting at (nt * K/64 + kb) * 1024.
 * Word h*512 + c*4 + j of a tile (h in {0,1}, c in [0,128), j in [0,4)) holds eight codes
 * of column nt*128 + c: for p in 0..3 and e in 0..1, the code of sorted row
 * kb*64 + h*32 + 8p + 2j + e sits at bit 4p + 16e.  One mask then turns the row pair
 * (8p + 2j, 8p + 2j + 1) into two fp16 lanes, a word is exactly what one thread of an
 * m16n8k16 register fragment needs for two 16-row k steps, the four words of one
 * (half, column) are one 16-byte load of 32 rows, and each 64x128 tile is one contiguous
 * 4 KiB bulk copy.
 * ---------------------------------------------------------------------------------------- */

/* GPTQ words -> tile layout.
 *   qweight   device int32 [K/8][N], read only
 *   perm      device int32 [K] or NULL; sorted row r takes logical row perm[r]
 *   b_packed  device int32 [K*N/8], written; must not overlap qweight
 *   status    device int32 or NULL; W4A16_DEV_PERM is OR-ed in when a perm entry is out of
 *             range (that row's codes are then written as 0)
 *   k, n      K % 128 == 0, N % 256 == 0 (marlin.rs module doc), both > 0
 * Alignment: qweight, b_packed 16 bytes; perm, status 4 bytes.
 * Source: vllm_marlin.rs `ferrum_vllm_gptq_marlin_repack` (GPTQ -> kernel tiles, has_perm). */
int w4_repack(const int32_t *qweight, const int32_t *perm, int32_t *b_packed, int32_t *status,
              int k, int n, cudaStream_t stream);

/* Gate/up interleave for the gated FFN epilogue (W4A16_FLAG_SWIGLU / _GEGLU).
 * transformer.rs, `encode_compressed_tensors_dense_swiglu` and the U4B8 GeGLU pipeline beside
 * it: gate = A Wg and up = A Wu are two W4A16 GEMMs over the same A, then h = act(gate) * up
 * feeds the down projection.  Here both run as one GEMM over a [K][2I] weight whose columns
 * alternate in blocks of 16 -- destination column 32b + r is gate column 16b + r for r < 16
 * and up column 16b + r - 16 for r >= 16 -- so each 128-column tile of the kernel holds 64
 * features' gate and up sums side by side and its epilogue writes act(gate) * up.
 * This permutes the columns of a row-major [rows][n2] array, n2 = 2I, from the planar order
 * (the I gate columns, then the I up columns) into that order; apply it to the GPTQ words
 * [K/8][2I] (elem_bytes 4) before w4_repack, and to the scales and zeros [G][2I]
 * (elem_bytes 2).  For w4a16_gemm, I must be a multiple of 128 (so 2I % 256 == 0).
 *   src, dst  device arrays of rows x n2 elements, not overlapping, aligned to elem_bytes
 *   n2        a positive multiple of 32;  elem_bytes 2 or 4 */
int w4_gate_up_interleave(const void *src, void *dst, int rows, int n2, int elem_bytes,
                          cudaStream_t stream);

/* FP8 E4M3 weights (W8A16).  Input: int32 [K/4][N], each word holding four K-consecutive E4M3
 * codes of one column, row 4r+i at byte i (little-endian) -- the input ABI of vllm_marlin.rs
 * `vllm_fp8_marlin_repack_raw_bits`; a checkpoint's row-major [N][K] bytes are transposed into
 * it.  Output (this library's FP8 tile layout, K*N/4 words): tile (nt, kb) covers rows
 * kb*64 .. kb*64+63 and columns nt*128 .. nt*128+127 at word (nt * K/64 + kb) * 2048; word
 * q*512 + c*4 + t (q, t in 0..3, c in 0..127) is the input word of rows kb*64 + 16q + 4t .. +3
 * of column nt*128 + c, so each thread of the kernel reads its column's 64 rows as four 16-byte
 * loads.  K % 128 == 0, N % 256 == 0; 16-byte aligned; the buffers must not overlap.
 * W4A16_TYPE_FE4M3 GEMMs (w4a16_gemm, _grouped, _moe_blocks) take these tiles, fp16 scales
 * [G][N] with group_size -1 or a positive multiple of 64 dividing K (the pages' FP8 Marlin
 * takes -1 or 128), no zero points, no act-order, fp16 activations.  They run on the
 * column-slice kernel for M <= 16 with N / 16 >= the SM count (W4A16_FLAG_FORCE_SLICE forces it;
 * M above 16 is then unsupported-shape)
 * and otherwise on the tcgen05 kernel; forcing the split-K small-M or the CUDA-core kernel is
 * rejected (those are 4-bit only).  Each code becomes its exact fp16 value
 * (cvt.rn.f16x2.e4m3x2); the product with the scale is rounded once. */
int w8_repack(const int32_t *qweight, int32_t *b_packed, int k, int n, cudaStream_t stream);

/* FP8 tiles -> the [K/4][N] input words (the inverse of w8_repack). */
int w8_unpack(const int32_t *b_packed, int32_t *qweight, int k, int n, cudaStream_t stream);

/* Tile layout -> GPTQ words of the sorted rows (the inverse of w4_repack; a permutation
 * applied at repack time is not undone).  Same shape, alignment and overlap rules. */
int w4_unpack(const int32_t *b_packed, int32_t *qweight, int k, int n, cudaStream_t stream);

/* Workspace bytes that w4a16_gemm needs for these sizes on a device with `num_sms`
 * multiprocessors (num_sms <= 0: query the current device; returns 0 if that fails or the
 * sizes are invalid).  The workspace holds a status word, the split-K tile counters, the
 * fp32 partial tiles and, with act-order, the gathered copy of A.  It must be zero-filled
 * once after allocation; the kernels leave it ready for the next call, of these or any other
 * sizes that need no more bytes, dense or grouped (counters reset themselves), so no per-call
 * memset is needed.  The size follows the token tile's height and can fall as m rises (257 rows
 * need more than 448): take the largest of the row counts in use.  The one exception: after w4a16_status has
 * reported W4A16_DEV_TIMEOUT, a CTA that gave up may have left its tile counters part-way, and
 * the next call would then reduce the wrong partials -- zero-fill the whole workspace again
 * (cudaMemsetAsync over its size) before reusing it.  Calls that run concurrently need
 * separate workspaces. */
size_t w4a16_workspace_size(int m, int n, int k, int group_size, unsigned flags, int num_sms);

/* The W4A16 GEMM.
 *   a          device fp16 [M][lda], lda >= K, lda % 8 == 0, 16-byte aligned
 *   b_packed   device int32 tile layout of the [K][N] codes (from w4_repack)
 *   c          device fp16 [M][ldc], ldc >= N, ldc % 8 == 0; written
 *   scales     device fp16 [G][N], G = K / group_size (1 for group_size -1)
 *   zeros      device fp16 [G][N] integer zero points in [0, 15], or NULL (u4b8).  The
 *              kernels form (q - z) exactly by integer arithmetic inside fp16 and do not check
 *              the values: a zero point that is not an integer in [0, 15] gives unspecified
 *              results (w4a16_zero_points_check reports such values)
 *   g_idx      device int32 [K] or NULL: group of each logical row (act-order)
 *   perm       device int32 [K] or NULL: the permutation that w4_repack applied, one that
 *              sorts g_idx (argsort; any order of the rows inside a group is accepted).
 *              Groups must be equal-sized (g_idx[perm[i]] == i/group_size, as GPTQ's desc_act
 *              layout is); a violation sets W4A16_DEV_GIDX.
 *   workspace  device, >= w4a16_workspace_size(...) bytes, 256-byte aligned, zero-filled once
 *   m          >= 0 (0 is a no-op);  n % 256 == 0;  k % 128 == 0
 *   group_size -1 (one group) or a positive multiple of 16 dividing K
 *              (transformer.rs `marlin_num_groups`; marlin.rs Marlin-MoE validation)
 *   weight_type W4A16_TYPE_U4B8 (zeros NULL), W4A16_TYPE_U4 (zeros and W4A16_FLAG_HAS_ZP) or
 *              W4A16_TYPE_FE4M3 (FP8 tiles from w8_repack; zeros NULL, see there)
 *   flags      W4A16_FLAG_*; ACT_ORDER exactly when g_idx and perm are given.  With
 *              W4A16_FLAG_SWIGLU or _GEGLU, N = 2I columns of interleaved gate/up weights
 *              (w4_gate_up_interleave) and c receives H [M][ldc], ldc >= I, with
 *              H[m][f] = act(gate[m][f]) * up[m][f] computed in fp32 from the fp32 sums and
 *              rounded once to fp16
 * Kernel choice (unless a W4A16_FLAG_FORCE_* flag picks one): M <= 8 -- and M <= 32 while
 * N / 16 <= 2 x the SM count -- with group_size -1 or a multiple of 64 and N / 16 >= the SM
 * count runs the column-slice kernel (no split-K); the rest of M <= 32 the split-K
 * register-fragment kernel; larger M the tcgen05 kernel.  All three give results within the
 * same tolerance of the exact product; they round differently, so their bits may differ.
 * Results are deterministic: a fixed reduction order makes repeated calls on the same device
 * with the same sizes and flags bit-identical.  Tuning overrides read once from the
 * environment (W4A16_STAGE_BLOCKS, W4A16_DECODE_ROWS, W4A16_DECODE_GRID, W4A16_TILE_TOKENS,
 * W4A16_SLICE, W4A16_PAIR_HALF; unset by default) change the kernel choice and tiling, and with them the
 * rounding order: results stay within tolerance but their bits can differ between processes
 * whose environments differ. */
int w4a16_gemm(const void *a, int lda, const int32_t *b_packed, void *c, int ldc,
               const void *scales, const void *zeros, const int32_t *g_idx, const int32_t *perm,
               void *workspace, size_t workspace_bytes, int m, int n, int k, int group_size,
               int weight_type, unsigned flags, cudaStream_t stream);

/* Which kernel w4a16_gemm runs for these sizes and flags on a device with `num_sms`
 * multiprocessors (num_sms <= 0: the current device): 0 the tcgen05 kernel, 1 the split-K
 * small-M kernel, 2 the column-slice small-M kernel; -1 for sizes or flags that w4a16_gemm
 * rejects.  Host code only (with num_sms > 0 it touches no GPU).  For tests and benchmarks:
 * the pages check the tile geometry a launch picked (marlin.rs, the profile-sink test of the
 * vLLM Marlin-MoE path). */
int w4a16_kernel_for(int m, int n, int k, int group_size, unsigned flags, int num_sms);

/* Device scratch of w4a16_gemm_noalloc, per GPU that loads the library (held until exit). */
#define W4A16_NOALLOC_SCRATCH_BYTES (32u * 1024u * 1024u)

/* w4a16_gemm without a workspace argument, for callers that cannot allocate device memory
 * (code running inside a host callback or an allocator hook, under a framework's sealed
 * memory pool, or in a plug-in whose host offers neither an allocator nor a workspace).  It
 * allocates nothing: the scratch that w4a16_gemm keeps in the caller's workspace lives in a
 * fixed device array of W4A16_NOALLOC_SCRATCH_BYTES inside the library.  The pages have no
 * counterpart of this entry point; it is this library's own.
 *   Arguments as w4a16_gemm, minus workspace / workspace_bytes, plus
 *   status_out  device int32 or NULL, 4-byte aligned: receives (stream-ordered) the call's
 *               device-side error bits (W4A16_DEV_*), 0 when all went well
 * It holds the tcgen05 kernel's token tiles to at most 192 rows (w4a16_gemm goes up to 256),
 * so that their partial-tile slots stay small; M above 192 then runs in tiles of 192 rows, a
 * little slower than w4a16_gemm where that would pick taller tiles.  The scratch a call needs
 * is the status header, one counter per CTA, two fp32 partial slots per CTA (SM count
 * x tile rows x 128 columns each) and, with act-order, the copy of A (M*K*2 bytes); a call for
 * which these exceed W4A16_NOALLOC_SCRATCH_BYTES (an act-order call with a large M*K, a very
 * large M, or a part with many more SMs) returns stage 2 with detail W4A16_ARG_SCRATCH and
 * launches nothing.
 * The first call on a device looks up the array's device address (once per device, cached
 * for the life of the process); make that first call before any stream capture.  A
 * cudaDeviceReset makes the cached address stale: calling this entry point after one is not
 * supported.  Each call clears the status word and tile
 * counters it needs on `stream` before its kernels run.  All calls on one device share the
 * array: calls whose work overlaps on the GPU (other streams, other host threads) race and
 * produce wrong results, so serialise them. */
int w4a16_gemm_noalloc(const void *a, int lda, const int32_t *b_packed, void *c, int ldc,
                       const void *scales, const void *zeros, const int32_t *g_idx,
                       const int32_t *perm, int32_t *status_out, int m, int n, int k,
                       int group_size, int weight_type, unsigned flags, cudaStream_t stream);

/* Workspace bytes for w4a16_gemm_grouped (same rules as w4a16_workspace_size). */
size_t w4a16_grouped_workspace_size(int n_pairs, int n_active, int n, int k, int group_size,
                                    unsigned flags, int num_sms);

/* Grouped (MoE) W4A16 GEMM over an expert-major CSR schedule (memra-engine mmq_ffi.rs,
 * `ExpertCsr`): for every active expert i (ex_ids[i], strictly increasing) and every pair p in
 * ex_pairs[ex_off[i] .. ex_off[i+1]):
 *     y[p][:] = a[pair_tok[p]][:] x dequant(B_{ex_ids[i]})
 * Output rows are pair-major; no routing weight is applied.
 *   a             device fp16 [n_tokens][lda]
 *   b_packed_stack device int32, expert e's tiles at word e*K*N/8
 *   y             device fp16 [n_pairs][ldy]
 *   scales_stack  device fp16, expert e's [G][N] scales at element e*G*N; zeros_stack alike
 *   ex_ids        device int32 [n_active];  ex_off device int32 [n_active+1];
 *   ex_pairs      device int32 [n_pairs];   pair_tok device int32 [n_pairs]
 *   n_active      1..W4A16_MAX_SEGMENTS; n_experts bounds ex_ids
 * Act-order is not supported here (W4A16_FLAG_ACT_ORDER is rejected), and every call runs the
 * tcgen05 kernel (W4A16_FLAG_FORCE_SIMT, _FORCE_MMA and _FORCE_SLICE are rejected).  With
 * W4A16_FLAG_SWIGLU / _GEGLU the experts' weights are interleaved gate/up projections of
 * N = 2I columns and y receives [n_pairs][ldy], ldy >= I, of act(gate) * up, as for
 * w4a16_gemm.
 * Out-of-range schedule entries are skipped and reported as W4A16_DEV_SCHEDULE. */
#define W4A16_MAX_SEGMENTS 1024
int w4a16_gemm_grouped(const void *a, int lda, const int32_t *b_packed_stack, void *y, int ldy,
                       const void *scales_stack, const void *zeros_stack, const int32_t *ex_ids,
                       const int32_t *ex_off, const int32_t *ex_pairs, const int32_t *pair_tok,
                       int n_active, int n_experts, int n_pairs, int n_tokens, int n, int k,
                       int group_size, int weight_type, unsigned flags, void *workspace,
                       size_t workspace_bytes, cudaStream_t stream);

/* ------------------------------------------------------------------------------------------
 * Block-routed MoE: the vLLM Marlin-MoE routing interface (ferrum-kernels 0.8.5 marlin.rs,
 * `ferrum_vllm_marlin_moe_f16` and `marlin_gemm_moe_vllm`), on the same tcgen05 kernel as
 * w4a16_gemm_grouped.  Rows are flattened (token, slot) ids, id = token * top_k + slot:
 *   sorted_token_ids  [num_tokens_past_padded] ids listed per expert, each expert's run
 *                     padded to a multiple of moe_block_size with the sentinel prob_m * top_k
 *   expert_ids        [num_tokens_past_padded / moe_block_size] expert of each block; with
 *                     is_ep, -1 marks an expert another rank holds (the block is skipped)
 *   num_tokens_past_padded  one device int32, the padded length (read on the device, so the
 *                     call needs no host synchronisation)
 * and for every non-sentinel row r of block b:
 *     c[id][:] = a[id / top_k][:] x dequant(B_{expert_ids[b]})   (x topk_weights[id] when
 *     mul_topk_weights is 1), rounded once to fp16;
 * rows of c that no entry names are not written.
 * ---------------------------------------------------------------------------------------- */
#define W4A16_MOE_MAX_BLOCKS 4096

/* Host builder of the routing above (vLLM's `moe_align_block_size`, as marlin.rs's doc has the
 * caller run it first): topk_ids [m * top_k] host int32, token-major (id t * top_k + j is token
 * t's j-th expert).  Experts in increasing order, each expert's ids in increasing order, an
 * expert with no ids gets no block.  sorted_token_ids needs `capacity` entries
 * (m * top_k + n_experts * (block_size - 1) always suffices), expert_ids capacity / block_size.
 * Returns num_tokens_past_padded, or -1 on an expert id out of range, a too small capacity or
 * bad sizes. */
int w4a16_moe_align_block_size(const int32_t *topk_ids, int m, int top_k, int n_experts,
                               int block_size, int capacity, int32_t *sorted_token_ids,
                               int32_t *expert_ids);

/* Workspace bytes for w4a16_gemm_moe_blocks (same rules as w4a16_workspace_size). */
size_t w4a16_moe_blocks_workspace_size(int max_padded, int moe_block_size, int n_experts, int n,
                                       int k, int group_size, unsigned flags, int num_sms);

/* The block-routed grouped GEMM.
 *   a               device fp16 [prob_m][lda]
 *   b_packed_stack, scales_stack, zeros_stack  as w4a16_gemm_grouped (expert e's tiles at word
 *                   e*K*N/8, its [G][N] scales / zeros at element e*G*N); zeros for U4 only
 *   c               device fp16 [prob_m * top_k][ldc] (ldc >= N, or >= N/2 with the gated flags)
 *   sorted_token_ids, expert_ids, num_tokens_past_padded  device int32, 4-byte aligned
 *   topk_weights    device fp32 [prob_m * top_k] (4-byte aligned), required when
 *                   mul_topk_weights is 1
 *   max_padded      capacity of sorted_token_ids: a multiple of moe_block_size, at most
 *                   W4A16_MOE_MAX_BLOCKS blocks; num_tokens_past_padded must not exceed it
 *   moe_block_size  8, 16, 32, 48 or 64;  top_k, prob_m, n_experts positive
 *   mul_topk_weights, is_ep  0 or 1
 *   flags           as w4a16_gemm_grouped (W4A16_FLAG_HAS_ZP, W4A16_FLAG_SWIGLU / _GEGLU, ...)
 *   workspace       >= w4a16_moe_blocks_workspace_size(...) bytes, 256-byte aligned,
 *                   zero-filled once (as w4a16_gemm's)
 * Three launches on `stream`: a one-CTA routing kernel that turns the blocks into the grouped
 * kernel's segments (runs of blocks of one expert, blocks of expert -1 dropped) in the
 * workspace, a gather of the rows' activations, and the grouped tcgen05 GEMM.  A padded length
 * that is negative, larger than max_padded or not a whole number of blocks, an expert id out of
 * range (or -1 without is_ep), an id other than a valid one or the sentinel, or more runs than
 * the schedule holds (min(blocks, 1024)) set W4A16_DEV_SCHEDULE; the affected rows are not
 * written. */
int w4a16_gemm_moe_blocks(const void *a, int lda, const int32_t *b_packed_stack, void *c, int ldc,
                          const void *scales_stack, const void *zeros_stack,
                          const int32_t *sorted_token_ids, const int32_t *expert_ids,
                          const int32_t *num_tokens_past_padded, const float *topk_weights,
                          int max_padded, int moe_block_size, int top_k, int mul_topk_weights,
                          int is_ep, int n_experts, int prob_m, int n, int k, int group_size,
                          int weight_type, unsigned flags, void *workspace, size_t workspace_bytes,
                          cudaStream_t stream);

/* Host-side schedule builder (memra-engine mmq_ffi.rs `ExpertCsr::from_token_routes`):
 * token-major routes selected[t*experts_per_token + j] -> expert-major CSR.  Host pointers;
 * ex_ids needs n_expert entries, ex_off n_expert+1, ex_pairs and pair_tok n_tokens*experts_per_token.
 * Returns the number of active experts, or a negative value on rejected input. */
int w4a16_csr_from_token_routes(int n_expert, int n_tokens, int experts_per_token,
                                const int32_t *selected, int32_t *ex_ids, int32_t *ex_off,
                                int32_t *ex_pairs, int32_t *pair_tok);

/* ------------------------------------------------------------------------------------------
 * The rest of a decode step around the W4A16 products: rotary positions with the write into a
 * paged key-value cache, the attention of one new token over that cache, and a whole expert
 * layer for a few tokens.  The pages have no kernels for these; they are this library's own.
 *
 * Paged cache: keys and values live in two arrays of the same layout.  Position i of a sequence
 * is token i % page_size of page block_table[i / page_size]; head c of it starts at element
 *     page * kv_page_stride + token * kv_token_stride + c * kv_head_stride
 * and is head_dim contiguous 16-bit values (fp16, or bf16 with W4A16_FLAG_BF16).  Any order of
 * tokens and heads inside a page, and any page size, can be expressed.  Offsets are 64-bit.
 * ---------------------------------------------------------------------------------------- */

/* Rotary positions with one to four axes (a text position; or time, height and width of images
 * and video) on q and k, and k and v written into the cache, in one launch.
 * Pair i < rot_dim / 2 of a head belongs to axis a when it lies in a's section (sections[0] pairs
 * of axis 0 first, then sections[1] of axis 1, ...).  With p = positions[a * ld_pos + t],
 * c = cos_sin[p * rot_dim + i] and s = cos_sin[p * rot_dim + rot_dim / 2 + i]:
 *     (x1, x2) -> (x1 c - x2 s, x2 c + x1 s)
 * on values i and rot_dim / 2 + i of the head (2i and 2i + 1 with W4A16_FLAG_ROPE_ADJACENT); values
 * rot_dim .. head_dim - 1 are copied.  Computed in fp32 and rounded once.
 *   q, k, v      device 16-bit; token t's heads start at element t * ldq (ldk, ldv), head h
 *                head_dim values further on; so the three parts of one fused projection's output
 *                can be passed as they lie
 *   q_out        device 16-bit [n_tokens][ldqo]; may be q itself (with ldqo == ldq), else must not
 *                overlap an input
 *   k_cache, v_cache  the paged cache; only the rows that slots name are written
 *   cos_sin      device fp32 [max_pos][rot_dim]: rot_dim / 2 cosines, then as many sines
 *   positions    device int32 [n_axes][ld_pos], ld_pos >= n_tokens
 *   slots        device int64 [n_tokens]: page * page_size + token in the page; negative: the
 *                token's k and v are not written (padding).  Two tokens must not share a slot
 *   status       device int32 or NULL: W4A16_DEV_POSITION is OR-ed in when a position is outside
 *                [0, max_pos) (values that need it are not written, nor, with 16-byte copies and a section
 *                that ends inside them, the rest of their eight pairs), W4A16_DEV_SLOT when a slot is
 *                past the cache (that token's k and v are not written)
 *   sections     host int32 [n_axes], non-negative, with sum rot_dim / 2;  n_axes 1..4
 *   n_heads, n_kv_heads  either may be 0 (its pointers are then not looked at)
 *   rot_dim      even, 2 .. head_dim
 *   flags        W4A16_FLAG_BF16, W4A16_FLAG_ROPE_ADJACENT
 * 16-bit buffers need 2-byte alignment only; with head_dim and rot_dim multiples of 16, strides
 * multiples of 8 and 16-byte aligned buffers the copies are 16 bytes wide. */
int w4a16_rope_append(const void *q, int ldq, const void *k, int ldk, const void *v, int ldv,
                      void *q_out, int ldqo, void *k_cache, void *v_cache, long long kv_page_stride,
                      long long kv_token_stride, long long kv_head_stride, const float *cos_sin,
                      int max_pos, const int32_t *positions, int ld_pos, const long long *slots,
                      int32_t *status, int n_tokens, int n_heads, int n_kv_heads, int head_dim,
                      int rot_dim, const int32_t *sections, int n_axes, int page_size, int n_pages,
                      unsigned flags, cudaStream_t stream);

/* Workspace bytes of w4a16_paged_attention (num_sms <= 0: the current device; 0 for sizes that it
 * rejects).  Zero-filled once after allocation, after which it serves calls of any sizes that need no
 * more bytes, in any order; calls that run concurrently need separate workspaces. */
size_t w4a16_paged_attention_workspace_size(int batch, int n_heads, int n_kv_heads, int head_dim,
                                            int num_sms);

/* Attention of one new token per sequence over the paged cache, the work split over the cache's
 * length and joined, in one launch.  For sequence b and query head h, with the KV head
 * c = h / (n_heads / n_kv_heads), over positions i in [max(0, len - window), len) (window 0: all):
 *     out[b][h] = sum_i p_i v_i,   p = softmax(scale q . k_i),   lse[b][h] = log sum_i e^(scale q . k_i)
 * The new token's own key and value are part of the cache (w4a16_rope_append writes them first).
 * A sequence of length 0 (or with scores of -inf alone) gets zeros and lse = -inf.  Rows of the cache
 * past a length are never read, whatever they hold.  Softmax and sums are fp32 (the scores of 256-wide
 * heads, at most eight per KV head, in one chain of tensor-core sums, which are cut off instead of rounded:
 * up to a bit and a half less than elsewhere).  p enters the value product as a 16-bit value plus a 16-bit
 * remainder, to 2^-17 (bf16) or 2^-23 (fp16; to 2^-40 absolute) of itself; a live value that is infinite
 * therefore gives NaN.
 *   q            device 16-bit [batch][ldq], head h at h * head_dim;  ldq % 8 == 0
 *   out          device 16-bit [batch][ldo];  ldo % 8 == 0;  lse  device fp32 [batch][n_heads] or NULL
 *   block_table  device int32 [batch][ld_table], ld_table >= max_pages; entries past a sequence's
 *                last page (and before a window's first) are not read
 *   seq_lens     device int32 [batch], read on the device: no host copy of the lengths is needed
 *   strides      multiples of 8 elements;  q, k_cache, v_cache, out 16-byte aligned
 *   batch        0 (a no-op) .. 4096;  head_dim 64, 128 or 256;  n_heads a multiple of n_kv_heads
 *   page_size, n_pages, max_pages  positive; max_pages x page_size bounds every length
 *   flags        W4A16_FLAG_BF16
 * A length outside [0, max_pages x page_size] is clamped and reported as W4A16_DEV_LENGTH; a page
 * number outside [0, n_pages) makes its positions masked and is reported as W4A16_DEV_PAGE.
 * Repeated calls with the same sizes and lengths are bit-identical. */
int w4a16_paged_attention(const void *q, int ldq, const void *k_cache, const void *v_cache,
                          long long kv_page_stride, long long kv_token_stride,
                          long long kv_head_stride, void *out, int ldo, float *lse,
                          const int32_t *block_table, int ld_table, const int32_t *seq_lens,
                          void *workspace, size_t workspace_bytes, int batch, int n_heads,
                          int n_kv_heads, int head_dim, int page_size, int n_pages, int max_pages,
                          int window, float scale, unsigned flags, cudaStream_t stream);

/* w4a16_rope_append with the heads of q and k normalised first, in the same launch:
 *     y = x rsqrt(mean(x^2) + eps) w
 * over a head's head_dim values, with the weights w = q_norm or k_norm; v is copied.  Sums are fp32 and nothing
 * is rounded between the norm and the rotation.  As w4a16_rope_append, but for:
 *   q_norm, k_norm  device 16-bit [head_dim], or NULL: those heads are not normalised
 *   eps          finite, not negative
 *   rot_dim      even, 0 .. head_dim; 0: no rotation, with n_axes 0 (cos_sin, positions and sections are then not
 *                looked at)
 * 16-byte copies also need q_norm and k_norm 16-byte aligned and head_dim at most 512. */
int w4a16_norm_rope_append(const void *q, int ldq, const void *k, int ldk, const void *v, int ldv,
                           const void *q_norm, const void *k_norm, float eps, void *q_out, int ldqo,
                           void *k_cache, void *v_cache, long long kv_page_stride,
                           long long kv_token_stride, long long kv_head_stride, const float *cos_sin,
                           int max_pos, const int32_t *positions, int ld_pos, const long long *slots,
                           int32_t *status, int n_tokens, int n_heads, int n_kv_heads, int head_dim,
                           int rot_dim, const int32_t *sections, int n_axes, int page_size, int n_pages,
                           unsigned flags, cudaStream_t stream);

/* ------------------------------------------------------------------------------------------
 * A paged cache held in 4 bits.  Each group of group_size values of a head (one token's) has a step s and a base b
 * of 16 bits (fp16, or bf16 with W4A16_FLAG_BF16), and each value a code in 0..15 that stands for code s + b:
 *     b = r(min),  s = r((max - min) / 15),  code = (x - b) / s to the nearest integer (ties to even), cut to 0..15
 * where r rounds to nearest even, from fp32; a group whose range rounds to 0 (bf16: to a subnormal number) has s = 0 and code 0.
 * A group without a finite range (it holds an infinity or a NaN, or max - min is beyond fp32, or its step or base rounds to
 * infinity) reads as NaN.  Records may be written by others too, with steps of either sign for which code s + b is finite
 * for every code.
 * Page p begins at byte p * page_stride, with one record per KV head, of w4a16_kv4_record_bytes bytes each:
 *     key codes [page_size][head_dim / 8] words, value codes the same, key (s, b) pairs
 *     [page_size][head_dim / group_size], value pairs the same
 * A word holds the codes of eight values in a row, value 8 w + i at bits 4 i .. 4 i + 3 of word w.  Words of a
 * row do not lie in order: with B = head_dim / 64, key word 8 b + 2 t + i (b < B, t < 4, i < 2) is at place
 * 16 (b / 2) + 4 t + 2 (b % 2) + i (B = 1: in order), value word 8 b + g (g < 8) at place g B + b.
 * head_dim 64, 128 or 256; group_size -1 (the head) or a multiple of 64 that divides head_dim; page_size
 * 1 .. W4A16_KV4_MAX_PAGE.  Position i of a sequence is token i % page_size of page block_table[i / page_size].
 * ---------------------------------------------------------------------------------------- */
#define W4A16_KV4_MAX_PAGE 65536

/* Bytes of one head's record in a page, a multiple of 16; 0 for sizes that the cache does not take. */
size_t w4a16_kv4_record_bytes(int page_size, int head_dim, int group_size);

/* w4a16_norm_rope_append into a cache held in 4 bits.  Keys are coded from norm and rotation in two fp32 parts: steps and
 * bases are those of exact arithmetic, and so are codes but for about three in 10^8, next to a border.
 * As w4a16_norm_rope_append, but for:
 *   cache        device, 16-byte aligned; page_stride in bytes, a multiple of 16, at least n_kv_heads records
 *   k_out, v_out device 16-bit, token t's heads at t * ldko (ldvo), or NULL: what the cache now stands for, rounded
 *                once, for a prompt's own attention.  Written for tokens without a slot too; may be k and v
 *                themselves (same leading dimensions)
 *   n_heads      may be 0;  n_kv_heads positive
 *   rot_dim      a multiple of 16
 * All 16-bit buffers and cos_sin 16-byte aligned, leading dimensions multiples of 8.  A key one of whose positions is
 * out of range (W4A16_DEV_POSITION) is not written at all, in no place. */
int w4a16_kv4_append(const void *q, int ldq, const void *k, int ldk, const void *v, int ldv,
                     const void *q_norm, const void *k_norm, float eps, void *q_out, int ldqo, void *cache,
                     long long page_stride, void *k_out, int ldko, void *v_out, int ldvo,
                     const float *cos_sin, int max_pos, const int32_t *positions, int ld_pos,
                     const long long *slots, int32_t *status, int n_tokens, int n_heads, int n_kv_heads,
                     int head_dim, int rot_dim, const int32_t *sections, int n_axes, int page_size,
                     int n_pages, int group_size, unsigned flags, cudaStream_t stream);

/* Workspace bytes of w4a16_kv4_attention: as w4a16_paged_attention_workspace_size, with the same rules.  One workspace
 * may serve calls of both. */
size_t w4a16_kv4_attention_workspace_size(int batch, int n_heads, int n_kv_heads, int head_dim, int num_sms);

/* w4a16_paged_attention over a cache held in 4 bits, whose values code s + b are used as they are: products and sums
 * are fp32, no key or value is rounded to 16 bits.  q and out are fp16, or bf16 with W4A16_FLAG_BF16, as are the
 * cache's steps and bases.  As w4a16_paged_attention, but for the cache (above) and these points: queries go in as fp16
 * scaled by a power of two per head, off by at most 2^-34 of the head's largest, or 2^-121 (fp16 is exact above 2^-23 of
 * the largest, bf16 above 2^-26; in bf16, queries beyond 2^112 are too large); p s goes into the value product to 2^-22
 * of itself, or to 2^-38 of the largest step of the values seen.  Sums of p times a value are divided by the sum of p at
 * the end, and have to stay within fp32 until then.  A group that reads as NaN makes NaN of what it touches.  page_size
 * at most W4A16_KV4_MAX_PAGE. */
int w4a16_kv4_attention(const void *q, int ldq, const void *cache, long long page_stride, void *out,
                        int ldo, float *lse, const int32_t *block_table, int ld_table,
                        const int32_t *seq_lens, void *workspace, size_t workspace_bytes, int batch,
                        int n_heads, int n_kv_heads, int head_dim, int page_size, int n_pages,
                        int max_pages, int group_size, int window, float scale, unsigned flags,
                        cudaStream_t stream);

/* The next token of each row of logits, from given uniform numbers.  With P_i = e^((l_i - max l) / T) and tokens
 * ordered by (logit falling, index rising):
 *     top_k keeps the first top_k; top_p, of these, the shortest beginning whose sum of P reaches top_p times their sum
 *     (one token at least); min_p, of these, those with P_i >= min_p;
 *     token = the first index i at which the sum of the kept P_j, j <= i, exceeds uniform times the sum of all kept.
 * P is held as a multiple of 2^-43, to 2^-30 of itself, and sums are exact: results do not depend on the batch and
 * repeats are identical.  One launch, no workspace.
 *   logits       device 16-bit [batch][ld] (fp16, or bf16 with W4A16_FLAG_BF16), 2-byte aligned (rows of 16-byte
 *                alignment are read in 16-byte loads); a NaN counts as -inf, and -inf is never chosen
 *   uniform      device fp32 [batch], in [0, 1)
 *   temperature  device fp32 [batch] or NULL (1): 0 .. 2^100; 0 takes the largest logit (the lowest index
 *                where some are equal) whatever the other settings; others below 2^-126 count as 2^-126
 *   top_k        device int32 [batch] or NULL: 0 and below: no limit
 *   top_p, min_p device fp32 [batch] or NULL (1, 0): top_p of 1 and above and min_p of 0 and below: no limit; min_p
 *                above 1 counts as 1
 *   tokens       device int32 [batch]
 *   logprobs     device fp32 [batch] or NULL: log of the token's share of the kept sum
 *   status       device int32 or NULL: W4A16_DEV_SETTING is OR-ed in for a row with a setting out of range or NaN; its
 *                token is -1 and its logprob NaN (with temperature 0: for a NaN in top_p or min_p alone)
 *   batch        0 (a no-op) .. 2^24;  vocab 1 .. 524288, ld >= vocab
 * A row without a logit above -inf gets token -1 and logprob -inf. */
int w4a16_sample(const void *logits, int ld, const float *uniform, const float *temperature,
                 const int32_t *top_k, const float *top_p, const float *min_p, int32_t *tokens,
                 float *logprobs, int32_t *status, int batch, int vocab, unsigned flags,
                 cudaStream_t stream);

/* Workspace bytes of w4a16_moe_layer (0 for sizes that it rejects).  Zero-filled once after
 * allocation, after which it serves calls of any sizes that need no more bytes, in any order; calls that
 * run concurrently need separate workspaces.  More tokens never need fewer bytes. */
size_t w4a16_moe_layer_workspace_size(int n_tokens, int hidden, int inter, int n_experts, int top_k);

/* A whole expert layer with 4-bit weights for a few tokens: router product, softmax, top-k, the
 * chosen experts' gated products and down products, the weighted sum and the residual.  For token t:
 *     l_e = router[e] . x_t;   P = softmax(l);   the top_k experts of largest l, best first (the
 *     lowest index where scores are equal);   w_j = P[e_j], divided by the sum of the chosen ones
 *     with W4A16_FLAG_MOE_RENORM;
 *     y_t = residual_t + sum_j w_j down_{e_j}( act(gate_{e_j} x_t) * (up_{e_j} x_t) )
 * with act silu (W4A16_FLAG_SWIGLU) or gelu_tanh (W4A16_FLAG_GEGLU).  All sums are fp32, (q - z) s is
 * not rounded, y is rounded once.  The inner activations go on as a 16-bit value plus a 16-bit remainder:
 * to 2^-17 of themselves in bf16; in fp16 to 2^-23, or to an absolute 2^-25 where that is more, and
 * whatever lies beyond 131008 is added in fp32 (a call that has such values takes longer).  Routing runs on the device:
 * no host synchronisation, and the call can be captured in a graph.  For more tokens than
 * 64 use the grouped entry points.
 *   x              device 16-bit [n_tokens][ldx];  residual 16-bit [n_tokens][ldr] or NULL
 *   router         device 16-bit [n_experts][hidden]
 *   gate_up        device int32, expert e's [hidden][2 inter] tiles at word e * hidden * 2 inter / 8:
 *                  columns interleaved by w4_gate_up_interleave, then w4_repack
 *   down           device int32, expert e's [inter][hidden] tiles (w4_repack)
 *   *_scales, *_zeros  device 16-bit [n_experts][G][N] (gate_up's columns interleaved too); zeros for
 *                  W4A16_TYPE_U4 only, with W4A16_FLAG_HAS_ZP, as for w4a16_gemm
 *   y              device 16-bit [n_tokens][ldy]; may be residual or x itself (same leading dimension)
 *   topk_ids, topk_weights  device int32 / fp32 [n_tokens][top_k] or NULL: the routing, written
 *   n_tokens       0 (a no-op) .. 64;  hidden % 256 == 0;  inter % 128 == 0;  both at most 65536
 *   n_experts      1 .. 512;  top_k 1 .. 16, at most n_experts
 *   group_size     -1, or a positive multiple of 64 that divides hidden and inter (sums are scaled per
 *                  64-row block: no groups of 16 or 32); no act-order
 *   flags          exactly one of W4A16_FLAG_SWIGLU / _GEGLU; W4A16_FLAG_BF16, _HAS_ZP, _MOE_RENORM,
 *                  _IS_K_FULL
 * 16-byte aligned buffers, leading dimensions multiples of 8.  A NaN score counts as the lowest when
 * experts are chosen; the token's output is then NaN.  Repeated calls are bit-identical. */
int w4a16_moe_layer(const void *x, int ldx, const void *router, const int32_t *gate_up,
                    const void *gate_up_scales, const void *gate_up_zeros, const int32_t *down,
                    const void *down_scales, const void *down_zeros, const void *residual, int ldr,
                    void *y, int ldy, int32_t *topk_ids, float *topk_weights, void *workspace,
                    size_t workspace_bytes, int n_tokens, int hidden, int inter, int n_experts,
                    int top_k, int group_size, int weight_type, unsigned flags, cudaStream_t stream);

/* ------------------------------------------------------------------------------------------
 * Checkpoint loading helpers (off the GEMM's path).
 * ---------------------------------------------------------------------------------------- */

/* AutoGPTQ packed zero points -> the fp16 zero points w4a16_gemm takes (host memory, host
 * code).  ferrum-kernels 0.8.4 vllm_marlin.rs, `repack_gptq_qzeros_to_marlin`: a checkpoint
 * stores `zero - 1`, eight 4-bit codes per int32 word along N, column 8w + i at bits 4i..4i+3,
 * so the runtime zero point is the stored code + 1, and a stored 15 (zero point 16, not a
 * 4-bit value) is rejected.
 *   qzeros  host int32 [groups][n / 8]
 *   zeros   host uint16 [groups][n], written: IEEE binary16 bit patterns of the zero points
 *           (integers 1..15), ready to copy to the device
 *   n       a positive multiple of 8
 * Returns 0, or stage 1 with W4A16_ARG_QZERO if any code is 15 (then nothing is written),
 * W4A16_ARG_SHAPE or W4A16_ARG_NULL. */
int w4_qzeros_to_zero_points(const int32_t *qzeros, int groups, int n, uint16_t *zeros);

/* Whether a checkpoint's packed zero words say "symmetric": every 4-bit code of every word is
 * 7 (zero point 8), so the weights can run as W4A16_TYPE_U4B8 without zero points
 * (vllm_marlin.rs, `gptq_qzeros_are_symmetric_code7`).  Host memory; returns 1 or 0 (0 for
 * an empty or NULL array). */
int w4_qzeros_symmetric_code7(const int32_t *qzeros, long long count);

/* Device check of fp16 zero points before they are handed to w4a16_gemm (whose kernels assume
 * integers in [0, 15] and do not check): ORs W4A16_DEV_ZERO into *status (device int32,
 * 4-byte aligned) if any of the `count` values is not an integer in [0, 15] or is NaN.
 * Asynchronous on `stream`; `zeros` is device fp16, 2-byte aligned.  Returns 0, a stage-1
 * status for bad arguments, or a stage-6 launch status. */
int w4a16_zero_points_check(const void *zeros, long long count, int32_t *status,
                            cudaStream_t stream);

/* Reads (synchronously, on `stream`) the device-side status word of a workspace and clears
 * it.  *device_bits receives the W4A16_DEV_* bits seen since the last read.  Returns 0, or a
 * stage-3 status if the copy failed. */
int w4a16_status(void *workspace, int *device_bits, cudaStream_t stream);

/* Self-test of the bounded wait used by every kernel: launches one block that waits on a
 * barrier nobody arrives at, for at most `limit_ns` nanoseconds, then records
 * W4A16_DEV_TIMEOUT in the workspace status word and returns normally.  The context stays
 * usable.  `workspace` needs 256 bytes. */
int w4a16_selftest_timeout(void *workspace, long long limit_ns, cudaStream_t stream);

/* Human-readable name of a status's stage ("ok", "invalid-argument", ...). */
const char *w4a16_status_string(int status);

/* ABI version of the loaded library (W4A16_ABI_VERSION). */
int w4a16_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* W4A16_H */
