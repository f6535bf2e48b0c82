/*
 * hm.h -- C ABI of the MI355X (gfx950) low-bit GEMM library.
 *
 * The library computes a linear layer Y[M,N] = X[M,K] . W_hat[N,K]^T whose
 * weights are stored in 4-bit form and dequantized inside the kernel, and the
 * grouped (MoE) variant in which every routed (token, expert) pair runs against
 * its expert's weights.  Sources, cited by page and section:
 *   - linear layer as X times W transposed, weights read once and reused over
 *     the M rows, about 2*M*N*K flops: ywsung.com note "How vLLM Humming
 *     computes 4 bits", section on one token vs many tokens;
 *   - 4-bit codes with a scale, q = round(w/s), restored as s*q, signed range
 *     -8..7, one 16-bit scale per 128 weights: same note, section on scales;
 *   - one common representation of weights, scales and zero points, then
 *     padding and re-ordering for the device, done once before inference
 *     (transform, then call the layer): same note, section on layout, and the
 *     aihaber.org article, Architecture;
 *   - the formats (INT4, MXFP4) and activation widths (16-bit, 8-bit):
 *     cocoloop.cn news item, format list; aihaber.org, hardware and format
 *     support; per-token FP8 activations: ywsung.com note, section on weight
 *     format / activation / backend;
 *   - tokens split per expert so that every expert's GEMM has its own M, and a
 *     grouped path over all experts: ywsung.com note, section on one token vs
 *     many tokens; aihaber.org, Performance.
 *
 * Conventions (every entry point):
 *   - Tensor pointers are DEVICE pointers unless stated; descriptors are host
 *     pointers.  The caller owns every buffer (weights, inputs, outputs,
 *     workspaces); the library allocates no device memory and keeps no state
 *     between calls.
 *   - Calls are asynchronous on `stream` (NULL = the default stream), never
 *     synchronize, and are safe to call from several host threads.
 *   - All argument checks happen before any launch.  On any error the call
 *     returns a non-zero hm_status and no kernel has been launched; outputs are
 *     untouched.  HM_ERR_HIP reports a failed launch.
 *   - Matrices are row-major and contiguous.  bf16 values are passed as their
 *     16-bit patterns (uint16_t).  Outputs are bf16, rounded to nearest even
 *     from an fp32 accumulator.
 *   - K must be a multiple of 128 for every format.  N is arbitrary.
 *   - Alignment: w_dev and workspaces 256 bytes, every other pointer 16 bytes
 *     (HM_ERR_ALIGN otherwise).
 *   - Inputs are finite; NaN or Inf in X, scales or weights gives unspecified
 *     (but memory-safe) results where an entry point does not say more.
 */
#ifndef HM_H
#define HM_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define HM_ABI_VERSION 2

typedef enum hm_status {
  HM_OK = 0,
  HM_ERR_NULL = 1,        /* a required pointer is NULL */
  HM_ERR_SHAPE = 2,       /* bad size, group or count */
  HM_ERR_ALIGN = 3,       /* pointer not aligned as required */
  HM_ERR_UNSUPPORTED = 4, /* unknown weight format or format/activation pair; arrays that overlap (hm_lora, hm_lora_grad, the int8 calls) */
  HM_ERR_WORKSPACE = 5,   /* buffer smaller than its size query */
  HM_ERR_HIP = 6,         /* a HIP launch failed */
  HM_ERR_ABI = 7,         /* descriptor abi field != HM_ABI_VERSION */
  HM_ERR_TUNING = 8       /* a tuning field out of range, or a forced kernel that cannot run this call */
} hm_status;

/* Weight number format (the "number format / scale unit / zero point" of the
 * quantization description, ywsung.com note, section on layout, figure on the
 * quantization description). */
typedef enum hm_wfmt {
  HM_W_INT4_SYM = 0, /* signed 4-bit two's complement q, bf16 scale per 128 along K: w = s*q */
  HM_W_UINT4_ZP = 1, /* unsigned 4-bit u, bf16 scale + 4-bit zero point per 128: w = s*(u-z) */
  HM_W_MXFP4 = 2,    /* E2M1 codes, E8M0 scale per 32 along K: w = e2m1(c) * 2^(b-127) */
  HM_W_MXINT4 = 3,   /* two's complement 4-bit q read as 1.2 fixed point, E8M0 scale per 32
                        along K: w = (q/4) * 2^(b-127); the format is named in the pages' lists
                        (cocoloop.cn item; aihaber.org article, hardware and format support)
                        without a definition, this is the MX-family reading */
  HM_W_UINT3_ZP = 4, /* unsigned 3-bit u, bf16 scale + 3-bit zero point per 128: w = s*(u-z) */
  HM_W_UINT2_ZP = 5, /* unsigned 2-bit u, bf16 scale + 2-bit zero point per 128: w = s*(u-z);
                        the pages list INT1..INT8 weights and name GPTQ INT3 as a compatibility
                        case (cocoloop.cn news item, format list and deployer section).  Both are
                        widened to the 4-bit zero-point device layout by hm_transform (exact; no
                        bandwidth saving over 4 bits) and run on every W4A16 kernel */
  HM_W_INT8_SYM = 6  /* signed 8-bit two's complement q, bf16 scale per 128 along K: w = s*q (own
                        device layout of 2 KiB tiles; the streaming (path 1) and 128 x 128
                        (path 4) kernels, and grouped streaming and 128-row units) */
} hm_wfmt;

/* Activation format (the compute option choosing A16, A8 or A4). */
typedef enum hm_afmt {
  HM_A_BF16 = 0,         /* X is bf16 [M,K]; x_scales unused (may be NULL) */
  HM_A_FP8_ROWSCALE = 1, /* X is OCP E4M3 bytes [M,K] with one fp32 scale per row: x = e4m3(c)*s[m] */
  HM_A_MXFP4 = 2         /* X is E2M1 codes [M][K/2] (value 2j in the low nibble of byte j) with E8M0
                            scale bytes [M][K/32] in x_scales: x = e2m1(c) * 2^(b-127) (W4A4) */
} hm_afmt;

/* Supported pairs: every weight format with HM_A_BF16 (W4A16: INT4_SYM,
 *                  UINT4_ZP, and MXFP4 / MXINT4, whose codes are scaled to
 *                  bf16 in the kernel; the pages list MXFP4 W4A16 among the
 *                  MoE results, aihaber.org article, performance section);
 *                  MXFP4 with HM_A_FP8_ROWSCALE (W4A8-MXFP4); MXFP4 with
 *                  HM_A_MXFP4 (W4A4: both operands E2M1 with E8M0 scales on
 *                  the scaled fp4 MFMA; the pages list W4A4 among the GEMM
 *                  types, cocoloop.cn news item, format list).  W4A4 runs on
 *                  the streaming kernel (path 1) and the 128 x 128 kernel
 *                  (path 4) only.
 * MXFP4 with bf16 rows requires every |w| < 2^128 (E8M0 scale bytes up to
 * 252 always satisfy it, up to 253 for MXINT4; larger products become inf,
 * and the row's sums NaN):
 * the dequantized weights enter the bf16 MFMA.  Subnormal products (scale
 * bytes 0..3) are kept exactly. */

/* Layer description (shapes, number format, group).  num_experts is 1 for a
 * dense layer.  group must be 128 for the INT4 formats and 32 for MXFP4. */
typedef struct hm_wdesc {
  int32_t abi;         /* HM_ABI_VERSION */
  int32_t wfmt;        /* hm_wfmt */
  int32_t group;       /* elements per scale along K */
  int32_t num_experts; /* >= 1 */
  int64_t n;           /* output features (rows of W), >= 1 */
  int64_t k;           /* input features, multiple of 128, >= 128 */
} hm_wdesc;

/* Explicit choices of one GEMM call (the pages' "Tuning Config": tile
 * shapes, launch shape and split of the work, chosen apart from the layer and
 * compute description; aihaber.org article, Architecture; ywsung.com note,
 * section on layout).  Pass NULL, or a zero-initialised struct with abi set,
 * for the library's default heuristic choice; any nonzero field overrides the
 * default for that one call (the library keeps no state).  Out-of-range
 * values, or a forced kernel that cannot run the call, give HM_ERR_TUNING
 * before any launch.  hm_gemm_plan / hm_moe_gemm_plan report what a given
 * tuning selects.  Every field has a documented default (0). */
typedef struct hm_tuning {
  int32_t abi;             /* HM_ABI_VERSION */
  int32_t path;            /* dense kernel: 0 default; 1 streaming (M <= 256); 2 128-row tiles
                              (W4A16 128 x 64 split over K, W4A8 64 x 128); 3 256 x 256 tiles;
                              4 128 x 128 tiles */
  int32_t stream_ks;       /* streaming: waves of a block splitting one column set's K: 0, 1, 2, 4, 8 */
  int32_t stream_nbw;      /* streaming: 16-column blocks per wave: 0, 1, 2 */
  int32_t stream_splits;   /* dense streaming: K split over blocks (fp32 partials): 0, 1 .. K/128 */
  int32_t stream_waves;    /* dense streaming: waves per block: 0, 4, 8 (8 needs stream_ks 2, 4 or 8) */
  int32_t moe_stream_rows; /* rows per grouped streaming unit: 0, 16, 32 */
  int32_t moe_stream_max;  /* largest expert (rows) taking streaming units: 0, 1 .. 4096 */
  int32_t moe_stream_nbw;  /* grouped streaming: 16-column blocks per wave: 0, 1, 2 */
  int32_t moe_stream_ks;   /* grouped streaming: waves splitting K: 0, 1, 2, 4 */
  int32_t moe_stream_lds_kb; /* grouped streaming: LDS per block in KiB: 0, 20 .. 159 */
  int32_t moe_big_min;     /* smallest expert remainder that takes a 256-row unit: 0, 1 .. 256;
                              -1: no 256-row units */
  int32_t moe_tile;        /* kernel of the up-to-128-row units: 0 default; 1 the 128-row tile
                              kernel of path 2; 2 the 128 x 128 kernel */
} hm_tuning;

/* ---------------------------------------------------------------- weights */

/* Bytes of the device weight buffer for `d` (all experts). */
hm_status hm_transform_size(const hm_wdesc* d, size_t* bytes);

/* Repack the standard format into the device layout (padding N to 16 and
 * re-ordering codes, scales and zero points so that each 64-lane wave reads
 * one 1 KiB tile of 16 columns x 128 K per 16-byte-per-lane load).  Run once
 * per weight, before inference.
 *   codes  [E][N][K/2] bytes, element k=2j in the low nibble of byte j,
 *          k=2j+1 in the high nibble (two's complement for INT4_SYM and
 *          MXINT4, unsigned for UINT4_ZP, E2M1 bits for MXFP4);
 *          UINT2_ZP: [E][N][K/4], element 4j+i at bits 2i..2i+1 of byte j;
 *          UINT3_ZP: [E][N][3K/8], element 8j+i at bits 3i..3i+2 of the
 *          little-endian 24-bit word of bytes 3j..3j+2;
 *          INT8_SYM: [E][N][K], one two's complement byte per element.
 *   scales INT4 formats: bf16 [E][N][K/128]; MXFP4, MXINT4: E8M0 bytes [E][N][K/32].
 *   zeros  zero-point formats only: bytes [E][N][K/128], the code's low 4 / 3 / 2
 *          bits used; else NULL.
 *   w_dev  output, w_bytes >= hm_transform_size.  Opaque; valid only for the
 *          same descriptor. */
hm_status hm_transform(const hm_wdesc* d, const uint8_t* codes, const void* scales,
                       const uint8_t* zeros, void* w_dev, size_t w_bytes, hipStream_t stream);

/* hm_transform of a gate_up weight (n = 2d rows: gate rows 0..d-1, up rows
 * d..2d-1, n a multiple of 32, else HM_ERR_SHAPE) into the gated device
 * layout that hm_moe_gemm_gated reads: device row 32 i + c holds gate row
 * 16 i + c and device row 32 i + 16 + c up row 16 i + c (c < 16), i.e. the
 * buffer equals hm_transform of the standard format with its rows so
 * permuted (hm_dequant of it returns the rows in that order).  Same size
 * (hm_transform_size) and arguments as hm_transform. */
hm_status hm_transform_gated(const hm_wdesc* d, const uint8_t* codes, const void* scales,
                             const uint8_t* zeros, void* w_dev, size_t w_bytes, hipStream_t stream);

/* Exact dequantization of one expert of a transformed buffer into fp32
 * out[N][K].  Every restored weight is exactly representable in fp32 for the
 * INT4 formats, and for MXFP4 with E8M0 scale bytes up to 252 (MXINT4: up to
 * 253); larger bytes give +-inf where the product leaves the fp32 range, and
 * byte 255 (the E8M0 NaN) gives NaN. */
hm_status hm_dequant(const hm_wdesc* d, const void* w_dev, size_t w_bytes, int32_t expert,
                     float* out, hipStream_t stream);

/* -------------------------------------------------------------- activations */

/* Per-token FP8: for each row m, s[m] = amax_k |x[m,k]| / 448 (fp32 division),
 * x8[m,k] = E4M3(x[m,k] / s[m]) with the division in fp32, round to nearest
 * even, saturating at +-448; a row of zeros gives s = 0 and zero codes.
 *   x bf16 [m][k]; x8 bytes [m][k]; row_scale fp32 [m].  k >= 1 (any k). */
hm_status hm_quant_fp8_rows(const uint16_t* x, int64_t m, int64_t k, uint8_t* x8,
                            float* row_scale, hipStream_t stream);

/* MXFP4 activation rows (the W4A4 pair: 4-bit weights with 4-bit
 * activations, cocoloop.cn news item, format list): per 32 consecutive values
 * of each row, the OCP MX rule -- shared exponent X = floor(log2 amax) - 2
 * clamped to [-127, 127], stored as the E8M0 byte X + 127 (0 for a zero
 * block), elements E2M1(x / 2^X) rounded to nearest even and saturated at
 * +-6 (negative values that round to zero keep the sign: code 8).
 *   x bf16 [m][k]; codes [m][k/2] bytes, value 2j in the low nibble of byte
 *   j; scales [m][k/32] E8M0 bytes.  k a multiple of 32; x and codes 16-byte
 *   aligned.  m = 0 is a no-op. */
hm_status hm_quant_mxfp4_rows(const uint16_t* x, int64_t m, int64_t k, uint8_t* codes, uint8_t* scales,
                              hipStream_t stream);

/* ---------------------------------------------------------------- dense GEMM */

/* Workspace bytes hm_gemm needs for this shape and tuning (may be 0). */
hm_status hm_gemm_workspace_size(const hm_wdesc* d, int32_t afmt, int64_t m, const hm_tuning* tune,
                                 size_t* bytes);

/* y[m][n] = bf16( sum_k x_hat[m,k] * w_hat[n,k] ), fp32 accumulation.
 *   w_dev      transformed weights (num_experts must be 1).
 *   x          bf16 [m][k] (HM_A_BF16), E4M3 bytes [m][k] (HM_A_FP8_ROWSCALE) or
 *              E2M1 codes [m][k/2] (HM_A_MXFP4).
 *   x_scales   fp32 [m] row scales for HM_A_FP8_ROWSCALE, E8M0 bytes [m][k/32]
 *              for HM_A_MXFP4 (4-byte aligned), else ignored.
 *   y          bf16 [m][n].
 *   ws         workspace of at least hm_gemm_workspace_size bytes (NULL if 0).
 *   tune       NULL for the default choice, else explicit choices (hm_tuning).
 * m = 0 is a no-op; m above 8388480 (65535 x 128) gives HM_ERR_SHAPE, here
 * and in the size and plan queries. */
hm_status hm_gemm(const hm_wdesc* d, const void* w_dev, int32_t afmt, const void* x,
                  const void* x_scales, int64_t m, uint16_t* y, void* ws, size_t ws_bytes,
                  const hm_tuning* tune, hipStream_t stream);

/* A short text naming the kernel path and tile configuration hm_gemm selects
 * for this shape and tuning (so a caller can confirm what actually runs). */
hm_status hm_gemm_plan(const hm_wdesc* d, int32_t afmt, int64_t m, const hm_tuning* tune, char* buf,
                       size_t buf_len);

/* ------------------------------------------------------------------- MoE */

/* Workspace bytes hm_moe_sort needs: 0 up to 4096 pairs (one workgroup),
 * else chunks x E x 4 for the per-chunk expert counts of the GPU-wide sort
 * (chunks of about 2048 pairs, at most 512 chunks: at most 1 MiB). */
hm_status hm_moe_sort_workspace_size(int64_t t, int32_t topk, int32_t num_experts, size_t* bytes);

/* Expert sort: pairs p = t*topk + j with ids topk_ids[t][j] (the expert
 * grouping of the MoE path: ywsung.com note, section on one token vs many
 * tokens; each expert's M follows its routing load).  Up to 4096 pairs one
 * workgroup counts and places them; more are cut into consecutive chunks,
 * one workgroup each: a counting pass writes every chunk's per-expert counts
 * to ws, and a placing pass gives each chunk its base positions from the
 * totals and the counts of the chunks before it.
 *   counts[e]        number of pairs routed to expert e        (int32 [E])
 *   offsets[e]       exclusive prefix sum, offsets[E] = pairs  (int32 [E+1])
 *   sorted_pairs[i]  pair ids grouped by expert, ascending within each
 *                    expert (stable)                           (int32 [t*topk])
 * Ids outside [0, E) are dropped (not counted, not placed); offsets[E] then
 * falls short of t*topk.  1 <= num_experts <= 512, topk <= num_experts,
 * t*topk < 2^31.  t = 0 is a no-op.  ws: hm_moe_sort_workspace_size bytes
 * (may be NULL when that is 0; HM_ERR_WORKSPACE when smaller), overwritten
 * by the call. */
hm_status hm_moe_sort(const int32_t* topk_ids, int64_t t, int32_t topk, int32_t num_experts,
                      int32_t* counts, int32_t* offsets, int32_t* sorted_pairs, void* ws,
                      size_t ws_bytes, hipStream_t stream);

/* Workspace bytes hm_moe_gemm needs for t tokens, topk and the tuning. */
hm_status hm_moe_gemm_workspace_size(const hm_wdesc* d, int32_t afmt, int64_t t, int32_t topk,
                                     const hm_tuning* tune, size_t* bytes);

/* Grouped GEMM over all experts in one call:
 *   y[p][:] = bf16( A_row(p) . W_hat_{e(p)}^T ) for every routed pair p,
 * where e(p) is the expert whose segment of sorted_pairs holds p.
 *   a            a_rows_are_pairs = 0: activations [t][k] and pair p uses row
 *                p / topk (gate/up projection);  = 1: [t*topk][k] and pair p
 *                uses row p (down projection).  bf16, or E4M3 bytes with
 *                a_scales (one fp32 per row of a) for HM_A_FP8_ROWSCALE, or
 *                E2M1 codes [rows][k/2] with E8M0 a_scales [rows][k/32] for
 *                HM_A_MXFP4.
 *   offsets, sorted_pairs  as produced by hm_moe_sort (device).
 *   y            bf16 [t*topk][n], rows in pair order; rows of dropped pairs
 *                are not written.
 *   ws           at least hm_moe_gemm_workspace_size bytes (the work lists
 *                of the schedule, written by the call).
 *   tune         NULL for the default choice, else explicit choices.
 * Activations of 4 GiB or more run their up-to-128-row units on the 128 x 128
 * kernel (64-bit row addressing) and take no 256-row units.
 * t = 0 is a no-op. */
hm_status hm_moe_gemm(const hm_wdesc* d, const void* w_dev, int32_t afmt, const void* a,
                      const void* a_scales, int32_t a_rows_are_pairs, int64_t t,
                      int32_t topk, const int32_t* offsets, const int32_t* sorted_pairs,
                      uint16_t* y, void* ws, size_t ws_bytes, const hm_tuning* tune,
                      hipStream_t stream);

/* A short text naming the unit kinds and kernels hm_moe_gemm schedules for
 * this call shape and tuning (no device access). */
hm_status hm_moe_gemm_plan(const hm_wdesc* d, int32_t afmt, int64_t t, int32_t topk,
                           int32_t a_rows_are_pairs, const hm_tuning* tune, char* buf, size_t buf_len);

/* The gate_up grouped GEMM with the gated activation in its epilogue (the
 * MoE feed-forward block of the pages: aihaber.org article on Humming, "what
 * problem does it solve"; ywsung.com note, section on one token vs many
 * tokens; the fusion is this library's, the formula that of hm_silu_mul):
 *   h[p][i] = bf16( silu(y[p][i]) * y[p][d + i] ),  y = hm_moe_gemm's bf16
 *   output for the same call, d = n / 2,
 * bit for bit what hm_moe_gemm followed by hm_silu_mul gives, without
 * writing or reading y.
 *   w_dev  from hm_transform_gated (same descriptor, n = 2d, n a multiple of
 *          32; HM_ERR_SHAPE otherwise): gate rows 0..d-1 and up rows
 *          d..2d-1 of the standard format, interleaved by 16-row blocks in
 *          the device layout so that a wave holds both halves of an output.
 *   h      bf16 [t*topk][n/2], rows in pair order; rows of dropped pairs are
 *          not written.
 *   ws     at least hm_moe_gemm_workspace_size bytes (the same schedule).
 * Other arguments and errors as hm_moe_gemm; the grouped streaming units
 * take two column blocks per wave (tune->moe_stream_nbw = 1 gives
 * HM_ERR_TUNING). */
hm_status hm_moe_gemm_gated(const hm_wdesc* d, const void* w_dev, int32_t afmt, const void* a,
                            const void* a_scales, int32_t a_rows_are_pairs, int64_t t,
                            int32_t topk, const int32_t* offsets, const int32_t* sorted_pairs,
                            uint16_t* h, void* ws, size_t ws_bytes, const hm_tuning* tune,
                            hipStream_t stream);

/* The plan text of hm_moe_gemm_gated (as hm_moe_gemm_plan). */
hm_status hm_moe_gemm_gated_plan(const hm_wdesc* d, int32_t afmt, int64_t t, int32_t topk,
                                 int32_t a_rows_are_pairs, const hm_tuning* tune, char* buf, size_t buf_len);

/* For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid allocation): the same
 * grouped GEMM as hm_moe_gemm, with the schedule's work lists kept in a
 * static device array of hm_moe_gemm_static_max_workspace() bytes (4 MiB)
 * inside the library instead of a caller workspace.  Each GPU holds its own
 * array until the process ends; its address is resolved once per device on
 * the first call with that device current.  The call allocates nothing.
 * Calls whose work lists exceed the array (hm_moe_gemm_workspace_size >
 * the maximum, about three million routed pairs with the default tuning)
 * return HM_ERR_WORKSPACE before any launch.  All calls on one GPU share the
 * array: calls that overlap in time on one GPU (different streams, or host
 * threads) race and must be serialized by the caller.  Every other argument,
 * check and result is as for hm_moe_gemm. */
size_t hm_moe_gemm_static_max_workspace(void);
hm_status hm_moe_gemm_static(const hm_wdesc* d, const void* w_dev, int32_t afmt, const void* a,
                             const void* a_scales, int32_t a_rows_are_pairs, int64_t t, int32_t topk,
                             const int32_t* offsets, const int32_t* sorted_pairs, uint16_t* y,
                             const hm_tuning* tune, hipStream_t stream);

/* ------------------------------------------------------- MoE block steps */

/* Gated activation between the gate_up and down grouped GEMMs of an MoE
 * feed-forward block (tokens split per expert, each token activating only
 * some experts: aihaber.org article on Humming, "what problem does it solve";
 * ywsung.com note "How vLLM Humming computes 4 bits", section on one token vs
 * many tokens; the pages give no formula, the reading is the plainest one):
 *   h[r][i] = bf16( silu(gu[r][i]) * gu[r][d + i] ),  silu(x) = x / (1 + exp(-x)),
 * computed in fp32 from the bf16 inputs, rounded to nearest even.
 *   gu   bf16 [rows][2d], row-major: gate in columns 0..d-1, up in d..2d-1
 *        (hm_moe_gemm's gate_up output with n = 2d, pair order kept);
 *   h    bf16 [rows][d] (the down projection's input, a_rows_are_pairs = 1).
 * Device pointers, caller-owned, 16-byte aligned; gu and h must not overlap.
 * rows = 0 is a no-op.  HM_ERR_NULL for a null pointer when rows > 0,
 * HM_ERR_SHAPE for rows < 0 or d <= 0, HM_ERR_ALIGN for a misaligned pointer,
 * HM_ERR_HIP if the launch fails. */
hm_status hm_silu_mul(const uint16_t* gu, int64_t rows, int64_t d, uint16_t* h, hipStream_t stream);

/* The gated activation and the per-token FP8 quantization of its rows in one
 * pass, for an MoE block whose down projection takes FP8 rows (per-token FP8
 * activations: ywsung.com note, section on weight format / activation /
 * backend): h8 and h_scales are exactly what hm_silu_mul followed by
 * hm_quant_fp8_rows on its bf16 output give (h rounded to bf16 first, then
 * s = amax/448 and E4M3(h/s)), without writing or reading the bf16 h.
 *   gu bf16 [rows][2d]; h8 E4M3 bytes [rows][d]; h_scales fp32 [rows].
 * d a multiple of 8 and at most 8192 (HM_ERR_SHAPE otherwise); gu and h8
 * 16-byte aligned, h_scales 4-byte aligned.  rows = 0 is a no-op. */
hm_status hm_silu_mul_fp8(const uint16_t* gu, int64_t rows, int64_t d, uint8_t* h8, float* h_scales,
                          hipStream_t stream);

/* Top-k weighted combine of an MoE block (same pages; the reading: each
 * token's output is its routing-weighted sum of its experts' outputs):
 *   out[t][c] = bf16( sum_{j = 0..topk-1} w[t][j] * y[t*topk + j][c] ),
 * summed in fp32 in ascending j, rounded to nearest even.
 *   y    bf16 [t*topk][n], pair order (hm_moe_gemm's down output);
 *   w    fp32 [t][topk] routing weights;
 *   out  bf16 [t][n].
 * Device pointers, caller-owned; y and out 16-byte aligned, w 4-byte aligned;
 * out must not overlap y or w.  t = 0 is a no-op.  HM_ERR_NULL for a null
 * pointer when t > 0, HM_ERR_SHAPE for t < 0, n <= 0 or topk < 1,
 * HM_ERR_ALIGN for a misaligned pointer, HM_ERR_HIP if the launch fails. */
hm_status hm_moe_combine(const uint16_t* y, const float* w, int64_t t, int32_t topk, int64_t n,
                         uint16_t* out, hipStream_t stream);

/* ------------------------------------------------ MoE rows in expert order */

/* Workspace bytes hm_moe_dispatch needs: 0 up to 32768 pairs, else those of
 * hm_moe_sort. */
hm_status hm_moe_dispatch_workspace_size(int64_t t, int32_t topk, int32_t num_experts, size_t* bytes);

/* Tokens sorted by expert: the stable order of hm_moe_sort and the token rows
 * in that order,
 *   xs[positions[p]][:] = x[p / topk][:]   for every routed pair p = t'*topk + j.
 *   x             bf16 [t][n];  topk_ids int32 [t][topk].
 *   xs            bf16 [t*topk][n]: row i is the row of pair sorted_pairs[i];
 *                 rows from offsets[E] on (as many as pairs were dropped) are
 *                 left as they were.
 *   counts, offsets, sorted_pairs   as hm_moe_sort writes them.
 *   positions     int32 [t][topk]: the row of xs that holds the pair, -1 for
 *                 a dropped pair (id outside [0, num_experts)).
 * hm_moe_gemm runs on the rows of xs with a_rows_are_pairs = 1, t*topk
 * "tokens", topk = 1, these offsets and the identity 0, 1, 2, ... as
 * sorted_pairs; its output is then in expert order too.  Its own gather
 * (a_rows_are_pairs = 0, sorted_pairs of hm_moe_sort) reads the tokens without
 * this copy: prefer it where the rows are not needed in expert order for
 * something else, such as an exchange between ranks or a gradient.
 * Any n >= 1; x and xs 16-byte aligned, the integer arrays 4-byte; limits on
 * t, topk and num_experts as hm_moe_sort.  t = 0 is a no-op: counts and
 * offsets are not written either.  No output may overlap x, topk_ids, ws or
 * another output.  ws: hm_moe_dispatch_workspace_size bytes. */
hm_status hm_moe_dispatch(const uint16_t* x, const int32_t* topk_ids, int64_t t, int32_t topk,
                          int32_t num_experts, int64_t n, uint16_t* xs, int32_t* counts, int32_t* offsets,
                          int32_t* sorted_pairs, int32_t* positions, void* ws, size_t ws_bytes,
                          hipStream_t stream);

/* The gradient of hm_moe_dispatch to its rows:
 *   dx[t'][c] = bf16( sum_j dxs[positions[t'][j]][c] ),
 * summed in fp32 in ascending j; positions outside [0, t*topk) (dropped
 * pairs) add nothing, a token with none routed gets zeros.
 *   dxs bf16 [t*topk][n] (rows that no position names are not read);
 *   positions int32 [t][topk]; dx bf16 [t][n], must not overlap dxs. */
hm_status hm_moe_dispatch_grad(const uint16_t* dxs, const int32_t* positions, int64_t t, int32_t topk,
                               int64_t n, uint16_t* dx, hipStream_t stream);

/* Expert-ordered rows back to their tokens with the routing weights applied
 * (hm_moe_combine for rows in expert order):
 *   out[t'][c] = bf16( sum_j w[t'][j] * ys[positions[t'][j]][c] ),
 * summed in fp32 in ascending j, dropped pairs left out.
 *   ys bf16 [t*topk][n]; w fp32 [t][topk]; out bf16 [t][n], must not overlap
 *   ys. */
hm_status hm_moe_collect(const uint16_t* ys, const float* w, const int32_t* positions, int64_t t,
                         int32_t topk, int64_t n, uint16_t* out, hipStream_t stream);

/* The gradient of hm_moe_collect:
 *   dys[positions[t'][j]][c] = bf16( w[t'][j] * dout[t'][c] ),
 *   dw[t'][j] = sum_c dout[t'][c] * ys[positions[t'][j]][c]   (fp32),
 * dw = 0 for a dropped pair; rows of dys that no position names are left as
 * they were.  No two positions in [0, t*topk) may be equal (hm_moe_dispatch
 * gives none), else which pair's row stays is unspecified, and so are their dw
 * where dys is ys.  With positions[t'][j] = t'*topk + j this is the gradient of
 * hm_moe_combine.
 *   dout bf16 [t][n]; ys, dys bf16 [t*topk][n]; w, dw fp32 [t][topk].  dys may
 *   be ys itself (each row is read before it is written); otherwise no
 *   overlaps.
 * For these three: any n in 1 .. 2^24, t = 0 is a no-op, bf16 arrays 16-byte
 * aligned, fp32 and int32 arrays 4-byte; topk >= 1, t*topk < 2^31.  For all
 * four: t < 2^24 and t * ceil(n / 512) < 2^26 (HM_ERR_SHAPE otherwise). */
hm_status hm_moe_collect_grad(const uint16_t* dout, const uint16_t* ys, const float* w,
                              const int32_t* positions, int64_t t, int32_t topk, int64_t n, uint16_t* dys,
                              float* dw, hipStream_t stream);

/* ------------------------------------------------------ low-rank adapters */

/* Low-rank adapters beside one linear layer (n output, k input features, as
 * its hm_wdesc): adapter e adds B_e A_e x, scaled, to the layer's output.
 * num_adapters are held side by side, and every row of a batch names its own. */
typedef struct hm_lora_desc {
  int32_t abi;          /* HM_ABI_VERSION */
  int32_t rank;         /* a multiple of 8, 8 .. 128 (smaller adapters are padded with zeros) */
  int32_t num_adapters; /* 1 .. 512 */
  int32_t reserved;     /* 0 */
  int64_t n;            /* output features, >= 1 */
  int64_t k;            /* input features, a multiple of 128, >= 128 */
} hm_lora_desc;

/* Workspace bytes hm_lora needs for m rows (may be 0). */
hm_status hm_lora_workspace_size(const hm_lora_desc* d, int64_t m, size_t* bytes);

/* Adapters of many requests at once beside a shared projection:
 *   h[m][:] = scales[e] * A_e x[m],  y[m][:] = bf16( base[m][:] + B_e h[m] ),
 * e = adapter_ids[m]; a row whose id is outside [0, num_adapters) has no
 * adapter: h = 0 and y = base.  Both products accumulate in fp32 and h enters
 * the second one with all its 24 bits (as three bf16 terms).  Infinities and
 * NaN among the inputs give what the formulas give in fp32, where h (here) and
 * g (in hm_lora_grad) are 0 or 2^-90 and more in size; they stay within the
 * rows and matrices of their adapter.
 *   x           bf16 [m][k];  adapter_ids int32 [m], in any order.
 *   a           bf16 [num_adapters][rank][k];  b bf16 [num_adapters][n][rank].
 *   scales      fp32 [num_adapters].
 *   base        bf16 [m][n], the shared projection's output (hm_gemm), or NULL
 *               for zeros.  May be y itself: the adapters are then added in
 *               place, and rows without an adapter are not touched.
 *   y           bf16 [m][n]; must not overlap an input in any other way
 *               (HM_ERR_UNSUPPORTED for x, a, b and base).
 *   h           fp32 [m][rank], what hm_lora_grad needs; NULL if not wanted.
 *   ws          hm_lora_workspace_size bytes, overwritten.
 * h and ws must overlap no other array.
 * m = 0 is a no-op; m up to 1048576, and m * n up to about 10^11 (a launch's
 * blocks; the size query and the call agree): HM_ERR_SHAPE above. */
hm_status hm_lora(const hm_lora_desc* d, const uint16_t* x, const int32_t* adapter_ids, const uint16_t* a,
                  const uint16_t* b, const float* scales, int64_t m, const uint16_t* base, uint16_t* y,
                  float* h, void* ws, size_t ws_bytes, hipStream_t stream);

/* Workspace bytes hm_lora_grad needs for m rows. */
hm_status hm_lora_grad_workspace_size(const hm_lora_desc* d, int64_t m, size_t* bytes);

/* The gradient of hm_lora to its rows and to both adapter matrices:
 *   g[m][:] = scales[e] * B_e^T dy[m],   dx[m][:] = bf16( dx_base[m][:] + A_e^T g[m] ),
 *   da[e] = bf16( sum over the rows m of e of g[m] x[m]^T ),
 *   db[e] = bf16( sum over the rows m of e of dy[m] h[m]^T ),
 * sums in fp32 in an order that the shapes and ids fix (equal calls give
 * equal bits); g and h enter the products with all their 24 bits.  (The gradient
 * to base is dy itself.)
 *   dy          bf16 [m][n];  x bf16 [m][k];  h fp32 [m][rank] from hm_lora.
 *   dx_base     bf16 [m][k], the gradient through the shared projection, or
 *               NULL for zeros; may be dx itself.
 *   dx          bf16 [m][k], or NULL if not wanted.  Rows without an adapter
 *               get dx_base.
 *   da          bf16 [num_adapters][rank][k];  db bf16 [num_adapters][n][rank];
 *               adapters that no row names get zeros.
 *   ws          hm_lora_grad_workspace_size bytes, overwritten.
 * dx, da and db must not overlap an input in any other way (HM_ERR_UNSUPPORTED
 * for dy, x, h, a, b and dx_base), nor each other; ws must overlap no other
 * array.
 * m = 0 writes zeros to da and db; limits as hm_lora. */
hm_status hm_lora_grad(const hm_lora_desc* d, const uint16_t* dy, const uint16_t* x, const float* h,
                       const int32_t* adapter_ids, const uint16_t* a, const uint16_t* b, const float* scales,
                       int64_t m, const uint16_t* dx_base, uint16_t* dx, uint16_t* da, uint16_t* db, void* ws,
                       size_t ws_bytes, hipStream_t stream);

/* ------------------------------------------------- 8-bit integer layers */

/* Linear layers whose activations and weights are both 8-bit integers, with
 * one fp32 scale per token (row of X) and one per output channel (row of W):
 *   x_hat[m,k] = x_scales[m] x8[m,k],   w_hat[n,k] = w_scales[n] w8[n,k]
 * (W8A8 among the GEMM types that the pages list, cocoloop.cn news item, format
 * list; per-token scales: ywsung.com note, section on weight format /
 * activation / backend).  Both are plain row-major int8 arrays, x8 [m][k] and
 * w8 [n][k], as hm_quant_int8_rows writes them (rows of W are its rows too), so
 * weights that change every training step need no repacking.  A training step
 * keeps the codes and scales of its rows, a byte a value, instead of the bf16
 * activations: the gradients below need nothing else of the forward pass.
 *
 * Sizes of all of them: 0 <= m <= 8388480; 1 <= n <= 2^22; k a multiple of 128,
 * 128 .. 130944 (every sum of k products then fits an int32: sums are exact);
 * ceil(m/128) ceil(n/128) <= 2^23, and the same of (m, k) and (n, k) for the
 * gradient.  HM_ERR_SHAPE otherwise.  Codes may be any int8, scales any finite
 * fp32; a NaN or infinite scale makes its row (token) or column (channel) of
 * the results NaN or infinite and leaves the others alone (of the gated
 * calls: a gate row's scale column i of h and columns i and d + i of dgu, an up
 * row's column i of h and of dgu, since du does not depend on u); where it is
 * summed over (hm_gemm_int8_grad) the sums are unspecified.  ws: at least the bytes that the
 * _workspace_size call names (NULL if 0), overwritten; calls that may run at the
 * same time need one each.  bf16 and int8 arrays are
 * 16-byte aligned, scales 4-byte, ws 256-byte (HM_ERR_ALIGN).  No output nor ws
 * may overlap an input or another output (HM_ERR_UNSUPPORTED). */

/* Codes and scales of rows, x bf16 [m][k] -> x8 int8 [m][k], row_scale fp32 [m]:
 *   row_scale[m] = amax_k |x[m,k]| / 127  (fp32 division),
 *   x8[m,k] = the whole number nearest to 127 x[m,k] / amax, ties to even,
 * the quotient exact (codes lie in -127..127).  A row of zeros gives scale 0 and
 * zero codes; a row that holds an infinity or a NaN gives scale NaN and zero
 * codes, so that products of it are NaN.  m = 0 is a no-op; any k >= 1, m k <=
 * 2^39 (HM_ERR_SHAPE). */
hm_status hm_quant_int8_rows(const uint16_t* x, int64_t m, int64_t k, int8_t* x8, float* row_scale,
                             hipStream_t stream);

/* Workspace bytes hm_gemm_int8 needs (may be 0). */
hm_status hm_gemm_int8_workspace_size(int64_t m, int64_t n, int64_t k, size_t* bytes);

/* y[m][n] = bf16( (sum_k x8[m,k] w8[n,k]) x_scales[m] w_scales[n] ): the sum as an
 * exact int32, converted to fp32 and multiplied in fp32 in this order.
 * m = 0 is a no-op. */
hm_status hm_gemm_int8(const int8_t* x8, const float* x_scales, const int8_t* w8, const float* w_scales,
                       int64_t m, int64_t n, int64_t k, uint16_t* y, void* ws, size_t ws_bytes,
                       hipStream_t stream);

/* Workspace bytes of the two gated calls (may be 0); n as there. */
hm_status hm_gemm_int8_gated_workspace_size(int64_t m, int64_t n, int64_t k, size_t* bytes);
hm_status hm_gemm_int8_gated_grad_workspace_size(int64_t m, int64_t n, int64_t k, size_t* bytes);

/* The first half of a gated feed-forward block: both projections, SiLU and the
 * product in one call.  w8 [n][k] holds n = 2d rows, gate rows 0..d-1, up rows
 * d..2d-1 (any d >= 1; an odd n gives HM_ERR_SHAPE); with g and u the fp32
 * products of hm_gemm_int8 before their rounding,
 *   h[m][i] = bf16( silu(g[m,i]) u[m,i] ),  silu(g) = g / (1 + exp(-g)).
 *   h bf16 [m][n/2].  m = 0 is a no-op.  (hm_gemm_int8 followed by hm_silu_mul
 * rounds g and u to bf16 in between.) */
hm_status hm_gemm_int8_gated(const int8_t* x8, const float* x_scales, const int8_t* w8, const float* w_scales,
                             int64_t m, int64_t n, int64_t k, uint16_t* h, void* ws, size_t ws_bytes,
                             hipStream_t stream);

/* The gradient of hm_gemm_int8_gated to its gate and up products, which are
 * computed again from the 8-bit rows (they are never stored): with s = 1 / (1 + exp(-g)),
 *   dgu[m][i]     = bf16( dh[m,i] u s (1 + g (1 - s)) ),
 *   dgu[m][d + i] = bf16( dh[m,i] g s ).
 *   dh bf16 [m][n/2]; dgu bf16 [m][n]: the dy of hm_gemm_int8_grad (and of
 * hm_lora_grad) for the gate_up projection.  m = 0 is a no-op. */
hm_status hm_gemm_int8_gated_grad(const uint16_t* dh, const int8_t* x8, const float* x_scales, const int8_t* w8,
                                  const float* w_scales, int64_t m, int64_t n, int64_t k, uint16_t* dgu, void* ws,
                                  size_t ws_bytes, hipStream_t stream);

/* Workspace bytes hm_gemm_int8_grad needs (for either gradient or both). */
hm_status hm_gemm_int8_grad_workspace_size(int64_t m, int64_t n, int64_t k, size_t* bytes);

/* The gradient of y = x_hat w_hat^T to its factors (quantization passes
 * gradients straight through, so they are those to the bf16 rows and weights
 * that the codes were made from):
 *   dx[m][k] = bf16( sum_n dy[m,n] w~[n,k] ),  w~ = bf16(w_scales[n] w8[n,k]),
 *   dw[n][k] = bf16( sum_m dy[m,n] x~[m,k] ),  x~ = bf16(x_scales[m] x8[m,k]),
 * summed in fp32 in an order that the sizes fix (equal calls give equal bits).
 *   dy bf16 [m][n];  dx bf16 [m][k] and dw bf16 [n][k]: either may be NULL if not
 *   wanted (both: HM_ERR_NULL); the scales and codes that only the other needs
 *   may be NULL then.  m = 0 writes zeros to dw.
 *   dx can be the dx_base of hm_lora_grad where the layer has adapters. */
hm_status hm_gemm_int8_grad(const uint16_t* dy, const int8_t* x8, const float* x_scales, const int8_t* w8,
                            const float* w_scales, int64_t m, int64_t n, int64_t k, uint16_t* dx, uint16_t* dw,
                            void* ws, size_t ws_bytes, hipStream_t stream);

/* Which of the int8 calls a plan is asked for. */
typedef enum hm_int8_op {
  HM_INT8_GEMM = 0,        /* hm_gemm_int8 */
  HM_INT8_GATED = 1,       /* hm_gemm_int8_gated */
  HM_INT8_GATED_GRAD = 2,  /* hm_gemm_int8_gated_grad */
  HM_INT8_GRAD = 3         /* hm_gemm_int8_grad: both gradients, dx first */
} hm_int8_op;

/* A short text naming the kernels and tiles that the call runs for these sizes
 * (no device access); HM_ERR_SHAPE for sizes that the call refuses, HM_ERR_UNSUPPORTED for
 * another op, HM_ERR_NULL without a buffer. */
hm_status hm_gemm_int8_plan(int32_t op, int64_t m, int64_t n, int64_t k, char* buf, size_t buf_len);

/* ------------------------------------------------------------ measurement */

/* Plain-read reference: reads `bytes` bytes of `buf` once with the 16-byte
 * loads the decode GEMM uses for its weights, `unroll` loads in flight per
 * lane (1, 2, 4 or 8) over `blocks` blocks of 256 threads (1 .. 65535), and
 * writes one xor-fold word per block to out[blocks] (so no load is skipped).
 * Computes nothing of the GEMM: its time is the bandwidth floor the
 * weight-streaming kernel is compared against.  bytes a positive multiple of
 * 16; buf and out 16- and 4-byte aligned; HM_ERR_SHAPE / HM_ERR_NULL /
 * HM_ERR_ALIGN before any launch. */
hm_status hm_read_probe(const void* buf, int64_t bytes, int32_t blocks, int32_t unroll, uint32_t* out,
                        hipStream_t stream);

/* Human-readable name of a status code (static string). */
const char* hm_status_string(int32_t status);  /* any value; unknown ones named so */

#ifdef __cplusplus
}
#endif

#endif /* HM_H */
