/*
 * moe_int8.h -- C ABI of libmoe_int8.so: the forward pass of a mixture-of-experts
 * feed-forward layer whose expert weights are stored as int8 (MI355X / gfx950).
 *
 * What the layer computes (Jamba-1.5 paper, "Model Architecture"): an MoE module
 * stands in for the MLP; a router scores n experts per token and the top K are
 * used (n=16, K=2 in Jamba). "Serving Considerations and Improvements" (the
 * ExpertsInt8 scheme): expert weights live in memory as INT8, are turned back
 * into BF16 values inside the fused MoE kernel, and activations stay BF16.
 *
 * Readings of what the paper leaves open, implemented by every call below:
 *   gate    p = softmax(l) over all E logits l = x . router_w[e] (+ bias[e]);
 *           the K largest logits, descending, exact ties to the lower index;
 *           w_k = p_k / sum of p over the K chosen experts.
 *   expert  SwiGLU: o = s_d * (q_d . h), h = silu(g) * u,
 *           g = s_g * (q_g . x), u = s_u * (q_u . x); no biases.
 *   int8    symmetric, one scale per output channel (row of an (out, in)
 *           matrix); moe_quantize_rows below produces the codes and scales.
 *   combine y_t = sum_k w_k * o_{t,k}; no capacity limit, no residual.
 * The contractions run on bf16 MFMA with fp32 accumulation: int8 codes become
 * bf16 exactly, activations given as fp32 are rounded to bf16 at the MFMA input,
 * the per-channel scale is applied to the fp32 sum, h is held as bf16, the
 * per-slot expert outputs (y_rows) as fp32.
 *
 * Conventions (all calls):
 *   - Pointers named x, router_w, y, w_*, s_*, topk_*, expert_offsets,
 *     sorted_slots, slot_to_row, y_rows and workspace are DEVICE pointers on
 *     the current HIP device, row-major, 16-byte aligned. The caller owns
 *     every buffer; the library allocates nothing and keeps no state between
 *     calls, so calls on different streams may run concurrently.
 *   - Work is enqueued on `stream` and is asynchronous; no call synchronises.
 *   - Arguments are validated before anything is enqueued. On error nothing is
 *     launched and a moe_status other than MOE_OK is returned; the message is
 *     available from moe_last_error() on the calling thread. A launch failure
 *     reported by HIP maps to MOE_ERR_HIP. Device-side faults surface at the
 *     caller's next synchronisation.
 *   - Expert weights are (out, in) matrices w_gate, w_up [E, f, d] and
 *     w_down [E, d, f] in the encoding shape->weight_fmt names (int8 unless
 *     stated), held by the FFN calls in the TILED LAYOUT that moe_pack_rows
 *     produces (see there). router_w [E, d] is row-major; scales
 *     s_gate, s_up [E, f], s_down [E, d] are row-major.
 *   - Slots: token t's k-th choice is slot s = t*K + k.
 *   - T = 0 is valid and enqueues nothing; once the shape is valid, no
 *     pointer is then checked (empty tensors may be NULL).
 *   - Debug checks: while the environment variable MOE_DEBUG is set (to a
 *     value other than "0"), the calls that take or produce a permutation
 *     also check it, on the host:
 *       moe_expert_ffn, moe_expert_gate_up, moe_expert_down,
 *       moe_expert_ffn_mxfp4, moe_grouped_mm_mxfp4,
 *       moe_expert_ffn_int8, moe_grouped_mm_int8: expert_offsets starts at
 *         0, never decreases and ends at most at T*K; where sorted_slots is
 *         given, its rows below off[E] hold distinct slots in [0, T*K);
 *       moe_combine, moe_combine_post: every slot_to_row entry is -1 or in [0, T*K);
 *       these run BEFORE anything is launched, so bad caller arrays are
 *       reported instead of being read out of bounds by a kernel;
 *       moe_permute, moe_forward, moe_forward_noalloc, moe_block_forward,
 *       moe_forward_gated, moe_block_forward_gated: after the permutation
 *         is computed, also that every id is in [0, E) (all slots placed),
 *         that each expert's rows hold its own slots in ascending order and
 *         that slot_to_row inverts sorted_slots.
 *     A failed check returns MOE_ERR_CHECK (moe_forward: before the down
 *     pass). The checks copy the arrays to the host and synchronise `stream`:
 *     they are for debugging, not for timed runs or graph capture.
 *   - Logging: while the environment variable MOE_LOG is set (to a value
 *     other than "0"), every call that runs an expert-FFN pass writes one line
 *     per pass to stderr ("[moe] <call> gate/up|down: <shape>; <schedule>"):
 *     the schedule (stream or tiled), and for the stream schedule the rows per
 *     pass, where the expert segments come from, and whether the down pass
 *     splits its reduction over workgroups; with MXFP4 weights the channels of
 *     an item, the rows of a pass and the slices of the reduction, or the tile
 *     and its order. Nothing else changes.
 */
#ifndef MOE_INT8_H
#define MOE_INT8_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t moe_status;
enum {
  MOE_OK = 0,
  MOE_ERR_NULL = 1,        /* a required pointer is NULL */
  MOE_ERR_SHAPE = 2,       /* a size is out of range or not a supported multiple */
  MOE_ERR_DTYPE = 3,       /* unknown dtype code */
  MOE_ERR_ALIGN = 4,       /* a pointer is not 16-byte aligned */
  MOE_ERR_WORKSPACE = 5,   /* workspace missing or smaller than required */
  MOE_ERR_UNSUPPORTED = 6, /* valid request the library does not support */
  MOE_ERR_HIP = 7,         /* a HIP runtime call failed */
  MOE_ERR_CHECK = 8        /* a MOE_DEBUG consistency check failed */
};

/* dtype codes */
enum { MOE_F32 = 0, MOE_BF16 = 1 };

/* Expert weight encodings (moe_shape.weight_fmt). MOE_W_INT8 is the layer
 * itself (ExpertsInt8). The other two are comparators for the paper's claims
 * ("Serving Considerations and Improvements": in-kernel INT8 dequantization is
 * faster than BF16 weights and as fast as FP8):
 *   MOE_W_INT8  int8 codes + per-output-channel scales (moe_quantize_rows);
 *   MOE_W_BF16  the bf16 weights themselves, no scales (s_* unused, may be NULL);
 *   MOE_W_FP8   OCP fp8 e4m3 codes + per-output-channel scales
 *               (moe_quantize_rows_fp8); every e4m3 value is exact in bf16.
 * All three are held in the tiled layout of their bytes (moe_pack_rows; a
 * bf16 matrix [rows, cols] is packed as int8 [rows, 2*cols]). The bf16 and
 * fp8 encodings need bf16 activations; on the TILED schedule their tensors
 * must also fit 32-bit byte offsets (x and h below 4 GiB, one expert's matrix
 * below 4 GiB), else MOE_ERR_UNSUPPORTED.
 *   MOE_W_MXFP4 4-bit codes with one power-of-two scale byte per 32 elements
 *               along the row (moe_quantize_mxfp4), a quarter of bf16's bytes.
 *               The w_* pointers hold the tiled codes, the s_* pointers the
 *               tiled scale bytes ([E, out, in/32]; scale_dtype is not used).
 *               Codes become bf16, scale included, so the products are exact
 *               (subnormal operands too) and the sums fp32 as for the others;
 *               weights of 2^128 and more, past bf16's largest number (codes
 *               of 4 and 6 under scale byte 253, of 2 and more under 254),
 *               become infinite. bf16 activations
 *               (else MOE_ERR_UNSUPPORTED), d and f multiples of 128 (else
 *               MOE_ERR_SHAPE). A pass that reads 4 GiB or more of x (gate/up)
 *               or h (down) takes the STREAM schedule on AUTO; asked for TILED
 *               it is refused with MOE_ERR_UNSUPPORTED.
 * Code 3 is not assigned. */
enum { MOE_W_INT8 = 0, MOE_W_BF16 = 1, MOE_W_FP8 = 2, MOE_W_MXFP4 = 4 };

/* expert-FFN schedule: AUTO picks STREAM when at most 64 rows fall on each
 * expert on average (T*K <= 64*E: decode) and TILED otherwise (prefill); with
 * MXFP4 weights the border is 16 rows for the down pass, 8 for the gate/up
 * pass and for products with MXFP4 activations (32 and 20 with few output
 * channels over all experts).
 * Both give results within the same tolerance of the exact layer; they are
 * not bit-identical to each other. Each is deterministic. */
enum { MOE_PATH_AUTO = 0, MOE_PATH_STREAM = 1, MOE_PATH_TILED = 2 };

typedef struct moe_shape {
  int32_t T;           /* tokens, >= 0                                     */
  int32_t d;           /* hidden size, multiple of 64, 64..65536            */
  int32_t f;           /* expert FFN width, multiple of 64, 64..131072      */
  int32_t E;           /* experts, 1..64                                    */
  int32_t K;           /* experts per token, 1..min(E, 8)                   */
  int32_t act_dtype;   /* x, router_w, y: MOE_F32 or MOE_BF16               */
  int32_t scale_dtype; /* s_gate, s_up, s_down: MOE_F32 or MOE_BF16         */
  int32_t ffn_path;    /* MOE_PATH_*                                        */
  int32_t weight_fmt;  /* MOE_W_*: encoding of w_gate, w_up, w_down        */
} moe_shape;

/* ABI version of this header (bumped on any signature change, and with new calls). */
#define MOE_ABI_VERSION 8
int32_t moe_abi_version(void);

/* Static description of a status code. */
const char* moe_status_str(moe_status status);

/* Message of the last failed call on this thread ("" if none). */
const char* moe_last_error(void);

/* Workspace, in bytes, that moe_forward needs for this shape (includes the
 * routing buffers, the permutation, h, y_rows and the FFN passes' own
 * workspaces, see moe_gate_up_workspace_size and moe_down_workspace_size). */
moe_status moe_workspace_size(const moe_shape* shape, size_t* bytes);

/* Workspace, in bytes, that moe_expert_ffn needs: h (T*K*f bf16), then the
 * down pass's workspace (moe_down_workspace_size), then the gate/up pass's
 * (moe_gate_up_workspace_size), each padded to 256. */
moe_status moe_ffn_workspace_size(const moe_shape* shape, size_t* bytes);

/* Workspace, in bytes, that the down pass can use:
 *   - STREAM schedule: fp32 partial sums [planes, T*K, d] for shapes whose
 *     weight-streaming down pass splits its reduction over workgroups (33 to
 *     64 rows per expert on average and too few output-channel groups to fill
 *     the GPU, e.g. a dense MLP at decode); 0 for every other stream shape;
 *   - TILED schedule: 256 bytes of tile claim words (see moe_expert_down). */
moe_status moe_down_workspace_size(const moe_shape* shape, size_t* bytes);

/* Workspace, in bytes, that the gate/up pass can use: 256 bytes of tile claim
 * words on the TILED schedule, 0 on the STREAM schedule (see moe_expert_gate_up). */
moe_status moe_gate_up_workspace_size(const moe_shape* shape, size_t* bytes);

/* Router and gate (paper: "Model Architecture", top K of n experts per token).
 *   x           [T, d]  act_dtype
 *   router_w    [E, d]  act_dtype
 *   router_bias [E] fp32 added to the logits, or NULL
 *   topk_ids    [T, K] int32 out: chosen experts, descending logit
 *   topk_w      [T, K] fp32  out: renormalised gate weights (sum to 1 per token)
 * Logits are fp32 dot products of the exact inputs. */
moe_status moe_route(const moe_shape* shape, const void* x, const void* router_w,
                     const float* router_bias, int32_t* topk_ids, float* topk_w,
                     hipStream_t stream);

/* Group the T*K slots by expert (stable: ascending slot inside an expert).
 * Source: Jamba-1.5 paper, "Model Architecture": each token is sent to the
 * top K of n experts, so every expert sees its own subset of the tokens; this
 * call gathers each expert's slots into one contiguous segment.
 *   topk_ids       [T*K] int32 in, values in [0, E)
 *   expert_offsets [E+1] int32 out: expert e owns sorted rows [off[e], off[e+1])
 *   sorted_slots   [T*K] int32 out: slot held by each sorted row
 *   slot_to_row    [T*K] int32 out: sorted row of each slot
 * An id outside [0, E) is not placed: its slot_to_row entry is -1 and the
 * sorted rows past off[E] hold -1. Bit-exact and deterministic. */
moe_status moe_permute(const moe_shape* shape, const int32_t* topk_ids,
                       int32_t* expert_offsets, int32_t* sorted_slots,
                       int32_t* slot_to_row, hipStream_t stream);

/* Expert SwiGLU FFNs on the permuted rows (the ExpertsInt8 contraction).
 * Source: Jamba-1.5 paper, "Serving Considerations and Improvements": the
 * expert weights stay INT8 in memory and become BF16 values inside the fused
 * MoE kernel, right before the contraction; activations stay BF16.
 *   x              [T, d] act_dtype (row of sorted row r is token sorted_slots[r] / K)
 *   expert_offsets [E+1], sorted_slots [T*K] from moe_permute
 *   w_gate, w_up   [E, f, d];  w_down [E, d, f] -- shape->weight_fmt encoding, tiled layout (moe_pack_rows)
 *   s_gate, s_up   [E, f] scale_dtype;  s_down [E, d] scale_dtype (unused for MOE_W_BF16)
 *   y_rows         [T*K, d] fp32 out: row r = output of sorted row r's expert
 *   workspace      >= moe_ffn_workspace_size bytes (holds h and the down pass's partial sums)
 * Rows past off[E] are left untouched. */
moe_status moe_expert_ffn(const moe_shape* shape, const void* x,
                          const int32_t* expert_offsets, const int32_t* sorted_slots,
                          const void* w_gate, const void* w_up, const void* w_down,
                          const void* s_gate, const void* s_up, const void* s_down,
                          float* y_rows, void* workspace, size_t workspace_bytes,
                          hipStream_t stream);

/* The two passes of moe_expert_ffn, callable on their own (same kernels;
 * source as moe_expert_ffn: Jamba-1.5 paper, "Serving Considerations and
 * Improvements"):
 * gate/up  h[r] = silu(s_g * (q_g . x_r)) * (s_u * (q_u . x_r))  for every sorted row r,
 *          h [T*K, f] bf16 out (rows past off[E] untouched).
 * down     y_rows[r] = s_d * (q_d . h[r]),  h [T*K, f] bf16 in, y_rows [T*K, d] fp32 out.
 * workspace (both passes): NULL, or 16-byte aligned and at least
 *          moe_gate_up_workspace_size / moe_down_workspace_size bytes (else
 *          MOE_ERR_ALIGN / MOE_ERR_WORKSPACE). Its contents need not be
 *          initialised. With it:
 *          - on the TILED schedule, the last tiles of each XCD's share are
 *            claimed through atomic counters in the workspace (cleared by the
 *            pass itself) by the workgroups of any XCD, so XCDs that run
 *            faster take more tiles; without it every workgroup's tile is
 *            fixed by its id;
 *          - on the STREAM schedule, a down pass that splits its reduction
 *            may spread the slices over workgroups (partial sums in the
 *            workspace, added in slice order by a second kernel); without it
 *            the slices stay inside one workgroup.
 *          The results are the same bit for bit either way.
 * moe_expert_ffn is moe_expert_gate_up followed by moe_expert_down on the same
 * stream, with the parts of its workspace after h as their workspaces. */
moe_status moe_expert_gate_up(const moe_shape* shape, const void* x, const int32_t* expert_offsets,
                              const int32_t* sorted_slots, const void* w_gate, const void* w_up,
                              const void* s_gate, const void* s_up, void* h, void* workspace,
                              size_t workspace_bytes, hipStream_t stream);
moe_status moe_expert_down(const moe_shape* shape, const void* h, const int32_t* expert_offsets,
                           const void* w_down, const void* s_down, float* y_rows, void* workspace,
                           size_t workspace_bytes, hipStream_t stream);

/* Weighted combine back to token order: y[t] = sum_k topk_w[t,k] * y_rows[slot_to_row[t*K+k]]
 * Source: Jamba-1.5 paper, "Model Architecture": the MoE module takes the
 * place of the MLP, so its output is the gate-weighted sum of the K chosen
 * experts' outputs, one [d] vector per token.
 * (k ascending, fp32, no atomics); a slot with row -1 contributes nothing.
 *   y [T, d] act_dtype out. */
moe_status moe_combine(const moe_shape* shape, const float* y_rows, const int32_t* slot_to_row,
                       const float* topk_w, void* y, hipStream_t stream);

/* The whole layer: route, permute, expert FFN, combine, enqueued on `stream`.
 * Sources: Jamba-1.5 paper, "Model Architecture" (an MoE module with n
 * experts, top K per token, in place of the MLP) and "Serving Considerations
 * and Improvements" (ExpertsInt8: int8 expert weights dequantized to BF16
 * inside the fused kernel).
 * Bit-identical to the four staged calls above with the same ffn_path.
 *   topk_ids_out [T, K] / topk_w_out [T, K]: optional copies of the routing (NULL to skip)
 *   workspace    >= moe_workspace_size bytes */
moe_status moe_forward(const moe_shape* shape, const void* x, const void* router_w,
                       const float* router_bias,
                       const void* w_gate, const void* w_up, const void* w_down,
                       const void* s_gate, const void* s_up, const void* s_down,
                       void* y, int32_t* topk_ids_out, float* topk_w_out,
                       void* workspace, size_t workspace_bytes, hipStream_t stream);

/* moe_forward without a caller workspace, for callers that cannot allocate
 * device memory (code under HIP graph capture, tight serving loops, harnesses
 * that forbid hipMalloc). Same arguments and results as moe_forward (bit for
 * bit), minus the workspace: the library keeps a fixed 32 MiB scratch array in
 * device memory on each GPU it runs on (held until the process ends) and uses
 * it as the workspace. A shape whose moe_workspace_size exceeds 32 MiB is
 * rejected with MOE_ERR_WORKSPACE before anything is enqueued (every
 * decode-sized layer fits: Jamba-1.5-Large at T=64 needs about 11 MiB). The
 * call allocates nothing. All calls on one GPU share that GPU's scratch, which
 * keeps the last call's contents: calls that overlap on one GPU (concurrent
 * streams, or host threads) race and must be serialised by the caller. */
moe_status moe_forward_noalloc(const moe_shape* shape, const void* x, const void* router_w,
                               const float* router_bias,
                               const void* w_gate, const void* w_up, const void* w_down,
                               const void* s_gate, const void* s_up, const void* s_down,
                               void* y, int32_t* topk_ids_out, float* topk_w_out, hipStream_t stream);

/* Dense int8-weight MLP (Jamba-1.5 paper, "Serving Considerations and
 * Improvements": ExpertsInt8 quantizes the MoE *and* the MLP weights). An MLP
 * layer is the MoE layer with one expert used by every token with weight 1:
 *   y = s_d * (q_d . h),  h = silu(s_g * (q_g . x)) * (s_u * (q_u . x)).
 * shape->E and shape->K must be 1; no router. Same kernels, weight encodings
 * and layouts as the MoE calls, same tolerance; the result is bitwise that of
 * moe_expert_ffn followed by moe_combine with weight 1 (when the down pass
 * splits its reduction over workgroups, the kernel that adds the slices
 * writes y itself).
 *   y [T, d] act_dtype out; workspace >= moe_mlp_workspace_size bytes. */
moe_status moe_mlp_workspace_size(const moe_shape* shape, size_t* bytes);
moe_status moe_mlp_forward(const moe_shape* shape, const void* x,
                           const void* w_gate, const void* w_up, const void* w_down,
                           const void* s_gate, const void* s_up, const void* s_down, void* y,
                           void* workspace, size_t workspace_bytes, hipStream_t stream);

/* ExpertsInt8 quantizer (paper: "Serving Considerations and Improvements":
 * quantized at load time in seconds, no calibration). Row-wise symmetric int8:
 *   a = max_i |w[r, i]|,  s[r] = a / 127 rounded once (nearest-even) to scale_dtype,
 *   q[r, i] = round-half-even(w[r, i] / s[r]) clamped to [-127, 127];
 *   an all-zero row gives s = 0 and q = 0.
 *   w [rows, cols] src_dtype (MOE_F32 or MOE_BF16), q [rows, cols] int8, s [rows].
 * Quantizing an (out, in) weight [E, out, in] is rows = E*out, cols = in.
 * cols must be a multiple of 16, 16..1048576. Non-finite inputs give
 * unspecified codes. Bit-exact (the rounding decisions are exact). */
moe_status moe_quantize_rows(int64_t rows, int32_t cols, int32_t src_dtype, const void* w,
                             int32_t scale_dtype, int8_t* q, void* s, hipStream_t stream);

/* FP8 comparator quantizer: as moe_quantize_rows with OCP e4m3 codes (the
 * paper compares ExpertsInt8 with FP8 weights, "Serving Considerations and
 * Improvements"). Row-wise symmetric, one scale per output channel:
 *   s[r] = max_i |w[r, i]| / 448 rounded once (nearest-even) to scale_dtype,
 *   q[r, i] = byte of the e4m3 value nearest to w[r, i] / s[r] (ties to the
 *   even mantissa), saturated to +-448; a zero value is byte 0x00;
 *   an all-zero row gives s = 0 and q = 0.
 * e4m3: sign, 4 exponent bits (bias 7), 3 mantissa bits, subnormals m*2^-9,
 * largest finite 448, bytes 0x7F/0xFF NaN (never produced).
 * Same sizes, dtypes and errors as moe_quantize_rows. Bit-exact. */
moe_status moe_quantize_rows_fp8(int64_t rows, int32_t cols, int32_t src_dtype, const void* w,
                                 int32_t scale_dtype, uint8_t* q, void* s, hipStream_t stream);

/* Quantizer and packer in one pass (load time: "Serving Considerations and
 * Improvements", quantized in seconds when the model is loaded): the codes of
 * moe_quantize_rows (weight_fmt MOE_W_INT8) or moe_quantize_rows_fp8
 * (MOE_W_FP8), written straight into the tiled layout of moe_pack_rows, so
 * the weights are read and the codes written once. Same scales, same codes
 * bit for bit as quantizing then packing.
 *   w [rows, cols] src_dtype in (rows % 16 == 0, cols % 64 == 0),
 *   q_tiled [rows*cols] bytes out (tiled layout), s [rows] scale_dtype out.
 * Errors as moe_quantize_rows; other weight_fmt values: MOE_ERR_DTYPE. */
moe_status moe_quantize_pack_rows(int64_t rows, int32_t cols, int32_t src_dtype, const void* w,
                                  int32_t scale_dtype, int32_t weight_fmt, void* q_tiled, void* s,
                                  hipStream_t stream);

/* Tiled int8 layout of the expert weights (load time, next to the quantizer).
 * The kernels read a wavefront's MFMA operands as whole 1 KiB blocks: a
 * row-major int8 matrix q [rows, cols] (rows % 16 == 0, cols % 64 == 0) is
 * stored as blocks of 16 rows x 64 columns; block (rg, ks) covers rows
 * 16*rg..+16 and columns 64*ks..+64 and sits at block index rg*(cols/64) + ks;
 * inside it, element (r, c) is byte 256*(c/16) + 16*r + (c%16). An expert
 * tensor [E, out, in] is packed as rows = E*out, cols = in.
 *   q [rows, cols] int8 row-major in, packed [rows*cols] int8 out (not in place).
 * A byte permutation: bit-exact. */
moe_status moe_pack_rows(int64_t rows, int32_t cols, const int8_t* q, int8_t* packed, hipStream_t stream);

/* ---------------------------------------------------------------- MXFP4
 * Microscaled 4-bit floating point (OCP MX): along a row of a matrix, each
 * block of 32 elements has one scale byte b worth 2^(b - 127) (255: not a
 * number), and an element is a 4-bit e2m1 code: sign, then the magnitudes
 * 0, 0.5, 1, 1.5, 2, 3, 4, 6. Two codes a byte, the even element in the low
 * half.
 *
 * Layouts of codes and scales:
 *   MOE_MX_ROWS   row-major: codes [rows, cols/2], scales [rows, cols/32];
 *                 cols a multiple of 32, 32..1048576.
 *   MOE_MX_TILED  what the kernels read weights in (rows % 16 == 0, cols % 128
 *                 == 0). Codes: the layout of moe_pack_rows over the cols/2
 *                 bytes of a row. Scales: with n = cols/128, the scale of row
 *                 r, columns 32*c .. +32 is byte
 *                   (r/16)*n*64 + 256*(k/4) + m*(16*(c%4) + r%16) + k%4,
 *                   k = c/4, m = min(4, n - 4*(k/4)).
 *                 An expert tensor [E, out, in] is rows = E*out, cols = in.
 *                 Fewer than 2^37 elements. */
enum { MOE_MX_ROWS = 0, MOE_MX_TILED = 1 };

/* Quantizer. Per block: b = floor(log2(max |w|)) - 2 + 127, at least 0 (an
 * all-zero block: 0); code = the e2m1 value nearest to w / 2^(b - 127), ties to
 * the even code, saturated to +-6, with the sign of w (so of -0 too). A block
 * holding an infinity or a NaN gets b = 255 and zero codes. Bit-exact.
 *   w [rows, cols] src_dtype in, q [rows*cols/2] and s [rows*cols/32] bytes out
 *   in `layout`; rows in [0, 2^31). */
moe_status moe_quantize_mxfp4(int64_t rows, int32_t cols, int32_t src_dtype, const void* w, int32_t layout,
                              uint8_t* q, uint8_t* s, hipStream_t stream);

/* The numbers that codes and scales stand for, in dst_dtype (exact; past the
 * type's largest number: infinite; a scale of 255: NaN). */
moe_status moe_dequantize_mxfp4(int64_t rows, int32_t cols, int32_t layout, const uint8_t* q, const uint8_t* s,
                                int32_t dst_dtype, void* w, hipStream_t stream);

/* Row-major codes and scales (a checkpoint's) -> MOE_MX_TILED; not in place. */
moe_status moe_pack_mxfp4(int64_t rows, int32_t cols, const uint8_t* q, const uint8_t* s, uint8_t* q_tiled,
                          uint8_t* s_tiled, hipStream_t stream);

/* Product grouped by expert, both operands in MXFP4 (the layer's own
 * contraction with 4-bit activations: the scaled MFMA takes both as they are).
 *   row r of expert e's segment [off[e], off[e+1]):
 *     out[r, n] = sum_k A[row(r), k] * W_e[n, k],                   n < f, k < d
 *     or, with a second matrix, silu(W_e . a) * (W2_e . a).
 *   shape: T tokens, K slots a token (rows of out: T*K; 1..8, more than E too: a
 *     shard holds some of a token's experts), d the reduction, f the output
 *     channels, E experts; weight_fmt MOE_W_MXFP4 (else MOE_ERR_DTYPE);
 *     act_dtype is out's type; scale_dtype is not used; ffn_path as for the
 *     expert FFN; d and f multiples of 128.
 *   a_q, a_s  codes and scales of A, row-major, d columns. With sorted_slots
 *     [T*K]: [T, .], row(r) = sorted_slots[r] / K; NULL: [T*K, .], row(r) = r.
 *   w_q, w_s, w2_q, w2_s  [E, f, d] tiled codes and scales (w2_*: both NULL for
 *     the plain product).
 *   out [T*K, f] act_dtype; rows past off[E] are left untouched.
 * Products are exact (within the range of fp32), sums fp32, one rounding. Any
 * segment lengths. Rows of codes past 32-bit byte offsets (4 GiB) take the
 * STREAM schedule throughout. */
moe_status moe_grouped_mm_mxfp4(const moe_shape* shape, const uint8_t* a_q, const uint8_t* a_s,
                                const int32_t* expert_offsets, const int32_t* sorted_slots, const uint8_t* w_q,
                                const uint8_t* w_s, const uint8_t* w2_q, const uint8_t* w2_s, void* out,
                                hipStream_t stream);

/* The expert FFN with MXFP4 weights AND activations, on the permuted rows:
 * x is quantized per token, gate/up with SwiGLU gives h (bf16), h is quantized
 * per row, down gives y_rows. As moe_expert_ffn with 4-bit products (2.5
 * times as fast at prefill) and the rounding of 4-bit activations.
 *   weight_fmt MOE_W_MXFP4; act_dtype is x's type; d, f multiples of 128;
 *   workspace >= moe_expert_ffn_mxfp4_workspace_size bytes. */
moe_status moe_expert_ffn_mxfp4_workspace_size(const moe_shape* shape, size_t* bytes);
moe_status moe_expert_ffn_mxfp4(const moe_shape* shape, const void* x, const int32_t* expert_offsets,
                                const int32_t* sorted_slots, const uint8_t* w_gate, const uint8_t* w_up,
                                const uint8_t* w_down, const uint8_t* s_gate, const uint8_t* s_up,
                                const uint8_t* s_down, float* y_rows, void* workspace, size_t workspace_bytes,
                                hipStream_t stream);

/* ---------------------------------------------------------------- gated routing
 * moe_route with a choice of scores, a bias that counts for the choice only (it
 * balances the experts' load), groups of experts, and weights as they are or
 * renormalised, scaled:
 *   l_e = x . router_w[e] (+ router_bias[e]);  s = softmax(l) over the E experts, or s_e = sigmoid(l_e)
 *   c_e = s_e + select_bias[e]
 *   a group is E / groups consecutive experts; its value is the largest c in it,
 *     or the sum of its two largest; the group_topk groups of the largest values stay
 *   of their experts the K with the largest c are taken, in descending order;
 *   w_k = s_k, divided by the sum of the K if renorm (0 if that is 0), times scale.
 * Ties, among groups too, go to the lower index. An expert whose c is -inf (a
 * bias of -inf takes it out of service) or NaN is never taken, and counts as
 * -inf for its group (as does a sum that is no number); where fewer than K are left, the other ids are -1 with
 * weight 0 (moe_permute does not place such slots, and they add nothing to the
 * combine). A token whose scores are no numbers gets ids of -1.
 * The values that decide the choice are compared in 64 bits, from exact inputs;
 * the weights come from logits with fp32 sums. */
enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 };
enum { MOE_GROUP_MAX = 0, MOE_GROUP_TOP2 = 1 };

typedef struct moe_gate {
  const float* select_bias; /* [E], or NULL: 0                                     */
  int32_t score;            /* MOE_SCORE_*                                         */
  int32_t groups;           /* 1..64, divides E; 1: no groups                      */
  int32_t group_topk;       /* 1..groups, group_topk * E / groups >= K             */
  int32_t group_by;         /* MOE_GROUP_*; TOP2 with two experts a group at least */
  int32_t renorm;           /* 0 or 1                                              */
  float scale;              /* finite                                              */
} moe_gate;

/* As moe_route; here shape->E may be up to 256 (a GPU that holds some of them, K at
 * least, permutes ids less its first expert's: ids outside [0, its experts) are not
 * placed; MOE_DEBUG's check of moe_permute reports such ids, -1 among them).
 *   workspace: NULL, or 16-byte aligned and at least moe_route_gated_workspace_size
 *     bytes (0 for shapes that have no use for it). With it the rows of few tokens
 *     are split over workgroups (half as long for 63 tokens and 64 experts). */
moe_status moe_route_gated_workspace_size(const moe_shape* shape, size_t* bytes);
moe_status moe_route_gated(const moe_shape* shape, const moe_gate* gate, const void* x, const void* router_w,
                           const float* router_bias, int32_t* topk_ids, float* topk_w, void* workspace,
                           size_t workspace_bytes, hipStream_t stream);

/* ---------------------------------------------------------------- int8 activations
 * Products of int8 rows, a scale each (moe_quantize_rows with fp32 scales), and the
 * layer's int8 weights, with both operands as they are in the int8 MFMA.
 *
 * Grouped by expert: row r of expert e's segment [off[e], off[e+1]):
 *     p[r, n] = a_s[row(r)] * w_s[e, n] * sum_k a_q[row(r), k] * w_q[e, n, k],    n < f, k < d
 *     out = p, or with a second matrix silu(p) * p2.
 *   shape: T tokens, K slots a token (rows of out: T*K; 1..8, more than E too: a
 *     shard holds some of a token's experts), d the reduction, f the output
 *     channels, E experts; weight_fmt MOE_W_INT8 (else MOE_ERR_DTYPE); act_dtype is
 *     out's type, scale_dtype that of w_s, w2_s; ffn_path as for the expert FFN.
 *   a_q, a_s  [rows, d] int8 row-major, [rows] fp32. With sorted_slots [T*K]: rows
 *     = T, row(r) = sorted_slots[r] / K; NULL: rows = T*K, row(r) = r.
 *   w_q, w_s, w2_q, w2_s  [E, f, d] tiled codes (moe_pack_rows) and [E, f] scales
 *     (w2_*: both NULL for the plain product).
 *   out [T*K, f] act_dtype, not overlapping any input (MOE_ERR_UNSUPPORTED); rows past off[E] are left untouched.
 * The sums are exact in int32; a sum becomes fp32 and takes its two scales there.
 * Any segment lengths. The schedules give the same bits; with
 * sorted_slots rows of a_q of 4 GiB and more take STREAM, whatever ffn_path asks for. */
moe_status moe_grouped_mm_int8(const moe_shape* shape, const int8_t* a_q, const float* a_s,
                               const int32_t* expert_offsets, const int32_t* sorted_slots, const int8_t* w_q,
                               const void* w_s, const int8_t* w2_q, const void* w2_s, void* out, hipStream_t stream);

/* The expert FFN with int8 weights AND activations, on the permuted rows: x is
 * quantized per token, gate/up with SwiGLU gives h (bf16), h is quantized per row
 * (moe_quantize_rows, fp32 scales), down gives y_rows. Rows past off[E] are neither
 * read nor written, in the workspace too. As moe_expert_ffn with int8
 * products (0.6 times as long at prefill) and the rounding of int8 activations. A
 * token with an infinity or a NaN, in x or h, gives unspecified numbers.
 *   weight_fmt MOE_W_INT8; act_dtype is x's type;
 *   workspace >= moe_expert_ffn_int8_workspace_size bytes. */
moe_status moe_expert_ffn_int8_workspace_size(const moe_shape* shape, size_t* bytes);
moe_status moe_expert_ffn_int8(const moe_shape* shape, const void* x, const int32_t* expert_offsets,
                               const int32_t* sorted_slots, const int8_t* w_gate, const int8_t* w_up,
                               const int8_t* w_down, const void* s_gate, const void* s_up, const void* s_down,
                               float* y_rows, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* The layer with a gate and a choice of activations: moe_route_gated, moe_permute, the
 * expert FFN (expert_act MOE_ACT_AS_IS: moe_expert_ffn, any weight encoding;
 * MOE_ACT_INT8: moe_expert_ffn_int8, weight_fmt MOE_W_INT8), moe_combine. Bit-identical to these
 * staged calls. shape->E up to 64, as for the other calls with weights. Slots
 * whose id is -1 are not placed and add nothing.
 *   workspace >= moe_gated_workspace_size bytes; the other arguments as in moe_forward.
 * Under MOE_DEBUG ids of -1 pass the check of the permutation. */
enum { MOE_ACT_AS_IS = 0, MOE_ACT_INT8 = 1 };
moe_status moe_gated_workspace_size(const moe_shape* shape, int32_t expert_act, size_t* bytes);
moe_status moe_forward_gated(const moe_shape* shape, const moe_gate* gate, int32_t expert_act, const void* x,
                             const void* router_w, const float* router_bias, const void* w_gate, const void* w_up,
                             const void* w_down, const void* s_gate, const void* s_up, const void* s_down, void* y,
                             int32_t* topk_ids_out, float* topk_w_out, void* workspace, size_t workspace_bytes,
                             hipStream_t stream);

/* ---------------------------------------------------------------- norms around the layer
 * rms(v) = v / sqrt(mean(v^2) + eps) over the d elements of a token, in fp32 (a
 * sum of squares past the fp32 range is infinite, as from an infinite element:
 * the token's finite elements become 0).
 *
 * Before the layer: n = rms(x) * weight.
 *   x, n [T, d], weight [d], all act_dtype; n may be x, and not overlap it
 *   otherwise (MOE_ERR_UNSUPPORTED). eps >= 0, finite. */
moe_status moe_norm_pre(const moe_shape* shape, const void* x, const void* weight, float eps, void* n,
                        hipStream_t stream);

/* After the layer, with y its output:
 *   out  = residual_scale * residual + block_scale * gate * (rms(y) * weight)
 *   next = rms(out) * next_weight      (the next block's moe_norm_pre)
 * in one pass, each rounded once; next is taken from the unrounded sum. */
typedef struct moe_post {
  const void* weight;      /* [d] act_dtype, or NULL: y without the norm                       */
  const void* gate;        /* [ceil(T / gate_tokens), d] act_dtype, token t takes row t /
                              gate_tokens; NULL: 1                                             */
  const void* next_weight; /* [d] act_dtype, or NULL: no next                                  */
  int32_t gate_tokens;     /* tokens that share a row of the gate, >= 1 (read with gate only)  */
  float residual_scale, block_scale;
  float eps, next_eps;     /* >= 0, finite                                                     */
} moe_post;

/* y [T, d], residual [T, d], out [T, d], next [T, d] (NULL without next_weight),
 * all act_dtype; out may be residual or y, next may be residual or y but not out;
 * other overlaps of these, and of out or next with post's arrays, are refused
 * (MOE_ERR_UNSUPPORTED). */
moe_status moe_norm_post(const moe_shape* shape, const moe_post* post, const void* y, const void* residual, void* out,
                         void* next, hipStream_t stream);

/* The same with y taken from the experts' rows, as moe_combine does (K = 1..8,
 * a slot with row -1 contributes nothing) but unrounded: one pass in place of
 * the combine and the norm. out and next may not overlap y_rows either. */
moe_status moe_combine_post(const moe_shape* shape, const moe_post* post, const float* y_rows,
                            const int32_t* slot_to_row, const float* topk_w, const void* residual, void* out,
                            void* next, hipStream_t stream);

/* A block: moe_norm_pre of the residual stream, the layer (moe_forward's steps
 * on it), moe_combine_post onto the stream; any weight encoding.
 *   residual [T, d] act_dtype; pre_weight [d] or NULL : x is given instead
 *   x [T, d] or NULL: the layer's input (the `next` of the block before), read
 *   when pre_weight is NULL; exactly one of the two is given
 *   out, next as in moe_norm_post (out may be residual)
 *   workspace >= moe_block_workspace_size bytes. */
moe_status moe_block_workspace_size(const moe_shape* shape, size_t* bytes);
moe_status moe_block_forward(const moe_shape* shape, const void* residual, const void* pre_weight, float pre_eps,
                             const void* x, const moe_post* post, const void* router_w, const float* router_bias,
                             const void* w_gate, const void* w_up, const void* w_down, const void* s_gate,
                             const void* s_up, const void* s_down, void* out, void* next, int32_t* topk_ids_out,
                             float* topk_w_out, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* The block with moe_forward_gated's steps in place of moe_forward's.
 *   workspace >= moe_block_gated_workspace_size bytes; the other arguments as in moe_block_forward. */
moe_status moe_block_gated_workspace_size(const moe_shape* shape, int32_t expert_act, size_t* bytes);
moe_status moe_block_forward_gated(const moe_shape* shape, const moe_gate* gate, int32_t expert_act,
                                   const void* residual, const void* pre_weight, float pre_eps, const void* x,
                                   const moe_post* post, const void* router_w, const float* router_bias,
                                   const void* w_gate, const void* w_up, const void* w_down, const void* s_gate,
                                   const void* s_up, const void* s_down, void* out, void* next, int32_t* topk_ids_out,
                                   float* topk_w_out, void* workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_INT8_H */
