// Launchers of the gfx950 kernels (host side). Arguments are validated by the
// C ABI layer before any of these is called; each returns the HIP status of
// its launch.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

hipError_t launch_router(const void* x, const void* router_w, const float* bias, int T, int d, int E, int K,
                         bool act_bf16, int32_t* topk_ids, float* topk_w, hipStream_t stream);

hipError_t launch_permute(const int32_t* ids, int S, int E, int32_t* offsets, int32_t* sorted_slots,
                          int32_t* slot_to_row, hipStream_t stream);

// Arguments of the expert FFN (both schedules).
struct FfnArgs {
  const void* x;              // [T, d] activations
  bool act_bf16;              // x dtype
  bool scale_bf16;            // scale dtype
  const int32_t* offsets;     // [E + 1]
  const int32_t* sorted_slots;  // [S]
  int wfmt;                   // weight encoding (WFmt: int8, bf16 or fp8)
  const int8_t* w_gate;       // [E, f, d], tiled layout of the weight bytes
  const int8_t* w_up;         // [E, f, d], tiled layout of the weight bytes
  const int8_t* w_down;       // [E, d, f], tiled layout of the weight bytes
  const void* s_gate;         // [E, f] (unused for bf16 weights)
  const void* s_up;           // [E, f]
  const void* s_down;         // [E, d]
  __bf16* h;                  // [S, f] scratch
  float* y_rows;              // [S, d] out
  float* part;                // [planes, S, d] scratch of a down pass split over workgroups, or null
  // A dense layer (E = K = 1, every token its own row with weight 1) whose
  // down pass splits its reduction over workgroups: the sum of the slices goes
  // straight to y ([T, d], act dtype), as the combine would write it, and
  // y_rows is not written. Null otherwise.
  void* y_dense;
  // gate/up from the expert ids (S <= 256, 32-row stream pass): ids [S] in,
  // the permutation (offsets, sorted_slots, slot_to_row) out; null otherwise
  const int32_t* ids;
  int32_t* perm_offsets;
  int32_t* perm_sorted;
  int32_t* perm_s2r;
  // tile claim words of the tiled gate/up and down passes ([8] each, zeroed by
  // the pass before use), or null: the static tile order throughout
  unsigned long long* claims_gate_up;
  unsigned long long* claims_down;
  int T, d, f, E, K, S;
};

// Bytes of one tiled pass's tile claim words (eight 64-bit words, padded).
constexpr size_t kTileClaimBytes = 256;

// Weight-streaming schedule for few rows per expert (decode): gate/up pass
// (x -> h) and down pass (h -> y_rows).
hipError_t launch_stream_gate_up(const FfnArgs& a, hipStream_t stream);
hipError_t launch_stream_down(const FfnArgs& a, hipStream_t stream);
// Partial-sum planes ([planes, S, d] fp32, in FfnArgs::part) with which the
// stream down pass splits its reduction over workgroups; 0: it does not. With
// part null the pass keeps the split inside one workgroup, with the same result.
int stream_down_planes(long S, int d, int f, int E);
// Whether the stream gate/up pass can take the expert ids instead of a
// permutation (FfnArgs::ids): at most 256 slots on the 32-row variant.
bool stream_gate_up_takes_ids(long S, int E);
// Tiled MFMA schedule for many rows per expert (prefill). bf16 and fp8
// weights need bf16 activations and dma_offsets_fit(T, S, d, f, bytes per
// weight); int8 weights take any shape.
bool dma_offsets_fit(long T, long S, long d, long f, int wbytes);
hipError_t launch_tiled_gate_up(const FfnArgs& a, hipStream_t stream);
hipError_t launch_tiled_down(const FfnArgs& a, hipStream_t stream);

hipError_t launch_combine(const float* y_rows, const int32_t* slot_to_row, const float* topk_w, int T, int d,
                          int K, bool act_bf16, void* y, hipStream_t stream);

hipError_t launch_dense_init(int T, int32_t* offsets, int32_t* sorted_slots, int32_t* slot_to_row, float* w,
                             hipStream_t stream);

hipError_t launch_pack_rows(long rows, int cols, const int8_t* src, int8_t* dst, hipStream_t stream);

// int8 codes (fp8 = false) or OCP e4m3 code bytes (fp8 = true), row-major or
// in the tiled layout (tiled = true: rows % 16 == 0, cols % 64 == 0)
hipError_t launch_quantize_rows(int64_t rows, int cols, bool src_bf16, const void* w, bool scale_bf16, int8_t* q,
                                void* s, bool fp8, bool tiled, hipStream_t stream);

// MXFP4 (mx_common.h): quantizer, dequantizer and packer. tiled: rows % 16 ==
// 0, cols % 128 == 0; row-major: cols % 32 == 0.
hipError_t launch_mx_quantize(int64_t rows, int cols, bool src_bf16, const void* w, bool tiled, uint8_t* q, uint8_t* s,
                              hipStream_t stream);
hipError_t launch_mx_dequantize(int64_t rows, int cols, bool tiled, const uint8_t* q, const uint8_t* s, bool dst_bf16,
                                void* w, hipStream_t stream);
hipError_t launch_mx_pack(int64_t rows, int cols, const uint8_t* q, const uint8_t* s, uint8_t* q_tiled,
                          uint8_t* s_tiled, hipStream_t stream);

// Products with MXFP4 weights over rows grouped by expert.
struct MxArgs {
  const void* a;                // rows: bf16 [., Kd], or MXFP4 codes [., Kd/2]
  const uint8_t* a_s;           // their scales [., Kd/32], or null: a is bf16
  const int32_t* offsets;       // [E + 1]
  const int32_t* sorted_slots;  // [S]: sorted row r reads row sorted_slots[r] / topk of a; null: row r
  int topk;
  long a_rows;                  // rows of a
  const uint8_t *w0, *s0;       // [E, N, Kd] codes and scales, tiled
  const uint8_t *w1, *s1;       // second matrix: out = silu(w0 . a) * (w1 . a); null: out = w0 . a
  void* out;                    // [S, N]
  bool out_bf16;                // else fp32
  unsigned long long* claims;   // tile claim words of the tiled kernel ([8], cleared by the launch), or null
  int E, N, Kd, S;
};
// What the two launches below take for these sizes: channels of an item (of each
// matrix), rows a pass and slices of the reduction; rows and channels of a tile
// (with two matrices half the channels are of each) and whether the queues' last
// tiles are claimed.
struct MxStreamPlan {
  int channels, rows, slices;
};
struct MxTilePlan {
  int rows, channels;
  bool claims;
};
MxStreamPlan mx_stream_plan(const MxArgs& a);
MxTilePlan mx_tile_plan(const MxArgs& a);
hipError_t launch_mx_stream(const MxArgs& a, hipStream_t stream);
// Whether rows of `cols` numbers (MXFP4 codes, or bf16) lie within 32-bit byte
// offsets, as launch_mx_tiled needs the rows of a to.
bool mx_tiled_offsets_fit(long rows, int cols, bool mx);
hipError_t launch_mx_tiled(const MxArgs& a, hipStream_t stream);

// Norms around the layer (block_norm.hip).
struct NormArgs {
  bool act_bf16;               // x, residual, weights, gate, out, next
  const void* x;               // [T, d]: normalised (residual null), or the layer's output y
  const float* y_rows;         // the experts' rows, combined into y; null: y is x
  const int32_t* slot_to_row;  // [T, K]
  const float* topk_w;         // [T, K]
  const void* residual;        // [T, d]; null: out = rms(x) * weight
  const void* weight;          // [d]; null after the block: y as it is
  const void* gate;            // [ceil(T / gate_tokens), d] or null
  const void* next_weight;     // [d] or null: no next
  void* out;                   // [T, d]
  void* next;                  // [T, d]
  float residual_scale, block_scale, eps, next_eps;
  int T, d, K, gate_tokens;
};
hipError_t launch_block_norm(const NormArgs& a, hipStream_t stream);

}  // namespace moe
