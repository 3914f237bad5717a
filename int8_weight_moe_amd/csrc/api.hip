// C ABI of libmoe_int8: argument validation, workspace layout and the
// enqueueing of the kernels. Nothing here allocates device memory or
// synchronises, except the checks that MOE_DEBUG turns on.
#include <stdarg.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <atomic>
#include <mutex>
#include <string>
#include <vector>

#include "../../include/moe_int8.h"
#include "debug_checks.h"
#include "kernels.h"

namespace {

thread_local char g_err[512] = "";

moe_status fail(moe_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
moe_status fail(moe_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return st;
}

moe_status hip_fail(hipError_t e, const char* what) {
  return fail(MOE_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// ---- MOE_DEBUG: permutation checks on the host (debug runs only)

// Set and not "0" at the time of the call.
bool debug_on() {
  const char* v = getenv("MOE_DEBUG");
  return v && v[0] && strcmp(v, "0") != 0;
}

// n int32 values from the device, after the work already enqueued on `stream`.
moe_status fetch_ints(const int32_t* dev, long n, std::vector<int32_t>& out, hipStream_t stream) {
  out.assign((size_t)n, 0);
  if (n <= 0) return MOE_OK;
  hipError_t e = hipMemcpyAsync(out.data(), dev, (size_t)n * sizeof(int32_t), hipMemcpyDeviceToHost, stream);
  if (e == hipSuccess) e = hipStreamSynchronize(stream);
  return e == hipSuccess ? MOE_OK : hip_fail(e, "MOE_DEBUG copy to the host");
}

moe_status debug_verdict(const std::string& m, const char* what) {
  return m.empty() ? MOE_OK : fail(MOE_ERR_CHECK, "MOE_DEBUG %s: %s", what, m.c_str());
}

// A caller's segment offsets and, when `sorted` is given, the slots of the
// rows they cover.
moe_status debug_inputs(const moe_shape* s, const int32_t* offsets, const int32_t* sorted, hipStream_t stream) {
  const long S = (long)s->T * s->K;
  std::vector<int32_t> off, srt;
  moe_status st = fetch_ints(offsets, s->E + 1, off, stream);
  if (st != MOE_OK) return st;
  st = debug_verdict(moe_debug::check_offsets(off.data(), s->E, S), "expert_offsets");
  if (st != MOE_OK || !sorted) return st;
  if ((st = fetch_ints(sorted, off[s->E], srt, stream)) != MOE_OK) return st;
  return debug_verdict(moe_debug::check_sorted(srt.data(), off[s->E], S), "sorted_slots");
}

// A caller's slot_to_row.
moe_status debug_rows(const moe_shape* s, const int32_t* s2r, hipStream_t stream) {
  const long S = (long)s->T * s->K;
  std::vector<int32_t> rows;
  moe_status st = fetch_ints(s2r, S, rows, stream);
  if (st != MOE_OK) return st;
  return debug_verdict(moe_debug::check_rows(rows.data(), S), "slot_to_row");
}

// The permutation the library produced from the expert ids.
moe_status debug_permutation(const moe_shape* s, const int32_t* ids, const int32_t* offsets, const int32_t* sorted,
                             const int32_t* s2r, hipStream_t stream) {
  const long S = (long)s->T * s->K;
  std::vector<int32_t> i, off, srt, rows;
  moe_status st;
  if ((st = fetch_ints(ids, S, i, stream)) != MOE_OK) return st;
  if ((st = fetch_ints(offsets, s->E + 1, off, stream)) != MOE_OK) return st;
  if ((st = fetch_ints(sorted, S, srt, stream)) != MOE_OK) return st;
  if ((st = fetch_ints(s2r, S, rows, stream)) != MOE_OK) return st;
  return debug_verdict(moe_debug::check_permutation(i.data(), off.data(), srt.data(), rows.data(), s->E, S),
                       "permutation");
}

constexpr size_t kAlign = 256;
size_t round_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

// Rows at or below this many per expert (on average) go to the weight-streaming schedule.
constexpr long kStreamRowsPerExpert = 64;
// The same with MXFP4 weights: for the down pass (whose schedule the workspaces
// are sized for), and for the gate/up pass and products of MXFP4 by MXFP4.
// Measured (us, stream / tiled; d 4096, f 14336, 16 experts): gate/up at 6 rows an
// expert 160 / 173, at 8 163 / 174, at 10 177 / 175, at 16 196 / 176; both in MXFP4
// (SwiGLU) at 8 rows 157 / 168, at 16 178 / 174; down at 16 114 / 122, at 32 212 / 135.
constexpr long kMxStreamRowsPerExpert = 16;
constexpr long kMxWideStreamRowsPerExpert = 8;
// With few channels in all, tiles leave most of the GPU idle and the streaming
// kernel's split reductions do not: the borders are 32 and 20 rows then. Measured
// (rows an expert): down, f 4096, d 4096, E 4 at 12 rows 13.6 / 28.9, at 32 26.6 / 32.2; f 8192,
// d 2048, E 8 at 32 47.9 / 62.6; gate/up, d 4096, f 4096, E 4 at 20 27.7 / 30.7, at 32 48.6 /
// 33.9; d 8192, f 2048, E 8 at 20 51.3 / 57.5; both in MXFP4 there at 20 29.3 / 30.2, at 32 51.6 / 31.9.
// Measured at 16384 channels and not between there and 65536; the length of the reduction has no part in
// it, which leaves one expert of many rows short of workgroups (dense layer, d 8192, f 24576: 124 us at
// 32 tokens, 260 at 33, where int8 weights take 187 and 145).
constexpr long kMxFewTilesRowsPerExpert = 32;
constexpr long kMxFewTilesWideRowsPerExpert = 20;
constexpr long kMxFewTilesChannels = 16384;

// routes: the call's K experts of a token are distinct ones of the E.
moe_status check_shape(const moe_shape* s, bool routes = true) {
  if (!s) return fail(MOE_ERR_NULL, "shape is NULL");
  if (s->T < 0) return fail(MOE_ERR_SHAPE, "T=%d must be >= 0", s->T);
  if (s->d < 64 || s->d > 65536 || s->d % 64) return fail(MOE_ERR_SHAPE, "d=%d must be a multiple of 64 in [64, 65536]", s->d);
  if (s->f < 64 || s->f > 131072 || s->f % 64) return fail(MOE_ERR_SHAPE, "f=%d must be a multiple of 64 in [64, 131072]", s->f);
  if (s->E < 1 || s->E > 64) return fail(MOE_ERR_SHAPE, "E=%d must be in [1, 64]", s->E);
  if (s->K < 1 || s->K > 8 || (routes && s->K > s->E))
    return fail(MOE_ERR_SHAPE, routes ? "K=%d must be in [1, min(E, 8)]" : "K=%d must be in [1, 8]", s->K);
  if ((long)s->T * s->K > (1L << 26)) return fail(MOE_ERR_SHAPE, "T*K=%ld exceeds 2^26", (long)s->T * s->K);
  if (s->act_dtype != MOE_F32 && s->act_dtype != MOE_BF16) return fail(MOE_ERR_DTYPE, "act_dtype=%d", s->act_dtype);
  if (s->scale_dtype != MOE_F32 && s->scale_dtype != MOE_BF16) return fail(MOE_ERR_DTYPE, "scale_dtype=%d", s->scale_dtype);
  if (s->ffn_path < MOE_PATH_AUTO || s->ffn_path > MOE_PATH_TILED) return fail(MOE_ERR_SHAPE, "ffn_path=%d", s->ffn_path);
  if ((s->weight_fmt < MOE_W_INT8 || s->weight_fmt > MOE_W_FP8) && s->weight_fmt != MOE_W_MXFP4) return fail(MOE_ERR_DTYPE, "weight_fmt=%d", s->weight_fmt);
  return MOE_OK;
}

#define REQUIRE_PTR(p)                                                         \
  do {                                                                         \
    if (!(p)) return fail(MOE_ERR_NULL, "%s is NULL", #p);                     \
    if (!aligned16(p)) return fail(MOE_ERR_ALIGN, "%s is not 16-byte aligned", #p); \
  } while (0)

// Scales are read for the scaled weight encodings (int8, fp8) only.
#define REQUIRE_SCALE(s, p)                                                    \
  do {                                                                         \
    if ((s)->weight_fmt != MOE_W_BF16) REQUIRE_PTR(p);                         \
  } while (0)

struct WsLayout {
  size_t ids, w, offsets, sorted, s2r, h, y_rows, part, part_bytes, claims, total;
};

bool use_stream(const moe_shape* s);
size_t down_ws_bytes(const moe_shape* s);

WsLayout forward_layout(const moe_shape* s) {
  const size_t S = (size_t)s->T * s->K;
  WsLayout L;
  size_t o = 0;
  L.ids = o;     o += round_up(S * 4);
  L.w = o;       o += round_up(S * 4);
  L.offsets = o; o += round_up((s->E + 1) * 4);
  L.sorted = o;  o += round_up(S * 4);
  L.s2r = o;     o += round_up(S * 4);
  L.h = o;       o += round_up(S * (size_t)s->f * 2);
  L.y_rows = o;  o += round_up(S * (size_t)s->d * 4);
  // partial sums of a stream down pass split over workgroups (none otherwise)
  L.part_bytes = use_stream(s) ? down_ws_bytes(s) : 0;
  L.part = o;    o += round_up(L.part_bytes);
  // tile claim words of the tiled gate/up and down passes (none for the stream schedule)
  L.claims = o;  o += use_stream(s) ? 0 : 2 * moe::kTileClaimBytes;
  L.total = o;
  return L;
}

// Workspace of the down pass: the stream schedule's fp32 partial sums of a
// reduction split over workgroups ([planes, S, d]; 0 bytes if it does not
// split), or the tiled schedule's tile claim words.
size_t down_ws_bytes(const moe_shape* s) {
  if (!use_stream(s)) return moe::kTileClaimBytes;
  if (s->weight_fmt == MOE_W_MXFP4) return 0;   // its stream pass splits inside the workgroup only
  const long S = (long)s->T * s->K;
  const int planes = moe::stream_down_planes(S, s->d, s->f, s->E);
  return (size_t)planes * (size_t)S * (size_t)s->d * 4;
}

// Workspace of the gate/up pass: the tiled schedule's tile claim words.
size_t gate_up_ws_bytes(const moe_shape* s) { return use_stream(s) ? 0 : moe::kTileClaimBytes; }

// moe_expert_ffn: h, then the down pass's workspace, then the gate/up pass's
size_t ffn_h_bytes(const moe_shape* s) { return round_up((size_t)s->T * s->K * (size_t)s->f * 2); }
size_t ffn_ws_bytes(const moe_shape* s) {
  return ffn_h_bytes(s) + round_up(down_ws_bytes(s)) + round_up(gate_up_ws_bytes(s));
}

bool use_stream(const moe_shape* s) {
  if (s->ffn_path == MOE_PATH_STREAM) return true;
  if (s->ffn_path == MOE_PATH_TILED) return false;
  if (s->weight_fmt == MOE_W_MXFP4) return (long)s->T * s->K <= kMxStreamRowsPerExpert * s->E;
  return (long)s->T * s->K <= kStreamRowsPerExpert * s->E;
}

// The passes of the expert FFN that a call runs.
enum { kGateUpPass = 1, kDownPass = 2, kBothPasses = 3 };

// What the FFN kernels accept beyond check_shape: the bf16 and fp8 weight
// encodings run with bf16 activations, and their tiled schedule addresses
// with 32-bit offsets. MXFP4 weights: only the rows that a pass reads (x, h) are
// addressed so; AUTO streams a pass whose rows do not fit (run_mx).
moe_status check_ffn(const moe_shape* s, int passes) {
  if (s->weight_fmt == MOE_W_INT8) return MOE_OK;
  if (s->act_dtype != MOE_BF16)
    return fail(MOE_ERR_UNSUPPORTED, "weight_fmt=%d needs bf16 activations", s->weight_fmt);
  if (s->weight_fmt == MOE_W_MXFP4) {
    if (s->d % 128 || s->f % 128)
      return fail(MOE_ERR_SHAPE, "MXFP4 weights need d=%d and f=%d to be multiples of 128", s->d, s->f);
    if (s->ffn_path != MOE_PATH_TILED) return MOE_OK;
    if ((passes & kGateUpPass) && !moe::mx_tiled_offsets_fit(s->T, s->d, false))
      return fail(MOE_ERR_UNSUPPORTED, "x is too large for the tiled schedule");
    if ((passes & kDownPass) && !moe::mx_tiled_offsets_fit((long)s->T * s->K, s->f, false))
      return fail(MOE_ERR_UNSUPPORTED, "h is too large for the tiled schedule");
    return MOE_OK;
  }
  const int wbytes = s->weight_fmt == MOE_W_BF16 ? 2 : 1;
  if (!use_stream(s) && !moe::dma_offsets_fit(s->T, (long)s->T * s->K, s->d, s->f, wbytes))
    return fail(MOE_ERR_UNSUPPORTED, "weight_fmt=%d: tensors too large for the tiled schedule", s->weight_fmt);
  return MOE_OK;
}

moe::FfnArgs ffn_args(const moe_shape* s, const void* x, const int32_t* offsets, const int32_t* sorted_slots,
                      const void* w_gate, const void* w_up, const void* w_down, const void* s_gate,
                      const void* s_up, const void* s_down, float* y_rows, __bf16* h) {
  moe::FfnArgs a;
  a.x = x;
  a.act_bf16 = s->act_dtype == MOE_BF16;
  a.scale_bf16 = s->scale_dtype == MOE_BF16;
  a.offsets = offsets;
  a.sorted_slots = sorted_slots;
  a.wfmt = s->weight_fmt;
  a.w_gate = static_cast<const int8_t*>(w_gate);
  a.w_up = static_cast<const int8_t*>(w_up);
  a.w_down = static_cast<const int8_t*>(w_down);
  a.s_gate = s_gate;
  a.s_up = s_up;
  a.s_down = s_down;
  a.h = h;
  a.y_rows = y_rows;
  a.part = nullptr;
  a.y_dense = nullptr;
  a.ids = nullptr;
  a.perm_offsets = a.perm_sorted = a.perm_s2r = nullptr;
  a.claims_gate_up = a.claims_down = nullptr;
  a.T = s->T;
  a.d = s->d;
  a.f = s->f;
  a.E = s->E;
  a.K = s->K;
  a.S = s->T * s->K;
  return a;
}

// ---- MOE_LOG: one line per FFN pass on stderr, naming the schedule it takes

// Set and not "0" at the time of the call.
bool log_on() {
  const char* v = getenv("MOE_LOG");
  return v && v[0] && strcmp(v, "0") != 0;
}

void log_pass(const char* call, bool gate_up, const moe_shape* s, const moe::FfnArgs& a) {
  const long S = (long)s->T * s->K;
  char how[192];
  if (!use_stream(s)) {
    snprintf(how, sizeof(how), "tiled schedule, %s",
             (gate_up ? a.claims_gate_up : a.claims_down) ? "the last tiles of each XCD queue claimed"
                                                          : "static tile order");
  } else if (gate_up) {
    snprintf(how, sizeof(how), "stream schedule, %d-row passes, expert segments %s", S > 32L * s->E ? 64 : 32,
             a.ids ? "derived from the expert ids (permutation written by the pass)" : "read from the permutation");
  } else {
    const int planes = moe::stream_down_planes(S, s->d, s->f, s->E);
    if (a.part && planes > 0) {
      snprintf(how, sizeof(how), "stream schedule, reduction split over workgroups in %d slices%s", planes,
               a.y_dense ? ", their sum written to y (combine folded in)" : "");
    } else {
      snprintf(how, sizeof(how), "stream schedule, %d-row passes, reduction inside the workgroup",
               S > 32L * s->E ? 64 : 32);
    }
  }
  static const char* const kFmt[] = {"int8", "bf16", "fp8"};
  fprintf(stderr, "[moe] %s %s: T=%d d=%d f=%d E=%d K=%d act=%s scale=%s weights=%s; %s\n", call,
          gate_up ? "gate/up" : "down", s->T, s->d, s->f, s->E, s->K, s->act_dtype == MOE_BF16 ? "bf16" : "f32",
          s->scale_dtype == MOE_BF16 ? "bf16" : "f32", kFmt[s->weight_fmt], how);
}

// The passes of the expert FFN as products with MXFP4 weights.
moe::MxArgs mx_gate_up(const moe::FfnArgs& a) {
  moe::MxArgs m;
  m.a = a.x;
  m.a_s = nullptr;
  m.offsets = a.offsets;
  m.sorted_slots = a.sorted_slots;
  m.topk = a.K;
  m.a_rows = a.T;
  m.w0 = reinterpret_cast<const uint8_t*>(a.w_gate);
  m.s0 = static_cast<const uint8_t*>(a.s_gate);
  m.w1 = reinterpret_cast<const uint8_t*>(a.w_up);
  m.s1 = static_cast<const uint8_t*>(a.s_up);
  m.out = a.h;
  m.out_bf16 = true;
  m.claims = a.claims_gate_up;
  m.E = a.E;
  m.N = a.f;
  m.Kd = a.d;
  m.S = a.S;
  return m;
}

moe::MxArgs mx_down(const moe::FfnArgs& a) {
  moe::MxArgs m;
  m.a = a.h;
  m.a_s = nullptr;
  m.offsets = a.offsets;
  m.sorted_slots = nullptr;
  m.topk = 1;
  m.a_rows = a.S;
  m.w0 = reinterpret_cast<const uint8_t*>(a.w_down);
  m.s0 = static_cast<const uint8_t*>(a.s_down);
  m.w1 = m.s1 = nullptr;
  m.out = a.y_rows;
  m.out_bf16 = false;
  m.claims = a.claims_down;
  m.E = a.E;
  m.N = a.d;
  m.Kd = a.f;
  m.S = a.S;
  return m;
}

// One product with MXFP4 weights; `call` and `what` name it in the log and in an error.
moe_status run_mx(const char* call, const char* what, const moe_shape* s, const moe::MxArgs& m, hipStream_t stream) {
  bool by_stream = use_stream(s);
  if (s->ffn_path == MOE_PATH_AUTO) {
    const bool wide = m.a_s || m.w1, few = (long)m.E * m.N <= kMxFewTilesChannels;
    const long rows = few ? (wide ? kMxFewTilesWideRowsPerExpert : kMxFewTilesRowsPerExpert)
                          : (wide ? kMxWideStreamRowsPerExpert : kMxStreamRowsPerExpert);
    by_stream = m.S <= rows * m.E;
  }
  // rows past the tiled kernel's 32-bit offsets (on TILED, bf16 rows are refused by check_ffn)
  if (!moe::mx_tiled_offsets_fit(m.a_rows, m.Kd, m.a_s != nullptr)) by_stream = true;
  if (log_on()) {
    char how[128];
    if (by_stream) {
      const moe::MxStreamPlan p = moe::mx_stream_plan(m);
      snprintf(how, sizeof(how), "stream schedule, %d-channel items, %d-row passes, reduction in %d slices", p.channels,
               p.rows, p.slices);
    } else {
      const moe::MxTilePlan p = moe::mx_tile_plan(m);
      snprintf(how, sizeof(how), "tiled schedule, %dx%d tiles, %s", p.rows, p.channels,
               p.claims ? "the last tiles of each XCD queue claimed" : "static tile order");
    }
    fprintf(stderr, "[moe] %s %s: rows=%d reduction=%d channels=%d E=%d act=%s weights=mxfp4 out=%s%s; %s\n", call, what,
            m.S, m.Kd, m.N, m.E, m.a_s ? "mxfp4" : "bf16", m.out_bf16 ? "bf16" : "f32", m.w1 ? " SwiGLU" : "", how);
  }
  const hipError_t e = by_stream ? moe::launch_mx_stream(m, stream) : moe::launch_mx_tiled(m, stream);
  if (e != hipSuccess) return hip_fail(e, what);
  return MOE_OK;
}

moe_status run_gate_up(const char* call, const moe_shape* s, const moe::FfnArgs& a, hipStream_t stream) {
  if (s->weight_fmt == MOE_W_MXFP4) return run_mx(call, "gate/up", s, mx_gate_up(a), stream);
  if (log_on()) log_pass(call, true, s, a);
  const hipError_t e = use_stream(s) ? moe::launch_stream_gate_up(a, stream) : moe::launch_tiled_gate_up(a, stream);
  if (e != hipSuccess) return hip_fail(e, "gate/up launch");
  return MOE_OK;
}

moe_status run_down(const char* call, const moe_shape* s, const moe::FfnArgs& a, hipStream_t stream) {
  if (s->weight_fmt == MOE_W_MXFP4) return run_mx(call, "down", s, mx_down(a), stream);
  if (log_on()) log_pass(call, false, s, a);
  const hipError_t e = use_stream(s) ? moe::launch_stream_down(a, stream) : moe::launch_tiled_down(a, stream);
  if (e != hipSuccess) return hip_fail(e, "down launch");
  return MOE_OK;
}

// MXFP4 codes and scales: sizes of a layout, and the pointers.
moe_status check_mxfp4(int64_t rows, int32_t cols, int32_t layout, const void* q, const void* s) {
  if (layout != MOE_MX_ROWS && layout != MOE_MX_TILED) return fail(MOE_ERR_SHAPE, "layout=%d", layout);
  if (rows < 0 || rows > 0x7fffffffL) return fail(MOE_ERR_SHAPE, "rows=%ld must be in [0, 2^31)", (long)rows);
  if (cols < 32 || cols > (1 << 20) || cols % 32) return fail(MOE_ERR_SHAPE, "cols=%d must be a multiple of 32 in [32, 2^20]", cols);
  if (layout == MOE_MX_TILED && (rows % 16 || cols % 128))
    return fail(MOE_ERR_SHAPE, "the tiled layout needs rows=%ld to be a multiple of 16 and cols=%d of 128", (long)rows, cols);
  if (layout == MOE_MX_TILED && rows * (int64_t)cols / 128 >= (1L << 30)) return fail(MOE_ERR_SHAPE, "matrix too large");
  if (rows == 0) return MOE_OK;
  REQUIRE_PTR(q);
  REQUIRE_PTR(s);
  return MOE_OK;
}

// Shape of a product with both operands in MXFP4.
moe_status check_mx_shape(const moe_shape* s, bool routes) {
  const moe_status st = check_shape(s, routes);
  if (st != MOE_OK) return st;
  if (s->weight_fmt != MOE_W_MXFP4) return fail(MOE_ERR_DTYPE, "weight_fmt=%d: this call takes MXFP4 weights", s->weight_fmt);
  if (s->d % 128 || s->f % 128)
    return fail(MOE_ERR_SHAPE, "MXFP4 weights need d=%d and f=%d to be multiples of 128", s->d, s->f);
  return MOE_OK;
}

// moe_block_forward's workspace: moe_forward's, then the normalised input.
size_t block_x_bytes(const moe_shape* s) {
  return round_up((size_t)s->T * s->d * (s->act_dtype == MOE_BF16 ? 2 : 4));
}

// Workspace of moe_expert_ffn_mxfp4: x in MXFP4, h, h in MXFP4.
struct MxFfnLayout {
  size_t xq, xs, h, hq, hs, total;
};

MxFfnLayout mx_ffn_layout(const moe_shape* s) {
  const size_t T = (size_t)s->T, S = T * s->K, d = (size_t)s->d, f = (size_t)s->f;
  MxFfnLayout L;
  size_t o = 0;
  L.xq = o; o += round_up(T * (d / 2));
  L.xs = o; o += round_up(T * (d / 32));
  L.h = o;  o += round_up(S * f * 2);
  L.hq = o; o += round_up(S * (f / 2));
  L.hs = o; o += round_up(S * (f / 32));
  L.total = o;
  return L;
}

bool finite_f32(float v) { return v - v == 0.f; }

moe_status check_eps(const char* what, float eps) {
  if (!finite_f32(eps) || eps < 0.f) return fail(MOE_ERR_SHAPE, "%s=%g must be finite and not negative", what, (double)eps);
  return MOE_OK;
}

// Whether two [T, d] act_dtype arrays share memory without being the same one.
bool overlap(const moe_shape* s, const void* a, const void* b) {
  const uintptr_t u = reinterpret_cast<uintptr_t>(a), v = reinterpret_cast<uintptr_t>(b);
  const uintptr_t bytes = (uintptr_t)s->T * s->d * (s->act_dtype == MOE_BF16 ? 2 : 4);
  return a && b && u != v && (u < v ? v - u : u - v) < bytes;
}

moe_status check_post(const moe_shape* s, const moe_post* p, const void* residual, const void* out, const void* next) {
  if (!p) return fail(MOE_ERR_NULL, "post is NULL");
  moe_status st;
  if (p->weight && (st = check_eps("eps", p->eps)) != MOE_OK) return st;
  if (p->next_weight && (st = check_eps("next_eps", p->next_eps)) != MOE_OK) return st;
  if (p->gate && p->gate_tokens < 1) return fail(MOE_ERR_SHAPE, "gate_tokens=%d must be at least 1", p->gate_tokens);
  if (s->T == 0) return MOE_OK;
  if (!aligned16(p->weight)) return fail(MOE_ERR_ALIGN, "weight is not 16-byte aligned");
  if (!aligned16(p->gate)) return fail(MOE_ERR_ALIGN, "gate is not 16-byte aligned");
  if (!aligned16(p->next_weight)) return fail(MOE_ERR_ALIGN, "next_weight is not 16-byte aligned");
  REQUIRE_PTR(residual);
  REQUIRE_PTR(out);
  if (overlap(s, out, residual)) return fail(MOE_ERR_UNSUPPORTED, "out overlaps residual and is not residual");
  if (!p->next_weight) return MOE_OK;
  REQUIRE_PTR(next);
  if (next == out || overlap(s, next, out)) return fail(MOE_ERR_UNSUPPORTED, "next overlaps out");
  if (overlap(s, next, residual)) return fail(MOE_ERR_UNSUPPORTED, "next overlaps residual");
  return MOE_OK;
}

// What every token's workgroup reads (post's arrays, the experts' rows) may not
// lie where another's writes out and next.
moe_status check_post_reads(const moe_shape* s, const moe_post* p, const float* y_rows, const void* out,
                            const void* next) {
  const size_t elem = s->act_dtype == MOE_BF16 ? 2 : 4, row = s->d * elem, bytes = s->T * row;
  const size_t gate_rows = p->gate ? ((size_t)s->T + p->gate_tokens - 1) / p->gate_tokens : 0;
  const struct {
    const char* name;
    const void* ptr;
    size_t bytes;
  } reads[] = {{"weight", p->weight, row},
               {"gate", p->gate, gate_rows * row},
               {"next_weight", p->next_weight, row},
               {"y_rows", y_rows, (size_t)s->T * s->K * s->d * 4}};
  for (const auto& r : reads)
    for (const void* w : {out, p->next_weight ? next : nullptr}) {
      const uintptr_t u = reinterpret_cast<uintptr_t>(r.ptr), v = reinterpret_cast<uintptr_t>(w);
      if (r.ptr && w && u < v + bytes && v < u + r.bytes)
        return fail(MOE_ERR_UNSUPPORTED, "%s overlaps %s", w == out ? "out" : "next", r.name);
    }
  return MOE_OK;
}

moe::NormArgs post_args(const moe_shape* s, const moe_post* p, const void* residual, void* out, void* next) {
  moe::NormArgs a = {};
  a.act_bf16 = s->act_dtype == MOE_BF16;
  a.residual = residual;
  a.weight = p->weight;
  a.gate = p->gate;
  a.next_weight = p->next_weight;
  a.out = out;
  a.next = next;
  a.residual_scale = p->residual_scale;
  a.block_scale = p->block_scale;
  a.eps = p->eps;
  a.next_eps = p->next_eps;
  a.T = s->T;
  a.d = s->d;
  a.K = s->K;
  a.gate_tokens = p->gate ? p->gate_tokens : 1;
  return a;
}

moe_status check_quantize(int64_t rows, int32_t cols, int32_t src_dtype, const void* w, int32_t scale_dtype,
                          const void* q, const void* s) {
  if (rows < 0 || rows > 0x7fffffffL) return fail(MOE_ERR_SHAPE, "rows=%ld must be in [0, 2^31)", (long)rows);
  if (cols < 16 || cols > (1 << 20) || cols % 16) return fail(MOE_ERR_SHAPE, "cols=%d must be a multiple of 16 in [16, 2^20]", cols);
  if (src_dtype != MOE_F32 && src_dtype != MOE_BF16) return fail(MOE_ERR_DTYPE, "src_dtype=%d", src_dtype);
  if (scale_dtype != MOE_F32 && scale_dtype != MOE_BF16) return fail(MOE_ERR_DTYPE, "scale_dtype=%d", scale_dtype);
  REQUIRE_PTR(w);
  REQUIRE_PTR(q);
  if (!s) return fail(MOE_ERR_NULL, "s is NULL");
  if ((reinterpret_cast<uintptr_t>(s) & 3u) != 0) return fail(MOE_ERR_ALIGN, "s is not 4-byte aligned");
  return MOE_OK;
}

// ---------------------------------------------------------------- fixed scratch of moe_forward_noalloc
// The allocation-free entry point keeps its workspace in this file-scope
// device array. Each GPU the library runs on holds its own copy until the
// process ends. In host code the name stands for a host-side shadow, not a
// device address: the device address is looked up once per device with
// hipGetSymbolAddress (with that device current) and kept in g_scratch_ptr.
constexpr size_t kScratchBytes = size_t(32) << 20;   // 32 MiB: the decode-sized layers
static __device__ __align__(256) unsigned char scratch[kScratchBytes];

constexpr int kMaxDevices = 64;
std::atomic<void*> g_scratch_ptr[kMaxDevices];
std::mutex g_scratch_mu;

moe_status scratch_on_current_device(void** out) {
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return fail(MOE_ERR_UNSUPPORTED, "device %d beyond the library's %d", dev, kMaxDevices);
  void* p = g_scratch_ptr[dev].load(std::memory_order_acquire);
  if (!p) {
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    p = g_scratch_ptr[dev].load(std::memory_order_relaxed);
    if (!p) {
      e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
      if (e != hipSuccess) return hip_fail(e, "hipGetSymbolAddress(scratch)");
      if (!p) return fail(MOE_ERR_HIP, "hipGetSymbolAddress(scratch) returned NULL");
      g_scratch_ptr[dev].store(p, std::memory_order_release);
    }
  }
  *out = p;
  return MOE_OK;
}

// post: null, or the norm and residual sum that take the combine's place (y is then unused).
moe_status forward_impl(const char* call, const moe_shape* s, const void* x, const void* router_w,
                       const float* router_bias, const void* w_gate, const void* w_up, const void* w_down,
                       const void* s_gate, const void* s_up, const void* s_down, void* y, int32_t* topk_ids_out,
                       float* topk_w_out, void* workspace, size_t workspace_bytes, hipStream_t stream,
                       moe::NormArgs* post = nullptr) {
  moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  st = check_ffn(s, kBothPasses);
  if (st != MOE_OK) return st;
  if (s->T == 0) return MOE_OK;   // nothing is read or written
  REQUIRE_PTR(x);
  REQUIRE_PTR(router_w);
  REQUIRE_PTR(w_gate);
  REQUIRE_PTR(w_up);
  REQUIRE_PTR(w_down);
  REQUIRE_SCALE(s, s_gate);
  REQUIRE_SCALE(s, s_up);
  REQUIRE_SCALE(s, s_down);
  if (!post) REQUIRE_PTR(y);
  REQUIRE_PTR(workspace);
  if (router_bias && !aligned16(router_bias)) return fail(MOE_ERR_ALIGN, "router_bias is not 16-byte aligned");
  if (topk_ids_out && !aligned16(topk_ids_out)) return fail(MOE_ERR_ALIGN, "topk_ids_out is not 16-byte aligned");
  if (topk_w_out && !aligned16(topk_w_out)) return fail(MOE_ERR_ALIGN, "topk_w_out is not 16-byte aligned");
  const WsLayout L = forward_layout(s);
  if (workspace_bytes < L.total)
    return fail(MOE_ERR_WORKSPACE, "workspace_bytes=%zu < required %zu", workspace_bytes, L.total);

  char* ws = static_cast<char*>(workspace);
  int32_t* ids = topk_ids_out ? topk_ids_out : reinterpret_cast<int32_t*>(ws + L.ids);
  float* wts = topk_w_out ? topk_w_out : reinterpret_cast<float*>(ws + L.w);
  int32_t* offsets = reinterpret_cast<int32_t*>(ws + L.offsets);
  int32_t* sorted = reinterpret_cast<int32_t*>(ws + L.sorted);
  int32_t* s2r = reinterpret_cast<int32_t*>(ws + L.s2r);
  __bf16* h = reinterpret_cast<__bf16*>(ws + L.h);
  float* y_rows = reinterpret_cast<float*>(ws + L.y_rows);

  hipError_t e = moe::launch_router(x, router_w, router_bias, s->T, s->d, s->E, s->K, s->act_dtype == MOE_BF16,
                                    ids, wts, stream);
  if (e != hipSuccess) return hip_fail(e, "router launch");
  moe::FfnArgs a = ffn_args(s, x, offsets, sorted, w_gate, w_up, w_down, s_gate, s_up, s_down, y_rows, h);
  if (L.part_bytes) a.part = reinterpret_cast<float*>(ws + L.part);
  if (!use_stream(s)) {
    a.claims_gate_up = reinterpret_cast<unsigned long long*>(ws + L.claims);
    a.claims_down = reinterpret_cast<unsigned long long*>(ws + L.claims + moe::kTileClaimBytes);
  }
  if (use_stream(s) && s->weight_fmt != MOE_W_MXFP4 && moe::stream_gate_up_takes_ids((long)s->T * s->K, s->E)) {
    // at most 256 slots: the gate/up pass derives the permutation from the ids
    // and writes it for the down pass and the combine (one launch fewer)
    a.ids = ids;
    a.perm_offsets = offsets;
    a.perm_sorted = sorted;
    a.perm_s2r = s2r;
    st = run_gate_up(call, s, a, stream);
    a.ids = nullptr;
    if (st == MOE_OK && debug_on()) st = debug_permutation(s, ids, offsets, sorted, s2r, stream);
  } else {
    e = moe::launch_permute(ids, s->T * s->K, s->E, offsets, sorted, s2r, stream);
    if (e != hipSuccess) return hip_fail(e, "permute launch");
    if (debug_on()) {
      st = debug_permutation(s, ids, offsets, sorted, s2r, stream);
      if (st != MOE_OK) return st;
    }
    st = run_gate_up(call, s, a, stream);
  }
  if (st != MOE_OK) return st;
  st = run_down(call, s, a, stream);
  if (st != MOE_OK) return st;
  if (post) {
    post->y_rows = y_rows;
    post->slot_to_row = s2r;
    post->topk_w = wts;
    e = moe::launch_block_norm(*post, stream);
    if (e != hipSuccess) return hip_fail(e, "norm launch");
    return MOE_OK;
  }
  e = moe::launch_combine(y_rows, s2r, wts, s->T, s->d, s->K, s->act_dtype == MOE_BF16, y, stream);
  if (e != hipSuccess) return hip_fail(e, "combine launch");
  return MOE_OK;
}

}  // namespace

extern "C" {

int32_t moe_abi_version(void) { return MOE_ABI_VERSION; }

const char* moe_status_str(moe_status st) {
  switch (st) {
    case MOE_OK: return "ok";
    case MOE_ERR_NULL: return "null pointer";
    case MOE_ERR_SHAPE: return "unsupported shape";
    case MOE_ERR_DTYPE: return "unknown dtype";
    case MOE_ERR_ALIGN: return "misaligned pointer";
    case MOE_ERR_WORKSPACE: return "workspace too small";
    case MOE_ERR_UNSUPPORTED: return "unsupported request";
    case MOE_ERR_HIP: return "HIP runtime error";
    case MOE_ERR_CHECK: return "MOE_DEBUG check failed";
    default: return "unknown status";
  }
}

const char* moe_last_error(void) { return g_err; }

moe_status moe_workspace_size(const moe_shape* shape, size_t* bytes) {
  moe_status st = check_shape(shape);
  if (st != MOE_OK) return st;
  if (!bytes) return fail(MOE_ERR_NULL, "bytes is NULL");
  *bytes = forward_layout(shape).total;
  return MOE_OK;
}

moe_status moe_ffn_workspace_size(const moe_shape* shape, size_t* bytes) {
  moe_status st = check_shape(shape);
  if (st != MOE_OK) return st;
  if (!bytes) return fail(MOE_ERR_NULL, "bytes is NULL");
  *bytes = ffn_ws_bytes(shape);
  return MOE_OK;
}

moe_status moe_route(const moe_shape* s, const void* x, const void* router_w, const float* router_bias,
                     int32_t* topk_ids, float* topk_w, hipStream_t stream) {
  moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  if (s->T == 0) return MOE_OK;   // nothing is read or written
  REQUIRE_PTR(x);
  REQUIRE_PTR(router_w);
  REQUIRE_PTR(topk_ids);
  REQUIRE_PTR(topk_w);
  if (router_bias && !aligned16(router_bias)) return fail(MOE_ERR_ALIGN, "router_bias is not 16-byte aligned");
  const hipError_t e = moe::launch_router(x, router_w, router_bias, s->T, s->d, s->E, s->K,
                                          s->act_dtype == MOE_BF16, topk_ids, topk_w, stream);
  if (e != hipSuccess) return hip_fail(e, "router launch");
  return MOE_OK;
}

moe_status moe_permute(const moe_shape* s, const int32_t* topk_ids, int32_t* expert_offsets,
                       int32_t* sorted_slots, int32_t* slot_to_row, hipStream_t stream) {
  moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  if (s->T == 0) return MOE_OK;   // nothing is read or written
  REQUIRE_PTR(topk_ids);
  REQUIRE_PTR(expert_offsets);
  REQUIRE_PTR(sorted_slots);
  REQUIRE_PTR(slot_to_row);
  const hipError_t e = moe::launch_permute(topk_ids, s->T * s->K, s->E, expert_offsets, sorted_slots,
                                           slot_to_row, stream);
  if (e != hipSuccess) return hip_fail(e, "permute launch");
  if (debug_on()) return debug_permutation(s, topk_ids, expert_offsets, sorted_slots, slot_to_row, stream);
  return MOE_OK;
}

moe_status moe_expert_ffn(const moe_shape* s, const void* x, const int32_t* expert_offsets,
                          const int32_t* sorted_slots, const void* w_gate, const void* w_up,
                          const void* w_down, const void* s_gate, const void* s_up, const void* s_down,
                          float* y_rows, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  st = check_ffn(s, kBothPasses);
  if (st != MOE_OK) return st;
  if (s->T == 0) return MOE_OK;   // nothing is read or written
  REQUIRE_PTR(x);
  REQUIRE_PTR(expert_offsets);
  REQUIRE_PTR(sorted_slots);
  REQUIRE_PTR(w_gate);
  REQUIRE_PTR(w_up);
  REQUIRE_PTR(w_down);
  REQUIRE_SCALE(s, s_gate);
  REQUIRE_SCALE(s, s_up);
  REQUIRE_SCALE(s, s_down);
  REQUIRE_PTR(y_rows);
  REQUIRE_PTR(workspace);
  const size_t need = ffn_ws_bytes(s);
  if (workspace_bytes < need)
    return fail(MOE_ERR_WORKSPACE, "workspace_bytes=%zu < required %zu", workspace_bytes, need);
  if (debug_on() && (st = debug_inputs(s, expert_offsets, sorted_slots, stream)) != MOE_OK) return st;
  moe::FfnArgs a = ffn_args(s, x, expert_offsets, sorted_slots, w_gate, w_up, w_down, s_gate, s_up, s_down, y_rows,
                            static_cast<__bf16*>(workspace));
  char* dws = static_cast<char*>(workspace) + ffn_h_bytes(s);
  if (use_stream(s)) {
    if (down_ws_bytes(s)) a.part = reinterpret_cast<float*>(dws);
  } else {
    a.claims_down = reinterpret_cast<unsigned long long*>(dws);
    a.claims_gate_up = reinterpret_cast<unsigned long long*>(dws + round_up(down_ws_bytes(s)));
  }
  st = run_gate_up("moe_expert_ffn", s, a, stream);
  if (st != MOE_OK) return st;
  return run_down("moe_expert_ffn", s, a, stream);
}

moe_status moe_expert_gate_up(const moe_shape* s, const void* x, const int32_t* expert_offsets,
                              const int32_t* sorted_slots, const void* w_gate, const void* w_up,
                              const void* s_gate, const void* s_up, void* h, void* workspace,
                              size_t workspace_bytes, hipStream_t stream) {
  moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  st = check_ffn(s, kGateUpPass);
  if (st != MOE_OK) return st;
  if (s->T == 0) return MOE_OK;   // nothing is read or written
  REQUIRE_PTR(x);
  REQUIRE_PTR(expert_offsets);
  REQUIRE_PTR(sorted_slots);
  REQUIRE_PTR(w_gate);
  REQUIRE_PTR(w_up);
  REQUIRE_SCALE(s, s_gate);
  REQUIRE_SCALE(s, s_up);
  REQUIRE_PTR(h);
  const size_t need = gate_up_ws_bytes(s);
  if (workspace) {
    if (!aligned16(workspace)) return fail(MOE_ERR_ALIGN, "workspace is not 16-byte aligned");
    if (workspace_bytes < need)
      return fail(MOE_ERR_WORKSPACE, "workspace_bytes=%zu < required %zu", workspace_bytes, need);
  }
  if (debug_on() && (st = debug_inputs(s, expert_offsets, sorted_slots, stream)) != MOE_OK) return st;
  moe::FfnArgs a = ffn_args(s, x, expert_offsets, sorted_slots, w_gate, w_up, nullptr, s_gate, s_up, nullptr,
                            nullptr, static_cast<__bf16*>(h));
  if (workspace && need) a.claims_gate_up = static_cast<unsigned long long*>(workspace);
  return run_gate_up("moe_expert_gate_up", s, a, stream);
}

moe_status moe_expert_down(const moe_shape* s, const void* h, const int32_t* expert_offsets, const void* w_down,
                           const void* s_down, float* y_rows, void* workspace, size_t workspace_bytes,
                           hipStream_t stream) {
  moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  st = check_ffn(s, kDownPass);
  if (st != MOE_OK) return st;
  if (s->T == 0) return MOE_OK;   // nothing is read or written
  REQUIRE_PTR(h);
  REQUIRE_PTR(expert_offsets);
  REQUIRE_PTR(w_down);
  REQUIRE_SCALE(s, s_down);
  REQUIRE_PTR(y_rows);
  const size_t need = down_ws_bytes(s);
  if (workspace) {
    if (!aligned16(workspace)) return fail(MOE_ERR_ALIGN, "workspace is not 16-byte aligned");
    if (workspace_bytes < need)
      return fail(MOE_ERR_WORKSPACE, "workspace_bytes=%zu < required %zu", workspace_bytes, need);
  }
  if (debug_on() && (st = debug_inputs(s, expert_offsets, nullptr, stream)) != MOE_OK) return st;
  moe::FfnArgs a = ffn_args(s, nullptr, expert_offsets, nullptr, nullptr, nullptr, w_down, nullptr, nullptr, s_down,
                            y_rows, static_cast<__bf16*>(const_cast<void*>(h)));
  if (workspace && need) {
    if (use_stream(s)) {
      a.part = static_cast<float*>(workspace);
    } else {
      a.claims_down = static_cast<unsigned long long*>(workspace);
    }
  }
  return run_down("moe_expert_down", s, a, stream);
}

moe_status moe_down_workspace_size(const moe_shape* shape, size_t* bytes) {
  moe_status st = check_shape(shape);
  if (st != MOE_OK) return st;
  if (!bytes) return fail(MOE_ERR_NULL, "bytes is NULL");
  *bytes = down_ws_bytes(shape);
  return MOE_OK;
}

moe_status moe_gate_up_workspace_size(const moe_shape* shape, size_t* bytes) {
  moe_status st = check_shape(shape);
  if (st != MOE_OK) return st;
  if (!bytes) return fail(MOE_ERR_NULL, "bytes is NULL");
  *bytes = gate_up_ws_bytes(shape);
  return MOE_OK;
}

moe_status moe_combine(const moe_shape* s, const float* y_rows, const int32_t* slot_to_row,
                       const float* topk_w, void* y, hipStream_t stream) {
  moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  if (s->T == 0) return MOE_OK;   // nothing is read or written
  REQUIRE_PTR(y_rows);
  REQUIRE_PTR(slot_to_row);
  REQUIRE_PTR(topk_w);
  REQUIRE_PTR(y);
  if (debug_on() && (st = debug_rows(s, slot_to_row, stream)) != MOE_OK) return st;
  const hipError_t e = moe::launch_combine(y_rows, slot_to_row, topk_w, s->T, s->d, s->K,
                                           s->act_dtype == MOE_BF16, y, stream);
  if (e != hipSuccess) return hip_fail(e, "combine launch");
  return MOE_OK;
}

moe_status moe_forward(const moe_shape* s, const void* x, const void* router_w, const float* router_bias,
                       const void* w_gate, const void* w_up, const void* w_down, const void* s_gate,
                       const void* s_up, const void* s_down, void* y, int32_t* topk_ids_out, float* topk_w_out,
                       void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return forward_impl("moe_forward", s, x, router_w, router_bias, w_gate, w_up, w_down, s_gate, s_up, s_down, y,
                      topk_ids_out, topk_w_out, workspace, workspace_bytes, stream);
}

moe_status moe_forward_noalloc(const moe_shape* s, const void* x, const void* router_w, const float* router_bias,
                               const void* w_gate, const void* w_up, const void* w_down, const void* s_gate,
                               const void* s_up, const void* s_down, void* y, int32_t* topk_ids_out,
                               float* topk_w_out, hipStream_t stream) {
  moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  const size_t need = forward_layout(s).total;
  if (need > kScratchBytes)
    return fail(MOE_ERR_WORKSPACE, "moe_forward_noalloc: this shape needs %zu bytes of scratch, more than the "
                "library's fixed %zu (use moe_forward with a caller workspace)", need, kScratchBytes);
  if (s->T == 0) return MOE_OK;
  void* ws = nullptr;
  st = scratch_on_current_device(&ws);
  if (st != MOE_OK) return st;
  return forward_impl("moe_forward_noalloc", s, x, router_w, router_bias, w_gate, w_up, w_down, s_gate, s_up,
                      s_down, y, topk_ids_out, topk_w_out, ws, kScratchBytes, stream);
}

moe_status moe_mlp_workspace_size(const moe_shape* shape, size_t* bytes) {
  moe_status st = check_shape(shape);
  if (st != MOE_OK) return st;
  if (!bytes) return fail(MOE_ERR_NULL, "bytes is NULL");
  if (shape->E != 1 || shape->K != 1) return fail(MOE_ERR_SHAPE, "the dense MLP needs E = K = 1");
  *bytes = forward_layout(shape).total;
  return MOE_OK;
}

moe_status moe_mlp_forward(const moe_shape* s, const void* x, const void* w_gate, const void* w_up,
                           const void* w_down, const void* s_gate, const void* s_up, const void* s_down, void* y,
                           void* workspace, size_t workspace_bytes, hipStream_t stream) {
  moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  st = check_ffn(s, kBothPasses);
  if (st != MOE_OK) return st;
  if (s->E != 1 || s->K != 1) return fail(MOE_ERR_SHAPE, "the dense MLP needs E = K = 1 (E=%d, K=%d)", s->E, s->K);
  if (s->T == 0) return MOE_OK;   // nothing is read or written
  REQUIRE_PTR(x);
  REQUIRE_PTR(w_gate);
  REQUIRE_PTR(w_up);
  REQUIRE_PTR(w_down);
  REQUIRE_SCALE(s, s_gate);
  REQUIRE_SCALE(s, s_up);
  REQUIRE_SCALE(s, s_down);
  REQUIRE_PTR(y);
  REQUIRE_PTR(workspace);
  const WsLayout L = forward_layout(s);
  if (workspace_bytes < L.total)
    return fail(MOE_ERR_WORKSPACE, "workspace_bytes=%zu < required %zu", workspace_bytes, L.total);
  char* ws = static_cast<char*>(workspace);
  float* wts = reinterpret_cast<float*>(ws + L.w);
  int32_t* offsets = reinterpret_cast<int32_t*>(ws + L.offsets);
  int32_t* sorted = reinterpret_cast<int32_t*>(ws + L.sorted);
  int32_t* s2r = reinterpret_cast<int32_t*>(ws + L.s2r);
  __bf16* h = reinterpret_cast<__bf16*>(ws + L.h);
  float* y_rows = reinterpret_cast<float*>(ws + L.y_rows);
  hipError_t e = moe::launch_dense_init(s->T, offsets, sorted, s2r, wts, stream);
  if (e != hipSuccess) return hip_fail(e, "dense init launch");
  moe::FfnArgs a = ffn_args(s, x, offsets, sorted, w_gate, w_up, w_down, s_gate, s_up, s_down, y_rows, h);
  if (L.part_bytes) a.part = reinterpret_cast<float*>(ws + L.part);
  if (!use_stream(s)) {
    a.claims_gate_up = reinterpret_cast<unsigned long long*>(ws + L.claims);
    a.claims_down = reinterpret_cast<unsigned long long*>(ws + L.claims + moe::kTileClaimBytes);
  }
  // with the down pass's reduction split over workgroups, the sum of its slices
  // is written to y directly (the combine of one expert of weight 1)
  if (L.part_bytes) a.y_dense = y;
  st = run_gate_up("moe_mlp_forward", s, a, stream);
  if (st != MOE_OK) return st;
  st = run_down("moe_mlp_forward", s, a, stream);
  if (st != MOE_OK || a.y_dense) return st;
  e = moe::launch_combine(y_rows, s2r, wts, s->T, s->d, 1, s->act_dtype == MOE_BF16, y, stream);
  if (e != hipSuccess) return hip_fail(e, "combine launch");
  return MOE_OK;
}

moe_status moe_quantize_rows(int64_t rows, int32_t cols, int32_t src_dtype, const void* w, int32_t scale_dtype,
                             int8_t* q, void* s, hipStream_t stream) {
  const moe_status st = check_quantize(rows, cols, src_dtype, w, scale_dtype, q, s);
  if (st != MOE_OK) return st;
  if (rows == 0) return MOE_OK;
  const hipError_t e = moe::launch_quantize_rows(rows, cols, src_dtype == MOE_BF16, w, scale_dtype == MOE_BF16, q,
                                                 s, false, false, stream);
  if (e != hipSuccess) return hip_fail(e, "quantize launch");
  return MOE_OK;
}

moe_status moe_quantize_rows_fp8(int64_t rows, int32_t cols, int32_t src_dtype, const void* w, int32_t scale_dtype,
                                 uint8_t* q, void* s, hipStream_t stream) {
  const moe_status st = check_quantize(rows, cols, src_dtype, w, scale_dtype, q, s);
  if (st != MOE_OK) return st;
  if (rows == 0) return MOE_OK;
  const hipError_t e = moe::launch_quantize_rows(rows, cols, src_dtype == MOE_BF16, w, scale_dtype == MOE_BF16,
                                                 reinterpret_cast<int8_t*>(q), s, true, false, stream);
  if (e != hipSuccess) return hip_fail(e, "quantize launch");
  return MOE_OK;
}

moe_status moe_quantize_pack_rows(int64_t rows, int32_t cols, int32_t src_dtype, const void* w,
                                  int32_t scale_dtype, int32_t weight_fmt, void* q_tiled, void* s,
                                  hipStream_t stream) {
  moe_status st = check_quantize(rows, cols, src_dtype, w, scale_dtype, q_tiled, s);
  if (st != MOE_OK) return st;
  if (rows % 16 || cols % 64) return fail(MOE_ERR_SHAPE, "rows=%ld must be a multiple of 16 and cols=%d of 64", (long)rows, cols);
  if (weight_fmt != MOE_W_INT8 && weight_fmt != MOE_W_FP8)
    return fail(MOE_ERR_DTYPE, "weight_fmt=%d: only the int8 and fp8 encodings are quantized", weight_fmt);
  if (rows == 0) return MOE_OK;
  const hipError_t e = moe::launch_quantize_rows(rows, cols, src_dtype == MOE_BF16, w, scale_dtype == MOE_BF16,
                                                 static_cast<int8_t*>(q_tiled), s, weight_fmt == MOE_W_FP8, true,
                                                 stream);
  if (e != hipSuccess) return hip_fail(e, "quantize launch");
  return MOE_OK;
}

moe_status moe_pack_rows(int64_t rows, int32_t cols, const int8_t* q, int8_t* packed, hipStream_t stream) {
  if (rows < 0 || rows % 16) return fail(MOE_ERR_SHAPE, "rows=%ld must be a non-negative multiple of 16", (long)rows);
  if (cols < 64 || cols > (1 << 20) || cols % 64) return fail(MOE_ERR_SHAPE, "cols=%d must be a multiple of 64 in [64, 2^20]", cols);
  if (rows * (int64_t)cols / 16 > 0x7fffffffL * 256L) return fail(MOE_ERR_SHAPE, "matrix too large");
  REQUIRE_PTR(q);
  REQUIRE_PTR(packed);
  if (q == packed) return fail(MOE_ERR_UNSUPPORTED, "packing cannot be done in place");
  if (rows == 0) return MOE_OK;
  const hipError_t e = moe::launch_pack_rows(rows, cols, q, packed, stream);
  if (e != hipSuccess) return hip_fail(e, "pack launch");
  return MOE_OK;
}

moe_status moe_quantize_mxfp4(int64_t rows, int32_t cols, int32_t src_dtype, const void* w, int32_t layout, uint8_t* q,
                              uint8_t* s, hipStream_t stream) {
  const moe_status st = check_mxfp4(rows, cols, layout, q, s);
  if (st != MOE_OK) return st;
  if (src_dtype != MOE_F32 && src_dtype != MOE_BF16) return fail(MOE_ERR_DTYPE, "src_dtype=%d", src_dtype);
  if (rows == 0) return MOE_OK;
  REQUIRE_PTR(w);
  const hipError_t e = moe::launch_mx_quantize(rows, cols, src_dtype == MOE_BF16, w, layout == MOE_MX_TILED, q, s, stream);
  if (e != hipSuccess) return hip_fail(e, "quantize launch");
  return MOE_OK;
}

moe_status moe_dequantize_mxfp4(int64_t rows, int32_t cols, int32_t layout, const uint8_t* q, const uint8_t* s,
                                int32_t dst_dtype, void* w, hipStream_t stream) {
  const moe_status st = check_mxfp4(rows, cols, layout, q, s);
  if (st != MOE_OK) return st;
  if (dst_dtype != MOE_F32 && dst_dtype != MOE_BF16) return fail(MOE_ERR_DTYPE, "dst_dtype=%d", dst_dtype);
  if (rows == 0) return MOE_OK;
  REQUIRE_PTR(w);
  const hipError_t e = moe::launch_mx_dequantize(rows, cols, layout == MOE_MX_TILED, q, s, dst_dtype == MOE_BF16, w, stream);
  if (e != hipSuccess) return hip_fail(e, "dequantize launch");
  return MOE_OK;
}

moe_status moe_pack_mxfp4(int64_t rows, int32_t cols, const uint8_t* q, const uint8_t* s, uint8_t* q_tiled,
                          uint8_t* s_tiled, hipStream_t stream) {
  moe_status st = check_mxfp4(rows, cols, MOE_MX_TILED, q, s);
  if (st != MOE_OK) return st;
  if (rows == 0) return MOE_OK;
  REQUIRE_PTR(q_tiled);
  REQUIRE_PTR(s_tiled);
  if (q == q_tiled || s == s_tiled) return fail(MOE_ERR_UNSUPPORTED, "packing cannot be done in place");
  const hipError_t e = moe::launch_mx_pack(rows, cols, q, s, q_tiled, s_tiled, stream);
  if (e != hipSuccess) return hip_fail(e, "pack launch");
  return MOE_OK;
}

moe_status moe_grouped_mm_mxfp4(const moe_shape* s, const uint8_t* a_q, const uint8_t* a_s,
                                const int32_t* expert_offsets, const int32_t* sorted_slots, const uint8_t* w_q,
                                const uint8_t* w_s, const uint8_t* w2_q, const uint8_t* w2_s, void* out,
                                hipStream_t stream) {
  moe_status st = check_mx_shape(s, false);
  if (st != MOE_OK) return st;
  if (s->T == 0) return MOE_OK;   // nothing is read or written
  REQUIRE_PTR(a_q);
  REQUIRE_PTR(a_s);
  REQUIRE_PTR(expert_offsets);
  if (!aligned16(sorted_slots)) return fail(MOE_ERR_ALIGN, "sorted_slots is not 16-byte aligned");
  REQUIRE_PTR(w_q);
  REQUIRE_PTR(w_s);
  if (w2_q || w2_s) {
    REQUIRE_PTR(w2_q);
    REQUIRE_PTR(w2_s);
  }
  REQUIRE_PTR(out);
  if (debug_on() && (st = debug_inputs(s, expert_offsets, sorted_slots, stream)) != MOE_OK) return st;
  moe::MxArgs m;
  m.a = a_q;
  m.a_s = a_s;
  m.offsets = expert_offsets;
  m.sorted_slots = sorted_slots;
  m.topk = s->K;
  m.a_rows = sorted_slots ? s->T : (long)s->T * s->K;
  m.w0 = w_q;
  m.s0 = w_s;
  m.w1 = w2_q;
  m.s1 = w2_s;
  m.out = out;
  m.out_bf16 = s->act_dtype == MOE_BF16;
  m.claims = nullptr;
  m.E = s->E;
  m.N = s->f;
  m.Kd = s->d;
  m.S = s->T * s->K;
  return run_mx("moe_grouped_mm_mxfp4", "product", s, m, stream);
}

moe_status moe_expert_ffn_mxfp4_workspace_size(const moe_shape* shape, size_t* bytes) {
  const moe_status st = check_mx_shape(shape, true);
  if (st != MOE_OK) return st;
  if (!bytes) return fail(MOE_ERR_NULL, "bytes is NULL");
  *bytes = mx_ffn_layout(shape).total;
  return MOE_OK;
}

moe_status moe_expert_ffn_mxfp4(const moe_shape* s, const void* x, const int32_t* expert_offsets,
                                const int32_t* sorted_slots, const uint8_t* w_gate, const uint8_t* w_up,
                                const uint8_t* w_down, const uint8_t* s_gate, const uint8_t* s_up,
                                const uint8_t* s_down, float* y_rows, void* workspace, size_t workspace_bytes,
                                hipStream_t stream) {
  moe_status st = check_mx_shape(s, true);
  if (st != MOE_OK) return st;
  if (s->T == 0) return MOE_OK;   // nothing is read or written
  REQUIRE_PTR(x);
  REQUIRE_PTR(expert_offsets);
  REQUIRE_PTR(sorted_slots);
  REQUIRE_PTR(w_gate);
  REQUIRE_PTR(w_up);
  REQUIRE_PTR(w_down);
  REQUIRE_PTR(s_gate);
  REQUIRE_PTR(s_up);
  REQUIRE_PTR(s_down);
  REQUIRE_PTR(y_rows);
  REQUIRE_PTR(workspace);
  const MxFfnLayout L = mx_ffn_layout(s);
  if (workspace_bytes < L.total)
    return fail(MOE_ERR_WORKSPACE, "workspace_bytes=%zu < required %zu", workspace_bytes, L.total);
  if (debug_on() && (st = debug_inputs(s, expert_offsets, sorted_slots, stream)) != MOE_OK) return st;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const long S = (long)s->T * s->K;
  moe::MxArgs m;
  m.offsets = expert_offsets;
  m.claims = nullptr;
  m.E = s->E;
  m.S = (int)S;

  hipError_t e = moe::launch_mx_quantize(s->T, s->d, s->act_dtype == MOE_BF16, x, false, ws + L.xq, ws + L.xs, stream);
  if (e != hipSuccess) return hip_fail(e, "quantize launch");
  m.a = ws + L.xq;
  m.a_s = ws + L.xs;
  m.sorted_slots = sorted_slots;
  m.topk = s->K;
  m.a_rows = s->T;
  m.w0 = w_gate;
  m.s0 = s_gate;
  m.w1 = w_up;
  m.s1 = s_up;
  m.out = ws + L.h;
  m.out_bf16 = true;
  m.N = s->f;
  m.Kd = s->d;
  st = run_mx("moe_expert_ffn_mxfp4", "gate/up", s, m, stream);
  if (st != MOE_OK) return st;

  // rows past off[E] hold whatever the workspace held: their codes are never read
  e = moe::launch_mx_quantize(S, s->f, true, ws + L.h, false, ws + L.hq, ws + L.hs, stream);
  if (e != hipSuccess) return hip_fail(e, "quantize launch");
  m.a = ws + L.hq;
  m.a_s = ws + L.hs;
  m.sorted_slots = nullptr;
  m.topk = 1;
  m.a_rows = S;
  m.w0 = w_down;
  m.s0 = s_down;
  m.w1 = m.s1 = nullptr;
  m.out = y_rows;
  m.out_bf16 = false;
  m.N = s->d;
  m.Kd = s->f;
  return run_mx("moe_expert_ffn_mxfp4", "down", s, m, stream);
}

moe_status moe_norm_pre(const moe_shape* s, const void* x, const void* weight, float eps, void* n, hipStream_t stream) {
  moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  if ((st = check_eps("eps", eps)) != MOE_OK) return st;
  if (s->T == 0) return MOE_OK;   // nothing is read or written
  REQUIRE_PTR(x);
  REQUIRE_PTR(weight);
  REQUIRE_PTR(n);
  if (overlap(s, n, x)) return fail(MOE_ERR_UNSUPPORTED, "n overlaps x and is not x");
  moe::NormArgs a = {};
  a.act_bf16 = s->act_dtype == MOE_BF16;
  a.x = x;
  a.weight = weight;
  a.out = n;
  a.eps = eps;
  a.T = s->T;
  a.d = s->d;
  const hipError_t e = moe::launch_block_norm(a, stream);
  if (e != hipSuccess) return hip_fail(e, "norm launch");
  return MOE_OK;
}

moe_status moe_norm_post(const moe_shape* s, const moe_post* post, const void* y, const void* residual, void* out,
                         void* next, hipStream_t stream) {
  moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  if ((st = check_post(s, post, residual, out, next)) != MOE_OK) return st;
  if (s->T == 0) return MOE_OK;   // nothing is read or written
  REQUIRE_PTR(y);
  if (overlap(s, out, y)) return fail(MOE_ERR_UNSUPPORTED, "out overlaps y and is not y");
  if (post->next_weight && overlap(s, next, y)) return fail(MOE_ERR_UNSUPPORTED, "next overlaps y");
  if ((st = check_post_reads(s, post, nullptr, out, next)) != MOE_OK) return st;
  moe::NormArgs a = post_args(s, post, residual, out, next);
  a.x = y;
  const hipError_t e = moe::launch_block_norm(a, stream);
  if (e != hipSuccess) return hip_fail(e, "norm launch");
  return MOE_OK;
}

moe_status moe_combine_post(const moe_shape* s, const moe_post* post, const float* y_rows, const int32_t* slot_to_row,
                            const float* topk_w, const void* residual, void* out, void* next, hipStream_t stream) {
  moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  if ((st = check_post(s, post, residual, out, next)) != MOE_OK) return st;
  if (s->T == 0) return MOE_OK;   // nothing is read or written
  REQUIRE_PTR(y_rows);
  REQUIRE_PTR(slot_to_row);
  REQUIRE_PTR(topk_w);
  if ((st = check_post_reads(s, post, y_rows, out, next)) != MOE_OK) return st;
  if (debug_on() && (st = debug_rows(s, slot_to_row, stream)) != MOE_OK) return st;
  moe::NormArgs a = post_args(s, post, residual, out, next);
  a.y_rows = y_rows;
  a.slot_to_row = slot_to_row;
  a.topk_w = topk_w;
  const hipError_t e = moe::launch_block_norm(a, stream);
  if (e != hipSuccess) return hip_fail(e, "norm launch");
  return MOE_OK;
}

moe_status moe_block_workspace_size(const moe_shape* shape, size_t* bytes) {
  const moe_status st = check_shape(shape);
  if (st != MOE_OK) return st;
  if (!bytes) return fail(MOE_ERR_NULL, "bytes is NULL");
  *bytes = round_up(forward_layout(shape).total) + block_x_bytes(shape);
  return MOE_OK;
}

moe_status moe_block_forward(const moe_shape* s, const void* residual, const void* pre_weight, float pre_eps,
                             const void* x, const moe_post* post, const void* router_w, const float* router_bias,
                             const void* w_gate, const void* w_up, const void* w_down, const void* s_gate,
                             const void* s_up, const void* s_down, void* out, void* next, int32_t* topk_ids_out,
                             float* topk_w_out, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  if ((st = check_ffn(s, kBothPasses)) != MOE_OK) return st;
  if ((st = check_post(s, post, residual, out, next)) != MOE_OK) return st;
  if (pre_weight && (st = check_eps("pre_eps", pre_eps)) != MOE_OK) return st;
  if (s->T == 0) return MOE_OK;   // nothing is read or written
  if (!x == !pre_weight)
    return fail(x ? MOE_ERR_UNSUPPORTED : MOE_ERR_NULL, "exactly one of x and pre_weight is given");
  if (!aligned16(pre_weight)) return fail(MOE_ERR_ALIGN, "pre_weight is not 16-byte aligned");
  REQUIRE_PTR(workspace);
  const size_t fwd = round_up(forward_layout(s).total), need = fwd + block_x_bytes(s);
  if (workspace_bytes < need)
    return fail(MOE_ERR_WORKSPACE, "workspace_bytes=%zu < required %zu", workspace_bytes, need);
  // everything forward_impl checks, before the first launch
  REQUIRE_PTR(router_w);
  REQUIRE_PTR(w_gate);
  REQUIRE_PTR(w_up);
  REQUIRE_PTR(w_down);
  REQUIRE_SCALE(s, s_gate);
  REQUIRE_SCALE(s, s_up);
  REQUIRE_SCALE(s, s_down);
  if (!aligned16(router_bias)) return fail(MOE_ERR_ALIGN, "router_bias is not 16-byte aligned");
  if (!aligned16(topk_ids_out)) return fail(MOE_ERR_ALIGN, "topk_ids_out is not 16-byte aligned");
  if (!aligned16(topk_w_out)) return fail(MOE_ERR_ALIGN, "topk_w_out is not 16-byte aligned");
  if (!aligned16(x)) return fail(MOE_ERR_ALIGN, "x is not 16-byte aligned");
  if ((st = check_post_reads(s, post, nullptr, out, next)) != MOE_OK) return st;
  moe::NormArgs pa = post_args(s, post, residual, out, next);
  if (pre_weight) {
    moe::NormArgs a = {};
    a.act_bf16 = s->act_dtype == MOE_BF16;
    a.x = residual;
    a.weight = pre_weight;
    a.out = static_cast<char*>(workspace) + fwd;
    a.eps = pre_eps;
    a.T = s->T;
    a.d = s->d;
    const hipError_t e = moe::launch_block_norm(a, stream);
    if (e != hipSuccess) return hip_fail(e, "norm launch");
    x = a.out;
  }
  return forward_impl("moe_block_forward", s, x, router_w, router_bias, w_gate, w_up, w_down, s_gate, s_up, s_down,
                      nullptr, topk_ids_out, topk_w_out, workspace, fwd, stream, &pa);
}

}  // extern "C"
