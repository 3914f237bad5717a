// The norms before and after the layer.
//
//   rms(v) = v / sqrt(mean(v^2) + eps), per token (row of d elements)
//   pre    n = rms(x) * weight
//   post   out  = residual_scale * residual + block_scale * gate * (rms(y) * weight)
//          next = rms(out) * next_weight
// y is given, or is the combine of the experts' rows, sum_k topk_w[k] *
// y_rows[row(k)]. Everything between the loads and the one rounding of each
// output is fp32; `next` is taken from the fp32 sum, not from its rounding to
// out's type.
//
// Bound by HBM: every operand is read once and every output written once. A
// token's row stays in registers from the load to the store (kChunks chunks of
// eight elements a thread), so the sums over the row cost two exchanges (lanes,
// then waves through LDS) and no second pass over memory. Each thread reads its
// elements of residual and x before it writes the same elements of out and n,
// so those pairs may share memory. Measured: combine, norms, gate and residual of
// 16384 tokens, d 8192, K 2, 351 us (5350 GB/s; 326 on inputs used just before); one token before the layer 2.6 us.
// For few tokens the kernel is a chain of dependent loads (row numbers, rows, then the operands behind each sum): 63
// tokens, d 4096, K 2, 4.6 us where the launch takes 2 and the bytes 0.9.
#include "kernels.h"
#include "device_common.h"

namespace moe {

namespace {

__device__ __forceinline__ void load8f(const __bf16* p, float (&v)[8]) {
  const u32x4 u = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8f(const float* p, float (&v)[8]) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = a[i];
    v[4 + i] = b[i];
  }
}
// kNt: a store that does not stay in the caches
template <bool kNt, typename T>
__device__ __forceinline__ void store_v(T* p, T v) {
  if constexpr (kNt) __builtin_nontemporal_store(v, p);
  else *p = v;
}
template <bool kNt>
__device__ __forceinline__ void store8f(__bf16* p, const float (&v)[8]) {
  bf16x8 o;
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = (__bf16)v[i];
  store_v<kNt>(reinterpret_cast<bf16x8*>(p), o);
}
template <bool kNt>
__device__ __forceinline__ void store8f(float* p, const float (&v)[8]) {
  store_v<kNt>(reinterpret_cast<f32x4*>(p), f32x4{v[0], v[1], v[2], v[3]});
  store_v<kNt>(reinterpret_cast<f32x4*>(p + 4), f32x4{v[4], v[5], v[6], v[7]});
}
// the experts' rows are read once
__device__ __forceinline__ void load8nt(const float* p, float (&v)[8]) {
  const f32x4 a = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p));
  const f32x4 b = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p + 4));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = a[i];
    v[4 + i] = b[i];
  }
}

// Sum over the workgroup's threads; the same value in every thread. `red` is
// used once per call: two calls in a row take two arrays.
template <int kThreads>
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  if constexpr (kThreads > kWave) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / kWave; ++w) v += red[w];
  }
  return v;
}

enum NormSource { kNormX, kNormY, kNormCombine };   // pre; post of a given y; post of the combine

template <typename Act, int kSrc, int kThreads, int kChunks, bool kNt>
__global__ __launch_bounds__(kThreads) void block_norm_kernel(NormArgs a) {
  __shared__ float red[2][16];
  const int t = blockIdx.y * gridDim.x + blockIdx.x;
  if (t >= a.T) return;
  const int d = a.d;
  const long row = (long)t * d;
  float v[kChunks][8];
  float sq = 0.f;
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int col = (c * kThreads + (int)threadIdx.x) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[c][i] = 0.f;
    if (col < d) {
      if constexpr (kSrc == kNormCombine) {
        for (int k = 0; k < a.K; ++k) {
          const int r = a.slot_to_row[(long)t * a.K + k];
          if (r < 0) continue;
          const float w = a.topk_w[(long)t * a.K + k];
          float u[8];
          load8nt(a.y_rows + (long)r * d + col, u);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[c][i] += w * u[i];
        }
      } else {
        load8f(static_cast<const Act*>(a.x) + row + col, v[c]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sq += v[c][i] * v[c][i];
    }
  }
  float scale = 1.f;
  if (a.weight) scale = 1.f / sqrtf(block_sum<kThreads>(sq, red[0]) / (float)d + a.eps);

  float sq2 = 0.f;
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int col = (c * kThreads + (int)threadIdx.x) * 8;
    if (col < d) {
      if (a.weight) {
        float w[8];
        load8f(static_cast<const Act*>(a.weight) + col, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] = v[c][i] * scale * w[i];
      }
      if constexpr (kSrc != kNormX) {
        float r[8];
        load8f(static_cast<const Act*>(a.residual) + row + col, r);
        if (a.gate) {
          float g[8];
          load8f(static_cast<const Act*>(a.gate) + (long)(t / a.gate_tokens) * d + col, g);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[c][i] *= g[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[c][i] = a.residual_scale * r[i] + a.block_scale * v[c][i];
          sq2 += v[c][i] * v[c][i];
        }
      }
      store8f<kNt>(static_cast<Act*>(a.out) + row + col, v[c]);
    }
  }
  if constexpr (kSrc != kNormX) {
    if (!a.next_weight) return;   // the same for every thread
    const float s2 = 1.f / sqrtf(block_sum<kThreads>(sq2, red[1]) / (float)d + a.next_eps);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int col = (c * kThreads + (int)threadIdx.x) * 8;
      if (col < d) {
        float w[8];
        load8f(static_cast<const Act*>(a.next_weight) + col, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = v[c][i] * s2 * w[i];
        store8f<kNt>(static_cast<Act*>(a.next) + row + col, w);
      }
    }
  }
}

template <typename Act, int kSrc>
hipError_t launch_norm(const NormArgs& a, hipStream_t stream) {
  // a grid dimension holds fewer than 2^32 threads
  const unsigned gx = (unsigned)min(a.T, 1 << 20);
  const dim3 grid(gx, (unsigned)((a.T + (long)gx - 1) / gx));
  const int n8 = a.d / 8;
#define MOE_NORM_CASE(TH, CH, NT) \
  hipLaunchKernelGGL((block_norm_kernel<Act, kSrc, TH, CH, NT>), grid, dim3(TH), 0, stream, a)
  // Few tokens: a chunk of eight elements a thread, for the shortest chain.
  // Many: the fewest threads that keep a row within four chunks, for the fewest
  // exchanges. Outputs that no cache would keep for the next reader (64 MiB on)
  // are stored past the caches (combine of 16384 x 8192: 365 -> 325 us, with
  // the experts' rows loaded the same way; of 16384 x 1024: 46 us against 44).
  const bool nt = (long)a.T * a.d * (long)sizeof(Act) >= (64L << 20);
  if (nt) {
    if (n8 <= 64 * 4) MOE_NORM_CASE(64, 4, true);
    else if (n8 <= 256 * 4) MOE_NORM_CASE(256, 4, true);
    else if (n8 <= 1024 * 4) MOE_NORM_CASE(1024, 4, true);
    else MOE_NORM_CASE(1024, 8, true);
  } else if (a.T < 1024 && n8 <= 1024) {
    if (n8 <= 64) MOE_NORM_CASE(64, 1, false);
    else if (n8 <= 256) MOE_NORM_CASE(256, 1, false);
    else MOE_NORM_CASE(1024, 1, false);
  } else if (n8 <= 64 * 4) MOE_NORM_CASE(64, 4, false);
  else if (n8 <= 256 * 4) MOE_NORM_CASE(256, 4, false);
  else if (n8 <= 1024 * 4) MOE_NORM_CASE(1024, 4, false);
  else MOE_NORM_CASE(1024, 8, false);
#undef MOE_NORM_CASE
  return hipGetLastError();
}

template <typename Act>
hipError_t dispatch_norm(const NormArgs& a, hipStream_t stream) {
  if (!a.residual) return launch_norm<Act, kNormX>(a, stream);
  return a.y_rows ? launch_norm<Act, kNormCombine>(a, stream) : launch_norm<Act, kNormY>(a, stream);
}

}  // namespace

hipError_t launch_block_norm(const NormArgs& a, hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  return a.act_bf16 ? dispatch_norm<__bf16>(a, stream) : dispatch_norm<float>(a, stream);
}

}  // namespace moe
