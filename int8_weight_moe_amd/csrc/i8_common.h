// Device-side pieces of the kernels whose products take both operands in int8.
//
//   out[r, n] = a_s[row(r)] * w_s[n] * sum_k a_q[row(r), k] * w_q[n, k]
//
// The sum is exact: int8 products in int32 (127 * 127 * 131072 < 2^31). Weights
// lie in the tiled layout of pack.hip: a 1 KiB block is 16 channels x 64 columns
// and lane l's 16 bytes at 16*l are channel l%16, columns 16*(l/16) .. +16 of it,
// which is one operand of the 16x16x64 int8 MFMA. The rows' operand holds the
// same columns of row l%16, so what matters of the instruction's column order
// is that both operands share it.
#pragma once

#include "device_common.h"

namespace moe {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kI8Step = 64;   // columns of one 1 KiB block

__device__ __forceinline__ i32x4 as_i32x4(uint4 v) { return __builtin_bit_cast(i32x4, v); }

// 16x16x64 int8 MFMA: lane l supplies row l%16 of its operand, columns 16*(l/16)
// .. +16. Result: lane l holds C[4*(l/16) + i][l%16], i = 0..3, rows from a and
// columns from b.
__device__ __forceinline__ i32x4 mfma_i8(i32x4 a, i32x4 b, i32x4 c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// Four consecutive scales (idx % 4 == 0).
__device__ __forceinline__ float4 i8_scale4(const void* s, bool bf16, long idx) {
  return bf16 ? load_scale4<true>(s, idx) : load_scale4<false>(s, idx);
}

// Four consecutive channels of one row from their sums, as out's type: the
// scaled sums (NMAT = 1), or silu(first) * second. A sum becomes fp32 (one
// rounding past 2^24) and takes its two scales, the channel's first. SwiGLU for an
// fp32 out takes the full-precision exponential and division; for a bf16 one the
// hardware's, whose errors are far below its rounding (the epilogue of a 128x256
// tile of 4096 columns: 2030 -> 1950 us with its four-fragment steps).
template <int NMAT, bool kOutBf16>
__device__ __forceinline__ void i8_store4(void* out, long o, const i32x4 (&acc)[NMAT], const float4 (&ws)[NMAT], float as) {
  f32x4 v;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    auto scaled = [&](int m) {
      const float s = q == 0 ? ws[m].x : q == 1 ? ws[m].y : q == 2 ? ws[m].z : ws[m].w;
      return (float)acc[m][q] * s * as;
    };
    v[q] = scaled(0);
    if constexpr (NMAT == 2) v[q] = (kOutBf16 ? silu(v[q]) : v[q] / (1.0f + expf(-v[q]))) * scaled(NMAT - 1);
  }
  if constexpr (kOutBf16) {
    bf16x4 b;
#pragma unroll
    for (int q = 0; q < 4; ++q) b[q] = (__bf16)v[q];
    *reinterpret_cast<bf16x4*>(static_cast<__bf16*>(out) + o) = b;
  } else {
    *reinterpret_cast<f32x4*>(static_cast<float*>(out) + o) = v;
  }
}

}  // namespace moe
