// Device-side pieces of the MXFP4 kernels (gfx950).
//
// MXFP4 (OCP microscaling): along a row, 32 elements share one scale byte b
// worth 2^(b - 127) (255: not a number); an element is a 4-bit e2m1 code (sign,
// magnitude 0, 0.5, 1, 1.5, 2, 3, 4, 6), two a byte, the even element in the
// low half.
//
// Tiled layout of a matrix [rows, cols] (rows % 16 == 0, cols % 128 == 0):
//   codes   the layout of pack.hip over the row's cols/2 bytes: 1 KiB blocks of
//           16 rows x 128 columns, block (rg, ks) at index rg*(cols/128) + ks;
//           lane l's 16 bytes at 16*l are row l%16, columns 32*(l/16) .. +32 of
//           the block: one scale group, and one lane's operand of the
//           16x16x128 scaled MFMA;
//   scales  one byte per lane and block, the bytes of four consecutive blocks
//           side by side, so a lane takes four steps' scales in one dword (and
//           the scaled MFMA picks one with its byte select): block (rg, ks),
//           lane l sits at rg*(cols/128)*64 + 256*(ks/4) + m*l + ks%4 with
//           m = min(4, cols/128 - 4*(ks/4)) (fewer than four in the last,
//           partial group of a row of blocks).
#pragma once

#include "device_common.h"

namespace moe {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kMxStep = 128;      // columns of one 1 KiB block
constexpr int kMxGroup = 4;       // blocks whose scales share a dword

// Byte of lane l's scale for block ks of a row group with n blocks, relative
// to the row group's scales.
__host__ __device__ __forceinline__ int mx_scale_at(int n, int ks, int l) {
  const int g = ks & ~3;
  const int m = n - g < 4 ? n - g : 4;
  return g * 64 + m * l + (ks - g);
}

// Two elements of the codes in byte kSel of `c`, times the scale, exactly (an
// element has two significant bits; its bf16 value is exact down to the
// smallest scale, and past the largest bf16 number it is infinite).
template <int kSel>
__device__ __forceinline__ bf16x2 mx_pair_bf16(uint32_t c, float scale) {
  return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, kSel);
}

// Eight elements (one dword of codes) as an MFMA operand.
__device__ __forceinline__ bf16x8 mx_bf16x8(uint32_t c, float scale) {
  const bf16x2 a = mx_pair_bf16<0>(c, scale), b = mx_pair_bf16<1>(c, scale), d = mx_pair_bf16<2>(c, scale),
               e = mx_pair_bf16<3>(c, scale);
  bf16x8 r;
  r[0] = a[0]; r[1] = a[1]; r[2] = b[0]; r[3] = b[1];
  r[4] = d[0]; r[5] = d[1]; r[6] = e[0]; r[7] = e[1];
  return r;
}

// The converts and the scaled MFMA read a scale's exponent bits only, so the
// byte moved into them is the scale for every b (0: 2^-127; 255: NaN).
__device__ __forceinline__ float mx_scale(uint32_t b) { return __uint_as_float(b << 23); }

// Byte j of a dword of scales.
template <int kJ>
__device__ __forceinline__ float mx_scale_of(uint32_t dword) {
  return __uint_as_float((kJ == 3 ? (dword >> 24) : ((dword >> (8 * kJ)) & 255u)) << 23);
}

// 16x16x128 MFMA with both operands in MXFP4: lane l supplies row l%16 of its
// operand, elements 32*(l/16) .. +32, and their scale in byte kSa / kSb of its
// scale dword. Products are exact; sums are fp32. Result as mfma_bf16.
template <int kSa, int kSb>
__device__ __forceinline__ f32x4 mfma_mx(uint4 a, uint4 b, f32x4 c, uint32_t sa, uint32_t sb) {
  const i32x8 av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const i32x8 bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, kSa, (int)sa, kSb, (int)sb);
}

// Four consecutive channels of one row from their sums: the sums themselves
// (NMAT = 1) or silu(first) * second, rounded once to the output type.
template <bool kOutBf16, int NMAT>
__device__ __forceinline__ void mx_store4(void* out, long o, const f32x4 (&acc)[NMAT]) {
  f32x4 v = acc[0];
  if constexpr (NMAT == 2) {
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = silu(v[q]) * acc[1][q];
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

// Scale byte of a block whose largest magnitude has the fp32 bits `amax`
// (sign cleared): 2^(floor(log2(amax)) - 2), so the block's largest element
// falls on 4 .. 6 (past 6: saturated); 255 if the block holds an infinity or a
// NaN (their bits are the largest).
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax) {
  const int e = (int)(amax >> 23);
  return e == 255 ? 255u : (uint32_t)max(e - 2, 0);
}

}  // namespace moe
