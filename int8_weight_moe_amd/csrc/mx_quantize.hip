// MXFP4 quantizer, dequantizer and packer (layouts in mx_common.h).
//
// Per block of 32 elements: b = floor(log2(max |w|)) - 2 + 127, at least 0;
// code = the e2m1 value nearest to w / 2^(b - 127) (ties to the even code),
// saturated to +-6, with the sign of w. A block holding an infinity or a NaN
// gets b = 255, which makes every element NaN. One power-of-two division and
// one rounding by the hardware's packed convert: bit-exact.
//
// Bound by HBM: each element is read once and its half byte written once.
// Eight elements a lane (16 bytes of bf16), four lanes a block: the largest
// magnitude takes two lane exchanges and every lane packs one dword of codes,
// so loads and row-major stores are contiguous over the wave. Measured: 16 x 14336
// rows of 4096 bf16 numbers into the tiled layout 416 us (5720 GB/s), back 446 us
// (5330 GB/s).
#include "kernels.h"
#include "mx_common.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;

// Eight consecutive elements as fp32.
template <bool kBf16>
__device__ __forceinline__ void load8(const void* w, long idx, float (&v)[8]) {
  if constexpr (kBf16) {
    const u32x4 u = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(w) + idx));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  } else {
    const f32x4* p = reinterpret_cast<const f32x4*>(static_cast<const float*>(w) + idx);
    const f32x4 a = __builtin_nontemporal_load(p), b = __builtin_nontemporal_load(p + 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  }
}

template <bool kBf16>
__device__ __forceinline__ void store8(void* w, long idx, uint32_t codes, float scale) {
  if constexpr (kBf16) {
    *reinterpret_cast<bf16x8*>(static_cast<__bf16*>(w) + idx) = mx_bf16x8(codes, scale);
  } else {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 0);
    const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 1);
    const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 2);
    const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 3);
    f32x4* p = reinterpret_cast<f32x4*>(static_cast<float*>(w) + idx);
    p[0] = f32x4{a[0], a[1], b[0], b[1]};
    p[1] = f32x4{c[0], c[1], d[0], d[1]};
  }
}

// One dword of codes from a lane's eight elements and its block's scale byte
// (the four lanes of a block hold it all). All lanes of the block call it.
__device__ __forceinline__ uint32_t quantize8(const float (&v)[8], uint32_t& scale_byte) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  m = max(m, (uint32_t)__shfl_xor((int)m, 1));
  m = max(m, (uint32_t)__shfl_xor((int)m, 2));
  scale_byte = mx_scale_byte(m);
  if (scale_byte == 255u) return 0u;
  const float s = mx_scale(scale_byte);
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], s, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], s, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], s, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], s, 3);
  return c;
}

// Row-major, seen as one run of `chunks` eight-element chunks (a row is a
// whole number of blocks, so chunks is a multiple of 4), one a thread: 100003 x
// 4096 fp32 numbers and back took 687 us so, 790, 833 and 854 with two, four and
// eight a thread, 909 with 2048 threads a CU that stride over the run.
template <bool kBf16>
__global__ __launch_bounds__(kThreads) void mx_quantize_kernel(const void* __restrict__ w, long chunks,
                                                               uint32_t* __restrict__ q, uint8_t* __restrict__ s) {
  const long i = (long)blockIdx.x * kThreads + threadIdx.x;
  if (i >= chunks) return;   // the four lanes of a block together
  float v[8];
  load8<kBf16>(w, i * 8, v);
  uint32_t b;
  q[i] = quantize8(v, b);
  if ((i & 3) == 0) s[i >> 2] = (uint8_t)b;
}

template <bool kBf16>
__global__ __launch_bounds__(kThreads) void mx_dequantize_kernel(const uint32_t* __restrict__ q,
                                                                 const uint8_t* __restrict__ s, long chunks,
                                                                 void* __restrict__ w) {
  const long i = (long)blockIdx.x * kThreads + threadIdx.x;
  if (i < chunks) store8<kBf16>(w, i * 8, q[i], mx_scale(s[i >> 2]));
}

// Tiled: a wave owns 16 rows x 512 columns (four blocks, one scale dword a
// lane; fewer in a row group's last part). Row r is one load of the wave: lane
// l holds columns 8*l .. +8, i.e. block l/16, dword l%4 of piece (l%16)/4 of
// row r. Codes and scales are put in order in LDS, so the stores are
// contiguous too.
template <bool kBf16>
__global__ __launch_bounds__(kThreads) void mx_quantize_tiled_kernel(const void* __restrict__ w, long parts, int cols,
                                                                     uint8_t* __restrict__ q,
                                                                     uint8_t* __restrict__ s) {
  __shared__ __attribute__((aligned(16))) uint32_t codes[kWaves][kMxGroup * 256];
  __shared__ __attribute__((aligned(16))) uint8_t scales[kWaves][kMxGroup * 64];
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int n = cols / kMxStep;
  const int gpr = (n + kMxGroup - 1) / kMxGroup;
  const long part = (long)blockIdx.x * kWaves + wave;
  const bool live = part < parts;
  const long rg = live ? part / gpr : 0;
  const int g = live ? (int)(part - rg * gpr) * kMxGroup : 0;
  const int m = min(kMxGroup, n - g);
  const int j = lane >> 4;                       // this lane's block of the part
  const bool mine = live && j < m;               // the same for the four lanes of a scale group
#pragma unroll 8
  for (int r = 0; r < 16; ++r) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
    if (mine) load8<kBf16>(w, (rg * 16 + r) * cols + (long)g * kMxStep + 8 * lane, v);
    uint32_t b;
    const uint32_t c = quantize8(v, b);
    const int piece = (lane & 15) >> 2;          // 32-column group of the block
    codes[wave][j * 256 + (piece * 16 + r) * 4 + (lane & 3)] = c;
    if (mine && (lane & 3) == 0) scales[wave][m * (piece * 16 + r) + j] = (uint8_t)b;
  }
  __syncthreads();
  if (!live) return;
  const long block0 = rg * n + g;
#pragma unroll
  for (int k = 0; k < kMxGroup; ++k)
    if (k < m)
      *reinterpret_cast<uint4*>(q + (block0 + k) * 1024 + 16 * lane) =
          *reinterpret_cast<const uint4*>(&codes[wave][k * 256 + lane * 4]);
  // 64*m bytes of scales, a multiple of 64, at a multiple of 64
  if (lane < 16 * m)
    *reinterpret_cast<uint32_t*>(s + block0 * 64 + 4 * lane) =
        *reinterpret_cast<const uint32_t*>(&scales[wave][4 * lane]);
}

template <bool kBf16>
__global__ __launch_bounds__(kThreads) void mx_dequantize_tiled_kernel(const uint8_t* __restrict__ q,
                                                                       const uint8_t* __restrict__ s, long parts,
                                                                       int cols, void* __restrict__ w) {
  __shared__ __attribute__((aligned(16))) uint32_t codes[kWaves][kMxGroup * 256];
  __shared__ __attribute__((aligned(16))) uint8_t scales[kWaves][kMxGroup * 64];
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int n = cols / kMxStep;
  const int gpr = (n + kMxGroup - 1) / kMxGroup;
  const long part = (long)blockIdx.x * kWaves + wave;
  const bool live = part < parts;
  const long rg = live ? part / gpr : 0;
  const int g = live ? (int)(part - rg * gpr) * kMxGroup : 0;
  const int m = min(kMxGroup, n - g);
  const long block0 = rg * n + g;
  if (live) {
#pragma unroll
    for (int k = 0; k < kMxGroup; ++k)
      if (k < m)
        *reinterpret_cast<uint4*>(&codes[wave][k * 256 + lane * 4]) =
            *reinterpret_cast<const uint4*>(q + (block0 + k) * 1024 + 16 * lane);
    if (lane < 16 * m)
      *reinterpret_cast<uint32_t*>(&scales[wave][4 * lane]) =
          *reinterpret_cast<const uint32_t*>(s + block0 * 64 + 4 * lane);
  }
  __syncthreads();
  const int j = lane >> 4;
  if (!live || j >= m) return;
  const int piece = (lane & 15) >> 2;
#pragma unroll 4
  for (int r = 0; r < 16; ++r)
    store8<kBf16>(w, (rg * 16 + r) * cols + (long)g * kMxStep + 8 * lane,
                  codes[wave][j * 256 + (piece * 16 + r) * 4 + (lane & 3)],
                  mx_scale(scales[wave][m * (piece * 16 + r) + j]));
}

// Row-major codes and scales -> tiled: one thread moves one 16-byte piece and
// its scale byte.
__global__ __launch_bounds__(kThreads) void mx_pack_kernel(const uint8_t* __restrict__ q,
                                                           const uint8_t* __restrict__ s, long pieces, int cols,
                                                           uint8_t* __restrict__ q_tiled,
                                                           uint8_t* __restrict__ s_tiled) {
  const long p = (long)blockIdx.x * kThreads + threadIdx.x;
  if (p >= pieces) return;
  const int n = cols / kMxStep;
  const long block = p >> 6;
  const int l = (int)(p & 63);
  const long rg = block / n;
  const int ks = (int)(block - rg * n);
  const long src = (rg * 16 + (l & 15)) * (long)(cols / 32) + ks * 4 + (l >> 4);   // 32-column group of the matrix
  *reinterpret_cast<uint4*>(q_tiled + p * 16) = *reinterpret_cast<const uint4*>(q + src * 16);
  s_tiled[rg * n * 64 + mx_scale_at(n, ks, l)] = s[src];
}

constexpr long kLaunchChunks = 1L << 30;   // of one launch: a grid holds fewer than 2^32 threads

}  // namespace

hipError_t launch_mx_quantize(int64_t rows, int cols, bool src_bf16, const void* w, bool tiled, uint8_t* q, uint8_t* s,
                              hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  if (tiled) {
    const long parts = rows / 16 * ((cols / kMxStep + kMxGroup - 1) / kMxGroup);
    const dim3 grid((unsigned)((parts + kWaves - 1) / kWaves));
    if (src_bf16)
      hipLaunchKernelGGL(mx_quantize_tiled_kernel<true>, grid, dim3(kThreads), 0, stream, w, parts, cols, q, s);
    else
      hipLaunchKernelGGL(mx_quantize_tiled_kernel<false>, grid, dim3(kThreads), 0, stream, w, parts, cols, q, s);
    return hipGetLastError();
  }
  const long chunks = rows * (long)(cols / 8);
  for (long c = 0; c < chunks; c += kLaunchChunks) {
    const long m = min(chunks - c, kLaunchChunks);
    const dim3 grid((unsigned)((m + kThreads - 1) / kThreads));
    const char* src = static_cast<const char*>(w) + c * (src_bf16 ? 16 : 32);
    uint32_t* qc = reinterpret_cast<uint32_t*>(q) + c;
    if (src_bf16)
      hipLaunchKernelGGL(mx_quantize_kernel<true>, grid, dim3(kThreads), 0, stream, src, m, qc, s + c / 4);
    else
      hipLaunchKernelGGL(mx_quantize_kernel<false>, grid, dim3(kThreads), 0, stream, src, m, qc, s + c / 4);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_mx_dequantize(int64_t rows, int cols, bool tiled, const uint8_t* q, const uint8_t* s, bool dst_bf16,
                                void* w, hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  if (tiled) {
    const long parts = rows / 16 * ((cols / kMxStep + kMxGroup - 1) / kMxGroup);
    const dim3 grid((unsigned)((parts + kWaves - 1) / kWaves));
    if (dst_bf16)
      hipLaunchKernelGGL(mx_dequantize_tiled_kernel<true>, grid, dim3(kThreads), 0, stream, q, s, parts, cols, w);
    else
      hipLaunchKernelGGL(mx_dequantize_tiled_kernel<false>, grid, dim3(kThreads), 0, stream, q, s, parts, cols, w);
    return hipGetLastError();
  }
  const long chunks = rows * (long)(cols / 8);
  for (long c = 0; c < chunks; c += kLaunchChunks) {
    const long m = min(chunks - c, kLaunchChunks);
    const dim3 grid((unsigned)((m + kThreads - 1) / kThreads));
    const uint32_t* qc = reinterpret_cast<const uint32_t*>(q) + c;
    char* dst = static_cast<char*>(w) + c * (dst_bf16 ? 16 : 32);
    if (dst_bf16)
      hipLaunchKernelGGL(mx_dequantize_kernel<true>, grid, dim3(kThreads), 0, stream, qc, s + c / 4, m, dst);
    else
      hipLaunchKernelGGL(mx_dequantize_kernel<false>, grid, dim3(kThreads), 0, stream, qc, s + c / 4, m, dst);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_mx_pack(int64_t rows, int cols, const uint8_t* q, const uint8_t* s, uint8_t* q_tiled,
                          uint8_t* s_tiled, hipStream_t stream) {
  const long pieces = rows * (long)(cols / 32);
  if (pieces == 0) return hipSuccess;
  hipLaunchKernelGGL(mx_pack_kernel, dim3((unsigned)((pieces + kThreads - 1) / kThreads)), dim3(kThreads), 0, stream,
                     q, s, pieces, cols, q_tiled, s_tiled);
  return hipGetLastError();
}

}  // namespace moe
