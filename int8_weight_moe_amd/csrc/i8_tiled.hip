// Products of int8 weights and int8 rows with many rows per expert (prefill): tiled MFMA.
//
//   out[r, n] = a_s[row(r)] * w_s[n] * sum_k a_q[row(r), k] * w_q[n, k],   or   silu(p0) * p1
//
// over the row segments of the experts. A workgroup of four waves owns a tile of
// kBM rows x kBN channels of one expert (with two matrices, kBN/2 channels of
// each); a wave owns all the rows and a quarter of the channels.
//   weights  are read by one wave only, so they go straight from memory to its
//            registers, one 1 KiB block per 16 channels and 64 columns, one step ahead;
//   rows     are shared by the waves and go through LDS, by direct global->LDS
//            loads, double buffered, one barrier a step. A step is 128 columns; the
//            16-byte chunks of a row are XOR-swizzled by the row number, so the
//            fragment reads (16 rows at one chunk) meet no bank conflict.
// Channels are MFMA rows and tokens MFMA columns, so a lane ends with four
// consecutive channels of one row. Sums are int32, exact.
// Tile order as in ffn_tiled.hip: groups of row tiles of one expert take every
// channel tile in turn, in eight contiguous XCD queues.
// Rows past the segment read row 0 of the tile and channels past N read channel
// 0; their results are not stored.
// Bound by the clock and the wait of each step: 8192 tokens of two experts of 16 (d 4096, f 14336, gate/up) 1804 to 1908 us
// by the card, 2.02 to 2.13 POP/s, the MFMAs busy 54% of the cycles at 1.9 GHz; 16384 tokens skewed (d 24576, f 8192, down) 5700
// to 6003 us, 2.20 to 2.31 POP/s, 64% at 1.7 GHz; no bank conflicts. A library product of these sizes reaches 2.1 and 2.45. Slower: two steps a barrier (1%),
// non-temporal weights (20 to 50%), 64 rows (17 to 33%), and one wave a SIMD on 256 rows x 256 channels (11 to 21%:
// nothing runs while it waits).
#include "i8_common.h"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kWaves = 4;
constexpr int kXcds = 8;
constexpr int KB = 2;               // 64-column blocks per step
constexpr int ROWB = KB * kI8Step;  // bytes of a row per step
constexpr int CPR = ROWB / 16;      // its 16-byte chunks
constexpr int RPI = 1024 / ROWB;    // rows per 1 KiB load

template <int NMAT, bool kOutBf16, int GM, int kBM, int kBN, int kWpe>
__global__ __launch_bounds__(kWaves* kWave) __attribute__((amdgpu_waves_per_eu(kWpe, kWpe))) void i8_tiled_kernel(
    I8Args a, int n_tiles) {
  constexpr int A_STAGE = kBM * ROWB;
  constexpr int A_INSTR = A_STAGE / 1024 / kWaves; // 1 KiB loads per wave and step
  constexpr int MB = kBM / 16;                     // row blocks (of every wave)
  constexpr int NB = kBN / 16 / kWaves;            // channel blocks of a wave
  constexpr int HALF = NB / NMAT;                  // of each matrix
  constexpr int CH_TILE = kBN / NMAT;
  __shared__ __attribute__((aligned(1024))) uint8_t As[2][A_STAGE];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int li = lane & 15;
  const int lg = lane >> 4;
  const int N = a.N, n = a.Kd / kI8Step;           // blocks along the reduction

  int e, row0, nrows, nt;
  {
    const TileGrid g = tile_grid<kBM>(a.offsets, a.E, n_tiles, kXcds, 1);
    const int tile = static_tile(g, kXcds);
    if (tile < 0) return;
    decode_tile<kBM, GM>(g, tile, a.E, n_tiles, e, row0, nrows, nt);
  }
  const int n0 = nt * CH_TILE;

  // ---- row sources: load j of this wave covers rows RPI*(wave + kWaves*j) + lane/CPR (so the first loads of all the
  // waves cover the first rows); byte offset of this lane's chunk at step 0, 32 bits from the tile's first row (128 rows of
  // 131072 at most), or for gathered rows from row 0 (i8_tiled_offsets_fit). Streamed instead, rows past 4 GiB take 6 to 40
  // times as long (90000 rows of 49152, E 8, f 4096: 91.2 / 14.7 ms).
  const int8_t* rows = a.sorted_slots ? a.a : a.a + (long)row0 * a.Kd;
  uint32_t a_off[A_INSTR];
#pragma unroll
  for (int j = 0; j < A_INSTR; ++j) {
    const int r = RPI * (wave + kWaves * j) + lane / CPR;
    const int rr = r < nrows ? r : 0;
    const uint32_t src = (uint32_t)(a.sorted_slots ? a.sorted_slots[row0 + rr] / a.topk : rr);
    a_off[j] = src * (uint32_t)a.Kd + (uint32_t)(((lane % CPR) ^ (r % CPR)) * 16);
  }
  // The second block of the last step of an odd number of blocks re-reads the first one: 64 bytes back for the lanes
  // whose chunk lies in it (a load covers whole swizzle periods, so the chunk is the same for every load).
  const uint32_t second = (((lane % CPR) ^ (lane / CPR % CPR)) & 4) ? 64u : 0u;
  auto step_off = [&](int step) { return (uint32_t)step * ROWB - (second & (2 * step + 1 >= n ? ~0u : 0u)); };

  // ---- weight sources: this lane's 16 bytes of block 0 of each channel block
  const int8_t* b_ptr[NB];
  int ch_of[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int ch = n0 + wave * (HALF * 16) + (j % HALF) * 16;
    ch_of[j] = ch;
    const long block = (((long)e * N + (ch < N ? ch : 0)) >> 4) * n;
    b_ptr[j] = (NMAT == 2 && j >= HALF ? a.w1 : a.w0) + block * 1024;
  }

  const int nsteps = (n + KB - 1) / KB;
  auto issue_a = [&](int step, int buf, auto mbc) {
    constexpr int LOADS = decltype(mbc)::value * 16 / RPI / kWaves;
    const uint32_t off = step_off(min(step, nsteps - 1));
#pragma unroll
    for (int j = 0; j < LOADS; ++j)
      dma16(rows, a_off[j] + off, lds_addr(&As[buf][0]) + (wave + kWaves * j) * 1024);
  };
  auto load_b = [&](int step, uint4 (&b)[NB][KB]) {
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int k = 0; k < KB; ++k) {
        const int8_t* p = b_ptr[j] + (long)min(step * KB + k, n - 1) * 1024;   // uniform
        b[j][k] = *reinterpret_cast<const uint4*>(p + 16u * (uint32_t)lane);
      }
  };

  i32x4 acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = i32x4{0, 0, 0, 0};

  auto main_loop = [&](auto mbc) {
    constexpr int MBV = decltype(mbc)::value;      // row blocks loaded and computed
    static_assert(MBV * 16 % (RPI * kWaves) == 0, "whole loads");
    uint4 b[2][NB][KB];
    issue_a(0, 0, mbc);
    load_b(0, b[0]);
    auto step = [&](auto bc, int st) {
      constexpr int B = decltype(bc)::value;
      if (st >= nsteps) return;
      // this step's loads have landed and every wave is past the buffers that the next ones overwrite
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));
      __builtin_amdgcn_s_barrier();
      issue_a(st + 1, 1 - B, mbc);
      load_b(st + 1, b[1 - B]);
#pragma unroll
      for (int k = 0; k < KB; ++k) {
        if (k > 0 && 2 * st + k >= n) break;
        constexpr int HB = MBV % 4 == 0 ? 4 : 2;   // row blocks whose fragments are read together (two: 3% slower)
#pragma unroll
        for (int h = 0; h < MBV; h += HB) {
          uint4 xf[HB];
#pragma unroll
          for (int i = 0; i < HB; ++i) {
            const int r = (h + i) * 16 + li;
            xf[i] = *reinterpret_cast<const uint4*>(&As[B][r * ROWB + (((4 * k + lg) ^ (r % CPR)) * 16)]);
          }
#pragma unroll
          for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int i = 0; i < HB; ++i) acc[h + i][j] = mfma_i8(as_i32x4(b[B][j][k]), as_i32x4(xf[i]), acc[h + i][j]);
        }
      }
    };
    for (int st = 0; st < nsteps; st += 2) {
      step(int_constant<0>{}, st);
      step(int_constant<1>{}, st + 1);
    }
  };
  // a segment's last tile skips the row blocks it does not have, in steps of two
  const int mb_valid = (nrows + 15) / 16;
  switch ((mb_valid + 1) / 2) {
    case 1: main_loop(int_constant<2>{}); break;
    case 2: main_loop(int_constant<MB < 4 ? MB : 4>{}); break;
    case 3: main_loop(int_constant<MB < 6 ? MB : 6>{}); break;
    default: main_loop(int_constant<MB>{}); break;
  }
  // no load may still be writing this workgroup's LDS when the waves exit
  __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));

  float4 ws[HALF][NMAT];
#pragma unroll
  for (int j = 0; j < HALF; ++j) {
    const long ch = (long)e * N + (ch_of[j] < N ? ch_of[j] : 0) + 4 * lg;
    ws[j][0] = i8_scale4(a.s0, a.scale_bf16, ch);
    if constexpr (NMAT == 2) ws[j][1] = i8_scale4(a.s1, a.scale_bf16, ch);
  }
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    const int r = i * 16 + li;
    if (r >= nrows) continue;
    const int rr = row0 + r;
    const float as = a.a_s[a.sorted_slots ? a.sorted_slots[rr] / a.topk : rr];
#pragma unroll
    for (int j = 0; j < HALF; ++j) {
      if (ch_of[j] >= N) continue;
      i32x4 v[NMAT];
      v[0] = acc[i][j];
      if constexpr (NMAT == 2) v[1] = acc[i][j + HALF];
      i8_store4<NMAT, kOutBf16>(a.out, (long)rr * N + ch_of[j] + 4 * lg, v, ws[j], as);
    }
  }
}

// Channel tiles of a row of tiles, and the most tiles that any segments make.
int tile_columns(const I8Args& a, int channels) {
  const int ch = a.w1 ? channels / 2 : channels;
  return (a.N + ch - 1) / ch;
}
long tile_bound(const I8Args& a, int rows, int channels) {
  return ((long)(a.S + rows - 1) / rows + a.E) * tile_columns(a, channels);
}

template <int NMAT, bool kOutBf16, int kBM, int kBN, int kWpe>
hipError_t launch_tile(const I8Args& a, hipStream_t stream) {
  constexpr int GM = 8;   // row tiles of an expert that take a channel tile together (4: 2 to 5% slower, 12: within 1%)
  const long per_xcd = (tile_bound(a, kBM, kBN) + kXcds - 1) / kXcds;
  hipLaunchKernelGGL((i8_tiled_kernel<NMAT, kOutBf16, GM, kBM, kBN, kWpe>), dim3((unsigned)(kXcds * per_xcd)),
                     dim3(kWaves * kWave), 0, stream, a, tile_columns(a, kBN));
  return hipGetLastError();
}

template <int NMAT, bool kOutBf16>
hipError_t launch_columns(const I8Args& a, hipStream_t stream) {
  return i8_tile_columns(a) == 128 ? launch_tile<NMAT, kOutBf16, 128, 128, 3>(a, stream)
                                   : launch_tile<NMAT, kOutBf16, 128, 256, 2>(a, stream);
}

}  // namespace

bool i8_tiled_offsets_fit(const I8Args& a) { return !a.sorted_slots || (uint64_t)a.a_rows * (uint64_t)a.Kd < (1ull << 32); }

bool i8_few_tiles(const I8Args& a) {
  return (long)max(min(a.E, a.S), (a.S + 127) / 128) * tile_columns(a, 128) < 256;
}

// Channels of a tile. Measured, us, 128 / 256: gate/up, d 4096, f 14336, E 16: 16 rows an expert 350 / 368, 32 348 / 378, 64
// 354 / 357, 128 499 / 486, 1024 2149 / 2034; d 4160, f 1472, E 40, 25 rows 60 / 64; one expert, 64 rows, d 8192, f 24576 95 / 106;
// down, d 24576, f 8192, E 16: 16 rows 690 / 609, 375 1419 / 1267, 2048 6998 / 5853; few tiles: d 14336, f 4096, 32 rows 180 / 199.
int i8_tile_columns(const I8Args& a) {
  return (a.w1 && a.S <= 64L * a.E) || tile_bound(a, 128, 256) < 512 ? 128 : 256;
}

hipError_t launch_i8_tiled(const I8Args& a, hipStream_t stream) {
  if (a.w1) return a.out_bf16 ? launch_columns<2, true>(a, stream) : launch_columns<2, false>(a, stream);
  return a.out_bf16 ? launch_columns<1, true>(a, stream) : launch_columns<1, false>(a, stream);
}

}  // namespace moe
