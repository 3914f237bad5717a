// Products of MXFP4 weights with many rows per expert (prefill): tiled MFMA.
//
//   out[r, n] = sum_k A[row(r), k] * W_e[n, k],   or   silu(W0 . a) * (W1 . a)
//
// over the row segments of the experts; A is bf16 (the expert FFN's passes) or
// MXFP4 (both operands in 4 bits). A workgroup of four waves owns a tile of
// kBM rows x kBN channels of one expert (with two matrices, kBN/2 channels of
// each); a wave owns all the rows and a quarter of the channels.
//   weights      are read by one wave only, so they go straight from memory to
//                its registers, one 1 KiB block per 16 channels and 128 columns
//                (16 bytes a lane: one scale group), one step ahead; a dword of
//                scales a lane holds four blocks' worth;
//   activations  are shared by the waves and go through LDS, by direct
//                global->LDS loads, double buffered, one barrier a step. A step
//                is 256 bytes of a bf16 row (128 columns) or 128 bytes of codes
//                (256 columns). The 16-byte chunks of a row are XOR-swizzled by
//                the row number, so the fragment reads (16 rows at one chunk)
//                meet no bank conflict with MXFP4 rows (counted: 0); with bf16
//                rows conflicts take 18% of the busy cycles. MXFP4 scales of the
//                rows: a dword (four scale groups) per row and block, four
//                blocks at a time.
// bf16 activations: the codes become bf16 in registers, exactly, scale
// included, and feed 16x16x32 bf16 MFMAs; MXFP4: the 16x16x128 scaled MFMA takes
// both operands as read. Channels are MFMA rows and tokens MFMA columns, so a
// lane ends with four consecutive channels of one row. Sums are fp32.
// Tile order as in ffn_tiled.hip: groups of row tiles of one expert take every
// channel tile in turn, in eight contiguous XCD queues.
// Bound by the MFMA rate at the clock that power leaves (1.5 to 1.8 of 2.4 GHz) and by
// the waits at each step: gate/up of 8192 tokens (d 4096, f 14336, E 16) 2727 us, 1411
// TFLOP/s, MFMA busy 72% of the cycles at 1.7 GHz, where a library bf16 product of that
// size reaches 1436; the same with MXFP4 activations 1143 us, 3366 TFLOP/s, 44% at 1.8 GHz;
// the down product of 16384 tokens (d 24576, f 8192) 3366 us, 3919 TFLOP/s, 57% at 1.5 GHz
// (a library MXFP4 product of 16384^3: 3462). Not faster: 32x32 MFMAs (5 to
// 9% slower), 256-row tiles of eight waves (4 to 7%), non-temporal weights (5 to 40%).
// Rows past the segment read row 0 of the tile and channels past N read channel
// 0; their results are not stored.
#include "kernels.h"
#include "mx_common.h"

namespace moe {

namespace {

constexpr int kWaves = 4;
constexpr int kXcds = 8;
constexpr int kClaimTail = 128;   // as in ffn_tiled.hip: the tiles of a queue's end that are claimed

// 4-byte-per-lane global->LDS load (see dma16): lane l's dword lands at lds + 4*l.
__device__ __forceinline__ void dma4(const void* base, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dword %1, %2" ::"s"(lds), "v"(voff), "s"(base) : "memory");
}

// Waves a SIMD must have room for, which is workgroups a CU: a smaller tile
// needs fewer accumulators, and more workgroups keep more weights in flight
// (bf16 activations of 128 rows fill LDS with two).
constexpr int waves_per_simd(bool mx_act, int rows, int channels) {
  return rows * channels >= 128 * 256 || (!mx_act && rows >= 128) ? 2 : 3;
}

template <bool kMxAct, int NMAT, bool kOutBf16, int GM, int kBM, int kBN>
__global__ __launch_bounds__(kWaves* kWave) __attribute__((amdgpu_waves_per_eu(waves_per_simd(kMxAct, kBM, kBN)))) void mx_tiled_kernel(
    MxArgs a, int n_tiles) {
  constexpr int KB = kMxAct ? 2 : 1;               // 128-column blocks per step
  constexpr int SPG = kMxGroup / KB;               // steps per scale group
  constexpr int ROWB = kMxAct ? 128 : 256;         // bytes of an activation row per step
  constexpr int CPR = ROWB / 16;                   // its 16-byte chunks
  static_assert(kBM == 64 || kBM == 128, "row scales: one or two loads of 64 a block");
  constexpr int A_STAGE = kBM * ROWB;
  constexpr int A_INSTR = A_STAGE / 1024 / kWaves; // 1 KiB loads per wave and step
  constexpr int RPI = 1024 / ROWB;                 // rows per load
  constexpr int MB = kBM / 16;                     // row blocks (of every wave)
  constexpr int NB = kBN / 16 / kWaves;            // channel blocks of a wave
  constexpr int HALF = NB / NMAT;                  // of each matrix
  constexpr int CH_TILE = kBN / NMAT;
  __shared__ __attribute__((aligned(1024))) uint8_t As[2][A_STAGE];
  __shared__ __attribute__((aligned(1024))) uint32_t Ss[2][kMxAct ? kMxGroup * kBM : 4];
  __shared__ int s_tile;

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int li = lane & 15;
  const int lg = lane >> 4;
  const int N = a.N, n = a.Kd / kMxStep;           // blocks along the reduction

  int e, row0, nrows, nt;
  {
    const TileGrid g = tile_grid<kBM>(a.offsets, a.E, n_tiles, kXcds, 1);
    const int tile = a.claims ? claimed_tail_tile(g, kXcds, kClaimTail, a.claims, &s_tile) : static_tile(g, kXcds);
    if (tile < 0) return;
    decode_tile<kBM, GM>(g, tile, a.E, n_tiles, e, row0, nrows, nt);
  }
  const int n0 = nt * CH_TILE;

  // ---- activation sources: load j of this wave covers rows RPI*(wave + kWaves*j) + lane/CPR (so the first loads of
  // all the waves cover the first rows); byte offset of this lane's chunk at step 0
  const uint32_t row_bytes = kMxAct ? (uint32_t)a.Kd / 2u : (uint32_t)a.Kd * 2u;
  uint32_t a_off[A_INSTR];
  auto src_row = [&](int r) {
    const int rr = row0 + (r < nrows ? r : 0);
    return (uint32_t)(a.sorted_slots ? a.sorted_slots[rr] / a.topk : rr);
  };
#pragma unroll
  for (int j = 0; j < A_INSTR; ++j) {
    const int r = RPI * (wave + kWaves * j) + lane / CPR;
    const int chunk = (lane % CPR) ^ (r % CPR);
    a_off[j] = src_row(r) * row_bytes + (uint32_t)(chunk * 16);
  }
  // The second block of the last step of an odd number of blocks re-reads the first one: 64 bytes back for the lanes
  // whose chunk lies in it (a load covers whole swizzle periods, so the chunk is the same for every load).
  const uint32_t second = KB == 2 && (((lane % CPR) ^ (lane / CPR % CPR)) & 4) ? 64u : 0u;
  auto step_off = [&](int step) {
    uint32_t off = (uint32_t)step * ROWB;
    if constexpr (KB == 2) off -= second & (2 * step + 1 >= n ? ~0u : 0u);
    return off;
  };
  // byte offsets of the scales of rows lane and 64 + lane
  uint32_t s_off[2] = {0, 0};
  if constexpr (kMxAct) {
    s_off[0] = src_row(lane) * (uint32_t)(n * 4);
    if constexpr (kBM > 64) s_off[1] = src_row(64 + lane) * (uint32_t)(n * 4);
  }

  // ---- weight sources: this lane's 16 bytes of block 0 of each channel block, and the row group's scales
  const uint8_t* b_ptr[NB];
  const uint8_t* s_ptr[NB];
  int ch_of[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int ch = n0 + wave * (HALF * 16) + (j % HALF) * 16;
    ch_of[j] = ch;
    const long block = (((long)e * N + (ch < N ? ch : 0)) >> 4) * n;
    b_ptr[j] = (NMAT == 2 && j >= HALF ? a.w1 : a.w0) + block * 1024;
    s_ptr[j] = (NMAT == 2 && j >= HALF ? a.s1 : a.s0) + block * 64;
  }

  const int nsteps = (n + KB - 1) / KB;
  // the first MBV row blocks of a step
  auto issue_a = [&](int step, int buf, auto mbc) {
    constexpr int LOADS = decltype(mbc)::value * 16 / RPI / kWaves;
    const uint32_t off = step_off(min(step, nsteps - 1));
#pragma unroll
    for (int j = 0; j < LOADS; ++j)
      dma16(a.a, a_off[j] + off, lds_addr(&As[buf][0]) + (wave + kWaves * j) * 1024);
  };
  // wave w copies the row scales of block w of the group (past the row's end: of its last block)
  auto issue_s = [&](int group, int buf) {
    if constexpr (kMxAct) {
      const uint32_t blk = (uint32_t)min(group * kMxGroup + wave, n - 1);
      dma4(a.a_s, s_off[0] + blk * 4u, lds_addr(&Ss[buf][wave * kBM]));
      if constexpr (kBM > 64) dma4(a.a_s, s_off[1] + blk * 4u, lds_addr(&Ss[buf][wave * kBM + 64]));
    }
  };
  auto load_b = [&](int step, uint4 (&b)[NB][KB]) {
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int k = 0; k < KB; ++k) {
        const uint8_t* p = b_ptr[j] + (long)min(step * KB + k, n - 1) * 1024;   // uniform
        b[j][k] = *reinterpret_cast<const uint4*>(p + 16u * (uint32_t)lane);
      }
  };
  auto load_sb = [&](int group, uint32_t (&s)[NB]) {
    const int m = min(kMxGroup, n - group * kMxGroup);
    if (m <= 0) return;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const uint8_t* p = s_ptr[j] + (long)group * 256;
      if (m == kMxGroup) {
        s[j] = *reinterpret_cast<const uint32_t*>(p + 4 * lane);
      } else {
        uint32_t v = 0;
        for (int q = 0; q < m; ++q) v |= (uint32_t)p[m * lane + q] << (8 * q);
        s[j] = v;
      }
    }
  };

  f32x4 acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int mb_valid = (nrows + 15) / 16;
  auto main_loop = [&](auto mbc) {
    constexpr int MBV = decltype(mbc)::value;      // row blocks loaded and computed
    static_assert(MBV * 16 % (RPI * kWaves) == 0, "whole loads");
    uint4 b[2][NB][KB];
    uint32_t sb[NB], sb_next[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) sb[j] = sb_next[j] = 0;
    issue_s(0, 0);
    issue_a(0, 0, mbc);
    load_b(0, b[0]);
    load_sb(0, sb_next);
    // one 128-column block of a step: J is its place in the scale group
    auto block = [&](auto jc, int buf, int gbuf, const uint4 (&w)[NB][KB]) {
      constexpr int J = decltype(jc)::value;
      constexpr int K = J % KB;
      if constexpr (kMxAct) {
        // two row blocks at a time: more fragments at once would spill
        constexpr int HB = 2;
#pragma unroll
        for (int h = 0; h < MBV; h += HB) {
          uint4 xf[HB];
          uint32_t xs[HB];
#pragma unroll
          for (int i = 0; i < HB; ++i) {
            const int r = (h + i) * 16 + li;
            xf[i] = *reinterpret_cast<const uint4*>(&As[buf][r * ROWB + (((4 * K + lg) ^ (r % CPR)) * 16)]);
            xs[i] = reinterpret_cast<const uint8_t*>(&Ss[gbuf][J * kBM + r])[lg];
          }
#pragma unroll
          for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int i = 0; i < HB; ++i) acc[h + i][j] = mfma_mx<J, 0>(w[j][K], xf[i], acc[h + i][j], sb[j], xs[i]);
        }
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          bf16x8 xf[MBV];
#pragma unroll
          for (int i = 0; i < MBV; ++i) {
            const int r = i * 16 + li;
            xf[i] = *reinterpret_cast<const bf16x8*>(&As[buf][r * ROWB + (((4 * lg + q) ^ (r % CPR)) * 16)]);
          }
#pragma unroll
          for (int j = 0; j < NB; ++j) {
            const uint32_t c = q == 0 ? w[j][0].x : q == 1 ? w[j][0].y : q == 2 ? w[j][0].z : w[j][0].w;
            const bf16x8 wf = mx_bf16x8(c, mx_scale_of<J>(sb[j]));
#pragma unroll
            for (int i = 0; i < MBV; ++i) acc[i][j] = mfma_bf16(wf, xf[i], acc[i][j]);
          }
        }
      }
    };
    auto step = [&](auto sc, int group) {
      constexpr int S = decltype(sc)::value;       // step within the group
      const int st = group * SPG + S;
      if (st >= nsteps) return;
      // This step's loads have landed and every wave is past the buffers that
      // the next ones overwrite. (Weights requested two steps ahead, left in
      // flight here: no faster, a step waits for its activations.)
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));
      __builtin_amdgcn_s_barrier();
      if constexpr (S == 0) {
#pragma unroll
        for (int j = 0; j < NB; ++j) sb[j] = sb_next[j];
        issue_s(group + 1, (group + 1) & 1);
        load_sb(group + 1, sb_next);
      }
      issue_a(st + 1, (S + 1) & 1, mbc);
      load_b(st + 1, b[(S + 1) & 1]);
      if constexpr (KB == 2) {
        block(int_constant<2 * S>{}, S & 1, group & 1, b[S & 1]);
        if (2 * st + 1 < n) block(int_constant<2 * S + 1>{}, S & 1, group & 1, b[S & 1]);
      } else {
        block(int_constant<S>{}, S & 1, group & 1, b[S & 1]);
      }
    };
    const int ngroups = (nsteps + SPG - 1) / SPG;
    for (int g = 0; g < ngroups; ++g) {
      step(int_constant<0>{}, g);
      step(int_constant<1>{}, g);
      if constexpr (SPG == 4) {
        step(int_constant<2>{}, g);
        step(int_constant<3>{}, g);
      }
    }
  };
  // a segment's last tile skips the row blocks it does not have, in steps of two
  switch ((mb_valid + 1) / 2) {
    case 1: main_loop(int_constant<2>{}); break;
    case 2: main_loop(int_constant<MB < 4 ? MB : 4>{}); break;
    case 3: main_loop(int_constant<MB < 6 ? MB : 6>{}); break;
    default: main_loop(int_constant<MB>{}); break;
  }
  // no load may still be writing this workgroup's LDS when the waves exit
  __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));

#pragma unroll
  for (int i = 0; i < MB; ++i) {
    const int r = i * 16 + li;
    if (r >= nrows) continue;
#pragma unroll
    for (int j = 0; j < HALF; ++j) {
      if (ch_of[j] >= N) continue;
      f32x4 v[NMAT];
      v[0] = acc[i][j];
      if constexpr (NMAT == 2) v[1] = acc[i][j + HALF];
      mx_store4<kOutBf16, NMAT>(a.out, (long)(row0 + r) * N + ch_of[j] + 4 * lg, v);
    }
  }
}

__global__ void zero_words_kernel(unsigned long long* __restrict__ claims) {
  if (threadIdx.x < kXcds) claims[threadIdx.x] = 0ull;
}

// Channel tiles of a row of tiles `channels` wide, and the most tiles that any
// segments make.
int tile_columns(const MxArgs& a, int channels) {
  const int ch = a.w1 ? channels / 2 : channels;
  return (a.N + ch - 1) / ch;
}
long tile_bound(const MxArgs& a, int rows, int channels) {
  return ((long)(a.S + rows - 1) / rows + a.E) * tile_columns(a, channels);
}

// Tile of a pass, in rows x channels: the rows from the rows an expert has on
// average, the channels from the tiles that makes (a tile of 128 x 256 runs
// twice a CU, one of 64 x 256 three times, the small ones three or four).
// Measured, in us (d, f as the pass's shape says; E = 16 unless stated):
//   gate/up, d 4096, f 14336: 64x256 / 128x256 / 64x128 at 32 rows an expert 204 / 222 / 218,
//     at 64 287 / 283 / 311, at 128 446 / 482 / 491, at 256 795 / 799 / 965, at 1024 2790 /
//     2669 / 3190; d 2048, f 1408, E 64, 17 rows 40 / 52 / 46; d 2048, f 2816, 512 rows
//     194 / 164 / 235; few tiles (d 896, f 4224, E 10, 36 rows) 20.8 / 25.2 / 19.9;
//   down, f 14336, d 4096: 64x256 / 128x256 / 64x128 / 128x128 at 32 rows 164 / 163 / 134 / 134,
//     at 64 194 / 190 / 183 / 170, at 128 251 / 305 / 282 / 320, at 512 763 / 774 / 847 / 888,
//     at 1024 1443 / 1443 / 1601 / 1718; f 2816, d 2048, 2048 rows 328 / 323 / 367 / 384;
//   MXFP4 activations, SwiGLU, d 4096, f 14336: 128x256 / 128x128 at 16 rows 184 / 174, at 64
//     198 / 194, at 128 253 / 279; few tiles (d 4480, f 1280, E 4, 640 rows) 29.2 / 21.7.
void pick_tile(const MxArgs& a, MxTilePlan& p) {
  const long S = a.S, E = a.E;
  // tiles of `rows` x `channels` if the rows spread evenly
  auto tiles = [&](int rows, int channels) {
    const long per_expert = S <= E * rows / 2 ? 2 : 2 * S / (E * rows) + 1;   // halves of a row tile, at least one tile
    return E * per_expert / 2 * tile_columns(a, channels);
  };
  auto tile = [&](int rows, int channels) {
    p.rows = rows;
    p.channels = channels;
  };
  if (a.a_s) return tile(128, S <= 64 * E || tiles(128, 256) < 512 ? 128 : 256);
  if (a.w1) return S > 160 * E ? tile(128, 256) : tile(64, tiles(64, 256) < 400 ? 128 : 256);
  // most experts fit 128 rows and not 64
  if (S > 48 * E && S <= 96 * E) return tile(128, tiles(128, 256) < 512 ? 128 : 256);
  return S > 512 * E ? tile(128, 256) : tile(64, tiles(64, 256) < 512 ? 128 : 256);
}

template <bool kMxAct, int NMAT, bool kOutBf16, int kBM, int kBN>
hipError_t launch_tile(MxArgs a, const MxTilePlan& p, hipStream_t stream) {
  // row tiles of an expert that take a channel tile together
  constexpr int GM = (NMAT == 2 || kMxAct) ? 8 : 4;
  const int n_tiles = tile_columns(a, kBN);
  const long per_xcd = (tile_bound(a, kBM, kBN) + kXcds - 1) / kXcds;
  long blocks = kXcds * per_xcd;
  if (!p.claims) a.claims = nullptr;
  if (a.claims) {
    // the static blocks of the longest queue, then one and a half times its tail
    blocks = kXcds * (per_xcd + min(per_xcd, (long)kClaimTail) / 2);
    hipLaunchKernelGGL(zero_words_kernel, dim3(1), dim3(kWave), 0, stream, a.claims);
  }
  hipLaunchKernelGGL((mx_tiled_kernel<kMxAct, NMAT, kOutBf16, GM, kBM, kBN>), dim3((unsigned)blocks), dim3(kWaves * kWave),
                     0, stream, a, n_tiles);
  return hipGetLastError();
}

template <bool kMxAct, int NMAT, bool kOutBf16>
hipError_t launch_tiled(const MxArgs& a, hipStream_t stream) {
  const MxTilePlan p = mx_tile_plan(a);
  const bool wide = p.channels == 256;
  if (p.rows == 128) {
    if (wide) return launch_tile<kMxAct, NMAT, kOutBf16, 128, 256>(a, p, stream);
    if constexpr (kMxAct || NMAT == 1) return launch_tile<kMxAct, NMAT, kOutBf16, 128, 128>(a, p, stream);
  } else if constexpr (!kMxAct) {
    return wide ? launch_tile<kMxAct, NMAT, kOutBf16, 64, 256>(a, p, stream)
                : launch_tile<kMxAct, NMAT, kOutBf16, 64, 128>(a, p, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace

bool mx_tiled_offsets_fit(long rows, int cols, bool mx) {
  return (uint64_t)rows * (uint64_t)cols * (mx ? 1 : 4) < (1ull << 33);
}

MxTilePlan mx_tile_plan(const MxArgs& a) {
  MxTilePlan p;
  pick_tile(a, p);
  // The claimed tail costs a launch (3 us) and an atomic in every block past the
  // static ones, of which there are many if the tile count's bound is loose; it
  // balances the XCDs over many rounds of long tiles. So: many tiles, several row
  // tiles an expert, a long reduction. (gate/up of 325 tokens, d 384, f 10496, E 9,
  // K 4, on 128x128 tiles: 181 us with it.)
  p.claims = a.claims && tile_bound(a, p.rows, p.channels) >= 2048 && a.S >= 4L * p.rows * a.E && a.Kd >= 2048;
  return p;
}

hipError_t launch_mx_tiled(const MxArgs& a, hipStream_t stream) {
  if (a.a_s) {
    if (a.w1) return a.out_bf16 ? launch_tiled<true, 2, true>(a, stream) : launch_tiled<true, 2, false>(a, stream);
    return a.out_bf16 ? launch_tiled<true, 1, true>(a, stream) : launch_tiled<true, 1, false>(a, stream);
  }
  if (a.w1) return a.out_bf16 ? launch_tiled<false, 2, true>(a, stream) : hipErrorInvalidValue;
  return a.out_bf16 ? hipErrorInvalidValue : launch_tiled<false, 1, false>(a, stream);
}

}  // namespace moe
