// Products of MXFP4 weights with few rows per expert (decode): the weights are
// streamed from HBM once.
//
//   out[r, n] = sum_k A[row(r), k] * W_e[n, k],   or   silu(W0 . a) * (W1 . a)
//
// for the rows r of every expert's segment; A is bf16 (the expert FFN's passes)
// or MXFP4 itself. A wave owns one (expert, 16*NG output channels) item and
// takes 16*RB rows a pass, with the channels as MFMA rows and the tokens as
// MFMA columns. Per 128-wide step it reads one 1 KiB block per 16 channels and
// matrix (16 bytes a lane: one scale group) and, every fourth step, one dword
// of scales a lane.
//   bf16 activations: the codes become bf16 in registers, exactly, scale
//     included, and feed four 16x16x32 bf16 MFMAs: lane group l/16 pairs its
//     columns 32*(l/16) + 8*i .. +8 with the same columns of its token's row;
//   MXFP4 activations: one 16x16x128 scaled MFMA takes both operands as read.
// Items are numbered over the experts that have rows. Sums are fp32; with few
// items the reduction is cut into KS slices of whole scale groups, streamed by
// the KS waves of a workgroup and added through LDS in ascending order.
// Bound by HBM: down of 64 tokens (d 8192, f 24576, E 16) 283 us, 6080 GB/s of codes,
// scales and rows; gate/up of one token (d 4096, f 14336, two experts) 23.2 us, 5370
// GB/s, start and end of the launch included; the MXFP4 product of 17 tokens 68.5 us.
#include "kernels.h"
#include "mx_common.h"

namespace moe {

namespace {

constexpr int kStreamWaves = 4;
constexpr int block_waves(int KS) { return KS > 1 ? KS : kStreamWaves; }

__device__ __forceinline__ uint32_t load_nt4(const void* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(p));
}

// A lane's scales of the m blocks of one scale group, in the bytes of a dword.
__device__ __forceinline__ uint32_t load_scales(const uint8_t* group, int m, int lane) {
  if (m == kMxGroup) return load_nt4(group + 4 * lane);
  uint32_t v = 0;
  for (int j = 0; j < m; ++j) v |= (uint32_t)group[m * lane + j] << (8 * j);
  return v;
}

template <bool kMxAct, int NMAT, int NG, int RB, int KS, bool kOutBf16, int U>
__global__ __launch_bounds__(block_waves(KS) * kWave) void mx_stream_kernel(MxArgs a) {
  constexpr int IPW = block_waves(KS) / KS;   // items per workgroup
  constexpr int AQ = kMxAct ? 1 : 4;          // 16-byte pieces of a token's row per lane and step
  __shared__ f32x4 red[KS > 1 ? KS - 1 : 1][NG][NMAT][kWave];
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int li = lane & 15;
  const int lg = lane >> 4;
  const int N = a.N, n = a.Kd / kMxStep;      // steps of a row

  const int gpe = N / (16 * NG);
  const int item = blockIdx.x * IPW + wave / KS;
  const int kslice = wave % KS;
  const int te = item / gpe;
  const int grp = item - te * gpe;
  int e, row0, nrows;
  // KS > 1: the workgroup is one item, so all its waves return here together
  if (!find_touched_expert(a.offsets, a.E, te, e, row0, nrows)) return;
  const int ch_base = grp * 16 * NG;

  const uint8_t* wp[NG][NMAT];
  const uint8_t* sp[NG][NMAT];
#pragma unroll
  for (int ng = 0; ng < NG; ++ng) {
    const long block = (((long)e * N + ch_base + ng * 16) >> 4) * n;
    wp[ng][0] = a.w0 + block * 1024 + 16 * lane;
    sp[ng][0] = a.s0 + block * 64;
    if constexpr (NMAT == 2) {
      wp[ng][1] = a.w1 + block * 1024 + 16 * lane;
      sp[ng][1] = a.s1 + block * 64;
    }
  }
  // this wave's slice, in scale groups
  const int groups = (n + kMxGroup - 1) / kMxGroup;
  const int g0 = kslice * groups / KS, g1 = (kslice + 1) * groups / KS;

  // weights and scales of the steps in use and of the next ones
  constexpr int UPG = kMxGroup / U;   // units per scale group
  uint4 w[2][U][NG][NMAT];
  uint32_t sc[2][NG][NMAT];           // scales of the group in use, and of the next
  const int s_begin = g0 * kMxGroup, s_end = min(g1 * kMxGroup, n);
  auto load_w = [&](int s, uint4 (&wb)[U][NG][NMAT]) {
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (s + j < s_end)
#pragma unroll
        for (int ng = 0; ng < NG; ++ng)
#pragma unroll
          for (int m = 0; m < NMAT; ++m) wb[j][ng][m] = load_nt16(wp[ng][m] + (long)(s + j) * 1024);
  };
  auto load_s = [&](int s, uint32_t (&sb)[NG][NMAT]) {
    const int m4 = min(kMxGroup, n - s);
#pragma unroll
    for (int ng = 0; ng < NG; ++ng)
#pragma unroll
      for (int m = 0; m < NMAT; ++m) sb[ng][m] = load_scales(sp[ng][m] + (long)s * 64, m4, lane);
  };

  for (int p0 = 0; p0 < nrows; p0 += 16 * RB) {
    const int nrb = min(RB, (nrows - p0 + 15) >> 4);
    // the first weights are requested before the row numbers are looked up
    if (s_begin < s_end) {
      load_w(s_begin, w[0]);
      load_s(s_begin, sc[0]);
    }
    const uint8_t* ap[RB];
    const uint8_t* asp[RB];
    bool aok[RB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      const int r = p0 + rb * 16 + li;
      aok[rb] = r < nrows;
      long src = 0;
      if (aok[rb]) src = a.sorted_slots ? a.sorted_slots[row0 + r] / a.topk : row0 + r;
      if constexpr (kMxAct) {
        ap[rb] = static_cast<const uint8_t*>(a.a) + src * (a.Kd / 2) + 16 * lg;
        asp[rb] = a.a_s + src * (a.Kd / 32) + lg;
      } else {
        ap[rb] = static_cast<const uint8_t*>(a.a) + src * (long)a.Kd * 2 + 64 * lg;
      }
    }
    f32x4 acc[RB][NG][NMAT];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
      for (int ng = 0; ng < NG; ++ng)
#pragma unroll
        for (int m = 0; m < NMAT; ++m) acc[rb][ng][m] = f32x4{0.f, 0.f, 0.f, 0.f};

    // U steps at a time (U divides a scale group), NRB row blocks present: the
    // activations of these steps are requested, then the weights of the next
    // ones, then the steps are computed. Loads return in order, so waiting for
    // the activations does not wait for the weights requested behind them.
    auto run = [&](auto nrbc) {
      constexpr int NRB = decltype(nrbc)::value;
      // unit UI of the group at step s0, whose scales are sb; its weights are wb
      auto unit = [&](auto uc, int s0, const uint4 (&wb)[U][NG][NMAT], const uint32_t (&sb)[NG][NMAT],
                      uint4 (&wn)[U][NG][NMAT], uint32_t (&sn)[NG][NMAT]) {
        constexpr int UI = decltype(uc)::value;
        const int s1 = s0 + UI * U;
        if (s1 >= s_end) return;
        uint4 av[U][NRB][AQ];
        uint32_t as[U][NRB];
#pragma unroll
        for (int j = 0; j < U; ++j)
#pragma unroll
          for (int rb = 0; rb < NRB; ++rb) {
            as[j][rb] = 0;
#pragma unroll
            for (int q = 0; q < AQ; ++q) av[j][rb][q] = make_uint4(0, 0, 0, 0);
            if (s1 + j < s_end && aok[rb]) {
              const uint8_t* p = ap[rb] + (long)(s1 + j) * (kMxAct ? 64 : 256);
#pragma unroll
              for (int q = 0; q < AQ; ++q) av[j][rb][q] = *reinterpret_cast<const uint4*>(p + 16 * q);
              if constexpr (kMxAct) as[j][rb] = asp[rb][(s1 + j) * 4];
            }
          }
        load_w(s1 + U, wn);
        if constexpr (UI == UPG - 1)
          if (s1 + U < s_end) load_s(s1 + U, sn);
        auto step = [&](auto jc) {
          constexpr int j = decltype(jc)::value;
          if constexpr (j < U) {
            constexpr int J = UI * U + j;
            if (s1 + j >= s_end) return;
#pragma unroll
            for (int ng = 0; ng < NG; ++ng)
#pragma unroll
              for (int m = 0; m < NMAT; ++m) {
                if constexpr (kMxAct) {
#pragma unroll
                  for (int rb = 0; rb < NRB; ++rb)
                    acc[rb][ng][m] = mfma_mx<J, 0>(wb[j][ng][m], av[j][rb][0], acc[rb][ng][m], sb[ng][m], as[j][rb]);
                } else {
                  const float s = mx_scale_of<J>(sb[ng][m]);
                  const uint32_t c[4] = {wb[j][ng][m].x, wb[j][ng][m].y, wb[j][ng][m].z, wb[j][ng][m].w};
#pragma unroll
                  for (int q = 0; q < 4; ++q) {
                    const bf16x8 wf = mx_bf16x8(c[q], s);
#pragma unroll
                    for (int rb = 0; rb < NRB; ++rb)
                      acc[rb][ng][m] = mfma_bf16(wf, as_bf16x8(av[j][rb][q]), acc[rb][ng][m]);
                  }
                }
              }
          }
        };
        step(int_constant<0>{});
        step(int_constant<1>{});
        step(int_constant<2>{});
        step(int_constant<3>{});
      };
      auto group = [&](auto pc, int s0) {
        constexpr int G = decltype(pc)::value;   // parity of the group
        // with one unit a group, the weight buffers alternate with the groups
        unit(int_constant<0>{}, s0, w[UPG == 1 ? G : 0], sc[G], w[UPG == 1 ? 1 - G : 1], sc[1 - G]);
        if constexpr (UPG >= 2) unit(int_constant<(UPG >= 2 ? 1 : 0)>{}, s0, w[1], sc[G], w[0], sc[1 - G]);
        if constexpr (UPG >= 4) {
          unit(int_constant<(UPG >= 4 ? 2 : 0)>{}, s0, w[0], sc[G], w[1], sc[1 - G]);
          unit(int_constant<(UPG >= 4 ? 3 : 0)>{}, s0, w[1], sc[G], w[0], sc[1 - G]);
        }
      };
      for (int s0 = s_begin; s0 < s_end; s0 += 2 * kMxGroup) {
        group(int_constant<0>{}, s0);
        group(int_constant<1>{}, s0 + kMxGroup);
      }
    };
    if (RB == 1 || nrb == 1) {
      run(int_constant<1>{});
    } else {
      run(int_constant<RB>{});
    }

    if constexpr (KS > 1) {
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) {
        if (rb < nrb) {
          if (kslice > 0) {
#pragma unroll
            for (int ng = 0; ng < NG; ++ng)
#pragma unroll
              for (int m = 0; m < NMAT; ++m) red[kslice - 1][ng][m][lane] = acc[rb][ng][m];
          }
          __syncthreads();
          if (kslice == 0) {
            for (int j = 0; j < KS - 1; ++j)
#pragma unroll
              for (int ng = 0; ng < NG; ++ng)
#pragma unroll
                for (int m = 0; m < NMAT; ++m) acc[rb][ng][m] += red[j][ng][m][lane];
          }
          __syncthreads();
        }
      }
      if (kslice > 0) continue;
    }
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      const int r = p0 + rb * 16 + li;
      if (rb < nrb && r < nrows) {
        const long o = (long)(row0 + r) * N + ch_base + 4 * lg;
#pragma unroll
        for (int ng = 0; ng < NG; ++ng) mx_store4<kOutBf16, NMAT>(a.out, o + ng * 16, acc[rb][ng]);
      }
    }
  }
}

// Items of 16*NG channels over the experts that can have rows (each has one of
// the S at least).
long stream_items(const MxArgs& a, int NG) { return (long)min(a.E, a.S) * (a.N / (16 * NG)); }

// Slices of the reduction, of whole scale groups (512 columns). Few items are
// split until HBM is busy; many are split in two, which balances the end of the
// pass, as long as a slice keeps four groups; in between the waves are kept from
// a little more than one round of the GPU (some 3000).
// Measured (us) for 1, 2, 4, 8 slices (items, groups): down of one token, f 14336
// (256, 28) -, 30.4, 19.8, 15.2; the MXFP4 product of one token, d 14336 (512, 28) -, 24.2,
// 15.9, 13.0; down of 8, 32 and 100 tokens (1024, 28) 83, 53, 59, - and -, 82, 82, 92 and 156,
// 96, 103, -; gate/up of one token, d 4096 (1792, 8) -, 22.8, 25.2, 28.7; d 8192 (1536, 16) -,
// 73.8, 70.9, 77.5; down of 64, f 24576 (2048, 48) 283, 301, 279, 300; gate/up of 32, d 4096
// (7168, 8) 164, 148, -, -; the MXFP4 product of 17 (7168, 8) 73.7, 65.7, 68.7, 77.7; gate/up of
// 64, d 8192 (12288, 16) 585, 536, 543, -.
int stream_slices(long items, int groups) {
  if (items >= 1024) {
    if (items >= 1536 && items < 4096 && groups >= 16) return 4;
    return groups >= 8 ? 2 : 1;
  }
  int ks = 1;
  while (ks < 8 && 2 * ks <= groups && (items * ks < 2048 || (items * ks < 4096 && groups / (2 * ks) >= 3))) ks *= 2;
  return ks;
}

// Channels per item: wide items read the rows' activations fewer times (a wave
// reads its rows' bf16 activations from L2 for every item: down of 64 tokens, d
// 8192, 534, 351 and 279 us for 16, 32 and 64 channels), narrow ones give few
// items more waves (gate/up of one token: 25.3 us for 16 channels, 27.3 for 32;
// down of one token: 15.4 us for 32, 20.5 for 64). MXFP4 activations are a
// quarter of the bytes: 32 channels pay for one matrix with many items (64
// tokens, d 24576, f 8192: 343 us for 16 channels, 282 for 32; 17 tokens, d 4096,
// f 14336: 69.4 and 68.3). N is a multiple of 128, so every width divides it.
int stream_width(const MxArgs& a) {
  if (a.a_s) return !a.w1 && stream_items(a, 2) >= 4096 ? 2 : 1;
  if (a.w1) return stream_items(a, 2) >= 1024 ? 2 : 1;
  if (stream_items(a, 4) >= 1024) return 4;
  return stream_items(a, 2) >= 256 ? 2 : 1;
}

// The most slices that stream_slices gives items of 16*NG channels: wide ones
// are chosen for 1024 items and more, with MXFP4 activations for 4096.
constexpr int most_slices(bool mx_act, int nmat, int ng) {
  if (mx_act) return ng == 2 ? 2 : 8;
  return ng == 4 || (nmat == 2 && ng == 2) ? 4 : 8;
}

template <bool kMxAct, int NMAT, int NG, int RB, bool kOutBf16, int U>
hipError_t launch_slices(const MxArgs& a, int slices, hipStream_t stream) {
  const long items = stream_items(a, NG);
  hipError_t e = hipErrorInvalidValue;
  auto launch = [&](auto ksc) {
    constexpr int KS = decltype(ksc)::value;
    if constexpr (KS <= most_slices(kMxAct, NMAT, NG)) {
      hipLaunchKernelGGL((mx_stream_kernel<kMxAct, NMAT, NG, RB, KS, kOutBf16, U>),
                         dim3((unsigned)(KS > 1 ? items : (items + kStreamWaves - 1) / kStreamWaves)),
                         dim3(block_waves(KS) * kWave), 0, stream, a);
      e = hipGetLastError();
    }
  };
  switch (slices) {
    case 1: launch(int_constant<1>{}); break;
    case 2: launch(int_constant<2>{}); break;
    case 4: launch(int_constant<4>{}); break;
    case 8: launch(int_constant<8>{}); break;
  }
  return e;
}

template <bool kMxAct, int NMAT, int RB, bool kOutBf16>
hipError_t launch_width(const MxArgs& a, const MxStreamPlan& p, hipStream_t stream) {
  constexpr int U = RB == 1 ? 2 : 1;   // two row blocks: more steps at once would spill
  if constexpr (kMxAct) {
    if constexpr (NMAT == 1)
      if (p.channels == 32) return launch_slices<true, 1, 2, RB, kOutBf16, 2>(a, p.slices, stream);
    return launch_slices<true, NMAT, 1, RB, kOutBf16, 2>(a, p.slices, stream);
  } else if constexpr (NMAT == 2) {
    if (p.channels == 32) return launch_slices<false, 2, 2, RB, kOutBf16, U>(a, p.slices, stream);
    return launch_slices<false, 2, 1, RB, kOutBf16, 1>(a, p.slices, stream);
  } else {
    if (p.channels == 64) return launch_slices<false, 1, 4, RB, kOutBf16, U>(a, p.slices, stream);
    if (p.channels == 32) return launch_slices<false, 1, 2, RB, kOutBf16, U>(a, p.slices, stream);
    return launch_slices<false, 1, 1, RB, kOutBf16, U>(a, p.slices, stream);
  }
}

template <bool kMxAct, int NMAT, bool kOutBf16>
hipError_t launch_rows(const MxArgs& a, hipStream_t stream) {
  const MxStreamPlan p = mx_stream_plan(a);
  return p.rows == 16 ? launch_width<kMxAct, NMAT, 1, kOutBf16>(a, p, stream)
                      : launch_width<kMxAct, NMAT, 2, kOutBf16>(a, p, stream);
}

}  // namespace

MxStreamPlan mx_stream_plan(const MxArgs& a) {
  MxStreamPlan p;
  const int ng = stream_width(a);
  p.channels = 16 * ng;
  // one row block per pass for up to eight rows an expert on average (an expert
  // with more than 16 streams its weights again), else two
  p.rows = a.S <= 8L * a.E ? 16 : 32;
  p.slices = stream_slices(stream_items(a, ng), (a.Kd / kMxStep + kMxGroup - 1) / kMxGroup);
  return p;
}

hipError_t launch_mx_stream(const MxArgs& a, hipStream_t stream) {
  if (a.a_s) {
    if (a.w1) return a.out_bf16 ? launch_rows<true, 2, true>(a, stream) : launch_rows<true, 2, false>(a, stream);
    return a.out_bf16 ? launch_rows<true, 1, true>(a, stream) : launch_rows<true, 1, false>(a, stream);
  }
  // bf16 activations: the expert FFN's gate/up (bf16 h) and down (fp32 rows) passes
  if (a.w1) return a.out_bf16 ? launch_rows<false, 2, true>(a, stream) : hipErrorInvalidValue;
  return a.out_bf16 ? hipErrorInvalidValue : launch_rows<false, 1, false>(a, stream);
}

}  // namespace moe
