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

template <bool kMxAct, int NMAT, int NG, int RB, int KS, bool kOutBf16>
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

  for (int p0 = 0; p0 < nrows; p0 += 16 * RB) {
    const int nrb = min(RB, (nrows - p0 + 15) >> 4);
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

    for (int g = g0; g < g1; ++g) {
      const int s0 = g * kMxGroup;
      const int m4 = min(kMxGroup, n - s0);
      uint4 w[kMxGroup][NG][NMAT];
      uint32_t sc[NG][NMAT];
#pragma unroll
      for (int ng = 0; ng < NG; ++ng)
#pragma unroll
        for (int m = 0; m < NMAT; ++m) {
          sc[ng][m] = load_scales(sp[ng][m] + s0 * 64, m4, lane);
#pragma unroll
          for (int j = 0; j < kMxGroup; ++j)
            if (j < m4) w[j][ng][m] = load_nt16(wp[ng][m] + (long)(s0 + j) * 1024);
        }
      auto step = [&](auto jc) {
        constexpr int j = decltype(jc)::value;
        if (j >= m4) return;
        uint4 av[RB][AQ];
        uint32_t as[RB];
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
          as[rb] = 0;
#pragma unroll
          for (int q = 0; q < AQ; ++q) av[rb][q] = make_uint4(0, 0, 0, 0);
          if (rb < nrb && aok[rb]) {
            const uint8_t* p = ap[rb] + (long)(s0 + j) * (kMxAct ? 64 : 256);
#pragma unroll
            for (int q = 0; q < AQ; ++q) av[rb][q] = *reinterpret_cast<const uint4*>(p + 16 * q);
            if constexpr (kMxAct) as[rb] = asp[rb][(s0 + j) * 4];
          }
        }
#pragma unroll
        for (int ng = 0; ng < NG; ++ng)
#pragma unroll
          for (int m = 0; m < NMAT; ++m) {
            if constexpr (kMxAct) {
#pragma unroll
              for (int rb = 0; rb < RB; ++rb)
                if (rb < nrb) acc[rb][ng][m] = mfma_mx<j, 0>(w[j][ng][m], av[rb][0], acc[rb][ng][m], sc[ng][m], as[rb]);
            } else {
              const float s = mx_scale_of<j>(sc[ng][m]);
              const uint32_t c[4] = {w[j][ng][m].x, w[j][ng][m].y, w[j][ng][m].z, w[j][ng][m].w};
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const bf16x8 wf = mx_bf16x8(c[q], s);
#pragma unroll
                for (int rb = 0; rb < RB; ++rb)
                  if (rb < nrb) acc[rb][ng][m] = mfma_bf16(wf, as_bf16x8(av[rb][q]), acc[rb][ng][m]);
              }
            }
          }
      };
      step(int_constant<0>{});
      step(int_constant<1>{});
      step(int_constant<2>{});
      step(int_constant<3>{});
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

template <bool kMxAct, int NMAT, int NG, int RB, bool kOutBf16>
hipError_t launch_ks(const MxArgs& a, hipStream_t stream) {
  const long items = (long)min(a.E, a.S) * (a.N / (16 * NG));   // an expert with rows has one of the S at least
  const int groups = (a.Kd / kMxStep + kMxGroup - 1) / kMxGroup;
  int ks = 1;
  while (ks < 8 && items * ks < 8192 && 2 * ks <= groups) ks *= 2;
#define MOE_MX_STREAM(KS)                                                                                       \
  hipLaunchKernelGGL((mx_stream_kernel<kMxAct, NMAT, NG, RB, KS, kOutBf16>),                                    \
                     dim3((unsigned)(KS > 1 ? items : (items + kStreamWaves - 1) / kStreamWaves)),              \
                     dim3(block_waves(KS) * kWave), 0, stream, a)
  switch (ks) {
    case 1: MOE_MX_STREAM(1); break;
    case 2: MOE_MX_STREAM(2); break;
    case 4: MOE_MX_STREAM(4); break;
    default: MOE_MX_STREAM(8); break;
  }
#undef MOE_MX_STREAM
  return hipGetLastError();
}

template <bool kMxAct, int NMAT, bool kOutBf16>
hipError_t launch_rb(const MxArgs& a, hipStream_t stream) {
  return launch_ks<kMxAct, NMAT, 1, 2, kOutBf16>(a, stream);
}

}  // namespace

hipError_t launch_mx_stream(const MxArgs& a, hipStream_t stream) {
  if (a.a_s) {
    if (a.w1) return a.out_bf16 ? launch_rb<true, 2, true>(a, stream) : launch_rb<true, 2, false>(a, stream);
    return a.out_bf16 ? launch_rb<true, 1, true>(a, stream) : launch_rb<true, 1, false>(a, stream);
  }
  // bf16 activations: the expert FFN's gate/up (bf16 h) and down (fp32 rows) passes
  if (a.w1) return a.out_bf16 ? launch_rb<false, 2, true>(a, stream) : hipErrorInvalidValue;
  return a.out_bf16 ? hipErrorInvalidValue : launch_rb<false, 1, false>(a, stream);
}

}  // namespace moe
