// Products of int8 weights and int8 rows with few rows per expert (decode): the
// weights are streamed from HBM once.
//
//   out[r, n] = a_s[row(r)] * w_s[n] * sum_k a_q[row(r), k] * w_q[n, k],   or   silu(p0) * p1
//
// for the rows r of every expert's segment. A workgroup owns one (expert, 16*NG output
// channels) item and takes 16*RB rows a pass, with the channels as MFMA rows and
// the tokens as MFMA columns. Per 64-wide step it reads one 1 KiB block per 16
// channels and matrix (16 bytes a lane) and 16 bytes a lane of the rows, U steps
// at a time: the rows of these steps are requested, then the weights of the next
// ones, then the steps are computed (loads return in order, so waiting for the
// rows does not wait for the weights behind them).
// Items are numbered over the experts that have rows. The reduction is cut
// into KS slices, streamed by the KS waves of the workgroup and added through
// LDS (integers: exact in any order). Where a tiled product would have
// fewer tiles than CUs the passes are spread over workgroups, whose weights come from the
// caches then (one expert, 450 rows, d 8960, f 896: 28 us, tiles 48).
// Bound by HBM: gate/up of one token (d 4096, f 14336, two experts) 39 us, 6.0
// TB/s; down of 64 tokens (d 24576, f 8192, E 16) 490 us, 6.6 TB/s.
#include "i8_common.h"
#include "kernels.h"

namespace moe {

namespace {

template <int NMAT, bool kOutBf16, int NG, int RB, int KS, int U>
__global__ __launch_bounds__(KS * kWave) void i8_stream_kernel(I8Args a) {
  static_assert(KS > 1, "the slices are added through LDS");
  __shared__ i32x4 red[KS - 1][NG][NMAT][kWave];
  const int lane = threadIdx.x & 63;
  const int kslice = threadIdx.x >> 6;
  const int li = lane & 15;
  const int lg = lane >> 4;
  const int N = a.N, n = a.Kd / kI8Step;      // steps of a row

  const int gpe = N / (16 * NG);
  const int te = blockIdx.x / gpe;
  const int grp = blockIdx.x - te * gpe;
  int e, row0, nrows;
  // the workgroup is one item, so all its waves return here together
  if (!find_touched_expert(a.offsets, a.E, te, e, row0, nrows)) return;
  const int ch_base = grp * 16 * NG;

  const int8_t* wp[NG][NMAT];
#pragma unroll
  for (int ng = 0; ng < NG; ++ng) {
    const long block = (((long)e * N + ch_base + ng * 16) >> 4) * n;
    wp[ng][0] = a.w0 + block * 1024 + 16 * lane;
    if constexpr (NMAT == 2) wp[ng][1] = a.w1 + block * 1024 + 16 * lane;
  }
  const int s_begin = (int)((long)kslice * n / KS), s_end = (int)((long)(kslice + 1) * n / KS);

  uint4 w[2][U][NG][NMAT];
  auto load_w = [&](int s, uint4 (&wb)[U][NG][NMAT]) {
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (s + j < s_end)
#pragma unroll
        for (int ng = 0; ng < NG; ++ng)
#pragma unroll
          for (int m = 0; m < NMAT; ++m) wb[j][ng][m] = load_nt16(wp[ng][m] + (long)(s + j) * 1024);
  };

  for (int p0 = blockIdx.y * 16 * RB; p0 < nrows; p0 += gridDim.y * 16 * RB) {
    const int nrb = min(RB, (nrows - p0 + 15) >> 4);
    // the first weights are requested before the row numbers are looked up
    load_w(s_begin, w[0]);
    const int8_t* ap[RB];
    long src[RB];
    bool aok[RB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      const int r = p0 + rb * 16 + li;
      aok[rb] = r < nrows;
      src[rb] = 0;
      if (aok[rb]) src[rb] = a.sorted_slots ? a.sorted_slots[row0 + r] / a.topk : row0 + r;
      ap[rb] = a.a + src[rb] * a.Kd + 16 * lg;
    }
    i32x4 acc[RB][NG][NMAT];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
      for (int ng = 0; ng < NG; ++ng)
#pragma unroll
        for (int m = 0; m < NMAT; ++m) acc[rb][ng][m] = i32x4{0, 0, 0, 0};

    auto run = [&](auto nrbc) {
      constexpr int NRB = decltype(nrbc)::value;   // row blocks present
      auto unit = [&](int s, const uint4 (&wb)[U][NG][NMAT], uint4 (&wn)[U][NG][NMAT]) {
        uint4 av[U][NRB];
#pragma unroll
        for (int j = 0; j < U; ++j)
#pragma unroll
          for (int rb = 0; rb < NRB; ++rb) {
            av[j][rb] = make_uint4(0, 0, 0, 0);
            if (s + j < s_end && aok[rb]) av[j][rb] = *reinterpret_cast<const uint4*>(ap[rb] + (long)(s + j) * kI8Step);
          }
        load_w(s + U, wn);
#pragma unroll
        for (int j = 0; j < U; ++j) {
          if (s + j >= s_end) break;
#pragma unroll
          for (int ng = 0; ng < NG; ++ng)
#pragma unroll
            for (int m = 0; m < NMAT; ++m)
#pragma unroll
              for (int rb = 0; rb < NRB; ++rb)
                acc[rb][ng][m] = mfma_i8(as_i32x4(wb[j][ng][m]), as_i32x4(av[j][rb]), acc[rb][ng][m]);
        }
      };
      for (int s = s_begin; s < s_end; s += 2 * U) {
        unit(s, w[0], w[1]);
        if (s + U < s_end) unit(s + U, w[1], w[0]);
      }
    };
    if (RB == 1 || nrb == 1) {
      run(int_constant<1>{});
    } else {
      run(int_constant<RB>{});
    }

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
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      const int r = p0 + rb * 16 + li;
      if (rb >= nrb || r >= nrows) continue;
      const float as = a.a_s[src[rb]];
#pragma unroll
      for (int ng = 0; ng < NG; ++ng) {
        const int ch = ch_base + ng * 16 + 4 * lg;
        float4 ws[NMAT];
        ws[0] = i8_scale4(a.s0, a.scale_bf16, (long)e * N + ch);
        if constexpr (NMAT == 2) ws[1] = i8_scale4(a.s1, a.scale_bf16, (long)e * N + ch);
        i8_store4<NMAT, kOutBf16>(a.out, (long)(row0 + r) * N + ch, acc[rb][ng], ws, as);
      }
    }
  }
}

// Items of 16*NG channels over the experts that can have rows (each has one of
// the S at least).
long stream_items(const I8Args& a, int NG) { return (long)min(a.E, a.S) * (a.N / (16 * NG)); }

template <int NMAT, bool kOutBf16, int NG, int RB, int KS, int U>
hipError_t launch(const I8Args& a, hipStream_t stream) {
  const long items = stream_items(a, NG);
  // the rows of an expert are known on the device alone: workgroups past its last pass return. Many rows come here if the call
  // asks for it, or gathered past 4 GiB: then fewer items than CUs share out their passes (66001 gathered rows of 65536, E 3,
  // f 64: 53.4 -> 1.9 ms).
  const int most = (a.S + 16 * RB - 1) / (16 * RB);
  const int passes = i8_few_tiles(a) ? min(16, most) : items < 256 ? min((int)(256 / items), most) : 1;
  hipLaunchKernelGGL((i8_stream_kernel<NMAT, kOutBf16, NG, RB, KS, U>),
                     dim3((unsigned)items, passes), dim3(KS * kWave), 0, stream, a);
  return hipGetLastError();
}

template <int NMAT, bool kOutBf16>
hipError_t launch_rows(const I8Args& a, hipStream_t stream) {
  switch (i8_stream_plan(a).rows) {
    case 16: return launch<NMAT, kOutBf16, 1, 1, 4, 4>(a, stream);
    case 32: return launch<NMAT, kOutBf16, 2, 2, 2, 4>(a, stream);
    default: return launch<NMAT, kOutBf16, 2, 4, 4, 2>(a, stream);
  }
}

}  // namespace

// Rows a pass, channels of an item, slices. Measured, us, weights that no cache
// holds (16r: 16 rows, 16 channels, 4 slices of 4 steps at a time; 32r: 32, 32, 2 of 4; 64r: 64, 32, 4 of 2):
//   gate/up, d 4096, f 14336, E 16: 2 slots 39 / 43 / 51, 32 slots 255 / 261 / 292, 128 slots
//     323 / 312 / 343; down, d 24576, f 8192, E 16, 128 slots 573 / 595 / 582;
//   one expert: 4 rows, d 24576, f 8192 39 / 55 / 49; 16 rows, gate/up, d 8192, f 24576 78 / 88 / 90; 64 rows, d 24576, f 8192
//     173 / 124 / 69 (128-row tiles: 150).
// More rows a pass cost registers, hence waves; an expert with more rows than a pass streams its weights again.
I8StreamPlan i8_stream_plan(const I8Args& a) {
  const long few = (long)min(a.E, a.S) * a.N / 32 < 2048;   // fewer 32-channel items than two waves a SIMD
  if (a.S <= (few ? 8L : 4L) * a.E) return {16, 16, 4};
  return a.S <= 8L * a.E ? I8StreamPlan{32, 32, 2} : I8StreamPlan{32, 64, 4};
}

long i8_stream_passes(const I8Args& a) {
  const long experts = min(a.E, a.S), rows = (a.S + experts - 1) / experts;
  return stream_items(a, 2) * ((rows + 63) / 64);
}

hipError_t launch_i8_stream(const I8Args& a, hipStream_t stream) {
  if (a.w1) return a.out_bf16 ? launch_rows<2, true>(a, stream) : launch_rows<2, false>(a, stream);
  return a.out_bf16 ? launch_rows<1, true>(a, stream) : launch_rows<1, false>(a, stream);
}

}  // namespace moe
