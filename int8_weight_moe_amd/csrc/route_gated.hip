// Gated routing: scores of a router's logits, groups of experts, top K.
//
//   l_e = x . router_w[e] (+ router_bias[e]);  s = softmax(l) or sigmoid(l)
//   c_e = s_e + select_bias[e], the value that decides the choice
//   groups: the group_topk of G groups of E/G consecutive experts with the
//     largest value (largest c, or the sum of the two largest)
//   the K experts of them with the largest c, descending; ties, here and among
//     groups, go to the lower index; -inf and NaN are never taken
//   w_k = s_k (/ their sum) * scale
//
// Logits: MFMA tiles of tokens x experts, the hidden dimension split over the
// waves of a workgroup. The sums of 32 products that an MFMA (fp32 inputs: eight)
// makes are added in fp64, so a logit is off by at most
//     delta = kMfmaUnits * 2^-23 * |x| |w_e|
// (the MFMA: see there; sum |x_i w_i| <= |x| |w_e|). |x|^2 and |w_e|^2 are taken
// on the way.
// Choice: one wave a token, first in fp32 with an error bound eps_e on every c_e
// (delta through the score's derivative, the evaluation, the bias's rounding). A
// decision between two values whose intervals overlap is not taken: the experts it
// hangs on are marked, the workgroup's waves compute their logits again in fp64, and the
// choice is repeated in fp64, until no decision hangs on an unrefined logit. So
// the ids are those of 64-bit values, at the price of fp32 ones.
#include "device_common.h"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kMaxExperts = 256;

// What an MFMA's sum of 32 products (a chain of eight fp32 ones) is taken to be off
// by, in 2^-23 of the sum of their magnitudes. Measured over random and one-sided sums
// with 24 bits between the terms: 2.3 at most.
constexpr float kMfmaUnits = 8.f;
constexpr float kUnit = 0x1p-23f;

__device__ __forceinline__ void load8d(const __bf16* p, double (&v)[8]) {
  const u32x4 u = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8d(const float* p, double (&v)[8]) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = a[i];
    v[4 + i] = b[i];
  }
}

// ---- reductions over a wave; the same value in every lane
template <int kCtrl, int kRows>
__device__ __forceinline__ float dpp_or(float v, float otherwise) {
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(otherwise), __float_as_int(v), kCtrl, kRows, 0xf, false));
}
__device__ __forceinline__ float wave_max(float v) {
  // shifts within a row of 16 by 1, 2, 4, 8, then rows 0 and 2 into 1 and 3, then row 1 into 2 and 3: lane 63 has all
  v = fmaxf(v, dpp_or<0x111, 0xf>(v, -INFINITY));
  v = fmaxf(v, dpp_or<0x112, 0xf>(v, -INFINITY));
  v = fmaxf(v, dpp_or<0x114, 0xf>(v, -INFINITY));
  v = fmaxf(v, dpp_or<0x118, 0xf>(v, -INFINITY));
  v = fmaxf(v, dpp_or<0x142, 0xa>(v, -INFINITY));
  v = fmaxf(v, dpp_or<0x143, 0xc>(v, -INFINITY));
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = fmax(v, __shfl_xor(v, off));
  return v;
}
template <typename Real>
__device__ __forceinline__ Real wave_sum(Real v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  return v;
}
__device__ __forceinline__ int wave_min(int v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = min(v, __shfl_xor(v, off));
  return v;
}

// a . b over d elements by one wave, in fp64; the same value in every lane.
template <typename Act>
__device__ __forceinline__ double dot64(const Act* __restrict__ a, const Act* __restrict__ b, int d) {
  double s = 0;
  for (int c = 8 * (threadIdx.x & 63); c < d; c += 8 * kWave) {
    double u[8], v[8];
    load8d(a + c, u);
    load8d(b + c, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fma(u[i], v[i], s);
  }
  return wave_sum(s);
}

__device__ __forceinline__ float exp_of(float v) { return expf(v); }
__device__ __forceinline__ double exp_of(double v) { return exp(v); }

// Largest and second largest of a lane's values and those of the lanes of its group (lanes_per_group consecutive ones).
template <typename Real>
struct Top2 {
  Real first = -INFINITY, second = -INFINITY;
  __device__ void add(Real v) {
    second = fmax(second, fmin(first, v));
    first = fmax(first, v);
  }
  __device__ void join(int lanes) {
    for (int off = 1; off < lanes; off <<= 1) {
      const Real f = __shfl_xor(first, off), s = __shfl_xor(second, off);
      second = fmax(fmin(first, f), fmax(second, s));
      first = fmax(first, f);
    }
  }
};

// A workgroup's tokens between their logits and their choice, in LDS.
struct TokenState {
  double* logit;       // [tokens][stride]
  float* x_norm;       // [tokens]  |x|, rounded up
  float* w_norm;       // [stride]  |w_e|, rounded up
  uint32_t* refined;   // [tokens][8] bit e: the logit is a 64-bit one
  uint16_t* work;      // (token << 8 | expert) to refine
  int* n_work;
  int stride;
};

// Experts of a lane in the choice: groups lie in lanes_per_group consecutive lanes
// each, expert i of group g in lane g*lanes + i%lanes, slot i/lanes.
struct ChoiceMap {
  int size, lanes, group, i0;
  __device__ ChoiceMap(const GateArgs& a, int lane) {
    size = a.E / a.groups;
    lanes = kWave;
    while (lanes * a.groups > kWave) lanes >>= 1;
    group = lane / lanes;
    i0 = lane % lanes;
  }
};

// One token's choice by one wave, in fp32 or (kFinal) fp64. Returns whether it is taken (and written); else the experts
// that it hangs on are appended to the work.
template <typename Real, int kSlots>
__device__ __forceinline__ bool choose(const GateArgs& a, const TokenState& s, int t, int32_t* ids, float* w, float units) {
  constexpr bool kDouble = sizeof(Real) == 8;
  const int lane = threadIdx.x & 63;
  const ChoiceMap map(a, lane);
  const double* logit = s.logit + t * s.stride;
  const float xn = s.x_norm[t];
  Real score[kSlots], arg[kSlots], c[kSlots], lo[kSlots], hi[kSlots];   // arg: the exponential's argument
  float delta[kSlots];
  int e_of[kSlots];
  bool open[kSlots];         // not refined
  Real m = -INFINITY;
  float dmax = 0.f;
#pragma unroll
  for (int j = 0; j < kSlots; ++j) {
    const int i = map.i0 + j * map.lanes;
    const bool valid = map.group < a.groups && i < map.size;
    const int e = valid ? map.group * map.size + i : -1;
    e_of[j] = e;
    open[j] = false;
    delta[j] = 0.f;
    score[j] = 0;
    if (valid) {
      score[j] = (Real)logit[e];
      open[j] = !((s.refined[t * 8 + (e >> 5)] >> (e & 31)) & 1u);
      if (open[j]) {
        const float wn = s.w_norm[e];
        delta[j] = units * kUnit * xn * wn;
        // norms that say nothing: past the fp32 range, or lost below it
        if (!(delta[j] < INFINITY) || ((xn < 0x1p-45f || wn < 0x1p-45f) && logit[e] != 0)) delta[j] = INFINITY;
      }
      m = fmax(m, score[j]);
      dmax = fmaxf(dmax, delta[j]);
    }
  }
  if (!a.sigmoid) {
    m = wave_max(m);
    // the sum of all exponentials matters next to a bias only: it scales every score alike
    dmax = a.select_bias ? wave_max(dmax) : 0.f;
    Real z = 0;
#pragma unroll
    for (int j = 0; j < kSlots; ++j)
      if (e_of[j] >= 0) {
        arg[j] = score[j] - m;
        score[j] = exp_of(arg[j]);
        z += score[j];
      }
    z = wave_sum(z);
#pragma unroll
    for (int j = 0; j < kSlots; ++j) score[j] /= z;
  }
#pragma unroll
  for (int j = 0; j < kSlots; ++j) {
    c[j] = lo[j] = hi[j] = -INFINITY;
    if (e_of[j] < 0) continue;
    Real part;               // the score's change with its logit
    float from = delta[j];
    if (a.sigmoid) {
      arg[j] = score[j];
      score[j] = 1 / (1 + exp_of(-score[j]));
      part = score[j] * (1 - score[j]);
    } else {
      part = score[j];
      from += dmax;
    }
    const Real b = a.select_bias ? (Real)a.select_bias[e_of[j]] : (Real)0;
    const Real v = score[j] + b;
    if (!(v > -INFINITY)) continue;
    // exp(x) - 1 <= 1.3 x up to 0.5
    Real eps = from <= 0.5f ? part * (Real)(1.3f * from) : (Real)INFINITY;
    if constexpr (!kDouble) {
      // the exponential and its argument's rounding, the sum of exponentials, the division; then the sum with b
      eps += score[j] * ((16 + fabsf(arg[j])) * kUnit) + (score[j] + fabsf(b)) * kUnit;
      eps = fmaxf(eps, 0x1p-120f);   // scores lost below the fp32 range
    }
    if (v == INFINITY) eps = 0;      // by its bias, whatever its score
    c[j] = v;
    lo[j] = v - eps;
    hi[j] = v + eps;
  }

  bool marks[kSlots];
#pragma unroll
  for (int j = 0; j < kSlots; ++j) marks[j] = false;
  if (a.groups > 1) {
    Top2<Real> vc, vlo, vhi;
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
      vc.add(c[j]);
      vlo.add(lo[j]);
      vhi.add(hi[j]);
    }
    vc.join(map.lanes);
    vlo.join(map.lanes);
    vhi.join(map.lanes);
    auto value = [&](const Top2<Real>& v) {
      const Real sum = a.top2 ? v.first + v.second : v.first;
      return sum > -INFINITY ? sum : (Real)-INFINITY;   // +inf and -inf too
    };
    const Real val = value(vc), val_lo = value(vlo), val_hi = value(vhi);
    int before = 0;
    for (int g = 0; g < a.groups; ++g) {
      const Real o = __shfl(val, g * map.lanes);
      before += o > val || (o == val && g < map.group);
    }
    const bool real = map.group < a.groups, kept = real && before < a.group_topk;
    const Real floor = -wave_max(kept ? -val_lo : (Real)-INFINITY);      // least value of a kept group
    const Real ceil = wave_max(real && !kept ? val_hi : (Real)-INFINITY);
    if (a.group_topk < a.groups && !(floor > ceil)) {
      const bool near = kept ? !(val_lo > ceil) : real && !(val_hi < floor);
      const Real least = a.top2 ? vlo.second : vlo.first;   // what a member needs to count in its group's value
#pragma unroll
      for (int j = 0; j < kSlots; ++j) marks[j] = near && open[j] && c[j] > -INFINITY && !(hi[j] < least);
    }
#pragma unroll
    for (int j = 0; j < kSlots; ++j)
      if (!kept) c[j] = lo[j] = hi[j] = -INFINITY;
  }

  // K rounds; lane k keeps round k's expert and lower end
  int rank[kSlots];
#pragma unroll
  for (int j = 0; j < kSlots; ++j) rank[j] = a.K;
  int my_id = -1;
  Real my_lo = -INFINITY, my_hi = -INFINITY;
  for (int k = 0; k < a.K; ++k) {
    Real v = -INFINITY;
#pragma unroll
    for (int j = 0; j < kSlots; ++j)
      if (rank[j] == a.K) v = fmax(v, c[j]);
    const Real top = wave_max(v);
    if (!(top > -INFINITY)) break;
    int e = kMaxExperts;
#pragma unroll
    for (int j = 0; j < kSlots; ++j)
      if (rank[j] == a.K && c[j] == top) e = min(e, e_of[j]);
    const uint64_t equal = __ballot(e < kMaxExperts);
    e = __popcll(equal) == 1 ? __builtin_amdgcn_readlane(e, __ffsll((unsigned long long)equal) - 1) : wave_min(e);
    Real l = -INFINITY, h = -INFINITY;
    bool mine = false;
#pragma unroll
    for (int j = 0; j < kSlots; ++j)
      if (e_of[j] == e) {
        rank[j] = k;
        l = lo[j];
        h = hi[j];
        mine = true;
      }
    const int owner = __ffsll((unsigned long long)__ballot(mine)) - 1;
    l = __shfl(l, owner);
    h = __shfl(h, owner);
    if (lane == k) {
      my_id = e;
      my_lo = l;
      my_hi = h;
    }
  }
  {
    // every pick lies above all that rank after it
    Real above = -INFINITY;
#pragma unroll
    for (int j = 0; j < kSlots; ++j)
      if (rank[j] == a.K) above = fmax(above, hi[j]);
    above = wave_max(above);
    for (int k = a.K - 1; k >= 0; --k) {
      const Real l = __shfl(my_lo, k), h = __shfl(my_hi, k);
      if (__shfl(my_id, k) >= 0 && !(l > above)) {
#pragma unroll
        for (int j = 0; j < kSlots; ++j) marks[j] = marks[j] || (open[j] && (rank[j] == k || (rank[j] > k && c[j] > -INFINITY && !(hi[j] < l))));
      }
      above = fmax(above, h);
    }
  }
  bool any = false;
#pragma unroll
  for (int j = 0; j < kSlots; ++j) any = any || marks[j];
  if (__any(any)) {
    // next to a bias a softmax hangs on every logit
    const bool all = !a.sigmoid && a.select_bias;
#pragma unroll
    for (int j = 0; j < kSlots; ++j)
      if (all ? open[j] : marks[j]) s.work[atomicAdd(s.n_work, 1)] = (uint16_t)(t << 8 | e_of[j]);
    return false;
  }

  // weights, in fp64 from the logits of the chosen
  double sk = 0;
  if (my_id >= 0) sk = a.sigmoid ? 1 / (1 + exp(-logit[my_id])) : exp(logit[my_id] - m);
  double total = wave_sum(sk);
  if (!a.renorm) {
    total = 1;
    if (!a.sigmoid) {
      total = 0;
      for (int e = lane; e < a.E; e += kWave) total += exp(logit[e] - m);
      total = wave_sum(total);
    }
  }
  if (lane < a.K) {
    ids[lane] = my_id;
    w[lane] = total > 0 ? (float)(sk / total * a.scale) : 0.f;
  }
  return true;
}

// The choice of the workgroup's tokens (kTok of them at most, n present) once their logits lie in LDS. All waves call
// it, after a barrier; wave v takes tokens v, v + kWaves, ...
template <typename Act, int kWaves, int kTok, int kSlots>
__device__ __forceinline__ void choose_all(const GateArgs& a, const TokenState& s, int tok0, int n, float units) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr int kMine = (kTok + kWaves - 1) / kWaves;
  uint32_t pending = 0;
#pragma unroll
  for (int i = 0; i < kMine; ++i)
    if (wave + kWaves * i < n) pending |= 1u << i;
  bool first = *s.n_work == 0;   // logits that are no numbers in fp32 are refined before any choice
  __syncthreads();               // every wave has read it before one adds to it
  for (;;) {
    if (first) {
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int t = wave + kWaves * i;
        const long o = (long)(tok0 + t) * a.K;
        if ((pending >> i & 1) && choose<float, kSlots>(a, s, t, a.topk_ids + o, a.topk_w + o, units)) pending &= ~(1u << i);
      }
      first = false;
      __syncthreads();
    }
    const int work = *s.n_work;
    if (work == 0) break;
    for (int i = wave; i < work; i += kWaves) {
      const int t = s.work[i] >> 8, e = s.work[i] & 255;
      const double v = dot64(static_cast<const Act*>(a.x) + (long)(tok0 + t) * a.d,
                             static_cast<const Act*>(a.router_w) + (long)e * a.d, a.d);
      if (lane == 0) {
        s.logit[t * s.stride + e] = a.router_bias ? v + a.router_bias[e] : v;
        atomicOr(&s.refined[t * 8 + (e >> 5)], 1u << (e & 31));
      }
    }
    __syncthreads();
    if (threadIdx.x == 0) *s.n_work = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int t = wave + kWaves * i;
      const long o = (long)(tok0 + t) * a.K;
      if ((pending >> i & 1) && choose<double, kSlots>(a, s, t, a.topk_ids + o, a.topk_w + o, units)) pending &= ~(1u << i);
    }
    __syncthreads();
  }
}

// Sum of a logit's parts, written with its bias; what is no number, or near the end of fp32's range, is left to fp64.
__device__ __forceinline__ void put_logit(const GateArgs& a, const TokenState& s, int t, int e, double v) {
  s.logit[t * s.stride + e] = a.router_bias ? v + a.router_bias[e] : v;
  if (!(fabs(v) < 0x1p120)) s.work[atomicAdd(s.n_work, 1)] = (uint16_t)(t << 8 | e);
}

// ------------------------------------------------------------------ up to 64 experts
constexpr int kTok = 16;
constexpr int kSlices = 16;

// One workgroup scores tpw <= 16 tokens against every expert (the MFMA tile keeps
// 16 rows; rows past tpw stay zero), EB blocks of 16 experts. Slice s of the hidden
// dimension is its 32-wide chunks s, s + 16, ...; wave w takes the slices w, w + kWaves, ..., U
// chunks requested together, and the slices' sums meet in LDS. A token's sums
// depend neither on tpw nor on kWaves.
template <typename Act, int EB, int kWaves>
__global__ __launch_bounds__(kWaves* kWave, 4) void route_gated_kernel(GateArgs a, int tpw) {
  constexpr int EP = 16 * EB;
  constexpr int U = sizeof(Act) == 2 ? 4 / EB : EB == 1 ? 2 : 1;   // more would spill
  constexpr int kSlots = EB <= 2 ? 1 : 2;   // a group has more than 32 / groups lanes
  __shared__ float part[kSlices][kTok][EP];
  __shared__ float norm_part[kSlices][kTok + EP];
  __shared__ double logit[kTok][EP];
  __shared__ float x_norm[kTok], w_norm[EP];
  __shared__ uint32_t refined[kTok][8];
  __shared__ uint16_t work[kTok * EP];
  __shared__ int n_work;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int li = lane & 15;
  const int lg = lane >> 4;
  const int tok0 = blockIdx.x * tpw;
  const int n = min(tpw, a.T - tok0);
  const int d = a.d;
  const Act* x = static_cast<const Act*>(a.x) + (long)(tok0 + min(li, n - 1)) * d + 8 * lg;
  const bool x_ok = li < n;
  const Act* wr = static_cast<const Act*>(a.router_w) + 8 * lg;
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  const int chunks = d >> 5;

#pragma unroll 1
  for (int slice = wave; slice < kSlices; slice += kWaves) {
    double acc[EB][4];
#pragma unroll
    for (int eb = 0; eb < EB; ++eb)
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[eb][r] = 0;
    f32x4 xx = zero, ww[EB];    // bf16: tiles of x.x and w.w, whose diagonals are the norms
    float xs = 0.f, wsum[EB];   // fp32: a lane's part of them
#pragma unroll
    for (int eb = 0; eb < EB; ++eb) {
      ww[eb] = zero;
      wsum[eb] = 0.f;
    }
    if constexpr (sizeof(Act) == 2) {
      bf16x8 u[2][U], v[2][U][EB];
      auto load = [&](int c0, bf16x8 (&un)[U], bf16x8 (&vn)[U][EB]) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int c = c0 + i * kSlices;
          un[i] = x_ok && c < chunks ? as_bf16x8(*reinterpret_cast<const uint4*>(x + 32 * c)) : zero_bf16x8();
#pragma unroll
          for (int eb = 0; eb < EB; ++eb) {
            const int e = eb * 16 + li;
            vn[i][eb] = e < a.E && c < chunks ? as_bf16x8(*reinterpret_cast<const uint4*>(wr + (long)e * d + 32 * c)) : zero_bf16x8();
          }
        }
      };
      auto add = [&](const bf16x8 (&un)[U], const bf16x8 (&vn)[U][EB]) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
          xx = mfma_bf16(un[i], un[i], xx);
#pragma unroll
          for (int eb = 0; eb < EB; ++eb) {
            const f32x4 p = mfma_bf16(un[i], vn[i][eb], zero);
            ww[eb] = mfma_bf16(vn[i][eb], vn[i][eb], ww[eb]);
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[eb][r] += (double)p[r];
          }
        }
      };
      load(slice, u[0], v[0]);
      for (int c0 = slice; c0 < chunks; c0 += 2 * kSlices * U) {
        load(c0 + kSlices * U, u[1], v[1]);
        add(u[0], v[0]);
        if (c0 + kSlices * U >= chunks) break;
        load(c0 + 2 * kSlices * U, u[0], v[0]);
        add(u[1], v[1]);
      }
    } else {
      f32x4 u[2][U][2], v[2][U][EB][2];
      auto load = [&](int c0, f32x4 (&un)[U][2], f32x4 (&vn)[U][EB][2]) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int c = c0 + i * kSlices;
          un[i][0] = un[i][1] = zero;
          if (x_ok && c < chunks) {
            const f32x4* p = reinterpret_cast<const f32x4*>(x + 32 * c);
            un[i][0] = p[0];
            un[i][1] = p[1];
          }
#pragma unroll
          for (int eb = 0; eb < EB; ++eb) {
            const int e = eb * 16 + li;
            vn[i][eb][0] = vn[i][eb][1] = zero;
            if (e < a.E && c < chunks) {
              const f32x4* p = reinterpret_cast<const f32x4*>(wr + (long)e * d + 32 * c);
              vn[i][eb][0] = p[0];
              vn[i][eb][1] = p[1];
            }
          }
        }
      };
      auto add = [&](const f32x4 (&un)[U][2], const f32x4 (&vn)[U][EB][2]) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
          f32x4 p[EB];
#pragma unroll
          for (int eb = 0; eb < EB; ++eb) p[eb] = zero;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float y = un[i][j >> 2][j & 3];
            xs += y * y;
#pragma unroll
            for (int eb = 0; eb < EB; ++eb) {
              const float z = vn[i][eb][j >> 2][j & 3];
              p[eb] = mfma_f32(y, z, p[eb]);
              wsum[eb] += z * z;
            }
          }
#pragma unroll
          for (int eb = 0; eb < EB; ++eb)
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[eb][r] += (double)p[eb][r];
        }
      };
      load(slice, u[0], v[0]);
      for (int c0 = slice; c0 < chunks; c0 += 2 * kSlices * U) {
        load(c0 + kSlices * U, u[1], v[1]);
        add(u[0], v[0]);
        if (c0 + kSlices * U >= chunks) break;
        load(c0 + 2 * kSlices * U, u[0], v[0]);
        add(u[1], v[1]);
      }
    }

    // lane l holds tokens 4*lg + r of expert 16*eb + li
#pragma unroll
    for (int eb = 0; eb < EB; ++eb)
#pragma unroll
      for (int r = 0; r < 4; ++r) part[slice][4 * lg + r][eb * 16 + li] = (float)acc[eb][r];
    if constexpr (sizeof(Act) == 2) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (4 * lg + r == li) {
          norm_part[slice][li] = xx[r];
#pragma unroll
          for (int eb = 0; eb < EB; ++eb) norm_part[slice][kTok + eb * 16 + li] = ww[eb][r];
        }
    } else {
      xs += __shfl_xor(xs, 16);
      xs += __shfl_xor(xs, 32);
      if (lg == 0) norm_part[slice][li] = xs;
#pragma unroll
      for (int eb = 0; eb < EB; ++eb) {
        wsum[eb] += __shfl_xor(wsum[eb], 16);
        wsum[eb] += __shfl_xor(wsum[eb], 32);
        if (lg == 0) norm_part[slice][kTok + eb * 16 + li] = wsum[eb];
      }
    }
  }
  const TokenState s = {&logit[0][0], x_norm, w_norm, &refined[0][0], work, &n_work, EP};
  if (threadIdx.x < kTok * 8) (&refined[0][0])[threadIdx.x] = 0;
  if (threadIdx.x == 0) n_work = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n * EP; i += kWaves * kWave) {
    const int t = i / EP, e = i % EP;
    double v = 0;
#pragma unroll
    for (int k = 0; k < kSlices; ++k) v += (double)part[k][t][e];
    if (e < a.E) put_logit(a, s, t, e, v);
  }
  if (threadIdx.x < kTok + EP) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < kSlices; ++k) v += norm_part[k][threadIdx.x];
    // the sum of squares is off by less than a thousandth
    v = sqrtf(v) * 1.01f;
    if (threadIdx.x < kTok) x_norm[threadIdx.x] = v;
    else w_norm[threadIdx.x - kTok] = v;
  }
  __syncthreads();
  // the parts of the slices are rounded to fp32 once more
  choose_all<Act, kWaves, kTok, kSlots>(a, s, tok0, n, kMfmaUnits + 1.f);
}

// ------------------------------------------------------------------ up to 256 experts
constexpr int kWideWaves = 16;
constexpr int kRowBytes = 256;   // of a token's row in a step

// One workgroup scores 16*TB tokens. Its 16 waves take a block of 16 experts each (KS = 1), or half of the chunks of
// one (KS = 2, up to 128 experts), and share the tokens' rows through LDS (direct loads, double buffered; 16-byte pieces
// XOR-swizzled by the row). The weights go to the registers of the one wave that needs them, a step ahead.
template <typename Act, int TB, int KS>
__global__ __launch_bounds__(kWideWaves* kWave) void route_gated_wide_kernel(GateArgs a) {
  constexpr int EP = kMaxExperts / KS;
  constexpr int TOK = 16 * TB;
  constexpr int CS = kRowBytes / (32 * (int)sizeof(Act));   // 32-wide chunks of a step: 4 or 2
  constexpr int WC = CS / KS;                               // of a wave
  constexpr int STAGE = TOK * kRowBytes;
  __shared__ __attribute__((aligned(1024))) uint8_t xs[2][STAGE];
  __shared__ double logit[TOK][EP];
  __shared__ float x_norm[TOK], w_norm[EP];
  __shared__ uint32_t refined[TOK][8];
  __shared__ uint16_t work[TOK * EP];
  __shared__ int n_work;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int li = lane & 15;
  const int lg = lane >> 4;
  const int tok0 = blockIdx.x * TOK;
  const int n = min(TOK, a.T - tok0);
  const int d = a.d;
  const int ks = wave / (16 / KS);
  const int e = (wave % (16 / KS)) * 16 + li;
  const bool active = (wave % (16 / KS)) * 16 < a.E;
  const TokenState s = {&logit[0][0], x_norm, w_norm, &refined[0][0], work, &n_work, EP};
  if (threadIdx.x < TOK * 8) (&refined[0][0])[threadIdx.x] = 0;
  if (threadIdx.x < TOK) x_norm[threadIdx.x] = 0.f;
  if (threadIdx.x < EP) w_norm[threadIdx.x] = 0.f;
  if (threadIdx.x == 0) n_work = 0;

  const uint8_t* x = static_cast<const uint8_t*>(a.x) + (long)tok0 * d * sizeof(Act);
  const Act* wr = static_cast<const Act*>(a.router_w) + (long)min(e, a.E - 1) * d + 8 * lg;
  const int chunks = d >> 5;
  const int nsteps = (chunks + CS - 1) / CS;
  // waves 0 .. 4*TB - 1 copy four rows each; the last step of bf16 rows may be half a step: its other half re-reads the first
  const int row = wave * 4 + (lane >> 4);
  const int piece = li ^ (row & 15);
  const uint32_t x_off = (uint32_t)min(row, n - 1) * (uint32_t)(d * (int)sizeof(Act)) + 16u * piece;
  auto issue_x = [&](int step, int buf) {
    if (wave >= 4 * TB || step >= nsteps) return;
    uint32_t off = x_off + (uint32_t)step * kRowBytes;
    if (step * CS + CS > chunks && piece >= 8) off -= 128;
    dma16(x, off, lds_addr(&xs[buf][0]) + wave * 1024);
  };
  constexpr int V = sizeof(Act) == 2 ? 1 : 2;   // 16-byte loads of a lane's 8 elements
  auto load_w = [&](int step, uint4 (&b)[WC][V]) {
#pragma unroll
    for (int i = 0; i < WC; ++i) {
      const int c = min(step * CS + i * KS + ks, chunks - 1);
#pragma unroll
      for (int h = 0; h < V; ++h) b[i][h] = reinterpret_cast<const uint4*>(wr + 32 * (long)c)[h];
    }
  };
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  double acc[TB][4];
#pragma unroll
  for (int tb = 0; tb < TB; ++tb)
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[tb][r] = 0;
  f32x4 xx = zero, ww = zero;
  float xsum = 0.f, wsum = 0.f;
  // a lane's 8 elements of chunk c of a step, token block tb
  auto x_piece = [&](int buf, int tb, int c, int h) {
    const int r = tb * 16 + li;
    const int p = V == 1 ? 4 * c + lg : 8 * c + 2 * lg + h;
    return *reinterpret_cast<const uint4*>(&xs[buf][r * kRowBytes + 16 * (p ^ li)]);
  };
  auto step_of = [&](int st, int buf, const uint4 (&b)[WC][V], uint4 (&bn)[WC][V]) {
    // this step's rows have landed, and every wave is past the buffer that the next ones overwrite
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));
    __builtin_amdgcn_s_barrier();
    issue_x(st + 1, 1 - buf);
    if (active && st + 1 < nsteps) load_w(st + 1, bn);
    if (active) {
      f32x4 p[TB];
#pragma unroll
      for (int i = 0; i < WC; ++i) {
        const int c = i * KS + ks;
        if (st * CS + c >= chunks) break;
        // sums of two chunks with bf16, of one (a chain of eight) with fp32
        if (V == 2 || i % 2 == 0)
#pragma unroll
          for (int tb = 0; tb < TB; ++tb) p[tb] = zero;
        if constexpr (V == 1) {
          const bf16x8 w = as_bf16x8(b[i][0]);
          ww = mfma_bf16(w, w, ww);
#pragma unroll
          for (int tb = 0; tb < TB; ++tb) p[tb] = mfma_bf16(as_bf16x8(x_piece(buf, tb, c, 0)), w, p[tb]);
        } else {
          const f32x4 w[2] = {__builtin_bit_cast(f32x4, b[i][0]), __builtin_bit_cast(f32x4, b[i][V - 1])};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            f32x4 u[TB];
#pragma unroll
            for (int tb = 0; tb < TB; ++tb) u[tb] = __builtin_bit_cast(f32x4, x_piece(buf, tb, c, h));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              wsum += w[h][j] * w[h][j];
#pragma unroll
              for (int tb = 0; tb < TB; ++tb) p[tb] = mfma_f32(u[tb][j], w[h][j], p[tb]);
            }
          }
        }
        if (V == 2 || i % 2 == 1 || i == WC - 1 || st * CS + c + KS >= chunks)
#pragma unroll
          for (int tb = 0; tb < TB; ++tb)
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[tb][r] += (double)p[tb][r];
      }
    }
    // the tokens' norms: wave tb takes token block tb
    if (wave < TB) {
#pragma unroll
      for (int c = 0; c < CS; ++c) {
        if (st * CS + c >= chunks) break;
#pragma unroll
        for (int h = 0; h < V; ++h) {
          const uint4 q = x_piece(buf, wave, c, h);
          if constexpr (V == 1) {
            xx = mfma_bf16(as_bf16x8(q), as_bf16x8(q), xx);
          } else {
            const f32x4 u = __builtin_bit_cast(f32x4, q);
#pragma unroll
            for (int j = 0; j < 4; ++j) xsum += u[j] * u[j];
          }
        }
      }
    }
  };
  uint4 b[2][WC][V];
  issue_x(0, 0);
  if (active) load_w(0, b[0]);
  for (int st = 0; st < nsteps; st += 2) {
    step_of(st, 0, b[0], b[1]);
    if (st + 1 < nsteps) step_of(st + 1, 1, b[1], b[0]);
  }

  // norms (1.01: the sum of squares is off by less than a thousandth), and the slices' sums
  if constexpr (V == 2) {
    xsum += __shfl_xor(xsum, 16);
    xsum += __shfl_xor(xsum, 32);
    wsum += __shfl_xor(wsum, 16);
    wsum += __shfl_xor(wsum, 32);
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    if (V == 1 ? 4 * lg + r != li : lg > 0 || r > 0) continue;
    if (wave < TB) x_norm[wave * 16 + li] = sqrtf(V == 1 ? xx[r] : xsum) * 1.01f;
    if (active && KS == 1) w_norm[e] = sqrtf(V == 1 ? ww[r] : wsum) * 1.01f;
    if (active && KS == 2) atomicAdd(&w_norm[e], V == 1 ? ww[r] : wsum);   // squares; two addends
  }
  if (KS == 2 && active && ks == 1) {
#pragma unroll
    for (int tb = 0; tb < TB; ++tb)
#pragma unroll
      for (int r = 0; r < 4; ++r) logit[tb * 16 + 4 * lg + r][e] = acc[tb][r];
  }
  __syncthreads();
  if (KS == 2 && threadIdx.x < EP) w_norm[threadIdx.x] = sqrtf(w_norm[threadIdx.x]) * 1.01f;
  if (active && ks == 0) {
#pragma unroll
    for (int tb = 0; tb < TB; ++tb)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = tb * 16 + 4 * lg + r;
        if (t < n && e < a.E) put_logit(a, s, t, e, KS == 2 ? acc[tb][r] + logit[t][e] : acc[tb][r]);
      }
  }
  __syncthreads();
  const float units = V == 1 ? 2 * kMfmaUnits : kMfmaUnits;
  // slots of a lane: experts of a group over its lanes, 8 at most; 4 if the groups are a power of two, as they mostly are
  const ChoiceMap map(a, lane);
  if (map.size <= 4 * map.lanes) choose_all<Act, kWideWaves, TOK, 4>(a, s, tok0, n, units);
  else choose_all<Act, kWideWaves, TOK, 8>(a, s, tok0, n, units);
}

template <typename Act, int EB>
void launch_narrow(const GateArgs& a, hipStream_t stream) {
  // as few tokens a workgroup as leave no CU without one, so that a small batch's reads of router_w are spread
  const int tpw = min(kTok, (a.T + 255) / 256);
  const dim3 grid((a.T + tpw - 1) / tpw);
  // few workgroups: the most waves each; many: two workgroups a CU, one of which loads while the other chooses
  if (grid.x <= 256) hipLaunchKernelGGL((route_gated_kernel<Act, EB, 16>), grid, dim3(16 * kWave), 0, stream, a, tpw);
  else hipLaunchKernelGGL((route_gated_kernel<Act, EB, 8>), grid, dim3(8 * kWave), 0, stream, a, tpw);
}

template <typename Act, int TB>
void launch_wide(const GateArgs& a, hipStream_t stream) {
  const dim3 grid((a.T + 16 * TB - 1) / (16 * TB)), block(kWideWaves * kWave);
  if (a.E <= 128) hipLaunchKernelGGL((route_gated_wide_kernel<Act, TB, 2>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((route_gated_wide_kernel<Act, TB, 1>), grid, block, 0, stream, a);
}

template <typename Act>
void launch(const GateArgs& a, hipStream_t stream) {
  if (a.E <= 16) launch_narrow<Act, 1>(a, stream);
  else if (a.E <= 32) launch_narrow<Act, 2>(a, stream);
  else if (a.E <= 64) launch_narrow<Act, 4>(a, stream);
  else if (a.T <= 256 * 16) launch_wide<Act, 1>(a, stream);
  else launch_wide<Act, 2>(a, stream);
}

}  // namespace

hipError_t launch_route_gated(const GateArgs& a, hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  if (a.act_bf16) launch<__bf16>(a, stream);
  else launch<float>(a, stream);
  return hipGetLastError();
}

}  // namespace moe
