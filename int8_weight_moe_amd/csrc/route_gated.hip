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
constexpr int kWaves = 16;

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
  uint32_t* work;      // (token << 16 | expert) to refine
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
      if (all ? open[j] : marks[j]) s.work[atomicAdd(s.n_work, 1)] = (uint32_t)t << 16 | (uint32_t)e_of[j];
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
template <typename Act, int kTok, int kSlots>
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
      const uint32_t p = s.work[i];
      const int t = p >> 16, e = p & 0xffff;
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
  if (!(fabs(v) < 0x1p120)) s.work[atomicAdd(s.n_work, 1)] = (uint32_t)t << 16 | (uint32_t)e;
}

// ------------------------------------------------------------------ up to 64 experts
constexpr int kTok = 16;

// One workgroup scores tpw <= 16 tokens against every expert (the MFMA tile keeps
// 16 rows; rows past tpw stay zero), EB blocks of 16 experts. Wave w takes the
// 32-wide chunks w, w + 16, ... of the hidden dimension, U of them requested
// together. A token's sums do not depend on tpw.
template <typename Act, int EB>
__global__ __launch_bounds__(kWaves* kWave) void route_gated_kernel(GateArgs a, int tpw) {
  constexpr int EP = 16 * EB;
  constexpr int U = EB == 4 ? 2 : sizeof(Act) == 2 ? 8 / EB : 4 / EB;
  constexpr int kSlots = EB <= 2 ? 1 : 2;   // a group has more than 32 / groups lanes
  __shared__ float part[kWaves][kTok][EP];
  __shared__ float norm_part[kWaves][kTok + EP];
  __shared__ double logit[kTok][EP];
  __shared__ float x_norm[kTok], w_norm[EP];
  __shared__ uint32_t refined[kTok][8], work[kTok * EP];
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

  double acc[EB][4];
#pragma unroll
  for (int eb = 0; eb < EB; ++eb)
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[eb][r] = 0;
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  f32x4 xx = zero, ww[EB];    // bf16: tiles of x.x and w.w, whose diagonals are the norms
  float xs = 0.f, wsum[EB];   // fp32: a lane's part of them
#pragma unroll
  for (int eb = 0; eb < EB; ++eb) {
    ww[eb] = zero;
    wsum[eb] = 0.f;
  }
  const int chunks = d >> 5;
  for (int c0 = wave; c0 < chunks; c0 += kWaves * U) {
    if constexpr (sizeof(Act) == 2) {
      bf16x8 u[U], v[U][EB];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int c = c0 + i * kWaves;
        u[i] = x_ok && c < chunks ? as_bf16x8(*reinterpret_cast<const uint4*>(x + 32 * c)) : zero_bf16x8();
#pragma unroll
        for (int eb = 0; eb < EB; ++eb) {
          const int e = eb * 16 + li;
          v[i][eb] = e < a.E && c < chunks ? as_bf16x8(*reinterpret_cast<const uint4*>(wr + (long)e * d + 32 * c)) : zero_bf16x8();
        }
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        xx = mfma_bf16(u[i], u[i], xx);
#pragma unroll
        for (int eb = 0; eb < EB; ++eb) {
          const f32x4 p = mfma_bf16(u[i], v[i][eb], zero);
          ww[eb] = mfma_bf16(v[i][eb], v[i][eb], ww[eb]);
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[eb][r] += (double)p[r];
        }
      }
    } else {
      f32x4 u[U][2], v[U][EB][2];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int c = c0 + i * kWaves;
        u[i][0] = u[i][1] = zero;
        if (x_ok && c < chunks) {
          const f32x4* p = reinterpret_cast<const f32x4*>(x + 32 * c);
          u[i][0] = p[0];
          u[i][1] = p[1];
        }
#pragma unroll
        for (int eb = 0; eb < EB; ++eb) {
          const int e = eb * 16 + li;
          v[i][eb][0] = v[i][eb][1] = zero;
          if (e < a.E && c < chunks) {
            const f32x4* p = reinterpret_cast<const f32x4*>(wr + (long)e * d + 32 * c);
            v[i][eb][0] = p[0];
            v[i][eb][1] = p[1];
          }
        }
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) xs += u[i][j >> 2][j & 3] * u[i][j >> 2][j & 3];
#pragma unroll
        for (int eb = 0; eb < EB; ++eb) {
          f32x4 p = zero;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float y = v[i][eb][j >> 2][j & 3];
            p = mfma_f32(u[i][j >> 2][j & 3], y, p);
            wsum[eb] += y * y;
          }
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[eb][r] += (double)p[r];
        }
      }
    }
  }

  // lane l holds tokens 4*lg + r of expert 16*eb + li
#pragma unroll
  for (int eb = 0; eb < EB; ++eb)
#pragma unroll
    for (int r = 0; r < 4; ++r) part[wave][4 * lg + r][eb * 16 + li] = (float)acc[eb][r];
  if constexpr (sizeof(Act) == 2) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (4 * lg + r == li) {
        norm_part[wave][li] = xx[r];
#pragma unroll
        for (int eb = 0; eb < EB; ++eb) norm_part[wave][kTok + eb * 16 + li] = ww[eb][r];
      }
  } else {
    xs += __shfl_xor(xs, 16);
    xs += __shfl_xor(xs, 32);
    if (lg == 0) norm_part[wave][li] = xs;
#pragma unroll
    for (int eb = 0; eb < EB; ++eb) {
      wsum[eb] += __shfl_xor(wsum[eb], 16);
      wsum[eb] += __shfl_xor(wsum[eb], 32);
      if (lg == 0) norm_part[wave][kTok + eb * 16 + li] = wsum[eb];
    }
  }
  const TokenState s = {&logit[0][0], x_norm, w_norm, &refined[0][0], work, &n_work, EP};
  if (threadIdx.x < kTok * 8) (&refined[0][0])[threadIdx.x] = 0;
  if (threadIdx.x == 0) n_work = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < kTok * EP; i += kWaves * kWave) {
    const int t = i / EP, e = i % EP;
    double v = 0;
#pragma unroll
    for (int k = 0; k < kWaves; ++k) v += (double)part[k][t][e];
    if (t < n && e < a.E) put_logit(a, s, t, e, v);
  }
  if (threadIdx.x < kTok + EP) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < kWaves; ++k) v += norm_part[k][threadIdx.x];
    // the sum of squares is off by less than a thousandth
    v = sqrtf(v) * 1.01f;
    if (threadIdx.x < kTok) x_norm[threadIdx.x] = v;
    else w_norm[threadIdx.x - kTok] = v;
  }
  __syncthreads();
  // the parts of the waves are rounded to fp32 once more
  choose_all<Act, kTok, kSlots>(a, s, tok0, n, kMfmaUnits + 1.f);
}

// ------------------------------------------------------------------ up to 256 experts
// One workgroup scores 16 tokens; wave w takes the experts 16*w .. +16 over the whole hidden dimension.
template <typename Act>
__global__ __launch_bounds__(kWaves* kWave) void route_gated_wide_kernel(GateArgs a, int tpw) {
  constexpr int EP = kMaxExperts;
  constexpr int U = 4;
  __shared__ double logit[kTok][EP];
  __shared__ float x_norm[kTok], w_norm[EP];
  __shared__ uint32_t refined[kTok][8], work[kTok * EP];
  __shared__ int n_work;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int li = lane & 15;
  const int lg = lane >> 4;
  const int tok0 = blockIdx.x * tpw;
  const int n = min(tpw, a.T - tok0);
  const int d = a.d;
  const int e = wave * 16 + li;
  const TokenState s = {&logit[0][0], x_norm, w_norm, &refined[0][0], work, &n_work, EP};
  if (threadIdx.x < kTok * 8) (&refined[0][0])[threadIdx.x] = 0;
  if (threadIdx.x == 0) n_work = 0;
  __syncthreads();
  if (wave * 16 < a.E) {
    const Act* x = static_cast<const Act*>(a.x) + (long)(tok0 + min(li, n - 1)) * d + 8 * lg;
    const Act* wr = static_cast<const Act*>(a.router_w) + (long)min(e, a.E - 1) * d + 8 * lg;
    double acc[4] = {0, 0, 0, 0};
    float xs = 0.f, wsum = 0.f;
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    f32x4 xx = zero, ww = zero;
    const int chunks = d >> 5;
    for (int c0 = 0; c0 < chunks; c0 += U) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (c0 + i >= chunks) break;
        if constexpr (sizeof(Act) == 2) {
          const bf16x8 u = as_bf16x8(*reinterpret_cast<const uint4*>(x + 32 * (c0 + i)));
          const bf16x8 v = as_bf16x8(*reinterpret_cast<const uint4*>(wr + 32 * (c0 + i)));
          const f32x4 p = mfma_bf16(u, v, zero);
          ww = mfma_bf16(v, v, ww);
          if (wave == 0) xx = mfma_bf16(u, u, xx);
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[r] += (double)p[r];
        } else {
          const f32x4* q = reinterpret_cast<const f32x4*>(x + 32 * (c0 + i));
          const f32x4* b = reinterpret_cast<const f32x4*>(wr + 32 * (c0 + i));
          f32x4 p = zero;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float y = q[j >> 2][j & 3], z = b[j >> 2][j & 3];
            p = mfma_f32(y, z, p);
            xs += y * y;
            wsum += z * z;
          }
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[r] += (double)p[r];
        }
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (4 * lg + r < n && e < a.E) put_logit(a, s, 4 * lg + r, e, acc[r]);
    if constexpr (sizeof(Act) == 2) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (4 * lg + r == li) {
          w_norm[e] = sqrtf(ww[r]) * 1.01f;
          if (wave == 0) x_norm[li] = sqrtf(xx[r]) * 1.01f;
        }
    } else {
      xs += __shfl_xor(xs, 16);
      xs += __shfl_xor(xs, 32);
      wsum += __shfl_xor(wsum, 16);
      wsum += __shfl_xor(wsum, 32);
      if (lg == 0) {
        w_norm[e] = sqrtf(wsum) * 1.01f;
        if (wave == 0) x_norm[li] = sqrtf(xs) * 1.01f;
      }
    }
  }
  __syncthreads();
  choose_all<Act, kTok, 8>(a, s, tok0, n, kMfmaUnits);
}

template <typename Act>
void launch(const GateArgs& a, hipStream_t stream) {
  // as few tokens a workgroup as leave no CU without one, so that a small batch's reads of router_w are spread
  const int tpw = min(kTok, (a.T + 255) / 256);
  const dim3 grid((a.T + tpw - 1) / tpw), block(kWaves * kWave);
  if (a.E <= 16) hipLaunchKernelGGL((route_gated_kernel<Act, 1>), grid, block, 0, stream, a, tpw);
  else if (a.E <= 32) hipLaunchKernelGGL((route_gated_kernel<Act, 2>), grid, block, 0, stream, a, tpw);
  else if (a.E <= 64) hipLaunchKernelGGL((route_gated_kernel<Act, 4>), grid, block, 0, stream, a, tpw);
  else hipLaunchKernelGGL((route_gated_wide_kernel<Act>), grid, block, 0, stream, a, tpw);
}

}  // namespace

hipError_t launch_route_gated(const GateArgs& a, hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  if (a.act_bf16) launch<__bf16>(a, stream);
  else launch<float>(a, stream);
  return hipGetLastError();
}

}  // namespace moe
