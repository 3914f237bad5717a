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
// waves of a workgroup, in blocks of 128 bytes of a row (whole cache lines). A
// block's sums are added in fp64, so a logit is taken to be off by at most
//     delta = kSumUnits * 2^-23 * |x| |w_e|
// (what the MFMAs' own sums round, as measured; sum |x_i w_i| <= |x| |w_e|).
// |x|^2 and |w_e|^2 are taken on the way.
// Choice: one wave a token, in fp32 with an error bound eps_e on every c_e (delta
// through the score's derivative, the evaluation, the bias's rounding). A decision
// between two values whose intervals overlap is not taken: the experts it hangs on
// are marked, the workgroup's waves compute their logits again in fp64, and the choice is
// repeated, in fp64 if it then hangs on the fp32 evaluation alone. So the ids are
// those of 64-bit values, at the price of fp32 ones.
//
// What bounds it: 16 experts, the reads of x (16384 x 8192 bf16 in 60 us, 4.5 TB/s of a copy's 4.8). 256 experts (8192 x
// 4096, 78 us): 50 us of logits, whose rows pass through LDS at 20 bytes a cycle and CU (nothing but the loads takes as
// long), then 14 us of choosing, 1000 instructions a token at four waves a SIMD, and 15 us for the tokens of each workgroup
// that are refined and chosen again. fp32 (2999 x 4096, 60 experts, 66 us): mostly the logits, whose
// workgroups of 12 tokens read all of router_w each. One token is 7.5 us of latency: rows to LDS, sums, choice.
#include "device_common.h"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kMaxExperts = 256;
// Up to so many tokens split rows of at least so many steps over workgroups, given a
// workspace. Measured, us, split / fused kernel: 1 token, d 8192, E 16 (8 steps) 7.8 / 9.9, d 4096 (4 steps) 8.0 / 7.8;
// d 8192, E 64 (32 steps): 63 tokens 13.2 / 26.0, 256 19.0 / 32.4, 1024 27.6 / 37.0, 2048 40.0 / 38.4; d 4096, E 256
// (64 steps): 16 tokens 21.6 / 44.7, 1024 39.8 / 56.8, 2048 58.2 / 57.9; d 8192, E 16: 1024 13.4 / 15.2, 2048 19.8 / 15.5.
constexpr int kSplitTokens = 1024, kSplitSteps = 8;

// What the fp32 sums of a block are taken to be off by, in 2^-23 of the sum of their
// terms' magnitudes: measured, not documented. A 16x16x32 bf16 MFMA cuts each of
// eight products (a lane's) off at 2^-24 of the power of two below the largest of
// them, adds them, and rounds to nearest as it adds each of the four such sums, cut
// off at some 2^-30, to the accumulator. Two of them make a block's sum: 7 products'
// 2^-24 of the largest, 8 roundings of 2^-24 and 8 cuts of 2^-30, 7.6 units. (Inputs
// bred for the largest error reach 7.51.)
// A chain of four 16x16x4 fp32 MFMAs rounds 16 sums by 2^-24 each: 8 (7.50 reached).
constexpr float kSumUnits = 8.f;
constexpr float kUnit = 0x1p-23f;

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
// The largest value of the lanes after this one, in lanes 0 .. 7 and of theirs.
__device__ __forceinline__ float after(float v) {
  v = dpp_or<0x101, 0xf>(v, -INFINITY);              // from the next lane of the row of 16
  v = fmaxf(v, dpp_or<0x101, 0xf>(v, -INFINITY));
  v = fmaxf(v, dpp_or<0x102, 0xf>(v, -INFINITY));
  return fmaxf(v, dpp_or<0x104, 0xf>(v, -INFINITY));
}
__device__ __forceinline__ double after(double v) {
  v = __shfl_down(v, 1);
#pragma unroll
  for (int off = 1; off <= 4; off <<= 1) v = fmax(v, __shfl_down(v, off));
  return v;
}
__device__ __forceinline__ int wave_min(int v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = min(v, __shfl_xor(v, off));
  return v;
}

// a . b over d elements by one wave, in fp64; the same value in every lane. Sixteen bytes a lane and load, U of them
// requested together: the rows come from afar, one load at a time took 12 us for 4096 elements.
template <typename Act>
__device__ __forceinline__ double dot64(const Act* __restrict__ a, const Act* __restrict__ b, int d) {
  constexpr int U = 4, V = 16 / sizeof(Act);
  double s = 0;
  for (int c0 = V * (threadIdx.x & 63); c0 < d; c0 += U * V * kWave) {
    uint4 u[U], v[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int c = c0 + i * V * kWave;
      u[i] = v[i] = make_uint4(0, 0, 0, 0);
      if (c < d) {
        u[i] = *reinterpret_cast<const uint4*>(a + c);
        v[i] = *reinterpret_cast<const uint4*>(b + c);
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t p[4] = {u[i].x, u[i].y, u[i].z, u[i].w}, q[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(Act) == 2) {
          s = fma((double)__uint_as_float(p[j] << 16), (double)__uint_as_float(q[j] << 16), s);
          s = fma((double)__uint_as_float(p[j] & 0xffff0000u), (double)__uint_as_float(q[j] & 0xffff0000u), s);
        } else {
          s = fma((double)__uint_as_float(p[j]), (double)__uint_as_float(q[j]), s);
        }
      }
    }
  }
  return wave_sum(s);
}

// The fp32 forms are the hardware's: one unit each, the exponential's with its argument's two roundings.
__device__ __forceinline__ float exp_of(float v) { return __builtin_amdgcn_exp2f(v * 1.44269504f); }
__device__ __forceinline__ double exp_of(double v) { return exp(v); }
__device__ __forceinline__ float inverse(float v) { return __builtin_amdgcn_rcpf(v); }
__device__ __forceinline__ double inverse(double v) { return 1 / v; }

// A lane's value, in every lane (lane: the same in all of them).
__device__ __forceinline__ int lane_value(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}
__device__ __forceinline__ double lane_value(double v, int lane) {
  const long long b = __double_as_longlong(v);
  const uint32_t lo = __builtin_amdgcn_readlane((int)b, lane), hi = __builtin_amdgcn_readlane((int)(b >> 32), lane);
  return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}

// Largest and second largest value of a group, whose values lie in consecutive lanes.
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
  __device__ Real value(bool top2) const {
    const Real sum = top2 ? first + second : first;
    return sum > -INFINITY ? sum : (Real)-INFINITY;   // +inf and -inf too
  }
};

// A workgroup's tokens between their logits and their choice, in LDS.
struct TokenState {
  double* logit;       // [tokens][stride]
  float* x_norm;       // [tokens]  |x|, rounded up
  float* w_norm;       // [stride]  |w_e|, rounded up
  float* bias;         // [stride]  select_bias, or 0
  uint32_t* refined;   // [tokens][8] bit e: the logit is a 64-bit one
  uint16_t* work;      // (token << 8 | expert) to refine
  int* n_work;
  int16_t* chosen;     // [tokens][8]
  double *top, *sum;   // [tokens]  what a softmax's exponentials are taken less of, and their sum where the weights need it
  int stride;
};

// Experts of a lane in the choice: a group lies in `lanes` consecutive lanes, its
// expert i in lane i % lanes of them, slot i / lanes.
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

// Compare and exchange: the larger value first, of equal ones the lower id (in fp32 equal values decide nothing: their
// intervals overlap).
template <typename Real>
__device__ __forceinline__ void order(Real& v0, Real& e0, int& i0, Real& v1, Real& e1, int& i1) {
  const bool swap = v1 > v0 || (sizeof(Real) == 8 && v1 == v0 && (i1 & 0xffff) < (i0 & 0xffff));
  const Real e = e0;
  const int i = i0;
  const Real least = fmin(v0, v1);
  v0 = fmax(v0, v1);
  v1 = least;
  e0 = swap ? e1 : e0;
  i0 = swap ? i1 : i0;
  e1 = swap ? e : e1;
  i1 = swap ? i : i1;
}

// A lane's slots in descending order, by exchanges of slots (i, j) that leave the larger in i (an odd-even merge sort).
template <int kSlots, typename Exchange>
__device__ __forceinline__ void sort_slots(Exchange exchange) {
  if constexpr (kSlots == 2) exchange(0, 1);
  if constexpr (kSlots >= 4) {
#pragma unroll
    for (int h = 0; h < kSlots; h += 4) {
      exchange(h, h + 1);
      exchange(h + 2, h + 3);
      exchange(h, h + 2);
      exchange(h + 1, h + 3);
      exchange(h + 1, h + 2);
    }
  }
  if constexpr (kSlots == 8) {
    exchange(0, 4);
    exchange(1, 5);
    exchange(2, 6);
    exchange(3, 7);
    exchange(2, 4);
    exchange(3, 5);
    exchange(1, 2);
    exchange(3, 4);
    exchange(5, 6);
  }
}

// Groups that rank before this lane's, whose value is val.
template <typename Real>
__device__ __forceinline__ int groups_before(const GateArgs& a, const ChoiceMap& map, Real val) {
  int before = 0;
  for (int g = 0; g < a.groups; ++g) {
    const Real o = lane_value(val, g * map.lanes);
    before += o > val || (o == val && g < map.group);
  }
  return before;
}

// Token t's choice stands: lane k has its k-th expert, or -1.
template <typename Real>
__device__ __forceinline__ void taken(const GateArgs& a, const TokenState& s, int t, int my_id, Real m) {
  const int lane = threadIdx.x & 63;
  if (lane < 8) s.chosen[t * 8 + lane] = (int16_t)my_id;
  if (a.sigmoid) return;
  if (lane == 0) s.top[t] = m;
  if (a.renorm) return;
  double sum = 0;
  for (int e = lane; e < a.E; e += kWave) sum += exp(s.logit[t * s.stride + e] - m);
  sum = wave_sum(sum);
  if (lane == 0) s.sum[t] = sum;
}

enum Choice { kTaken, kRefine, kInDouble };

// One token's choice by one wave, in fp32 or fp64: taken (into s.chosen); or the experts whose logits it hangs on are
// appended to the work; or (fp32) it hangs on the rounding of refined ones, or on values past the range.
template <typename Real, int kSlots>
__device__ __forceinline__ Choice choose(const GateArgs& a, const TokenState& s, int t) {
  constexpr bool kDouble = sizeof(Real) == 8;
  constexpr Real kNone = -INFINITY;
  constexpr int kOpen = 1 << 16, kMark = 1 << 17;   // beside an expert's id: not refined; the choice hangs on its logit
  const int lane = threadIdx.x & 63;
  const ChoiceMap map(a, lane);
  const double* logit = s.logit + t * s.stride;
  const float xn = s.x_norm[t];
  Real arg[kSlots], c[kSlots], eps[kSlots];   // arg: the exponential's argument; c +- eps: the value that decides
  float delta[kSlots];
  int id[kSlots];                             // -1: no expert
  Real m = kNone;
  float dmax = 0.f;
  bool far = false;
#pragma unroll
  for (int j = 0; j < kSlots; ++j) {
    const int i = map.i0 + j * map.lanes;
    const int e = map.group * map.size + i;
    id[j] = -1;
    delta[j] = 0.f;
    arg[j] = 0;
    if (map.group < a.groups && i < map.size) {
      const double l = logit[e];
      arg[j] = (Real)l;
      far = far || l >= 0x1p120 || (l <= -0x1p120 && l > -INFINITY);
      id[j] = e;
      if (!((s.refined[t * 8 + (e >> 5)] >> (e & 31)) & 1u)) {
        id[j] = e | kOpen;
        const float wn = s.w_norm[e];
        delta[j] = kSumUnits * kUnit * xn * wn;
        // norms that say nothing: past the fp32 range, or lost below it
        if (!(delta[j] < INFINITY) || xn < 0x1p-45f || wn < 0x1p-45f) delta[j] = INFINITY;
      }
      m = fmax(m, arg[j]);
      dmax = fmaxf(dmax, delta[j]);
    }
  }
  if constexpr (!kDouble)
    if (__any(far)) return kInDouble;
  // A softmax's sum z of all exponentials is off by up to dmax of itself. It scales every score alike, so the order
  // of the c is that of z c = exponential + z b: what it moves there, |b| dmax of the sum, is the error that counts.
  const bool all = !a.sigmoid && a.select_bias;
  Real z = 1;
  if (!a.sigmoid) {
    m = wave_max(m);
    // Exponentials are taken less of the largest logit. Rounded to fp32 it is off by one at most up to 2^24; by 64 from 2^30 on,
    // which takes them all to 0 or the largest to infinity.
    if constexpr (!kDouble)
      if (!(fabsf(m) <= 0x1p24f)) return kInDouble;
    dmax = all ? wave_max(dmax) : 0.f;
    z = 0;
#pragma unroll
    for (int j = 0; j < kSlots; ++j)
      if (id[j] >= 0) {
        arg[j] = (Real)(logit[id[j] & 0xffff] - (double)m);   // before it is rounded: the difference may be far smaller
        c[j] = exp_of(arg[j]);
        z += c[j];
      }
    z = wave_sum(z);
  }
  const Real inv_z = kDouble ? z : inverse(z);
#pragma unroll
  for (int j = 0; j < kSlots; ++j) {
    Real v = kNone, err = 0;
    if (id[j] >= 0) {
      const Real score = a.sigmoid ? inverse(1 + exp_of(-arg[j])) : kDouble ? c[j] / z : c[j] * inv_z;
      const Real b = s.bias[id[j] & 0xffff];
      v = score + b;
      // the score's change with its logit: s (1 - s), or s; exp(x) - 1 <= 1.3 x up to 0.5
      const Real part = a.sigmoid ? score * (1 - score) : score;
      err = part * (Real)(1.3f * delta[j]);
      if (all) err += fabs(b) * (Real)(1.3f * dmax);
      if (!(delta[j] <= 0.5f) || (all && !(dmax <= 0.5f))) err = INFINITY;
      if constexpr (!kDouble) {
        // The exponential (one unit) and its argument's roundings (to fp32, of log2(e), of the product); 1 + it and the
        // inverse, or the product with one; the sum with b; a softmax's sum of up to eight and six additions matters
        // next to a bias, as above.
        const float own = 2 + 2 * fminf(fabsf(arg[j]), 200.f);   // past it the score is 0 or 1, and 0 * infinity no number
        err += kUnit * (score * (a.sigmoid ? (1 - score) * own + 3 : own + 4) + fabsf(b) * (all ? 17 : 1));
        err = fmaxf(err, 0x1p-120f);           // scores lost below the fp32 range
      }
      if (!(v > kNone)) v = kNone;
      if (v == kNone || v == INFINITY) err = 0;   // by the bias, whatever the score
    }
    c[j] = v;
    eps[j] = err;
  }

  bool hangs = false;   // experts may be marked
  // what a refined logit leaves open: in fp32 the evaluation, in fp64 a softmax's sum next to a bias
  auto unsure = [&](int i) { return i >= 0 && (!kDouble || (i & kOpen) || (all && dmax > 0.f)); };
  if (a.groups > 1) {
    Top2<Real> vc;
#pragma unroll
    for (int j = 0; j < kSlots; ++j) vc.add(c[j]);
    vc.join(map.lanes);
    const Real val = vc.value(a.top2);
    Real lo, hi, least;    // ends of the group's value, and what a member needs to count in it
    if constexpr (kDouble) {
      Top2<Real> vlo, vhi;
#pragma unroll
      for (int j = 0; j < kSlots; ++j) {
        vlo.add(c[j] - eps[j]);
        vhi.add(c[j] + eps[j]);
      }
      vlo.join(map.lanes);
      vhi.join(map.lanes);
      lo = vlo.value(a.top2);
      hi = vhi.value(a.top2);
      least = a.top2 ? vlo.second : vlo.first;
    } else {
      // wider ends that cost one exchange
      Real e = 0;
#pragma unroll
      for (int j = 0; j < kSlots; ++j) e = fmaxf(e, eps[j]);
      e = wave_max(e);
      lo = val - (a.top2 ? 2 * e : e);
      hi = val + (a.top2 ? 2 * e : e);
      least = (a.top2 ? vc.second : vc.first) - e;
    }
    const int before = groups_before(a, map, val);
    const bool real = map.group < a.groups, kept = real && before < a.group_topk;
    if (a.group_topk < a.groups) {
      const Real floor = -wave_max(kept ? -lo : kNone);      // least value of a kept group
      const Real ceil = wave_max(real && !kept ? hi : kNone);
      if (!(floor > ceil)) {
        hangs = true;
        const bool near = kept ? !(lo > ceil) : real && !(hi < floor);
#pragma unroll
        for (int j = 0; j < kSlots; ++j)
          if (near && unsure(id[j]) && c[j] > kNone && !(c[j] + eps[j] < least)) id[j] |= kMark;
      }
    }
#pragma unroll
    for (int j = 0; j < kSlots; ++j)
      if (!kept) {
        c[j] = kNone;
        eps[j] = 0;
      }
  }

  // a lane's experts in descending order
  sort_slots<kSlots>([&](int i, int j) { order(c[i], eps[i], id[i], c[j], eps[j], id[j]); });
  // K rounds: the largest of the lanes' first ones, which its lane then drops; lane k keeps round k's
  int my_id = -1;
  Real my_lo = kNone, my_hi = kNone;
  for (int k = 0; k < a.K; ++k) {
    const Real top = wave_max(c[0]);
    if (!(top > kNone)) break;
    const uint64_t equal = __ballot(c[0] == top);
    int owner = __ffsll((unsigned long long)equal) - 1;
    if (kDouble && __popcll(equal) > 1) {
      const int e = c[0] == top ? id[0] & 0xffff : kMaxExperts;
      owner = __ffsll((unsigned long long)__ballot(e == wave_min(e))) - 1;
    }
    const Real err = lane_value(eps[0], owner);
    const int i = lane_value(id[0], owner);
    if (lane == k) {
      my_id = i;
      my_lo = top - err;
      my_hi = top + err;
    }
    if (lane == owner) {
#pragma unroll
      for (int j = 0; j + 1 < kSlots; ++j) {
        c[j] = c[j + 1];
        eps[j] = eps[j + 1];
        id[j] = id[j + 1];
      }
      c[kSlots - 1] = kNone;
      eps[kSlots - 1] = 0;
      id[kSlots - 1] = -1;
    }
  }
  // every pick has to lie above all that rank after it
  Real above = kNone;
#pragma unroll
  for (int j = 0; j < kSlots; ++j) above = fmax(above, c[j] + eps[j]);
  above = fmax(wave_max(above), after(my_hi));
  const uint64_t bad = __ballot(my_id >= 0 && !(my_lo > above));
  if (bad) {
    // such picks, and what ranks after the first of them and may lie above the lowest of their lower ends
    const Real lo = -wave_max(bad >> lane & 1 ? -my_lo : kNone);
    hangs = true;
#pragma unroll
    for (int j = 0; j < kSlots; ++j)
      if (unsure(id[j]) && c[j] > kNone && !(c[j] + eps[j] < lo)) id[j] |= kMark;
    if (lane >= __ffsll((unsigned long long)bad) - 1 && unsure(my_id) && !(my_hi < lo)) my_id |= kMark;
  }
  if (hangs) {
    bool on_open = my_id >= 0 && (my_id & kMark) && (my_id & kOpen), marked = my_id >= 0 && (my_id & kMark);
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
      const bool mark = id[j] >= 0 && (id[j] & kMark);
      marked = marked || mark;
      on_open = on_open || (mark && (id[j] & kOpen));
    }
    if (__any(marked)) {
      const bool some = __any(on_open);
      if (!kDouble && !some) return kInDouble;
      // the marked ones; if these are refined, every logit of the sum
      auto append = [&](int i) {
        if (i >= 0 && (i & kOpen) && (!some || (i & kMark))) s.work[atomicAdd(s.n_work, 1)] = (uint16_t)(t << 8 | (i & 0xff));
      };
      append(my_id);
#pragma unroll
      for (int j = 0; j < kSlots; ++j) append(id[j]);
      return kRefine;
    }
  }

  taken(a, s, t, my_id >= 0 ? my_id & 0xffff : -1, m);
  return kTaken;
}

// Ids and weights of the workgroup's n tokens once all are chosen, in fp64 from the logits of the chosen: a thread each
// (by each token's own wave: 66.0 -> 64.3 us with the hardware's exponentials above, 16384 tokens, 16 experts).
__device__ __forceinline__ void write_chosen(const GateArgs& a, const TokenState& s, int tok0, int n) {
  for (int i = threadIdx.x; i < 8 * n; i += blockDim.x) {
    const int t = i >> 3, k = i & 7;
    const int id = k < a.K ? s.chosen[i] : -1;
    double sk = 0;
    if (id >= 0) {
      const double l = s.logit[t * s.stride + id];
      sk = a.sigmoid ? 1 / (1 + exp(-l)) : exp(l - s.top[t]);
    }
    double total = a.sigmoid ? 1 : s.sum[t];
    if (a.renorm) {
      total = sk;
#pragma unroll
      for (int off = 4; off >= 1; off >>= 1) total += __shfl_xor(total, off);
    }
    if (k < a.K) {
      const long at = (long)(tok0 + t) * a.K + k;
      a.topk_ids[at] = id;
      a.topk_w[at] = total > 0 ? (float)(sk / total * a.scale) : 0.f;
    }
  }
}

// The choice of the workgroup's tokens (kTok of them at most, n present) once their logits lie in LDS. All waves call
// it, after a barrier; wave v takes tokens v, v + kWaves, ...
template <typename Act, int kWaves, int kTok, int kSlots>
__device__ __forceinline__ void choose_all(const GateArgs& a, const TokenState& s, int tok0, int n) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr int kMine = (kTok + kWaves - 1) / kWaves;
  uint32_t pending = 0;
#pragma unroll
  for (int i = 0; i < kMine; ++i)
    if (wave + kWaves * i < n) pending |= 1u << i;
  for (;;) {
    // logits that are no numbers in fp32 are in the work before any choice
    const int work = *s.n_work;
    if (work > 0) {
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
    }
    __syncthreads();   // every wave has read the number before one adds to it
#pragma unroll 1
    for (int i = 0; i < kMine; ++i) {
      if (!(pending >> i & 1)) continue;
      const int t = wave + kWaves * i;
      Choice c = choose<float, kSlots>(a, s, t);
      if (c == kInDouble) c = choose<double, kSlots>(a, s, t);
      if (c == kTaken) pending &= ~(1u << i);
    }
    __syncthreads();
    if (*s.n_work == 0) break;   // a token that is not taken has added to it
  }
  write_chosen(a, s, tok0, n);
}

// A logit's sum, written with its bias, once the norms are known. What is no number, or near the end of fp32's range, is
// left to fp64; the zeros of a token or an expert of zeros (a padded batch) are exact as they are.
__device__ __forceinline__ void put_logit(const GateArgs& a, const TokenState& s, int t, int e, double v) {
  s.logit[t * s.stride + e] = a.router_bias ? v + a.router_bias[e] : v;
  if (!(fabs(v) < 0x1p120)) s.work[atomicAdd(s.n_work, 1)] = (uint16_t)(t << 8 | e);
  else if (v == 0 && (s.x_norm[t] == 0.f || s.w_norm[e] == 0.f)) atomicOr(&s.refined[t * 8 + (e >> 5)], 1u << (e & 31));
}

// ------------------------------------------------------------------ logits
// A block is 128 bytes of a row of x or router_w: 64 bf16 or 32 fp32 elements.
// Lane l of a wave holds the 32 bytes at 32*(l/16) of row l%16, of x and of w alike.
// Rows go through LDS: direct loads of 8 rows an instruction, whose eight lanes a
// row read one cache line (lanes that read their MFMA rows themselves touch 64 lines an
// instruction, and stay at 14 bytes a cycle and CU). The 16-byte pieces of a row are XOR-swizzled by its number.
constexpr int kBlockBytes = 128;
constexpr int kTileBytes = 16 * kBlockBytes;   // a block of 16 rows

struct Block {
  uint4 h[2];
};

// This lane's part of a block of 16 rows in LDS.
__device__ __forceinline__ Block lds_block(const uint8_t* tile) {
  const int li = threadIdx.x & 15, lg = (threadIdx.x & 63) >> 4;
  Block b;
#pragma unroll
  for (int h = 0; h < 2; ++h) b.h[h] = *reinterpret_cast<const uint4*>(tile + li * kBlockBytes + 16 * ((2 * lg + h) ^ (li & 7)));
  return b;
}

// The block's sums x . w of 16 rows by 16, added to acc in fp64: one sum of two MFMAs (bf16), two of four (fp32). The
// conversions and additions are what the sums cost: one a MFMA took 1.6 times as long with 256 experts.
template <typename Act>
__device__ __forceinline__ void add_block(const Block& x, const Block& w, double (&acc)[4]) {
  f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (sizeof(Act) == 2) {
      p = mfma_bf16(as_bf16x8(x.h[h]), as_bf16x8(w.h[h]), p);
      if (h == 0) continue;
    } else {
      const f32x4 u = __builtin_bit_cast(f32x4, x.h[h]), v = __builtin_bit_cast(f32x4, w.h[h]);
      p = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < 4; ++j) p = mfma_f32(u[j], v[j], p);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[r] += (double)p[r];
  }
}

// The squares of 16 rows, block by block: with bf16 the diagonal of a tile rows . rows (an MFMA costs its wave
// nothing next to the sums' additions), with fp32 a lane's share of its row. A sum of 0 stands for a row of zeros alone:
// where fp32 loses the squares (elements below 2^-63) it is kLost, which no choice takes for a norm (1 to 2% of the time for 256
// experts; reading such rows again instead: 50 -> 66 us for 16384 tokens of 16 experts, half of them padding).
template <typename Act>
struct Squares {
  static constexpr uint32_t kMagnitudes = sizeof(Act) == 2 ? 0x7fff7fffu : 0x7fffffffu;   // -0 is a zero
  static constexpr float kLost = 0x1p-120f;
  f32x4 tile = {0.f, 0.f, 0.f, 0.f};
  float mine = 0.f;
  uint32_t bits = 0;   // of this lane's share of its row
  __device__ void add(const Block& b) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      bits |= b.h[h].x | b.h[h].y;
      bits |= b.h[h].z | b.h[h].w;
      if constexpr (sizeof(Act) == 2) {
        tile = mfma_bf16(as_bf16x8(b.h[h]), as_bf16x8(b.h[h]), tile);
      } else {
        const f32x4 u = __builtin_bit_cast(f32x4, b.h[h]);
#pragma unroll
        for (int j = 0; j < 4; ++j) mine += u[j] * u[j];
      }
    }
  }
  // out[row], by the lanes that hold a row's sum
  __device__ void store(float* out) {
    const int li = threadIdx.x & 15, lg = (threadIdx.x & 63) >> 4;
    bool holds = lg == 0;
    if constexpr (sizeof(Act) == 2) {
      holds = lg == li >> 2;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (4 * lg + r == li) mine = tile[r];
    } else {
      mine += __shfl_xor(mine, 16);
      mine += __shfl_xor(mine, 32);
    }
    if (__any(holds && mine == 0.f)) {
      bits |= __shfl_xor(bits, 16);
      bits |= __shfl_xor(bits, 32);
      if (mine == 0.f && (bits & kMagnitudes)) mine = kLost;
    }
    if (holds) out[li] = mine;
  }
};

// A norm from its square, whose own sum is off by less than a thousandth, rounded up.
__device__ __forceinline__ float norm_of(float square) { return sqrtf(square) * 1.01f; }

// Shape of a logits tile: NEB blocks of 16 experts by TB blocks of 16 tokens by KS slices of the hidden dimension (block b
// belongs to slice b % KS); wave (eb, ks) has expert block eb and slice ks, and all token blocks. A step is a
// block of every slice; its rows lie in one of D stages of LDS, requested D - 1 steps ahead.
template <int NEB, int TB, int kWaves, int D>
struct Tile {
  static constexpr int KS = kWaves / NEB;
  static constexpr int EP = 16 * NEB;
  static constexpr int TOK = 16 * TB;
  static constexpr int kStage = (kWaves + KS * TB) * kTileBytes;
  // the sums of the slices, then the choice's state, take the stages' place
  static constexpr int kSums = KS * TOK * EP * 8;
  static constexpr int kState = TOK * EP * (8 + 2);
  static constexpr int kLds = D * kStage > kSums ? (D * kStage > kState ? D * kStage : kState) : (kSums > kState ? kSums : kState);
};

// Sums of x . w over the steps [s0, s1) of one workgroup's tokens, in fp64: sum[ks][token][expert] in LDS (lds, after a
// barrier), the squares of the rows in x_sq [KS][TOK] and w_sq [KS][EP].
template <typename Act, int NEB, int TB, int kWaves, int D>
__device__ __forceinline__ void tile_logits(const GateArgs& a, int tok0, int n, int s0, int s1, uint8_t* lds, float* x_sq,
                                            float* w_sq) {
  using S = Tile<NEB, TB, kWaves, D>;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int li = lane & 15;
  const int lg = lane >> 4;
  const int eb = wave % NEB, ks = wave / NEB;
  const long row_bytes = (long)a.d * sizeof(Act);
  const int blocks = (int)(row_bytes / kBlockBytes);

  // sources: lane l of a load reads 16 bytes of row l/8 of eight rows, at the place that its LDS slot must hold
  const int r8 = lane >> 3;
  const uint32_t piece = 16u * (uint32_t)((lane & 7) ^ r8);
  const uint8_t* xb = static_cast<const uint8_t*>(a.x) + tok0 * row_bytes;      // offsets below 32 rows: 32 bits
  const uint8_t* wb = static_cast<const uint8_t*>(a.router_w);                  // 256 rows of 65536 at most
  uint32_t w_off[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) w_off[h] = (uint32_t)(min(eb * 16 + h * 8 + r8, a.E - 1) * row_bytes) + piece;
  constexpr int XN = 2 * TB;                          // loads of a slice's token rows, dealt to its NEB waves
  constexpr int XI = (XN + NEB - 1) / NEB;
  uint32_t x_off[XI];
#pragma unroll
  for (int i = 0; i < XI; ++i) x_off[i] = (uint32_t)(min((eb + NEB * i) * 8 + r8, n - 1) * row_bytes) + piece;
  const int x_loads = eb < XN ? (XN - eb + NEB - 1) / NEB : 0;

  // Workgroups start at different steps: rows a power of two apart lie in the same memory channels, which workgroups in
  // step would ask for all at once (16384 tokens, 16 experts: 64 -> 52 us without the choice). The sums of fp32 sums
  // lose nothing in fp64 unless one is 2^-27 of the others, so their order does not show.
  const int turn = (blockIdx.x >> 3) % (s1 - s0);
  auto turned = [&](int st) { return st + turn >= s1 ? st + turn - (s1 - s0) : st + turn; };
  const uint32_t base = lds_addr(lds);
  auto issue = [&](int st) {
    // past the end the last step again, so that a wave's loads stay countable
    const uint32_t off = (uint32_t)min(turned(min(st, s1 - 1)) * S::KS + ks, blocks - 1) * kBlockBytes;
    const uint32_t stage = base + (uint32_t)(st % D) * S::kStage;
#pragma unroll
    for (int h = 0; h < 2; ++h) dma16(wb, w_off[h] + off, stage + wave * kTileBytes + h * 1024);
#pragma unroll
    for (int i = 0; i < XI; ++i)
      if (i < x_loads) dma16(xb, x_off[i] + off, stage + (kWaves + ks * TB) * kTileBytes + (eb + NEB * i) * 1024);
  };
  // all but the loads of the last `steps` steps have landed
  auto wait = [&](auto steps) {
    constexpr int K = decltype(steps)::value;
    if constexpr (K == 0) __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));
    else if (x_loads == XI) __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(K * (2 + XI)));
    else __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(K * (2 + XI - 1)));
  };

  double acc[TB][4];
#pragma unroll
  for (int tb = 0; tb < TB; ++tb)
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[tb][r] = 0;
  Squares<Act> xs[TB], ws;
#pragma unroll
  for (int i = 0; i < D - 1; ++i) issue(s0 + i);
  for (int st = s0; st < s1; ++st) {
    // this step's rows have landed, and every wave is past the stage that the next ones overwrite
    asm volatile("" ::: "memory");
    wait(int_constant<D - 2>{});
    __builtin_amdgcn_s_barrier();
    issue(st + D - 1);
    if (turned(st) * S::KS + ks < blocks) {
      const uint8_t* stage = lds + (st % D) * S::kStage;
      const Block w = lds_block(stage + wave * kTileBytes);
      ws.add(w);
#pragma unroll
      for (int tb = 0; tb < TB; ++tb) {
        const Block x = lds_block(stage + (kWaves + ks * TB + tb) * kTileBytes);
        if (eb == tb % NEB) xs[tb].add(x);
        add_block<Act>(x, w, acc[tb]);
      }
    }
  }
  __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));   // the loads past the end too
  __syncthreads();
  // lane l holds tokens 16*tb + 4*lg + r of expert 16*eb + li
  double* sum = reinterpret_cast<double*>(lds) + ks * S::TOK * S::EP;
#pragma unroll
  for (int tb = 0; tb < TB; ++tb) {
#pragma unroll
    for (int r = 0; r < 4; ++r) sum[(tb * 16 + 4 * lg + r) * S::EP + eb * 16 + li] = acc[tb][r];
    if (eb == tb % NEB) xs[tb].store(x_sq + ks * S::TOK + tb * 16);
  }
  ws.store(w_sq + ks * S::EP + eb * 16);
  __syncthreads();
}

// What a workgroup's choice needs besides the logits.
template <int TOK, int EP>
struct ChoiceLds {
  double top[TOK], sum[TOK];
  float x_norm[TOK], w_norm[EP], bias[EP];
  uint32_t refined[TOK][8];
  int n_work;
  int16_t chosen[TOK * 8];
};

// Logits and choice of 16*TB tokens in one workgroup.
template <typename Act, int NEB, int TB, int kWaves, int D, int kSlots>
__global__ __launch_bounds__(kWaves* kWave, 4) void route_gated_kernel(GateArgs a, int tpw) {
  using S = Tile<NEB, TB, kWaves, D>;
  constexpr int EP = S::EP, TOK = S::TOK, KS = S::KS;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S::kLds];
  __shared__ float x_sq[KS * TOK], w_sq[KS * EP];
  __shared__ ChoiceLds<TOK, EP> c;
  const int tok0 = blockIdx.x * tpw;
  const int n = min(tpw, a.T - tok0);
  const int blocks = (int)((long)a.d * sizeof(Act) / kBlockBytes);
  if (threadIdx.x < TOK * 8) (&c.refined[0][0])[threadIdx.x] = 0;
  if (threadIdx.x == 0) c.n_work = 0;
  if (threadIdx.x < a.E) c.bias[threadIdx.x] = a.select_bias ? a.select_bias[threadIdx.x] : 0.f;
  tile_logits<Act, NEB, TB, kWaves, D>(a, tok0, n, 0, (blocks + KS - 1) / KS, lds, x_sq, w_sq);

  // the slices' sums, each thread's before any is overwritten
  constexpr int kPer = (TOK * EP + kWaves * kWave - 1) / (kWaves * kWave);
  double v[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int at = threadIdx.x + i * kWaves * kWave;
    v[i] = 0;
    if (at < TOK * EP)
#pragma unroll
      for (int k = 0; k < KS; ++k) v[i] += reinterpret_cast<const double*>(lds)[k * TOK * EP + at];
  }
  for (int i = threadIdx.x; i < TOK + EP; i += kWaves * kWave) {
    float q = 0.f;
#pragma unroll
    for (int k = 0; k < KS; ++k) q += i < TOK ? x_sq[k * TOK + i] : w_sq[k * EP + i - TOK];
    if (i < TOK) c.x_norm[i] = norm_of(q);
    else c.w_norm[i - TOK] = norm_of(q);
  }
  __syncthreads();
  const TokenState s = {reinterpret_cast<double*>(lds), c.x_norm, c.w_norm, c.bias, &c.refined[0][0],
                        reinterpret_cast<uint16_t*>(lds + TOK * EP * 8), &c.n_work, c.chosen, c.top, c.sum, EP};
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int at = threadIdx.x + i * kWaves * kWave, t = at / EP, e = at % EP;
    if (t < n && e < a.E) put_logit(a, s, t, e, v[i]);
  }
  __syncthreads();
  choose_all<Act, kWaves, TOK, kSlots>(a, s, tok0, n);
}

// ------------------------------------------------------------------ few tokens
// One workgroup of the fused kernel walks the whole of a long row step by step, each a trip to memory. Few tokens split
// the row over workgroups instead: one kernel writes the splits' sums and squares to the workspace, the next adds them
// and chooses.
struct SplitSums {
  double* sum;          // [splits][T][E]
  float *x_sq, *w_sq;   // [splits][T], [splits][E]
  int splits, steps;    // steps of a split
};

template <typename Act, int NEB>
__global__ __launch_bounds__(16 * kWave, 4) void route_logits_kernel(GateArgs a, SplitSums p) {
  constexpr int kWaves = 16, D = 2;
  using S = Tile<NEB, 1, kWaves, D>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S::kLds];
  __shared__ float x_sq[S::KS * S::TOK], w_sq[S::KS * S::EP];
  const int tok0 = blockIdx.x * 16, split = blockIdx.y;
  const int n = min(16, a.T - tok0);
  const int blocks = (int)((long)a.d * sizeof(Act) / kBlockBytes);
  const int nsteps = (blocks + S::KS - 1) / S::KS;
  // every split has a step: splits = ceil(nsteps / steps)
  tile_logits<Act, NEB, 1, kWaves, D>(a, tok0, n, split * p.steps, min((split + 1) * p.steps, nsteps), lds, x_sq, w_sq);
  for (int i = threadIdx.x; i < n * S::EP; i += kWaves * kWave) {
    const int t = i / S::EP, e = i % S::EP;
    if (e >= a.E) continue;
    double v = 0;
#pragma unroll
    for (int k = 0; k < S::KS; ++k) v += reinterpret_cast<const double*>(lds)[k * S::TOK * S::EP + i];
    p.sum[((long)split * a.T + tok0 + t) * a.E + e] = v;
  }
  for (int i = threadIdx.x; i < n + a.E; i += kWaves * kWave) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < S::KS; ++k) v += i < n ? x_sq[k * S::TOK + i] : w_sq[k * S::EP + i - n];
    if (i < n) p.x_sq[(long)split * a.T + tok0 + i] = v;
    else if (blockIdx.x == 0) p.w_sq[(long)split * a.E + i - n] = v;
  }
}

template <typename Act, int EP, int kSlots>
__global__ __launch_bounds__(4 * kWave) void route_choose_kernel(GateArgs a, SplitSums p) {
  constexpr int kWaves = 4;
  __shared__ double logit[EP];
  __shared__ uint16_t work[EP];
  __shared__ ChoiceLds<1, EP> c;
  const int t = blockIdx.x;
  if (threadIdx.x < 8) c.refined[0][threadIdx.x] = 0;
  if (threadIdx.x == 0) c.n_work = 0;
  __syncthreads();
  const TokenState s = {logit, c.x_norm, c.w_norm, c.bias, &c.refined[0][0], work, &c.n_work, c.chosen, c.top, c.sum, EP};
  static_assert(EP <= kWaves * kWave, "an expert a thread");
  const int e = threadIdx.x;
  double v = 0;
  if (e < a.E) {
    float q = 0.f;
#pragma unroll 8
    for (int k = 0; k < p.splits; ++k) {
      v += p.sum[((long)k * a.T + t) * a.E + e];
      q += p.w_sq[(long)k * a.E + e];
    }
    c.w_norm[e] = norm_of(q);
    c.bias[e] = a.select_bias ? a.select_bias[e] : 0.f;
  }
  if (threadIdx.x >= (kWaves - 1) * kWave) {
    float q = 0.f;
    for (int k = threadIdx.x & 63; k < p.splits; k += kWave) q += p.x_sq[(long)k * a.T + t];
    q = wave_sum(q);
    if ((threadIdx.x & 63) == 0) c.x_norm[0] = norm_of(q);
  }
  __syncthreads();
  if (e < a.E) put_logit(a, s, 0, e, v);
  __syncthreads();
  choose_all<Act, kWaves, 1, kSlots>(a, s, t, 1);
}

// Blocks of 16 experts of a tile, and the splits of few tokens' rows; splits 0: the fused kernel.
int expert_blocks(int E) { return E <= 16 ? 1 : E <= 32 ? 2 : E <= 64 ? 4 : E <= 128 ? 8 : 16; }
SplitSums split_of(int T, int d, int E, bool act_bf16) {
  SplitSums p = {};
  const int blocks = (int)((long)d * (act_bf16 ? 2 : 4) / kBlockBytes), slices = 16 / expert_blocks(E);
  const int nsteps = (blocks + slices - 1) / slices, tiles = (T + 15) / 16;
  if (T == 0 || T > kSplitTokens || nsteps < kSplitSteps) return p;
  const int most = 256 / tiles;                      // a workgroup a CU
  p.steps = (nsteps + most - 1) / most;
  p.splits = (nsteps + p.steps - 1) / p.steps;
  return p;
}

template <typename Act, int NEB, int kSlots>
void launch_split(const GateArgs& a, const SplitSums& p, hipStream_t stream) {
  hipLaunchKernelGGL((route_logits_kernel<Act, NEB>), dim3((a.T + 15) / 16, p.splits), dim3(16 * kWave), 0, stream, a, p);
  hipLaunchKernelGGL((route_choose_kernel<Act, 16 * NEB, kSlots>), dim3(a.T), dim3(4 * kWave), 0, stream, a, p);
}

template <typename Act, int NEB, int TB, int kWaves, int kSlots>
void launch_tile(const GateArgs& a, int tpw, hipStream_t stream) {
  constexpr int D = NEB == 1 ? 2 : 3;
  hipLaunchKernelGGL((route_gated_kernel<Act, NEB, TB, kWaves, D, kSlots>), dim3((a.T + tpw - 1) / tpw), dim3(kWaves * kWave), 0,
                     stream, a, tpw);
}

template <typename Act, int NEB, int kSlots>
void launch_experts(const GateArgs& a, hipStream_t stream) {
  SplitSums p = split_of(a.T, a.d, a.E, a.act_bf16);
  if (p.splits && a.workspace) {
    p.sum = static_cast<double*>(a.workspace);
    p.x_sq = reinterpret_cast<float*>(p.sum + (long)p.splits * a.T * a.E);
    p.w_sq = p.x_sq + (long)p.splits * a.T;
    return launch_split<Act, NEB, kSlots>(a, p, stream);
  }
  if constexpr (NEB <= 4) {
    // As few tokens a workgroup as leave no CU without one, so that a small batch's reads of router_w are spread. Few
    // workgroups: the most waves each; many: two workgroups a CU, one of which loads while the other chooses.
    const int tpw = min(16, (a.T + 255) / 256);
    if ((a.T + tpw - 1) / tpw <= 256) launch_tile<Act, NEB, 1, 16, kSlots>(a, tpw, stream);
    else launch_tile<Act, NEB, 1, 8, kSlots>(a, tpw, stream);
  } else if (a.T <= 16 * 256) {
    launch_tile<Act, NEB, 1, 16, kSlots>(a, 16, stream);
  } else {
    // tokens spread over the CUs, which leaves each fewer to choose for (5000 tokens, 256 experts: 76.3 -> 73.9 us; up to
    // 4096 it gains nothing: a wave has one token at most, 2000 tokens 55.5 -> 56.5 us)
    launch_tile<Act, NEB, 2, 16, kSlots>(a, min(32, (a.T + 255) / 256), stream);
  }
}

// Slots of a lane: a group's experts over its lanes, of which there are more than 32 / groups, so at most E / 32: 4 for 128
// experts; for 256 experts 8, or 4 if the groups are a power of two, as they mostly are.
template <typename Act>
void launch(const GateArgs& a, hipStream_t stream) {
  int lanes = kWave;
  while (lanes * a.groups > kWave) lanes >>= 1;
  if (a.E <= 16) launch_experts<Act, 1, 1>(a, stream);
  else if (a.E <= 32) launch_experts<Act, 2, 1>(a, stream);
  else if (a.E <= 64) launch_experts<Act, 4, 2>(a, stream);
  else if (a.E <= 128) launch_experts<Act, 8, 4>(a, stream);
  else if (a.E / a.groups <= 4 * lanes) launch_experts<Act, 16, 4>(a, stream);
  else launch_experts<Act, 16, 8>(a, stream);
}

}  // namespace

size_t route_gated_workspace(int T, int d, int E, bool act_bf16) {
  const SplitSums p = split_of(T, d, E, act_bf16);
  return (size_t)p.splits * ((size_t)T * E * 8 + (size_t)(T + E) * 4);
}

hipError_t launch_route_gated(const GateArgs& a, hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  if (a.act_bf16) launch<__bf16>(a, stream);
  else launch<float>(a, stream);
  return hipGetLastError();
}

}  // namespace moe
