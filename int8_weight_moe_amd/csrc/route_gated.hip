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
// Which experts are taken is decided by values in 64 bits.
#include "device_common.h"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kMaxExperts = 256;
constexpr int kSlots = kMaxExperts / kWave;   // experts of a lane: lane + 64*j
constexpr int kWaves = 4;

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

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  return v;
}
__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = fmax(v, __shfl_xor(v, off));
  return v;
}

// a . b over d elements by one wave; the same value in every lane.
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

// The choice for one token by one wave, from the logits of the lane's experts.
__device__ __forceinline__ void choose(const GateArgs& a, const double (&l)[kSlots], double* choice, double* value,
                                       int32_t* ids, float* w) {
  const int lane = threadIdx.x & 63;
  double s[kSlots], c[kSlots];
  if (a.sigmoid) {
#pragma unroll
    for (int j = 0; j < kSlots; ++j) s[j] = 1 / (1 + exp(-l[j]));
  } else {
    double m = -INFINITY, z = 0;
#pragma unroll
    for (int j = 0; j < kSlots; ++j)
      if (lane + kWave * j < a.E) m = fmax(m, l[j]);
    m = wave_max(m);
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
      s[j] = lane + kWave * j < a.E ? exp(l[j] - m) : 0;
      z += s[j];
    }
    z = wave_sum(z);
#pragma unroll
    for (int j = 0; j < kSlots; ++j) s[j] /= z;
  }
#pragma unroll
  for (int j = 0; j < kSlots; ++j) {
    const int e = lane + kWave * j;
    c[j] = -INFINITY;
    if (e < a.E) {
      const double v = a.select_bias ? s[j] + a.select_bias[e] : s[j];
      if (v > -INFINITY) c[j] = v;
    }
  }
  if (a.groups > 1) {
    const int size = a.E / a.groups;
#pragma unroll
    for (int j = 0; j < kSlots; ++j)
      if (lane + kWave * j < a.E) choice[lane + kWave * j] = c[j];
    __builtin_amdgcn_wave_barrier();
    __threadfence_block();
    if (lane < a.groups) {
      double m1 = -INFINITY, m2 = -INFINITY;
      for (int i = 0; i < size; ++i) {
        const double v = choice[lane * size + i];
        m2 = fmax(m2, fmin(m1, v));
        m1 = fmax(m1, v);
      }
      value[lane] = a.top2 ? m1 + m2 : m1;
    }
    __builtin_amdgcn_wave_barrier();
    __threadfence_block();
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
      const int e = lane + kWave * j;
      if (e < a.E) {
        const int g = e / size;
        int before = 0;
        for (int i = 0; i < a.groups; ++i) before += value[i] > value[g] || (value[i] == value[g] && i < g);
        if (before >= a.group_topk) c[j] = -INFINITY;
      }
    }
  }
  double total = 0, mine = 0;
  int my_id = -1;
  for (int k = 0; k < a.K; ++k) {
    double v = c[0], sv = s[0];
    int e = lane;
#pragma unroll
    for (int j = 1; j < kSlots; ++j)
      if (c[j] > v) {
        v = c[j];
        sv = s[j];
        e = lane + kWave * j;
      }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
      const double ov = __shfl_xor(v, off), os = __shfl_xor(sv, off);
      const int oe = __shfl_xor(e, off);
      if (ov > v || (ov == v && oe < e)) {
        v = ov;
        sv = os;
        e = oe;
      }
    }
    const bool taken = v > -INFINITY;
    if (!taken) sv = 0;
    total += sv;
    if (lane == k) {
      mine = sv;
      my_id = taken ? e : -1;
    }
#pragma unroll
    for (int j = 0; j < kSlots; ++j)
      if (e == lane + kWave * j) c[j] = -INFINITY;
  }
  if (lane < a.K) {
    if (a.renorm) mine = total > 0 ? mine / total : 0;
    ids[lane] = my_id;
    w[lane] = (float)(mine * a.scale);
  }
}

template <typename Act>
__global__ __launch_bounds__(kWaves* kWave) void route_gated_kernel(GateArgs a) {
  __shared__ double logit[kMaxExperts], value[kWave];
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const long t = blockIdx.x;
  const Act* x = static_cast<const Act*>(a.x) + t * a.d;
  const Act* wr = static_cast<const Act*>(a.router_w);
  for (int e = wave; e < a.E; e += kWaves) {
    const double v = dot64(x, wr + (long)e * a.d, a.d);
    if (lane == 0) logit[e] = a.router_bias ? v + a.router_bias[e] : v;
  }
  __syncthreads();
  if (wave > 0) return;
  double l[kSlots];
#pragma unroll
  for (int j = 0; j < kSlots; ++j) l[j] = lane + kWave * j < a.E ? logit[lane + kWave * j] : 0;
  choose(a, l, logit, value, a.topk_ids + t * a.K, a.topk_w + t * a.K);
}

}  // namespace

hipError_t launch_route_gated(const GateArgs& a, hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  if (a.act_bf16) {
    hipLaunchKernelGGL((route_gated_kernel<__bf16>), dim3(a.T), dim3(kWaves * kWave), 0, stream, a);
  } else {
    hipLaunchKernelGGL((route_gated_kernel<float>), dim3(a.T), dim3(kWaves * kWave), 0, stream, a);
  }
  return hipGetLastError();
}

}  // namespace moe
