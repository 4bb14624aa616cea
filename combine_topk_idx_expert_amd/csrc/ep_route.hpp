// ep_route.hpp -- routing to experts: scores, a balance bias, expert groups,
// top-k and renormalised weights, and the gradient of the weights.
//
// The choice of the experts is that of exact arithmetic on the scores plus
// the bias, ties to the lowest expert; the kernels decide it in 64 bits, where
// scores that fp32 would merge still differ.  Without a bias, and without
// sums of scores over a group, the logits order the experts as the scores do
// and are compared directly.
#pragma once

#include <hip/hip_fp16.h>

#include "ep_device.hpp"

namespace ep {

constexpr int kMaxRouteGroups = 64;  // one lane a group

struct RouteArgs {
  const void* logits;    // [T][stride], E used
  int64_t stride;        // elements between rows
  const float* bias;     // [E] or null
  const uint8_t* mask;   // [T] or null; 0: the token is not routed
  int64_t* idx;          // [T][K]
  float* w;              // [T][K]
  int T, E, K, G, TG;
  int sigmoid;           // 1: sigmoid scores, 0: softmax
  int top2;              // group score: 1 sum of the two largest, 0 the largest
  int renorm;
  float scale;
};

struct RouteBwdArgs {
  const void* logits;
  int64_t stride;
  const int64_t* idx;    // [T][K]
  const float* gw;       // [T][K] gradient of the weights
  void* grad;            // [T][E], the logits' type
  int T, E, K;
  int sigmoid, renorm;
  float scale;
};

struct F32 {
  typedef float type;
  static __device__ __forceinline__ float load(const void* p, int64_t i) { return ((const float*)p)[i]; }
  static __device__ __forceinline__ void store(void* p, int64_t i, float v) { ((float*)p)[i] = v; }
  // eight values to an address that is a multiple of 16 bytes
  static __device__ __forceinline__ void store8(void* p, int64_t i, const float* v) {
    typedef float f32x4 __attribute__((ext_vector_type(4)));
    *(f32x4*)((float*)p + i) = f32x4{v[0], v[1], v[2], v[3]};
    *(f32x4*)((float*)p + i + 4) = f32x4{v[4], v[5], v[6], v[7]};
  }
};
struct Bf16 {
  typedef uint16_t type;
  static __device__ __forceinline__ float load(const void* p, int64_t i) {
    return __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16);
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, float v) {
    ((uint16_t*)p)[i] = __builtin_bit_cast(uint16_t, (__bf16)v);
  }
  static __device__ __forceinline__ void store8(void* p, int64_t i, const float* v) {
    *(u32x4*)((uint16_t*)p + i) = u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                        pack_bf16x2(v[6], v[7])};
  }
};
struct F16 {
  typedef uint16_t type;
  static __device__ __forceinline__ float load(const void* p, int64_t i) { return (float)((const _Float16*)p)[i]; }
  static __device__ __forceinline__ void store(void* p, int64_t i, float v) { ((_Float16*)p)[i] = (_Float16)v; }
  static __device__ __forceinline__ void store8(void* p, int64_t i, const float* v) {
    typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
    *(f16x8*)((_Float16*)p + i) = f16x8{(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3],
                                        (_Float16)v[4], (_Float16)v[5], (_Float16)v[6], (_Float16)v[7]};
  }
};

constexpr float kNegInf = -__builtin_inff();

// A logit as the scores take it: +Inf counts as the largest finite value, so
// that no score is a quotient of infinities; -0 becomes +0, since the two tie.
__device__ __forceinline__ float clean_logit(float x) { return (x > 3.402823466e38f ? 3.402823466e38f : x) + 0.0f; }

__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ double wave_max(double v) {
  for (int o = 32; o > 0; o >>= 1) v = fmax(v, __shfl_xor(v, o, 64));
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// Largest (key, lowest index) over the wave; idx < 0 where a lane has none.
__device__ __forceinline__ void wave_best(double& key, int& idx) {
  for (int o = 32; o > 0; o >>= 1) {
    const double k2 = __shfl_xor(key, o, 64);
    const int i2 = __shfl_xor(idx, o, 64);
    const bool take = i2 >= 0 && (idx < 0 || k2 > key || (k2 == key && i2 < idx));
    key = take ? k2 : key;
    idx = take ? i2 : idx;
  }
}

// One row by one wave, all in 64 bits.  key: E doubles of LDS that the wave
// has to itself.
template <typename IO>
__device__ void route_row(const RouteArgs& a, int64_t row, double* key) {
  const int lane = lane_id();
  const int64_t base = row * a.stride;
  const bool live = !a.mask || a.mask[row] != 0;
  const bool by_logit = !a.bias && (a.G == 1 || !a.top2);
  bool nan = false;
  double m = -__builtin_inf();
  for (int e = lane; e < a.E; e += kWave) {
    const float x = IO::load(a.logits, base + e);
    nan |= x != x;
    m = fmax(m, (double)clean_logit(x));  // fmax passes over NaN
  }
  const bool any_nan = ballot(nan) != 0;
  m = wave_max(m);
  double sum = 1.0;
  if (!a.sigmoid && (!by_logit || !a.renorm)) {
    sum = 0.0;
    for (int e = lane; e < a.E; e += kWave) {
      const float x = IO::load(a.logits, base + e);
      if (x > kNegInf) sum += exp((double)clean_logit(x) - m);
    }
    sum = wave_sum(sum);
  }
  // keys; -Inf marks an expert that cannot be chosen
  for (int e = lane; e < a.E; e += kWave) {
    const float x = IO::load(a.logits, base + e);
    double k = -__builtin_inf();
    if (x > kNegInf) {
      const double v = (double)clean_logit(x);
      k = by_logit ? v : a.sigmoid ? 1.0 / (1.0 + exp(-v)) : exp(v - m) / sum;
      if (a.bias) k += (double)a.bias[e];
      if (!(k > -__builtin_inf())) k = -__builtin_inf();
    }
    key[e] = k;
  }
  wave_sync();
  if (a.G > 1) {
    // lane g scores group g; groups are ranked by counting those ahead
    const int gs = a.E / a.G;
    double s = -__builtin_inf();
    if (lane < a.G) {
      double m1 = -__builtin_inf(), m2 = -__builtin_inf();
      for (int i = 0; i < gs; ++i) {
        const double k = key[lane * gs + i];
        if (k > m1) {
          m2 = m1;
          m1 = k;
        } else if (k > m2) {
          m2 = k;
        }
      }
      s = a.top2 && m2 > -__builtin_inf() ? m1 + m2 : m1;
    }
    int ahead = 0;
    for (int g = 0; g < a.G; ++g) {
      const double o = __shfl(s, g, 64);
      ahead += (o > s || (o == s && g < lane)) ? 1 : 0;
    }
    const uint64_t keep = ballot(lane < a.G && ahead < a.TG);
    wave_sync();
    for (int e = lane; e < a.E; e += kWave)
      if (!((keep >> (e / gs)) & 1)) key[e] = -__builtin_inf();
    wave_sync();
  }
  int mine = -1;  // lane j holds choice j
  for (int j = 0; j < a.K; ++j) {
    double best = -__builtin_inf();
    int at = -1;
    for (int e = lane; e < a.E; e += kWave) {
      const double k = key[e];
      if (k > best) {
        best = k;
        at = e;
      }
    }
    wave_best(best, at);
    if (at < 0) break;
    if (lane == j) mine = at;
    if (lane == 0) key[at] = -__builtin_inf();
    wave_sync();
  }
  // Weights.  Renormalised ones are formed relative to the largest chosen
  // score, so that their sum neither overflows nor vanishes:
  //   softmax: exp(x - top), sigmoid: exp(x - t) / (1 + exp(x)), t = min(top, 0).
  const bool have = mine >= 0;
  const double x = have ? (double)clean_logit(IO::load(a.logits, base + mine)) : 0.0;
  double w = 0.0;
  if (a.renorm) {
    const double top = wave_max(have ? x : -__builtin_inf());
    if (have) {
      const double t = fmin(top, 0.0);
      w = !a.sigmoid ? exp(x - top) : x > 0.0 ? 1.0 / (1.0 + exp(-x)) : exp(x - t) / (1.0 + exp(x));
    }
    const double total = wave_sum(w);
    if (have) w /= total;
  } else if (have) {
    w = a.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - m) / sum;
  }
  if (lane < a.K) {
    const bool put = have && live;
    a.idx[row * a.K + lane] = put ? mine : -1;
    a.w[row * a.K + lane] = !put ? 0.0f : any_nan ? __uint_as_float(0x7FC00000u) : (float)(w * (double)a.scale);
  }
  wave_sync();
}

// One row a wave, up to four waves a workgroup.  LDS: E doubles a wave.
constexpr int kRouteWaves = 4;

template <typename IO>
__global__ __launch_bounds__(kRouteWaves* kWave) void route_kernel(RouteArgs a) {
  extern __shared__ double route_lds[];
  const int wave = threadIdx.x / kWave;
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x / kWave) + wave;
  if (row >= a.T) return;
  route_row<IO>(a, row, route_lds + (size_t)wave * a.E);
}

// Gradient of the logits from the gradient g of the weights, one row a wave.
// With c the scale and w the weights of the chosen experts j:
//   sigmoid, renormalised: dx_j = w_j (1 - s_j) (g_j - sum g w / c)
//   sigmoid:               dx_j = c g_j s_j (1 - s_j)
//   softmax, renormalised: dx_j = w_j (g_j - sum g w / c)
//   softmax:               dx_e = c p_e ([e chosen] g_e - sum g_j p_j), every e
// Experts that were not chosen get 0 in the first three.  An expert named by
// two slots of a token gets the sum of both slots' terms.
template <typename IO>
__global__ __launch_bounds__(kRouteWaves* kWave) void route_backward_kernel(RouteBwdArgs a) {
  extern __shared__ float grad_lds[];
  const int lane = lane_id();
  const int wave = threadIdx.x / kWave;
  const int64_t row = (int64_t)blockIdx.x * kRouteWaves + wave;
  if (row >= a.T) return;
  float* buf = grad_lds + (size_t)wave * a.E;
  const int64_t base = row * a.stride;
  int at = -1;
  float g = 0.0f;
  if (lane < a.K) {
    const int64_t e = a.idx[row * a.K + lane];
    if (e >= 0 && e < a.E) {
      at = (int)e;
      g = a.gw[row * a.K + lane];
    }
  }
  const bool have = at >= 0;
  const float x = have ? clean_logit(IO::load(a.logits, base + at)) : kNegInf;
  double m = -__builtin_inf(), sum = 1.0;
  const bool dense = !a.sigmoid && !a.renorm;
  if (dense) {
    for (int e = lane; e < a.E; e += kWave) m = fmax(m, (double)clean_logit(IO::load(a.logits, base + e)));
    m = wave_max(m);
    sum = 0.0;
    for (int e = lane; e < a.E; e += kWave) sum += exp((double)clean_logit(IO::load(a.logits, base + e)) - m);
    sum = wave_sum(sum);
  }
  double d = 0.0, inner = 0.0;
  if (a.renorm) {
    const double top = wave_max(have ? (double)x : -__builtin_inf());
    const double t = fmin(top, 0.0);
    double w = 0.0;
    if (have && x > kNegInf)
      w = !a.sigmoid ? exp(x - top) : x > 0.0f ? 1.0 / (1.0 + exp(-(double)x)) : exp(x - t) / (1.0 + exp((double)x));
    const double total = wave_sum(w);
    if (total > 0.0) w /= total;
    const double mean = wave_sum(have ? g * w : 0.0);
    d = w * (g - mean) * a.scale;
    if (a.sigmoid) d /= 1.0 + exp((double)x);
  } else if (a.sigmoid) {
    const double s = 1.0 / (1.0 + exp(-(double)x));
    d = have && x > kNegInf ? a.scale * g * s / (1.0 + exp((double)x)) : 0.0;
  } else {
    const double p = have && x > kNegInf ? exp(x - m) / sum : 0.0;
    d = a.scale * g * p;
    inner = wave_sum(have ? g * p : 0.0);
  }
  if (!have) d = 0.0;
  // slots that name the same expert: the first of them carries the sum
  double total = 0.0;
  bool first = have;
  for (int j = 0; j < a.K; ++j) {
    const int o = __shfl(at, j, 64);
    const double dj = __shfl(d, j, 64);
    if (o == at) {
      total += dj;
      if (j < lane) first = false;
    }
  }
  for (int e = lane; e < a.E; e += kWave) {
    float v = 0.0f;
    if (dense) {
      const float xe = IO::load(a.logits, base + e);
      v = (float)(-(double)a.scale * inner * (exp((double)clean_logit(xe) - m) / sum));
      if (ballot(have) == 0) v = 0.0f;
    }
    buf[e] = v;
  }
  wave_sync();
  if (first) buf[at] = (float)(buf[at] + total);
  wave_sync();
  for (int e = lane; e < a.E; e += kWave) IO::store(a.grad, row * a.E + e, buf[e]);
}

}  // namespace ep
