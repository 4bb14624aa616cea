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

// Pairs of 16-bit magnitudes: their running maxima (v_pk_max_u16), the larger of
// the two at the end.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t max_magnitude16(uint32_t m, u32x4 w) {
  u16x2 r = __builtin_bit_cast(u16x2, m);
#pragma unroll
  for (int i = 0; i < 4; ++i) r = __builtin_elementwise_max(r, __builtin_bit_cast(u16x2, w[i] & 0x7FFF7FFFu));
  return __builtin_bit_cast(uint32_t, r);
}
__device__ __forceinline__ uint32_t larger16(uint32_t m) { return max(m >> 16, m & 0xFFFFu); }

// 16 bytes at any address a value may have: the memory unit takes them in one
// access.
typedef u32x4 u32x4_at2 __attribute__((aligned(2)));
typedef u32x4 u32x4_at4 __attribute__((aligned(4)));

struct F32 {
  typedef float type;
  typedef u32x4_at4 piece;
  static __device__ __forceinline__ float load(const void* p, int64_t i) { return ((const float*)p)[i]; }
  // one element that no neighbour is read with
  static __device__ __forceinline__ float load_nt(const void* p, int64_t i) {
    return __builtin_nontemporal_load((const float*)p + i);
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, float v) { ((float*)p)[i] = v; }
  static __device__ __forceinline__ void unpack(u32x4 w, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(w[i]);
  }
  // running maximum of magnitudes in a word, and at the end its fp32 bits
  static __device__ __forceinline__ uint32_t max_magnitude(uint32_t m, u32x4 w) {
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
    return m;
  }
  static __device__ __forceinline__ uint32_t magnitude_bits(uint32_t m) { return m; }
  // 16 bytes of values, to any address
  static __device__ __forceinline__ void store_piece(float* p, const float* v) {
    typedef float f32x4 __attribute__((ext_vector_type(4)));
    __builtin_nontemporal_store(__builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]}), (piece*)p);
  }
  // eight values to any address
  static __device__ __forceinline__ void store8(void* p, int64_t i, const float* v) {
    typedef float f32x4 __attribute__((ext_vector_type(4)));
    *(u32x4_at4*)((float*)p + i) = __builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]});
    *(u32x4_at4*)((float*)p + i + 4) = __builtin_bit_cast(u32x4, f32x4{v[4], v[5], v[6], v[7]});
  }
};
struct Bf16 {
  typedef uint16_t type;
  typedef u32x4_at2 piece;
  static __device__ __forceinline__ uint32_t max_magnitude(uint32_t m, u32x4 w) { return max_magnitude16(m, w); }
  static __device__ __forceinline__ uint32_t magnitude_bits(uint32_t m) { return larger16(m) << 16; }
  static __device__ __forceinline__ float load(const void* p, int64_t i) {
    return __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16);
  }
  static __device__ __forceinline__ float load_nt(const void* p, int64_t i) {
    return __uint_as_float((uint32_t)__builtin_nontemporal_load((const uint16_t*)p + i) << 16);
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, float v) {
    ((uint16_t*)p)[i] = __builtin_bit_cast(uint16_t, (__bf16)v);
  }
  static __device__ __forceinline__ void unpack(u32x4 w, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16_lo(w[i]);
      f[2 * i + 1] = bf16_hi(w[i]);
    }
  }
  static __device__ __forceinline__ void store_piece(uint16_t* p, const float* v) {
    __builtin_nontemporal_store(u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                      pack_bf16x2(v[6], v[7])}, (piece*)p);
  }
  static __device__ __forceinline__ void store8(void* p, int64_t i, const float* v) {
    *(u32x4_at2*)((uint16_t*)p + i) = u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                            pack_bf16x2(v[6], v[7])};
  }
};
struct F16 {
  typedef uint16_t type;
  typedef u32x4_at2 piece;
  static __device__ __forceinline__ uint32_t max_magnitude(uint32_t m, u32x4 w) { return max_magnitude16(m, w); }
  static __device__ __forceinline__ uint32_t magnitude_bits(uint32_t m) {
    return __float_as_uint((float)__builtin_bit_cast(_Float16, (uint16_t)larger16(m)));  // (infinities and NaN stay)
  }
  static __device__ __forceinline__ float load(const void* p, int64_t i) { return (float)((const _Float16*)p)[i]; }
  static __device__ __forceinline__ float load_nt(const void* p, int64_t i) {
    return (float)__builtin_bit_cast(_Float16, __builtin_nontemporal_load((const uint16_t*)p + i));
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, float v) { ((_Float16*)p)[i] = (_Float16)v; }
  static __device__ __forceinline__ void unpack(u32x4 w, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = (float)__builtin_bit_cast(_Float16, (uint16_t)w[i]);
      f[2 * i + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[i] >> 16));
    }
  }
  static __device__ __forceinline__ void store_piece(uint16_t* p, const float* v) {
    typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
    const f16x8 h = {(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3],
                     (_Float16)v[4], (_Float16)v[5], (_Float16)v[6], (_Float16)v[7]};
    __builtin_nontemporal_store(__builtin_bit_cast(u32x4, h), (piece*)p);
  }
  static __device__ __forceinline__ void store8(void* p, int64_t i, const float* v) {
    typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
    *(u32x4_at2*)((_Float16*)p + i) = __builtin_bit_cast(
        u32x4, f16x8{(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3], (_Float16)v[4], (_Float16)v[5],
                     (_Float16)v[6], (_Float16)v[7]});
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

// Value of lane (lane ^ X), X < 16, by DPP.
template <int X>
__device__ __forceinline__ int xor_lane(int v) {
  if constexpr (X >= 8) return xor_lane<15 ^ X>(__builtin_amdgcn_mov_dpp(v, 0x140, 0xF, 0xF, true));  // mirror of 16
  else if constexpr (X >= 4) return xor_lane<7 ^ X>(__builtin_amdgcn_mov_dpp(v, 0x141, 0xF, 0xF, true));  // mirror of 8
  else if constexpr (X == 3) return __builtin_amdgcn_mov_dpp(v, 0x1B, 0xF, 0xF, true);
  else if constexpr (X == 2) return __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, true);
  else if constexpr (X == 1) return __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, true);
  else return v;
}
template <int X>
__device__ __forceinline__ float xor_lane(float v) { return __int_as_float(xor_lane<X>(__float_as_int(v))); }
template <int X>
__device__ __forceinline__ double xor_lane(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)(uint32_t)xor_lane<X>((int)(uint32_t)b) |
                                        (uint64_t)(uint32_t)xor_lane<X>((int)(uint32_t)(b >> 32)) << 32);
}

__device__ __forceinline__ double lane_value(double v, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)b, lane);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_max(double v) {
  v = fmax(v, xor_lane<1>(v));
  v = fmax(v, xor_lane<2>(v));
  v = fmax(v, xor_lane<7>(v));
  v = fmax(v, xor_lane<15>(v));
  return fmax(fmax(lane_value(v, 0), lane_value(v, 16)), fmax(lane_value(v, 32), lane_value(v, 48)));
}
__device__ __forceinline__ double wave_sum(double v) {
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
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
  // keys; -Inf marks an expert that cannot be chosen
  double sum = 1.0;
  const bool soft = !a.sigmoid && (!by_logit || !a.renorm);
  if (soft) {
    sum = 0.0;
    for (int e = lane; e < a.E; e += kWave) {
      const float x = IO::load(a.logits, base + e);
      const double p = x > kNegInf ? exp((double)clean_logit(x) - m) : 0.0;
      sum += p;
      key[e] = p;
    }
    sum = wave_sum(sum);
  }
  for (int e = lane; e < a.E; e += kWave) {
    const float x = IO::load(a.logits, base + e);
    double k = -__builtin_inf();
    if (x > kNegInf) {
      const double v = (double)clean_logit(x);
      k = by_logit ? v : a.sigmoid ? 1.0 / (1.0 + exp(-v)) : key[e] / sum;
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
#pragma unroll 4
      for (int i = 0; i < gs; ++i) {
        const double k = key[lane * gs + i];
        m2 = fmax(m2, fmin(m1, k));
        m1 = fmax(m1, k);
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
  // Every lane has the best of its experts at hand; the best lane gives its up and
  // looks for its next.
  int mine = -1;  // lane j holds choice j
  double best;
  int at;
  auto look = [&]() {
    best = -__builtin_inf();
    at = -1;
#pragma unroll 4
    for (int e = lane; e < a.E; e += kWave) {
      const double k = key[e];
      at = k > best ? e : at;
      best = fmax(best, k);
    }
  };
  look();
  for (int j = 0; j < a.K; ++j) {
    const double top = wave_max(best);
    if (!(top > -__builtin_inf())) break;
    uint64_t tied = ballot(best == top);
    int first = __builtin_amdgcn_readlane(at, __builtin_ctzll(tied));
    for (tied &= tied - 1; tied; tied &= tied - 1)
      first = min(first, __builtin_amdgcn_readlane(at, __builtin_ctzll(tied)));
    if (lane == j) mine = first;
    if (at == first) {
      key[first] = -__builtin_inf();
      look();
    }
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

// --------------------------------------------------------------------------
// Several rows a wave: LPR lanes share a row of at most LPR * VPL experts and
// K <= 8 * R choices.  A lane owns `seg` consecutive experts, or what is left of
// its group, brought to its registers through LDS (memory is read in whole lines).
//
// Keys are fp32.  A key's bits are taken as the high word of a double, whose
// order is that of the floats (all of them finite doubles, -Inf included), with
// the expert in the low word (inverted for positive keys): one v_max_f64 and one
// v_min_f64 exchange key and expert, and equal keys stand in the order of the
// experts.  (Waves without a negative key skip the inversion by sign, two operations
// a key.)  A lane sorts eights of its keys, keeps the best eight, and three or
// four bitonic merges over its neighbours leave the row's best eight in every lane.
// More than eight choices (R = 2) take a second round over the keys below the eighth
// (65536 x 256 bf16, top 10: 28 us, against 178 with one row a wave in 64 bits).
//
// The definition orders the keys by their exact values.  Logits are exact.
// Scores are not: a row where two neighbours among the choices, the last choice
// and the best expert left out, or a kept and a dropped group, lie within the
// error of the fp32 scores (and are not equal for being made of equal numbers)
// is done over in 64 bits by the whole wave (route_row), rows of masked tokens too.
// How many that are depends on the data, since the margins do not shrink with small
// scores.  Top 8 of 256: one row in 800 to 1100 for normal logits of deviation 1.5; one in
// 22 for sigmoids of deviation 5 under a bias of deviation 0.001; one in 8 for softmax of
// deviation 5 under a bias of 0.0008; nearly all for saturated sigmoids (deviation 8)
// without a bias but with sums of two.
//
// Vector instructions bound it, 180 a row of 256 with groups and bias: 262144 rows
// of fp32 in 92 us, 3.2 TB/s; 32768 rows of bf16 by logits 9-10 us; one
// row 5.3 us, a wave's latency.  One row a wave in 64 bits took 759 and 38 us.

// Over the N (8 or 16) lanes of a row; every lane gets the result.
template <int N>
__device__ __forceinline__ float lanes_max(float v) {
  v = fmaxf(v, xor_lane<1>(v));
  v = fmaxf(v, xor_lane<2>(v));
  v = fmaxf(v, xor_lane<7>(v));
  if (N == 16) v = fmaxf(v, xor_lane<15>(v));
  return v;
}
template <int N>
__device__ __forceinline__ float lanes_sum(float v) {
  v += xor_lane<1>(v);
  v += xor_lane<2>(v);
  v += xor_lane<7>(v);
  if (N == 16) v += xor_lane<15>(v);
  return v;
}
template <int N>
__device__ __forceinline__ int lanes_sum(int v) {
  v += xor_lane<1>(v);
  v += xor_lane<2>(v);
  v += xor_lane<7>(v);
  if (N == 16) v += xor_lane<15>(v);
  return v;
}

// v_max_f64 and v_min_f64 as they are: fmax would first quiet operands that the
// compiler cannot prove to be no signalling NaN (a third more instructions), and
// the keys are none.
__device__ __forceinline__ double max64(double a, double b) {
  double r;
  asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}
__device__ __forceinline__ double min64(double a, double b) {
  double r;
  asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}
__device__ __forceinline__ void exchange(double& a, double& b) {  // the larger first
  const double hi = max64(a, b), lo = min64(a, b);
  a = hi;
  b = lo;
}
__device__ __forceinline__ void sort8(double (&v)[8]) {
  exchange(v[0], v[2]); exchange(v[1], v[3]); exchange(v[4], v[6]); exchange(v[5], v[7]);
  exchange(v[0], v[4]); exchange(v[1], v[5]); exchange(v[2], v[6]); exchange(v[3], v[7]);
  exchange(v[0], v[1]); exchange(v[2], v[3]); exchange(v[4], v[5]); exchange(v[6], v[7]);
  exchange(v[2], v[4]); exchange(v[3], v[5]);
  exchange(v[1], v[4]); exchange(v[3], v[6]);
  exchange(v[1], v[2]); exchange(v[3], v[4]); exchange(v[5], v[6]);
}
// The best eight of two falling lists of eight, falling.
__device__ __forceinline__ void merge8(double (&v)[8], const double (&o)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = max64(v[i], o[7 - i]);
#pragma unroll
  for (int d = 4; d > 0; d >>= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!(i & d)) exchange(v[i], v[i + d]);
}
template <int X>
__device__ __forceinline__ void merge8_lane(double (&v)[8]) {
  double o[8];
  // two wait states between the writes above and the DPP reads
  asm("s_nop 1" : "+v"(v[0]), "+v"(v[1]), "+v"(v[2]), "+v"(v[3]), "+v"(v[4]), "+v"(v[5]), "+v"(v[6]), "+v"(v[7]));
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = xor_lane<X>(v[i]);
  merge8(v, o);
}

// BY_SIGN: inverted for positive keys only, else always.
template <bool BY_SIGN>
__device__ __forceinline__ double tagged(float k, int e) {
  const uint32_t hi = __float_as_uint(k);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | (uint32_t)(~e ^ (BY_SIGN ? (int)hi >> 31 : 0)));
}
__device__ __forceinline__ float key_of(double d) {
  return __uint_as_float((uint32_t)(__builtin_bit_cast(uint64_t, d) >> 32));
}
__device__ __forceinline__ int expert_of(double d, int by_sign) {
  const uint64_t b = __builtin_bit_cast(uint64_t, d);
  return ~((int)(uint32_t)b ^ (((int)(uint32_t)(b >> 32) >> 31) & by_sign));
}

// The best eight of a lane's keys, falling, in rounds after the first of those that
// come after list[7].
template <int VPL, bool BY_SIGN>
__device__ __forceinline__ void best_of_lane(const float (&key)[VPL], int e0, int round, double (&list)[8]) {
  const double limit = list[7];
#pragma unroll
  for (int c = 0; c < VPL; c += 8) {
    double v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = tagged<BY_SIGN>(key[c + i], e0 + c + i);
      if (round > 0) v[i] = v[i] < limit ? v[i] : tagged<true>(kNegInf, 0);
    }
    sort8(v);
    if (c == 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) list[i] = v[i];
    } else {
      merge8(list, v);
    }
  }
}

// Where a row's logits are in LDS: share l of `seg` experts at l * pitch (pitch a
// multiple of 4 and odd in 16-byte units: no bank conflicts), where no group ends
// within four experts that are stored at once; otherwise one after the other (pitch
// and magic 0).
struct RouteLanes {
  int seg;        // experts of a lane, at most VPL
  int gs;         // experts of a group (without groups: all)
  int shift;      // 1 << shift lanes of a group
  int pitch;      // floats between lanes in LDS, 0: experts one after the other
  int row_pitch;  // floats between rows in LDS, a multiple of 4
  int magic;      // e / seg == (e * magic) >> 20 for e < 512
  int pad;        // some lane has fewer than VPL experts
  int bias_vec;   // the bias can be read 16 bytes at a time
};

// log2(e) * x for exp2, and the hardware's exp2 and reciprocal: the scores of
// the first pass, whose errors the margins below bound.
__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }

// A choice's score relative to the largest of the token's: softmax exp(x - best),
// sigmoid exp(x - t) / (1 + exp(x)), t = min(best, 0).
__device__ __forceinline__ float choice_weight(float x, float best, int sigmoid) {
  if (!sigmoid) return expf(x - best);
  const float a = expf(-fabsf(x));
  const float top = x > 0.0f ? 1.0f : best < 0.0f ? expf(x - best) : a;
  return top / (1.0f + a);
}

template <typename IO, int LPR, int VPL, int R>
__global__ __launch_bounds__(kWave) void route_lanes_kernel(RouteArgs a, RouteLanes p) {
  constexpr int kRows = kWave / LPR;
  typedef float f32x4 __attribute__((ext_vector_type(4)));
  extern __shared__ float lanes_lds[];  // [kRows][row_pitch], and VPL that are read past the end
  const int lane = threadIdx.x;
  const int l = lane % LPR;
  const int64_t row0 = (int64_t)blockIdx.x * kRows;
  const int64_t row = min(row0 + lane / LPR, (int64_t)a.T - 1);
  const int64_t base = row * a.stride;
  float* const row_lds = lanes_lds + (lane / LPR) * p.row_pitch;
  const int group = l >> p.shift, share = l & ((1 << p.shift) - 1);
  const int e0 = group * p.gs + share * p.seg;
  const int have = group < a.G ? max(0, min(p.seg, p.gs - share * p.seg)) : 0;
  const float* const mine = row_lds + (p.pitch ? l * p.pitch : have > 0 ? e0 : 0);
  const bool by_logit = !a.bias && (a.G == 1 || !a.top2);
  bool by_sign = by_logit;  // keys below zero stand in order too

  // logits to LDS
  constexpr int V = 16 / sizeof(typename IO::type);
  constexpr int kChunks = (VPL + V - 1) / V;
  const typename IO::type* src = (const typename IO::type*)a.logits + base;
  const int chunks = a.E / V;
  auto place = [&](int e) {
    const int o = (e * p.magic) >> 20;
    return row_lds + o * p.pitch + (e - o * p.seg);
  };
  u32x4 raw[kChunks];
#pragma unroll
  for (int j = 0; j < kChunks; ++j) {
    const int c = j * LPR + l;
    raw[j] = c < chunks ? *(const typename IO::piece*)(src + c * V) : u32x4{0, 0, 0, 0};
  }
  const int last = chunks * V + l;  // fewer than V <= LPR are left
  float end = 0.0f;
  if (a.E % V != 0 && last < a.E) end = IO::load(a.logits, base + last);
#pragma unroll
  for (int j = 0; j < kChunks; ++j) {
    const int c = j * LPR + l;
    if (c < chunks) {
      float f[V];
      IO::unpack(raw[j], f);
#pragma unroll
      for (int i = 0; i < V; i += 4) *(f32x4*)place(c * V + i) = f32x4{f[i], f[i + 1], f[i + 2], f[i + 3]};
    }
  }
  if (a.E % V != 0 && last < a.E) *place(last) = end;
  wave_sync();

  // this lane's logits.  Rows of numbers alone go straight on; where the wave has an
  // infinity or a NaN, kNegInf marks what cannot be chosen.
  float key[VPL];
  float top = kNegInf;
  if (p.pitch) {
#pragma unroll
    for (int i = 0; i < VPL; i += 4) {
      const f32x4 v = *(const f32x4*)(mine + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) key[i + j] = v[j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = mine[i];
  }
  if (p.pad) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = i < have ? key[i] : 0.0f;
  }
  float size = 0.0f;  // NaN if one of them is
#pragma unroll
  for (int i = 0; i < VPL; i += 2)
    size = __builtin_elementwise_maximum(__builtin_elementwise_maximum(size, fabsf(key[i])), fabsf(key[i + 1]));
  const bool special = ballot(!(size < __builtin_inff())) != 0;
  bool any_nan = false;
  if (special) {
    bool nan = false;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const float x = i < have ? key[i] : kNegInf;
      nan |= x != x;
      key[i] = x != x ? kNegInf : clean_logit(x);
    }
    const uint64_t row_lanes = (LPR == 16 ? 0xFFFFull : 0xFFull) << (lane - l);
    any_nan = (ballot(nan) & row_lanes) != 0;
  } else if (p.pad) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = i < have ? key[i] : kNegInf;
  }
  float total = 1.0f;
  if (!a.sigmoid && (!by_logit || !a.renorm)) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) top = fmaxf(top, key[i]);
    top = fmaxf(lanes_max<LPR>(top), -3.402823466e38f);  // finite, also in a row without a choice
    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < VPL; ++i) sum[i % 4] += fast_exp(key[i] - top);  // 0 for kNegInf
    total = lanes_sum<LPR>((sum[0] + sum[1]) + (sum[2] + sum[3]));
  }
  if (by_logit) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] += 0.0f;  // -0 ties with +0
  } else {
    if (a.sigmoid) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) key[i] = __builtin_amdgcn_rcpf(1.0f + fast_exp(-key[i]));
    } else {
      const float inv = __builtin_amdgcn_rcpf(total);
#pragma unroll
      for (int i = 0; i < VPL; ++i) key[i] = fast_exp(key[i] - top) * inv;
    }
    if (special) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) key[i] = i < have && mine[i] > kNegInf ? key[i] : kNegInf;
    } else if (p.pad) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) key[i] = i < have ? key[i] : kNegInf;
    }
    if (a.bias) {
      // rounded score plus bias in every branch: keys of equal parts tie wherever their bias is read
#pragma clang fp contract(off)
      float best = kNegInf, worst = 0.0f;
      if (p.bias_vec) {
#pragma unroll
        for (int i = 0; i < VPL; i += 4) {
          const f32x4 b = *(const f32x4*)(a.bias + (i < have ? e0 + i : 0));
#pragma unroll
          for (int j = 0; j < 4; ++j) key[i + j] += b[j];
        }
      } else {
#pragma unroll
        for (int i = 0; i < VPL; i += 4) {
          if (i >= have) continue;
          if (e0 + i + 4 <= a.E) {  // (a neighbour's bias leaves -Inf, or makes a NaN that is cleared below)
            const u32x4 b = *(const u32x4_at4*)(a.bias + e0 + i);
#pragma unroll
            for (int j = 0; j < 4; ++j) key[i + j] += __uint_as_float(b[j]);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) key[i + j] += a.bias[min(e0 + i + j, a.E - 1)];
          }
        }
      }
#pragma unroll
      for (int i = 0; i < VPL; i += 2)
        best = __builtin_elementwise_maximum(__builtin_elementwise_maximum(best, key[i]), key[i + 1]);
#pragma unroll
      for (int i = 0; i < VPL; i += 2) worst = fminf(fminf(worst, key[i]), key[i + 1]);
      by_sign = ballot(worst < 0.0f) != 0;
      // a key of -Inf or NaN cannot be chosen; one of +Inf is decided in 64 bits
      if (ballot(!(best < __builtin_inff()))) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) key[i] = key[i] > kNegInf ? fminf(key[i], 3.402823466e38f) : kNegInf;
      }
    }
  }
  // Two keys of the row keep their order where they differ by more than the error of
  // their difference.  In units of u = 2^-24, sigmoid: the exponent's 2.3 |x| u
  // weighs x s (1 - s) < 0.23, exp2 0.5 u, the sum u, the reciprocal 2 u: below 4.1 u
  // a score.  Softmax, of the largest score: two scores' exponent (0.9 u at most),
  // exp2 2 u and product u each, and the sum's error, a common factor: 14 additions,
  // exp2 2 u, the exponents 2.3 ln E u, the reciprocal 2 u: 41 u in all, below 2^-18.
  // The sum with the bias is added where keys are compared.
  const float margin0 = a.sigmoid ? 0x1p-20f : 0x1p-18f * __builtin_amdgcn_rcpf(total);
  bool unsure = false, lane_kept = true;

  if (a.G > 1) {
    float m1 = kNegInf, m2 = kNegInf;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      m2 = __builtin_amdgcn_fmed3f(m1, m2, key[i]);  // m1 >= m2: the second of the three
      m1 = fmaxf(m1, key[i]);
    }
    auto join = [&](float o1, float o2) {
      m2 = fmaxf(fmaxf(m2, o2), fminf(m1, o1));
      m1 = fmaxf(m1, o1);
    };
    // lanes of one group are neighbours: after each merge all of them agree
    if (p.shift >= 1) join(xor_lane<1>(m1), xor_lane<1>(m2));
    if (p.shift >= 2) join(xor_lane<2>(m1), xor_lane<2>(m2));
    if (p.shift >= 3) join(xor_lane<7>(m1), xor_lane<7>(m2));
    const int g = group;
    // Groups past the last own nothing: -Inf, behind every other or tied with an empty one.
    // A sum below fp32 (experts switched off by a bias of its lowest value) counts as the
    // lowest value, before an empty group; two such sums are equal, and decided in 64 bits.
    const float s = a.top2 && m2 > kNegInf ? fmaxf(m1 + m2, -3.402823466e38f) : m1;
    int ahead = 0;
    auto count = [&](float o, int ol) {
      const int og = ol >> p.shift;
      ahead += (o > s) | ((o == s) & (og < g)) ? 1 : 0;
    };
    count(xor_lane<1>(s), l ^ 1);
    count(xor_lane<2>(s), l ^ 2);
    count(xor_lane<3>(s), l ^ 3);
    count(xor_lane<4>(s), l ^ 4);
    count(xor_lane<5>(s), l ^ 5);
    count(xor_lane<6>(s), l ^ 6);
    count(xor_lane<7>(s), l ^ 7);
    if (LPR == 16) {
      count(xor_lane<8>(s), l ^ 8);
      count(xor_lane<9>(s), l ^ 9);
      count(xor_lane<10>(s), l ^ 10);
      count(xor_lane<11>(s), l ^ 11);
      count(xor_lane<12>(s), l ^ 12);
      count(xor_lane<13>(s), l ^ 13);
      count(xor_lane<14>(s), l ^ 14);
      count(xor_lane<15>(s), l ^ 15);
    }
    // every lane of a group ahead counted
    const bool kept = g < a.G && (ahead >> p.shift) < a.TG;
    if (!by_logit) {
      const float worst = -lanes_max<LPR>(kept ? -s : kNegInf);  // of the kept groups
      const float best = lanes_max<LPR>(!kept && g < a.G ? s : kNegInf);
      const float margin = (a.top2 ? 2.0f : 1.0f) * margin0 + 0x1p-21f * fmaxf(fabsf(worst), fabsf(best));
      unsure |= best > kNegInf && !(worst - best > margin);
    }
    lane_kept = kept;
  }

  double list[8], own[8];
  const double none = tagged<true>(kNegInf, 0);
  double mine_d[R];  // lane l < 8 of the row holds choices l, l + 8, ..
#pragma unroll
  for (int c = 0; c < R; ++c) {
    if (by_sign)
      best_of_lane<VPL, true>(key, e0, c, list);
    else
      best_of_lane<VPL, false>(key, e0, c, list);
#pragma unroll
    for (int i = 0; i < 8; ++i) own[i] = list[i] = lane_kept ? list[i] : none;
    merge8_lane<1>(list);
    merge8_lane<2>(list);
    merge8_lane<7>(list);
    if (LPR == 16) merge8_lane<15>(list);
    mine_d[c] = list[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) mine_d[c] = l == i ? list[i] : mine_d[c];
  }

  bool chosen[R];
  int e[R];
  float x[R];
#pragma unroll
  for (int c = 0; c < R; ++c) {
    chosen[c] = (R == 1 || l < 8) && c * 8 + l < a.K && key_of(mine_d[c]) > kNegInf;
    e[c] = chosen[c] ? expert_of(mine_d[c], by_sign ? -1 : 0) : 0;
    x[c] = chosen[c] ? clean_logit(*place(e[c])) : kNegInf;
  }

  if (!by_logit) {
    float kf[R], b[R], largest = 0.0f;
#pragma unroll
    for (int c = 0; c < R; ++c) {
      kf[c] = chosen[c] ? key_of(mine_d[c]) : 0.0f;
      b[c] = a.bias && chosen[c] ? a.bias[e[c]] : 0.0f;
      largest = fmaxf(largest, fabsf(kf[c]));
    }
    const float margin = margin0 + 0x1p-22f * lanes_max<LPR>(largest);
    // neighbours among the choices
#pragma unroll
    for (int c = 0; c < R; ++c) {
      float k2 = __shfl_down(kf[c], 1, 64), x2 = __shfl_down(x[c], 1, 64), b2 = __shfl_down(b[c], 1, 64);
      bool next = __shfl_down((int)chosen[c], 1, 64) != 0 && l + 1 < min(8, a.K - c * 8);
      if (c + 1 < R) {
        const int first = lane - l;
        const float k3 = __shfl(kf[c + 1 < R ? c + 1 : c], first, 64), x3 = __shfl(x[c + 1 < R ? c + 1 : c], first, 64);
        const float b3 = __shfl(b[c + 1 < R ? c + 1 : c], first, 64);
        const bool n3 = __shfl((int)chosen[c + 1 < R ? c + 1 : c], first, 64) != 0;
        k2 = l == 7 ? k3 : k2;
        x2 = l == 7 ? x3 : x2;
        b2 = l == 7 ? b3 : b2;
        next = l == 7 ? n3 : next;
      }
      unsure |= chosen[c] && next && !(kf[c] - k2 > margin) && !(x[c] == x2 && b[c] == b2);
    }
    // the last choice against those left out; it is one of the last round's
    const int at = a.K - 1 - (R - 1) * 8;
    double last_d = list[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) last_d = at == i ? list[i] : last_d;
    const float last = key_of(last_d);
    const bool full = last > kNegInf;
    const float from = last - margin;
    // the best key left out: a lane's choices are the first of its eight; eight
    // of one lane leave its ninth unknown
    float out = key_of(own[7]);
    out = own[7] < last_d ? out : __builtin_inff();
#pragma unroll
    for (int i = 6; i >= 0; --i) out = own[i] < last_d ? key_of(own[i]) : out;
    out = lanes_max<LPR>(lane_kept ? out : kNegInf);
    if (ballot(full && out >= from)) {
      const float xk = __shfl(x[R - 1], lane - l + at, 64), bk = __shfl(b[R - 1], lane - l + at, 64);
      int other = 0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        if (!(full && lane_kept && i < have && key[i] >= from)) continue;
        other += clean_logit(mine[i]) == xk && (!a.bias || a.bias[e0 + i] == bk) ? 0 : 1;
      }
      other = lanes_sum<LPR>(other);
      int among = 0;
#pragma unroll
      for (int c = 0; c < R; ++c) among += chosen[c] && !(x[c] == xk && b[c] == bk) ? 1 : 0;
      unsure |= full && other != lanes_sum<LPR>(among);
    }
  }

  // weights, as route_row forms them
  float w[R], best = kNegInf, sum = 0.0f;
#pragma unroll
  for (int c = 0; c < R; ++c) best = fmaxf(best, x[c]);
  if (a.renorm) best = lanes_max<LPR>(best);
#pragma unroll
  for (int c = 0; c < R; ++c) {
    w[c] = 0.0f;
    if (chosen[c])
      w[c] = a.renorm ? choice_weight(x[c], best, a.sigmoid)
             : a.sigmoid ? choice_weight(x[c], 0.0f, 1)
                         : expf(x[c] - top) / total;
    sum += w[c];
  }
  if (a.renorm) sum = lanes_sum<LPR>(sum);
#pragma unroll
  for (int c = 0; c < R; ++c) {
    const int k = c * 8 + l;
    if ((R == 1 || l < 8) && k < a.K && row0 + lane / LPR < a.T) {
      const bool put = chosen[c] && (!a.mask || a.mask[row] != 0);
      if (a.renorm && chosen[c]) w[c] /= sum;
      a.idx[row * a.K + k] = put ? e[c] : -1;
      a.w[row * a.K + k] = !put ? 0.0f : any_nan ? __uint_as_float(0x7FC00000u) : w[c] * a.scale;
    }
  }

  // the rows whose order fp32 does not settle
  uint64_t redo = ballot(unsure && row0 + lane / LPR < a.T);
  if (redo) {
    wave_sync();
    for (int r = 0; r < kRows; ++r)
      if ((redo >> (r * LPR)) & (LPR == 16 ? 0xFFFFull : 0xFFull))
        route_row<IO>(a, row0 + r, (double*)lanes_lds);
  }
}

// Gradient of the logits from the gradient g of the weights, one row a wave.
// With c the scale and w the weights of the chosen experts j:
//   sigmoid, renormalised: dx_j = w_j (1 - s_j) (g_j - sum g w / c)
//   sigmoid:               dx_j = c g_j s_j (1 - s_j)
//   softmax, renormalised: dx_j = w_j (g_j - sum g w / c)
//   softmax:               dx_e = c p_e ([e chosen] g_e - sum g_j p_j), every e
// Experts that were not chosen get 0 in the first three.  An expert named by
// two slots of a token gets the sum of both slots' terms.  Logits of -Inf have
// score 0; NaN (compared as "not <= -Inf") goes on into all that its score enters.
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
    m = fmax(wave_max(m), (double)-3.402823466e38f);  // finite, also in a row of -Inf
    sum = 0.0;
    for (int e = lane; e < a.E; e += kWave) sum += exp((double)clean_logit(IO::load(a.logits, base + e)) - m);
    sum = wave_sum(sum);
  }
  double d = 0.0, inner = 0.0;
  if (a.renorm) {
    const double top = wave_max(have ? (double)x : -__builtin_inf());
    const double t = fmin(top, 0.0);
    double w = 0.0;
    if (have && !(x <= kNegInf))
      w = !a.sigmoid ? exp(x - top) : x > 0.0f ? 1.0 / (1.0 + exp(-(double)x)) : exp(x - t) / (1.0 + exp((double)x));
    const double total = wave_sum(w);
    if (total != 0.0) w /= total;
    const double mean = wave_sum(have ? g * w : 0.0);
    d = w * (g - mean) * a.scale;
    if (a.sigmoid) d /= 1.0 + exp((double)x);
  } else if (a.sigmoid) {
    const double s = 1.0 / (1.0 + exp(-(double)x));
    d = have && !(x <= kNegInf) ? a.scale * g * s / (1.0 + exp((double)x)) : 0.0;
  } else {
    const double p = have && !(x <= kNegInf) ? exp(x - m) / sum : 0.0;
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
      if (ballot(have) == 0 || sum == 0.0) v = 0.0f;  // (a row of -Inf has no score)
    }
    buf[e] = v;
  }
  wave_sync();
  if (first) buf[at] = (float)(buf[at] + total);
  wave_sync();
  for (int e = lane; e < a.E; e += kWave) IO::store(a.grad, row * a.E + e, buf[e]);
}

// The same with LPR lanes a row (K <= LPR), kWave / LPR rows a wave, a lane a
// choice, in 32 bits.  What has to move is the gradient (and, with a softmax
// that is not renormalised, the logits): the choices' terms are put into rows of
// zeros in LDS, the rows go out in 16-byte pieces, and the terms are taken out
// again, so that the zeros are written to LDS once for all rows of a wave.  Memory
// bounds it: 262144 x 256 fp32 in 80 us, of which the chosen logits, a line each, are
// 25; dense, 131072 x 256 bf16 in 33 us, 4.3 TB/s (one row a wave: 189 and 179 us).
// NCH > 0: the dense form with a lane's NCH pieces of the row in registers, read
// and raised once; 0: every other case (vec: dense rows of whole pieces).
// The rows in registers are raised by the hardware's exp2 (fast_exp): a score d below
// the row's largest is off by 3 u d relative, u = 2^-24 (the difference, the factor
// log2 e, their product), one by expf by u d, and is 0 below the normal range.  d exp(-d)
// < 0.37, so that this adds 0.8 u of the largest score to an error of several u.
template <typename IO, int LPR, int NCH>
__global__ __launch_bounds__(kWave) void route_backward_lanes_kernel(RouteBwdArgs a, int vec) {
  constexpr int kRows = kWave / LPR;
  constexpr int V = 16 / sizeof(typename IO::type);
  extern __shared__ float terms[];  // [kRows][E]
  const int lane = threadIdx.x;
  const int l = lane % LPR;
  const bool dense = !a.sigmoid && !a.renorm;
  float* const row_terms = terms + (lane / LPR) * a.E;
  for (int i = lane; i < kRows * a.E; i += kWave) terms[i] = 0.0f;
  wave_sync();
  for (int64_t row0 = (int64_t)blockIdx.x * kRows; row0 < a.T; row0 += (int64_t)gridDim.x * kRows) {
    const int64_t row = row0 + lane / LPR;
    const bool live = row < a.T;
    const int64_t base = (live ? row : 0) * a.stride;
    int at = -1;
    float g = 0.0f;
    if (live && l < a.K) {
      const int64_t e = a.idx[row * a.K + l];
      if (e >= 0 && e < a.E) {
        at = (int)e;
        g = a.gw[row * a.K + l];
      }
    }
    const bool have = at >= 0;
    const float x = have ? clean_logit(IO::load_nt(a.logits, base + at)) : kNegInf;
    // softmax over the whole row: maximum and sum in one pass
    float m = kNegInf, sum = 0.0f;
    float e[NCH > 0 ? NCH : 1][V], rest = kNegInf;
    const int last = a.E / V * V + l;  // fewer than V <= LPR values are no whole piece
    if (NCH > 0) {
      const typename IO::type* src = (const typename IO::type*)a.logits + base;
      bool nan = false;
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        const int c = j * LPR + l;
        const bool in = c < a.E / V;
        IO::unpack(!in ? u32x4{0, 0, 0, 0} : *(const typename IO::piece*)(src + c * V), e[j]);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          nan |= in && e[j][i] != e[j][i];
          e[j][i] = in ? clean_logit(e[j][i]) : kNegInf;
          m = fmaxf(m, e[j][i]);
        }
      }
      if (a.E % V != 0 && last < a.E) {
        const float x = IO::load(a.logits, base + last);
        nan |= x != x;
        rest = clean_logit(x);
        m = fmaxf(m, rest);
      }
      m = fmaxf(lanes_max<LPR>(m), -3.402823466e38f);  // finite, also in a row of -Inf
#pragma unroll
      for (int j = 0; j < NCH; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          e[j][i] = fast_exp(e[j][i] - m);
          sum += e[j][i];
        }
      rest = fast_exp(rest - m);
      sum += rest;
      sum = lanes_sum<LPR>(nan ? __uint_as_float(0x7FC00000u) : sum);
    } else if (dense) {
      auto add = [&](const float* f, int n) {
        float top = m;
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (i < n) top = fmaxf(top, clean_logit(f[i]));
        const float old = m > kNegInf ? sum * expf(m - top) : sum;
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (i < n && !(f[i] <= kNegInf)) s += expf(clean_logit(f[i]) - top);  // NaN stays NaN
        sum = old + s;
        m = top;
      };
      if (vec) {
        const typename IO::type* src = (const typename IO::type*)a.logits + base;
        for (int c = l; c < a.E / V; c += LPR) {
          float f[V];
          IO::unpack(*(const typename IO::piece*)(src + c * V), f);
          add(f, V);
        }
      } else {
        for (int e = l; e < a.E; e += LPR) {
          float f[V] = {IO::load(a.logits, base + e)};
          add(f, 1);
        }
      }
      const float top = fmaxf(lanes_max<LPR>(m), -3.402823466e38f);
      sum = lanes_sum<LPR>(m > kNegInf ? sum * expf(m - top) : sum);
      m = top;
    }
    float d = 0.0f, inner = 0.0f;
    if (a.renorm) {
      const float top = lanes_max<LPR>(x);
      const float t = fminf(top, 0.0f);
      float w = 0.0f;
      if (!(x <= kNegInf))
        w = !a.sigmoid ? expf(x - top) : x > 0.0f ? 1.0f / (1.0f + expf(-x)) : expf(x - t) / (1.0f + expf(x));
      const float total = lanes_sum<LPR>(w);
      if (total != 0.0f) w /= total;
      const float mean = lanes_sum<LPR>(have ? g * w : 0.0f);
      d = w * (g - mean) * a.scale;
      if (a.sigmoid) d /= 1.0f + expf(x);
    } else if (a.sigmoid) {
      if (!(x <= kNegInf)) d = a.scale * g / ((1.0f + expf(-x)) * (1.0f + expf(x)));
    } else {
      const float p = !(x <= kNegInf) ? expf(x - m) / sum : 0.0f;
      d = a.scale * g * p;
      inner = a.scale * lanes_sum<LPR>(have ? g * p : 0.0f);
    }
    if (!have) d = 0.0f;
    // slots that name the same expert: the first of them carries the sum
    float total = d;
    bool first = have;
    auto other = [&](int oat, float od, int ol) {
      const bool same = oat == at;
      total += same ? od : 0.0f;
      first = first && !(same && ol < l);
    };
    other(xor_lane<1>(at), xor_lane<1>(d), l ^ 1);
    other(xor_lane<2>(at), xor_lane<2>(d), l ^ 2);
    other(xor_lane<3>(at), xor_lane<3>(d), l ^ 3);
    other(xor_lane<4>(at), xor_lane<4>(d), l ^ 4);
    other(xor_lane<5>(at), xor_lane<5>(d), l ^ 5);
    other(xor_lane<6>(at), xor_lane<6>(d), l ^ 6);
    other(xor_lane<7>(at), xor_lane<7>(d), l ^ 7);
    if (LPR == 16) {
      other(xor_lane<8>(at), xor_lane<8>(d), l ^ 8);
      other(xor_lane<9>(at), xor_lane<9>(d), l ^ 9);
      other(xor_lane<10>(at), xor_lane<10>(d), l ^ 10);
      other(xor_lane<11>(at), xor_lane<11>(d), l ^ 11);
      other(xor_lane<12>(at), xor_lane<12>(d), l ^ 12);
      other(xor_lane<13>(at), xor_lane<13>(d), l ^ 13);
      other(xor_lane<14>(at), xor_lane<14>(d), l ^ 14);
      other(xor_lane<15>(at), xor_lane<15>(d), l ^ 15);
    }
    if (first) row_terms[at] = total;
    wave_sync();
    if (NCH == 0 && !dense) {
      // rows are neighbours in memory: the wave writes them as one
      const int n = (int)min((int64_t)kRows, a.T - row0) * a.E, pieces = n / V;
      typename IO::type* dst = (typename IO::type*)a.grad + row0 * a.E;
      for (int c = lane; c < pieces; c += kWave) {
        float f[V];
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = terms[c * V + i];
        IO::store_piece(dst + c * V, f);
      }
      if (pieces * V + lane < n) IO::store(a.grad, row0 * a.E + pieces * V + lane, terms[pieces * V + lane]);
    } else if (live) {
      const bool any = inner != 0.0f || (ballot(have) >> (lane - l) & (LPR == 16 ? 0xFFFFull : 0xFFull)) != 0;
      // a token without a choice gets zeros, whatever its logits, and so does a row of -Inf, which has no score
      const float back = any && sum != 0.0f ? -inner / sum : 0.0f;
      if (NCH > 0) {
        typename IO::type* dst = (typename IO::type*)a.grad + row * a.E;
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
          const int c = j * LPR + l;
          if (c >= a.E / V) break;
          float t[V];
#pragma unroll
          for (int i = 0; i < V; ++i) t[i] = row_terms[c * V + i] + (any ? back * e[j][i] : 0.0f);
          IO::store_piece(dst + c * V, t);
        }
        if (a.E % V != 0 && last < a.E)
          IO::store(a.grad, row * a.E + last, row_terms[last] + (any ? back * rest : 0.0f));
      } else if (vec) {
        const typename IO::type* src = (const typename IO::type*)a.logits + base;
        typename IO::type* dst = (typename IO::type*)a.grad + row * a.E;
        for (int c = l; c < a.E / V; c += LPR) {
          float f[V], t[V];
#pragma unroll
          for (int i = 0; i < V; ++i) t[i] = row_terms[c * V + i];
          if (any) {
            IO::unpack(*(const typename IO::piece*)(src + c * V), f);
#pragma unroll
            for (int i = 0; i < V; ++i) t[i] += back * expf(clean_logit(f[i]) - m);
          }
          IO::store_piece(dst + c * V, t);
        }
      } else {
        for (int e = l; e < a.E; e += LPR) {
          float t = row_terms[e];
          if (any) t += back * expf(clean_logit(IO::load(a.logits, base + e)) - m);
          IO::store(a.grad, row * a.E + e, t);
        }
      }
    }
    wave_sync();
    if (first) row_terms[at] = 0.0f;
    wave_sync();
  }
}

}  // namespace ep
