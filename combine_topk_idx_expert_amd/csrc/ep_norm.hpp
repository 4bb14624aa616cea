// ep_norm.hpp -- root-mean-square norm of rows, with the residual's addition
// and E4M3 output; its gradient; E4M3 quantising of rows.
#pragma once

#include "ep_route.hpp"  // F32 / Bf16 / F16 element access

namespace ep {

// ------------------------------------------------------------------ E4M3 codes

// The scale of a block of channels from the largest magnitude's bits (they order
// like the magnitudes, NaN above infinity): amax / 448, correctly rounded.
__device__ __forceinline__ float e4m3_scale(uint32_t m) {
  if (m >= 0x7F800000u) return __uint_as_float(m > 0x7F800000u ? 0x7FC00000u : 0x7F800000u);
  return __uint_as_float(m) / 448.0f;
}

// Codes of four values, E4M3 of the fp32 quotient x / scale.  A scale of 0 (zeros,
// and magnitudes below 448 times the smallest fp32 value) gives signed zeros.  A
// subnormal scale is so coarse that quotients pass 448: they are cut there.
__device__ __forceinline__ uint32_t e4m3_codes4(const float* x, float scale) {
  const uint32_t m = __float_as_uint(scale);
  float q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    q[i] = m == 0 ? __builtin_copysignf(0.0f, x[i]) : x[i] / scale;
    q[i] = __builtin_amdgcn_fmed3f(q[i], -448.0f, 448.0f);
  }
  uint32_t w = e4m3x4_hw(q[0], q[1], q[2], q[3]);
  if (__builtin_expect(m >= 0x7F800000u, 0)) {
    // a block holding NaN has codes 0x7F; one of infinities 0x7F for those and signed zeros
    w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t b = __float_as_uint(x[i]);
      w |= (m > 0x7F800000u || (b & 0x7FFFFFFFu) >= 0x7F800000u ? 0x7Fu : (b >> 24) & 0x80u) << (8 * i);
    }
  }
  return w;
}

typedef uint32_t u32x2_at1 __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t u32_at1 __attribute__((aligned(1)));

// V codes (4 or 8) to any address; the last ones of a row one by one.
template <int V>
__device__ __forceinline__ void store_codes(uint8_t* p, const uint32_t* w, int left) {
  if (left >= V) {
    if constexpr (V == 8)
      __builtin_nontemporal_store(u32x2{w[0], w[1]}, (u32x2_at1*)p);
    else
      __builtin_nontemporal_store(w[0], (u32_at1*)p);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j < left) p[j] = (uint8_t)(w[j / 4] >> (8 * (j % 4)));
  }
}

// The largest of the magnitudes' bits over the lanes that share a block of 128
// channels: 16 lanes of eight values, or 32 of four.
template <int V>
__device__ __forceinline__ uint32_t block_max(uint32_t m) {
  m = row16_max_u32(m);
  if constexpr (V == 4) m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
  return m;
}

struct QuantFp8Args {
  const void* x;
  int64_t stride;  // elements between rows of x
  uint8_t* codes;  // [N][H]
  float* scales;   // block b of row r at r * row_step + b * block_step
  int64_t row_step, block_step;
  uint32_t N;
  int H;
  uint32_t nb;  // blocks of a row
};

// Sixteen lanes a block of 128 channels, eight values a lane, whatever the row's
// length.  Bound by memory: DESIGN's table has its rate.
template <typename IO>
__global__ __launch_bounds__(256) void quantize_fp8_kernel(QuantFp8Args a) {
  constexpr int V = 16 / sizeof(typename IO::type);
  const uint32_t b = blockIdx.x * 16 + threadIdx.x / 16;
  const uint32_t row = b / a.nb;  // (N * nb < 2^31)
  const uint32_t blk = b - row * a.nb;
  const bool any = row < a.N;
  const int col = (int)blk * 128 + (int)(threadIdx.x % 16) * 8;
  const int left = any ? a.H - col : 0;
  const int64_t base = (int64_t)row * a.stride + col;
  float f[8];
  if (left >= 8) {
#pragma unroll
    for (int j = 0; j < 8; j += V)
      IO::unpack(__builtin_nontemporal_load((const typename IO::piece*)((const typename IO::type*)a.x + base + j)), f + j);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = j < left ? IO::load(a.x, base + j) : 0.0f;
  }
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(f[j]) & 0x7FFFFFFFu);
  m = row16_max_u32(m);
  const float scale = e4m3_scale(m);
  if (!any) return;
  if (threadIdx.x % 16 == 0) a.scales[row * a.row_step + blk * a.block_step] = scale;
  const uint32_t w[2] = {e4m3_codes4(f, scale), e4m3_codes4(f + 4, scale)};
  store_codes<8>(a.codes + (int64_t)row * a.H + col, w, left);
}

// ------------------------------------------------------------------------ norm

struct NormArgs {
  const void* x;
  const void* residual;  // null: none
  const void* weight;    // [H]
  void* total;           // [N][H] x + residual; null without a residual
  void* y;               // [N][H] or null
  uint8_t* codes;        // [N][H] or null
  float* scales;         // [N][nb]
  int64_t x_stride, r_stride;
  int64_t N;
  int H;
  int weight32;  // the weight is fp32
  float eps;
};

// 16 bytes of a row from element `at` on, `left` of them the row's; zeros behind it.
template <typename IO, int V>
__device__ __forceinline__ void load_values(const void* p, int64_t at, int left, float* f) {
  if (left >= V) {
    IO::unpack(__builtin_nontemporal_load((const typename IO::piece*)((const typename IO::type*)p + at)), f);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] = j < left ? IO::load(p, at + j) : 0.0f;
  }
}

template <typename IO, int V>
__device__ __forceinline__ void store_values(void* p, int64_t at, int left, const float* f) {
  if (left >= V) {
    IO::store_piece((typename IO::type*)p + at, f);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j < left) IO::store(p, at + j, f[j]);
  }
}

// V weights from column c on; they are read for every row and stay in the caches.
template <typename IO, int V>
__device__ __forceinline__ void load_weight(const void* p, int weight32, int c, int left, float* f) {
  if (left < V) {
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] = j < left ? (weight32 ? F32::load(p, c + j) : IO::load(p, c + j)) : 0.0f;
  } else if (weight32) {
#pragma unroll
    for (int j = 0; j < V; j += 4) F32::unpack(*(const F32::piece*)((const float*)p + c + j), f + j);
  } else {
    IO::unpack(*(const typename IO::piece*)((const typename IO::type*)p + c), f);
  }
}

__device__ __forceinline__ float wave_sum(float v) {
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// Sum (or maximum of bits) over the W waves that share a row.  `part` has room for
// W values; calls that follow each other use different room.
template <int W>
__device__ __forceinline__ float team_sum(float v, float* part) {
  v = wave_sum(v);
  if constexpr (W > 1) {
    if (lane_id() == 0) part[threadIdx.x / kWave] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int w = 1; w < W; ++w) v += part[w];
  }
  return v;
}
template <int W>
__device__ __forceinline__ uint32_t team_max(uint32_t v, uint32_t* part) {
  for (int o = 32; o > 0; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o, 64));
  if constexpr (W > 1) {
    if (lane_id() == 0) part[threadIdx.x / kWave] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int w = 1; w < W; ++w) v = max(v, part[w]);
  }
  return v;
}

// Squares that leave fp32: sums above this lost some to infinity or may soon; small
// ones lost some to zero, which shows if eps is as small.
__device__ __forceinline__ bool squares_left_range(float ss, float eps) {
  return !(ss < 0x1p120f) || (ss < 0x1p-80f && eps < 0x1p-60f);
}

// Power of two for the row of largest magnitude m (its bits): large ones come to 2^50,
// where 2^15 squares still fit and values 2^-100 of the largest keep their bits, small
// ones near 1, but never so far up that eps scaled likewise would leave fp32.  An
// infinity or NaN stays what it is.
__device__ __forceinline__ int scale_exponent(uint32_t m) {
  const int e = (int)(m >> 23) - 127;
  return e > 0 ? 50 - e : min(-e, 60);
}

// W waves a row (W = 1: four rows a workgroup), NC pieces of 16 bytes a lane: the row
// stays in fp32 registers from its one read to the outputs, so each byte moves
// once.  Sums of squares are fp32 in a fixed order.  y is formed from the unrounded
// sum x + residual; the stored sum is that value rounded once.  Memory bounds it; the
// launch code says which rows take how many waves.
template <typename IO, int W, int NC>
__global__ __launch_bounds__(W < 4 ? 256 : W * kWave) void norm_kernel(NormArgs a) {
  constexpr int V = 16 / sizeof(typename IO::type);
  __shared__ float part[3][W];
  const int64_t row = W == 1 ? (int64_t)blockIdx.x * 4 + threadIdx.x / kWave : blockIdx.x;
  if (row >= a.N) return;  // (W == 1: no barrier follows)
  const int t = W == 1 ? lane_id() : (int)threadIdx.x;
  float f[NC][V];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = (t + i * W * kWave) * V;
    load_values<IO, V>(a.x, row * a.x_stride + c, a.H - c, f[i]);
  }
  if (a.residual) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = (t + i * W * kWave) * V;
      float r[V];
      load_values<IO, V>(a.residual, row * a.r_stride + c, a.H - c, r);
#pragma unroll
      for (int j = 0; j < V; ++j) f[i][j] += r[j];
      store_values<IO, V>(a.total, row * a.H + c, a.H - c, f[i]);
    }
  }
  auto squares = [&]() {
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) ss = __builtin_fmaf(f[i][j], f[i][j], ss);
    return ss;
  };
  float ss = team_sum<W>(squares(), part[0]);
  float eps = a.eps;
  if (__builtin_expect(squares_left_range(ss, eps), 0)) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) m = max(m, __float_as_uint(f[i][j]) & 0x7FFFFFFFu);
    const int e = scale_exponent(team_max<W>(m, (uint32_t*)part[1]));
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) f[i][j] = ldexpf(f[i][j], e);
    eps = ldexpf(eps, 2 * e);
    ss = team_sum<W>(squares(), part[2]);
  }
  const float r = 1.0f / sqrtf(ss / (float)a.H + eps);
  const int nb = (a.H + 127) / 128;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = (t + i * W * kWave) * V;
    const int left = a.H - c;
    float w[V];
    load_weight<IO, V>(a.weight, a.weight32, c, left, w);
#pragma unroll
    for (int j = 0; j < V; ++j) f[i][j] *= r * w[j];
    if (a.y) store_values<IO, V>(a.y, row * a.H + c, left, f[i]);
    if (a.codes) {
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < V; ++j) m = max(m, __float_as_uint(f[i][j]) & 0x7FFFFFFFu);
      m = block_max<V>(m);
      const float scale = e4m3_scale(m);
      if (left > 0) {
        if (c % 128 == 0) a.scales[row * nb + c / 128] = scale;
        uint32_t o[V / 4];
#pragma unroll
        for (int j = 0; j < V / 4; ++j) o[j] = e4m3_codes4(f[i] + 4 * j, scale);
        store_codes<V>(a.codes + row * a.H + c, o, left);
      }
    }
  }
}

// -------------------------------------------------------------------- gradient

struct NormBwdArgs {
  const void* x;        // what was normalised
  const void* weight;   // [H]
  const void* grad;     // [N][H] of y
  const void* through;  // [N][H] added to the gradient of x; null: none
  void* grad_x;         // [N][H]
  float* partial;       // [teams][H]
  int64_t x_stride, g_stride, t_stride;
  int64_t N;
  int teams;
  int H;
  int weight32;
  float eps;
};

// With n = x / rms and rms = sqrt(mean x^2 + eps):
//   dx = (g w - n mean(g w n)) / rms,   dw = sum over rows of g n.
// A team of W waves (W = 1: four teams a workgroup) takes every teams-th row, holds x
// and g of it in registers and the weight's gradient of its columns over all its rows;
// those sums are joined by norm_weight_kernel in a fixed order.  The two sums over a
// row share one barrier, and rows in turn use one of two places for them.
template <typename IO, int W, int NC>
__global__ __launch_bounds__(W < 4 ? 256 : W * kWave) void norm_backward_kernel(NormBwdArgs a) {
  constexpr int V = 16 / sizeof(typename IO::type);
  __shared__ float part[2][2][W];
  __shared__ float redo[3][W];
  const int wave = threadIdx.x / kWave;
  const int team = W == 1 ? (int)blockIdx.x * 4 + wave : (int)blockIdx.x;
  if (team >= a.teams) return;  // (W == 1: no barrier follows)
  const int t = W == 1 ? lane_id() : (int)threadIdx.x;
  float dw[NC][V];
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) dw[i][j] = 0.0f;
  int turn = 0;
  for (int64_t row = team; row < a.N; row += a.teams, turn ^= 1) {
    float x[NC][V], g[NC][V];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = (t + i * W * kWave) * V;
      load_values<IO, V>(a.x, row * a.x_stride + c, a.H - c, x[i]);
      load_values<IO, V>(a.grad, row * a.g_stride + c, a.H - c, g[i]);
    }
    float ss = 0.0f, dot = 0.0f;
    auto sums = [&]() {
      ss = dot = 0.0f;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int c = (t + i * W * kWave) * V;
        float w[V];
        load_weight<IO, V>(a.weight, a.weight32, c, a.H - c, w);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          ss = __builtin_fmaf(x[i][j], x[i][j], ss);
          dot = __builtin_fmaf(g[i][j] * w[j], x[i][j], dot);
        }
      }
      ss = wave_sum(ss);
      dot = wave_sum(dot);
    };
    sums();
    if constexpr (W > 1) {
      float(*p)[W] = part[turn];
      if (lane_id() == 0) {
        p[0][wave] = ss;
        p[1][wave] = dot;
      }
      __syncthreads();
      ss = p[0][0];
      dot = p[1][0];
#pragma unroll
      for (int w = 1; w < W; ++w) {
        ss += p[0][w];
        dot += p[1][w];
      }
    }
    float eps = a.eps, back = 1.0f;
    if (__builtin_expect(squares_left_range(ss, eps), 0)) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) m = max(m, __float_as_uint(x[i][j]) & 0x7FFFFFFFu);
      const int e = scale_exponent(team_max<W>(m, (uint32_t*)redo[0]));
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) x[i][j] = ldexpf(x[i][j], e);
      eps = ldexpf(eps, 2 * e);
      back = ldexpf(1.0f, e);
      sums();
      if constexpr (W > 1) {
        if (lane_id() == 0) {
          redo[1][wave] = ss;
          redo[2][wave] = dot;
        }
        __syncthreads();
        ss = redo[1][0];
        dot = redo[2][0];
#pragma unroll
        for (int w = 1; w < W; ++w) {
          ss += redo[1][w];
          dot += redo[2][w];
        }
        __syncthreads();  // the next row may come here too
      }
    }
    const float r = 1.0f / sqrtf(ss / (float)a.H + eps);
    const float mean = dot * r / (float)a.H;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = (t + i * W * kWave) * V;
      const int left = a.H - c;
      float w[V], d[V];
      load_weight<IO, V>(a.weight, a.weight32, c, left, w);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float n = x[i][j] * r;
        dw[i][j] = __builtin_fmaf(g[i][j], n, dw[i][j]);
        d[j] = (g[i][j] * w[j] - n * mean) * r * back;
      }
      if (a.through) {
        float p[V];
        load_values<IO, V>(a.through, row * a.t_stride + c, left, p);
#pragma unroll
        for (int j = 0; j < V; ++j) d[j] += p[j];
      }
      store_values<IO, V>(a.grad_x, row * a.H + c, left, d);
    }
  }
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = (t + i * W * kWave) * V;
#pragma unroll
    for (int j = 0; j < V; j += 4) {
      if (c + j + 4 <= a.H)
        *(u32x4_at4*)(a.partial + (int64_t)team * a.H + c + j) =
            u32x4{__float_as_uint(dw[i][j]), __float_as_uint(dw[i][j + 1]), __float_as_uint(dw[i][j + 2]),
                  __float_as_uint(dw[i][j + 3])};
      else
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (c + j + k < a.H) a.partial[(int64_t)team * a.H + c + j + k] = dw[i][j + k];
    }
  }
}

// grad_w[c] = sum over the teams of partial[.][c], in a fixed order: 32 columns a
// workgroup, 32 slices of teams.
__global__ __launch_bounds__(1024) void norm_weight_kernel(const float* __restrict__ partial, int teams, int H,
                                                           float* __restrict__ grad_w) {
  __shared__ float part[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x % 32;
  const int s = threadIdx.x / 32;
  float sum = 0.0f;
  if (c < H) {
#pragma unroll 8
    for (int k = s; k < teams; k += 32) sum += partial[(int64_t)k * H + c];
  }
  part[s][threadIdx.x % 32] = sum;
  __syncthreads();
  if (s == 0 && c < H) {
#pragma unroll
    for (int k = 1; k < 32; ++k) sum += part[k][threadIdx.x];
    grad_w[c] = sum;
  }
}

}  // namespace ep
