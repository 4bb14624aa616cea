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

// Codes of four values, E4M3 of the fp32 quotient x / scale, for any scale.  A scale of 0
// (zeros, and magnitudes below 448 times the smallest fp32 value) gives signed zeros.  A
// subnormal scale is so coarse that quotients pass 448: they are cut there.
__device__ __forceinline__ uint32_t e4m3_divided4(const float* x, float scale) {
  const uint32_t m = __float_as_uint(scale);
  float q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    q[i] = m == 0 ? __builtin_copysignf(0.0f, x[i]) : x[i] / scale;
    q[i] = __builtin_amdgcn_fmed3f(q[i], -448.0f, 448.0f);
  }
  uint32_t w = e4m3x4_hw(q[0], q[1], q[2], q[3]);
  if (m >= 0x7F800000u) {
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

// The same by products with both ends of an interval around 1 / scale that holds the fp32
// rounding of x / scale for every x: where E4M3 rounds both products to one code, that is the
// quotient's.  `doubt` gathers the others (one value in some 100000).
__device__ __forceinline__ uint32_t e4m3_codes4(const float* x, float inv_lo, float inv_hi, uint32_t& doubt) {
  const uint32_t w = e4m3x4_hw(x[0] * inv_lo, x[1] * inv_lo, x[2] * inv_lo, x[3] * inv_lo);
  doubt |= w ^ e4m3x4_hw(x[0] * inv_hi, x[1] * inv_hi, x[2] * inv_hi, x[3] * inv_hi);
  return w;
}

// V codes (4 or 8); those in doubt, and blocks whose scale or quotients may leave the normal
// range, by division.  The reciprocal is off by 2^-23, three products and the quotient by
// 2^-24 each: less than 2^-21.
template <int V>
__device__ __forceinline__ void e4m3_codes(const float* x, float scale, uint32_t* w) {
  uint32_t doubt = scale > 0x1p-100f && scale < 0x1p100f ? 0 : 1;
  const float inv = __builtin_amdgcn_rcpf(scale);
  const float inv_lo = inv * (1.0f - 0x1p-21f), inv_hi = inv * (1.0f + 0x1p-21f);
#pragma unroll
  for (int j = 0; j < V / 4; ++j) w[j] = e4m3_codes4(x + 4 * j, inv_lo, inv_hi, doubt);
  if (__builtin_expect(doubt != 0, 0)) {
#pragma unroll
    for (int j = 0; j < V / 4; ++j) w[j] = e4m3_divided4(x + 4 * j, scale);
  }
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
// channels: 16 lanes of eight values, or 32 of four (of L lanes of a row).
template <int V, int L>
__device__ __forceinline__ uint32_t block_max(uint32_t m) {
  m = row16_max_u32(m);
  if constexpr (V == 4 && L > 16) m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
  return m;
}

// Blocks of a lane: two of 16-bit values (32768 x 4096 bf16: 77 us, with one 83, with four 76),
// one of fp32 (111; 114).
template <typename IO>
constexpr int kQuantBlocks = sizeof(typename IO::type) == 2 ? 2 : 1;

struct QuantFp8Args {
  const void* x;
  int64_t stride;  // elements between rows of x
  uint8_t* codes;  // [N][H]
  float* scales;   // block b of row r at r * row_step + b * block_step
  int64_t row_step, block_step;
  uint32_t N;
  int H;
  uint32_t nb;     // blocks of a row
  uint32_t magic;  // b / nb = b * magic >> shift for b < 2^31
  int shift;
};

// Sixteen lanes a block of 128 channels, eight values a lane, whatever the row's length; a
// lane has kBlocks blocks and asks for all of them first.  Memory and vector instructions
// (some 70 a block and lane) bound it: 65536 x 2048 bf16 75 us, 5.4 TB/s.
template <typename IO>
__global__ __launch_bounds__(256) void quantize_fp8_kernel(QuantFp8Args a) {
  typedef typename IO::type T;
  constexpr int V = 16 / sizeof(T), kBlocks = kQuantBlocks<IO>;
  const int lane_col = (int)(threadIdx.x % 16) * 8;
  uint32_t row[kBlocks], blk[kBlocks];
  int left[kBlocks];
  u32x4 raw[kBlocks][8 / V];
#pragma unroll
  for (int k = 0; k < kBlocks; ++k) {
    const uint32_t b = (blockIdx.x * kBlocks + k) * 16 + threadIdx.x / 16;
    row[k] = (uint32_t)((uint64_t)b * a.magic >> a.shift);
    blk[k] = b - row[k] * a.nb;
    const int col = (int)blk[k] * 128 + lane_col;
    left[k] = row[k] < a.N ? a.H - col : 0;
    const T* src = (const T*)a.x + ((int64_t)row[k] * a.stride + col);
#pragma unroll
    for (int j = 0; j < 8 / V; ++j) {
      raw[k][j] = u32x4{0, 0, 0, 0};
      if (left[k] >= 8) raw[k][j] = __builtin_nontemporal_load((const typename IO::piece*)(src + j * V));
    }
    if (a.H % 8 != 0 && left[k] > 0 && left[k] < 8) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t v = 0;
        if (j < left[k]) v = V == 8 ? (uint32_t)((const uint16_t*)src)[j] : ((const uint32_t*)src)[j];
        raw[k][j / V][j % V * 4 / V] |= v << (V == 8 ? 16 * (j % 2) : 0);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kBlocks; ++k) {
    float f[8];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8 / V; ++j) {
      m = IO::max_magnitude(m, raw[k][j]);
      IO::unpack(raw[k][j], f + j * V);
    }
    m = row16_max_u32(IO::magnitude_bits(m));
    const float scale = e4m3_scale(m);
    if (row[k] < a.N) {
      if (threadIdx.x % 16 == 0) a.scales[row[k] * a.row_step + blk[k] * a.block_step] = scale;
      uint32_t w[2];
      e4m3_codes<8>(f, scale, w);
      store_codes<8>(a.codes + (int64_t)row[k] * a.H + (int)blk[k] * 128 + lane_col, w, left[k]);
    }
  }
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

// 16 bytes of a row from column c on; zeros past the row's end.
template <typename IO>
__device__ __forceinline__ u32x4 load_piece(const typename IO::type* src, int c, int H) {
  constexpr int V = 16 / sizeof(typename IO::type);
  u32x4 raw{0, 0, 0, 0};
  if (c + V <= H) raw = __builtin_nontemporal_load((const typename IO::piece*)(src + c));
  return raw;
}
// The last piece of a row that does not hold whole ones.
template <typename IO>
__device__ __forceinline__ void load_tail(const typename IO::type* src, int c, int H, u32x4& raw) {
  constexpr int V = 16 / sizeof(typename IO::type);
  if (c < H && c + V > H) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      uint32_t b = 0;
      if (c + j < H) b = V == 8 ? (uint32_t)((const uint16_t*)src)[c + j] : ((const uint32_t*)src)[c + j];
      raw[j * 4 / V] |= b << (V == 8 ? 16 * (j % 2) : 0);
    }
  }
}

// The pieces of a row that a lane has: piece i begins at column (t + i * STEP) * V.  All are
// asked for before the first is used.
template <typename IO, int NC, int STEP>
struct RowPieces {
  static constexpr int V = 16 / sizeof(typename IO::type);
  u32x4 raw[NC];
  __device__ __forceinline__ void load(const void* p, int64_t row_at, int t, int H) {
    const typename IO::type* src = (const typename IO::type*)p + row_at;
#pragma unroll
    for (int i = 0; i < NC; ++i) raw[i] = load_piece<IO>(src, (t + i * STEP) * V, H);
    if (H % V != 0) {
#pragma unroll
      for (int i = 0; i < NC; ++i) load_tail<IO>(src, (t + i * STEP) * V, H, raw[i]);
    }
  }
};

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

// A row is a team's of L lanes: 16 or 32 (several rows a wave), 64, or whole waves.
template <int L>
__device__ __forceinline__ float team_lanes_sum(float v) {
  constexpr int kLanes = L < kWave ? L : kWave;
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// Sum (or maximum of bits) over a team.  `part` has room for a value of each of its waves;
// calls that follow each other use different room.
template <int L>
__device__ __forceinline__ float team_sum(float v, float* part) {
  v = team_lanes_sum<L>(v);
  if constexpr (L > kWave) {
    if (lane_id() == 0) part[threadIdx.x / kWave] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int w = 1; w < L / kWave; ++w) v += part[w];
  }
  return v;
}
template <int L>
__device__ __forceinline__ uint32_t team_max(uint32_t v, uint32_t* part) {
  constexpr int kLanes = L < kWave ? L : kWave;
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o, 64));
  if constexpr (L > kWave) {
    if (lane_id() == 0) part[threadIdx.x / kWave] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int w = 1; w < L / kWave; ++w) v = max(v, part[w]);
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

// L lanes a row (up to 64: 256 / L rows a workgroup), NC pieces of 16 bytes a lane: the row
// stays in fp32 registers from its one read to the outputs, so each byte moves
// once.  Sums of squares are fp32 in a fixed order.  y is formed from the unrounded
// sum x + residual; the stored sum is that value rounded once.  Memory bounds it
// (32768 x 7168 bf16 with residual, rows and codes 364 us, 5.8 TB/s); the launch code says
// which rows take how many lanes.
template <typename IO, int L, int NC>
__global__ __launch_bounds__(L <= kWave ? 256 : L) void norm_kernel(NormArgs a) {
  constexpr int V = 16 / sizeof(typename IO::type);
  __shared__ float part[3][L <= kWave ? 1 : L / kWave];
  const int64_t row = L <= kWave ? (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L : blockIdx.x;
  if (row >= a.N) return;  // (up to 64 lanes: no barrier follows, and no lane of another row is asked)
  const int t = threadIdx.x % L;
  float f[NC][V];
  RowPieces<IO, NC, L> x, res;
  x.load(a.x, row * a.x_stride, t, a.H);
  if (a.residual) res.load(a.residual, row * a.r_stride, t, a.H);
#pragma unroll
  for (int i = 0; i < NC; ++i) IO::unpack(x.raw[i], f[i]);
  if (a.residual) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = (t + i * L) * V;
      float r[V];
      IO::unpack(res.raw[i], r);
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
  float ss = team_sum<L>(squares(), part[0]);
  float eps = a.eps;
  if (__builtin_expect(squares_left_range(ss, eps), 0)) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) m = max(m, __float_as_uint(f[i][j]) & 0x7FFFFFFFu);
    const int e = scale_exponent(team_max<L>(m, (uint32_t*)part[1]));
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) f[i][j] = ldexpf(f[i][j], e);
    eps = ldexpf(eps, 2 * e);
    ss = team_sum<L>(squares(), part[2]);
  }
  const float r = 1.0f / sqrtf(ss / (float)a.H + eps);
  const int nb = (a.H + 127) / 128;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = (t + i * L) * V;
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
      m = block_max<V, L>(m);
      const float scale = e4m3_scale(m);
      if (left > 0) {
        if (c % 128 == 0) a.scales[row * nb + c / 128] = scale;
        uint32_t o[V / 4];
        e4m3_codes<V>(f[i], scale, o);
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
  float* partial;       // [groups][H]
  int64_t x_stride, g_stride, t_stride;
  int64_t N;
  int groups;           // workgroups
  int H;
  int weight32;
  float eps;
};

// With n = x / rms and rms = sqrt(mean x^2 + eps):
//   dx = (g w - n mean(g w n)) / rms,   dw = sum over rows of g n.
// A team of L lanes (up to 64: 256 / L teams a workgroup) takes every kTeams * groups-th row,
// holds x and g of it in registers (as they were read: unpacking them twice costs less than
// their room) and the weight's gradient of its columns over all its rows.  A workgroup's teams
// join those at the end, and norm_weight_kernel those of all workgroups, in a fixed order.
// The two sums over a row share one barrier, and rows in turn use one of two places for
// them.  Where registers allow the weight stays in registers and the next row is on its way
// while a row is worked on.  Memory bounds it: 262144 x 4096 bf16 with the residual's gradient
// 1.60 ms, 5.4 TB/s; 32768 x 7168 319 us, 5.9.
template <typename IO, int L, int NC>
__global__ __launch_bounds__(L <= kWave ? 256 : L) void norm_backward_kernel(NormBwdArgs a) {
  constexpr int V = 16 / sizeof(typename IO::type);
  constexpr int W = L <= kWave ? 1 : L / kWave;
  constexpr int kTeams = L <= kWave ? 256 / L : 1;  // of a workgroup
  constexpr bool kAhead = NC * V <= (L == 256 ? 16 : 8);
  static_assert(kTeams == 1 || NC == 1, "a workgroup's teams join one piece a lane");
  __shared__ float part[2][2][W];
  __shared__ float redo[3][W];
  const int wave = threadIdx.x / kWave;
  const int teams = a.groups * kTeams;
  const int team = (int)blockIdx.x * kTeams + (kTeams > 1 ? (int)threadIdx.x / L : 0);
  const int t = threadIdx.x % L;
  auto column = [&](int i) { return (t + i * L) * V; };
  float dw[NC][V], kept[kAhead ? NC : 1][V];
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) dw[i][j] = 0.0f;
  if (kAhead) {
#pragma unroll
    for (int i = 0; i < NC; ++i) load_weight<IO, V>(a.weight, a.weight32, column(i), a.H - column(i), kept[kAhead ? i : 0]);
  }
  auto weight = [&](int i, float* w) {
    if (kAhead) {
#pragma unroll
      for (int j = 0; j < V; ++j) w[j] = kept[kAhead ? i : 0][j];
    } else {
      load_weight<IO, V>(a.weight, a.weight32, column(i), a.H - column(i), w);
    }
  };
  RowPieces<IO, NC, L> x, g, p, x1, g1, p1;
  auto fetch = [&](int64_t row, auto& x_, auto& g_, auto& p_) {
    x_.load(a.x, row * a.x_stride, t, a.H);
    g_.load(a.grad, row * a.g_stride, t, a.H);
    if (kAhead && a.through) p_.load(a.through, row * a.t_stride, t, a.H);
  };
  int turn = 0;
  if (kAhead && team < a.N) fetch(team, x1, g1, p1);
  for (int64_t row = team; row < a.N; row += teams, turn ^= 1) {
    if (kAhead) {
      x = x1;
      g = g1;
      p = p1;
      if (row + teams < a.N) fetch(row + teams, x1, g1, p1);
    } else {
      fetch(row, x, g, p);
    }
    float ss = 0.0f, dot = 0.0f;
    auto sums = [&](float up) {
      ss = dot = 0.0f;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        float w[V], xf[V], gf[V];
        weight(i, w);
        IO::unpack(x.raw[i], xf);
        IO::unpack(g.raw[i], gf);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float xs = xf[j] * up;
          ss = __builtin_fmaf(xs, xs, ss);
          dot = __builtin_fmaf(gf[j] * w[j], xs, dot);
        }
      }
      ss = team_lanes_sum<L>(ss);
      dot = team_lanes_sum<L>(dot);
    };
    sums(1.0f);
    if constexpr (W > 1) {
      float(*q)[W] = part[turn];
      if (lane_id() == 0) {
        q[0][wave] = ss;
        q[1][wave] = dot;
      }
      __syncthreads();
      ss = q[0][0];
      dot = q[1][0];
#pragma unroll
      for (int w = 1; w < W; ++w) {
        ss += q[0][w];
        dot += q[1][w];
      }
    }
    float eps = a.eps, up = 1.0f;
    if (__builtin_expect(squares_left_range(ss, eps), 0)) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        float xf[V];
        IO::unpack(x.raw[i], xf);
#pragma unroll
        for (int j = 0; j < V; ++j) m = max(m, __float_as_uint(xf[j]) & 0x7FFFFFFFu);
      }
      const int e = scale_exponent(team_max<L>(m, (uint32_t*)redo[0]));
      up = ldexpf(1.0f, e);
      eps = ldexpf(eps, 2 * e);
      sums(up);
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
      const int c = column(i);
      float w[V], xf[V], gf[V], d[V];
      weight(i, w);
      IO::unpack(x.raw[i], xf);
      IO::unpack(g.raw[i], gf);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float n = xf[j] * up * r;
        dw[i][j] = __builtin_fmaf(gf[j], n, dw[i][j]);
        d[j] = (gf[j] * w[j] - n * mean) * r * up;
      }
      if (a.through) {
        if (!kAhead) {
          const typename IO::type* src = (const typename IO::type*)a.through + row * a.t_stride;
          p.raw[i] = load_piece<IO>(src, c, a.H);
          if (a.H % V != 0) load_tail<IO>(src, c, a.H, p.raw[i]);
        }
        float q[V];
        IO::unpack(p.raw[i], q);
#pragma unroll
        for (int j = 0; j < V; ++j) d[j] += q[j];
      }
      store_values<IO, V>(a.grad_x, row * a.H + c, a.H - c, d);
    }
  }
  if constexpr (kTeams > 1) {
    __shared__ float sums_of[256][V + 1];
#pragma unroll
    for (int j = 0; j < V; ++j) sums_of[threadIdx.x][j] = dw[0][j];
    __syncthreads();
    if (threadIdx.x >= L) return;
    for (int k = 1; k < kTeams; ++k)
#pragma unroll
      for (int j = 0; j < V; ++j) dw[0][j] += sums_of[k * L + t][j];
  }
  float* const out = a.partial + (int64_t)blockIdx.x * a.H;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = column(i);
#pragma unroll
    for (int j = 0; j < V; j += 4) {
      if (c + j + 4 <= a.H) {
        *(u32x4_at4*)(out + c + j) = u32x4{__float_as_uint(dw[i][j]), __float_as_uint(dw[i][j + 1]),
                                           __float_as_uint(dw[i][j + 2]), __float_as_uint(dw[i][j + 3])};
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (c + j + k < a.H) out[c + j + k] = dw[i][j + k];
      }
    }
  }
}

// grad_w[c] = sum of partial[.][c], in a fixed order: 32 columns a workgroup, 32 slices of
// the rows of sums.
__global__ __launch_bounds__(1024) void norm_weight_kernel(const float* __restrict__ partial, int rows, int H,
                                                           float* __restrict__ grad_w) {
  __shared__ float part[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x % 32;
  const int s = threadIdx.x / 32;
  float sum = 0.0f;
  if (c < H) {
#pragma unroll 8
    for (int k = s; k < rows; k += 32) sum += partial[(int64_t)k * H + c];
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
