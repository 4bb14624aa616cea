// ep_int8.hpp -- int8 rows: quantising them, and their product with int8
// weights, scaled for each row (token) and each output channel.
#pragma once

#include "ep_route.hpp"  // F32 / Bf16 / F16 element access

namespace ep {

typedef int i32x4 __attribute__((ext_vector_type(4)));

struct QuantArgs {
  const void* x;
  int64_t stride;  // elements between rows of x
  int8_t* codes;   // [N][H]
  float* scales;   // [N]
  int64_t N;
  int H;
};

// scale = amax / 127 (fp32, correctly rounded), code = the whole number nearest
// to x / scale, ties to even, of the exact quotient.  A row of zeros has scale
// 0 and codes 0; a row holding NaN or an infinity has scale NaN and codes 0, so
// that what is made of it is NaN and seen.
__device__ __forceinline__ int8_t int8_code(float x, float scale) {
  if (!(scale > 0.0f)) return 0;
  const double q = rint((double)x / (double)scale);
  return (int8_t)(int)fmin(fmax(q, -127.0), 127.0);
}

constexpr int kQuantThreads = 256;

template <typename IO>
__global__ __launch_bounds__(kQuantThreads) void quantize_kernel(QuantArgs a) {
  __shared__ uint32_t part[kQuantThreads / kWave];
  const int64_t row = blockIdx.x;
  const int64_t base = row * a.stride;
  // magnitudes order like unsigned integers, NaN and infinities above the rest
  uint32_t m = 0;
  for (int i = threadIdx.x; i < a.H; i += kQuantThreads)
    m = max(m, __float_as_uint(IO::load(a.x, base + i)) & 0x7FFFFFFFu);
  for (int o = 32; o > 0; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, 64));
  if (lane_id() == 0) part[threadIdx.x / kWave] = m;
  __syncthreads();
  for (int w = 0; w < kQuantThreads / kWave; ++w) m = max(m, part[w]);
  const float scale = m >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : __uint_as_float(m) / 127.0f;
  if (threadIdx.x == 0) a.scales[row] = scale;
  for (int i = threadIdx.x; i < a.H; i += kQuantThreads)
    a.codes[row * a.H + i] = int8_code(IO::load(a.x, base + i), scale);
}

struct MatmulArgs {
  const int8_t* a;           // [M][K]
  const float* a_scale;      // [M]
  const int8_t* w;           // [G][N][K]; dense: [N][K]
  const float* w_scale;      // [G][N]
  const int64_t* row_start;  // [G], null: dense
  const int32_t* row_count;  // [G]
  void* out;                 // [M][N], gated: [M][N / 2]
  int64_t M;
  int G, N, K;
  int width;                 // columns of out
};

// Rows [lo, hi) of group g.  Ranges come from device memory the host has not
// seen, so they are cut to the rows that exist.
__device__ __forceinline__ void group_rows(const MatmulArgs& a, int g, int64_t& lo, int64_t& hi) {
  if (!a.row_start) {
    lo = 0;
    hi = a.M;
    return;
  }
  const int64_t s = a.row_start[g], n = a.row_count[g];
  const bool any = s >= 0 && s < a.M && n > 0;
  lo = any ? s : 0;
  hi = any ? (n < a.M - s ? s + n : a.M) : 0;
}

__device__ __forceinline__ float silu(float g) { return g / (1.0f + expf(-g)); }

// Product of 16-row tiles, four waves a workgroup, each with 16 output columns
// (gated: the gate and the up channel of 16 columns), straight from memory.
// v_mfma_i32_16x16x64_i8 with the weights as first operand: lane l holds 16
// bytes of channel l % 16 and of row l % 16 at k = (l / 16) * 16, and gets
// channels (l / 16) * 4 + 0..3 of row l % 16.
constexpr int kRowTile = 16;

template <typename IO, bool GATED>
__global__ __launch_bounds__(256) void matmul_rows_kernel(MatmulArgs a) {
  const int lane = lane_id();
  const int wave = threadIdx.x / kWave;
  const int g = blockIdx.y;
  int64_t lo, hi;
  group_rows(a, g, lo, hi);
  const int c0 = ((int)blockIdx.x * 4 + wave) * 16;
  if (c0 >= a.width) return;
  const int q = lane >> 4, r = lane & 15;
  const int8_t* w = a.w + (int64_t)g * a.N * a.K;
  const float* ws = a.w_scale + (int64_t)g * a.N;
  const int ch = min(c0 + r, a.width - 1);
  const int8_t* w0 = w + (int64_t)ch * a.K;
  const int8_t* w1 = GATED ? w0 + (int64_t)a.width * a.K : nullptr;
  for (int64_t m0 = lo + (int64_t)blockIdx.z * kRowTile; m0 < hi; m0 += (int64_t)gridDim.z * kRowTile) {
    const int64_t row = m0 + r;
    const int8_t* x = a.a + (row < hi ? row : hi - 1) * a.K;
    i32x4 acc0 = {0, 0, 0, 0}, acc1 = {0, 0, 0, 0};
    for (int k0 = 0; k0 < a.K; k0 += 64) {
      const int k = k0 + q * 16;
      i32x4 xv = {0, 0, 0, 0}, wv = {0, 0, 0, 0}, uv = {0, 0, 0, 0};
      if (k < a.K) {
        xv = *(const i32x4*)(x + k);
        wv = *(const i32x4*)(w0 + k);
        if (GATED) uv = *(const i32x4*)(w1 + k);
      }
      acc0 = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv, xv, acc0, 0, 0, 0);
      if (GATED) acc1 = __builtin_amdgcn_mfma_i32_16x16x64_i8(uv, xv, acc1, 0, 0, 0);
    }
    if (row < hi) {
      const float sa = a.a_scale[row];
      for (int i = 0; i < 4; ++i) {
        const int c = c0 + q * 4 + i;
        if (c >= a.width) break;
        float v = (float)acc0[i] * sa * ws[c];
        if (GATED) v = silu(v) * ((float)acc1[i] * sa * ws[a.width + c]);
        IO::store(a.out, row * a.width + c, v);
      }
    }
  }
}

// Rows of every expert of a handle: where they start in the expanded tensors
// and how many there are (fixed windows: those that were kept).
__global__ __launch_bounds__(256) void expert_rows_kernel(const int64_t* __restrict__ window_row_base,
                                                          const int64_t* __restrict__ expert_offset,
                                                          const int32_t* __restrict__ n_e, int E, int El, int cap,
                                                          int64_t* __restrict__ start, int32_t* __restrict__ count) {
  const int e = blockIdx.x * 256 + threadIdx.x;
  if (e >= E) return;
  const int r = e / El;
  int64_t off = expert_offset[(int64_t)r * (El + 1) + (e - r * El)];
  int64_t n = n_e[e];
  if (cap > 0) {
    off = off < cap ? off : cap;
    n = n < cap - off ? n : cap - off;
  }
  start[e] = window_row_base[r] + off;
  count[e] = (int32_t)n;
}

}  // namespace ep
