// ep_int8.hpp -- int8 rows: quantising them; the rows of every expert.
#pragma once

#include "ep_route.hpp"  // F32 / Bf16 / F16 element access

namespace ep {

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
//
// m: the largest magnitude's bits (magnitudes order like unsigned integers, NaN
// and infinities above the rest).
__device__ __forceinline__ float int8_scale(uint32_t m) {
  return m >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : __uint_as_float(m) / 127.0f;
}

// The code by a 64-bit quotient, for rows of any scale.
__device__ __forceinline__ int8_t int8_code(float x, float scale) {
  if (!(scale > 0.0f)) return 0;
  const double q = rint((double)x / (double)scale);
  return (int8_t)(int)fmin(fmax(q, -127.0), 127.0);
}

// The code of x by a product with inv = 1 / scale, as its low byte: adding
// 1.5 * 2^23 rounds to a whole number (to even) and leaves it in the low bits.
// The rest d = x - r * scale is exact where |d| is near scale / 2 (a multiple of
// half a step of scale, below 2^24 of them), so |d| < scale / 2 says that r is
// the nearest code; `off` gathers the largest |d|.
__device__ __forceinline__ uint32_t int8_code_fast(float x, float scale, float inv, float& off) {
  const float t = x * inv + 12582912.0f;
  const float r = t - 12582912.0f;
  off = fmaxf(off, fabsf(__builtin_fmaf(-r, scale, x)));
  return __float_as_uint(t);
}

// The codes of 16 bytes of values.  Where a quotient lies on or within rounding of
// a border between two codes (one piece in some thousand) or the row's scale is
// tiny, they are done over in 64 bits.
template <typename IO>
struct Int8Piece {
  static constexpr int V = 16 / sizeof(typename IO::type);
  typedef uint32_t codes __attribute__((ext_vector_type(V / 4)));
  typedef codes codes_at1 __attribute__((aligned(1)));

  float scale, inv, half;
  bool plain;  // neither 1 / scale nor the rests leave the normal range
  __device__ __forceinline__ explicit Int8Piece(float s)
      : scale(s), inv(1.0f / s), half(0.5f * s), plain(s > 0x1p-100f) {}

  __device__ __forceinline__ codes operator()(u32x4 raw) const {
    float f[V];
    IO::unpack(raw, f);
    uint32_t b[V];
    float off = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) b[j] = int8_code_fast(f[j], scale, inv, off);
    if (!plain || off >= half) {
#pragma unroll
      for (int j = 0; j < V; ++j) b[j] = (uint8_t)int8_code(f[j], scale);
    }
    codes o;
#pragma unroll
    for (int j = 0; j < V / 4; ++j) {
      const uint32_t lo = __builtin_amdgcn_perm(b[4 * j + 1], b[4 * j], 0x0C0C0400u);
      const uint32_t hi = __builtin_amdgcn_perm(b[4 * j + 3], b[4 * j + 2], 0x0C0C0400u);
      o[j] = lo | hi << 16;
    }
    return o;
  }
};

__device__ __forceinline__ uint32_t wave_max_bits(uint32_t m) {
  for (int o = 32; o > 0; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, 64));
  return m;
}

// Rows of whole pieces held in registers, WAVES waves a row: a lane has NC pieces
// of 16 bytes, so every byte is read once.  Memory bounds it: 262144 x 4096 bf16 in
// 515 us, 6.25 TB/s.  Many rows take a wave each (no barrier); few rows four
// waves, for the latency.
template <typename IO, int WAVES, int NC>
__global__ __launch_bounds__(256) void quantize_rows_kernel(QuantArgs a) {
  typedef Int8Piece<IO> Piece;
  constexpr int V = Piece::V;
  constexpr int kRows = 4 / WAVES;
  __shared__ uint32_t part[4];
  const int lane = lane_id();
  const int wave = threadIdx.x / kWave;
  const int64_t row = (int64_t)blockIdx.x * kRows + (WAVES == 1 ? wave : 0);
  if (row >= a.N) return;
  const int chunks = a.H / V;
  const int c0 = (WAVES == 1 ? 0 : wave * kWave) + lane;
  const typename IO::type* src = (const typename IO::type*)a.x + row * a.stride;
  u32x4 raw[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = c0 + i * WAVES * kWave;
    raw[i] = u32x4{0, 0, 0, 0};
    if (c < chunks) raw[i] = __builtin_nontemporal_load((const typename IO::piece*)(src + c * V));
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < NC; ++i) m = IO::max_magnitude(m, raw[i]);
  m = wave_max_bits(IO::magnitude_bits(m));
  if (WAVES > 1) {
    if (lane == 0) part[wave] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WAVES; ++w) m = max(m, part[w]);
  }
  const float scale = int8_scale(m);
  if (threadIdx.x % (WAVES * kWave) == 0) a.scales[row] = scale;
  const Piece piece(scale);
  int8_t* dst = a.codes + row * a.H;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = c0 + i * WAVES * kWave;
    // one piece after the other: left alone, the compiler starts all eight of them
    // (fp32: 230 registers in place of 56, 2.8 TB/s in place of 6)
    asm volatile("" : "+v"(raw[i][0]), "+v"(raw[i][1]), "+v"(raw[i][2]), "+v"(raw[i][3]));
    const typename Piece::codes o = piece(raw[i]);
    if (c < chunks) __builtin_nontemporal_store(o, (typename Piece::codes_at1*)(dst + c * V));
  }
}

// Rows of any length, a workgroup a row: two passes, the second out of the caches.
constexpr int kQuantThreads = 256;

template <typename IO>
__global__ __launch_bounds__(kQuantThreads) void quantize_kernel(QuantArgs a) {
  typedef Int8Piece<IO> Piece;
  constexpr int V = Piece::V;
  __shared__ uint32_t part[kQuantThreads / kWave];
  const int64_t row = blockIdx.x;
  const int64_t base = row * a.stride;
  const typename IO::type* src = (const typename IO::type*)a.x + base;
  const int chunks = a.H / V;
  uint32_t m = 0;
#pragma unroll 4
  for (int c = threadIdx.x; c < chunks; c += kQuantThreads)
    m = IO::max_magnitude(m, *(const typename IO::piece*)(src + (int64_t)c * V));
  m = IO::magnitude_bits(m);
  const int last = chunks * V + (int)threadIdx.x;  // fewer than V values are left
  const float x = last < a.H ? IO::load(a.x, base + last) : 0.0f;
  m = wave_max_bits(max(m, __float_as_uint(x) & 0x7FFFFFFFu));
  if (lane_id() == 0) part[threadIdx.x / kWave] = m;
  __syncthreads();
  for (int w = 0; w < kQuantThreads / kWave; ++w) m = max(m, part[w]);
  const float scale = int8_scale(m);
  if (threadIdx.x == 0) a.scales[row] = scale;
  const Piece piece(scale);
  int8_t* dst = a.codes + row * a.H;
  for (int c = threadIdx.x; c < chunks; c += kQuantThreads)
    *(typename Piece::codes_at1*)(dst + (int64_t)c * V) = piece(*(const typename IO::piece*)(src + (int64_t)c * V));
  if (last < a.H) dst[last] = int8_code(x, scale);
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
