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
  int64_t least, most;       // groups of other sizes are not this launch's
};

// Rows [lo, hi) of group g, none if its size is not this launch's.  Ranges come
// from device memory the host has not seen, so they are cut to the rows that exist.
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
  if (hi - lo < a.least || hi - lo > a.most) hi = lo;
}

// g / (1 + exp(-g)).  Below -87 the quotient's denominator leaves fp32 while its value
// does not, so neither form lets it grow so far.
// For a 16-bit result the hardware's exp2 and reciprocal (a third of the operations),
// of the denominator times 2^-16: the exponent's rounding makes a relative error below
// 2^-17, where the result's own is 2^-9 or 2^-12; a score below 2^-142 is 0.
// For fp32, 1 + exp(-g) is exp(-g) below -60, and half the exponent twice stays in range.
template <typename IO>
__device__ __forceinline__ float silu(float g) {
  if (sizeof(typename IO::type) == 2) {
    const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(g, -1.44269504f, -16.0f));
    return g * (__builtin_amdgcn_rcpf(0x1p-16f + e) * 0x1p-16f);
  }
  if (g < -60.0f) {
    const float h = expf(0.5f * g);
    return g * h * h;
  }
  return g / (1.0f + expf(-g));
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00020000);
}

constexpr uint32_t kBeyond = 0x80000000u;  // past the size of every descriptor here: reads zero

typedef __attribute__((address_space(3))) uint8_t lds_byte;

// 16 or 4 bytes a lane from memory to dst + lane * 16 or 4.
__device__ __forceinline__ void load16_to_lds(__amdgpu_buffer_rsrc_t r, void* dst, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_byte*)dst, 16, (int)off, 0, 0, 0);
}
__device__ __forceinline__ void load4_to_lds(__amdgpu_buffer_rsrc_t r, void* dst, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_byte*)dst, 4, (int)off, 0, 0, 0);
}

// N neighbouring columns of one row of out, from fp32.
template <typename IO, int N>
__device__ __forceinline__ void store_row(const MatmulArgs& a, int64_t row, int col, int end, const float* v) {
  const int64_t at = row * a.width + col;
  if (N % 8 == 0 && col + N <= end) {
#pragma unroll
    for (int j = 0; j < N; j += 8) IO::store8(a.out, at + j, v + j);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (col + j < end) IO::store(a.out, at + j, v[j]);
  }
}

// Few rows to a weight matrix: the weights are read once, and the waves of a
// workgroup take a share of the inner dimension each, so that a narrow matrix
// keeps many loads in flight.  A workgroup has 16 * MT rows by NT channel tiles
// of 16; the KW waves join their sums, which are whole numbers and do not depend
// on the split, through LDS.  Bound by the memory where weights are many (32 groups
// of 3 rows, 7168 x 4096 gated: 149 us, 6.3 TB/s of weights), else by the loads of
// the CU with the most workgroups, ~24 bytes a clock (one row: 7.4 us).
//
// A wave has a ring of S stages of LDS to itself and no barrier before the end:
// it loads 128 bytes of its rows and channels straight into a stage, eight
// lanes a row (loads in the lanes' MFMA places ask for 64 pieces of 16 bytes
// each, four times the address work: 30 us against 12 at 256 x 7168 x 4096), and
// waits for its own loads alone.  LDS image: 128 bytes a row, chunk ^ (row & 7).
//
// v_mfma_i32_16x16x64_i8 with the weights as first operand: lane l holds 16
// bytes of channel l % 16 and of row l % 16, and gets channels (l / 16) * 4 +
// 0..3 of row l % 16.  The NO column tiles take their columns in turn, four at a
// time, so that a lane ends with 4 * NO neighbours.  GATED: the second half of
// the channel tiles are the ups of the first half's columns.
template <typename IO, bool GATED, int MT, int NT, int KW, int S>
__global__ __launch_bounds__(KW* kWave) void matmul_split_kernel(MatmulArgs a) {
  constexpr int NO = GATED ? NT / 2 : NT;
  constexpr int BC = 16 * NO;
  constexpr int kStage = (MT + NT) * 2048;
  constexpr int kLoads = 2 * (MT + NT);  // a wave and stage
  static_assert(S * (MT + NT) * 2 >= MT * NT, "the sums fit where the stages were");
  __shared__ __attribute__((aligned(1024))) uint8_t split_lds[KW * S * kStage];
  const int lane = lane_id();
  const int wave = uniform((int)threadIdx.x / kWave);
  const int g = blockIdx.z;
  int64_t lo, hi;
  group_rows(a, g, lo, hi);
  const int q = lane >> 4, r = lane & 15;
  const int K = a.K;
  const int c0 = (int)blockIdx.x * BC;
  const int cols = min(BC, a.width - c0);
  const int8_t* w = a.w + (int64_t)g * a.N * K;
  const float* ws = a.w_scale + (int64_t)g * a.N;
  const __amdgpu_buffer_rsrc_t rw = buffer_of(w + (int64_t)c0 * K, (int64_t)cols * K);
  const __amdgpu_buffer_rsrc_t ru = buffer_of(w + (int64_t)(c0 + (GATED ? a.width : 0)) * K, (int64_t)cols * K);
  const int steps = (K + 127) / 128;
  const int share = (steps + KW - 1) / KW;
  const int s0 = min(wave * share, steps), s1 = min(s0 + share, steps);
  const uint32_t chunk = (uint32_t)((lane & 7) ^ (lane >> 3)) * 16;
  const uint32_t w_off = (uint32_t)((lane >> 5) * 4 * NO + ((lane >> 3) & 3)) * K + chunk;
  const uint32_t a_off = (uint32_t)(lane >> 3) * K + chunk;
  uint8_t* const mine = split_lds + wave * (S * kStage);
  const int frag = r * 128 + ((q ^ (r & 7)) * 16);  // first half of a step; the second: ^ 64

  for (int64_t m0 = lo + (int64_t)blockIdx.y * (16 * MT); m0 < hi; m0 += (int64_t)gridDim.y * (16 * MT)) {
    const int rows = (int)min((int64_t)(16 * MT), hi - m0);
    const __amdgpu_buffer_rsrc_t ra = buffer_of(a.a + m0 * K, (int64_t)rows * K);
    i32x4 acc[MT][NT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[m][n] = i32x4{0, 0, 0, 0};
    // step s into stage d; a step past the share loads zeros, so that the count of loads stays
    auto load = [&](int s, int d) {
      const uint32_t k0 = (uint32_t)s * 128;
      uint8_t* st = mine + d * kStage;
      const bool in = s < s1;
      uint32_t oa = in && k0 + chunk < (uint32_t)K ? a_off + k0 : kBeyond;
      uint32_t ow = in ? w_off + k0 : kBeyond;
      asm("" : "+v"(oa), "+v"(ow));
#pragma unroll
      for (int j = 0; j < 2 * NT; ++j) {
        const int n = j / 2;
        load16_to_lds(n < NO ? rw : ru, st + j * 1024, ow + (uint32_t)((j % 2) * 8 * NO + n % NO * 4) * K);
      }
#pragma unroll
      for (int j = 0; j < 2 * MT; ++j) load16_to_lds(ra, st + NT * 2048 + j * 1024, oa + (uint32_t)(j * 8) * K);
    };
#pragma unroll
    for (int d = 0; d < S; ++d) load(s0 + d, d);
    int d = 0;
    for (int s = s0; s < s1; ++s) {
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kLoads * (S - 1)) : "memory");
      const uint8_t* st = mine + d * kStage + frag;
      const uint8_t* st1 = mine + d * kStage + (frag ^ 64);
      i32x4 wv[2][NT], av[2][MT];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int n = 0; n < NT; ++n) wv[h][n] = *(const i32x4*)((h ? st1 : st) + n * 2048);
#pragma unroll
        for (int m = 0; m < MT; ++m) av[h][m] = *(const i32x4*)((h ? st1 : st) + (NT + m) * 2048);
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the stage has been read: load over it
      load(s + S, d);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int n = 0; n < NT; ++n)
            acc[m][n] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[h][n], av[h][m], acc[m][n], 0, 0, 0);
      d = d + 1 == S ? 0 : d + 1;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();  // every wave has left its stages
    i32x4* const part = (i32x4*)split_lds;  // [KW][MT][NT][64]
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) part[((wave * MT + m) * NT + n) * kWave + lane] = acc[m][n];
    __syncthreads();
    // wave m of the row tiles joins and writes tile m
    for (int m = wave; m < MT; m += KW) {
      i32x4 sum[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        sum[n] = part[(m * NT + n) * kWave + lane];
#pragma unroll
        for (int k = 1; k < KW; ++k) sum[n] += part[((k * MT + m) * NT + n) * kWave + lane];
      }
      const int row = m * 16 + r;
      if (row < rows) {
        const float s = a.a_scale[m0 + row];
        const int col = c0 + q * 4 * NO;
        float v[NO * 4];
#pragma unroll
        for (int n = 0; n < NO; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = min(col + n * 4 + i, a.width - 1);
            float y = (float)sum[n][i] * s * ws[c];
            if (GATED) y = silu<IO>(y) * ((float)sum[n + NT / 2][i] * s * ws[a.width + c]);
            v[n * 4 + i] = y;
          }
        store_row<IO, NO * 4>(a, m0 + row, col, a.width, v);
      }
    }
    __syncthreads();
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
