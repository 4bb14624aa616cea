// ep_product.hpp -- products of rows with the weights of their group (expert) or
// with one matrix, the inner dimension contiguous in both: what their kernels
// share, and the kernel for few rows.
#pragma once

#include "ep_route.hpp"  // F32 / Bf16 / F16 element access

namespace ep {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// The arithmetic of a product: the matrix instruction on 16 bytes a lane of each
// operand (weights first), its sums, and what the scales belong to.
enum Scales { kNoScales, kRowScales, kBlockScales };

// int8 with a scale for each row and channel: sums are exact.
struct Int8Math {
  typedef i32x4 acc;
  static constexpr Scales kScales = kRowScales;
  static __device__ __forceinline__ acc mfma(i32x4 w, i32x4 a, acc c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(w, a, c, 0, 0, 0);
  }
};
// 16-bit values, sums in fp32.
struct Bf16Math {
  typedef f32x4 acc;
  typedef __bf16 operand __attribute__((ext_vector_type(8)));
  static constexpr Scales kScales = kNoScales;
  static __device__ __forceinline__ acc mfma(i32x4 w, i32x4 a, acc c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(operand, w), __builtin_bit_cast(operand, a), c, 0, 0, 0);
  }
  // 128 bytes of the inner dimension
  struct frag {
    i32x4 v[2];
  };
  static __device__ __forceinline__ frag make(i32x4 lo, i32x4 hi) { return frag{{lo, hi}}; }
};
struct F16Math {
  typedef f32x4 acc;
  typedef _Float16 operand __attribute__((ext_vector_type(8)));
  static constexpr Scales kScales = kNoScales;
  static __device__ __forceinline__ acc mfma(i32x4 w, i32x4 a, acc c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(operand, w), __builtin_bit_cast(operand, a), c, 0, 0, 0);
  }
  // 128 bytes of the inner dimension
  struct frag {
    i32x4 v[2];
  };
  static __device__ __forceinline__ frag make(i32x4 lo, i32x4 hi) { return frag{{lo, hi}}; }
};
// E4M3 with a scale for each 128 channels of a row and 128 x 128 of a weight: the
// products of a block are summed by the instruction, and scaled when they are added
// to the fp32 sums of all blocks.
// The instruction for 128 channels aligns groups of up to 16 products to the largest of
// them and cuts, toward zero, what lies 2^-14 and more below it.  Measured, in 2-norm: sums of
// normal values are 1.2e-5 off, with channels 50 times the others 6e-5, sums of one sign and
// exponents over the whole type 7e-5 too small.  The result's own rounding is 1.7e-3 for bf16
// and 2e-4 for fp16.  (Its operands' own scales, powers of two, are unused.)
struct Fp8Math {
  typedef f32x4 acc;
  typedef i32x8 frag;
  static constexpr Scales kScales = kBlockScales;
  static __device__ __forceinline__ frag make(i32x4 lo, i32x4 hi) {
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  }
  static __device__ __forceinline__ acc mfma128(const frag& w, const frag& a) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, acc{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0, 0, 0);
  }
};
// The same for fp32 results, which would show that: E4M3 values are bf16 values too, and
// the bf16 instruction adds in fp32 (at half the rate, and eight conversions for 16
// bytes).
struct Fp8ExactMath {
  typedef f32x4 acc;
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  struct frag {
    Bf16Math::operand v[4];
  };
  static constexpr Scales kScales = kBlockScales;
  static __device__ __forceinline__ frag make(i32x4 lo, i32x4 hi) {
    frag f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int codes = (j < 2 ? lo : hi)[j % 2 * 2 + i];
        const bf16x2 x = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, 1.0f, false);
        const bf16x2 y = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, 1.0f, true);
        f.v[j][4 * i] = x[0];
        f.v[j][4 * i + 1] = x[1];
        f.v[j][4 * i + 2] = y[0];
        f.v[j][4 * i + 3] = y[1];
      }
    return f;
  }
  static __device__ __forceinline__ acc mfma128(const frag& w, const frag& a) {
    acc c{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[j], a.v[j], c, 0, 0, 0);
    return c;
  }
};

struct MatmulArgs {
  const uint8_t* a;          // [M] rows of K bytes
  const float* a_scale;      // row scales: [M]; block scales: see a_row_step
  const uint8_t* w;          // [G][N] channels of K bytes; dense: [N]
  const float* w_scale;      // row scales: [G][N]; block scales: [G][N blocks][K blocks]
  const int64_t* row_start;  // [G], null: dense
  const int32_t* row_count;  // [G]
  void* out;                 // [M][N], gated: [M][N / 2]
  int64_t M;
  int G, N, K;
  int width;                 // columns of out
  int64_t least, most;       // groups of other sizes are not this launch's
  void* pre;                 // gated, 16-bit: [M][N], the product before the gate; or null
  int64_t a_row_step, a_block_step;  // block b of row r has scale a_scale[r * a_row_step + b * a_block_step]
  int slices;                // gradients: parts of the inner dimension, each with an out of its own; else 1
};

// Blocks of 128 channels of the weights: gated, each half has blocks of its own.
__device__ __forceinline__ const float* block_scales(const MatmulArgs& a, bool gated, int g, int col, bool up) {
  const int nb = (a.width + 127) / 128, kb = (a.K + 127) / 128;
  return a.w_scale + ((int64_t)g * nb * (gated ? 2 : 1) + (up ? nb : 0) + col / 128) * kb;
}

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
typedef __attribute__((address_space(1))) const uint8_t global_byte;

// 16 or 4 bytes a lane from memory to dst + lane * 16 or 4.
__device__ __forceinline__ void load16_to_lds(__amdgpu_buffer_rsrc_t r, void* dst, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_byte*)dst, 16, (int)off, 0, 0, 0);
}
__device__ __forceinline__ void load4_to_lds(__amdgpu_buffer_rsrc_t r, void* dst, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_byte*)dst, 4, (int)off, 0, 0, 0);
}

// Values [at, at + N) of out that lie before column `end`, from fp32; col is the first's.
template <typename IO, int N>
__device__ __forceinline__ void store_cols(void* out, int64_t at, int col, int end, const float* v) {
  if (N % 8 == 0 && col + N <= end) {
#pragma unroll
    for (int j = 0; j < N; j += 8) IO::store8(out, at + j, v + j);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (col + j < end) IO::store(out, at + j, v[j]);
  }
}

// The scaled sums of NT channel tiles of one row (tile n: columns col + 4 n + 0..3 of
// out; gated, the second half of the tiles are the ups of the first half's columns) to
// out, and before the gate to pre where it is asked for (PRE: 16-bit products may.  Asked in
// the gated int8 tiles, too, it took 209 registers for 203 and 17 scalar spills more).
template <typename IO, bool GATED, bool PRE, int NT>
__device__ __forceinline__ void store_row(const MatmulArgs& a, int64_t row, int col, int end, const float* y) {
  constexpr int NO = GATED ? NT / 2 : NT;
  if constexpr (GATED) {
    if (PRE && a.pre) {
      const int64_t at = row * a.N + col;
      store_cols<IO, NO * 4>(a.pre, at, col, end, y);
      store_cols<IO, NO * 4>(a.pre, at + a.width, col, end, y + NO * 4);
    }
    float v[NO * 4];
#pragma unroll
    for (int i = 0; i < NO * 4; ++i) v[i] = silu<IO>(y[i]) * y[i + NO * 4];
    store_cols<IO, NO * 4>(a.out, row * a.width + col, col, end, v);
  } else {
    store_cols<IO, NO * 4>(a.out, row * a.width + col, col, end, y);
  }
}

// Few rows to a weight matrix: the weights are read once, and the waves of a
// workgroup take a share of the inner dimension each, so that a narrow matrix
// keeps many loads in flight.  A workgroup has 16 * MT rows by NT channel tiles
// of 16; the KW waves join their sums, in a fixed order, through LDS.  For int8, bound by the
// memory where weights are many (32 groups of 3 rows, 7168 x 4096 gated: 154 us, 6.1 TB/s
// of weights), else by the loads of the CU with the most workgroups, ~24 bytes a clock
// (one row: 7.4 us).
//
// A wave has a ring of S stages of LDS to itself and no barrier before the end:
// it loads 128 bytes of its rows and channels straight into a stage, eight
// lanes a row (loads in the lanes' MFMA places ask for 64 pieces of 16 bytes
// each, four times the address work: 30 us against 12 at 256 x 7168 x 4096), and
// waits for its own loads alone.  LDS image: 128 bytes a row, chunk ^ (row & 7).
//
// A matrix instruction has the weights as first operand: lane l holds 16
// bytes of channel l % 16 and of row l % 16, and gets channels (l / 16) * 4 +
// 0..3 of row l % 16.  The NO column tiles take their columns in turn, four at a
// time, so that a lane ends with 4 * NO neighbours.  GATED: the second half of
// the channel tiles are the ups of the first half's columns.
//
// E4M3 rows and 16-bit rows take the same way: 32 groups of 3 E4M3 rows, 7168 x 4096 gated,
// 162 us, 5.8 TB/s of weights, of 16-bit rows 303 us, 6.2; one row 6.8 us, a 16-bit one 10.5.
//
// Block scales: a step is a block, so its scales are loaded with it, one float a lane:
// rows 0..16 * MT - 1, then the columns' block of the weights (gated: two).
template <typename AR, typename IO, bool GATED, int MT, int NT, int KW, int S>
__global__ __launch_bounds__(KW* kWave) void matmul_split_kernel(MatmulArgs a) {
  constexpr int NO = GATED ? NT / 2 : NT;
  constexpr int BC = 16 * NO;
  constexpr bool kBlocks = AR::kScales == kBlockScales;
  constexpr int kScaleLoads = kBlocks ? (MT > 2 ? 2 : 1) : 0;
  constexpr int kStage = (MT + NT) * 2048 + (kBlocks ? 512 : 0);
  constexpr int kLoads = 2 * (MT + NT) + kScaleLoads;  // a wave and stage
  typedef typename AR::acc acc_t;
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
  const uint8_t* w = a.w + (int64_t)g * a.N * K;
  const float* ws = a.w_scale + (int64_t)g * a.N;  // row scales
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
    acc_t acc[MT][NT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[m][n] = acc_t{0, 0, 0, 0};
    // this lane's scales of block 0 (rows past the last one, which are not stored, have its)
    const float* sp[2] = {};
    int64_t sp_step[2] = {};
    if constexpr (kBlocks) {
      const bool row_lane = lane < (MT > 2 ? 64 : 32);
      const float* const rp = a.a_scale + (m0 + min(lane, rows - 1)) * a.a_row_step;
      const float* const wp = block_scales(a, GATED, g, c0, GATED && (lane & 1));
      sp[0] = row_lane ? rp : wp;
      sp_step[0] = row_lane ? a.a_block_step : 1;
      sp[1] = wp;
      sp_step[1] = 1;
    }
    // step s into stage d; a step past the share loads zeros, so that the count of loads stays
    auto load = [&](int s, int d) {
      const uint32_t k0 = (uint32_t)s * 128;
      uint8_t* st = mine + d * kStage;
      const bool in = s < s1;
      const bool inner = in && k0 + chunk < (uint32_t)K;
      uint32_t oa = inner ? a_off + k0 : kBeyond;
      // (what follows a channel may be NaN; times zero only whole numbers vanish)
      uint32_t ow = (AR::kScales == kRowScales ? in : inner) ? w_off + k0 : kBeyond;
      asm("" : "+v"(oa), "+v"(ow));
#pragma unroll
      for (int j = 0; j < 2 * NT; ++j) {
        const int n = j / 2;
        load16_to_lds(n < NO ? rw : ru, st + j * 1024, ow + (uint32_t)((j % 2) * 8 * NO + n % NO * 4) * K);
      }
#pragma unroll
      for (int j = 0; j < 2 * MT; ++j) load16_to_lds(ra, st + NT * 2048 + j * 1024, oa + (uint32_t)(j * 8) * K);
      if constexpr (kBlocks) {
        const int b = min(s, steps - 1);
#pragma unroll
        for (int j = 0; j < kScaleLoads; ++j)
          __builtin_amdgcn_global_load_lds((global_byte*)(sp[j] + b * sp_step[j]),
                                           (lds_byte*)(st + (MT + NT) * 2048 + j * 256), 4, 0, 0);
      }
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
      float sa[MT], sw[2];
      if constexpr (kBlocks) {
        const float* sc = (const float*)(mine + d * kStage + (MT + NT) * 2048);
#pragma unroll
        for (int m = 0; m < MT; ++m) sa[m] = sc[m * 16 + r];
        sw[0] = sc[MT > 2 ? 64 : 32];
        sw[1] = sc[(MT > 2 ? 64 : 32) + 1];
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the stage has been read: load over it
      load(s + S, d);
      if constexpr (kBlocks) {
        typename AR::frag wf[NT], af[MT];
#pragma unroll
        for (int n = 0; n < NT; ++n) wf[n] = AR::make(wv[0][n], wv[1][n]);
#pragma unroll
        for (int m = 0; m < MT; ++m) af[m] = AR::make(av[0][m], av[1][m]);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int n = 0; n < NT; ++n)
            acc[m][n] += AR::mfma128(wf[n], af[m]) * (sa[m] * sw[n / NO]);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n) acc[m][n] = AR::mfma(wv[h][n], av[h][m], acc[m][n]);
      }
      d = d + 1 == S ? 0 : d + 1;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();  // every wave has left its stages
    acc_t* const part = (acc_t*)split_lds;  // [KW][MT][NT][64]
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) part[((wave * MT + m) * NT + n) * kWave + lane] = acc[m][n];
    __syncthreads();
    // wave m of the row tiles joins and writes tile m
    for (int m = wave; m < MT; m += KW) {
      acc_t sum[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        sum[n] = part[(m * NT + n) * kWave + lane];
#pragma unroll
        for (int k = 1; k < KW; ++k) sum[n] += part[((k * MT + m) * NT + n) * kWave + lane];
      }
      const int row = m * 16 + r;
      if (row < rows) {
        const int col = c0 + q * 4 * NO;
        const float s = AR::kScales == kRowScales ? a.a_scale[m0 + row] : 1.0f;
        float y[NT * 4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            y[n * 4 + i] = (float)sum[n][i];
            if (AR::kScales == kRowScales) {
              const int c = min(col + n % NO * 4 + i, a.width - 1);
              y[n * 4 + i] = y[n * 4 + i] * s * ws[(n < NO ? 0 : a.width) + c];
            }
          }
        store_row<IO, GATED, AR::kScales == kNoScales, NT>(a, m0 + row, col, a.width, y);
      }
    }
    __syncthreads();
  }
}

// ---- tiles

// Starts of the groups' row tiles: pre[g] tiles come before group g, pre[G] in
// all.  Groups do not overlap, so there are at most M / BM + G tiles; ranges that
// say otherwise are cut there, which keeps every index in range.
template <int THREADS, int BM>
__device__ void tile_starts(const MatmulArgs& a, int* pre) {
  const int most = (int)(a.M / BM) + a.G;
  for (int g = threadIdx.x; g < a.G; g += THREADS) {
    int64_t lo, hi;
    group_rows(a, g, lo, hi);
    pre[g] = (int)((hi - lo + BM - 1) / BM);  // below 2^24
  }
  __syncthreads();
  if (threadIdx.x < kWave) {
    int carry = 0;
    for (int g0 = 0; g0 < a.G; g0 += kWave) {
      const int g = g0 + (int)threadIdx.x;
      const int v = g < a.G ? pre[g] : 0;
      int x = v;
      for (int o = 1; o < kWave; o <<= 1) {
        const int y = __shfl_up(x, o, 64);
        if ((int)threadIdx.x >= o) x += y;
      }
      if (g < a.G) pre[g] = min(carry + x - v, most);
      carry = min(carry + __shfl(x, kWave - 1, 64), most);
    }
    if (threadIdx.x == 0) pre[a.G] = carry;
  }
  __syncthreads();
}

struct Tile {
  int g;        // group
  int64_t m0;   // first row
  int rows;     // 1..BM
  int c0;       // first column of out
  int cols;     // 1..BN (BN / 2 gated)
};

// Tile t of all: the group is the last one whose tiles start at or before t
// (64 starts are compared at once, of G <= 4096 in two rounds).  Within a group
// strips of eight channel tiles, in each all row tiles, so that the tiles that
// run at once on an XCD share both operands.
template <int BM, int BC>
__device__ __forceinline__ Tile locate(const MatmulArgs& a, const int* pre, int n_tiles, int t) {
  Tile x;
  int g = 0;
  if (a.G > 1) {
    const int lane = lane_id();
    int base = 0, stride = (a.G + kWave - 1) / kWave;
    if (stride > 1) {
      const int i = lane * stride;
      base = (__popcll(ballot(i < a.G && pre[min(i, a.G)] * n_tiles <= t)) - 1) * stride;
    }
    // stride <= 64 groups are left
    const int i = base + lane;
    g = base + __popcll(ballot((stride == 1 || lane < stride) && i < a.G && pre[min(i, a.G)] * n_tiles <= t)) - 1;
    g = uniform(g);
  }
  const int first = uniform(pre[g]);
  const int m_tiles = uniform(pre[g + 1]) - first;
  const int in = t - first * n_tiles;
  const int strip = in / (8 * m_tiles);
  const int wide = min(8, n_tiles - strip * 8);
  const int rest = in - strip * 8 * m_tiles;
  int64_t lo, hi;
  group_rows(a, g, lo, hi);
  x.g = g;
  x.m0 = lo + (int64_t)(rest / wide) * BM;
  x.rows = (int)min((int64_t)BM, hi - x.m0);
  x.c0 = (strip * 8 + rest % wide) * BC;
  x.cols = min(BC, a.width - x.c0);
  return x;
}

}  // namespace ep
