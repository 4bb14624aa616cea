// ep_half_grad.hpp -- gradients of the 16-bit product: of the rows and of the
// weights, in tiles staged through LDS; the gate's gradient.
#pragma once

#include "ep_product_tile.hpp"

namespace ep {

// y = a w^T has the gradients d w (of the rows; inner dimension: channels) and, for
// each group, d^T a (of its weights; inner dimension: the group's rows).  The inner
// dimension is not contiguous in w, and in neither operand of d^T a: their stages in
// LDS are images of 64 inner indexes by BM or BN values, read with ds_read_b64_tr_b16.
// For 16 lanes that instruction takes four rows of 16 values (lane i: 8 bytes of row
// i / 4, values 4 (i % 4)..) and gives lane i the four of column i, so two of them make
// a lane's operand of the matrix instruction.
//
// Stream of steps, two stages, one barrier a step, order of tiles and halves as in
// ep_product_tile.hpp, with one difference: a wave's column tiles are 16 neighbouring
// columns each, and v_permlane16_swap gives a lane eight neighbours of a row at the end.
// (65536 rows of 32 experts, 4096 x 4096: rows 1.9 ms, weights 2.0, 1.1e15 operations a second.)
//
// Image of a strided operand: index k has 512 (256) bytes, blocks of 32 bytes (16 values)
// in the order block ^ f(k), f(k) = k % 4 + 4 (k / 8 % 2): the eight k whose blocks 32
// lanes read together meet all banks.  Indexes past the end lie past the descriptor, which
// starts anew at each step, so offsets stay in 32 bits for any number of rows; columns
// past the last hold the next row's values and are not stored.
struct Strided {
  const uint8_t* at;  // the stream's next step
  int64_t left;       // indexes from there on
  int64_t stride;     // bytes between indexes
  int64_t tail;       // bytes of an index from the tile's first value on
  __device__ __forceinline__ void start(const uint8_t* p, int64_t n, int64_t stride_, int64_t tail_) {
    at = p;
    left = n;
    stride = stride_;
    tail = tail_;
  }
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t step() {
    const int64_t n = left < 64 ? left : 64;
    const __amdgpu_buffer_rsrc_t r = buffer_of(at, n > 0 ? (n - 1) * stride + tail : 0);
    at += 64 * stride;
    left -= 64;
    return r;
  }
};

__device__ __forceinline__ Strided pick(bool first, const Strided& x, const Strided& y) {
  return Strided{first ? x.at : y.at, first ? x.left : y.left, first ? x.stride : y.stride, first ? x.tail : y.tail};
}

// Where lane's 16 bytes of a load of 1 KiB come from, from the step's first index on:
// loads go round the waves, WIDTH values an index.
template <int WIDTH>
__device__ __forceinline__ uint32_t strided_source(int wave, int lane, uint32_t stride) {
  constexpr int kLanes = WIDTH / 8;  // of an index
  const int k = wave * (64 / kLanes) + lane / kLanes;
  const int f = (k & 3) | (k >> 3 & 1) << 2;
  const int piece = lane % kLanes;
  return (uint32_t)k * stride + (uint32_t)(((piece >> 1) ^ f) * 2 + (piece & 1)) * 16;
}

// The byte of the image that lane reads for block `block`: index q * 8 + i / 4, the
// second half of its operand four indexes on, the step's second half 32 indexes on.
template <int WIDTH>
__device__ __forceinline__ uint32_t strided_frag(int lane, int block) {
  const int q = lane >> 4, i = lane & 15;
  const int f = i >> 2 | (q & 1) << 2;
  return (uint32_t)(q * 8 + (i >> 2)) * (WIDTH * 2) + (uint32_t)(block ^ f) * 32 + (i & 3) * 8;
}

// (`__restrict__` gives the reads alias information; without any the compiler waits for all
// direct loads to LDS in flight before each of them: 4.44 against 2.1 ms for 65536 rows of 32 experts, 4096 x 4096.)
template <int WIDTH>
__device__ __forceinline__ i32x4 read_strided(const uint8_t* __restrict__ at) {
  typedef short i16x4 __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
  typedef int i32x2 __attribute__((ext_vector_type(2)));
  const i32x2 lo = __builtin_bit_cast(i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)at));
  const i32x2 hi = __builtin_bit_cast(i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(at + 4 * WIDTH * 2)));
  return i32x4{lo[0], lo[1], hi[0], hi[1]};
}

// Where tiles are few and the inner dimension long, each is computed by several workgroups,
// a slice of the inner dimension each, into fp32 results that join_slices_kernel adds in a
// fixed order.
//
// MatmulArgs here: a = d [M][N], K its row's bytes; w = the weights [G][N][width], or for
// the weights' gradient the rows a [M][width]; out = [M][width] or [G][N][width].
//
// Tile t of the weights' gradient: strips of eight column tiles, in each all row tiles.
template <int BM, int BN>
__device__ __forceinline__ Tile locate_weights(const MatmulArgs& a, int m_tiles, int n_tiles, int t) {
  Tile x;
  const int each = m_tiles * n_tiles;
  x.g = t / each;
  const int in = t - x.g * each;
  const int strip = in / (8 * m_tiles);
  const int wide = min(8, n_tiles - strip * 8);
  const int rest = in - strip * 8 * m_tiles;
  x.m0 = (int64_t)(rest / wide) * BM;
  x.rows = min(BM, a.N - (int)x.m0);
  x.c0 = (strip * 8 + rest % wide) * BN;
  x.cols = min(BN, a.width - x.c0);
  return x;
}

template <typename AR, typename IO, bool WEIGHTS, int BM, int BN, int WM, int WN, bool HALVES>
__global__ __launch_bounds__(WM* WN* kWave) void half_grad_kernel(MatmulArgs a, int n_tiles) {
  typedef StepShape<BM, BN, WM, WN, false> S;
  constexpr int MT = S::MT, NT = S::NT;
  constexpr int kImageA = BM * S::kRowBytes;
  static_assert(MT % 4 == 0 && NT == 4 && BN == 256 && (BM == 256 || BM == 128), "fragment registers and images");
  typedef typename AR::frag frag_t;
  extern __shared__ uint8_t tile_lds[];
  int* const pre = (int*)(tile_lds + 2 * S::kStage);
  const int lane = lane_id();
  const int wave = uniform((int)threadIdx.x / kWave);
  const int wm = wave / WN, wn = wave % WN;
  const int q = lane >> 4, r = lane & 15;

  const int m_tiles = (a.N + BM - 1) / BM;
  int each;  // tiles of a slice
  if constexpr (WEIGHTS) {
    each = a.G * m_tiles * n_tiles;
  } else {
    tile_starts<S::kThreads, BM>(a, pre);
    each = uniform(pre[a.G]) * n_tiles;
  }
  const int total = each * a.slices;
  const int K = a.K;
  const int per = gridDim.x / 8;
  const int slot = gridDim.x % 8 == 0 ? ((int)blockIdx.x % 8) * per + (int)blockIdx.x / 8 : (int)blockIdx.x;
  if (slot >= total) return;

  auto tile = [&](int t) {
    if constexpr (WEIGHTS)
      return locate_weights<BM, BN>(a, m_tiles, n_tiles, t % each);
    else
      return locate<BM, BN>(a, pre, n_tiles, t % each);
  };
  // Inner indexes [lo, hi) of tile t: the group's rows or the channels, or a slice of them.
  auto inner = [&](int t, const Tile& x, int64_t& lo, int64_t& hi) {
    lo = 0;
    hi = a.N;
    if constexpr (WEIGHTS) group_rows(a, x.g, lo, hi);
    if (a.slices > 1) {
      const int64_t len = ((hi - lo + a.slices - 1) / a.slices + 63) / 64 * 64;
      lo = min(hi, lo + t / each * len);
      hi = min(hi, lo + len);
    }
  };
  // steps of a tile (without indexes one of zeros)
  auto steps_of = [&](int64_t lo, int64_t hi) { return max(1, (int)((hi - lo + 63) / 64)); };

  // ---- producer: the stream of loads
  const uint32_t chunk = (uint32_t)((lane & 7) ^ (lane >> 3)) * 16;
  const uint32_t lane_off_a = WEIGHTS ? strided_source<BM>(wave, lane, (uint32_t)K) : (uint32_t)(lane >> 3) * K + chunk;
  const uint32_t lane_off_w = strided_source<BN>(wave, lane, (uint32_t)a.width * 2);
  // Where the loads of a tile come from.  (The one behind the last tile reads zeros.)
  struct Source {
    int steps;
    Strided a, w;                // strided operands (a: of the weights' gradient)
    __amdgpu_buffer_rsrc_t rows; // rows' gradient: d's rows, and the bytes of them that the tile needs
    uint32_t from, to;
  };
  int p_tile = slot, p_step = 0;
  uint32_t p_stage = 0;
  auto next_source = [&]() {
    const bool any = p_tile < total;
    const int t = any ? p_tile : slot;
    const Tile x = tile(t);
    const int64_t row = (int64_t)a.width * 2;
    int64_t lo, hi;
    inner(t, x, lo, hi);
    Source s;
    s.steps = steps_of(lo, hi);
    s.from = (uint32_t)lo * 2;
    s.to = (uint32_t)hi * 2;
    const int64_t n = any ? hi - lo : 0;
    if constexpr (WEIGHTS) {
      s.a.start(a.a + lo * K + x.m0 * 2, n, K, K - x.m0 * 2);
      s.w.start(a.w + lo * row + (int64_t)x.c0 * 2, n, row, row - (int64_t)x.c0 * 2);
      s.rows = buffer_of(a.a, 0);
    } else {
      s.a.start(a.a, 0, 0, 0);
      s.w.start(a.w + ((int64_t)x.g * a.N + lo) * row + (int64_t)x.c0 * 2, n, row, row - (int64_t)x.c0 * 2);
      s.rows = buffer_of(a.a + x.m0 * K, any ? (int64_t)x.rows * K : 0);
    }
    p_tile += gridDim.x;
    return s;
  };
  Source src = next_source(), next_src = src;
  __amdgpu_buffer_rsrc_t ra, rw;  // of the stream's next step
  auto describe = [&]() {
    ra = WEIGHTS ? src.a.step() : src.rows;
    rw = src.w.step();
  };
  describe();
  // load i of this wave's kLoads for the next step of the stream
  auto load_one = [&](int i) {
    uint8_t* st = tile_lds + p_stage;
    if (i < S::kLoadsA) {
      const int at = (i * S::kWaves + wave) * 1024;
      uint32_t off = lane_off_a;
      asm("" : "+v"(off));  // one register and an addition a load, rather than a register a load
      if constexpr (WEIGHTS) {
        // 1 KiB is 512 / BM indexes
        load16_to_lds(ra, st + at, off + (uint32_t)(i * S::kWaves * (512 / BM)) * K);
      } else {
        const uint32_t k0 = src.from + (uint32_t)p_step * S::kRowBytes;
        off += k0 + (uint32_t)((i * S::kWaves + wave) * 8) * K;
        load16_to_lds(ra, st + at, k0 + chunk < src.to ? off : kBeyond);
      }
    } else {
      const int j = i - S::kLoadsA;
      uint32_t off = lane_off_w;
      asm("" : "+v"(off));
      load16_to_lds(rw, st + kImageA + (j * S::kWaves + wave) * 1024,
                    off + (uint32_t)(j * S::kWaves * (512 / BN) * 2) * a.width);
    }
  };
  // The stream goes on by a step, in next_src after a tile's last.
  auto advance = [&]() {
    const bool last = p_step == src.steps - 1;
    if (WEIGHTS) {
      src.a = pick(last, next_src.a, src.a);
    } else {
      src.rows = last ? next_src.rows : src.rows;
      src.from = last ? next_src.from : src.from;
      src.to = last ? next_src.to : src.to;
    }
    src.w = pick(last, next_src.w, src.w);
    src.steps = last ? next_src.steps : src.steps;
    p_step = last ? 0 : p_step + 1;
    p_stage ^= S::kStage;
    describe();
  };

  // ---- consumer
  auto row_of = [](int m) { return m < MT / 2 ? m * 16 : (m - MT / 2) * 16 + BM / 2; };  // row tile m of wave row 0
  const uint32_t frag0 = r * S::kRowBytes + (q ^ (r & 7)) * 16, frag1 = frag0 ^ 64;  // of the two halves of a step
  uint32_t a_at[4], w_at[NT];
#pragma unroll
  for (int m = 0; m < 4; ++m)
    a_at[m] = WEIGHTS ? strided_frag<BM>(lane, (wm * (MT / 2) * 16 + row_of(m)) / 16)
                      : (uint32_t)((wm * (MT / 2) * 16 + row_of(m)) * S::kRowBytes);
#pragma unroll
  for (int n = 0; n < NT; ++n) w_at[n] = kImageA + strided_frag<BN>(lane, wn * NT + n);
  uint32_t cur = 0;  // the current stage
  f32x4 acc[MT][NT];
  frag_t av[2], wv[NT];
  auto read_a = [&](uint32_t stage, int slot_, int m) {
    // (row tiles 4..7 of 256 rows: eight blocks, or 128 rows, on)
    const uint8_t* at = tile_lds + stage + a_at[m % 4] + (m / 4) * (WEIGHTS ? 8 * 32 : 128 * S::kRowBytes);
    if constexpr (WEIGHTS)
      av[slot_] = AR::make(read_strided<BM>(at), read_strided<BM>(at + 32 * BM * 2));
    else
      av[slot_] = AR::make(*(const i32x4*)(at + frag0), *(const i32x4*)(at + frag1));
  };
  auto w_half = [&](uint32_t stage, int n, int h) {
    return read_strided<BN>(tile_lds + stage + w_at[n] + h * 32 * BN * 2);
  };
  // One step of MTN row tiles.
  auto step = [&](auto mtn) {
    constexpr int MTN = decltype(mtn)::value;
    constexpr int kLoading = MTN * 5 / 8;  // row tiles that share the loads
    constexpr int kEach = (S::kLoads - S::kFirst + kLoading - 1) / kLoading;
    const uint32_t next = cur ^ S::kStage;
    if (p_step == src.steps - 1) next_src = next_source();
#pragma unroll
    for (int u = 0; u < MTN; ++u) {
      constexpr int kLast = MTN - 1;
      if (u == kLast) {
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        read_a(next, 0, 0);
#pragma unroll
        for (int i = 0; i < S::kFirst; ++i) load_one(i);
      }
      // the other loads of the step that the last row tile of the step before began
#pragma unroll
      for (int i = S::kFirst + u * kEach; i < min(S::kFirst + (u + 1) * kEach, S::kLoads); ++i) load_one(i);
      if (u == kLoading - 1) advance();
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          acc[u][n] = AR::mfma(wv[n].v[h], av[u % 2].v[h], acc[u][n]);
          if (u == kLast) wv[n].v[h] = w_half(next, n, h);
        }
      if (u + 2 < MTN) read_a(cur, u % 2, u + 2);
      if (u == kLast) read_a(next, 1, 1);
      __builtin_amdgcn_sched_barrier(0);
    }
    cur = next;
  };

  // the stream's first step and the beginning of its second, and the first fragments
  for (int i = 0; i < S::kLoads; ++i) load_one(i);
  if (src.steps == 1) next_src = next_source();
  advance();
  for (int i = 0; i < S::kFirst; ++i) load_one(i);
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(S::kFirst) : "memory");
#pragma unroll
  for (int n = 0; n < NT; ++n) wv[n] = AR::make(w_half(0, n, 0), w_half(0, n, 1));
  read_a(0, 0, 0);
  read_a(0, 1, 1);

  for (int t = slot; t < total; t += gridDim.x) {
    const Tile x = tile(t);
    int64_t lo, hi;
    inner(t, x, lo, hi);
    const int steps = steps_of(lo, hi);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[m][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    auto run = [&](auto mtn) {
      for (int s = 0; s < steps; ++s) step(mtn);
    };
    if (!HALVES || x.rows > BM / 2)
      run(std::integral_constant<int, MT>{});
    else
      run(std::integral_constant<int, HALVES ? MT / 2 : MT>{});

    // epilogue: lane (q, r) has columns 4 q.. of row r of each 16 x 16; of two column
    // tiles odd q's of the first and even q's of the second trade places
    int er = r, eq = q;
    asm volatile("" : "+v"(er), "+v"(eq));  // what follows is not kept in registers over the steps
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int row = wm * (MT / 2) * 16 + row_of(m) + er;
      const int64_t first = WEIGHTS ? ((int64_t)(t / each) * a.G + x.g) * a.N : (int64_t)(t / each) * a.M;
      const int64_t at = (first + x.m0 + row) * a.width;
#pragma unroll
      for (int n = 0; n < NT; n += 2) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(acc[m][n][i]), __float_as_uint(acc[m][n + 1][i]),
                                                          false, false);
          v[i] = __uint_as_float(s[0]);
          v[4 + i] = __uint_as_float(s[1]);
        }
        const int col = x.c0 + wn * S::CW + (n + (eq & 1)) * 16 + (eq >> 1) * 8;
        if (row < x.rows) store_cols<IO, 8>(a.out, at + col, col, x.c0 + x.cols, v);
      }
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load into LDS outlives the workgroup
}

// The sum of the slices' results (parts: [slices] of the whole) for the rows of each group;
// the weights' gradient is one group of all its rows.  width is a multiple of 8.
template <typename IO>
__global__ __launch_bounds__(256) void join_slices_kernel(MatmulArgs a, const float* __restrict__ parts) {
  const int col = ((int)blockIdx.x * 64 + (int)threadIdx.x % 64) * 8;
  if (col >= a.width) return;
  int64_t lo, hi;
  group_rows(a, blockIdx.z, lo, hi);
  for (int64_t row = lo + blockIdx.y * 4 + threadIdx.x / 64; row < hi; row += (int64_t)gridDim.y * 4) {
    const int64_t at = row * a.width + col;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.0f;
    for (int k = 0; k < a.slices; ++k) {
      const float* p = parts + (int64_t)k * a.M * a.width + at;
      float f[8];
      F32::unpack(*(const F32::piece*)p, f);
      F32::unpack(*(const F32::piece*)(p + 4), f + 4);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += f[j];
    }
    IO::store8(a.out, at, v);
  }
}

// Gradient of the gate: with out = silu(g) u,
//   dg = grad u s (1 + g (1 - s)),  du = grad g s,  s = 1 / (1 + exp(-g)).
// Rounded to the rows' type, as the products' operands have to be; their sums are fp32.  s
// comes from the hardware's exp2 and reciprocal, as in silu: a step of fp32 each, and less
// than 2^-17 of s from the rounded exponent, far below that rounding.  Scaled by 2^-16, the
// denominator stays in fp32 down to gates of -98; an s below 2^-142 is 0.
// The small factors are multiplied first, and by half, since s (1 + g (1 - s)) reaches 1.1: a
// product leaves fp32 only if the gradient does.  g and u that were rounded to an infinity
// count as fp32's largest, so that a shut gate, or a grad of 0, gives 0 and not NaN.
// Bound by memory: 65536 x 2048 bf16 231 to 238 us, 5.7 to 5.8 TB/s.
template <typename IO>
__global__ __launch_bounds__(256) void gate_backward_kernel(const void* __restrict__ pre, const void* __restrict__ grad,
                                                            int64_t pieces, int width, void* __restrict__ out) {
  typedef typename IO::type T;
  const int per = width / 8;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < pieces; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / per;
    const int64_t at = row * 2 * width + (i - row * per) * 8;
    float g[8], u[8], d[8], dg[8], du[8];
    IO::unpack(__builtin_nontemporal_load((const typename IO::piece*)((const T*)pre + at)), g);
    IO::unpack(__builtin_nontemporal_load((const typename IO::piece*)((const T*)pre + at + width)), u);
    IO::unpack(__builtin_nontemporal_load((const typename IO::piece*)((const T*)grad + i * 8)), d);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (__builtin_isinf(g[j])) g[j] = __builtin_copysignf(0x1.fffffep127f, g[j]);
      if (__builtin_isinf(u[j])) u[j] = __builtin_copysignf(0x1.fffffep127f, u[j]);
      const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(g[j], -1.44269504f, -16.0f));
      const float s = __builtin_amdgcn_rcpf(0x1p-16f + e) * 0x1p-16f;
      du[j] = d[j] * (g[j] * s);
      dg[j] = 2.0f * (d[j] * (u[j] * (0.5f * (s * (1.0f + g[j] * (1.0f - s))))));
    }
    IO::store_piece((T*)out + at, dg);
    IO::store_piece((T*)out + at + width, du);
  }
}

}  // namespace ep
