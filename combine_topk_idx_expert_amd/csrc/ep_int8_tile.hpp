// ep_int8_tile.hpp -- int8 product in tiles staged through LDS.
#pragma once

#include <type_traits>

#include "ep_int8.hpp"

namespace ep {

// A workgroup computes BM rows x BN channels at a time, WM x WN waves, over
// steps of 128 bytes of the inner dimension.  Both operands have the inner
// dimension contiguous; their tiles go from memory straight to LDS (16 bytes a
// lane, two buffers: step t + 1 is on its way while step t is multiplied).
//
// LDS image: 128 bytes a row, its eight 16-byte chunks in the order
// chunk ^ (row & 7), so that the 16 lanes that read one chunk of 16 rows for
// v_mfma_i32_16x16x64_i8 meet all banks.  The direct loads write lane l of a
// wave at l * 16, so the order is made by the addresses they read.
//
// Rows beyond the group's last one and channels beyond the last are beyond the
// buffer descriptor's size and arrive as zeros; so do chunks of A past the
// inner size (those of W may hold anything, their partners are zero).
//
// Rows of a wave: 16-row tiles mt = 0..MT-1 in two halves of the tile, so that
// a tile with at most BM / 2 rows costs half the products.
// GATED: of the 16 * NT channels of a wave the first half are gates and the
// second half the ups of the same columns.
template <int BM, int BN, int WM, int WN>
struct TileShape {
  static constexpr int kThreads = WM * WN * kWave;
  static constexpr int kWaves = WM * WN;
  static constexpr int MT = BM / WM / 16, NT = BN / WN / 16;
  static constexpr int kStep = 128;
  static constexpr int kStage = (BM + BN) * kStep;
  static constexpr int kLoadsA = BM / 8 / kWaves, kLoadsW = BN / 8 / kWaves;  // direct loads a wave and step
  static size_t lds(int groups) { return 2 * (size_t)kStage + (BM + BN) * 4 + ((size_t)groups + 1) * 4; }
};

typedef __attribute__((address_space(3))) uint8_t lds_byte;

__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t r, uint8_t* dst, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_byte*)dst, 16, (int)off, 0, 0, 0);
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00020000);
}

// Every wave's direct loads so far have landed, and every wave is here.
__device__ __forceinline__ void step_sync() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Starts of the groups' row tiles: pre[g] tiles come before group g, pre[G] in all.
template <int THREADS, int BM>
__device__ void tile_starts(const MatmulArgs& a, int* pre) {
  for (int g = threadIdx.x; g < a.G; g += THREADS) {
    int64_t lo, hi;
    group_rows(a, g, lo, hi);
    pre[g] = (int)((hi - lo + BM - 1) / BM);
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
      if (g < a.G) pre[g] = carry + x - v;
      carry += __shfl(x, kWave - 1, 64);
    }
    if (threadIdx.x == 0) pre[a.G] = carry;
  }
  __syncthreads();
}

// Products of one step for MTN row tiles by NT channel tiles, as 2 * MTN units
// (half of the step, row tile) of NT products.  A unit's row fragment is read
// kAhead units before it is used and the channel fragments of the second half
// during the first one; sched_barrier keeps the compiler from moving the reads
// back to their uses.
template <int MTN, int MT, int NT>
__device__ __forceinline__ void tile_step(const uint8_t* __restrict__ la, const uint8_t* __restrict__ lw, int sw0,
                                          int sw1, int half_rows, i32x4 (&acc)[MT][NT]) {
  constexpr int kAhead = 3;
  constexpr int kUnits = 2 * MTN;
  i32x4 wv[2][NT], av[kAhead + 1];
  auto read_a = [&](int u) {
    const int m = u % MTN;
    return *(const i32x4*)(la + (m < MT / 2 ? m * 2048 : half_rows * 128 + (m - MT / 2) * 2048) + (u / MTN ? sw1 : sw0));
  };
#pragma unroll
  for (int n = 0; n < NT; ++n) wv[0][n] = *(const i32x4*)(lw + n * 2048 + sw0);
#pragma unroll
  for (int u = 0; u < kAhead; ++u) av[u] = read_a(u);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    if (u + kAhead < kUnits) av[(u + kAhead) % (kAhead + 1)] = read_a(u + kAhead);
    if (u < NT && MTN >= NT) wv[1][u] = *(const i32x4*)(lw + u * 2048 + sw1);
    const int m = u % MTN;
#pragma unroll
    for (int n = 0; n < NT; ++n)
      acc[m][n] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[u / MTN][n], av[u % (kAhead + 1)], acc[m][n], 0, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
  }
}

template <typename IO, bool GATED, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM* WN* kWave) void matmul_tile_kernel(MatmulArgs a, int n_tiles) {
  typedef TileShape<BM, BN, WM, WN> S;
  constexpr int MT = S::MT, NT = S::NT;
  constexpr int BC = GATED ? BN / 2 : BN;  // columns of out
  extern __shared__ uint8_t tile_lds[];
  uint8_t* const stage0 = tile_lds;
  float* const sa = (float*)(tile_lds + 2 * S::kStage);
  float* const sw = sa + BM;
  int* const pre = (int*)(sw + BN);
  const int lane = lane_id();
  const int wave = uniform((int)threadIdx.x / kWave);
  const int wm = wave / WN, wn = wave % WN;
  const int q = lane >> 4, r = lane & 15;

  tile_starts<S::kThreads, BM>(a, pre);
  const int total = uniform(pre[a.G]) * n_tiles;
  const int K = a.K;
  const int steps = (K + S::kStep - 1) / S::kStep;
  // neighbouring tiles on one XCD (workgroups go round the 8 XCDs in turn)
  const int per = gridDim.x / 8;
  const int slot = gridDim.x % 8 == 0 ? ((int)blockIdx.x % 8) * per + (int)blockIdx.x / 8 : (int)blockIdx.x;

  for (int t = slot; t < total; t += gridDim.x) {
    // group: the last one whose tiles start at or before t
    int g = 0;
    for (int lo = 0, hi = a.G; hi - lo > 1;) {
      const int mid = (lo + hi) / 2;
      if (uniform(pre[mid]) * n_tiles <= t) lo = mid; else hi = mid;
      g = lo;
    }
    const int m_tiles = uniform(pre[g + 1]) - uniform(pre[g]);
    const int in = t - uniform(pre[g]) * n_tiles;
    // strips of eight channel tiles, in each all row tiles, so that what runs
    // at once on an XCD shares both operands
    const int strip = in / (8 * m_tiles);
    const int wide = min(8, n_tiles - strip * 8);
    const int rest = in - strip * 8 * m_tiles;
    const int mi = rest / wide, ni = strip * 8 + rest % wide;
    int64_t lo, hi;
    group_rows(a, g, lo, hi);
    const int64_t m0 = lo + (int64_t)mi * BM;
    const int rows = (int)min((int64_t)BM, hi - m0);
    const int c0 = ni * BC;
    const int cols = min(BC, a.width - c0);
    const int8_t* w = a.w + (int64_t)g * a.N * K;
    const __amdgpu_buffer_rsrc_t ra = buffer_of(a.a + m0 * K, (int64_t)rows * K);
    const __amdgpu_buffer_rsrc_t rw = buffer_of(w + (int64_t)c0 * K, (int64_t)cols * K);
    const __amdgpu_buffer_rsrc_t ru = buffer_of(w + (int64_t)(c0 + (GATED ? a.width : 0)) * K, (int64_t)cols * K);

    const uint32_t chunk = (uint32_t)((lane & 7) ^ (lane >> 3)) * 16;
    const uint32_t lane_off = (uint32_t)(lane >> 3) * K + chunk;
    auto load_step = [&](int step, uint8_t* st) {
      const uint32_t k0 = (uint32_t)step * S::kStep;
      uint32_t off = lane_off + k0;
      asm("" : "+v"(off));  // one register and an addition a load, rather than a register a load
      const uint32_t offa = k0 + chunk < (uint32_t)K ? off : 0x80000000u;
#pragma unroll
      for (int i = 0; i < S::kLoadsA; ++i) {
        const int row = (i * S::kWaves + wave) * 8;
        if (row < rows) load_to_lds(ra, st + row * S::kStep, offa + (uint32_t)row * K);
      }
#pragma unroll
      for (int i = 0; i < S::kLoadsW; ++i) {
        const int row = (i * S::kWaves + wave) * 8;
        constexpr int CW = BN / WN;  // channels of a wave
        if (!GATED)
          load_to_lds(rw, st + (BM + row) * S::kStep, off + (uint32_t)row * K);
        else
          load_to_lds((row % CW) < CW / 2 ? rw : ru, st + (BM + row) * S::kStep,
                      off + (uint32_t)((row / CW) * (CW / 2) + row % (CW / 2)) * K);
      }
    };

    __syncthreads();  // the previous tile's readers of the buffers and the scales are done
    load_step(0, stage0);
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));  // nothing that follows is kept in registers over the tiles
    for (int i = tid; i < BM + BN; i += S::kThreads) {
      if (i < BM) {
        sa[i] = i < rows ? a.a_scale[m0 + i] : 0.0f;
      } else {
        const int c = i - BM;
        constexpr int CW = BN / WN;
        const int col = GATED ? (c / CW) * (CW / 2) + c % (CW / 2) : c;
        const bool up = GATED && (c % CW) >= CW / 2;
        sw[c] = col < cols ? a.w_scale[(int64_t)g * a.N + (up ? a.width : 0) + c0 + col] : 0.0f;
      }
    }
    i32x4 acc[MT][NT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[m][n] = i32x4{0, 0, 0, 0};

    const int sw0 = r * 128 + ((q ^ (lane & 7)) * 16);
    const int sw1 = r * 128 + (((4 + q) ^ (lane & 7)) * 16);
    const int a_base = wm * (MT / 2) * 2048;
    const int w_base = BM * S::kStep + wn * NT * 2048;
    auto run = [&](auto mtn) {
      for (int s = 0; s < steps; ++s) {
        step_sync();  // step s has landed for every wave; the other buffer is free
        const uint8_t* cur = stage0 + (s & 1) * S::kStage;
        if (s + 1 < steps) load_step(s + 1, stage0 + ((s + 1) & 1) * S::kStage);
        tile_step<decltype(mtn)::value, MT, NT>(cur + a_base, cur + w_base, sw0, sw1, BM / 2, acc);
      }
    };
    if (rows > BM / 2)
      run(std::integral_constant<int, MT>{});
    else
      run(std::integral_constant<int, MT / 2>{});

    // epilogue: lane holds channels q * 4 + 0..3 of row r of every tile
    constexpr int NO = GATED ? NT / 2 : NT;
    int er = r, eq = q;
    asm volatile("" : "+v"(er), "+v"(eq));
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int row = (m < MT / 2 ? 0 : BM / 2) + wm * (MT / 2) * 16 + (m % (MT / 2)) * 16 + er;
      if (row >= rows) continue;
      const float s = sa[row];
#pragma unroll
      for (int n = 0; n < NO; ++n) {
        const int col = wn * (NO * 16) + n * 16 + eq * 4;
        const int64_t at = (m0 + row) * a.width + c0 + col;
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] = (float)acc[m][n][i] * s * sw[wn * (NT * 16) + n * 16 + eq * 4 + i];
          if (GATED) v[i] = silu(v[i]) * ((float)acc[m][n + NT / 2][i] * s * sw[wn * (NT * 16) + (n + NT / 2) * 16 + eq * 4 + i]);
        }
        if (col + 4 <= cols && a.width % 4 == 0) {
          IO::store4(a.out, at, v);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (col + i < cols) IO::store(a.out, at + i, v[i]);
        }
      }
    }
  }
}

}  // namespace ep
