// ep_int8_tile.hpp -- int8 product in tiles staged through LDS.
#pragma once

#include <type_traits>

#include "ep_product.hpp"

namespace ep {

// A workgroup of WM x WN waves computes tiles of BM rows x BN channels, one
// after the other, in steps of 64 bytes of the inner dimension.  Both operands
// have the inner dimension contiguous; their pieces go from memory straight to
// LDS (16 bytes a lane) into a ring of four stages.
//
// The steps of all tiles of a workgroup form one stream.  In step s the waves
//   - wait until their loads for step s + 1 have landed, and meet,
//   - start the loads of step s + 3 (into the stage that step s - 1 left),
//   - multiply step s, reading the fragments of its later row tiles and, near
//     its end, the first ones of step s + 1.
// So a load has two steps to arrive, no fragment is waited for behind a
// barrier, and the next tile's first steps arrive during a tile's epilogue.
//
// What bounds it: a step takes 1470 cycles (256 x 256; 990 at 128 x 256) against 1024
// (512) of products.  The direct loads alone come at ~24 bytes a clock and CU (a
// probe of them from the L2: 42 to 54), and more stages change nothing; and
// under int8 products the clock falls to 1.7-1.9 GHz of 2.4.  65536 rows of 64 groups,
// 7168 x 4096 gated: 1775 us, 2.17e15 operations a second; 16384 rows, 2048 x 7168:
// 341 us; 1003 x 2048 x 7168 (128 x 256): 22 us.
//
// LDS image of a stage: 64 bytes a row, its four 16-byte chunks in the order
// chunk ^ order(row / 4 % 4), so that the lanes that ds_read_b128 serves
// together (16 rows of one chunk, or 8 rows each of two) meet all banks; the
// order (row / 4) % 4 itself had a conflict on every second read.  Direct loads
// write lane l at l * 16, so the order is made by the addresses they read.
//
// Rows beyond the group's last one and channels beyond the last are beyond the
// buffer descriptor's size and arrive as zeros; so do chunks of A past the
// inner size (those of W may hold anything, their partners are zero).
//
// Row tiles of a wave: mt = 0..MT-1, in two halves of the tile, so that a tile
// with at most BM / 2 rows costs half the products (HALVES).
// GATED: of the 16 * NT channels of a wave the first half are gates and the
// second half the ups of the same columns.
//
// Lane l of an MFMA gets channels (l / 16) * 4 + 0..3 of its first operand, so
// the NO column tiles of a wave take their channels in turn, four at a time:
// row i of column tile n is column (i / 4) * 4 * NO + n * 4 + i % 4, and a lane
// ends with 4 * NO neighbouring columns of a row (16-byte stores, whole lines a
// wave).
template <int BM, int BN, int WM, int WN>
struct TileShape {
  static constexpr int kWaves = WM * WN;
  static constexpr int kThreads = kWaves * kWave;
  static constexpr int MT = BM / WM / 16, NT = BN / WN / 16;
  static constexpr int CW = BN / WN;  // channels of a wave
  static constexpr int kStep = 64;
  static constexpr int kStage = (BM + BN) * kStep;
  static constexpr int kStages = 4;
  static constexpr int kLoadsA = BM / 16 / kWaves, kLoadsW = BN / 16 / kWaves;  // direct loads a wave and step
  static constexpr int kLoads = kLoadsA + kLoadsW;
  static constexpr int kScales = BM + BN;  // floats of a tile
  static_assert(kLoadsA >= 1 && kLoadsW >= 1, "a load covers 16 rows");
  static size_t lds(int groups) { return kStages * ((size_t)kStage + kScales * 4) + ((size_t)groups + 1) * 4; }
};

__device__ __forceinline__ int chunk_order(int g) { return ((g ^ (g >> 1)) & 1) * 2 + (g >> 1); }  // 0, 2, 3, 1

// All but the newest N of this wave's loads have landed, and every wave is here.
template <int N>
__device__ __forceinline__ void step_sync() {
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(N) : "memory");
}

template <typename IO, bool GATED, int BM, int BN, int WM, int WN, bool HALVES>
__global__ __launch_bounds__(WM* WN* kWave) void matmul_tile_kernel(MatmulArgs a, int n_tiles) {
  typedef TileShape<BM, BN, WM, WN> S;
  constexpr int MT = S::MT, NT = S::NT, CW = S::CW;
  constexpr int BC = GATED ? BN / 2 : BN;  // columns of out
  constexpr int NO = GATED ? NT / 2 : NT;  // column tiles of out a wave
  constexpr int kPair = 2 * S::kStage;     // the stages of an even and the next odd step
  static_assert(MT % 4 == 0 && NT == 4, "fragment rings");
  extern __shared__ uint8_t tile_lds[];
  float* const scales = (float*)(tile_lds + S::kStages * S::kStage);  // [kStages][BM + BN]
  int* const pre = (int*)(scales + S::kStages * S::kScales);
  const int lane = lane_id();
  const int wave = uniform((int)threadIdx.x / kWave);
  const int wm = wave / WN, wn = wave % WN;
  const int q = lane >> 4, r = lane & 15;

  tile_starts<S::kThreads, BM>(a, pre);
  const int total = uniform(pre[a.G]) * n_tiles;
  const int K = a.K;
  const int steps = (K + 2 * S::kStep - 1) / (2 * S::kStep) * 2;  // even: stages and registers take turns
  // neighbouring tiles on one XCD (workgroups go round the 8 XCDs in turn)
  const int per = gridDim.x / 8;
  const int slot = gridDim.x % 8 == 0 ? ((int)blockIdx.x % 8) * per + (int)blockIdx.x / 8 : (int)blockIdx.x;
  if (slot >= total) return;

  // ---- producer: the stream of loads
  const uint32_t chunk = (uint32_t)((lane & 3) ^ chunk_order(lane >> 4)) * 16;
  const uint32_t lane_off = (uint32_t)(lane >> 2) * K + chunk;
  const uint32_t lane_off_w = (uint32_t)((lane >> 4) * 4 * NO + ((lane >> 2) & 3)) * K + chunk;
  int p_tile = slot, p_step = steps, p_ring = 0, p_stage = 0;
  __amdgpu_buffer_rsrc_t ra, rw, ru;
  auto next_tile = [&]() {  // descriptors of tile p_tile, and its scales on their way
    const bool any = p_tile < total;
    const Tile x = locate<BM, BC>(a, pre, n_tiles, any ? p_tile : slot);
    const uint8_t* w = a.w + (int64_t)x.g * a.N * K;
    ra = buffer_of(a.a + x.m0 * K, any ? (int64_t)x.rows * K : 0);
    rw = buffer_of(w + (int64_t)x.c0 * K, any ? (int64_t)x.cols * K : 0);
    if (GATED) ru = buffer_of(w + (int64_t)(x.c0 + a.width) * K, any ? (int64_t)x.cols * K : 0);
    const __amdgpu_buffer_rsrc_t rs = buffer_of(a.a_scale + x.m0, any ? x.rows * 4 : 0);
    const __amdgpu_buffer_rsrc_t rc = buffer_of(a.w_scale + (int64_t)x.g * a.N, any ? a.N * 4 : 0);
    float* dst = scales + p_ring * S::kScales;
    for (int i = wave; i < S::kScales / kWave; i += S::kWaves) {
      int e = i * kWave + lane;
      asm volatile("" : "+v"(e));
      if (i * kWave < BM) {
        load4_to_lds(rs, dst + i * kWave, (uint32_t)e * 4);
      } else {
        const int c = e - BM;  // gated: the columns' gates, then their ups
        const int col = c % BC;
        const int ch = x.c0 + col + (c >= BC ? a.width : 0);
        load4_to_lds(rc, dst + i * kWave, col < x.cols ? (uint32_t)ch * 4 : kBeyond);
      }
    }
    p_ring = (p_ring + 1) % S::kStages;
    p_tile += gridDim.x;
    p_step = 0;
  };
  // load i of this wave's kLoads for the next step of the stream
  auto load_one = [&](int i) {
    const uint32_t k0 = (uint32_t)p_step * S::kStep;
    uint32_t off = lane_off + k0;
    asm("" : "+v"(off));  // one register and an addition a load, rather than a register a load
    uint8_t* st = tile_lds + p_stage * S::kStage;
    if (i < S::kLoadsA) {
      const int row = (i * S::kWaves + wave) * 16;
      load16_to_lds(ra, st + row * S::kStep, k0 + chunk < (uint32_t)K ? off + (uint32_t)row * K : kBeyond);
    } else {
      // LDS row `row` + 0..15: column tile n of wave column v
      const int row = ((i - S::kLoadsA) * S::kWaves + wave) * 16;
      const int v = row / CW, n = row % CW / 16;
      uint32_t offw = lane_off_w + k0;
      asm("" : "+v"(offw));
      load16_to_lds(GATED && n >= NO ? ru : rw, st + (BM + row) * S::kStep,
                    offw + (uint32_t)(v * 16 * NO + n % NO * 4) * K);
    }
  };
  auto advance = [&]() {
    ++p_step;
    p_stage = (p_stage + 1) % S::kStages;
  };

  // ---- consumer
  const int frag = r * S::kStep + ((q ^ chunk_order(r >> 2)) * 16);
  const uint32_t a_lane = wm * (MT / 2) * 16 * S::kStep + frag;
  const uint32_t w_lane = BM * S::kStep + wn * CW * S::kStep + frag;
  uint32_t pair = 0;  // 0 or kPair: the current pair of stages
  i32x4 acc[MT][NT], av[4], wv[2][NT];
  auto read_a = [&](uint32_t at, int h, int m) {
    return *(const i32x4*)(tile_lds + at + h * S::kStage + (m < MT / 2 ? m : m - MT / 2 + BM / 32) * 16 * S::kStep);
  };
  auto read_w = [&](uint32_t at, int h, int n) {
    return *(const i32x4*)(tile_lds + at + h * S::kStage + n * 16 * S::kStep);
  };
  // One step; h: its place in the pair.
  auto step = [&](auto hc, auto mtn) {
    constexpr int h = decltype(hc)::value, MTN = decltype(mtn)::value;
    step_sync<S::kLoads>();
    if (p_step == steps) next_tile();
    const uint32_t next = h ? kPair - pair : pair;
    const uint32_t a_at = a_lane + pair, a_next = a_lane + next, w_next = w_lane + next;
#pragma unroll
    for (int u = 0; u < MTN; ++u) {
      constexpr int kW0 = MTN > 4 ? 2 : 0;  // the next step's channel fragments: units kW0..kW0 + NT - 1
      av[(u + 3) % 4] = u + 3 < MTN ? read_a(a_at, h, u + 3) : read_a(a_next, 1 - h, u + 3 - MTN);
      if (u >= kW0 && u < kW0 + NT) wv[1 - h][u - kW0] = read_w(w_next, 1 - h, u - kW0);
#pragma unroll
      for (int i = u; i < S::kLoads; i += MTN) load_one(i);
#pragma unroll
      for (int n = 0; n < NT; ++n)
        acc[u][n] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[h][n], av[u % 4], acc[u][n], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
    advance();
  };

  // the first three steps of the stream, and the first fragments
  for (int s = 0; s < 3; ++s) {
    if (p_step == steps) next_tile();
    for (int i = 0; i < S::kLoads; ++i) load_one(i);
    advance();
  }
  step_sync<2 * S::kLoads>();
#pragma unroll
  for (int n = 0; n < NT; ++n) wv[0][n] = read_w(w_lane, 0, n);
#pragma unroll
  for (int u = 0; u < 3; ++u) av[u] = read_a(a_lane, 0, u);

  int c_ring = 0;
  for (int t = slot; t < total; t += gridDim.x) {
    const Tile x = locate<BM, BC>(a, pre, n_tiles, t);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[m][n] = i32x4{0, 0, 0, 0};
    auto run = [&](auto mtn) {
      for (int s = 0; s < steps; s += 2) {
        step(std::integral_constant<int, 0>{}, mtn);
        step(std::integral_constant<int, 1>{}, mtn);
        pair = kPair - pair;
      }
    };
    if (!HALVES || x.rows > BM / 2)
      run(std::integral_constant<int, MT>{});
    else
      run(std::integral_constant<int, HALVES ? MT / 2 : MT>{});

    // epilogue: a lane holds columns wn * 16 * NO + q * 4 * NO + 0..4 * NO - 1 of
    // row r of every row tile
    const float* sa = scales + c_ring * S::kScales;
    c_ring = (c_ring + 1) % S::kStages;
    int er = r, eq = q;
    asm volatile("" : "+v"(er), "+v"(eq));  // what follows is not kept in registers over the steps
    const int col = wn * 16 * NO + eq * 4 * NO;
    float sw[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) sw[n][i] = sa[BM + (n < NO ? 0 : BC) + col + (n % NO) * 4 + i];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int row = (m < MT / 2 ? 0 : BM / 2) + wm * (MT / 2) * 16 + (m % (MT / 2)) * 16 + er;
      if (row >= x.rows) continue;
      const float s = sa[row];
      float y[NT * 4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) y[n * 4 + i] = (float)acc[m][n][i] * s * sw[n][i];
      store_row<IO, GATED, false, NT>(a, x.m0 + row, x.c0 + col, x.c0 + x.cols, y);
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load into LDS outlives the workgroup
}

}  // namespace ep
