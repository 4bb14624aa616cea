// ep_product_tile.hpp -- products of E4M3 rows with block scales and of 16-bit rows in
// tiles staged through LDS, in steps of 128 bytes.
#pragma once

#include <type_traits>

#include "ep_product.hpp"

namespace ep {

// A workgroup of WM x WN waves computes tiles of BM rows x BN channels, one after the
// other, in steps of 128 bytes of the inner dimension; the steps of all its tiles form one
// stream, as in ep_int8_tile.hpp.  With block scales a step is a block: one matrix
// instruction for each 16 x 16 of a wave's share, and what it gives is scaled and added to
// the fp32 sums by vector instructions while the next ones run.  16-bit values take two,
// which add to the sums themselves.
//
// Two stages of LDS (a step each).  A wave goes through its row tiles in order; before the
// last it has all fragments of the step in registers, waits for its own loads of the next
// step, and meets the others: then the next step may be read and this one's stage loaded
// over, two loads at once and the others over the first row tiles of the next step (all at
// once they hold up the products behind them: E4M3 7%, 16-bit 3%).  So there is one barrier
// a step, a load has at least three row tiles to arrive, and fragments are read two row
// tiles ahead, those of the weights behind their last use.
// Against steps of 64 bytes with four stages (ep_int8_tile.hpp) the loads ask for whole
// lines of 128 bytes, half as many requests, and barriers are half as many.  Measured:
// 16-bit, 65536 x 4096 x 4096 gated 1.64 to 1.69 ms (64-byte steps 1.85), 4096^3 102 us (115),
// 8192^3 815 to 945 us with the box and its clock; E4M3, 65536 x 4096 x 4096 gated 1.01 to 1.05 ms.
// What bounds it (8192^3): 16-bit matrix instructions run 66% of the cycles (the library's 86%),
// E4M3's 52%, beside vector instructions, two thirds of them the scaling, in 38%.  A SIMD's
// two waves could run both at once, but pass the same barrier and so the same phase.  By count a
// step of 256 x 256 reads 192 KiB of LDS and writes 64 KiB, at 128 bytes a clock 2048 cycles,
// which is what its matrix instructions take (128 of 16 cycles a SIMD, E4M3 64 of 32); how
// much of the rest is waiting for LDS was not measured.  The clock falls to 1.5 to 1.9 GHz.
//
// LDS image: 128 bytes a row, chunk ^ (row & 7).  Columns of a wave's channel tiles, rows
// past the group's and channels past the last as in ep_int8_tile.hpp.  With block scales
// a stage holds behind the rows their scales of the block, and the two of the weights: of
// the tile's two blocks of columns, or of its gates and its ups.
template <int BM, int BN, int WM, int WN, bool BLOCKS>
struct StepShape {
  static constexpr int kWaves = WM * WN;
  static constexpr int kThreads = kWaves * kWave;
  static constexpr int MT = BM / WM / 16, NT = BN / WN / 16;
  static constexpr int CW = BN / WN;
  static constexpr int kRowBytes = 128;
  static constexpr int kScaleAt = (BM + BN) * kRowBytes;
  static constexpr int kStage = kScaleAt + (BLOCKS ? kThreads * 4 : 0);
  static constexpr int kLoadsA = BM / 8 / kWaves, kLoadsW = BN / 8 / kWaves;  // direct loads a wave and step
  static constexpr int kLoads = kLoadsA + kLoadsW + (BLOCKS ? 1 : 0);         // the last of scales
  static constexpr int kFirst = 2;  // of them right behind the barrier
  static_assert(BM / kWave < kWaves, "a wave is left for the weights' scales");
  static size_t lds(int groups) { return 2 * (size_t)kStage + ((size_t)groups + 1) * 4; }
};

template <typename AR, typename IO, bool GATED, int BM, int BN, int WM, int WN, bool HALVES>
__global__ __launch_bounds__(WM* WN* kWave) void product_tile_kernel(MatmulArgs a, int n_tiles) {
  constexpr bool kBlocks = AR::kScales == kBlockScales;
  typedef StepShape<BM, BN, WM, WN, kBlocks> S;
  constexpr int MT = S::MT, NT = S::NT, CW = S::CW;
  constexpr int BC = GATED ? BN / 2 : BN;  // columns of out
  constexpr int NO = GATED ? NT / 2 : NT;  // column tiles of out a wave
  static_assert(MT % 4 == 0, "fragment registers take turns, also in half tiles");
  static_assert(BC <= 256 && 128 % (16 * NO) == 0, "a wave's columns lie in one block");
  extern __shared__ uint8_t tile_lds[];
  int* const pre = (int*)(tile_lds + 2 * S::kStage);
  const int lane = lane_id();
  const int wave = uniform((int)threadIdx.x / kWave);
  const int wm = wave / WN, wn = wave % WN;
  const int q = lane >> 4, r = lane & 15;

  tile_starts<S::kThreads, BM>(a, pre);
  const int total = uniform(pre[a.G]) * n_tiles;
  const int K = a.K;
  const int steps = (K + 127) / 128;
  const int per = gridDim.x / 8;
  const int slot = gridDim.x % 8 == 0 ? ((int)blockIdx.x % 8) * per + (int)blockIdx.x / 8 : (int)blockIdx.x;
  if (slot >= total) return;

  // ---- producer: the stream of loads
  const uint32_t chunk = (uint32_t)((lane & 7) ^ (lane >> 3)) * 16;
  const uint32_t lane_off = (uint32_t)(lane >> 3) * K + chunk;
  const uint32_t lane_off_w = (uint32_t)((lane >> 5) * 4 * NO + ((lane >> 3) & 3)) * K + chunk;
  // Where the loads of a tile come from.  (The one behind the last tile reads zeros.)
  struct Source {
    __amdgpu_buffer_rsrc_t a, w, u;
    const float* scale;  // this lane's, of the next step
    int64_t scale_step;
  };
  int p_tile = slot, p_step = 0;
  uint32_t p_stage = 0;
  auto next_source = [&]() {
    const bool any = p_tile < total;
    const Tile x = locate<BM, BC>(a, pre, n_tiles, any ? p_tile : slot);
    const uint8_t* w = a.w + (int64_t)x.g * a.N * K;
    Source n;
    n.a = buffer_of(a.a + x.m0 * K, any ? (int64_t)x.rows * K : 0);
    n.w = buffer_of(w + (int64_t)x.c0 * K, any ? (int64_t)x.cols * K : 0);
    n.u = GATED ? buffer_of(w + (int64_t)(x.c0 + a.width) * K, any ? (int64_t)x.cols * K : 0) : n.w;
    // (rows and columns past the tile's have the scale of its last)
    n.scale = nullptr;
    n.scale_step = 0;
    if (kBlocks && wave < BM / kWave) {
      n.scale = a.a_scale + (x.m0 + min(wave * kWave + lane, x.rows - 1)) * a.a_row_step;
      n.scale_step = a.a_block_step;
    } else if (kBlocks) {
      const int col = GATED ? x.c0 : min(x.c0 + (lane & 1) * 128, a.width - 1);
      n.scale = block_scales(a, GATED, x.g, col, GATED && (lane & 1));
      n.scale_step = 1;
    }
    p_tile += gridDim.x;
    return n;
  };
  Source src = next_source(), next_src = src;
  // load i of this wave's kLoads for the next step of the stream
  auto load_one = [&](int i) {
    const uint32_t k0 = (uint32_t)p_step * 128;
    uint8_t* st = tile_lds + p_stage;
    if (kBlocks && i == S::kLoads - 1) {
      __builtin_amdgcn_global_load_lds((global_byte*)src.scale, (lds_byte*)(st + S::kScaleAt + wave * kWave * 4), 4, 0, 0);
    } else if (i < S::kLoadsA) {
      const int row = (i * S::kWaves + wave) * 8;
      uint32_t off = lane_off + k0;
      asm("" : "+v"(off));  // one register and an addition a load, rather than a register a load
      load16_to_lds(src.a, st + row * S::kRowBytes, k0 + chunk < (uint32_t)K ? off + (uint32_t)row * K : kBeyond);
    } else {
      // LDS rows `row` + 0..7: half of column tile n of wave column v
      const int row = ((i - S::kLoadsA) * S::kWaves + wave) * 8;
      const int v = row / CW, n = row % CW / 16, half = row % 16 / 8;
      uint32_t off = lane_off_w + k0;
      asm("" : "+v"(off));
      off += (uint32_t)(v * 16 * NO + n % NO * 4 + half * 8 * NO) * K;
      load16_to_lds(GATED && n >= NO ? src.u : src.w, st + (BM + row) * S::kRowBytes, k0 + chunk < (uint32_t)K ? off : kBeyond);
    }
  };
  // The stream goes on by a step, in next_src after a tile's last.
  auto advance = [&]() {
    const bool last = p_step == steps - 1;
    src.a = last ? next_src.a : src.a;
    src.w = last ? next_src.w : src.w;
    if (GATED) src.u = last ? next_src.u : src.u;
    if (kBlocks) {
      src.scale = last ? next_src.scale : src.scale + src.scale_step;
      src.scale_step = last ? next_src.scale_step : src.scale_step;
    }
    p_step = last ? 0 : p_step + 1;
    p_stage ^= S::kStage;
  };

  // ---- consumer
  // the two halves of a step in an image row
  const uint32_t frag0 = r * S::kRowBytes + (q ^ (r & 7)) * 16, frag1 = frag0 ^ 64;
  const uint32_t a_at = wm * (MT / 2) * 16 * S::kRowBytes, w_at = (BM + wn * CW) * S::kRowBytes;
  const uint32_t sa_lane = S::kScaleAt + (wm * (MT / 2) * 16 + r) * 4;
  uint32_t cur = 0;  // the current stage
  f32x4 acc[MT][NT], p[NT];
  typename AR::frag av[2], wv[NT];
  float sa[2], sw[2], s_prev[2];
  auto row_of = [](int m) { return m < MT / 2 ? m * 16 : (m - MT / 2) * 16 + BM / 2; };
  auto read_a = [&](uint32_t stage, int slot_, int m) {
    const uint8_t* at = tile_lds + (stage + a_at) + row_of(m) * S::kRowBytes;
    av[slot_] = AR::make(*(const i32x4*)(at + frag0), *(const i32x4*)(at + frag1));
    if (kBlocks) sa[slot_] = *(const float*)(tile_lds + stage + sa_lane + row_of(m) * 4);
  };
  auto w_half = [&](uint32_t stage, int n, uint32_t frag) {
    return *(const i32x4*)(tile_lds + (stage + w_at) + n * 16 * S::kRowBytes + frag);
  };
  auto read_w = [&](uint32_t stage, int n) { wv[n] = AR::make(w_half(stage, n, frag0), w_half(stage, n, frag1)); };
  auto read_sw = [&](uint32_t stage) {
    const float* s = (const float*)(tile_lds + stage + S::kScaleAt) + BM;
    sw[0] = s[GATED ? 0 : wn * 16 * NO / 128];
    if (GATED) sw[1] = s[1];
  };
  // the products in p, of row tile m and column tile n, to the sums
  auto add = [&](int m, int n) {
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[m][n][i] = __builtin_fmaf(p[n][i], s_prev[n / NO], acc[m][n][i]);
  };
  // One step of MTN row tiles.
  auto step = [&](auto mtn) {
    constexpr int MTN = decltype(mtn)::value;
    constexpr int kLoading = MTN * 5 / 8;  // row tiles that share the loads
    constexpr int kEach = (S::kLoads - S::kFirst + kLoading - 1) / kLoading;
    const uint32_t next = cur ^ S::kStage;
    // (here, since a branch further down lets the sums' additions sink past it)
    if (p_step == steps - 1) next_src = next_source();
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
      if constexpr (kBlocks) {
        const float s0 = sa[u % 2] * sw[0], s1 = GATED ? sa[u % 2] * sw[1] : s0;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          add(u == 0 ? kLast : u - 1, n);
          p[n] = AR::mfma128(wv[n], av[u % 2]);
          if (u == kLast) read_w(next, n);
        }
        s_prev[0] = s0;
        s_prev[1] = s1;
        if (u == kLast) read_sw(next);
      } else {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          acc[u][n] = AR::mfma(wv[n].v[0], av[u % 2].v[0], acc[u][n]);
          if (u == kLast) wv[n].v[0] = w_half(next, n, frag0);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          acc[u][n] = AR::mfma(wv[n].v[1], av[u % 2].v[1], acc[u][n]);
          if (u == kLast) wv[n].v[1] = w_half(next, n, frag1);
        }
      }
      if (u + 2 < MTN) read_a(cur, u % 2, u + 2);
      if (u == kLast) read_a(next, 1, 1);
      __builtin_amdgcn_sched_barrier(0);
    }
    cur = next;
  };
  auto run = [&](auto mtn) {
    for (int s = 0; s < steps; ++s) step(mtn);
    if constexpr (kBlocks) {
#pragma unroll
      for (int n = 0; n < NT; ++n) add(decltype(mtn)::value - 1, n);
    }
  };

  // the stream's first step and the beginning of its second, and the first fragments
  for (int i = 0; i < S::kLoads; ++i) load_one(i);
  if (steps == 1) next_src = next_source();
  advance();
  for (int i = 0; i < S::kFirst; ++i) load_one(i);
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(S::kFirst) : "memory");
#pragma unroll
  for (int n = 0; n < NT; ++n) read_w(0, n);
  if (kBlocks) read_sw(0);
  read_a(0, 0, 0);
  read_a(0, 1, 1);

  for (int t = slot; t < total; t += gridDim.x) {
    const Tile x = locate<BM, BC>(a, pre, n_tiles, t);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[m][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (kBlocks) {
#pragma unroll
      for (int n = 0; n < NT; ++n) p[n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      s_prev[0] = s_prev[1] = 0.0f;
    }
    if (!HALVES || x.rows > BM / 2)
      run(std::integral_constant<int, MT>{});
    else
      run(std::integral_constant<int, HALVES ? MT / 2 : MT>{});

    int er = r, eq = q;
    asm volatile("" : "+v"(er), "+v"(eq));  // what follows is not kept in registers over the steps
    const int col = wn * 16 * NO + eq * 4 * NO;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int row = wm * (MT / 2) * 16 + row_of(m) + er;
      if (row >= x.rows) continue;
      float y[NT * 4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) y[n * 4 + i] = acc[m][n][i];
      store_row<IO, GATED, !kBlocks, NT>(a, x.m0 + row, x.c0 + col, x.c0 + x.cols, y);
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load into LDS outlives the workgroup
}

}  // namespace ep
