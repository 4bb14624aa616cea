// ep_norm.hip -- host side of the norm, its gradient and the E4M3 quantising of
// rows: argument checks and launch configuration.
#include <algorithm>

#include "ep_host.hpp"
#include "ep_norm.hpp"

using namespace ep;

namespace {

ep_status validate_rows(int32_t type, int64_t num_rows, int32_t num_cols, int32_t most) {
  if (!known_type(type)) return fail(EP_ERR_SHAPE, "unknown element type %d", type);
  if (num_rows < 0 || num_cols < 1) return fail(EP_ERR_SHAPE, "bad sizes: %lld rows of %d", (long long)num_rows, num_cols);
  if (num_rows > EP_MAX_QUANT_ROWS || num_cols > most)
    return fail(EP_ERR_OVERFLOW, "%lld rows of %d: at most %d rows of %d", (long long)num_rows, num_cols,
                EP_MAX_QUANT_ROWS, most);
  return EP_OK;
}

ep_status validate_stride(const char* name, int64_t stride, int32_t num_cols) {
  if (stride < num_cols) return fail(EP_ERR_SHAPE, "%s stride %lld below num_cols %d", name, (long long)stride, num_cols);
  if (stride > (int64_t)1 << 40) return fail(EP_ERR_OVERFLOW, "%s stride %lld too large", name, (long long)stride);
  return EP_OK;
}

ep_status validate_norm(int32_t type, int64_t num_rows, int32_t num_cols, int32_t weight_type, float eps) {
  const ep_status st = validate_rows(type, num_rows, num_cols, EP_MAX_NORM_COLS);
  if (st != EP_OK) return st;
  if (weight_type != type && weight_type != EP_TYPE_F32)
    return fail(EP_ERR_SHAPE, "the weight's type %d must be the rows' or fp32", weight_type);
  if (!(eps > 0.0f && eps - eps == 0.0f)) return fail(EP_ERR_SHAPE, "eps must be positive and finite");
  return EP_OK;
}

template <typename IO, int L, int NC>
ep_status launch_norm(const NormArgs& a, hipStream_t s) {
  constexpr int kRows = L <= kWave ? 256 / L : 1;
  norm_kernel<IO, L, NC><<<(unsigned)((a.N + kRows - 1) / kRows), L <= kWave ? 256 : L, 0, s>>>(a);
  EP_LAUNCHED("norm_kernel");
  return EP_OK;
}

// Lanes of a row: 16, 32 or 64 (no barrier) where they hold it in one piece each, 64 with two
// pieces where there are rows for all CUs; else four waves, and sixteen for the longest.
// (32768 rows of 4096 bf16: four waves of two pieces 201 us, a wave of eight 475.)  Rows for
// less than all CUs take sixteen waves of one piece, for the latency.
template <typename IO>
ep_status launch_norm(const NormArgs& a, hipStream_t s) {
  constexpr int V = 16 / sizeof(typename IO::type);
  const int pieces = (a.H + V - 1) / V;
  if (pieces <= 16) return launch_norm<IO, 16, 1>(a, s);
  if (pieces <= 32) return launch_norm<IO, 32, 1>(a, s);
  if (pieces <= 64) return launch_norm<IO, 64, 1>(a, s);
  if (pieces <= 2 * 64 && a.N >= 4 * kCUs) return launch_norm<IO, 64, 2>(a, s);
  if (a.N <= kCUs && pieces > 256 && pieces <= 1024) return launch_norm<IO, 1024, 1>(a, s);
  if (pieces <= 128) return launch_norm<IO, 128, 1>(a, s);
  if (pieces <= 256) return launch_norm<IO, 256, 1>(a, s);
  if (pieces <= 2 * 256) return launch_norm<IO, 256, 2>(a, s);
  if (pieces <= 4 * 256) return launch_norm<IO, 256, 4>(a, s);
  if (pieces <= 2 * 1024) return launch_norm<IO, 1024, 2>(a, s);
  if (pieces <= 4 * 1024) return launch_norm<IO, 1024, 4>(a, s);
  if constexpr (V == 4) return launch_norm<IO, 1024, 8>(a, s);
  return fail(EP_ERR_SHAPE, "rows too long");  // not reached: validate_rows bounds them
}

// The gradient's teams of lanes, pieces of a lane, and workgroups.
struct NormTeams {
  int lanes, nc, groups;
};

// Every workgroup writes a row of fp32 sums, so there are no more than the card can use, and
// for few rows one for every four.  (262144 x 4096 bf16: 256 lanes of two pieces, three
// workgroups a CU 1610 us, four without the next row ahead 1690; 512 lanes of one 1840.
// 65536 x 2048: three 177 us, five 201.)
NormTeams norm_teams(int32_t type, int64_t N, int32_t H) {
  const int v = 16 / (int)type_bytes(type);
  const int pieces = (H + v - 1) / v;
  NormTeams t{1024, 1, 0};
  if (pieces <= 16) t.lanes = 16;
  else if (pieces <= 32) t.lanes = 32;
  else if (pieces <= 64) t.lanes = 64;
  else if (pieces <= 128) t.lanes = 128;
  else if (pieces <= 256) t.lanes = 256;
  else if (pieces <= 512) t.lanes = 256, t.nc = 2;
  else while (t.nc * 1024 < pieces) t.nc *= 2;
  const int64_t full = kCUs * (t.lanes == 1024 ? 1 : t.lanes == 256 ? 3 : t.lanes == 128 ? 10 : 5);
  const int64_t rows = t.lanes <= kWave ? 256 / t.lanes : 1;  // at once in a workgroup
  const int64_t all = (N + rows - 1) / rows;
  t.groups = (int)std::min(full, std::max<int64_t>(std::min<int64_t>(all, kCUs), all / 4));
  return t;
}

template <typename IO, int L, int NC>
ep_status launch_norm_backward(const NormBwdArgs& a, hipStream_t s) {
  norm_backward_kernel<IO, L, NC><<<a.groups, L <= kWave ? 256 : L, 0, s>>>(a);
  EP_LAUNCHED("norm_backward_kernel");
  return EP_OK;
}

template <typename IO>
ep_status launch_norm_backward(const NormBwdArgs& a, const NormTeams& t, hipStream_t s) {
  if (t.lanes == 16) return launch_norm_backward<IO, 16, 1>(a, s);
  if (t.lanes == 32) return launch_norm_backward<IO, 32, 1>(a, s);
  if (t.lanes == 64) return launch_norm_backward<IO, 64, 1>(a, s);
  if (t.lanes == 128) return launch_norm_backward<IO, 128, 1>(a, s);
  if (t.lanes == 256 && t.nc == 2) return launch_norm_backward<IO, 256, 2>(a, s);
  if (t.lanes == 256) return launch_norm_backward<IO, 256, 1>(a, s);
  if (t.nc == 1) return launch_norm_backward<IO, 1024, 1>(a, s);
  if (t.nc == 2) return launch_norm_backward<IO, 1024, 2>(a, s);
  if (t.nc == 4) return launch_norm_backward<IO, 1024, 4>(a, s);
  if constexpr (sizeof(typename IO::type) == 4) return launch_norm_backward<IO, 1024, 8>(a, s);
  return fail(EP_ERR_SHAPE, "rows too long");  // not reached: validate_rows bounds them
}

}  // namespace

extern "C" {

ep_status ep_quantize_fp8(int32_t type, const void* x, int64_t num_rows, int32_t num_cols, int64_t row_stride,
                          uint32_t flags, uint8_t* codes, float* scales, void* stream) {
  if (flags & ~(uint32_t)EP_FP8_SCALES_COL_MAJOR) return fail(EP_ERR_SHAPE, "unknown quantise flags 0x%x", flags);
  ep_status st = validate_rows(type, num_rows, num_cols, EP_MAX_QUANT_COLS);
  if (st != EP_OK || num_rows == 0) return st;
  if (st = validate_stride("row", row_stride, num_cols); st != EP_OK) return st;
  const int64_t nb = ((int64_t)num_cols + 127) / 128;
  if (num_rows * nb >= (int64_t)1 << 31)
    return fail(EP_ERR_OVERFLOW, "%lld rows of %d: 2^31 scales or more", (long long)num_rows, num_cols);
  if (!x || !codes || !scales) return fail(EP_ERR_NULL, "x / codes / scales is NULL");
  if (misaligned(x, type_bytes(type)) || misaligned(scales, 4))
    return fail(EP_ERR_SHAPE, "x / scales must be aligned to their element size");
  const bool cols = flags & EP_FP8_SCALES_COL_MAJOR;
  QuantFp8Args a{x, row_stride, codes, scales, cols ? 1 : nb, cols ? num_rows : 1, (uint32_t)num_rows, num_cols,
                 (uint32_t)nb, 0, 31};
  while ((int64_t)1 << (a.shift - 31) < nb) ++a.shift;
  a.magic = (uint32_t)((((uint64_t)1 << a.shift) + nb - 1) / nb);
  return with_type(type, [&](auto io) -> ep_status {
    constexpr int kEach = 16 * kQuantBlocks<decltype(io)>;
    const unsigned blocks = (unsigned)((num_rows * nb + kEach - 1) / kEach);
    quantize_fp8_kernel<decltype(io)><<<blocks, 256, 0, (hipStream_t)stream>>>(a);
    EP_LAUNCHED("quantize_fp8_kernel");
    return EP_OK;
  });
}

ep_status ep_rms_norm(int32_t type, const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                      const void* weight, int32_t weight_type, float eps, int64_t num_rows, int32_t num_cols,
                      void* total, void* y, uint8_t* codes, float* scales, void* stream) {
  ep_status st = validate_norm(type, num_rows, num_cols, weight_type, eps);
  if (st != EP_OK || num_rows == 0) return st;
  if (st = validate_stride("x", x_stride, num_cols); st != EP_OK) return st;
  if (!x || !weight || (residual && !total)) return fail(EP_ERR_NULL, "x / weight / total is NULL");
  if (!y && !codes) return fail(EP_ERR_NULL, "y and codes are NULL: nothing to write");
  if (codes && !scales) return fail(EP_ERR_NULL, "scales is NULL");
  if (residual)
    if (st = validate_stride("residual", residual_stride, num_cols); st != EP_OK) return st;
  const uintptr_t b = type_bytes(type);
  if (misaligned(x, b) || misaligned(residual, b) || misaligned(weight, type_bytes(weight_type)) || misaligned(total, b) ||
      misaligned(y, b) || misaligned(scales, 4))
    return fail(EP_ERR_SHAPE, "every array must be aligned to its element size");
  NormArgs a{x, residual, weight, total, y, codes, scales, x_stride, residual_stride, num_rows, num_cols,
             weight_type == EP_TYPE_F32, eps};
  return with_type(type, [&](auto io) { return launch_norm<decltype(io)>(a, (hipStream_t)stream); });
}

ep_status ep_rms_norm_backward_workspace(int32_t type, int64_t num_rows, int32_t num_cols, int64_t* bytes) {
  if (!bytes) return fail(EP_ERR_NULL, "bytes is NULL");
  const ep_status st = validate_rows(type, num_rows, num_cols, EP_MAX_NORM_COLS);
  if (st != EP_OK) return st;
  *bytes = (int64_t)norm_teams(type, num_rows, num_cols).groups * num_cols * (int64_t)sizeof(float);
  return EP_OK;
}

ep_status ep_rms_norm_backward(int32_t type, const void* x, int64_t x_stride, const void* weight, int32_t weight_type,
                               float eps, const void* grad, int64_t grad_stride, const void* grad_total,
                               int64_t grad_total_stride, int64_t num_rows, int32_t num_cols, void* grad_x,
                               float* grad_weight, void* workspace, void* stream) {
  ep_status st = validate_norm(type, num_rows, num_cols, weight_type, eps);
  if (st != EP_OK) return st;
  if (!grad_weight) return fail(EP_ERR_NULL, "grad_weight is NULL");
  if (misaligned(grad_weight, 4)) return fail(EP_ERR_SHAPE, "grad_weight must be 4-byte aligned");
  const NormTeams t = norm_teams(type, num_rows, num_cols);
  hipStream_t s = (hipStream_t)stream;
  if (num_rows > 0) {
    if (st = validate_stride("x", x_stride, num_cols); st != EP_OK) return st;
    if (st = validate_stride("grad", grad_stride, num_cols); st != EP_OK) return st;
    if (!x || !weight || !grad || !grad_x || !workspace)
      return fail(EP_ERR_NULL, "x / weight / grad / grad_x / workspace is NULL");
    if (grad_total)
      if (st = validate_stride("grad_total", grad_total_stride, num_cols); st != EP_OK) return st;
    const uintptr_t b = type_bytes(type);
    if (misaligned(x, b) || misaligned(weight, type_bytes(weight_type)) || misaligned(grad, b) ||
        misaligned(grad_total, b) || misaligned(grad_x, b) || misaligned(workspace, 4))
      return fail(EP_ERR_SHAPE, "every array must be aligned to its element size");
    NormBwdArgs a{x, weight, grad, grad_total, grad_x, (float*)workspace, x_stride, grad_stride, grad_total_stride,
                  num_rows, t.groups, num_cols, weight_type == EP_TYPE_F32, eps};
    st = with_type(type, [&](auto io) { return launch_norm_backward<decltype(io)>(a, t, s); });
    if (st != EP_OK) return st;
  }
  norm_weight_kernel<<<(num_cols + 31) / 32, 1024, 0, s>>>((const float*)workspace, t.groups, num_cols, grad_weight);
  EP_LAUNCHED("norm_weight_kernel");
  return EP_OK;
}

}  // extern "C"
