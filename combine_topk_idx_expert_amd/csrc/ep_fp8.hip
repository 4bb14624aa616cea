// ep_fp8.hip -- host side of the E4M3 product: argument checks and launch.
#include "ep_product_launch.hpp"

using namespace ep;

extern "C" ep_status ep_matmul_fp8(const uint8_t* a, const float* a_scale, int64_t num_rows, const uint8_t* w,
                                   const float* w_scale, int32_t num_groups, const int64_t* row_start,
                                   const int32_t* row_count, int32_t inner, int32_t outer, uint32_t flags,
                                   int32_t out_type, void* out, void* stream) {
  const ep_status st =
      validate_matmul(num_rows, num_groups, outer, flags, EP_MATMUL_GATED | EP_FP8_SCALES_COL_MAJOR);
  if (st != EP_OK) return st;
  if (!known_type(out_type)) return fail(EP_ERR_SHAPE, "unknown element type %d", out_type);
  const bool gated = flags & EP_MATMUL_GATED;
  if (inner < 16 || inner % 16 != 0 || inner > EP_MAX_MATMUL_INNER)
    return fail(EP_ERR_SHAPE, "inner %d must be a multiple of 16 in [16, %d]", inner, EP_MAX_MATMUL_INNER);
  if (num_rows == 0) return EP_OK;
  if (!a || !a_scale || !w || !w_scale || !out) return fail(EP_ERR_NULL, "a / a_scale / w / w_scale / out is NULL");
  if (num_groups > 0 && (!row_start || !row_count)) return fail(EP_ERR_NULL, "row_start / row_count is NULL");
  if (misaligned(a, 16) || misaligned(w, 16) || misaligned(out, 16) || misaligned(a_scale, 4) ||
      misaligned(w_scale, 4) || misaligned(row_start, 8) || misaligned(row_count, 4))
    return fail(EP_ERR_SHAPE, "a / w / out must be 16-byte aligned, other arrays aligned to their element size");
  const bool cols = flags & EP_FP8_SCALES_COL_MAJOR;
  MatmulArgs m{a, a_scale, w, w_scale, num_groups > 0 ? row_start : nullptr, num_groups > 0 ? row_count : nullptr,
               out, num_rows, std::max(num_groups, 1), outer, inner, gated ? outer / 2 : outer, 0, num_rows, nullptr,
               cols ? 1 : (inner + 127) / 128, cols ? num_rows : 1, 1};
  return with_type(out_type, [&](auto io) {
    typedef std::conditional_t<std::is_same_v<decltype(io), F32>, Fp8ExactMath, Fp8Math> AR;
    return gated ? launch_matmul<AR, decltype(io), true>(m, (hipStream_t)stream)
                 : launch_matmul<AR, decltype(io), false>(m, (hipStream_t)stream);
  });
}

extern "C" ep_status ep_debug_product_kernels(int64_t num_rows, int32_t num_groups, int32_t outer, uint32_t flags,
                                              int32_t out_type, uint32_t* kernels) {
  if (!kernels) return fail(EP_ERR_NULL, "kernels is NULL");
  const ep_status st = validate_matmul(num_rows, num_groups, outer, flags);
  if (st != EP_OK) return st;
  if (!known_type(out_type)) return fail(EP_ERR_SHAPE, "unknown element type %d", out_type);
  const bool gated = flags & EP_MATMUL_GATED;
  const int width = gated ? outer / 2 : outer;
  *kernels = num_rows == 0             ? 0
             : out_type == EP_TYPE_F32 ? product_kernels<Fp8ExactMath>(num_rows, num_groups, width, gated)
                                       : product_kernels<Bf16Math>(num_rows, num_groups, width, gated);
  return EP_OK;
}

extern "C" ep_status ep_debug_split_shape(int64_t num_rows, int32_t num_groups, int32_t inner_bytes, int32_t outer,
                                          uint32_t flags, int32_t* shape) {
  if (!shape) return fail(EP_ERR_NULL, "shape is NULL");
  const ep_status st = validate_matmul(num_rows, num_groups, outer, flags);
  if (st != EP_OK) return st;
  if (inner_bytes < 1 || inner_bytes > 2 * EP_MAX_MATMUL_INNER)
    return fail(EP_ERR_SHAPE, "inner_bytes %d must lie in [1, %d]", inner_bytes, 2 * EP_MAX_MATMUL_INNER);
  const bool gated = flags & EP_MATMUL_GATED;
  MatmulArgs m{};
  m.M = num_rows;
  m.G = std::max(num_groups, 1);
  m.N = outer;
  m.K = inner_bytes;
  m.width = gated ? outer / 2 : outer;
  const uint32_t kernels = num_rows == 0 ? 0 : matmul_kernels(num_rows, num_groups, m.width, gated);
  m.most = kernels == EP_KERNEL_SPLIT ? num_rows : kFewRows;
  const SplitShape t = kernels & EP_KERNEL_SPLIT ? split_shape(m, gated) : SplitShape{};
  shape[0] = t.rows * 16;
  shape[1] = t.cols * 16;
  shape[2] = t.waves;
  return EP_OK;
}
