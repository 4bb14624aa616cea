// ep_half.hip -- host side of the 16-bit product: argument checks and launch.
#include "ep_product_launch.hpp"

using namespace ep;

namespace {

// inner and, for the gradient, outer: 16 bytes are whole numbers of values.
ep_status validate_half(int32_t type, int64_t num_rows, int32_t num_groups, int32_t inner, int32_t outer, uint32_t flags) {
  const ep_status st = validate_matmul(num_rows, num_groups, outer, flags);
  if (st != EP_OK) return st;
  if (type != EP_TYPE_BF16 && type != EP_TYPE_F16) return fail(EP_ERR_SHAPE, "element type %d must be bf16 or fp16", type);
  if (inner < 8 || inner % 8 != 0 || inner > EP_MAX_MATMUL_INNER)
    return fail(EP_ERR_SHAPE, "inner %d must be a multiple of 8 in [8, %d]", inner, EP_MAX_MATMUL_INNER);
  return EP_OK;
}

}  // namespace

extern "C" {

ep_status ep_matmul(int32_t type, const void* a, int64_t num_rows, const void* w, int32_t num_groups,
                    const int64_t* row_start, const int32_t* row_count, int32_t inner, int32_t outer, uint32_t flags,
                    void* pre, void* out, void* stream) {
  const ep_status st = validate_half(type, num_rows, num_groups, inner, outer, flags);
  if (st != EP_OK) return st;
  const bool gated = flags & EP_MATMUL_GATED;
  if (pre && !gated) return fail(EP_ERR_SHAPE, "pre belongs to a gated product");
  if (num_rows == 0) return EP_OK;
  if (!a || !w || !out) return fail(EP_ERR_NULL, "a / w / out is NULL");
  if (num_groups > 0 && (!row_start || !row_count)) return fail(EP_ERR_NULL, "row_start / row_count is NULL");
  if (misaligned(a, 16) || misaligned(w, 16) || misaligned(out, 16) || misaligned(pre, 16) || misaligned(row_start, 8) ||
      misaligned(row_count, 4))
    return fail(EP_ERR_SHAPE, "a / w / out / pre must be 16-byte aligned, other arrays aligned to their element size");
  MatmulArgs m{(const uint8_t*)a, nullptr, (const uint8_t*)w, nullptr, num_groups > 0 ? row_start : nullptr,
               num_groups > 0 ? row_count : nullptr, out, num_rows, std::max(num_groups, 1), outer, inner * 2,
               gated ? outer / 2 : outer, 0, num_rows, pre, 0, 0};
  hipStream_t s = (hipStream_t)stream;
  if (type == EP_TYPE_BF16)
    return gated ? launch_matmul<Bf16Math, Bf16, true>(m, s) : launch_matmul<Bf16Math, Bf16, false>(m, s);
  return gated ? launch_matmul<F16Math, F16, true>(m, s) : launch_matmul<F16Math, F16, false>(m, s);
}

}  // extern "C"
