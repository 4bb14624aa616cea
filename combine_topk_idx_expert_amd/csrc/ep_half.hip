// ep_half.hip -- host side of the 16-bit product and its gradients: argument checks
// and launch configuration.
#include "ep_half_grad.hpp"
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

ep_status validate_half_backward(int32_t type, int64_t num_rows, int32_t num_groups, int32_t inner, int32_t outer,
                                 uint32_t flags) {
  const ep_status st = validate_half(type, num_rows, num_groups, inner, outer, flags);
  if (st != EP_OK) return st;
  const int whole = flags & EP_MATMUL_GATED ? 16 : 8;
  if (outer % whole != 0) return fail(EP_ERR_SHAPE, "outer %d must be a multiple of %d", outer, whole);
  return EP_OK;
}

template <typename AR, typename IO, bool WEIGHTS, int BM, bool HALVES>
ep_status launch_half_grad(const MatmulArgs& a, int64_t most, int n_tiles, hipStream_t s) {
  typedef TileShape<BM, 256, 2, 4> S;
  if (most >= (int64_t)1 << 31) return fail(EP_ERR_OVERFLOW, "gradient of %lld tiles is too large", (long long)most);
  const int grid = (int)std::min<int64_t>(most, kCUs);
  half_grad_kernel<AR, IO, WEIGHTS, BM, 256, 2, 4, HALVES>
      <<<grid, S::kThreads, S::lds(WEIGHTS ? 0 : a.G, false), s>>>(a, n_tiles);
  EP_LAUNCHED("half_grad_kernel");
  return EP_OK;
}

// Rows' gradient: tiles as the product of that width has them.
template <typename AR, typename IO>
ep_status launch_grad_rows(const MatmulArgs& a, hipStream_t s) {
  const int n_tiles = (a.width + 255) / 256;
  if (matmul_kernels(a.M, a.row_start ? a.G : 0, a.width, false) & EP_KERNEL_TILES_256)
    return launch_half_grad<AR, IO, false, 256, true>(a, (a.M / 256 + a.G) * n_tiles, n_tiles, s);
  return launch_half_grad<AR, IO, false, 128, false>(a, (a.M / 128 + a.G) * n_tiles, n_tiles, s);
}

// Weights' gradient: 256 x 256 once such tiles fill three quarters of the CUs.
template <typename AR, typename IO>
ep_status launch_grad_weights(const MatmulArgs& a, hipStream_t s) {
  const int n_tiles = (a.width + 255) / 256;
  const int64_t tall = (int64_t)a.G * ((a.N + 255) / 256) * n_tiles;
  if (tall >= 3 * kCUs / 4) return launch_half_grad<AR, IO, true, 256, true>(a, tall, n_tiles, s);
  return launch_half_grad<AR, IO, true, 128, false>(a, (int64_t)a.G * ((a.N + 127) / 128) * n_tiles, n_tiles, s);
}

template <typename IO>
ep_status launch_gate_backward(const void* pre, const void* grad, int64_t rows, int width, void* out, hipStream_t s) {
  const int64_t pieces = rows * (width / 8);
  const int blocks = (int)std::min<int64_t>((pieces + 255) / 256, 32 * kCUs);
  gate_backward_kernel<IO><<<blocks, 256, 0, s>>>(pre, grad, pieces, width, out);
  EP_LAUNCHED("gate_backward_kernel");
  return EP_OK;
}

template <typename AR, typename IO>
ep_status matmul_backward(const MatmulArgs& rows, const MatmulArgs& weights, const void* pre, const void* grad, void* space,
                          int32_t grad_w_type, hipStream_t s) {
  if (pre && rows.M > 0) {
    const ep_status st = launch_gate_backward<IO>(pre, grad, rows.M, rows.N / 2, space, s);
    if (st != EP_OK) return st;
  }
  if (rows.out && rows.M > 0) {
    const ep_status st = launch_grad_rows<AR, IO>(rows, s);
    if (st != EP_OK) return st;
  }
  if (!weights.out) return EP_OK;
  return grad_w_type == EP_TYPE_F32 ? launch_grad_weights<AR, F32>(weights, s) : launch_grad_weights<AR, IO>(weights, s);
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

ep_status ep_matmul_backward_workspace(int64_t num_rows, int32_t outer, uint32_t flags, int64_t* bytes) {
  if (!bytes) return fail(EP_ERR_NULL, "bytes is NULL");
  const ep_status st = validate_matmul(num_rows, 0, outer, flags);
  if (st != EP_OK) return st;
  *bytes = flags & EP_MATMUL_GATED ? num_rows * outer * 2 : 0;
  return EP_OK;
}

ep_status ep_matmul_backward(int32_t type, const void* a, int64_t num_rows, const void* w, const void* grad,
                             const void* pre, int32_t num_groups, const int64_t* row_start, const int32_t* row_count,
                             int32_t inner, int32_t outer, uint32_t flags, void* grad_a, void* grad_w,
                             int32_t grad_w_type, void* workspace, void* stream) {
  const ep_status st = validate_half_backward(type, num_rows, num_groups, inner, outer, flags);
  if (st != EP_OK) return st;
  const bool gated = flags & EP_MATMUL_GATED;
  if (grad_w_type != type && grad_w_type != EP_TYPE_F32)
    return fail(EP_ERR_SHAPE, "grad_w's type %d must be the rows' or fp32", grad_w_type);
  if (!grad_a && !grad_w) return fail(EP_ERR_NULL, "grad_a and grad_w are NULL: nothing to write");
  if (num_groups > 0 && (!row_start || !row_count)) return fail(EP_ERR_NULL, "row_start / row_count is NULL");
  if (num_rows > 0 && (!a || !w || !grad)) return fail(EP_ERR_NULL, "a / w / grad is NULL");
  if (num_rows > 0 && gated && (!pre || !workspace)) return fail(EP_ERR_NULL, "pre / workspace is NULL");
  if (!gated && pre) return fail(EP_ERR_SHAPE, "pre belongs to a gated product");
  if (misaligned(a, 16) || misaligned(w, 16) || misaligned(grad, 16) || misaligned(pre, 16) || misaligned(grad_a, 16) ||
      misaligned(grad_w, 16) || misaligned(workspace, 16) || misaligned(row_start, 8) || misaligned(row_count, 4))
    return fail(EP_ERR_SHAPE, "tensors and workspace must be 16-byte aligned, other arrays aligned to their element size");
  const uint8_t* d = (const uint8_t*)(gated ? workspace : grad);
  const int64_t* start = num_groups > 0 ? row_start : nullptr;
  const int32_t* count = num_groups > 0 ? row_count : nullptr;
  const int G = std::max(num_groups, 1);
  const MatmulArgs r{d, nullptr, (const uint8_t*)w, nullptr, start, count, grad_a, num_rows, G, outer, outer * 2, inner,
                     0, num_rows, nullptr, 0, 0};
  MatmulArgs g = r;
  g.w = (const uint8_t*)a;
  g.out = grad_w;
  hipStream_t s = (hipStream_t)stream;
  return type == EP_TYPE_BF16 ? matmul_backward<Bf16Math, Bf16>(r, g, pre, grad, workspace, grad_w_type, s)
                              : matmul_backward<F16Math, F16>(r, g, pre, grad, workspace, grad_w_type, s);
}

}  // extern "C"
