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

// How a gradient is cut: tiles of 256 or 128 rows by 256 columns, slices of the inner dimension.
struct GradPlan {
  bool tall;
  int n_tiles, slices;
  int64_t most;  // tiles of a slice, at most
};

// Slices for fewer tiles of 128 rows than half the CUs, as many as cost least: a tile takes
// 0.45 us for 32 inner indexes, and slices 5 us and the writing and reading of their fp32
// results, at 4 TB/s.  (32768 rows, 512 x 512: 8 tiles; the weights' gradient in one piece
// 446 us, in 32 slices 40; 10999 rows of 15 groups, 1512 x 112: 90 tiles, one slice 18 us,
// two 25; the rows' gradient of one row, 4096 x 4096: 54 us, in 16 slices 16.)
int best_slices(int64_t tiles, int64_t inner, int64_t result_bytes) {
  const int most = (int)std::min<int64_t>(kCUs / std::max<int64_t>(tiles, 1), inner / 128);
  int best = 1;
  double least = 0.45 * inner / 32;
  for (int k = 2; k <= most; ++k) {
    const double t = 0.45 * inner / 32 / k + 5 + 2e-6 / 4 * k * result_bytes;
    if (t < least) least = t, best = k;
  }
  return best;
}

// Rows' gradient: width = inner of the product, its inner dimension are the channels.  Tiles of
// 256 rows where an int8 product of that width takes them (the rule that dense 16-bit products
// have instead, tall_tiles, was not timed for gradients).
GradPlan plan_rows(int64_t M, int G, int inner, int outer) {
  const bool tall = matmul_kernels(M, G, inner, false) & EP_KERNEL_TILES_256;
  const int rows = tall ? 256 : 128;
  GradPlan p{tall, (inner + 255) / 256, 1, 0};
  // (each group's last row tile may be partly filled; no more groups than rows have any)
  p.most = (G == 0 ? (M + rows - 1) / rows : M / rows + std::min<int64_t>(G, M)) * p.n_tiles;
  if (!tall) p.slices = best_slices(p.most, outer, M * inner * 4);
  return p;
}

// Weights' gradient: channels by inner, over the rows of a group.  Tiles of 256 channels once
// they fill three quarters of the CUs.
GradPlan plan_weights(int64_t M, int G, int inner, int outer) {
  const int64_t groups = std::max(G, 1);
  GradPlan p{false, (inner + 255) / 256, 1, 0};
  p.tall = groups * ((outer + 255) / 256) * p.n_tiles >= 3 * kCUs / 4;
  p.most = groups * ((outer + (p.tall ? 255 : 127)) / (p.tall ? 256 : 128)) * p.n_tiles;
  if (!p.tall) p.slices = best_slices(p.most, M / groups, groups * outer * inner * 4);
  return p;
}

int64_t round_up(int64_t n) { return (n + 255) / 256 * 256; }

// The workspace: the gate's gradient, then the slices of one gradient after the other.
int64_t gate_bytes(int64_t M, int outer, bool gated) { return gated ? round_up(M * outer * 2) : 0; }
int64_t slice_bytes(const GradPlan& p, int64_t rows, int width) {
  return p.slices > 1 ? (int64_t)p.slices * rows * width * 4 : 0;
}

template <typename AR, typename IO, bool WEIGHTS, int BM, bool HALVES>
ep_status launch_half_grad(const MatmulArgs& a, const GradPlan& p, hipStream_t s) {
  typedef StepShape<BM, 256, 2, 4, false> S;
  const int64_t most = p.most * a.slices;
  if (most >= (int64_t)1 << 31) return fail(EP_ERR_OVERFLOW, "gradient of %lld tiles is too large", (long long)most);
  const int grid = (int)std::min<int64_t>(most, kCUs);
  half_grad_kernel<AR, IO, WEIGHTS, BM, 256, 2, 4, HALVES>
      <<<grid, S::kThreads, S::lds(WEIGHTS ? 0 : a.G), s>>>(a, p.n_tiles);
  EP_LAUNCHED("half_grad_kernel");
  return EP_OK;
}

template <typename IO>
ep_status launch_join(const MatmulArgs& a, const float* parts, hipStream_t s) {
  const int64_t mean = (a.M + a.G - 1) / a.G;
  const dim3 grid((a.width + 511) / 512, (unsigned)std::min<int64_t>((mean + 3) / 4, 4096), a.G);
  join_slices_kernel<IO><<<grid, 256, 0, s>>>(a, parts);
  EP_LAUNCHED("join_slices_kernel");
  return EP_OK;
}

// IO: the result's type; `space` holds the slices.
template <typename AR, typename IO, bool WEIGHTS>
ep_status launch_grad(MatmulArgs a, const GradPlan& p, void* space, hipStream_t s) {
  if (p.tall) return launch_half_grad<AR, IO, WEIGHTS, 256, true>(a, p, s);
  if (p.slices == 1) return launch_half_grad<AR, IO, WEIGHTS, 128, false>(a, p, s);
  MatmulArgs parts = a;
  parts.slices = a.slices = p.slices;
  parts.out = space;
  const ep_status st = launch_half_grad<AR, F32, WEIGHTS, 128, false>(parts, p, s);
  if (st != EP_OK) return st;
  if (WEIGHTS) {  // every row of the result
    a.M = (int64_t)a.G * a.N;
    a.G = 1;
    a.row_start = nullptr;
  }
  return launch_join<IO>(a, (const float*)space, s);
}

template <typename IO>
ep_status launch_gate_backward(const void* pre, const void* grad, int64_t rows, int width, void* out, hipStream_t s) {
  const int64_t pieces = rows * (width / 8);
  const int blocks = (int)std::min<int64_t>((pieces + 255) / 256, 32 * kCUs);
  gate_backward_kernel<IO><<<blocks, 256, 0, s>>>(pre, grad, pieces, width, out);
  EP_LAUNCHED("gate_backward_kernel");
  return EP_OK;
}

// `rows` and `weights` are the two gradients' arguments (out null: not wanted).
template <typename AR, typename IO>
ep_status matmul_backward(const MatmulArgs& rows, const MatmulArgs& weights, const void* pre, const void* grad,
                          void* workspace, int32_t grad_w_type, hipStream_t s) {
  const int64_t M = rows.M;
  const int G = rows.row_start ? rows.G : 0;
  uint8_t* space = (uint8_t*)workspace + gate_bytes(M, rows.N, pre != nullptr);
  if (pre && M > 0) {
    const ep_status st = launch_gate_backward<IO>(pre, grad, M, rows.N / 2, workspace, s);
    if (st != EP_OK) return st;
  }
  if (rows.out && M > 0) {
    const ep_status st = launch_grad<AR, IO, false>(rows, plan_rows(M, G, rows.width, rows.N), space, s);
    if (st != EP_OK) return st;
  }
  if (!weights.out) return EP_OK;
  const GradPlan p = plan_weights(M, G, rows.width, rows.N);
  return grad_w_type == EP_TYPE_F32 ? launch_grad<AR, F32, true>(weights, p, space, s)
                                    : launch_grad<AR, IO, true>(weights, p, space, s);
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
               gated ? outer / 2 : outer, 0, num_rows, pre, 0, 0, 1};
  hipStream_t s = (hipStream_t)stream;
  if (type == EP_TYPE_BF16)
    return gated ? launch_matmul<Bf16Math, Bf16, true>(m, s) : launch_matmul<Bf16Math, Bf16, false>(m, s);
  return gated ? launch_matmul<F16Math, F16, true>(m, s) : launch_matmul<F16Math, F16, false>(m, s);
}

ep_status ep_matmul_backward_workspace(int64_t num_rows, int32_t num_groups, int32_t inner, int32_t outer,
                                       uint32_t flags, int64_t* bytes) {
  if (!bytes) return fail(EP_ERR_NULL, "bytes is NULL");
  const ep_status st = validate_half_backward(EP_TYPE_BF16, num_rows, num_groups, inner, outer, flags);
  if (st != EP_OK) return st;
  const GradPlan r = plan_rows(num_rows, num_groups, inner, outer), w = plan_weights(num_rows, num_groups, inner, outer);
  *bytes = gate_bytes(num_rows, outer, flags & EP_MATMUL_GATED) +
           std::max(slice_bytes(r, num_rows, inner), slice_bytes(w, (int64_t)std::max(num_groups, 1) * outer, inner));
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
  if (num_rows > 0 && gated && !pre) return fail(EP_ERR_NULL, "pre is NULL");
  int64_t space = 0;
  if (ep_matmul_backward_workspace(num_rows, num_groups, inner, outer, flags, &space) == EP_OK && space > 0 && !workspace)
    return fail(EP_ERR_NULL, "workspace is NULL");
  if (!gated && pre) return fail(EP_ERR_SHAPE, "pre belongs to a gated product");
  if (misaligned(a, 16) || misaligned(w, 16) || misaligned(grad, 16) || misaligned(pre, 16) || misaligned(grad_a, 16) ||
      misaligned(grad_w, 16) || misaligned(workspace, 16) || misaligned(row_start, 8) || misaligned(row_count, 4))
    return fail(EP_ERR_SHAPE, "tensors and workspace must be 16-byte aligned, other arrays aligned to their element size");
  const uint8_t* d = (const uint8_t*)(gated ? workspace : grad);
  const int64_t* start = num_groups > 0 ? row_start : nullptr;
  const int32_t* count = num_groups > 0 ? row_count : nullptr;
  const int G = std::max(num_groups, 1);
  const MatmulArgs r{d, nullptr, (const uint8_t*)w, nullptr, start, count, grad_a, num_rows, G, outer, outer * 2, inner,
                     0, num_rows, nullptr, 0, 0, 1};
  MatmulArgs g = r;
  g.w = (const uint8_t*)a;
  g.out = grad_w;
  hipStream_t s = (hipStream_t)stream;
  return type == EP_TYPE_BF16 ? matmul_backward<Bf16Math, Bf16>(r, g, pre, grad, workspace, grad_w_type, s)
                              : matmul_backward<F16Math, F16>(r, g, pre, grad, workspace, grad_w_type, s);
}

ep_status ep_debug_backward_plan(int64_t num_rows, int32_t num_groups, int32_t inner, int32_t outer, uint32_t flags,
                                 int32_t* plan) {
  if (!plan) return fail(EP_ERR_NULL, "plan is NULL");
  const ep_status st = validate_half_backward(EP_TYPE_BF16, num_rows, num_groups, inner, outer, flags);
  if (st != EP_OK) return st;
  const GradPlan r = plan_rows(num_rows, num_groups, inner, outer), w = plan_weights(num_rows, num_groups, inner, outer);
  plan[0] = r.tall ? 256 : 128;
  plan[1] = r.slices;
  plan[2] = w.tall ? 256 : 128;
  plan[3] = w.slices;
  return EP_OK;
}

}  // extern "C"
