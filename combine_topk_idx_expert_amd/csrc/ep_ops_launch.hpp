// ep_ops_launch.hpp -- argument checks and launch configuration of the router and
// of int8 quantising.
//
// Part of ep_api.hip's translation unit: it is included there, inside the
// anonymous namespace, after the error helpers (fail, EP_LAUNCHED) it uses.
#pragma once

ep_status validate_route(const ep_route_config* c, int32_t type, int64_t num_tokens, int64_t row_stride) {
  if (!c) return fail(EP_ERR_NULL, "route config is NULL");
  if (c->num_experts < 1 || c->num_experts > EP_MAX_EXPERTS)
    return fail(EP_ERR_SHAPE, "num_experts %d outside [1, %d]", c->num_experts, EP_MAX_EXPERTS);
  if (c->num_topk < 1 || c->num_topk > EP_MAX_TOPK)
    return fail(EP_ERR_SHAPE, "num_topk %d outside [1, %d]", c->num_topk, EP_MAX_TOPK);
  if (c->num_groups < 1 || c->num_groups > EP_MAX_ROUTE_GROUPS || c->num_experts % c->num_groups != 0)
    return fail(EP_ERR_SHAPE, "num_groups %d must divide num_experts %d and lie in [1, %d]", c->num_groups,
                c->num_experts, EP_MAX_ROUTE_GROUPS);
  if (c->topk_groups < 1 || c->topk_groups > c->num_groups)
    return fail(EP_ERR_SHAPE, "topk_groups %d outside [1, %d]", c->topk_groups, c->num_groups);
  if (c->num_topk > c->topk_groups * (c->num_experts / c->num_groups))
    return fail(EP_ERR_SHAPE, "num_topk %d exceeds the %d experts of topk_groups groups", c->num_topk,
                c->topk_groups * (c->num_experts / c->num_groups));
  if (c->score != EP_SCORE_SOFTMAX && c->score != EP_SCORE_SIGMOID)
    return fail(EP_ERR_SHAPE, "unknown score %d", c->score);
  if (c->group_score != EP_GROUP_MAX && c->group_score != EP_GROUP_TOP2)
    return fail(EP_ERR_SHAPE, "unknown group score %d", c->group_score);
  if (!(c->scale - c->scale == 0.0f)) return fail(EP_ERR_SHAPE, "scale must be finite");
  if (type != EP_TYPE_F32 && type != EP_TYPE_BF16 && type != EP_TYPE_F16)
    return fail(EP_ERR_SHAPE, "unknown element type %d", type);
  if (num_tokens < 0) return fail(EP_ERR_SHAPE, "num_tokens %lld < 0", (long long)num_tokens);
  if (num_tokens > 0 && row_stride < c->num_experts)
    return fail(EP_ERR_SHAPE, "row_stride %lld below num_experts %d", (long long)row_stride, c->num_experts);
  if (num_tokens > EP_MAX_ROUTE_TOKENS)
    return fail(EP_ERR_OVERFLOW, "num_tokens %lld above %d", (long long)num_tokens, EP_MAX_ROUTE_TOKENS);
  if (row_stride > ((int64_t)1 << 40)) return fail(EP_ERR_OVERFLOW, "row_stride %lld too large", (long long)row_stride);
  return EP_OK;
}

template <typename IO, int LPR, int VPL, int R>
ep_status launch_route_lanes(const RouteArgs& a, RouteLanes p, hipStream_t s) {
  constexpr int kRows = kWave / LPR;
  p.pad = p.seg != VPL || p.gs * a.G != p.seg * LPR;
  const size_t lds = std::max(((size_t)kRows * p.row_pitch + VPL) * sizeof(float), (size_t)a.E * sizeof(double));
  route_lanes_kernel<IO, LPR, VPL, R><<<(a.T + kRows - 1) / kRows, kWave, lds, s>>>(a, p);
  EP_LAUNCHED("route_lanes_kernel");
  return EP_OK;
}

template <typename IO, int LPR, int VPL>
ep_status launch_route_lanes(const RouteArgs& a, const RouteLanes& p, hipStream_t s) {
  return a.K <= 8 ? launch_route_lanes<IO, LPR, VPL, 1>(a, p, s) : launch_route_lanes<IO, LPR, VPL, 2>(a, p, s);
}

// Up to 512 experts and 16 choices: several rows a wave.  A group is 1, 2, 4 or 8
// lanes of eight, or of sixteen where eight lanes of 32 experts do not hold it;
// routers for which that does not come out, and wider ones, take one row a wave.
template <typename IO>
ep_status launch_route(const RouteArgs& a, hipStream_t s) {
  for (int lanes = 8; a.K <= 16 && lanes <= 16; lanes *= 2) {
    if (a.G > lanes) continue;
    RouteLanes p{};
    p.gs = a.E / a.G;
    while (a.G << (p.shift + 1) <= lanes && (a.G == 1 || p.shift < 3)) ++p.shift;
    const int wide = 1 << p.shift;
    p.seg = (p.gs + wide - 1) / wide;
    if (a.G == 1) p.seg = (p.seg + 3) / 4 * 4;
    if (p.seg > 32) continue;
    if (a.G == 1 || (p.gs == wide * p.seg && p.seg % 4 == 0)) {
      p.pitch = 4 * ((p.seg + 3) / 4 | 1);
      p.row_pitch = lanes * p.pitch;
      p.magic = (1 << 20) / p.seg + 1;
    } else {
      p.row_pitch = (a.E + 3) / 4 * 4;
    }
    p.bias_vec = p.seg % 4 == 0 && p.gs % 4 == 0 && !misaligned(a.bias, 16);
    if (lanes == 16) return launch_route_lanes<IO, 16, 32>(a, p, s);
    if (p.seg <= 8 && a.K <= 8) return launch_route_lanes<IO, 8, 8, 1>(a, p, s);
    if (p.seg <= 16) return launch_route_lanes<IO, 8, 16>(a, p, s);
    return launch_route_lanes<IO, 8, 32>(a, p, s);
  }
  const int waves = a.E > 2048 ? kRouteWaves / 2 : kRouteWaves;  // at most 64 KiB of LDS
  const int blocks = (a.T + waves - 1) / waves;
  route_kernel<IO><<<blocks, waves * kWave, (size_t)waves * a.E * sizeof(double), s>>>(a);
  EP_LAUNCHED("route_kernel");
  return EP_OK;
}

template <typename IO, int LPR>
ep_status launch_route_backward_lanes(const RouteBwdArgs& a, hipStream_t s) {
  constexpr int kRows = kWave / LPR, V = 16 / sizeof(typename IO::type);
  const bool dense = !a.sigmoid && !a.renorm;
  const int vec = a.E % V == 0;
  const size_t lds = (size_t)kRows * a.E * sizeof(float);
  const int blocks = (int)std::min<int64_t>((a.T + kRows - 1) / kRows, 16 * kCUs);
  const int pieces = (a.E / V + LPR - 1) / LPR;  // of a row, a lane
  if (dense && pieces <= 2)
    route_backward_lanes_kernel<IO, LPR, 2><<<blocks, kWave, lds, s>>>(a, vec);
  else if (dense && pieces <= 4)
    route_backward_lanes_kernel<IO, LPR, 4><<<blocks, kWave, lds, s>>>(a, vec);
  else if (dense && pieces <= 8)
    route_backward_lanes_kernel<IO, LPR, 8><<<blocks, kWave, lds, s>>>(a, vec);
  else
    route_backward_lanes_kernel<IO, LPR, 0><<<blocks, kWave, lds, s>>>(a, vec);
  EP_LAUNCHED("route_backward_lanes_kernel");
  return EP_OK;
}

// Up to 16 choices of 1024 experts: several rows a wave (at most 32 KiB of LDS).
template <typename IO>
ep_status launch_route_backward(const RouteBwdArgs& a, hipStream_t s) {
  if (a.E <= 1024 && a.K <= 8) return launch_route_backward_lanes<IO, 8>(a, s);
  if (a.E <= 1024 && a.K <= 16) return launch_route_backward_lanes<IO, 16>(a, s);
  const int blocks = (a.T + kRouteWaves - 1) / kRouteWaves;
  const size_t lds = (size_t)kRouteWaves * a.E * sizeof(float);
  route_backward_kernel<IO><<<blocks, kRouteWaves * kWave, lds, s>>>(a);
  EP_LAUNCHED("route_backward_kernel");
  return EP_OK;
}

template <typename IO, int WAVES>
ep_status launch_quantize_rows(const QuantArgs& a, int nc, hipStream_t s) {
  const int blocks = (int)((a.N * WAVES + 3) / 4);
  if (nc <= 1)
    quantize_rows_kernel<IO, WAVES, 1><<<blocks, 256, 0, s>>>(a);
  else if (nc <= 2)
    quantize_rows_kernel<IO, WAVES, 2><<<blocks, 256, 0, s>>>(a);
  else if (nc <= 4)
    quantize_rows_kernel<IO, WAVES, 4><<<blocks, 256, 0, s>>>(a);
  else
    quantize_rows_kernel<IO, WAVES, 8><<<blocks, 256, 0, s>>>(a);
  EP_LAUNCHED("quantize_rows_kernel");
  return EP_OK;
}

template <typename IO>
ep_status launch_quantize(const QuantArgs& a, hipStream_t s) {
  constexpr int V = 16 / sizeof(typename IO::type);
  const int chunks = a.H / V;
  const bool whole = a.H % V == 0;
  if (whole && a.N >= 4 * kCUs && chunks <= 8 * kWave) return launch_quantize_rows<IO, 1>(a, (chunks + 63) / 64, s);
  if (whole && chunks <= 8 * 4 * kWave) return launch_quantize_rows<IO, 4>(a, (chunks + 255) / 256, s);
  quantize_kernel<IO><<<(int)a.N, kQuantThreads, 0, s>>>(a);
  EP_LAUNCHED("quantize_kernel");
  return EP_OK;
}
