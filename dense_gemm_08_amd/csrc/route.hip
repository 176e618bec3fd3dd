// route.hip -- routing of tokens to experts (dense_gemm_route and its gradient,
// include/dense_gemm.h) on the MI355X (gfx950).  Host side: the plan
// (route_plan in plan_experts.cpp), the launches and the C ABI entry points.
// The kernels are in route_kernel.h.
#include "layer_host.h"
#include "plan_experts.h"
#include "route_kernel.h"

namespace dg {

namespace {

void set_routing(RouteParams& p, const void* logits, int64_t ld, int64_t T, int64_t E, int64_t k,
                 const dense_gemm_routing& r) {
  p.logits = logits;
  p.ld = ld;
  p.T = (int)T;
  p.E = (int)E;
  p.k = (int)k;
  p.sigmoid = r.score == DENSE_GEMM_SIGMOID;
  p.renorm = r.renorm;
  p.scale = r.scale;
}

// f(lanes per token, experts per lane) for E experts: 16 lanes up to 512 experts
// for the choice (4096 tokens of 512: 16.4 us, 28 with a wave a token), up to 256
// for the gradient (16384 of 512: 20.7, 17.3 so), a wave beyond.
template <int MOST16, typename Launch>
void by_experts(int64_t E, Launch&& launch) {
  using std::integral_constant;
  if (E <= 64)
    launch(integral_constant<int, 16>(), integral_constant<int, 4>());
  else if (E <= 128)
    launch(integral_constant<int, 16>(), integral_constant<int, 8>());
  else if (E <= 256)
    launch(integral_constant<int, 16>(), integral_constant<int, 16>());
  else if (E <= 512)
    launch(integral_constant<int, MOST16 == 512 ? 16 : 64>(), integral_constant<int, MOST16 == 512 ? 32 : 8>());
  else
    launch(integral_constant<int, 64>(), integral_constant<int, 16>());
}

template <typename F>
dense_gemm_status run_route(const RouteParams& p, const RoutePlan& plan, hipStream_t stream) {
  by_experts<512>(p.E, [&](auto lanes, auto per) {
    hipLaunchKernelGGL((route_choose<F, decltype(lanes)::value, decltype(per)::value>),
                       dim3((unsigned)plan.blocks), dim3(ROUTE_THREADS), 0, stream, p);
  });
  if (plan.blocks > 1)
    hipLaunchKernelGGL(route_place, dim3((unsigned)plan.blocks), dim3(ROUTE_THREADS), 0, stream, p);
  return launched();
}

template <typename F>
dense_gemm_status run_grad(const RouteGradParams& p, hipStream_t stream) {
  by_experts<256>(p.E, [&](auto lanes, auto per) {
    constexpr int tokens = ROUTE_GRAD_THREADS / decltype(lanes)::value;
    const int64_t blocks = ((int64_t)p.T + tokens - 1) / tokens, most = 1 << 16;
    hipLaunchKernelGGL((route_grad<F, decltype(lanes)::value, decltype(per)::value>),
                       dim3((unsigned)(blocks < most ? blocks : most)), dim3(ROUTE_GRAD_THREADS), 0,
                       stream, p);
  });
  return launched();
}

}  // namespace

}  // namespace dg

using namespace dg;

extern "C" {

dense_gemm_status dense_gemm_route(int fmt, int64_t T, int64_t E, int64_t k, const void* logits,
                                   int64_t ldl, const dense_gemm_routing* routing, void* weights,
                                   void* experts, void* places, void* ends, void* tokens,
                                   void* workspace, size_t workspace_bytes, hipStream_t stream) {
  dense_gemm_status st = route_validate(fmt, T, E, k, logits, ldl, routing, weights, experts, places,
                                        ends, tokens);
  if (st != DENSE_GEMM_OK) return st;
  int cus, xcds;
  st = device_topology(&cus, &xcds);
  if (st != DENSE_GEMM_OK) return st;
  const RoutePlan plan = route_plan(T, E);
  if (plan.bytes > 0) {
    if (workspace == nullptr || workspace_bytes < plan.bytes) return DENSE_GEMM_WORKSPACE_TOO_SMALL;
    if (((uintptr_t)workspace & 255) != 0) return DENSE_GEMM_MISALIGNED;
  }
  RouteParams p = {};
  set_routing(p, logits, ldl, T, E, k, *routing);
  p.bias = (const float*)routing->bias;
  p.weights = (float*)weights;
  p.experts = (int32_t*)experts;
  p.places = (int32_t*)places;
  p.ends = (int32_t*)ends;
  p.tokens = (int32_t*)tokens;
  p.counts = plan.blocks > 1 ? (uint32_t*)workspace : nullptr;
  p.groups = routing->groups;
  p.group_size = (int)(E / routing->groups);
  p.top_groups = routing->top_groups;
  // (where all groups stay their values do not matter)
  p.group_top = p.top_groups < p.groups ? routing->group_top : 1;
  p.ranked = p.bias == nullptr;
  // (up to 1024 experts, a group of m: e (2^20 + m) / m 2^-20 exceeds e / m by
  // less than 1 / m)
  p.group_inverse = (int)(((1 << 20) + p.group_size - 1) / p.group_size);
  for (int wide = 0; wide < 2; ++wide) {
    int& n = p.group_lanes[wide];
    n = 1;
    while (n < 16 && 2 * n * p.groups <= (wide ? 64 : 16)) n *= 2;
  }
  p.k_inverse = (int)(((1 << 20) + k - 1) / k);
  p.chunks = (int)plan.chunks;
  if (fmt == DENSE_GEMM_F32) return run_route<float>(p, plan, stream);
  return fmt == DENSE_GEMM_BF16 ? run_route<__bf16>(p, plan, stream) : run_route<_Float16>(p, plan, stream);
}

dense_gemm_status dense_gemm_route_workspace_size(int64_t T, int64_t E, int64_t k, size_t* bytes) {
  if (bytes == nullptr) return DENSE_GEMM_BAD_ARG;
  const void* any = (const void*)(uintptr_t)16;
  const dense_gemm_routing r = {nullptr, DENSE_GEMM_SOFTMAX, 0, 1.0f, 1, 1, 1};
  const dense_gemm_status st = route_validate(DENSE_GEMM_F32, T, E, k, any, E, &r, any, any, any, any, any);
  if (st == DENSE_GEMM_OK) *bytes = route_plan(T, E).bytes;
  return st;
}

dense_gemm_status dense_gemm_route_grad(int fmt, int64_t T, int64_t E, int64_t k, const void* logits,
                                        int64_t ldl, const dense_gemm_routing* routing,
                                        const void* experts, const void* dweights, void* dlogits,
                                        int64_t ldd, hipStream_t stream) {
  bool done;
  dense_gemm_status st = route_grad_validate(fmt, T, E, k, logits, ldl, routing, experts, dweights,
                                             dlogits, ldd, &done);
  if (st != DENSE_GEMM_OK || done) return st;
  int cus, xcds;
  st = device_topology(&cus, &xcds);
  if (st != DENSE_GEMM_OK) return st;
  RouteGradParams p = {};
  set_routing(p, logits, ldl, T, E, k, *routing);
  p.experts = (int32_t*)const_cast<void*>(experts);
  p.dweights = (const float*)dweights;
  p.dlogits = dlogits;
  p.ldd = ldd;
  if (fmt == DENSE_GEMM_F32) return run_grad<float>(p, stream);
  return fmt == DENSE_GEMM_BF16 ? run_grad<__bf16>(p, stream) : run_grad<_Float16>(p, stream);
}

}  // extern "C"
