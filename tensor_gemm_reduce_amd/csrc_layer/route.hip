// route.hip -- C entry points of the router, its plan and the rows' combination
// (gemm_rs_experts.h).
#include "host.hpp"

#include "gemm_rs_experts.h"
#include "route.hpp"

using namespace gemm_rs_layer;

namespace {

// Tokens per workgroup: all of a few, for which one launch is faster than three (256 experts in groups, 16 / 64 tokens: 16 / 35 us
// so, 1024 in three launches 24); else one for each of its waves, or up to
// kRouteTokens while two workgroups for every CU are left.  At most as many as its threads have choices for.
constexpr int kRouteAlone = 32;
int route_tokens(int64_t T, int k, int threads)
{
    int64_t n = T <= kRouteAlone ? kRouteAlone : threads / 64;
    while (n < kRouteTokens && T > n * 2 * kCus) n *= 2;
    const int most = threads / k;
    return n < most ? (int)n : most;
}

int route_values(int E) { return E <= 64 ? 1 : E <= 128 ? 2 : E <= 256 ? 4 : E <= 512 ? 8 : 16; }

// Choices per workgroup of the router's call; of gemm_rs_expert_plan's, at least as many.
int route_chunk(int64_t T, int E, int k) { return route_tokens(T, k, route_threads(route_values(E))) * k; }

size_t plan_bytes(int64_t ids, int E, int chunk)
{
    const int64_t chunks = ceil_div(ids, chunk);
    return chunks > 1 ? (size_t)((chunks + 1) * E) * sizeof(int32_t) : 0;
}

bool plan_sizes(int64_t T, int32_t E, int32_t k)
{
    return T >= 0 && E >= 1 && E <= GEMM_RS_ROUTE_MAX_EXPERTS && k >= 1 && k <= GEMM_RS_ROUTE_MAX_CHOICES;
}

PlanArgs plan_args(int64_t T, int E, int k, int chunk, const int32_t* experts, const gemm_rs_expert_plan_args& p, void* workspace)
{
    PlanArgs a = {};
    a.experts = experts;
    a.offsets = p.offsets;
    a.tokens = p.tokens;
    a.slots = p.slots;
    a.ids = T * k;
    a.E = E;
    a.k = k;
    a.chunk = chunk;
    a.chunks = (int)ceil_div(a.ids, chunk);
    a.totals = static_cast<int32_t*>(workspace);
    a.hist = a.totals + E;
    return a;
}

void plan_check(Checker& c, int64_t T, const gemm_rs_expert_plan_args* p, const void* experts, size_t need, const void* workspace,
                size_t bytes)
{
    if (!p) return c.fail(GEMM_RS_ERR_INVALID_ARG);
    c.need(p->offsets, 4);
    if (T > 0) {
        c.need(experts, 4);
        c.need(p->tokens, 4);
        c.need(p->slots, 4);
    }
    if (need > 0) {
        if (!workspace || bytes < need) c.fail(GEMM_RS_ERR_SCRATCH);
        else c.need(workspace, 4);
    }
}

// What follows the counts of more than one workgroup.
int plan_rest(const PlanArgs& a, void* stream)
{
    const int rc = launch(plan_scan_kernel, dim3((unsigned)a.E), kScanThreads, a, stream, "plan_scan_kernel");
    return rc != GEMM_RS_OK ? rc
                            : launch(plan_place_kernel, dim3((unsigned)a.chunks), (int)ceil_div(a.chunk, 64) * 64, a, stream,
                                     "plan_place_kernel");
}

template <int SEG, int NV>
int route_launch(const RouteArgs& a, bool wide, void* stream)
{
    const dim3 grid((unsigned)ceil_div(a.T, a.tokens));
    return launch(wide ? route_kernel<SEG, NV, true> : route_kernel<SEG, NV, false>, grid, route_threads(NV), a, stream,
                  "gemm_rs_route");
}

template <int SEG, int NV>
int grad_launch(const RouteGradArgs& a, void* stream)
{
    return launch(route_backward_kernel<SEG, NV>, dim3((unsigned)ceil_div(a.T, 4 * (64 / SEG))), 256, a, stream,
                  "gemm_rs_route_backward");
}

// The smallest segment of lanes and number of values that hold the experts; f<SEG, NV>().
#define ROUTE_FORMS(E, whole, f, ...)                              \
    (E) <= 8 && !(whole)    ? f<8, 1>(__VA_ARGS__)                 \
    : (E) <= 16 && !(whole) ? f<16, 1>(__VA_ARGS__)                \
    : (E) <= 32 && !(whole) ? f<32, 1>(__VA_ARGS__)                \
    : (E) <= 64             ? f<64, 1>(__VA_ARGS__)                \
    : (E) <= 128            ? f<64, 2>(__VA_ARGS__)                \
    : (E) <= 256            ? f<64, 4>(__VA_ARGS__)                \
    : (E) <= 512            ? f<64, 8>(__VA_ARGS__)                \
                            : f<64, 16>(__VA_ARGS__)

bool combine_ok(int32_t dtype, int64_t T, int64_t R, int64_t N, int32_t k)
{
    return dtype >= GEMM_RS_DTYPE_BF16 && dtype <= GEMM_RS_DTYPE_F32 && T >= 0 && R >= 0 && N >= 1 && k >= 1;
}

bool combine_fits(int64_t T, int64_t R, int64_t N, int32_t k)
{
    return T <= kMaxThreads / kCombineThreads && R < kMaxRows && N <= (1 << 22) && k <= GEMM_RS_ROUTE_MAX_CHOICES;
}

}  // namespace

extern "C" {

int gemm_rs_route_validate(const gemm_rs_route_config* c)
{
    if (!c || c->dtype < GEMM_RS_DTYPE_BF16 || c->dtype > GEMM_RS_DTYPE_F32 || c->E < 1 || c->k < 1 ||
        (c->score != GEMM_RS_SCORE_SOFTMAX && c->score != GEMM_RS_SCORE_SIGMOID) ||
        (c->renormalise != 0 && c->renormalise != 1) || c->groups < 1 || c->keep_groups < 1 ||
        c->keep_groups > c->groups || !isfinite(c->scale) || c->k > c->E || c->E % c->groups != 0)
        return GEMM_RS_ERR_INVALID_ARG;
    if (c->E > GEMM_RS_ROUTE_MAX_EXPERTS || c->k > GEMM_RS_ROUTE_MAX_CHOICES || c->groups > 64)
        return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
    return GEMM_RS_OK;
}

size_t gemm_rs_expert_plan_workspace(int64_t T, int32_t E, int32_t k)
{
    return plan_sizes(T, E, k) && T < kMaxRows && T * k < kMaxRows ? plan_bytes(T * k, E, route_chunk(T, E, k)) : 0;
}

int gemm_rs_route(const gemm_rs_route_config* c, int64_t T, const void* logits, int64_t logits_stride, const float* bias,
                  float* weights, int32_t* experts, const gemm_rs_expert_plan_args* plan, void* workspace, size_t workspace_bytes,
                  void* stream)
{
    int rc = gemm_rs_route_validate(c);
    if (rc != GEMM_RS_OK) return rc;
    if (T < 0) return GEMM_RS_ERR_INVALID_ARG;
    if (T >= kMaxRows || T * c->k >= kMaxRows) return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
    const int tokens = route_chunk(T, c->E, c->k) / c->k;  // of a workgroup
    if (ceil_div(T, tokens) * route_threads(route_values(c->E)) > kMaxThreads) return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
    Checker k;
    plan_check(k, T, plan, experts, gemm_rs_expert_plan_workspace(T, c->E, c->k), workspace, workspace_bytes);
    if (T > 0) {
        k.need(logits, elem_bytes(c->dtype));
        k.stride(logits_stride, c->E);
        k.need(weights, 4);
    }
    k.maybe(bias, 4);
    if (k.code != GEMM_RS_OK) return k.code;
    if ((rc = check_device()) != GEMM_RS_OK) return rc;
    RouteArgs a = {};
    a.logits = logits;
    a.bias = bias;
    a.weights = weights;
    a.experts = experts;
    a.T = T;
    a.stride = logits_stride;
    a.dtype = c->dtype;
    a.E = c->E;
    a.k = c->k;
    a.sigmoid = c->score == GEMM_RS_SCORE_SIGMOID;
    a.renormalise = c->renormalise;
    a.groups = c->groups;
    a.keep = c->keep_groups;
    a.scale = c->scale;
    a.tokens = tokens;
    a.plan = plan_args(T, c->E, c->k, a.tokens * c->k, experts, *plan, workspace);
    if (T == 0)  // offsets of nothing
        return launch(plan_count_kernel, dim3(1), kPlanIds, [&] { a.plan.chunks = 1; return a.plan; }(), stream, "gemm_rs_route");
    const bool wide = bias || c->groups > 1;
    rc = ROUTE_FORMS(c->E, c->groups > 1, route_launch, a, wide, stream);
    return rc != GEMM_RS_OK || a.plan.chunks == 1 ? rc : plan_rest(a.plan, stream);
}

int gemm_rs_expert_plan(int64_t T, int32_t E, int32_t k, const int32_t* experts, const gemm_rs_expert_plan_args* plan, void* workspace,
                 size_t workspace_bytes, void* stream)
{
    if (T < 0 || E < 1 || k < 1) return GEMM_RS_ERR_INVALID_ARG;
    if (!plan_sizes(T, E, k) || T >= kMaxRows || T * k >= kMaxRows) return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
    Checker c;
    plan_check(c, T, plan, experts, gemm_rs_expert_plan_workspace(T, E, k), workspace, workspace_bytes);
    if (c.code != GEMM_RS_OK) return c.code;
    int rc = check_device();
    if (rc != GEMM_RS_OK) return rc;
    PlanArgs a = plan_args(T, E, k, kPlanIds, experts, *plan, workspace);
    if (a.chunks == 0) a.chunks = 1;
    rc = launch(plan_count_kernel, dim3((unsigned)a.chunks), kPlanIds, a, stream, "gemm_rs_expert_plan");
    return rc != GEMM_RS_OK || a.chunks == 1 ? rc : plan_rest(a, stream);
}

int gemm_rs_route_backward(const gemm_rs_route_config* c, int64_t T, const void* logits, int64_t logits_stride,
                           const int32_t* experts, const float* dweights, void* dlogits, int64_t dlogits_stride, void* stream)
{
    int rc = gemm_rs_route_validate(c);
    if (rc != GEMM_RS_OK) return rc;
    if (T < 0) return GEMM_RS_ERR_INVALID_ARG;
    if (T >= kMaxThreads / 64 - 8) return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return GEMM_RS_OK;
    Checker k;
    k.need(logits, elem_bytes(c->dtype));
    k.stride(logits_stride, c->E);
    k.need(experts, 4);
    k.need(dweights, 4);
    k.need(dlogits, elem_bytes(c->dtype));
    k.stride(dlogits_stride, c->E);
    if (k.code != GEMM_RS_OK) return k.code;
    if ((rc = check_device()) != GEMM_RS_OK) return rc;
    RouteGradArgs a = {};
    a.logits = logits;
    a.experts = experts;
    a.dweights = dweights;
    a.dlogits = dlogits;
    a.T = T;
    a.stride = logits_stride;
    a.dstride = dlogits_stride;
    a.dtype = c->dtype;
    a.E = c->E;
    a.k = c->k;
    a.sigmoid = c->score == GEMM_RS_SCORE_SIGMOID;
    a.renormalise = c->renormalise;
    a.scale = c->scale;
    return ROUTE_FORMS(c->E, false, grad_launch, a, stream);
}

int gemm_rs_combine(int32_t dtype, int64_t T, int64_t R, int64_t N, int32_t k, const void* y, int64_t y_stride,
                    const int32_t* slots, const float* weights, void* out, int64_t out_stride, void* stream)
{
    if (!combine_ok(dtype, T, R, N, k)) return GEMM_RS_ERR_INVALID_ARG;
    if (!combine_fits(T, R, N, k)) return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return GEMM_RS_OK;
    Checker c;
    if (R > 0) {
        c.need(y, elem_bytes(dtype));
        c.stride(y_stride, N);
    }
    c.need(slots, 4);
    c.maybe(weights, 4);
    c.need(out, elem_bytes(dtype));
    c.stride(out_stride, N);
    if (c.code != GEMM_RS_OK) return c.code;
    const int rc = check_device();
    if (rc != GEMM_RS_OK) return rc;
    CombineArgs a = {};
    a.y = y;
    a.slots = slots;
    a.weights = weights;
    a.out = out;
    a.T = T;
    a.R = R;
    a.y_stride = y_stride;
    a.out_stride = out_stride;
    a.N = (int)N;
    a.k = k;
    void (*kern)(CombineArgs) = dtype == GEMM_RS_DTYPE_BF16  ? combine_kernel<__bf16>
                                : dtype == GEMM_RS_DTYPE_F16 ? combine_kernel<_Float16>
                                                             : combine_kernel<float>;
    return launch(kern, dim3((unsigned)T, (unsigned)ceil_div(N, kCombineThreads * 8)), kCombineThreads, a, stream,
                  "gemm_rs_combine");
}

int gemm_rs_combine_backward(int32_t dtype, int64_t T, int64_t R, int64_t N, int32_t k, const void* dout,
                             int64_t dout_stride, const void* y, int64_t y_stride, const int32_t* slots,
                             const float* weights, void* dy, int64_t dy_stride, float* dweights, void* stream)
{
    if (!combine_ok(dtype, T, R, N, k)) return GEMM_RS_ERR_INVALID_ARG;
    if (!combine_fits(T, R, N, k)) return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
    if (R > 0 && (y != nullptr) != (dweights != nullptr)) return GEMM_RS_ERR_INVALID_ARG;
    if (T == 0) return GEMM_RS_OK;
    Checker c;
    c.need(dout, elem_bytes(dtype));
    c.stride(dout_stride, N);
    c.need(slots, 4);
    c.maybe(weights, 4);
    c.maybe(dweights, 4);
    if (R > 0) {
        c.need(dy, elem_bytes(dtype));
        c.stride(dy_stride, N);
        c.maybe(y, elem_bytes(dtype));
        if (y) c.stride(y_stride, N);
    }
    if (c.code != GEMM_RS_OK) return c.code;
    const int rc = check_device();
    if (rc != GEMM_RS_OK) return rc;
    CombineArgs a = {};
    a.dout = dout;
    a.y = y;
    a.slots = slots;
    a.weights = weights;
    a.dy = dy;
    a.dweights = dweights;
    a.T = T;
    a.R = R;
    a.dout_stride = dout_stride;
    a.y_stride = y_stride;
    a.dy_stride = dy_stride;
    a.N = (int)N;
    a.k = k;
    void (*kern)(CombineArgs) = dtype == GEMM_RS_DTYPE_BF16  ? combine_backward_kernel<__bf16>
                                : dtype == GEMM_RS_DTYPE_F16 ? combine_backward_kernel<_Float16>
                                                             : combine_backward_kernel<float>;
    return launch(kern, dim3((unsigned)T), kCombineThreads, a, stream, "gemm_rs_combine_backward");
}

}  // extern "C"
