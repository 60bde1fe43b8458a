// block_norm.hip -- C entry points of the block norm and its gradients (gemm_rs_layer.h).
#include "host.hpp"

#include "block_norm.hpp"

using namespace gemm_rs_layer;

namespace {

// Threads per workgroup: eight columns each, 1024 for wider rows.
int norm_threads(int n)
{
    return n <= 1024 ? 128 : n <= 2048 ? 256 : n <= 3072 ? 384 : n <= 4096 ? 512 : n <= 6144 ? 768 : 1024;
}

template <class T, class R, int MAXP>
int norm_forward_sized(const NormArgs& a, void* stream)
{
    auto go = [&](void (*k)(NormArgs), int threads) {
        return launch(k, dim3((unsigned)a.rows), threads, a, stream, "gemm_rs_block_norm");
    };
    switch (norm_threads(a.n)) {
    case 128: return go(norm_forward_kernel<T, R, 128, 1, MAXP>, 128);
    case 256: return go(norm_forward_kernel<T, R, 256, 1, MAXP>, 256);
    case 384: return go(norm_forward_kernel<T, R, 384, 1, MAXP>, 384);
    case 512: return go(norm_forward_kernel<T, R, 512, 1, MAXP>, 512);
    case 768: return go(norm_forward_kernel<T, R, 768, 1, MAXP>, 768);
    default:
        return a.n <= 8192 ? go(norm_forward_kernel<T, R, 1024, 1, MAXP>, 1024) : go(norm_forward_kernel<T, R, 1024, 4, MAXP>, 1024);
    }
}

template <class T, class R>
int norm_forward(const NormArgs& a, void* stream)
{
    return a.nparts == 1 ? norm_forward_sized<T, R, 1>(a, stream) : norm_forward_sized<T, R, 8>(a, stream);
}

template <class T, class R>
int norm_backward(const NormGradArgs& a, int grid, void* stream)
{
    const int threads = norm_threads(a.n);
    auto go = [&](void (*k)(NormGradArgs)) {
        return launch(k, dim3((unsigned)grid), threads, a, stream, "gemm_rs_block_norm_backward");
    };
    if (a.n > 16384) return go(norm_backward_wide_kernel<T, R, 4>);
    if (a.n > 8192) return go(norm_backward_wide_kernel<T, R, 2>);
    switch (threads) {
    case 128: return go(norm_backward_kernel<T, R, 128>);
    case 256: return go(norm_backward_kernel<T, R, 256>);
    case 384: return go(norm_backward_kernel<T, R, 384>);
    case 512: return go(norm_backward_kernel<T, R, 512>);
    case 768: return go(norm_backward_kernel<T, R, 768>);
    default: return go(norm_backward_kernel<T, R, 1024>);
    }
}

// f(T, R) for the configuration's types
template <class F>
int norm_types(const gemm_rs_norm_config& c, F f)
{
    const bool wide = c.residual_dtype == GEMM_RS_DTYPE_F32;
    switch (c.dtype) {
    case GEMM_RS_DTYPE_BF16: return wide ? f((__bf16)0, 0.f) : f((__bf16)0, (__bf16)0);
    case GEMM_RS_DTYPE_F16: return wide ? f((_Float16)0, 0.f) : f((_Float16)0, (_Float16)0);
    default: return f(0.f, 0.f);
    }
}

int norm_sums(const gemm_rs_norm_config& c)
{
    return (c.pre_norm ? 1 : 0) + (c.post_norm ? 1 : 0) + (c.gate == GEMM_RS_GATE_CHANNEL ? 1 : 0);
}


// Workgroups of the backward pass, each with one row of partial sums: as many as give
// every CU 16 waves (fewer leave a row's waits uncovered, more write more partial rows:
// 4096 rows of 8192 columns 180 / 135 / 146 us with 8 / 16 / 32 waves, of 4096 columns
// 84 / 82 / 87, of 2048 columns 34 / 32 / 40).  With more rows than CUs a workgroup takes
// two at least (1021 rows of 1000 columns 20 us with one, 16 with two, 16 with four; 512 rows
// of 4096 columns 21, 18, 20; 200 rows of 256 columns 7.7, 9.2).
int norm_groups(const gemm_rs_norm_config& c, int64_t rows)
{
    const int64_t most = kCus * (16 * 64 / norm_threads(c.width));
    if (rows > kCus && norm_sums(c) > 0) rows = rows < 2 * kCus ? kCus : ceil_div(rows, 2);
    return (int)(rows < most ? rows : most);
}

}  // namespace

extern "C" {

int gemm_rs_norm_validate(const gemm_rs_norm_config* c)
{
    if (!c || c->dtype < GEMM_RS_DTYPE_BF16 || c->dtype > GEMM_RS_DTYPE_F32 ||
        (c->residual_dtype != c->dtype && c->residual_dtype != GEMM_RS_DTYPE_F32) || c->gate < GEMM_RS_GATE_NONE ||
        c->gate > GEMM_RS_GATE_FULL || (c->post_norm != 0 && c->post_norm != 1) ||
        (c->pre_norm != 0 && c->pre_norm != 1) || !(c->eps >= 0.f) || !isfinite(c->eps) || !isfinite(c->block_scale) ||
        !isfinite(c->residual_scale))
        return GEMM_RS_ERR_INVALID_ARG;
    if (c->parts < 1 || c->parts > GEMM_RS_NORM_MAX_PARTS) return GEMM_RS_ERR_INVALID_ARG;
    if (c->width < 1 || c->width > GEMM_RS_NORM_MAX_WIDTH) return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
    return GEMM_RS_OK;
}

int gemm_rs_block_norm(const gemm_rs_norm_config* c, int64_t rows, const gemm_rs_norm_args* g, void* stream)
{
    int rc = gemm_rs_norm_validate(c);
    if (rc != GEMM_RS_OK) return rc;
    if (!g || rows < 0) return GEMM_RS_ERR_INVALID_ARG;
    if (rows > kMaxThreads / 1024) return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
    if (rows == 0) return GEMM_RS_OK;
    const size_t eb = elem_bytes(c->dtype), rb = elem_bytes(c->residual_dtype);
    Checker k;
    for (int i = 0; i < c->parts; ++i) k.need(g->parts[i], eb);
    k.stride(g->part_stride, c->width);
    k.maybe(g->residual, rb);
    if (g->residual) k.stride(g->residual_stride, c->width);
    if (c->post_norm) k.need(g->post_weight, eb);
    if (c->gate != GEMM_RS_GATE_NONE) k.need(g->gate, eb);
    if (c->gate == GEMM_RS_GATE_FULL) k.stride(g->gate_stride, c->width);
    k.need(g->h, rb);
    k.stride(g->h_stride, c->width);
    if (c->pre_norm) {
        k.need(g->pre_weight, eb);
        k.need(g->z, eb);
        k.stride(g->z_stride, c->width);
    }
    k.maybe(g->y, eb);
    if (g->y) k.stride(g->y_stride, c->width);
    k.maybe(g->rstd, 4);
    // in place: row by row, so only with the same rows
    if (g->h == g->residual && g->h_stride != g->residual_stride) k.fail(GEMM_RS_ERR_INVALID_ARG);
    if (g->y && g->y == g->parts[0] && (c->parts != 1 || g->y_stride != g->part_stride)) k.fail(GEMM_RS_ERR_INVALID_ARG);
    if (k.code != GEMM_RS_OK) return k.code;
    if ((rc = check_device()) != GEMM_RS_OK) return rc;
    NormArgs a = {};
    for (int i = 0; i < c->parts; ++i) a.parts[i] = g->parts[i];
    a.residual = g->residual;
    a.post_weight = c->post_norm ? g->post_weight : nullptr;
    a.gate = c->gate != GEMM_RS_GATE_NONE ? g->gate : nullptr;
    a.pre_weight = c->pre_norm ? g->pre_weight : nullptr;
    a.h = g->h;
    a.z = g->z;
    a.y = g->y;
    a.rstd = g->rstd;
    a.part_stride = g->part_stride;
    a.residual_stride = g->residual_stride;
    a.gate_stride = g->gate_stride;
    a.h_stride = g->h_stride;
    a.z_stride = g->z_stride;
    a.y_stride = g->y_stride;
    a.rows = rows;
    a.eps = c->eps;
    a.block_scale = c->block_scale;
    a.residual_scale = c->residual_scale;
    a.n = c->width;
    a.nparts = c->parts;
    a.gate_kind = c->gate;
    return norm_types(*c, [&](auto t, auto r) { return norm_forward<decltype(t), decltype(r)>(a, stream); });
}

size_t gemm_rs_block_norm_workspace(const gemm_rs_norm_config* c, int64_t rows)
{
    if (gemm_rs_norm_validate(c) != GEMM_RS_OK || rows <= 0) return 0;
    return (size_t)norm_groups(*c, rows) * norm_sums(*c) * c->width * sizeof(float);
}

int gemm_rs_block_norm_backward(const gemm_rs_norm_config* c, int64_t rows, const gemm_rs_norm_grad_args* g,
                                void* workspace, size_t workspace_bytes, void* stream)
{
    int rc = gemm_rs_norm_validate(c);
    if (rc != GEMM_RS_OK) return rc;
    if (!g || rows < 0) return GEMM_RS_ERR_INVALID_ARG;
    if (rows > kMaxThreads / 1024) return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
    const size_t eb = elem_bytes(c->dtype), rb = elem_bytes(c->residual_dtype);
    const bool channel = c->gate == GEMM_RS_GATE_CHANNEL;
    Checker k;
    if (c->pre_norm) k.need(g->dpre_weight, 4);
    if (c->post_norm) k.need(g->dpost_weight, 4);
    if (channel) k.need(g->dgate, 4);
    if (rows > 0) {
        if (c->pre_norm) {
            k.need(g->dz, eb);
            k.stride(g->dz_stride, c->width);
            k.need(g->h, rb);
            k.stride(g->h_stride, c->width);
            k.need(g->pre_weight, eb);
        }
        k.maybe(g->dh, rb);
        if (g->dh) k.stride(g->dh_stride, c->width);
        if (c->post_norm || c->gate != GEMM_RS_GATE_NONE) {
            k.need(g->y, eb);
            k.stride(g->y_stride, c->width);
        }
        if (c->post_norm) k.need(g->post_weight, eb);
        if (c->post_norm || c->pre_norm) k.need(g->rstd, 4);
        if (c->gate != GEMM_RS_GATE_NONE) k.need(g->gate, eb);
        if (c->gate == GEMM_RS_GATE_TOKEN || c->gate == GEMM_RS_GATE_FULL) k.need(g->dgate, eb);
        if (c->gate == GEMM_RS_GATE_FULL) {
            k.stride(g->gate_stride, c->width);
            k.stride(g->dgate_stride, c->width);
        }
        k.maybe(g->dresidual, rb);
        if (g->dresidual) k.stride(g->dresidual_stride, c->width);
        k.need(g->dy, eb);
        k.stride(g->dy_stride, c->width);
        if (g->dresidual && g->dresidual == g->dh && g->dresidual_stride != g->dh_stride) k.fail(GEMM_RS_ERR_INVALID_ARG);
        if (c->pre_norm && g->dy == g->dz && g->dy_stride != g->dz_stride) k.fail(GEMM_RS_ERR_INVALID_ARG);
        const size_t ws = gemm_rs_block_norm_workspace(c, rows);
        if (ws > 0) {
            if (workspace_bytes < ws || !workspace) k.fail(GEMM_RS_ERR_SCRATCH);
            else k.need(workspace, 16);
        }
    }
    if (k.code != GEMM_RS_OK) return k.code;
    if ((rc = check_device()) != GEMM_RS_OK) return rc;
    const int grid = norm_groups(*c, rows), sums = norm_sums(*c);
    if (rows > 0) {
        NormGradArgs a = {};
        a.dz = g->dz;
        a.dh = g->dh;
        a.h = g->h;
        a.y = g->y;
        a.rstd = g->rstd;
        a.post_weight = c->post_norm ? g->post_weight : nullptr;
        a.gate = c->gate != GEMM_RS_GATE_NONE ? g->gate : nullptr;
        a.pre_weight = c->pre_norm ? g->pre_weight : nullptr;
        a.dresidual = g->dresidual;
        a.dy = g->dy;
        a.dgate = g->dgate;
        a.partial = static_cast<float*>(workspace);
        a.dz_stride = g->dz_stride;
        a.dh_stride = g->dh_stride;
        a.h_stride = g->h_stride;
        a.y_stride = g->y_stride;
        a.gate_stride = g->gate_stride;
        a.dresidual_stride = g->dresidual_stride;
        a.dy_stride = g->dy_stride;
        a.dgate_stride = g->dgate_stride;
        a.rows = rows;
        a.block_scale = c->block_scale;
        a.residual_scale = c->residual_scale;
        a.n = c->width;
        a.gate_kind = c->gate;
        a.sums = sums;
        rc = norm_types(*c, [&](auto t, auto r) { return norm_backward<decltype(t), decltype(r)>(a, grid, stream); });
        if (rc != GEMM_RS_OK) return rc;
    }
    if (sums == 0) return GEMM_RS_OK;
    NormSumsArgs s = {};
    s.partial = static_cast<const float*>(workspace);
    s.n = c->width;
    s.sums = sums;
    s.groups = grid;
    int i = 0;
    if (c->pre_norm) s.out[i++] = g->dpre_weight;
    if (c->post_norm) s.out[i++] = g->dpost_weight;
    if (channel) s.out[i++] = static_cast<float*>(g->dgate);
    const dim3 blocks((unsigned)ceil_div(c->width, kSumCols), (unsigned)sums);
    // a batch of loads per thread
    if (grid <= 8 * 16)
        return launch(norm_sums_kernel<16>, blocks, kSumCols * 16, s, stream, "gemm_rs_block_norm_backward");
    return launch(norm_sums_kernel<32>, blocks, kSumCols * 32, s, stream, "gemm_rs_block_norm_backward");
}

}  // extern "C"
