// checkpoint.hip -- C entry points of the 8-bit checkpoint and the weight gradient
// (gemm_rs_layer.h), and the error messages.
#include "host.hpp"

#include "checkpoint.hpp"

using namespace gemm_rs_layer;

namespace {

// dy in whole 4-byte words (buffer loads check bounds by the word), and 64 of its rows
// within a buffer resource's 2^31 bytes.
bool wgrad_fast(const gemm_rs_wgrad_args& g)
{
    return g.M > 0 && aligned(g.dy, 4) && g.dy_stride % 2 == 0 && g.N % 2 == 0 && g.dy_stride < (1 << 23);
}

// A share of a cut tile is at least this many steps of 64 tokens: shorter ones cost more
// in starts and in joining than they spread (us with 6 / 8 / 12 steps: 2048 x 1024 x 1024
// 19.9 / 19.8 / 24.3, 4096 x 512 x 512 20.2 / 19.5 / 23.4, 16384 x 256 x 128 21.8 / 19.3 /
// 21.7, 1000 x 300 x 200 15.0 / 14.0 / 19.2).
constexpr int kWgMinSteps = 8;

// The number of shares that the tiles of the last round are best cut into, or 0 if they are
// better left whole: by what a step costs there (small tiles: 0.8 us, 1.3 with two
// workgroups per CU; big ones 1.1, since fewer of them run at a higher clock), and by
// starting the join and moving a piece for every tile and share.  Measured, us, BF16
// results, cut / whole: 1000 x 8192 x 1100 39 / 40, 2000 x 6000 x 1500 61 / 69,
// 2048 x 8192 x 3584 172 / 160, 3000 x 8192 x 3584 198 / 180, 4096 x 1280 x 8192 107 / 107,
// 4096 x 8192 x 1024 85 / 105, 6000 x 4000 x 2000 112 / 146, 32768 x 8192 x 3584 1697 / 1726;
// with 512 / 256 shares: 16384 x 700 x 300 40 / 34, 3000 x 1500 x 700 33 / 28,
// 16384 x 512 x 512 30 / 27.
int wgrad_shares(bool big, int64_t rest, int64_t steps)
{
    auto ns = [&](int64_t groups) { return big ? 1100 : groups <= kCus ? 800 : 1300; };
    int64_t best = 0, cost = steps * ns(rest);
    for (int64_t most = big ? kCus : 2 * kCus; most >= kCus / 2; most /= 2) {
        int64_t shares = rest * steps / kWgMinSteps;
        shares = shares < most ? shares : most;
        if (shares <= rest) continue;
        const int64_t c = rest * steps / shares * ns(shares) + 1500 + (rest + shares) * (big ? 62 : 35);
        if (c < cost) {
            cost = c;
            best = shares;
        }
    }
    return (int)best;
}

// Neighbouring shares of one XCD (each reads the tiles' rows of its own tokens) or of all:
// short shares are mostly better the first way (us, first / second: 2048 x 1024 x 1024,
// 8 steps, 19.8 / 23.4; 8000 x 2300 x 2300, 40 steps, 113 / 118; but 3000 x 1500 x 700,
// 13 steps, 28.8 / 27.1, and 12300 x 1030 x 1000, 15 steps, 61.5 / 58.5), long ones the
// second (10000 x 2000 x 3500, 69 steps, 167 / 158; 16384 x 3000 x 2500, 120 steps, 313 / 261).
constexpr int kWgDealtSteps = 48;

// The 256 x 256 tile reads and turns its operands half as often for the same outputs, but
// starts and ends slower: for products of at least kWgBigSteps steps, and kWgBigWork of
// its steps per CU.  Where the two meet depends on how the tiles fill the CUs and on the
// bytes of a result; the thresholds are those from which the big tile is at most some 8%
// behind with either result.  Measured, us (256 / 128), FP32 results added to a running sum:
// 2048 x 8192 x 3584 194 / 187 (32 steps), 2560 x 8192 x 3584 228 / 228 (40),
// 3008 x 8192 x 3584 257 / 265 (47), 3008 x 8192 x 1024 77 / 74, 3008 x 2048 x 3584 78 / 73,
// 4096 x 7168 x 1280 112 / 112 (64), 10000 x 8192 x 3584 592 / 754 (157); BF16 results:
// 2560 x 8192 x 1024 72 / 61 (40), 3008 x 8192 x 1024 71 / 69, 4096 x 1280 x 8192 105 / 117,
// 32768 x 8192 x 3584 1700 / 2556 (512); 8192 x 1024 x 1024 46 / 40 (8 a CU), 5000 x 1024 x
// 2048 47 / 45 (10), 16384 x 2048 x 512 58 / 61 (16), 3500 x 3000 x 1500 66 / 86 (16).
// What that gives away: with BF16 results, tiles that leave few CUs idle in their last round
// are faster big from 12 or 16 steps on (1024 x 8192 x 2048, 256 tiles, 43 / 53; 2560 x 8192 x
// 2048 85 / 116; 2048 x 6144 x 2048, 192 tiles, 62 / 72; 2048 x 8192 x 3584, 448, 130 / 161).
constexpr int kWgBigSteps = 44, kWgBigWork = 12;

WgradPlan wgrad_plan(const gemm_rs_wgrad_args& g, int& big)
{
    auto tiles = [&](int t) { return ceil_div(g.N, t) * ceil_div(g.K, t); };
    const int64_t steps = ceil_div(g.M, kWgRows);
    big = steps >= kWgBigSteps && tiles(256) * steps >= kWgBigWork * kCus;
    const int edge = big ? 256 : 128, slots = big ? kCus : 2 * kCus;
    WgradPlan p = {};
    p.tiles_n = (int)ceil_div(g.N, edge);
    p.tiles_k = (int)ceil_div(g.K, edge);
    p.steps = steps;
    const int64_t all = (int64_t)p.tiles_n * p.tiles_k, rest = all % slots;
    p.full = (int)(all - rest);
    const int shares = wgrad_shares(big, rest, steps);
    if (shares == 0) p.full = (int)all;
    p.shares = shares;
    p.grid = (int)(p.full >= slots || shares >= slots ? slots : p.full > shares ? p.full : shares);
    p.dealt = shares > 0 && (shares < p.grid || rest * p.steps / shares >= kWgDealtSteps);
    return p;
}

int64_t wgrad_cut(const WgradPlan& p) { return (int64_t)p.tiles_n * p.tiles_k - p.full; }

// Waves per workgroup of the join: by the pieces a tile has (wgrad_join_kernel).
int wgrad_join_waves(const WgradPlan& p) { return p.shares > 6 * wgrad_cut(p) ? 4 : 1; }

template <class A, class B>
int launch2(void (*kernel)(A, B), dim3 grid, int threads, int lds, const A& a, const B& b, void* stream)
{
    void* p[] = {const_cast<A*>(&a), const_cast<B*>(&b)};
    const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, dim3(threads), p, lds,
                                         static_cast<hipStream_t>(stream));
    return e == hipSuccess ? GEMM_RS_OK : hip_fail(e, "gemm_rs_ckpt_wgrad");
}

template <class T, int WN, int WK>
int wgrad_run(const WgradArgs& a, const WgradPlan& p, int device, void* stream)
{
    constexpr int kLds = WgradTile<WN, WK>::kLds;
    static std::atomic<bool> allowed[kMaxDevices];  // the LDS of one workgroup, once per device
    if (!allowed[device].load(std::memory_order_relaxed)) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(wgrad_kernel<T, WN, WK>),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
        if (e != hipSuccess) return hip_fail(e, "hipFuncSetAttribute");
        allowed[device].store(true, std::memory_order_relaxed);
    }
    int rc = launch2(wgrad_kernel<T, WN, WK>, dim3((unsigned)p.grid), kWgThreads, kLds, a, p, stream);
    if (rc != GEMM_RS_OK || p.shares == 0) return rc;
    const dim3 grid((unsigned)wgrad_cut(p), 4 * WN);
    return wgrad_join_waves(p) == 4 ? launch2(wgrad_join_kernel<T, WN, WK, 4>, grid, 256, 0, a, p, stream)
                                    : launch2(wgrad_join_kernel<T, WN, WK, 1>, grid, 64, 0, a, p, stream);
}

}  // namespace

extern "C" {

const char* gemm_rs_layer_strerror(int code)
{
    switch (code) {
    case GEMM_RS_OK: return "ok";
    case GEMM_RS_ERR_INVALID_ARG: return "invalid argument";
    case GEMM_RS_ERR_UNSUPPORTED_SHAPE: return "unsupported shape";
    case GEMM_RS_ERR_MISALIGNED: return "misaligned buffer";
    case GEMM_RS_ERR_NO_DEVICE: return "the current device is not a gfx950";
    case GEMM_RS_ERR_HIP: return g_hip_msg[0] ? g_hip_msg : "HIP error";
    case GEMM_RS_ERR_SCRATCH: return "workspace missing or too small";
    default: return "unknown error";
    }
}

static int ckpt_check(int32_t dtype, int64_t M, int64_t K, const void* x, int64_t stride, const void* q,
                      const void* exps)
{
    if (dtype < GEMM_RS_DTYPE_BF16 || dtype > GEMM_RS_DTYPE_F32 || M < 0 || K < 1) return GEMM_RS_ERR_INVALID_ARG;
    if (M >= kMaxRows || K > (1 << 22) || M * (ceil_div(K, 32) * 2) > kMaxThreads - kCkptThreads)
        return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
    if (M == 0) return GEMM_RS_OK;
    Checker k;
    k.need(x, elem_bytes(dtype));
    k.stride(stride, K);
    k.need(q, 16);
    k.need(exps, 1);
    return k.code;
}

static CkptArgs ckpt_args(int64_t M, int64_t K, int64_t stride)
{
    CkptArgs a = {};
    a.rows = M;
    a.stride = stride;
    a.K = (int)K;
    a.chunks = (int)ceil_div(K, 32) * 2;
    return a;
}

int gemm_rs_ckpt_pack(int32_t dtype, int64_t M, int64_t K, const void* x, int64_t x_stride, void* q, void* exps,
                      void* stream)
{
    int rc = ckpt_check(dtype, M, K, x, x_stride, q, exps);
    if (rc != GEMM_RS_OK || M == 0) return rc;
    if ((rc = check_device()) != GEMM_RS_OK) return rc;
    CkptArgs a = ckpt_args(M, K, x_stride);
    a.x = x;
    a.q = static_cast<int8_t*>(q);
    a.e = static_cast<int8_t*>(exps);
    void (*kern)(CkptArgs) = dtype == GEMM_RS_DTYPE_BF16  ? ckpt_pack_kernel<__bf16>
                             : dtype == GEMM_RS_DTYPE_F16 ? ckpt_pack_kernel<_Float16>
                                                          : ckpt_pack_kernel<float>;
    return launch(kern, dim3((unsigned)ceil_div(M * a.chunks, kCkptThreads)), kCkptThreads, a, stream, "gemm_rs_ckpt_pack");
}

int gemm_rs_ckpt_unpack(int32_t dtype, int64_t M, int64_t K, const void* q, const void* exps, void* x,
                        int64_t x_stride, void* stream)
{
    int rc = ckpt_check(dtype, M, K, x, x_stride, q, exps);
    if (rc != GEMM_RS_OK || M == 0) return rc;
    if ((rc = check_device()) != GEMM_RS_OK) return rc;
    CkptArgs a = ckpt_args(M, K, x_stride);
    a.out = x;
    a.q = static_cast<int8_t*>(const_cast<void*>(q));
    a.e = static_cast<int8_t*>(const_cast<void*>(exps));
    void (*kern)(CkptArgs) = dtype == GEMM_RS_DTYPE_BF16  ? ckpt_unpack_kernel<__bf16>
                             : dtype == GEMM_RS_DTYPE_F16 ? ckpt_unpack_kernel<_Float16>
                                                          : ckpt_unpack_kernel<float>;
    return launch(kern, dim3((unsigned)ceil_div(M * a.chunks, kCkptThreads)), kCkptThreads, a, stream,
                  "gemm_rs_ckpt_unpack");
}

static int wgrad_check(const gemm_rs_wgrad_args* g)
{
    if (!g || (g->dtype != GEMM_RS_DTYPE_BF16 && g->dtype != GEMM_RS_DTYPE_F16) ||
        (g->out_dtype != g->dtype && g->out_dtype != GEMM_RS_DTYPE_F32) || g->M < 0 || g->N < 1 || g->K < 1)
        return GEMM_RS_ERR_INVALID_ARG;
    if (g->M >= kMaxRows || g->N > (1 << 22) || g->K > (1 << 22)) return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
    return GEMM_RS_OK;
}

int gemm_rs_ckpt_wgrad_plan(const gemm_rs_wgrad_args* g, gemm_rs_wgrad_info* info)
{
    const int rc = wgrad_check(g);
    if (rc != GEMM_RS_OK) return rc;
    if (!info) return GEMM_RS_ERR_INVALID_ARG;
    if (!wgrad_fast(*g)) {
        const int64_t tiles = ceil_div(g->N, kWgTile) * ceil_div(g->K, kWgTile);
        *info = {0, kWgTile, (int32_t)tiles, 0, 0, (int32_t)tiles, 0, 0};
        return GEMM_RS_OK;
    }
    int big;
    const WgradPlan p = wgrad_plan(*g, big);
    *info = {1, big ? 256 : 128, p.full, (int32_t)wgrad_cut(p), p.shares, p.grid, p.dealt, p.shares ? wgrad_join_waves(p) : 0};
    return GEMM_RS_OK;
}

size_t gemm_rs_ckpt_wgrad_workspace(const gemm_rs_wgrad_args* g)
{
    if (wgrad_check(g) != GEMM_RS_OK || !wgrad_fast(*g)) return 0;
    int big;
    const WgradPlan p = wgrad_plan(*g, big);
    if (p.shares == 0) return 0;
    return (size_t)(p.shares + wgrad_cut(p) - 1) * (big ? WgradTile<4, 4>::kFloats : WgradTile<2, 2>::kFloats) * sizeof(float);
}

int gemm_rs_ckpt_wgrad(const gemm_rs_wgrad_args* g, void* workspace, size_t workspace_bytes, void* stream)
{
    int rc = wgrad_check(g);
    if (rc != GEMM_RS_OK) return rc;
    Checker k;
    if (g->M > 0) {
        k.need(g->dy, 2);
        k.stride(g->dy_stride, g->N);
        k.need(g->q, 16);
        k.need(g->exps, 1);
    }
    k.maybe(g->add, 4);
    if (g->add) k.stride(g->add_stride, g->K);
    k.need(g->dw, elem_bytes(g->out_dtype));
    k.stride(g->dw_stride, g->K);
    if (g->add && g->add == g->dw && (g->out_dtype != GEMM_RS_DTYPE_F32 || g->add_stride != g->dw_stride))
        k.fail(GEMM_RS_ERR_INVALID_ARG);
    const size_t ws = gemm_rs_ckpt_wgrad_workspace(g);
    if (ws > 0) {
        if (workspace_bytes < ws || !workspace) k.fail(GEMM_RS_ERR_SCRATCH);
        else k.need(workspace, 16);
    }
    if (k.code != GEMM_RS_OK) return k.code;
    int device = 0;
    if ((rc = check_device(&device)) != GEMM_RS_OK) return rc;
    WgradArgs a = {};
    a.dy = g->dy;
    a.q = static_cast<const int8_t*>(g->q);
    a.e = static_cast<const int8_t*>(g->exps);
    a.add = g->add;
    a.dw = g->dw;
    a.M = g->M;
    a.dy_stride = g->dy_stride;
    a.add_stride = g->add_stride;
    a.dw_stride = g->dw_stride;
    a.N = (int)g->N;
    a.K = (int)g->K;
    a.Kp = (int)ceil_div(g->K, 32) * 32;
    a.out_f32 = g->out_dtype == GEMM_RS_DTYPE_F32;
    const bool bf16 = g->dtype == GEMM_RS_DTYPE_BF16;
    if (!wgrad_fast(*g)) {
        const dim3 grid((unsigned)ceil_div(g->K, kWgTile), (unsigned)ceil_div(g->N, kWgTile));
        return launch(bf16 ? wgrad_any_kernel<__bf16> : wgrad_any_kernel<_Float16>, grid, kWgThreads, a, stream,
                      "gemm_rs_ckpt_wgrad");
    }
    int big;
    WgradPlan p = wgrad_plan(*g, big);
    p.pieces = static_cast<float*>(workspace);
    if (bf16) return big ? wgrad_run<__bf16, 4, 4>(a, p, device, stream) : wgrad_run<__bf16, 2, 2>(a, p, device, stream);
    return big ? wgrad_run<_Float16, 4, 4>(a, p, device, stream) : wgrad_run<_Float16, 2, 2>(a, p, device, stream);
}

}  // extern "C"
