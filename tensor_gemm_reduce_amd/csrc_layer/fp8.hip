// fp8.hip -- C entry points of the 8-bit floating-point matrices and their products
// (gemm_rs_experts.h).
#include "host.hpp"

#include "gemm_rs_experts.h"
#include "fp8.hpp"

using namespace gemm_rs_layer;

namespace {

constexpr int64_t kMaxWidth = 1 << 22;
constexpr int64_t kFewRows = 16;  // of the kernel for few rows, which has a form for twice as many
constexpr int64_t kMaxResource = (int64_t(1) << 31) - 1;  // bytes of a buffer resource below kOob

int64_t blocks_of(int64_t n) { return GEMM_RS_FP8_BLOCKS(n); }
int64_t pitch_of(int64_t rows) { return GEMM_RS_FP8_SCALE_ROWS(rows); }  // bytes from a block's scales to the next one's
int64_t scale_bytes(int64_t rows, int64_t cols) { return GEMM_RS_FP8_SCALE_BYTES(rows, cols); }
int64_t up16(int64_t n) { return ceil_div(n, 16) * 16; }
bool is_float(int dtype) { return dtype >= GEMM_RS_DTYPE_BF16 && dtype <= GEMM_RS_DTYPE_F32; }

template <class A>
using Kernel = void (*)(A);

template <class A>
Kernel<A> pick(int dtype, Kernel<A> bf16, Kernel<A> f16, Kernel<A> f32)
{
    return dtype == GEMM_RS_DTYPE_BF16 ? bf16 : dtype == GEMM_RS_DTYPE_F16 ? f16 : f32;
}

int quant_rows(int dtype, int64_t M, int64_t K, const void* x, int64_t stride, void* q, void* s, void* stream)
{
    Fp8QuantArgs a = {};
    a.x = x;
    a.q = static_cast<uint8_t*>(q);
    a.s = static_cast<uint8_t*>(s);
    a.M = M;
    a.stride = stride;
    a.K = (int)K;
    a.blocks = (int)blocks_of(K);
    a.pitch = (int)pitch_of(M);
    a.q_pitch = a.blocks * kFp8Block;
    return launch(pick(dtype, fp8_quant_kernel<__bf16>, fp8_quant_kernel<_Float16>, fp8_quant_kernel<float>),
                  dim3((unsigned)ceil_div(ceil_div(M, 16) * a.blocks, 4)), 256, a, stream, "gemm_rs_fp8_quant");
}

// blocks: of 128 rows of x, those of all experts where there are any
int quant_columns(int dtype, int64_t M, int64_t K, int64_t x_rows, const void* x, int64_t stride, const int32_t* offsets,
                  const int32_t* tokens, int64_t E, int64_t blocks, void* q, void* s, void* stream)
{
    Fp8QuantArgs a = {};
    a.x = x;
    a.q = static_cast<uint8_t*>(q);
    a.s = static_cast<uint8_t*>(s);
    a.M = M;
    a.stride = stride;
    a.K = (int)K;
    a.pitch = (int)pitch_of(K);
    a.q_pitch = blocks * kFp8Block;
    a.offsets = offsets;
    a.tokens = tokens;
    a.E = (int)E;
    a.x_rows = x_rows;
    return launch(pick(dtype, fp8_quant_t_kernel<__bf16>, fp8_quant_t_kernel<_Float16>, fp8_quant_t_kernel<float>),
                  dim3((unsigned)blocks, (unsigned)ceil_div(K, 64)), 256, a, stream, "gemm_rs_fp8_quant_transposed");
}

// A launch has threads for all of the rows' blocks.
bool quant_fits(int64_t M, int64_t K) { return ceil_div(M, 16) * blocks_of(K) <= kMaxThreads / 64 - 4; }

int quant_check(int32_t dtype, int64_t M, int64_t K, const void* x, int64_t stride, const void* q, const void* s)
{
    if (!is_float(dtype) || M < 0 || K < 1) return GEMM_RS_ERR_INVALID_ARG;
    if (M >= kMaxRows || K > kMaxWidth || !quant_fits(M, K)) return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
    if (M == 0) return GEMM_RS_OK;
    Checker c;
    c.need(x, elem_bytes(dtype));
    c.stride(stride, K);
    c.need(q, 16);
    c.need(s, 16);
    return c.code;
}

// A workgroup's LDS past 64 KB, allowed once per device.
template <class K>
int allow_lds(K kernel, int bytes, int device, std::atomic<bool>* allowed)
{
    if (allowed[device].load(std::memory_order_relaxed)) return GEMM_RS_OK;
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return hip_fail(e, "hipFuncSetAttribute");
    allowed[device].store(true, std::memory_order_relaxed);
    return GEMM_RS_OK;
}

// How a product runs: tiles of `tile` x `tile`, or the kernel for few rows, 16 or 32 of them at a time.
struct Fp8Form {
    int tile, stages;
    int64_t tiles_m, tiles_n, tiles, grid;
};

template <int W, int NS, int MODE, class T>
int tile_launch(Fp8Args& a, const Fp8Form& f, int device, void* stream)
{
    typedef Fp8Tile<W, NS, MODE> Tile;
    static std::atomic<bool> allowed[kMaxDevices];
    const int rc = allow_lds(fp8_kernel<W, NS, MODE, T>, Tile::kLds, device, allowed);
    if (rc != GEMM_RS_OK) return rc;
    a.tiles_n = (int)f.tiles_n;
    a.tiles_m = (int)f.tiles_m;
    void* p[] = {&a};
    const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(fp8_kernel<W, NS, MODE, T>), dim3((unsigned)f.grid), dim3(256), p,
                                         Tile::kLds, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? GEMM_RS_OK : hip_fail(e, "fp8_kernel");
}

// The kernel for few rows: a dense product's up to twice its tile, and experts' while their tiles of 128 x 128 would leave
// more than half of the CUs idle.  us so, and with tiles: dense, 7168 x 8192, 16 rows 17 / 28, 32 26 / 28; 2 of 8 experts of
// 4096 x 6144 for 1 token 12 / 26, 8 tokens 34 / 29, 64 62 / 30; 6 of 64 of 1408 x 2048, 4 tokens 14 / 13, 32 41 / 34.
bool takes_few(int64_t M, int64_t N, int64_t E)
{
    if (E == 0) return M <= 2 * kFewRows;
    return ceil_div(M, E) <= kFewRows && (E < M ? E : M) * ceil_div(N, 128) < kCus / 2;
}

template <int MF, int MODE, class X, class T>
int few_launch(const Fp8Args& a, const Fp8Form& f, void* stream)
{
    constexpr int kWaves = 8;
    return launch(fp8_few_kernel<kWaves, MF, MODE, X, T>, dim3((unsigned)f.tiles_n, (unsigned)f.tiles_m), 64 * kWaves, a, stream,
                  "fp8_few_kernel");
}

// 0: tiles of 256 x 256, 1: of 128 x 128 with two workgroups per CU, 2: with one: by the time of their rounds of tiles over
// the CUs, which is so much for each step and for the rest.  In tenths of a us; measured, us, BF16 results, 2 / 8 / 28 / 64
// steps: 128 tiles of 256 x 256 10 / 16 / 40 / 80, 256 of them 12 / 20 / 50 / 103; 128 x 128, two per CU: 256 tiles 6 / 8 / 24
// / 45, 512 7 / 11 / 30 / 63, 1024 11 / 21 / 58 / 124; one per CU: 256 tiles 6 / 9 / 20 / 39, 512 10 / 14 / 35 / 73.  FP32
// results: 256 tiles of 256 x 256 21 / 38 / 95 / 197; 128 x 128, two per CU: 256 tiles 8 / 11 / 29 / 60, 512 10 / 18 / 51 /
// 110; one per CU, 256 tiles: 8 / 12 / 30 / 63, which is never taken.  It takes the fastest of the three, or one within 7%,
// for 1024 x 4096 .. 8192 x 8192 with 8 steps or more; at two steps the second is up to 20% faster than the first, which
// is taken from 256 tiles on.
int tile_choice(bool exact, int64_t big, int64_t small, int64_t steps)
{
    const int64_t whole = exact ? 16 * steps + 70 : 9 * steps + 55, rest = small % (2 * kCus);
    const int64_t cost[3] = {ceil_div(big, kCus) * (exact ? 29 * steps + 100 : 14 * steps + 80),
                             small / (2 * kCus) * whole + (rest > kCus ? whole : rest == 0 ? 0 : exact ? 9 * steps + 60 : (13 * steps + 90) / 2),
                             ceil_div(small, kCus) * (exact ? 9 * steps + 60 : (11 * steps + 110) / 2)};
    if (cost[0] <= cost[1] && cost[0] <= cost[2]) return 0;
    return cost[1] < cost[2] ? 1 : 2;
}

// rows: of the experts' (kSums), whose steps are not known here, but their number on average
int form_of(int mode, int out_dtype, int64_t M, int64_t N, int64_t K, int64_t E, int64_t rows, Fp8Form& f)
{
    const bool exact = out_dtype == GEMM_RS_DTYPE_F32, grouped = mode == kByExpert || mode == kGather;
    const int64_t experts = E < M ? E : M;  // that can have a row
    // rows of tiles: exact, or a bound, and what to expect
    auto rows_of = [&](int64_t edge) { return grouped ? M / edge + experts : ceil_div(M, edge); };
    auto tiles = [&](int64_t edge) {
        return (grouped ? M / edge + (experts + 1) / 2 : rows_of(edge)) * ceil_div(N, edge) * (mode == kSums ? E : 1);
    };
    if (mode != kSums && takes_few(M, N, E)) {
        const int few = mode == kDense && M > kFewRows ? 2 * kFewRows : kFewRows;
        f = {few, 0, rows_of(few), ceil_div(N, kFewTile)};
        f.tiles = f.grid = f.tiles_m * f.tiles_n;
        return GEMM_RS_OK;
    }
    const int choice = tile_choice(exact, tiles(256), tiles(128), mode == kSums ? rows / E / kFp8Block + 1 : blocks_of(K));
    const int edge = choice == 0 ? 256 : 128;
    f = {edge, choice == 2 && !exact ? 4 : 2, rows_of(edge), ceil_div(N, edge)};
    f.tiles = f.tiles_m * f.tiles_n * (mode == kSums ? E : 1);
    f.grid = ceil_div(f.tiles_m * f.tiles_n, 8) * 8 * (mode == kSums ? E : 1);
    if (f.grid >= int64_t(1) << 31) return GEMM_RS_ERR_UNSUPPORTED_SHAPE;  // tiles are counted in 32 bits
    if (choice == 0 && f.grid > kCus) f.grid = kCus;
    return f.grid * 256 > kMaxThreads ? GEMM_RS_ERR_UNSUPPORTED_SHAPE : GEMM_RS_OK;
}

template <int MODE, class T>
int product(Fp8Args& a, const Fp8Form& f, int device, void* stream)
{
    if constexpr (MODE != kSums)
        if (f.tile == kFewRows) return few_launch<1, MODE, Fp8Few, T>(a, f, stream);
    if constexpr (MODE == kDense)
        if (f.tile == 2 * kFewRows) return few_launch<2, MODE, Fp8Few, T>(a, f, stream);
    if (f.tile == 256) return tile_launch<4, 2, MODE, T>(a, f, device, stream);
    if constexpr (!fp8_exact<T>)
        if (f.stages == 4) return tile_launch<2, 4, MODE, T>(a, f, device, stream);
    return tile_launch<2, 2, MODE, T>(a, f, device, stream);
}

// The product of a few rows that are quantised on the way: x and x_pitch are the matrix itself.
template <int MODE>
int few_of(int x_dtype, int out_dtype, const Fp8Args& a, const Fp8Form& f, void* stream)
{
    if (x_dtype == GEMM_RS_DTYPE_F32) return few_launch<1, MODE, float, float>(a, f, stream);
    if (x_dtype == GEMM_RS_DTYPE_F16)
        return out_dtype == GEMM_RS_DTYPE_F32 ? few_launch<1, MODE, _Float16, float>(a, f, stream)
                                              : few_launch<1, MODE, _Float16, _Float16>(a, f, stream);
    return out_dtype == GEMM_RS_DTYPE_F32 ? few_launch<1, MODE, __bf16, float>(a, f, stream)
                                          : few_launch<1, MODE, __bf16, __bf16>(a, f, stream);
}

template <int MODE>
int product_of(int out_dtype, Fp8Args& a, const Fp8Form& f, int device, void* stream)
{
    return out_dtype == GEMM_RS_DTYPE_BF16  ? product<MODE, __bf16>(a, f, device, stream)
           : out_dtype == GEMM_RS_DTYPE_F16 ? product<MODE, _Float16>(a, f, device, stream)
                                            : product<MODE, float>(a, f, device, stream);
}

bool fp8_args_ok(const gemm_rs_fp8_args* g)
{
    return g && (is_float(g->x_dtype) || g->x_dtype == GEMM_RS_DTYPE_FP8) && is_float(g->out_dtype) && g->M >= 0 && g->N >= 1 &&
           g->K >= 1 && g->x_rows >= 0 && g->E >= 0;
}

// x is quantised by the product's own kernel: few rows, not too many bytes of them for every 16 columns to read again, and of
// few blocks, since a wave's conversions stand in the way of its weights' loads.  us so, and with a kernel before it: 1 x 1024 x
// 1024 3.2 / 5.1, 1 x 8192 x 1024 5.1 / 5.7, 16 x 8192 x 1024 6.3 / 7.1, 8 x 2048 x 4096 7.9 / 7.9, 1 x 7168 x 8192 20.5 / 15.8.
constexpr int64_t kFewBytes = 17 << 20, kFewInputs = 4096;

bool few_raw(const gemm_rs_fp8_args& g)
{
    return g.x_dtype != GEMM_RS_DTYPE_FP8 && (g.out_dtype == g.x_dtype || g.out_dtype == GEMM_RS_DTYPE_F32) &&
           takes_few(g.M, g.N, g.E) && (g.E > 0 || g.M <= kFewRows) && g.K <= kFewInputs &&
           ceil_div(g.N, kFewTile) * g.M <= kFewBytes / (g.K * elem_bytes(g.x_dtype));
}

// q and scales of x in the workspace
size_t quant_bytes(int64_t rows, int64_t K) { return (size_t)(up16(GEMM_RS_FP8_Q_BYTES(rows, K)) + up16(scale_bytes(rows, K))); }

// The sizes and the kind of a product, and how it runs.
int fp8_form(const gemm_rs_fp8_args* g, Fp8Form& f)
{
    if (!fp8_args_ok(g)) return GEMM_RS_ERR_INVALID_ARG;
    if (g->E ? !g->offsets : g->offsets || g->tokens) return GEMM_RS_ERR_INVALID_ARG;
    if (g->tokens ? g->x_rows == 0 && g->M > 0 : g->x_rows != g->M) return GEMM_RS_ERR_INVALID_ARG;
    if (g->M >= kMaxRows || g->x_rows >= kMaxRows || g->N > kMaxWidth || g->K > kMaxWidth || g->E > GEMM_RS_ROUTE_MAX_EXPERTS ||
        scale_bytes(g->x_rows, g->K) > kMaxResource || scale_bytes(g->N, g->K) > kMaxResource ||
        (g->tokens && GEMM_RS_FP8_Q_BYTES(g->x_rows, g->K) > kMaxResource))
        return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
    f = {};
    if (g->M == 0) return GEMM_RS_OK;
    if (g->x_dtype != GEMM_RS_DTYPE_FP8 && !quant_fits(g->x_rows, g->K)) return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
    return form_of(g->E == 0 ? kDense : g->tokens ? kGather : kByExpert, g->out_dtype, g->M, g->N, g->K, g->E, 0, f);
}

int fp8_product(const gemm_rs_fp8_args* g, bool experts, void* workspace, size_t workspace_bytes, void* stream)
{
    if (g && experts != (g->E != 0)) return GEMM_RS_ERR_INVALID_ARG;
    Fp8Form form;
    int rc = fp8_form(g, form);
    if (rc != GEMM_RS_OK || g->M == 0) return rc;
    const int64_t blocks = blocks_of(g->K), pitch = blocks * kFp8Block;
    const bool raw = g->x_dtype != GEMM_RS_DTYPE_FP8;
    Checker c;
    c.need(g->x, raw ? elem_bytes(g->x_dtype) : 16);
    if (raw) c.stride(g->x_stride, g->K);
    else c.need(g->x_scales, 16);
    c.need(g->w, 16);
    c.need(g->w_scales, 16);
    c.maybe(g->offsets, 4);
    c.maybe(g->tokens, 4);
    c.maybe(g->add, 4);
    if (g->add) c.stride(g->add_stride, g->N);
    c.need(g->out, elem_bytes(g->out_dtype));
    c.stride(g->out_stride, g->N);
    if (g->add && (g->out_dtype != GEMM_RS_DTYPE_F32 || (g->add == g->out && g->add_stride != g->out_stride)))
        c.fail(GEMM_RS_ERR_INVALID_ARG);
    const size_t ws = gemm_rs_fp8_workspace(g);
    if (ws > 0) {
        if (!workspace || workspace_bytes < ws) c.fail(GEMM_RS_ERR_SCRATCH);
        else c.need(workspace, 16);
    }
    if (c.code != GEMM_RS_OK) return c.code;
    int device = 0;
    if ((rc = check_device(&device)) != GEMM_RS_OK) return rc;
    Fp8Args a = {};
    a.x = static_cast<const uint8_t*>(g->x);
    a.xs = static_cast<const uint8_t*>(g->x_scales);
    const bool few = few_raw(*g);
    if (raw && !few) {
        uint8_t* q = static_cast<uint8_t*>(workspace);
        uint8_t* s = q + up16(g->x_rows * pitch);
        rc = quant_rows(g->x_dtype, g->x_rows, g->K, g->x, g->x_stride, q, s, stream);
        if (rc != GEMM_RS_OK) return rc;
        a.x = q;
        a.xs = s;
    }
    a.w = static_cast<const uint8_t*>(g->w);
    a.ws = static_cast<const uint8_t*>(g->w_scales);
    a.offsets = g->offsets;
    a.tokens = g->tokens;
    a.add = g->add;
    a.out = g->out;
    a.M = g->M;
    a.x_rows = g->x_rows;
    a.x_pitch = few ? g->x_stride * elem_bytes(g->x_dtype) : pitch;
    a.w_pitch = pitch;
    a.w_expert = g->N * pitch;
    a.ws_expert = scale_bytes(g->N, g->K);
    a.add_stride = g->add_stride;
    a.out_stride = g->out_stride;
    a.xs_bytes = scale_bytes(g->x_rows, g->K);
    a.ws_bytes = a.ws_expert;
    a.N = (int)g->N;
    a.K = (int)g->K;
    a.E = (int)g->E;
    a.steps = (int)blocks;
    a.xs_pitch = (int)pitch_of(g->x_rows);
    a.ws_pitch = (int)pitch_of(g->N);
    if (few)
        return !experts    ? few_of<kDense>(g->x_dtype, g->out_dtype, a, form, stream)
               : g->tokens ? few_of<kGather>(g->x_dtype, g->out_dtype, a, form, stream)
                           : few_of<kByExpert>(g->x_dtype, g->out_dtype, a, form, stream);
    return !experts    ? product_of<kDense>(g->out_dtype, a, form, device, stream)
           : g->tokens ? product_of<kGather>(g->out_dtype, a, form, device, stream)
                       : product_of<kByExpert>(g->out_dtype, a, form, device, stream);
}

bool wgrad_ok(const gemm_rs_experts_wgrad_args* g)
{
    return g && is_float(g->dtype) && (g->out_dtype == g->dtype || g->out_dtype == GEMM_RS_DTYPE_F32) && g->M >= 0 && g->N >= 1 &&
           g->K >= 1 && g->E >= 1 && g->x_rows >= 0;
}

// Blocks of 128 rows that the experts' rows make at most.
int64_t wgrad_blocks(const gemm_rs_experts_wgrad_args& g) { return g.M / kFp8Block + (g.E < g.M ? g.E : g.M); }

bool wgrad_fits(const gemm_rs_experts_wgrad_args& g)
{
    return g.M < kMaxRows && g.x_rows < kMaxRows && g.N <= kMaxWidth && g.K <= kMaxWidth && g.E <= GEMM_RS_ROUTE_MAX_EXPERTS &&
           wgrad_blocks(g) * kFp8Block <= kMaxResource / 256 && pitch_of(g.N) * wgrad_blocks(g) <= kMaxResource &&
           pitch_of(g.K) * wgrad_blocks(g) <= kMaxResource && ceil_div(g.N, 64) <= 65535 && ceil_div(g.K, 64) <= 65535;
}

int wgrad_form(const gemm_rs_experts_wgrad_args* g, Fp8Form& f)
{
    if (!wgrad_ok(g) || (!g->tokens && g->x_rows != g->M)) return GEMM_RS_ERR_INVALID_ARG;
    if (!wgrad_fits(*g)) return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
    return form_of(kSums, g->out_dtype, g->N, g->K, 0, g->E, g->x_rows > 0 ? g->M : 0, f);
}

int64_t wgrad_operand(int64_t rows, int64_t blocks) { return up16(rows * blocks * kFp8Block) + up16(pitch_of(rows) * blocks); }

}  // namespace

extern "C" {

int gemm_rs_fp8_quant(int32_t dtype, int64_t M, int64_t K, const void* x, int64_t x_stride, void* q, void* scales, void* stream)
{
    int rc = quant_check(dtype, M, K, x, x_stride, q, scales);
    if (rc != GEMM_RS_OK || M == 0) return rc;
    if ((rc = check_device()) != GEMM_RS_OK) return rc;
    return quant_rows(dtype, M, K, x, x_stride, q, scales, stream);
}

int gemm_rs_fp8_quant_transposed(int32_t dtype, int64_t M, int64_t K, const void* x, int64_t x_stride, void* q, void* scales,
                                 void* stream)
{
    int rc = quant_check(dtype, M, K, x, x_stride, q, scales);
    if (rc != GEMM_RS_OK || M == 0) return rc;
    if (ceil_div(K, 64) > 65535 || blocks_of(M) * 256 > kMaxThreads) return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
    if ((rc = check_device()) != GEMM_RS_OK) return rc;
    return quant_columns(dtype, M, K, M, x, x_stride, nullptr, nullptr, 0, blocks_of(M), q, scales, stream);
}

int gemm_rs_fp8_pack(int32_t dtype, int64_t E, int64_t N, int64_t K, int32_t transpose, const void* w, void* q, void* scales,
                     void* stream)
{
    if (!is_float(dtype) || E < 1 || N < 1 || K < 1 || (transpose != 0 && transpose != 1)) return GEMM_RS_ERR_INVALID_ARG;
    if (E > 65535 || N > kMaxWidth || K > kMaxWidth) return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
    Checker c;
    c.need(w, elem_bytes(dtype));
    c.need(q, 16);
    c.need(scales, 16);
    if (c.code != GEMM_RS_OK) return c.code;
    const int rc = check_device();
    if (rc != GEMM_RS_OK) return rc;
    Fp8PackArgs a = {};
    const int64_t rows = transpose ? K : N, cols = transpose ? N : K;
    a.w = w;
    a.q = static_cast<uint8_t*>(q);
    a.s = static_cast<uint8_t*>(scales);
    a.N = (int)N;
    a.K = (int)K;
    a.transpose = transpose;
    a.w_expert = N * K;
    a.q_pitch = blocks_of(cols) * kFp8Block;
    a.q_expert = rows * a.q_pitch;
    a.s_expert = scale_bytes(rows, cols);
    a.pitch = (int)pitch_of(rows);
    return launch(pick(dtype, fp8_pack_kernel<__bf16>, fp8_pack_kernel<_Float16>, fp8_pack_kernel<float>),
                  dim3((unsigned)blocks_of(K), (unsigned)blocks_of(N), (unsigned)E), 256, a, stream, "gemm_rs_fp8_pack");
}

size_t gemm_rs_fp8_workspace(const gemm_rs_fp8_args* g)
{
    if (!fp8_args_ok(g) || g->M == 0 || g->x_dtype == GEMM_RS_DTYPE_FP8 || g->x_rows >= kMaxRows || g->K > kMaxWidth || few_raw(*g))
        return 0;
    return quant_bytes(g->x_rows, g->K);
}

int gemm_rs_fp8_plan(const gemm_rs_fp8_args* g, gemm_rs_fp8_info* info)
{
    Fp8Form f;
    const int rc = fp8_form(g, f);
    if (rc != GEMM_RS_OK) return rc;
    if (!info) return GEMM_RS_ERR_INVALID_ARG;
    *info = {f.tile, f.stages, g->M > 0 && few_raw(*g), (int32_t)f.tiles, (int32_t)f.grid};
    return GEMM_RS_OK;
}

int gemm_rs_fp8_linear(const gemm_rs_fp8_args* g, void* workspace, size_t workspace_bytes, void* stream)
{
    return fp8_product(g, false, workspace, workspace_bytes, stream);
}

int gemm_rs_experts_linear(const gemm_rs_fp8_args* g, void* workspace, size_t workspace_bytes, void* stream)
{
    return fp8_product(g, true, workspace, workspace_bytes, stream);
}

size_t gemm_rs_experts_wgrad_workspace(const gemm_rs_experts_wgrad_args* g)
{
    if (!wgrad_ok(g) || !wgrad_fits(*g) || g->M == 0 || g->x_rows == 0) return 0;
    const int64_t blocks = wgrad_blocks(*g);
    return (size_t)(wgrad_operand(g->N, blocks) + wgrad_operand(g->K, blocks));
}

int gemm_rs_experts_wgrad_plan(const gemm_rs_experts_wgrad_args* g, gemm_rs_fp8_info* info)
{
    Fp8Form f;
    const int rc = wgrad_form(g, f);
    if (rc != GEMM_RS_OK) return rc;
    if (!info) return GEMM_RS_ERR_INVALID_ARG;
    *info = {f.tile, f.stages, 0, (int32_t)f.tiles, (int32_t)f.grid};
    return GEMM_RS_OK;
}

int gemm_rs_experts_wgrad(const gemm_rs_experts_wgrad_args* g, void* workspace, size_t workspace_bytes, void* stream)
{
    Fp8Form form;
    int rc = wgrad_form(g, form);
    if (rc != GEMM_RS_OK) return rc;
    const bool any = g->M > 0 && g->x_rows > 0;
    Checker c;
    c.need(g->offsets, 4);
    c.maybe(g->tokens, 4);
    if (any) {
        c.need(g->dy, elem_bytes(g->dtype));
        c.stride(g->dy_stride, g->N);
        c.need(g->x, elem_bytes(g->dtype));
        c.stride(g->x_stride, g->K);
    }
    c.maybe(g->add, 4);
    c.need(g->dw, elem_bytes(g->out_dtype));
    if (g->add && g->out_dtype != GEMM_RS_DTYPE_F32) c.fail(GEMM_RS_ERR_INVALID_ARG);
    const size_t need = gemm_rs_experts_wgrad_workspace(g);
    if (need > 0) {
        if (!workspace || workspace_bytes < need) c.fail(GEMM_RS_ERR_SCRATCH);
        else c.need(workspace, 16);
    }
    if (c.code != GEMM_RS_OK) return c.code;
    int device = 0;
    if ((rc = check_device(&device)) != GEMM_RS_OK) return rc;
    Fp8Args a = {};
    const int64_t blocks = any ? wgrad_blocks(*g) : 0;
    if (any) {
        uint8_t* y = static_cast<uint8_t*>(workspace);
        uint8_t* ys = y + up16(g->N * blocks * kFp8Block);
        uint8_t* x = y + wgrad_operand(g->N, blocks);
        uint8_t* xs = x + up16(g->K * blocks * kFp8Block);
        rc = quant_columns(g->dtype, g->M, g->N, g->M, g->dy, g->dy_stride, g->offsets, nullptr, g->E, blocks, y, ys, stream);
        if (rc == GEMM_RS_OK)
            rc = quant_columns(g->dtype, g->M, g->K, g->x_rows, g->x, g->x_stride, g->offsets, g->tokens, g->E, blocks, x, xs, stream);
        if (rc != GEMM_RS_OK) return rc;
        a.x = y;
        a.xs = ys;
        a.w = x;
        a.ws = xs;
    }
    a.offsets = g->offsets;
    a.add = g->add;
    a.out = g->dw;
    a.M = g->N;
    a.x_rows = g->N;
    a.rows = any ? g->M : 0;
    a.x_pitch = a.w_pitch = blocks * kFp8Block;
    a.out_expert = g->N * g->K;
    a.add_stride = a.out_stride = g->K;
    a.xs_bytes = pitch_of(g->N) * blocks;
    a.ws_bytes = pitch_of(g->K) * blocks;
    a.N = (int)g->K;
    a.E = (int)g->E;
    a.xs_pitch = (int)pitch_of(g->N);
    a.ws_pitch = (int)pitch_of(g->K);
    return product_of<kSums>(g->out_dtype, a, form, device, stream);
}

}  // extern "C"
