// w4.hip -- C entry points of the product with 4-bit weights (gemm_rs_layer.h).
#include <type_traits>

#include "host.hpp"

#include "w4.hpp"

using namespace gemm_rs_layer;

namespace {

W4Layout w4_layout(const gemm_rs_w4_config& c)
{
    W4Layout l;
    l.N = c.N;
    l.K = c.K;
    l.group = c.group;
    l.tiles = (int)ceil_div(c.N, kW4Tile);
    l.blocks = (int)ceil_div(c.K, kW4Block);
    l.groups = (int)ceil_div(c.K, c.group);
    l.subs = c.group >= c.K || c.group % 128 == 0 ? 1 : c.group % 64 == 0 ? 2 : 4;
    const int64_t tb = (int64_t)l.tiles * l.blocks;
    l.scale_at = tb * 1024;
    l.zero_at = l.scale_at + tb * kW4Tile * l.subs * 2;
    l.bytes = l.zero_at + (c.zero_points ? tb * kW4Tile * l.subs : 0);
    return l;
}

// f(SUBS, ZEROS) for the layout, as compile-time constants
template <class F>
int w4_forms(const W4Layout& l, bool zeros, F f)
{
    auto subs = [&](auto z) {
        switch (l.subs) {
        case 1: return f(std::integral_constant<int, 1>(), z);
        case 2: return f(std::integral_constant<int, 2>(), z);
        default: return f(std::integral_constant<int, 4>(), z);
        }
    };
    return zeros ? subs(std::true_type()) : subs(std::false_type());
}

template <class T, int WAVES, int NT, int MF, bool FEW, int WA, int XA>
int w4_launch(const gemm_rs_w4_config& c, const W4Args& a, void* stream)
{
    const dim3 grid((unsigned)ceil_div(a.l.tiles, NT), (unsigned)ceil_div(a.M, 16 * MF));
    return w4_forms(a.l, c.zero_points, [&](auto subs, auto zeros) {
        return launch(w4_kernel<T, WAVES, NT, MF, FEW, WA, XA, decltype(subs)::value, decltype(zeros)::value>, grid, 64 * WAVES, a,
                      stream, "gemm_rs_w4_linear");
    });
}

template <class T, int NT>
int w4_tile_launch(const gemm_rs_w4_config& c, const W4Args& a, void* stream)
{
    const dim3 grid((unsigned)ceil_div(a.M, kW4Rows), (unsigned)ceil_div(a.l.tiles, 4 * NT));
    return w4_forms(a.l, c.zero_points, [&](auto subs, auto zeros) {
        return launch(w4_tile_kernel<T, NT, decltype(subs)::value, decltype(zeros)::value>, grid, 512, a, stream,
                      "gemm_rs_w4_linear");
    });
}

// Up to 32 rows: the kernel whose waves split K, with one tile of columns and more waves
// per workgroup where the tiles are no more than the CUs, else two tiles.  Measured, us
// (one / two): 3584 x 4096 at 4 rows 4.7 / 6.2, at 9 5.5 / 7.0, at 24 7.1 / 8.5; 7168 x 8192
// at 4 rows 12.1 (8 waves) / 10.7, at 9 15.4 / 11.5, at 24 20 / 14.4.
//
// More rows: whichever of six kernels costs least, as rounds of workgroups over the CUs
// times a round's cost.  A round takes a time that grows with the columns per workgroup,
// though not from zero (all run the whole of K).  Measured at K = 8192 with 64 rows, us for
// groups of 128 and of 32: the kernel above with 16 columns 19, 20; with 32 columns 29, 37;
// the kernel whose workgroups keep 64 rows in LDS with 64 columns 36, 40; 128: 44, 52; 192:
// 55, 68; 256: 66, 84.  The table has no entry for the group, zero points or K, which move
// the six alike: with 2048 rows 42, 43, 38, 50, 62, 76 for groups of 128, 42, 45, 42, 55, 74,
// 88 for groups of 32, 48, 57, 56, 78, 99, 132 with zero points too, and 16, 21, 15, 22, 29,
// 40 at K = 2048.  It takes the fastest of the six, or one within 2%, for 500 x 7168 x 8192,
// 500 x 6144 x 2048 and 2000 x 8192 x 3584 with groups of 128, of 32, and of 64 and 32 with
// zero points: 500 x 7168 x 8192, groups of 32 with zero points, 192 / 256 columns 196 / 139.
template <class T>
int w4_run(const gemm_rs_w4_config& c, const W4Args& a, void* stream)
{
    const bool narrow = a.l.tiles <= kCus;
    if (a.M <= 4)
        return narrow ? w4_launch<T, 16, 1, 1, true, 2, 2>(c, a, stream) : w4_launch<T, 8, 2, 1, true, 4, 4>(c, a, stream);
    if (a.M <= 16)
        return narrow ? w4_launch<T, 16, 1, 1, false, 2, 2>(c, a, stream) : w4_launch<T, 8, 2, 1, false, 4, 4>(c, a, stream);
    if (a.M <= 32)
        return narrow ? w4_launch<T, 8, 1, 2, false, 2, 1>(c, a, stream) : w4_launch<T, 8, 2, 2, false, 2, 1>(c, a, stream);
    constexpr int kTiles[6] = {1, 2, 4, 8, 12, 16}, kCost[6] = {3, 5, 6, 8, 10, 12};
    int best = 0;
    int64_t cost = INT64_MAX;
    for (int i = 0; i < 6; ++i) {
        const int64_t rounds = ceil_div(ceil_div(a.M, kW4Rows) * ceil_div(a.l.tiles, kTiles[i]), kCus);
        if (rounds * kCost[i] < cost) {
            cost = rounds * kCost[i];
            best = i;
        }
    }
    switch (best) {
    case 0: return w4_launch<T, 8, 1, 4, false, 2, 1>(c, a, stream);
    case 1: return w4_launch<T, 4, 2, 4, false, 2, 1>(c, a, stream);
    case 2: return w4_tile_launch<T, 1>(c, a, stream);
    case 3: return w4_tile_launch<T, 2>(c, a, stream);
    case 4: return w4_tile_launch<T, 3>(c, a, stream);
    default: return w4_tile_launch<T, 4>(c, a, stream);
    }
}

}  // namespace

extern "C" {

int gemm_rs_w4_validate(const gemm_rs_w4_config* c)
{
    if (!c || c->N < 0 || c->K < 0 || c->group <= 0 || (c->zero_points != 0 && c->zero_points != 1) ||
        (c->dtype != GEMM_RS_DTYPE_BF16 && c->dtype != GEMM_RS_DTYPE_F16))
        return GEMM_RS_ERR_INVALID_ARG;
    // packing takes a wave per tile and block
    if (c->K < 2 || c->K % 2 != 0 || c->K > (1 << 22) || c->N < 1 || c->N > (1 << 22) ||
        ceil_div(c->N, kW4Tile) * ceil_div(c->K, kW4Block) * 64 > kMaxThreads)
        return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
    if (c->group % 32 != 0 && c->group != c->K) return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
    return GEMM_RS_OK;
}

size_t gemm_rs_w4_packed_bytes(const gemm_rs_w4_config* c)
{
    return gemm_rs_w4_validate(c) == GEMM_RS_OK ? (size_t)w4_layout(*c).bytes : 0;
}

int gemm_rs_w4_pack(const gemm_rs_w4_config* c, const void* q, const void* scales, const void* zeros, void* packed,
                    void* stream)
{
    int rc = gemm_rs_w4_validate(c);
    if (rc != GEMM_RS_OK) return rc;
    Checker k;
    k.need(q, 1);
    k.need(scales, 2);
    k.need(packed, 16);
    if ((zeros != nullptr) != (c->zero_points != 0)) k.fail(GEMM_RS_ERR_INVALID_ARG);
    if (k.code != GEMM_RS_OK) return k.code;
    if ((rc = check_device()) != GEMM_RS_OK) return rc;
    W4PackArgs a;
    a.l = w4_layout(*c);
    a.q = static_cast<const uint8_t*>(q);
    a.scales = static_cast<const uint16_t*>(scales);
    a.zeros = static_cast<const uint8_t*>(zeros);
    a.packed = static_cast<char*>(packed);
    a.bf16 = c->dtype == GEMM_RS_DTYPE_BF16;
    return launch(w4_pack_kernel, dim3((unsigned)((int64_t)a.l.tiles * a.l.blocks)), 64, a, stream, "gemm_rs_w4_pack");
}

int gemm_rs_w4_linear(const gemm_rs_w4_config* c, const void* packed, int64_t M, const void* x, int64_t x_stride,
                      void* y, int64_t y_stride, void* stream)
{
    int rc = gemm_rs_w4_validate(c);
    if (rc != GEMM_RS_OK) return rc;
    if (M < 0) return GEMM_RS_ERR_INVALID_ARG;
    if (M > (1 << 20)) return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
    if (M == 0) return GEMM_RS_OK;
    Checker k;
    k.need(packed, 16);
    k.need(x, 2);
    k.need(y, 2);
    k.stride(x_stride, c->K);
    k.stride(y_stride, c->N);
    if (k.code != GEMM_RS_OK) return k.code;
    if ((rc = check_device()) != GEMM_RS_OK) return rc;
    W4Args a;
    a.l = w4_layout(*c);
    a.packed = static_cast<const char*>(packed);
    a.x = x;
    a.y = y;
    a.M = M;
    a.x_stride = x_stride;
    a.y_stride = y_stride;
    return c->dtype == GEMM_RS_DTYPE_BF16 ? w4_run<__bf16>(*c, a, stream) : w4_run<_Float16>(*c, a, stream);
}

}  // extern "C"
