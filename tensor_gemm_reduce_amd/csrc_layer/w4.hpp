// w4.hpp -- the product of a few tokens with 4-bit weights:
//   y[m][n] = sum over groups g of s[n][g] sum_{k in g} x[m][k] (q[n][k] - z[n][g])
//
// The weight bytes bound it (at up to about 64 tokens), so they are laid out once
// in the order the waves consume them, and everything else is arranged around
// reading them at full rate.
//   - A nibble becomes a 16-bit float by two bit operations per pair: placed in the
//     mantissa of 16.0 it reads as 16 + q exactly.
//   - The MFMA multiplies x by 16 + q; the group's FP32 accumulator starts at
//     -(16 + z) times the sum of the group's inputs, which an MFMA with a constant
//     gives for every column at once.  No weight is rounded, and none has its zero
//     point subtracted by itself.
//   - The group's accumulator times its scale is added to the result's (FP32).
#pragma once

#include "common.hpp"

namespace gemm_rs_layer {

constexpr int kW4Tile = 16;    // rows of w per tile: the columns of one MFMA
constexpr int kW4Block = 128;  // inputs per block of a tile: 64 lanes x 16 bytes

// Packed weights: tiles x blocks of 1 KiB of nibbles, then the scales, then the
// zero points, each [tile][block][row of the tile][sub], with `subs` (1, 2 or 4)
// scales per row and block.
//   Word t (0..3) of lane l holds row l % 16, inputs 32 t + 8 (l / 16) + 0..7 of
//   the block: nibble i < 4 is input 2 i, nibble 4 + i input 2 i + 1, so a shift
//   and a mask give the pair (2 i, 2 i + 1) in the halves of a word.
struct W4Layout {
    int N, K, group;
    int tiles, blocks, groups, subs;  // groups: per row, as given
    int64_t scale_at, zero_at, bytes;
};

struct W4PackArgs {
    W4Layout l;
    const uint8_t* q;
    const uint16_t* scales;
    const uint8_t* zeros;
    char* packed;
};

// One wave per (tile, block).  Weights past N or K are stored as zeros with a zero
// scale, so they add nothing.
__global__ __launch_bounds__(64) void w4_pack_kernel(const W4PackArgs a)
{
    const int lane = threadIdx.x;
    const int64_t tb = blockIdx.x;
    const int tile = (int)(tb / a.l.blocks), block = (int)(tb % a.l.blocks);
    const int n = tile * kW4Tile + lane % 16;
    u32x4 w;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        uint32_t v = 0;
        const int k = block * kW4Block + 32 * t + 8 * (lane / 16);
        for (int j = 0; j < 8; ++j) {
            uint32_t nib = 0;
            if (n < a.l.N && k + j < a.l.K)
                nib = (a.q[(int64_t)n * (a.l.K / 2) + (k + j) / 2] >> (4 * ((k + j) & 1))) & 15u;
            v |= nib << (4 * (j / 2 + 4 * (j & 1)));
        }
        w[t] = v;
    }
    *reinterpret_cast<u32x4*>(a.packed + (tb * 64 + lane) * 16) = w;
    const int per = kW4Tile * a.l.subs;
    if (lane < per) {
        const int row = lane / a.l.subs, k = block * kW4Block + (lane % a.l.subs) * (kW4Block / a.l.subs);
        const int nn = tile * kW4Tile + row;
        const bool in = nn < a.l.N && k < a.l.K;
        const int64_t g = (int64_t)nn * a.l.groups + (in ? k / a.l.group : 0);
        reinterpret_cast<uint16_t*>(a.packed + a.l.scale_at)[tb * per + lane] = in ? a.scales[g] : (uint16_t)0;
        if (a.zeros) reinterpret_cast<uint8_t*>(a.packed + a.l.zero_at)[tb * per + lane] = in ? a.zeros[g] & 15u : 0u;
    }
}

template <class T>
struct W4Type;
template <>
struct W4Type<__bf16> {
    typedef bf16x8 frag;
    static constexpr uint32_t kMask = 0x00780078u, kMagic = 0x41804180u;  // 16.0 in both halves
    static constexpr int kShift = 3;                                      // the nibble's place in the mantissa
    static __device__ __forceinline__ f32x4 mfma(frag a, frag b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};
template <>
struct W4Type<_Float16> {
    typedef f16x8 frag;
    static constexpr uint32_t kMask = 0x03C003C0u, kMagic = 0x4C004C00u;
    static constexpr int kShift = 6;
    static __device__ __forceinline__ f32x4 mfma(frag a, frag b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};

// The eight weights of a word as 16 + q.
template <class T>
__device__ __forceinline__ typename W4Type<T>::frag w4_expand(uint32_t w)
{
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int sh = 4 * i - W4Type<T>::kShift;
        const uint32_t b = sh >= 0 ? w >> (sh >= 0 ? sh : 0) : w << (sh < 0 ? -sh : 0);
        v[i] = (b & W4Type<T>::kMask) | W4Type<T>::kMagic;
    }
    return __builtin_bit_cast(typename W4Type<T>::frag, v);
}

// A value in all eight places.
template <class T>
__device__ __forceinline__ typename W4Type<T>::frag w4_constant(float v)
{
    typename W4Type<T>::frag f;
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = (T)v;
    return f;
}

// Within 16 lanes, lane i takes lane i + N's register (zero past the end).
template <int N>
__device__ __forceinline__ i32x4 lanes_down(const i32x4& v)
{
    i32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __builtin_amdgcn_update_dpp(0, v[i], 0x100 + N, 0xF, 0xF, true);
    return r;
}

struct W4Args {
    W4Layout l;
    const char* packed;
    const void* x;
    void* y;
    int64_t M, x_stride, y_stride;
};

// What one block of 128 inputs brings: the weights, scales and zero points of NT tiles.
template <class T, int NT, int SUBS, bool ZEROS>
struct W4Block {
    u32x4 w[NT];
    T sc[NT][SUBS];
    uint8_t z[NT][SUBS];

    // tb: tile 0's index of the block; tiles are `blocks` apart.  Tiles past the last read it again.
    __device__ __forceinline__ void load(const W4Args& a, int tile0, int b)
    {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int tile = min(tile0 + t, a.l.tiles - 1);
            const int64_t tb = (int64_t)tile * a.l.blocks + b;
            w[t] = *reinterpret_cast<const u32x4*>(a.packed + (tb * 64 + lane) * 16);
            const int64_t at = tb * (kW4Tile * SUBS) + (lane & 15) * SUBS;
            typedef T scales_t __attribute__((ext_vector_type(SUBS)));
            typedef uint8_t zeros_t __attribute__((ext_vector_type(SUBS)));
            const scales_t s = *reinterpret_cast<const scales_t*>(a.packed + a.l.scale_at + at * 2);
            zeros_t zz;
            if constexpr (ZEROS) zz = *reinterpret_cast<const zeros_t*>(a.packed + a.l.zero_at + at);
#pragma unroll
            for (int u = 0; u < SUBS; ++u) {
                sc[t][u] = s[u];
                z[t][u] = ZEROS ? zz[u] : 8;
            }
        }
    }
    // acc[t][f] += the block's product with the rows x[f] (four steps of 32 inputs).  The part of the zero points,
    // -(16 + z) times the sum of a row's inputs, is where a group's accumulator starts: that sum is one MFMA per step
    // for all the tiles.
    template <int MF>
    __device__ __forceinline__ void multiply(const typename W4Type<T>::frag (&x)[MF][4], f32x4 (&acc)[NT][MF]) const
    {
        constexpr int kSteps = 4 / SUBS;  // steps per scale
        const typename W4Type<T>::frag unit = w4_constant<T>(ZEROS ? -1.f : -24.f);
#pragma unroll
        for (int u = 0; u < SUBS; ++u) {
            f32x4 start[MF] = {};
#pragma unroll
            for (int k = 0; k < kSteps; ++k)
#pragma unroll
                for (int f = 0; f < MF; ++f) start[f] = W4Type<T>::mfma(x[f][u * kSteps + k], unit, start[f]);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                f32x4 g[MF];
#pragma unroll
                for (int f = 0; f < MF; ++f) g[f] = ZEROS ? start[f] * (float)(16 + z[t][u]) : start[f];
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
                    const typename W4Type<T>::frag q = w4_expand<T>(w[t][u * kSteps + k]);
#pragma unroll
                    for (int f = 0; f < MF; ++f) g[f] = W4Type<T>::mfma(x[f][u * kSteps + k], q, g[f]);
                }
                const float scale = (float)sc[t][u];
#pragma unroll
                for (int f = 0; f < MF; ++f)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[t][f][r] = __builtin_fmaf(g[f][r], scale, acc[t][f][r]);
            }
        }
    }
};

// Few rows: a workgroup computes NT tiles of 16 columns for up to 16 MF rows; its
// waves split the blocks of K and add up through LDS at the end, in wave order.
//   - Each wave keeps the weights of the next WA blocks and the rows of the next XA in
//     flight, in registers that a block's loads refill in place once it is multiplied
//     (a copy from one set to another would wait for the loads).
//   - A load of x takes four rows' 256 bytes of a block, so whole lines; the fragments
//     (16 rows x 64 bytes) are made in the wave's own part of LDS, 16-byte chunk c of
//     row m at c ^ m % 16.  Loading fragments directly touches 16 half lines per
//     instruction, of rows that share their cache set when they are a power of two
//     apart (7168 x 8192, 24 rows, nothing else changed: 18.5 us so, 16.2 by LDS).
//   - FEW (at most four rows) needs no LDS for it: the one load puts row m of step t
//     into lane 4 t + m of each 16, and a step's fragment is that register shifted down
//     4 t lanes (its rows past the fourth are other steps', and not stored).
template <class T, int WAVES, int NT, int MF, bool FEW, int WA, int XA, int SUBS, bool ZEROS>
__global__ __launch_bounds__(64 * WAVES) void w4_kernel(const W4Args a)
{
    static_assert(WA % XA == 0 && (!FEW || MF == 1), "register rings");
    typedef typename W4Type<T>::frag frag;
    typedef W4Block<T, NT, SUBS, ZEROS> Block;
    constexpr int kLoads = FEW ? 1 : 4 * MF;
    constexpr int kRow = kW4Block * 2, kArea = FEW ? 0 : 16 * MF * kRow;  // bytes of a row's block; of a wave's rows
    constexpr int kPart = NT * MF * 64 * 16;                              // of a wave's results
    __shared__ __attribute__((aligned(16))) char lds[WAVES * (kArea > kPart ? kArea : kPart)];
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6);
    char* const area = lds + wave * kArea;
    const int tile0 = blockIdx.x * NT;
    const int64_t m0 = (int64_t)blockIdx.y * (16 * MF);
    const int loads = FEW ? 1 : (int)min((a.M - m0 + 3) / 4, (int64_t)kLoads);
    f32x4 acc[NT][MF] = {};
    // Load i of a block: row 4 i + lane / 16, 16-byte chunk lane % 16 (FEW: row lane % 4, chunk lane % 16 / 4 of the
    // step's four and step lane / 16 changed over).  A row past the last reads that again; rows of loads that are left
    // out hold anything.  Neither's results are stored.
    const int l16 = lane & 15, r0 = lane >> 4;
    const int col0 = FEW ? 32 * (l16 >> 2) + 8 * r0 : 8 * l16;
    auto row = [&](int i) {
        const int64_t m = FEW ? l16 & 3 : m0 + 4 * i + r0;
        return static_cast<const T*>(a.x) + (m < a.M ? m : a.M - 1) * a.x_stride;
    };
    auto load_x = [&](vec8<T> (&x)[kLoads], int b) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            if (i < loads) x[i] = *reinterpret_cast<const vec8<T>*>(row(i) + b * kW4Block + col0);
    };
    auto fragments = [&](const vec8<T> (&x)[kLoads], frag (&s)[MF][4]) {
        if constexpr (FEW) {
            const i32x4 v = __builtin_bit_cast(i32x4, x[0]);
            s[0][0] = __builtin_bit_cast(frag, v);
            s[0][1] = __builtin_bit_cast(frag, lanes_down<4>(v));
            s[0][2] = __builtin_bit_cast(frag, lanes_down<8>(v));
            s[0][3] = __builtin_bit_cast(frag, lanes_down<12>(v));
        } else {
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                if (i < loads)
                    *reinterpret_cast<u32x4*>(area + (4 * i + r0) * kRow + ((l16 ^ ((4 * i + r0) & 15)) * 16)) =
                        __builtin_bit_cast(u32x4, x[i]);
#pragma unroll
            for (int f = 0; f < MF; ++f)
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    s[f][t] = *reinterpret_cast<const frag*>(area + (16 * f + l16) * kRow + (((4 * t + r0) ^ l16) * 16));
        }
    };
    const int b0 = (int)((int64_t)a.l.blocks * wave / WAVES), b1 = (int)((int64_t)a.l.blocks * (wave + 1) / WAVES);
    const int whole = min(b1, a.l.K / kW4Block);  // the last block may end past K
    Block w[WA];
    vec8<T> x[XA][kLoads];
    frag s[MF][4];
#pragma unroll
    for (int i = 0; i < WA; ++i)
        if (b0 + i < whole) {
            w[i].load(a, tile0, b0 + i);
            if (i < XA) load_x(x[i], b0 + i);
        }
    for (int b = b0; b < whole; b += WA) {
#pragma unroll
        for (int i = 0; i < WA; ++i) {
            if (b + i < whole) {
                fragments(x[i % XA], s);
                if (b + i + XA < whole) load_x(x[i % XA], b + i + XA);
                w[i].multiply(s, acc);
            }
            if (b + i + WA < whole) w[i].load(a, tile0, b + i + WA);
        }
    }
    if (whole < b1) {
        w[0].load(a, tile0, b1 - 1);
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            if (i < loads) x[0][i] = load8(row(i), (b1 - 1) * kW4Block + col0, a.l.K);
        fragments(x[0], s);
        w[0].multiply(s, acc);
    }
    __syncthreads();
    f32x4* const part = reinterpret_cast<f32x4*>(lds);  // [wave][tile][16 rows][lane]
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int f = 0; f < MF; ++f) part[((wave * NT + t) * MF + f) * 64 + lane] = acc[t][f];
    __syncthreads();
    // lane l of a tile holds rows 4 (l / 16) .. + 3 of column l % 16
    for (int i = threadIdx.x; i < NT * MF * 64; i += 64 * WAVES) {
        const int l = i & 63, f = (i >> 6) % MF, t = (i >> 6) / MF;
        f32x4 sum = part[i];
#pragma unroll
        for (int v = 1; v < WAVES; ++v) sum += part[v * NT * MF * 64 + i];
        const int n = (tile0 + t) * kW4Tile + (l & 15);
        if (n >= a.l.N) continue;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int64_t m = m0 + f * 16 + 4 * (l >> 4) + r;
            if (m < a.M) static_cast<T*>(a.y)[m * a.y_stride + n] = (T)sum[r];
        }
    }
}

// Many rows: 64 rows x 64 NT columns per workgroup, four waves of 64 x 16 NT over the
// whole of K.  The rows' block of x goes through LDS (16-byte chunk c of row m at
// c ^ m % 16), two blocks ahead in registers; each wave expands its own weights.
constexpr int kW4Rows = 64;

template <class T, int NT, int SUBS, bool ZEROS>
__global__ __launch_bounds__(256, 2) void w4_tile_kernel(const W4Args a)
{
    typedef typename W4Type<T>::frag frag;
    typedef W4Block<T, NT, SUBS, ZEROS> Block;
    constexpr int kRow = kW4Block * 2;  // bytes of a row's block
    __shared__ __attribute__((aligned(16))) char lds[2][kW4Rows * kRow];
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6);
    const int tile0 = (blockIdx.y * 4 + wave) * NT;
    const int64_t m0 = (int64_t)blockIdx.x * kW4Rows;
    const int chunk = threadIdx.x & 15, r0 = threadIdx.x >> 4;
    const T* xrow[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        int64_t m = m0 + r0 + 16 * i;
        m = m < a.M ? m : a.M - 1;
        xrow[i] = static_cast<const T*>(a.x) + m * a.x_stride;
    }
    vec8<T> xr[4];
    auto load_x = [&](int b) {
        if (b >= a.l.blocks) return;
#pragma unroll
        for (int i = 0; i < 4; ++i) xr[i] = load8(xrow[i], b * kW4Block + chunk * 8, a.l.K);
    };
    auto put_x = [&](char* stage) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<u32x4*>(stage + (r0 + 16 * i) * kRow + ((chunk ^ r0) * 16)) = __builtin_bit_cast(u32x4, xr[i]);
    };
    f32x4 acc[NT][4] = {};
    Block w[2];
    load_x(0);
    w[0].load(a, tile0, 0);
    if (a.l.blocks > 1) w[1].load(a, tile0, 1);
    put_x(lds[0]);
    load_x(1);
    __syncthreads();
    for (int b = 0; b < a.l.blocks; b += 2) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (b + i < a.l.blocks) {
                frag x[4][4];
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int f = 0; f < 4; ++f)
                        x[f][t] = *reinterpret_cast<const frag*>(lds[i] + (f * 16 + (lane & 15)) * kRow +
                                                                 (((4 * t + (lane >> 4)) ^ (lane & 15)) * 16));
                if (b + i + 1 < a.l.blocks) put_x(lds[i ^ 1]);
                load_x(b + i + 2);
                w[i].multiply(x, acc);
                if (b + i + 2 < a.l.blocks) w[i].load(a, tile0, b + i + 2);
                __syncthreads();
            }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int n = (tile0 + t) * kW4Tile + (lane & 15);
        if (n >= a.l.N) continue;
#pragma unroll
        for (int f = 0; f < 4; ++f)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int64_t m = m0 + f * 16 + 4 * (lane >> 4) + r;
                if (m < a.M) static_cast<T*>(a.y)[m * a.y_stride + n] = (T)acc[t][f][r];
            }
    }
}

}  // namespace gemm_rs_layer
