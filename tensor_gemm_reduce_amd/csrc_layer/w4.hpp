// w4.hpp -- the product of a few tokens with 4-bit weights:
//   y[m][n] = sum over groups g of s[n][g] sum_{k in g} x[m][k] (q[n][k] - z[n][g])
//
// The weight bytes bound it (at up to about 64 tokens), so they are laid out once
// in the order the waves consume them, and everything else is arranged around
// reading them at full rate.
//   - A nibble becomes a 16-bit float by two bit operations per pair: placed in the
//     mantissa of 16.0 it reads as 16 + q exactly.
//   - The MFMA multiplies x by 16 + q, a second one by the constant -(16 + z), both
//     into the group's FP32 accumulator, so no vector instruction subtracts the zero
//     point and nothing is rounded before the scale.
//   - The group's accumulator times its scale (FP32) is added to the result's.
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

// -(16 + z) in all eight places.
template <class T>
__device__ __forceinline__ typename W4Type<T>::frag w4_offset(uint32_t z)
{
    uint32_t v = ((z | (z << 16)) << W4Type<T>::kShift) | W4Type<T>::kMagic | 0x80008000u;
    return __builtin_bit_cast(typename W4Type<T>::frag, (u32x4{v, v, v, v}));
}

struct W4Args {
    W4Layout l;
    const char* packed;
    const void* x;
    void* y;
    int64_t M, x_stride, y_stride;
};

// A workgroup computes NT tiles of 16 columns for up to 16 MF rows; its waves
// split the blocks of K and add up through LDS at the end, in wave order.
template <class T, int WAVES, int NT, int MF, int SUBS, bool ZEROS>
__global__ __launch_bounds__(64 * WAVES) void w4_kernel(const W4Args a)
{
    typedef typename W4Type<T>::frag frag;
    constexpr int kSteps = 4 / SUBS;  // MFMA steps (32 inputs) per scale
    __shared__ f32x4 part[WAVES][NT][MF][64];
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6);
    const int tile0 = blockIdx.x * NT;
    const int64_t m0 = (int64_t)blockIdx.y * (16 * MF);
    f32x4 acc[NT][MF] = {};
    // rows past the last read it again; their results are not stored
    const T* xrow[MF];
#pragma unroll
    for (int f = 0; f < MF; ++f) {
        int64_t m = m0 + f * 16 + (lane & 15);
        m = m < a.M ? m : a.M - 1;
        xrow[f] = static_cast<const T*>(a.x) + m * a.x_stride;
    }
    const int b0 = (int)((int64_t)a.l.blocks * wave / WAVES), b1 = (int)((int64_t)a.l.blocks * (wave + 1) / WAVES);
    for (int b = b0; b < b1; ++b) {
        u32x4 w[NT];
        float sc[NT][SUBS];
        uint32_t z[NT][SUBS];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int tile = min(tile0 + t, a.l.tiles - 1);
            const int64_t tb = (int64_t)tile * a.l.blocks + b;
            w[t] = *reinterpret_cast<const u32x4*>(a.packed + (tb * 64 + lane) * 16);
            const int64_t at = tb * (kW4Tile * SUBS) + (lane & 15) * SUBS;
#pragma unroll
            for (int s = 0; s < SUBS; ++s) {
                sc[t][s] = (float)reinterpret_cast<const T*>(a.packed + a.l.scale_at)[at + s];
                z[t][s] = ZEROS ? reinterpret_cast<const uint8_t*>(a.packed + a.l.zero_at)[at + s] : 8u;
            }
        }
        frag x[MF][4];
#pragma unroll
        for (int f = 0; f < MF; ++f)
#pragma unroll
            for (int t = 0; t < 4; ++t)
                x[f][t] = __builtin_bit_cast(frag, load8(xrow[f], b * kW4Block + t * 32 + (lane >> 4) * 8, a.l.K));
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int s = 0; s < SUBS; ++s) {
                const frag off = w4_offset<T>(z[t][s]);
                f32x4 g[MF] = {};
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
                    const frag b8 = w4_expand<T>(w[t][s * kSteps + k]);
#pragma unroll
                    for (int f = 0; f < MF; ++f) {
                        g[f] = W4Type<T>::mfma(x[f][s * kSteps + k], b8, g[f]);
                        g[f] = W4Type<T>::mfma(x[f][s * kSteps + k], off, g[f]);
                    }
                }
#pragma unroll
                for (int f = 0; f < MF; ++f) acc[t][f] += g[f] * sc[t][s];
            }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int f = 0; f < MF; ++f) part[wave][t][f][lane] = acc[t][f];
    __syncthreads();
    // lane l of a tile holds rows 4 (l / 16) .. + 3 of column l % 16
    for (int i = threadIdx.x; i < NT * MF * 64; i += 64 * WAVES) {
        const int l = i & 63, f = (i >> 6) % MF, t = (i >> 6) / MF;
        f32x4 s = part[0][t][f][l];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) s += part[w][t][f][l];
        const int n = (tile0 + t) * kW4Tile + (l & 15);
        if (n >= a.l.N) continue;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int64_t m = m0 + f * 16 + 4 * (l >> 4) + r;
            if (m < a.M) static_cast<T*>(a.y)[m * a.y_stride + n] = (T)s[r];
        }
    }
}

}  // namespace gemm_rs_layer
