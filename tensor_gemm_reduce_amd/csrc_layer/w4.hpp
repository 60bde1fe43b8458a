// w4.hpp -- the product of a few tokens with 4-bit weights:
//   y[m][n] = sum over groups g of s[n][g] sum_{k in g} x[m][k] (q[n][k] - z[n][g])
//
// The weight bytes bound it for a few tokens, so they are laid out once in the order
// the waves consume them and read at full rate; from some 16 tokens on the vector
// instructions that expand weights and apply scales do, beside the MFMAs.
//   - A nibble becomes a 16-bit float by two bit operations per pair: placed in the
//     mantissa of 16 o it reads as (16 + q) o exactly, o a power of two.
//   - The MFMA multiplies x by (16 + q) o; the group's FP32 accumulator starts at
//     -(16 + z) o times the sum of the group's inputs, which is taken once for every
//     column.  No weight is rounded, and none has its zero point subtracted by itself.
//   - The group's accumulator times its scale is added to the result's (FP32), which is
//     divided by o at the end.
//   - o is 1 in F16.  In BF16, whose inputs reach FP32's largest value, 31 x summed over
//     a block's 128 inputs would be an infinity from |x| of some 2^116 on, over groups of
//     32 from 2^118, even where y is small.  o = 2^-12 keeps every such sum below 2^128 for
//     any finite x.  Nothing is lost at the other end: inputs are multiples of 2^-133, so
//     the products are of 2^-145, which FP32 holds down to 2^-149; only the result's own
//     sum is rounded there, by 2^-138 of y at most, a 32nd of BF16's last place.
#pragma once

#include <type_traits>

#include "common.hpp"

namespace gemm_rs_layer {

constexpr int kW4Tile = 16;    // rows of w per tile: the columns of one MFMA
constexpr int kW4Block = 128;  // inputs per block of a tile: 64 lanes x 16 bytes

// Packed weights: tiles x blocks of 1 KiB of nibbles, then the scales, then the
// zero points, each [tile][block][row of the tile][sub], with `subs` (1, 2 or 4)
// scales per row and block.
//   Word t (0..3) of lane l holds row l % 16, inputs 32 t + 8 (l / 16) + 0..7 of
//   the block.  Turned right by w4_turn(type, i) bits it holds inputs 2 i and 2 i + 1
//   at the top of the mantissas of its two halves, so a pair costs a turn (none for
//   i = 0) and one and-or.
struct W4Layout {
    int N, K, group;
    int tiles, blocks, groups, subs;  // groups: per row, as given
    int64_t scale_at, zero_at, bytes;
};

constexpr __device__ int w4_turn(bool bf16, int i) { return i < 2 ? 4 * i : i == 2 ? (bf16 ? 8 : 28) : bf16 ? 28 : 24; }

struct W4PackArgs {
    W4Layout l;
    const uint8_t* q;
    const uint16_t* scales;
    const uint8_t* zeros;
    char* packed;
    int bf16;
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
            const uint32_t at = nib << ((a.bf16 ? 3 : 6) + 16 * (j & 1));
            const int turn = w4_turn(a.bf16, j / 2);
            v |= at << turn | (turn ? at >> (32 - turn) : 0u);
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
    static constexpr float kOne = 0x1p-12f;  // what a weight of 1 is multiplied as
    static constexpr uint32_t kOnes = 0x39803980u;  // it in both halves
    static constexpr uint32_t kMask = 0x00780078u, kMagic = 0x3B803B80u;  // the nibbles' places; 16 of it in both halves
    static constexpr bool kBf16 = true;
    static __device__ __forceinline__ f32x4 mfma(frag a, frag b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ float add2(uint32_t v, float c)  // both halves times kOne, and c
    {
        return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, v), __builtin_bit_cast(bf16x2, kOnes), c, false);
    }
};
template <>
struct W4Type<_Float16> {
    typedef f16x8 frag;
    static constexpr float kOne = 1.f;
    static constexpr uint32_t kOnes = 0x3C003C00u, kMask = 0x03C003C0u, kMagic = 0x4C004C00u;
    static constexpr bool kBf16 = false;
    static __device__ __forceinline__ f32x4 mfma(frag a, frag b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ float add2(uint32_t v, float c)
    {
        return __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, v), __builtin_bit_cast(f16x2, kOnes), c, false);
    }
};

// The eight weights of a word as (16 + q) kOne.  The constants sit in a scalar and a vector
// register: and-or takes neither as a literal, and one scalar.
template <class T>
__device__ __forceinline__ typename W4Type<T>::frag w4_expand(uint32_t w)
{
    uint32_t mask = W4Type<T>::kMask, magic = W4Type<T>::kMagic;
    asm("" : "+s"(mask));
    asm("" : "+v"(magic));
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = ((i ? __builtin_amdgcn_alignbit(w, w, w4_turn(W4Type<T>::kBf16, i)) : w) & mask) | magic;
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

// What a sum of inputs times kOne is multiplied by: all of -(16 + 8) where every zero point is 8, else the sign.
template <bool ZEROS>
constexpr float w4_unit()
{
    return ZEROS ? -1.f : -24.f;
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
    typedef T scales_t __attribute__((ext_vector_type(SUBS)));
    typedef uint8_t zeros_t __attribute__((ext_vector_type(SUBS)));
    scales_t sc[NT];
    zeros_t z[NT];

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
            sc[t] = *reinterpret_cast<const scales_t*>(a.packed + a.l.scale_at + at * 2);
            if constexpr (ZEROS) z[t] = *reinterpret_cast<const zeros_t*>(a.packed + a.l.zero_at + at);
        }
    }
    // g[t][f] += step k (32 inputs) of the block's product with the rows x[f]; after a group's last step acc += its scale
    // times g.  The part of the zero points, -(16 + z) times the sum of a row's inputs, is where g starts: start(u, f)
    // gives that sum of sub-block u times kOne w4_unit.
    template <int MF, class F>
    __device__ __forceinline__ void step(const typename W4Type<T>::frag (&x)[MF], int k, f32x4 (&g)[NT][MF],
                                         f32x4 (&acc)[NT][MF], F start) const
    {
        constexpr int kSteps = 4 / SUBS;  // steps per scale
        const int u = k / kSteps;
        f32x4 s[MF];
        if (k % kSteps == 0)
#pragma unroll
            for (int f = 0; f < MF; ++f) s[f] = start(u, f);
#pragma unroll
        for (int t0 = 0; t0 < NT; t0 += 2) {
#pragma unroll
            for (int t = t0; t < NT && t < t0 + 2; ++t) {
                if (k % kSteps == 0)
#pragma unroll
                    for (int f = 0; f < MF; ++f) g[t][f] = ZEROS ? s[f] * (float)(16 + z[t][u]) : s[f];
                const typename W4Type<T>::frag q = w4_expand<T>(w[t][k]);
#pragma unroll
                for (int f = 0; f < MF; ++f) g[t][f] = W4Type<T>::mfma(x[f], q, g[t][f]);
            }
            if (k % kSteps == kSteps - 1)
#pragma unroll
                for (int t = t0; t < NT && t < t0 + 2; ++t) {
                    const float scale = (float)sc[t][u];
#pragma unroll
                    for (int f = 0; f < MF; ++f) {
#pragma unroll
                        for (int r = 0; r < 4; ++r) acc[t][f][r] = __builtin_fmaf(g[t][f][r], scale, acc[t][f][r]);
                        asm volatile("" : "+v"(acc[t][f]));  // here, not gathered behind the last step with every g kept
                    }
                }
        }
    }
    // The whole block, the sums taken by an MFMA per step for all the tiles at once.
    template <int MF>
    __device__ __forceinline__ void multiply(const typename W4Type<T>::frag (&x)[4][MF], f32x4 (&acc)[NT][MF]) const
    {
        const typename W4Type<T>::frag unit = w4_constant<T>(W4Type<T>::kOne * w4_unit<ZEROS>());
        f32x4 g[NT][MF];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            step(x[k], k, g, acc, [&](int u, int f) {
                f32x4 s = {};
#pragma unroll
                for (int i = u * (4 / SUBS); i < (u + 1) * (4 / SUBS); ++i) s = W4Type<T>::mfma(x[i][f], unit, s);
                return s;
            });
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
// Measured, 7168 x 8192 with groups of 128: 1 row 10.0 us (3.1 TB/s, of which starting and
// ending take 2.5 us), 4 rows 10.7, 24 rows 14.5; 8192 x 1024: 1 row 3.4, 24 rows 4.5.
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
    auto fragments = [&](const vec8<T> (&x)[kLoads], frag (&s)[4][MF]) {
        if constexpr (FEW) {
            const i32x4 v = __builtin_bit_cast(i32x4, x[0]);
            s[0][0] = __builtin_bit_cast(frag, v);
            s[1][0] = __builtin_bit_cast(frag, lanes_down<4>(v));
            s[2][0] = __builtin_bit_cast(frag, lanes_down<8>(v));
            s[3][0] = __builtin_bit_cast(frag, lanes_down<12>(v));
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
                    s[t][f] = *reinterpret_cast<const frag*>(area + (16 * f + l16) * kRow + (((4 * t + r0) ^ l16) * 16));
        }
    };
    const int b0 = (int)((int64_t)a.l.blocks * wave / WAVES), b1 = (int)((int64_t)a.l.blocks * (wave + 1) / WAVES);
    const int whole = min(b1, a.l.K / kW4Block);  // the last block may end past K
    Block w[WA];
    vec8<T> x[XA][kLoads];
    frag s[4][MF];
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
            if (m < a.M) static_cast<T*>(a.y)[m * a.y_stride + n] = (T)(sum[r] / W4Type<T>::kOne);
        }
    }
}

// Many rows: 64 rows x 64 NT columns per workgroup.  Two sets of four waves take half of
// K's blocks each, a wave 64 x 16 NT, and add up through LDS at the end.  A set's rows of
// a block go through LDS (16-byte chunk c of row m at c ^ m % 16), two blocks ahead in
// registers; each wave expands its own weights, once for its 64 rows.  Whoever writes a
// row's inputs also sums them for the zero points: sums by MFMA, as the kernel above takes
// them, would repeat in every wave and cost 1 / NT of the product.
// MFMAs and vector instructions bound it together: two waves share a SIMD, and a pair of
// tiles is scaled right behind its MFMAs, so that the two kinds run after each other more
// than side by side.  7168 x 8192, 500 rows: 71 us (823 TFLOP/s) with groups of 128, when
// MFMAs take 42% of the busy cycles and the rest of the vector instructions 41%; 87 with
// groups of 32 (34% and 60%: four times the scales' multiply-adds); 139 with groups of 32 and
// zero points (21% and 62%: a multiply per start of a group as well, and NT = 4 keeps 32
// registers in scratch; 15 with groups of 64).  6144 x 2048, 500 rows, groups of 32: 22.8 us
// (552 TFLOP/s; 25% and 50%).
constexpr int kW4Rows = 64;

// Adds another lane's value, within 16 lanes.
template <int CTRL>
__device__ __forceinline__ float w4_lanes_add(float v)
{
    return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}

template <class T, int NT, int SUBS, bool ZEROS>
__global__ __launch_bounds__(512, 2) void w4_tile_kernel(const W4Args a)
{
    typedef typename W4Type<T>::frag frag;
    typedef W4Block<T, NT, SUBS, ZEROS> Block;
    constexpr int kRow = kW4Block * 2;  // bytes of a row's block
    struct Stage {
        char x[kW4Rows * kRow];
        float sum[SUBS][kW4Rows];
    };
    __shared__ __attribute__((aligned(16))) char lds[4 * sizeof(Stage)];
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6), set = wave >> 2;
    Stage* const stage = reinterpret_cast<Stage*>(lds) + 2 * set;
    const int tile0 = (blockIdx.y * 4 + (wave & 3)) * NT;
    const int64_t m0 = (int64_t)blockIdx.x * kW4Rows;
    const int chunk = threadIdx.x & 15, r0 = (threadIdx.x & 255) >> 4;
    const int share = a.l.K / kW4Block / 2, b0 = set * share;
    auto xrow = [&](int i) {  // rows past the last read it again, and are not stored
        const int64_t m = m0 + r0 + 16 * i;
        return static_cast<const T*>(a.x) + (m < a.M ? m : a.M - 1) * a.x_stride;
    };
    vec8<T> xr[4];
    auto load_x = [&](int b) {
#pragma unroll
        for (int i = 0; i < 4; ++i) xr[i] = *reinterpret_cast<const vec8<T>*>(xrow(i) + b * kW4Block + chunk * 8);
    };
    auto put_x = [&](Stage& st) {
        float sum[4] = {};  // of the row's sub-block, over the 16 / SUBS lanes that hold it
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const u32x4 v = __builtin_bit_cast(u32x4, xr[i]);
            *reinterpret_cast<u32x4*>(st.x + (r0 + 16 * i) * kRow + ((chunk ^ r0) * 16)) = v;
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[i] = W4Type<T>::add2(v[j], sum[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] = w4_lanes_add<0xB1>(sum[i]);  // lane ^ 1
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] = w4_lanes_add<0x4E>(sum[i]);  // lane ^ 2
        if constexpr (SUBS < 4)
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[i] = w4_lanes_add<0x141>(sum[i]);  // the other four of eight
        if constexpr (SUBS < 2)
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[i] = w4_lanes_add<0x140>(sum[i]);  // the other eight of sixteen
        const float lo = chunk & 1 ? sum[1] : sum[0], hi = chunk & 1 ? sum[3] : sum[2];
        if (chunk % (16 / SUBS) < 4)
            st.sum[chunk / (16 / SUBS)][r0 + 16 * (chunk & 3)] = (chunk & 2 ? hi : lo) * w4_unit<ZEROS>();
    };
    f32x4 acc[NT][4] = {};
    auto multiply = [&](const Stage& st, const Block& w, auto load) {
        frag x[2][4];
        auto read_x = [&](int k) {
#pragma unroll
            for (int f = 0; f < 4; ++f)
                x[k & 1][f] = *reinterpret_cast<const frag*>(st.x + (f * 16 + (lane & 15)) * kRow +
                                                             (((4 * k + (lane >> 4)) ^ (lane & 15)) * 16));
        };
        read_x(0);
        load();
        f32x4 g[NT][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (k < 3) read_x(k + 1);
            w.step(x[k & 1], k, g, acc, [&](int u, int f) {
                return *reinterpret_cast<const f32x4*>(&st.sum[u][f * 16 + 4 * (lane >> 4)]);
            });
        }
    };
    Block w[2];
    if (share > 0) {
        load_x(b0);
        w[0].load(a, tile0, b0);
        if (share > 1) w[1].load(a, tile0, b0 + 1);
        put_x(stage[0]);
        if (share > 1) load_x(b0 + 1);
    }
    for (int j = 0; j < share; j += 2) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (j + i < share) {
                __syncthreads();
                multiply(stage[i], w[i], [&] {
                    if (j + i + 1 < share) put_x(stage[i ^ 1]);
                    if (j + i + 2 < share) load_x(b0 + j + i + 2);
                });
                if (j + i + 2 < share) w[i].load(a, tile0, b0 + j + i + 2);
            }
    }
    // The block without a partner, and the one that ends past K
    const int last = 2 * share + set;
    __syncthreads();
    if (last < a.l.blocks) {
        w[0].load(a, tile0, last);
#pragma unroll
        for (int i = 0; i < 4; ++i) xr[i] = load8(xrow(i), last * kW4Block + chunk * 8, a.l.K);
        put_x(stage[0]);
    }
    __syncthreads();
    if (last < a.l.blocks) multiply(stage[0], w[0], [] {});
    __syncthreads();
    f32x4* const part = reinterpret_cast<f32x4*>(lds) + (wave & 3) * (NT * 4 * 64) + lane;
    static_assert(sizeof(lds) >= 4 * NT * 4 * 64 * 16, "the second set's results");
    if (set)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int f = 0; f < 4; ++f) part[(t * 4 + f) * 64] = acc[t][f];
    __syncthreads();
    if (set) return;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int n = (tile0 + t) * kW4Tile + (lane & 15);
#pragma unroll
        for (int f = 0; f < 4; ++f) {
            const f32x4 y = acc[t][f] + part[(t * 4 + f) * 64];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int64_t m = m0 + f * 16 + 4 * (lane >> 4) + r;
                if (n < a.l.N && m < a.M) static_cast<T*>(a.y)[m * a.y_stride + n] = (T)(y[r] / W4Type<T>::kOne);
            }
        }
    }
}

}  // namespace gemm_rs_layer
