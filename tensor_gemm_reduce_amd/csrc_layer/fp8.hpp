// fp8.hpp -- matrices in e4m3 with a power-of-two scale for each block of 128 inputs,
// and their products, dense and by expert.
//
// The scale is the smallest power of two that brings a block to at most 448, e4m3's
// largest value: quantising then has one rounding, to e4m3, which no reciprocal can
// turn, and the scale is an E8M0 byte, which the scaled MFMA takes beside its operands.
// So the products of a block of 128 are scaled where they are summed, in FP32, without
// a vector instruction, and the matrix instructions alone bound a large product.
// How the instruction orders its inputs inside a block does not matter: both operands
// are read in the same order, and all of a block has one scale.
#pragma once

#include <type_traits>
#include <utility>

#include "common.hpp"

namespace gemm_rs_layer {

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kFp8Block = 128;
constexpr int kFp8MinExp = -126;

// The exponent of a block from the bits of its largest magnitude: E - 8 for 2^E .. 1.75 2^E,
// else E - 7, since 448 = 1.75 2^8.
__device__ __forceinline__ int fp8_exponent(uint32_t top)
{
    const int e = (int)(top >> 23) - 127 - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return e > kFp8MinExp ? e : kFp8MinExp;
}
// A block of zeros has the scale one, and so has a block of NaN: what they hold needs no other, and the lowest costs FP32
// products a second pass.
__device__ __forceinline__ int fp8_block_exponent(uint32_t top) { return top == 0 || top >= 0x7F800000u ? 0 : fp8_exponent(top); }

// Four values times 2^-e as e4m3 bytes; all NaN in a block with an infinity or a NaN.
__device__ __forceinline__ uint32_t fp8_word(float a, float b, float c, float d)
{
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}
constexpr uint32_t kFp8Nan4 = 0x7F7F7F7Fu;

__device__ __forceinline__ float fp8_inverse(int e) { return __uint_as_float((uint32_t)(127 - e) << 23); }

struct Fp8QuantArgs {
    const void* x;
    uint8_t *q, *s;
    int64_t M, stride;  // rows of x
    int K, blocks;      // columns; blocks of 128 of the result's rows
    int pitch;          // bytes from a block's scales to the next one's
    int64_t q_pitch;    // bytes of a row of q
    // transposed: the rows of each expert by themselves
    const int32_t *offsets, *tokens;
    int E;
    int64_t x_rows;
};

// A wave takes 16 rows of one block, 16 lanes and 16 bytes a lane (BF16) for each row.
template <class T>
__global__ __launch_bounds__(256) void fp8_quant_kernel(const Fp8QuantArgs a)
{
    const int lane = threadIdx.x & 63, l16 = lane & 15;
    const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int64_t r0 = id / a.blocks * 16;
    const int kb = (int)(id % a.blocks), col = kb * kFp8Block + l16 * 8;
    vec8<T> v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = r0 + 4 * i + lane / 16;
        v[i] = vec8<T>{};
        if (r < a.M) v[i] = load8(static_cast<const T*>(a.x) + r * a.stride, col, a.K);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = r0 + 4 * i + lane / 16;
        float f[8];
        widen<T>(v[i], f);
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(f[j]) & 0x7FFFFFFFu);
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
        const bool bad = top >= 0x7F800000u;
        const int e = fp8_block_exponent(top);
        const float inv = fp8_inverse(e);
        u32x2 w = {fp8_word(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                   fp8_word(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv)};
        if (bad) w = u32x2{kFp8Nan4, kFp8Nan4};
        if (r < a.M) {
            *reinterpret_cast<u32x2*>(a.q + r * a.q_pitch + col) = w;
            if (l16 == 0) a.s[(int64_t)kb * a.pitch + r] = (uint8_t)(e + 127);
        }
    }
}

// The lane's expert among e0 .. e0 + 63: rows a .. b - 1, within 0 .. M.
__device__ __forceinline__ void expert_rows(const int32_t* offsets, int E, int64_t M, int e, int& a, int& b)
{
    a = b = 0;
    if (e < E) {
        const int m = (int)M;
        a = min(max(offsets[e], 0), m);
        b = min(max(offsets[e + 1], a), m);
    }
}

struct RowTile {
    int e, m0, m1;  // expert, first row, end of the expert's rows
};

// Tile `id` of the experts' rows, `rows` rows a tile, expert by expert; false if there are
// fewer.  For a whole wave, with uniform results.
__device__ __forceinline__ bool find_tile(const int32_t* offsets, int E, int64_t M, int rows, int id, RowTile& t)
{
    const int lane = threadIdx.x & 63;
    int carry = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
        int a, b;
        expert_rows(offsets, E, M, e0 + lane, a, b);
        const int n = (b - a + rows - 1) / rows;
        int s = n;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(s, d);
            if (lane >= d) s += o;
        }
        const uint64_t past = __ballot(carry + s > id);
        if (past) {
            const int at = __ffsll((unsigned long long)past) - 1;
            const int before = carry + __builtin_amdgcn_readlane(s, at) - __builtin_amdgcn_readlane(n, at);
            t.e = e0 + at;
            t.m0 = __builtin_amdgcn_readlane(a, at) + (uni(id) - before) * rows;
            t.m1 = __builtin_amdgcn_readlane(b, at);
            return true;
        }
        carry += __builtin_amdgcn_readlane(s, 63);
    }
    return false;
}

// Tiles of `rows` rows of the experts before `last`.
__device__ __forceinline__ int tiles_before(const int32_t* offsets, int E, int64_t M, int rows, int last)
{
    int n = 0;
    for (int e0 = 0; e0 < last; e0 += 64) {
        int a, b;
        const int e = e0 + (threadIdx.x & 63);
        expert_rows(offsets, E, M, e < last ? e : E, a, b);
        n += (b - a + rows - 1) / rows;
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) n += __shfl_xor(n, d);
    return uni(n);
}

// 128 rows x 64 columns of x as 64 rows of one block: a thread holds 4 rows x 8 columns, the
// columns' maxima meet in LDS, and a column's four bytes go there as one word, from where
// whole rows of the result are written.
template <class T>
__global__ __launch_bounds__(256) void fp8_quant_t_kernel(const Fp8QuantArgs a)
{
    constexpr int kCols = 64, kPitch = kFp8Block + 16;
    __shared__ uint32_t top[kCols];
    __shared__ __attribute__((aligned(16))) uint8_t out[kCols * kPitch];
    const int tid = threadIdx.x, cg = tid % 8, rg = tid / 8, c0 = blockIdx.y * kCols, col = c0 + cg * 8;
    int64_t m0 = (int64_t)blockIdx.x * kFp8Block, m1 = a.M;
    if (a.offsets) {
        RowTile t;
        if (!find_tile(a.offsets, a.E, a.M, kFp8Block, blockIdx.x, t)) return;
        m0 = t.m0;
        m1 = t.m1;
    }
    if (tid < kCols) top[tid] = 0;
    vec8<T> v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        int64_t r = m0 + rg * 4 + i;
        v[i] = vec8<T>{};
        if (r >= m1) continue;
        if (a.tokens) r = a.tokens[r];
        if (r >= 0 && r < a.x_rows) v[i] = load8(static_cast<const T*>(a.x) + r * a.stride, col, a.K);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max(m, __float_as_uint((float)v[i][j]) & 0x7FFFFFFFu);
#pragma unroll
        for (int d = 8; d < 64; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
        if ((tid & 63) < 8) atomicMax(&top[cg * 8 + j], m);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t m = top[cg * 8 + j];
        const bool bad = m >= 0x7F800000u;
        const float inv = fp8_inverse(fp8_block_exponent(m));
        const uint32_t w = fp8_word((float)v[0][j] * inv, (float)v[1][j] * inv, (float)v[2][j] * inv, (float)v[3][j] * inv);
        *reinterpret_cast<uint32_t*>(out + (cg * 8 + j) * kPitch + rg * 4) = bad ? kFp8Nan4 : w;
    }
    __syncthreads();
    const int64_t kb = blockIdx.x;
    if (tid < kCols && c0 + tid < a.K) {
        a.s[kb * a.pitch + c0 + tid] = (uint8_t)(fp8_block_exponent(top[tid]) + 127);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int c = tid / 8 + 32 * i;
        if (c0 + c < a.K)
            *reinterpret_cast<u32x4*>(a.q + (c0 + c) * a.q_pitch + kb * kFp8Block + tid % 8 * 16) =
                *reinterpret_cast<const u32x4*>(out + c * kPitch + tid % 8 * 16);
    }
}

struct Fp8PackArgs {
    const void* w;
    uint8_t *q, *s;
    int N, K, transpose;
    int64_t w_expert, q_expert, s_expert;  // elements, bytes and bytes of an expert
    int64_t q_pitch;
    int pitch;
};

// A workgroup takes a block of 128 x 128: a thread holds eight columns of eight rows 16 apart.
template <class T>
__global__ __launch_bounds__(256) void fp8_pack_kernel(const Fp8PackArgs a)
{
    constexpr int kPitch = kFp8Block + 16;
    __shared__ uint32_t top;
    __shared__ __attribute__((aligned(16))) uint8_t out[kFp8Block * kPitch];
    const int tid = threadIdx.x, cg = tid % 16, rg = tid / 16, n0 = blockIdx.y * kFp8Block, k0 = blockIdx.x * kFp8Block;
    const T* w = static_cast<const T*>(a.w) + blockIdx.z * a.w_expert;
    uint8_t *q = a.q + blockIdx.z * a.q_expert, *s = a.s + blockIdx.z * a.s_expert;
    if (tid == 0) top = 0;
    vec8<T> v[8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int n = n0 + rg + 16 * i;
        v[i] = vec8<T>{};
        if (n < a.N) v[i] = load8(w + (int64_t)n * a.K, k0 + cg * 8, a.K);
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint((float)v[i][j]) & 0x7FFFFFFFu);
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
    __syncthreads();
    if ((tid & 63) == 0) atomicMax(&top, m);
    __syncthreads();
    m = top;
    const bool bad = m >= 0x7F800000u;
    const int e = fp8_block_exponent(m);
    const float inv = fp8_inverse(e);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float f[8];
        widen<T>(v[i], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] *= inv;
        u32x2 b = {fp8_word(f[0], f[1], f[2], f[3]), fp8_word(f[4], f[5], f[6], f[7])};
        if (bad) b = u32x2{kFp8Nan4, kFp8Nan4};
        const int r = rg + 16 * i;
        if (a.transpose) {
#pragma unroll
            for (int j = 0; j < 8; ++j) out[(cg * 8 + j) * kPitch + r] = (uint8_t)(b[j / 4] >> (8 * (j % 4)));
        } else
            *reinterpret_cast<u32x2*>(out + r * kPitch + cg * 8) = b;
    }
    __syncthreads();
    // rows of the result: n, or k where transposed; padding rows of it are not kept, its padding columns are zeros
    const int rows = a.transpose ? a.K : a.N, r0 = a.transpose ? k0 : n0, kb = a.transpose ? blockIdx.y : blockIdx.x;
    if (tid < kFp8Block && r0 + tid < rows) s[(int64_t)kb * a.pitch + r0 + tid] = (uint8_t)(e + 127);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = tid / 8 + 32 * i;
        u32x4 b = *reinterpret_cast<const u32x4*>(out + r * kPitch + tid % 8 * 16);
        if (r0 + r < rows) *reinterpret_cast<u32x4*>(q + (int64_t)(r0 + r) * a.q_pitch + kb * kFp8Block + tid % 8 * 16) = b;
    }
}

// ---- the products -----------------------------------------------------------------------

enum Fp8Mode { kDense = 0, kByExpert = 1, kGather = 2, kSums = 3 };

// out[m][n] = add + sum_k x[m][k] w[n][k].
//   kDense   all rows with one w
//   kByExpert   the rows of each expert with its own; kGather: the row of x is tokens[m]
//   kSums    a result for each expert, the sum over its own blocks of the columns of x and w
struct Fp8Args {
    const uint8_t *x, *w, *xs, *ws;
    const int32_t *offsets, *tokens;
    const float* add;
    void* out;
    int64_t M, x_rows, rows;  // rows of the result; of x; of the experts (kSums)
    int64_t x_pitch, w_pitch, w_expert, ws_expert, out_expert, add_stride, out_stride;
    int64_t xs_bytes, ws_bytes;
    int N, K, E, steps;       // steps of 128 inputs
    int xs_pitch, ws_pitch;
    int tiles_m, tiles_n;
};

// Results in FP32 take every product whole.  For 16-bit results the scaled MFMA does all of it at twice the rate, but it lines the
// products of eight neighbouring inputs up with the largest of them and drops from each what lies below that one's 2^-13
// (measured; the sums with the accumulator are FP32's).  A product has eight bits, so those from 2^-5 of the largest on lose
// nothing; all eight together lose less than 2^-10 of it.  That is a quarter of BF16's half step, 2^-8, and two of F16's, 2^-11: a
// sum that one product makes up nearly alone may be off by that in F16 without cancelling.  On activations and weights: 501 x
// 7168 x 8192 in F16 is 2.100e-4 from the exact results (2-norm) instead of 2.079e-4 with every product whole, and 11% of
// the results round to the other neighbour; 1 x 8192 x 1024 in BF16 1.663e-3 either way, 2%.  FP32's half step is 2^-24, so there the
// operands are multiplied in BF16, at half the rate, and block by block where their scales are past BF16's.
template <class T>
constexpr bool fp8_exact = std::is_same<T, float>::value;

// Which of four scales may have values q 2^e that are no normal BF16 numbers: below 2^-117 the smallest are not, 2^-9 2^e, above
// 2^119 the largest, 448 2^e.  The highest bit of each byte is 0 where the byte's upper four bits are all alike, 2^-127 ..
// 2^-112 and 2^113 and above, which takes the fewest instructions.
__device__ __forceinline__ uint32_t fp8_near(uint32_t s)
{
    const uint32_t d = s ^ (s << 1);
    return d | (d << 1) | (d << 2);
}

__device__ __forceinline__ float fp8_scale(uint32_t byte) { return __uint_as_float((byte & 255u) << 23); }

// Quarter q (eight values) of a fragment times its scale.
__device__ __forceinline__ bf16x8 fp8_to_bf16(const i32x8& f, int q, float scale)
{
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bf16x2 p = i & 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(f[2 * q + i / 2], scale, true)
                               : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(f[2 * q + i / 2], scale, false);
        v[i] = __builtin_bit_cast(uint32_t, p);
    }
    return __builtin_bit_cast(bf16x8, v);
}

template <int... I, class F>
__device__ __forceinline__ void each_of(std::integer_sequence<int, I...>, F f)
{
    (f(std::integral_constant<int, I>()), ...);
}
template <int N, class F>
__device__ __forceinline__ void each(F f)
{
    each_of(std::make_integer_sequence<int, N>(), f);
}

// Tiles of 64 W x 64 W results by 2 x 2 waves of 32 W x 32 W, in steps of 128 inputs, NS stages in LDS.
//   - Stages are loaded into LDS directly, 16-byte chunk c of row r at chunk c ^ r / 2 % 8: 16 consecutive rows, as the
//     fragments are read, lie in different banks.
//   - A wave's LDS row 32 i + r holds matrix row W r + i: the W fragments of a lane then belong to W neighbouring rows,
//     whose scales are one load, and the MFMA picks the byte.  w is the MFMA's first operand, so a lane ends with 4 W
//     neighbouring columns of a row.
//   - A step has two halves of 64 inputs.  While the first is multiplied, the second's fragments are read; then the next
//     step's stage has to have come, and a barrier frees this one; while the second is multiplied, this stage is filled
//     for step s + NS and the next step's first fragments are read.
// W = 4, NS = 2: one workgroup per CU, whose waves have 256 accumulators each.  In 8192^3 (390 .. 415 us, 2.65 .. 2.8
//   PFLOP/s) the matrix instructions are busy for 79% of the cycles, at the 1.8 GHz that the power limit leaves; in 32768 x
//   8192 x 3584 (784 .. 919 us at 2.0 .. 1.6 GHz) for 63%: a quarter of the cycles are waits, and 23% of the requests miss
//   the L2.  One load beside each MFMA: two or four at a time cost 3% and 8%.  Half steps in
//   four stages, with more time for a load to arrive, but half lines a request, are 6% slower (8192^3: 393 / 417 us).
//   It keeps its workgroups for all tiles: the next tile's first stages are on their way before a tile's results are
//   stored (8192 x 8192 x 1024: 72 us, 79 without).
// W = 2, NS = 2: two workgroups per CU.  LDS bounds it: 96 KB a step are 768 cycles at 128 bytes each, the MFMAs 512.
// W = 2, NS = 4: for products of no more tiles than CUs, where a workgroup has the CU to itself and its loads' latency
//   would bound it (501 x 7168 x 8192: 34 us, 48 with two stages).
template <int W, int NS, int MODE>
struct Fp8Tile {
    static constexpr int kRows = 64 * W;
    static constexpr int kOperand = kRows * kFp8Block;
    static constexpr int kStage = 2 * kOperand;
    static constexpr bool kKeeps = W == 4;       // workgroups stay for all tiles
    static constexpr int kArea = 4096;           // of a wave's results on their way out
    static constexpr int kOut = kKeeps ? NS * kStage : 0;              // where the areas begin
    static constexpr int kScale = NS * kStage + (kKeeps ? 4 * kArea : 0);  // and the scales: [wave][stage][1 + W][64 lanes]
    static constexpr int kScaleStage = 256 * (MODE == kGather ? 1 + W : 2);
    static constexpr int kLds = kScale + 4 * NS * kScaleStage;
};

struct Fp8Place {
    int e, n0, s0, s1;  // expert, first column, steps
    int64_t m0, m1;     // first row, end of rows
};

template <int W, int NS, int MODE, bool EXACT>
struct Fp8Run {
    typedef Fp8Tile<W, NS, MODE> Tile;
    static constexpr int kLoads = 2 * W;  // a thread's, of an operand and stage
    static constexpr int kScales = MODE == kGather ? 1 + W : 2;  // loads of a step's scales
    static constexpr int kStep = 2 * kLoads + kScales;
    static constexpr int kMf = W * W;     // MFMAs of a half step, or (EXACT) of a quarter of it

    const Fp8Args& a;
    char *const lds, *put, *put_scales;  // where the wave's loads of a stage begin, and of its scales
    f32x16 (&acc)[W][W];  // [row of x][row of w]
    i32x4 f[2][2 * W][2];  // fragments of w, then of x, in two chunks
    bf16x8 wide[2][EXACT ? 2 * W : 1];  // a quarter of a half step: w's, then x's
    int sx[2][MODE == kGather ? W : 1], sw[2];  // scales of an even and an odd step
    uint32_t far_x = 0, far_w = 0;  // EXACT: the scales' bytes that were not fp8_near (W = 2: w's in the upper half of far_x)
    uint32_t xo[MODE == kGather ? kLoads : 1], wo;  // a thread's chunk of a stage, first or of each load
    uint32_t sxo[MODE == kGather ? W : 1], swo;
    uint32_t get[2][4];  // LDS offsets of the lane's chunks of the first stage: operand, chunk
    __amdgpu_buffer_rsrc_t rx, rw, rsx, rsw;
    int step0, step1;

    __device__ __forceinline__ Fp8Run(const Fp8Args& args, char* l, f32x16 (&c)[W][W]) : a(args), lds(l), acc(c)
    {
        const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6), r = lane & 31, h = lane >> 5;
        put = l + wave * 1024;
        put_scales = l + Tile::kScale + wave * NS * Tile::kScaleStage;
#pragma unroll
        for (int c4 = 0; c4 < 4; ++c4) {  // chunks of half c4 / 2 of a step: 2 h + c4 % 2
            const int at = (4 * (c4 / 2) + 2 * h + c4 % 2) ^ (r / 2 % 8);
            get[0][c4] = ((wave >> 1) * 32 * W + r) * kFp8Block + at * 16;
            get[1][c4] = Tile::kOperand + ((wave & 1) * 32 * W + r) * kFp8Block + at * 16;
        }
    }
    __device__ __forceinline__ void setup(const Fp8Place& p)
    {
        int tid = threadIdx.x;
        __asm__ __volatile__("" : "+v"(tid));  // keeps what follows from being held in registers over all tiles
        const int lane = tid & 63, wave = uni(tid >> 6), wm = wave >> 1, wn = wave & 1;
        // load j: LDS row 32 j + tid / 8, so matrix row `row` + rows_of(j)
        const int chunk = (tid % 8) ^ (tid / 16 % 8), row = W * (tid / 8);
        const int nrows = (int)(a.N - p.n0 < Tile::kRows ? a.N - p.n0 : Tile::kRows);
        const int mrows = (int)(p.m1 - p.m0 < Tile::kRows ? p.m1 - p.m0 : Tile::kRows);
        const int e = MODE == kSums ? 0 : p.e;
        step0 = p.s0;
        step1 = p.s1;
        rw = __builtin_amdgcn_make_buffer_rsrc((void*)(a.w + e * a.w_expert + p.n0 * a.w_pitch), 0, (int)(nrows * a.w_pitch),
                                               kRsrcFlags);
        wo = (uint32_t)row * (uint32_t)a.w_pitch + chunk * 16;
        rsw = __builtin_amdgcn_make_buffer_rsrc((void*)(a.ws + e * a.ws_expert), 0, (int)a.ws_bytes, kRsrcFlags);
        swo = p.n0 + wn * 32 * W + W * (lane & 31);
        if constexpr (MODE == kGather) {
            rx = __builtin_amdgcn_make_buffer_rsrc((void*)a.x, 0, (int)(a.x_rows * a.x_pitch), kRsrcFlags);
            auto token = [&](int r) {
                const int t = r < mrows ? a.tokens[p.m0 + r] : -1;
                return t < a.x_rows ? t : -1;
            };
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const int t = token(row + rows_of(j));
                xo[j] = t >= 0 ? (uint32_t)t * (uint32_t)a.x_pitch + chunk * 16 : kOob;
            }
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const int t = token(wm * 32 * W + W * (lane & 31) + i);
                sxo[i] = t >= 0 ? t : kOob;
            }
        } else {
            rx = __builtin_amdgcn_make_buffer_rsrc((void*)(a.x + p.m0 * a.x_pitch), 0, (int)(mrows * a.x_pitch), kRsrcFlags);
            xo[0] = (uint32_t)row * (uint32_t)a.x_pitch + chunk * 16;
            sxo[0] = (uint32_t)p.m0 + wm * 32 * W + W * (lane & 31);
        }
        rsx = __builtin_amdgcn_make_buffer_rsrc((void*)a.xs, 0, (int)a.xs_bytes, kRsrcFlags);
    }
    static constexpr __device__ int rows_of(int j) { return j / W * 32 * W + j % W; }
    // Load j of the 2 kLoads of inputs k .. k + 127 into stage Q; skip: past() of the step.
    template <int Q>
    __device__ __forceinline__ void load(int j, int k, uint32_t skip) const
    {
        const bool w = j >= kLoads;
        const int i = w ? j - kLoads : j;
        const uint32_t off = (w ? wo + (uint32_t)rows_of(i) * (uint32_t)a.w_pitch
                              : MODE == kGather ? xo[i % (MODE == kGather ? kLoads : 1)]
                                                : xo[0] + (uint32_t)rows_of(i) * (uint32_t)a.x_pitch) | skip;
        lds_void_t* to = (lds_void_t*)(put + Q * Tile::kStage + (w ? Tile::kOperand : 0) + i * 4096);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(w ? rw : rx, to, 16, off, k, 0, 0);
    }
    // Steps past the last read zeros, from an offset past every resource (and not from where their inputs would be): masks,
    // no selects that might become one per lane.
    __device__ __forceinline__ int live(int s) const { return uni((s - step1) >> 31); }
    __device__ __forceinline__ uint32_t past(int s) const { return ~(uint32_t)live(s) & kOob; }
    __device__ __forceinline__ int inputs(int s) const { return (s & live(s)) * kFp8Block; }
    // The scales go through LDS too, a dword for each lane: in registers, the compiler would wait for them, and so for
    // everything before them, by its own count.
    template <int Q>
    __device__ __forceinline__ void load_scales(int s) const
    {
        const uint32_t skip = past(s);
        const int in = s & live(s), kw = in * a.ws_pitch, kx = in * a.xs_pitch;
        auto load = [&](const __amdgpu_buffer_rsrc_t& r, uint32_t off, int k, int slot) {
            lds_void_t* to = (lds_void_t*)(put_scales + Q * Tile::kScaleStage + slot * 256);
            if constexpr (W == 4) __builtin_amdgcn_raw_ptr_buffer_load_lds(r, to, 4, off, k, 0, 0);
            else __builtin_amdgcn_raw_ptr_buffer_load_lds(r, to, 2, off, k, 0, 0);
        };
        load(rsw, swo | skip, kw, 0);
        if constexpr (MODE == kGather) {
#pragma unroll
            for (int i = 0; i < W; ++i) {
                lds_void_t* to = (lds_void_t*)(put_scales + Q * Tile::kScaleStage + (1 + i) * 256);
                const uint32_t off = sxo[i] | skip;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rsx, to, 1, off, kx, 0, 0);
            }
        } else
            load(rsx, sxo[0] | skip, kx, 1);
        __builtin_amdgcn_sched_barrier(0);  // the waits count them
    }
    // Counts the scales of a step in.
    template <int P>
    __device__ __forceinline__ void see_scales(int s)
    {
        uint32_t x = (uint32_t)sx[P & 1][0], w = (uint32_t)sw[P & 1];
        if constexpr (MODE == kGather) {
            x = __builtin_amdgcn_perm((uint32_t)sx[P & 1][1], x, 0x0C0C0400);  // the lowest bytes, side by side
            if constexpr (W == 4)
                x |= __builtin_amdgcn_perm((uint32_t)sx[P & 1][3], (uint32_t)sx[P & 1][2], 0x04000C0C);
        }
        const uint32_t on = P == 0 ? ~0u : (uint32_t)live(s);  // an even step is there
        if constexpr (W == 2) far_x |= on & ~fp8_near((x & 0xFFFFu) | w << 16);
        else {
            far_x |= on & ~fp8_near(x);
            far_w |= on & ~fp8_near(w);
        }
    }
    // Whether one of the wave's rows of x or w has a block of such a scale.
    __device__ __forceinline__ bool far(const Fp8Place& p) const
    {
        const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6), row = W * (lane & 31);
        auto bytes = [&](int64_t left) { return (left <= 0 ? 0u : left >= W ? ~0u >> (32 - 8 * W) : (1u << (8 * (int)left)) - 1) & 0x80808080u; };
        const uint32_t x = bytes(p.m1 - p.m0 - (wave >> 1) * 32 * W - row), w = bytes(a.N - p.n0 - (wave & 1) * 32 * W - row);
        return W == 2 ? __any(far_x & (x | w << 16)) : __any((far_x & x) | (far_w & w));
    }
    template <int Q>
    __device__ __forceinline__ void read_scales()
    {
        const char* p = put_scales + Q * Tile::kScaleStage + (threadIdx.x & 63) * 4;
        sw[Q & 1] = *reinterpret_cast<const int*>(p);
#pragma unroll
        for (int i = 0; i < (MODE == kGather ? W : 1); ++i) sx[Q & 1][i] = *reinterpret_cast<const int*>(p + (1 + i) * 256);
    }
    // chunk c of half u of fragment i (w's, then x's) of stage Q
    template <int Q>
    __device__ __forceinline__ i32x4 read(int u, int i, int c) const
    {
        return *reinterpret_cast<const i32x4*>(lds + Q * Tile::kStage + i % W * 32 * kFp8Block + get[i < W][2 * u + c]);
    }
    template <int U>
    __device__ __forceinline__ i32x8 fragment(int i) const
    {
        return __builtin_shufflevector(f[U][i][0], f[U][i][1], 0, 1, 2, 3, 4, 5, 6, 7);
    }
    // piece i (w's, then x's) of quarter q of half U in BF16, scaled
    template <int U, int P>
    __device__ __forceinline__ void widen_piece(int q, int i)
    {
        const bool w = i < W;
        const int t = w ? i : i - W;
        const uint32_t s = w ? (uint32_t)sw[P & 1] >> (8 * t) : MODE == kGather ? (uint32_t)sx[P & 1][MODE == kGather ? t : 0]
                                                                                : (uint32_t)sx[P & 1][0] >> (8 * t);
        wide[q & 1][i] = fp8_to_bf16(fragment<U>(i), q, fp8_scale(s));
    }
    // the same piece of the quarter after q
    template <int U, int P>
    __device__ __forceinline__ void widen_next(int q, int piece)
    {
        if (q < 3) widen_piece<U, P>(q + 1, piece);
        else if (U == 0) widen_piece<1, P>(0, piece);
        else widen_piece<0, (P + 1) % NS>(0, piece);
    }
    // MFMA M of half U of a step on stage P
    template <int U, int P, int M>
    __device__ __forceinline__ void multiply()
    {
        constexpr int i = M % kMf / W, j = M % W;
        if constexpr (EXACT) {
            constexpr int q = M / kMf, piece = M % kMf;
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wide[q & 1][j], wide[q & 1][W + i], acc[i][j], 0, 0, 0);
            if constexpr (piece < 2 * W) widen_next<U, P>(q, piece);
        } else if constexpr (MODE == kGather)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fragment<U>(j), fragment<U>(W + i), acc[i][j], 0, 0, j,
                                                                         sw[P & 1], 0, sx[P & 1][i]);
        else
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fragment<U>(j), fragment<U>(W + i), acc[i][j], 0, 0, j,
                                                                         sw[P & 1], i, sx[P & 1][0]);
    }
    // This wave's LDS reads have ended, and its memory instructions but the last LEFT; the wait is a builtin: the compiler
    // then knows.
    template <int LEFT>
    static __device__ __forceinline__ void wait()
    {
        constexpr int n = LEFT < 63 ? LEFT : 63;
        __builtin_amdgcn_s_waitcnt((n & 15) | (n >> 4) << 14 | 7 << 4);
    }
    static __device__ __forceinline__ void barrier()
    {
        __asm__ __volatile__("s_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    }
    // Takes the constancy of these from the compiler, which would give every sum with them a register of its own.
    __device__ __forceinline__ void hide()
    {
        __asm__ __volatile__("" : "+v"(wo));
        if constexpr (MODE != kGather) __asm__ __volatile__("" : "+v"(xo[0]));
#pragma unroll
        for (int c = 0; c < 4; ++c) __asm__ __volatile__("" : "+v"(get[0][c]), "+v"(get[1][c]));
    }
    // Step s on stage P.  STORES: those that may still be on their way, issued behind the loads of the step after it.
    template <int P, int STORES>
    __device__ __forceinline__ void step(int s, bool stores)
    {
        constexpr int kAll = EXACT ? 4 * kMf : kMf, kReads = 4 * W, kPer = 2;  // reads beside an MFMA
        hide();
        each<kAll>([&](auto m) {
            constexpr int M = decltype(m)::value;
            multiply<0, P, M>();
#pragma unroll
            for (int i = kPer * M; i < kPer * (M + 1) && i < kReads; ++i) f[1][i / 2][i % 2] = read<P>(1, i / 2, i % 2);
            __builtin_amdgcn_sched_barrier(0);
        });
        if constexpr (EXACT) see_scales<P>(s);
        if (STORES > 0 && stores) wait<(NS - 2) * kStep + STORES>();
        else wait<(NS - 2) * kStep>();
        barrier();
        read_scales<(P + 1) % NS>();
        const uint32_t skip = past(s + NS);
        const int at = inputs(s + NS);
        each<kAll>([&](auto m) {
            constexpr int M = decltype(m)::value;
            multiply<1, P, M>();
#pragma unroll
            for (int i = M * 2 * kLoads / kMf; i < (M + 1) * 2 * kLoads / kMf && i < 2 * kLoads; ++i) load<P>(i, at, skip);
#pragma unroll
            for (int i = kPer * M; i < kPer * (M + 1) && i < kReads; ++i) f[0][i / 2][i % 2] = read<(P + 1) % NS>(0, i / 2, i % 2);
            __builtin_amdgcn_sched_barrier(0);
        });
        load_scales<P>(s + NS);
    }
    // The first NS stages, in the order that the waits count.
    __device__ __forceinline__ void fill()
    {
        each<NS>([&](auto q) {
            constexpr int Q = decltype(q)::value;
            const int at = inputs(step0 + Q);
            const uint32_t skip = past(step0 + Q);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < 2 * kLoads; ++j) load<Q>(j, at, skip);
            __builtin_amdgcn_sched_barrier(0);
            load_scales<Q>(step0 + Q);
        });
    }
    // All steps, behind fill(); stores: STORES stores have been issued since.
    template <int STORES>
    __device__ __forceinline__ void run(bool stores)
    {
        if (STORES > 0 && stores) wait<(NS - 1) * kStep + STORES>();
        else wait<(NS - 1) * kStep>();
        barrier();
#pragma unroll
        for (int i = 0; i < 4 * W; ++i) f[0][i / 2][i % 2] = read<0>(0, i / 2, i % 2);
        read_scales<0>();
        far_x = far_w = 0;
        if constexpr (EXACT)
#pragma unroll
            for (int i = 0; i < 2 * W; ++i) widen_piece<0, 0>(0, i);
        // in twos: a step past the last multiplies the zeros its loads gave
        for (int s = step0; s < step1; s += NS) {
            step<0, STORES>(s, stores && s == step0);
            step<1, 0>(s + 1, false);
            if constexpr (NS == 4) {
                if (s + 2 >= step1) break;
                step<2, 0>(s + 2, false);
                step<3, 0>(s + 3, false);
            }
        }
        wait<0>();
        barrier();
    }
};

// The results of a wave leave through LDS, so that whole lines are stored: 128 bytes of 32 rows at a time, 16-byte chunk c of
// a row at chunk c ^ r.  A lane has 4 W neighbouring columns of a row for each g.  Direct stores of those, 16 bytes in
// each of 64 lines an instruction, were slower: 2048 x 3584 x 8192 66 us instead of 60, 4096^3 64 instead of 56, 8192 x
// 3584 x 2048 in FP32 128 instead of 106.
// Rows that start at whole lines of 128 bytes are stored past the caches, which hold x and w for the tiles to come: 32768 x
// 8192 x 3584 803 us without, 767 with; the gradients of 64 experts' weights, 738 MB in FP32, 360 .. 379 and 321 .. 347.
// Others go through the caches, which join the parts of a line: the same gradients with rows of 2045 instead of 2048 575 us
// past them and 444 so, 8192 x 8185 x 1024 124 and 79, 8192 x 3581 x 2048 in FP32 154 and 107.  Rows at 64 bytes, which
// go with the others, gain or lose (8192 x 8160 x 1024 94 and 78, 32768 x 8160 x 3584 794 and 838).
// area: the wave's own 4 KB; m0, n0: the wave's first row and column.  FULL: no row or column past the end, so that every
// wave has the same number of stores.
// Accumulators stay where they are, in AGPRs and in one piece: the compiler otherwise takes them apart on the way from the
// loop to the stores, and keeps parts of them in scratch memory.
template <int W>
__device__ __forceinline__ void fp8_hold(f32x16 (&acc)[W])
{
#pragma unroll
    for (int j = 0; j < W; ++j) __asm__ __volatile__("" : "+a"(acc[j]));
}

template <int W, class T>
struct Fp8Store {
    static constexpr int kPer = 16 / sizeof(T);    // elements of a chunk
    static constexpr int kCols = 128 / sizeof(T);  // columns at a time
    static constexpr int kChunks = 8;              // of a row
    static constexpr int kRows = 64 / kChunks;     // rows of an instruction
    static constexpr int kStores = W * (32 * W / kCols) * (32 / kRows);
    typedef T chunk_t __attribute__((ext_vector_type(kPer)));
    typedef T out_t __attribute__((ext_vector_type(kPer), aligned(sizeof(T))));

    template <bool FULL>
    static __device__ __forceinline__ void run(const Fp8Args& a, char* area, int64_t shift, int64_t m0, int64_t m1, int n0,
                                               f32x16 (&acc)[W][W])
    {
        int lane = threadIdx.x & 63;
        __asm__ __volatile__("" : "+v"(lane));  // keeps the addresses from being held in registers over all tiles
        const int r = lane & 31, h = lane >> 5, c = lane % kChunks;
        const bool lines = ((reinterpret_cast<uint64_t>(a.out) | (uint64_t)shift * sizeof(T) | (uint64_t)a.out_stride * sizeof(T)) & 127) == 0;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if constexpr (W == 4) fp8_hold<W>(acc[i]);
#pragma unroll
            for (int c0 = 0; c0 < 32 * W; c0 += kCols) {
                __asm__ __volatile__("" ::: "memory");  // the LDS operations of a wave complete in order
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int g = c0 / (8 * W); g < (c0 + kCols) / (8 * W); ++g)
#pragma unroll
                    for (int p = 0; p < 4 * W; p += kPer) {
                        chunk_t v;
#pragma unroll
                        for (int q = 0; q < kPer; ++q) v[q] = (T)acc[i][(p + q) % W][4 * g + (p + q) / W];
                        const int at = (W * (8 * g + 4 * h) - c0 + p) / kPer;
                        *reinterpret_cast<chunk_t*>(area + (r * kChunks + (at ^ (r & (kChunks - 1)))) * 16) = v;
                    }
                __asm__ __volatile__("" ::: "memory");
                __builtin_amdgcn_sched_barrier(0);
                const int n = n0 + c0 + c * kPer;
#pragma unroll
                for (int k = 0; k < 32 / kRows; ++k) {
                    const int row = k * kRows + lane / kChunks;
                    const int64_t m = m0 + W * row + i;
                    out_t v = *reinterpret_cast<const chunk_t*>(area + (row * kChunks + (c ^ (row & (kChunks - 1)))) * 16);
                    if (!FULL && (m >= m1 || n >= a.N)) continue;
                    T* out = static_cast<T*>(a.out) + shift + m * a.out_stride + n;
                    if (FULL || n + kPer <= a.N) {
                        if constexpr (fp8_exact<T>)
                            if (a.add) v += *reinterpret_cast<const out_t*>(a.add + shift + m * a.add_stride + n);
                        if (lines) {  // the empty statements keep the compiler from making one store of the two, through the caches
                            __asm__ __volatile__("" ::: "memory");
                            __builtin_nontemporal_store(v, reinterpret_cast<out_t*>(out));
                            __asm__ __volatile__("" ::: "memory");
                        } else
                            *reinterpret_cast<out_t*>(out) = v;
                    } else {
#pragma unroll
                        for (int q = 0; q < kPer - 1; ++q)
                            if (n + q < a.N) {
                                if constexpr (fp8_exact<T>)
                                    if (a.add) v[q] += a.add[shift + m * a.add_stride + n + q];
                                out[q] = v[q];
                            }
                    }
                }
            }
        }
        __asm__ __volatile__("" ::: "memory");
    }
};

// The results of a wave with scales that may take its values out of BF16, computed again: the products of a block are summed as
// they are, in FP32, and the sum is scaled by both scales at once.  A tile of 32 x 32 at a time, straight from memory: for values
// below 2^-103 and above 2^120, which programs seldom have.  With one such row in every tile 4096 x 4096 x 384 takes 127 us
// instead of 27, 8192 x 8192 x 1024 890 instead of 140; looking for them costs 1 to 3% (501 x 7168 x 8192 59 / 61 us, 8192 x
// 8192 x 1024 134 / 135).
template <int W, int MODE>
__device__ __forceinline__ void fp8_scaled_apart(const Fp8Args& a, const Fp8Place& p, int64_t shift, int64_t m0, int n0)
{
    const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5, e = MODE == kSums ? 0 : p.e;
#pragma unroll 1
    for (int ij = 0; ij < W * W; ++ij) {
        const int i = ij / W, j = ij % W, n = min(n0 + W * r + j, a.N - 1);  // rows past the last are read again, and not stored
        const int64_t m = m0 + W * r + i;
        int64_t row = m < p.m1 ? m : p.m1 - 1;
        bool none = false;
        if constexpr (MODE == kGather) {
            row = a.tokens[row];
            none = row < 0 || row >= a.x_rows;
            if (none) row = 0;
        }
        const uint8_t *x = a.x + row * a.x_pitch + 64 * h, *xs = a.xs + row;
        const uint8_t *w = a.w + e * a.w_expert + n * a.w_pitch + 64 * h, *ws = a.ws + e * a.ws_expert + n;
        f32x16 sum = {};
#pragma unroll 1
        for (int64_t s = p.s0; s < p.s1; ++s) {
            const int ex = xs[s * a.xs_pitch], ew = ws[s * a.ws_pitch];
            f32x16 part = {};
#pragma unroll
            for (int c = 0; c < 4; c += 2) {
                i32x4 fx[2], fw[2];
#pragma unroll
                for (int d = 0; d < 2; ++d) {
                    fx[d] = none ? i32x4{} : *reinterpret_cast<const i32x4*>(x + s * kFp8Block + (c + d) * 16);
                    fw[d] = *reinterpret_cast<const i32x4*>(w + s * kFp8Block + (c + d) * 16);
                }
                const i32x8 qx = __builtin_shufflevector(fx[0], fx[1], 0, 1, 2, 3, 4, 5, 6, 7);
                const i32x8 qw = __builtin_shufflevector(fw[0], fw[1], 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    part = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fp8_to_bf16(qw, q, 1.f), fp8_to_bf16(qx, q, 1.f), part, 0, 0, 0);
            }
#pragma unroll
            for (int g = 0; g < 16; ++g) sum[g] += ldexpf(part[g], ex + __shfl(ew, 8 * (g / 4) + 4 * h + g % 4) - 254);
        }
        if (m < p.m1) {
#pragma unroll
            for (int g = 0; g < 16; ++g) {
                const int at = n0 + W * (8 * (g / 4) + 4 * h + g % 4) + j;
                if (at >= a.N) continue;
                float v = sum[g];
                if (a.add) v += a.add[shift + m * a.add_stride + at];
                static_cast<float*>(a.out)[shift + m * a.out_stride + at] = v;
            }
        }
    }
}

// Where tile `id` of tiles_m x tiles_n is: groups of four tile rows, column by column, so that the 32 tiles an XCD works on
// at a time share rows of x and of w, and the group's rows of x (3.7 MB at 3584 inputs) stay in its L2 while the columns go
// by: 32768 x 8192 x 3584 takes 816 / 798 / 870 us with groups of 3 / 4 / 8, 8192^3 402 / 391 / 391.
__device__ __forceinline__ void fp8_place(int id, int tiles_m, int tiles_n, int& tm, int& tn)
{
    const int per = 4 * tiles_n, g = id / per, left = tiles_m - 4 * g, rows = left < 4 ? left : 4, r = id - g * per;
    tm = 4 * g + r % rows;
    tn = r / rows;
}

// EXACT: quarters of the fragments are turned to BF16, scaled, beside the MFMAs of the quarter before.  BF16 holds every value
// q 2^e with e = -117 .. 119 as a normal number; a wave that has met a scale past fp8_near's computes its results again.
template <int W, int NS, int MODE, class T>
__global__ __launch_bounds__(256, W == 4 || NS == 4 ? 1 : 2) void fp8_kernel(const Fp8Args a)
{
    typedef Fp8Tile<W, NS, MODE> Tile;
    typedef Fp8Store<W, T> Store;
    extern __shared__ __attribute__((aligned(1024))) char lds[];
    constexpr bool kGrouped = MODE == kByExpert || MODE == kGather;
    const int wave = uni(threadIdx.x >> 6);
    const int tiles_m = kGrouped ? tiles_before(a.offsets, a.E, a.M, Tile::kRows, a.E) : a.tiles_m;
    // Workgroups are dealt to the 8 XCDs in turn: those of one XCD take neighbouring tiles, an eighth of all, or of each
    // expert's where those differ in their steps.
    const int all = tiles_m * a.tiles_n, per = (all + 7) / 8, mine = (int)gridDim.x / 8;
    const int first = (int)blockIdx.x % 8 * per;
    auto place = [&](int& i, Fp8Place& p) {
        p.e = 0;
        if constexpr (MODE == kSums)
            while (i / per < a.E && first + i % per >= all) i += mine;  // an XCD's eighth may be short
        if (MODE == kSums ? i / per >= a.E : i >= per) return false;
        int id = first + i % per;
        if (id >= all) return false;
        p.s0 = 0;
        p.s1 = a.steps;
        if constexpr (MODE == kSums) {
            p.e = i / per;
            p.s0 = tiles_before(a.offsets, a.E, a.rows, kFp8Block, p.e);
            p.s1 = tiles_before(a.offsets, a.E, a.rows, kFp8Block, p.e + 1);
        }
        int tm, tn;
        fp8_place(id, tiles_m, a.tiles_n, tm, tn);
        p.n0 = tn * Tile::kRows;
        p.m0 = (int64_t)tm * Tile::kRows;
        p.m1 = a.M;
        if constexpr (kGrouped) {
            RowTile t;
            if (!find_tile(a.offsets, a.E, a.M, Tile::kRows, tm, t)) return false;
            p.e = t.e;
            p.m0 = t.m0;
            p.m1 = t.m1;
        }
        return true;
    };
    int i = (int)blockIdx.x / 8;
    Fp8Place p;
    if (!place(i, p)) return;
    f32x16 acc[W][W];
    Fp8Run<W, NS, MODE, fp8_exact<T>> run(a, lds, acc);
    run.setup(p);
    run.fill();
    bool full = false;
    for (;;) {
#pragma unroll
        for (int u = 0; u < W; ++u)
#pragma unroll
            for (int v = 0; v < W; ++v) acc[u][v] = f32x16{};
        run.template run<Tile::kKeeps ? Store::kStores : 0>(full);
        if constexpr (W == 4)
#pragma unroll
            for (int u = 0; u < W; ++u) fp8_hold<W>(acc[u]);
        const int64_t shift = MODE == kSums ? p.e * a.out_expert : 0, m0 = p.m0 + (wave >> 1) * 32 * W, m1 = p.m1;
        const int n0 = p.n0 + (wave & 1) * 32 * W;
        const bool far = fp8_exact<T> && run.far(p);
        const Fp8Place at = p;
        bool more = false;
        if constexpr (Tile::kKeeps) {
            i += mine;
            more = place(i, p);
            if (more) {
                run.setup(p);
                run.fill();
            }
        }
        char* area = lds + Tile::kOut + wave * Tile::kArea;
        full = m0 + 32 * W <= m1 && n0 + 32 * W <= a.N && !far;
        if (far) {
            if constexpr (fp8_exact<T>) fp8_scaled_apart<W, MODE>(a, at, shift, m0, n0);
        } else if (full) Store::template run<true>(a, area, shift, m0, m1, n0, acc);
        else Store::template run<false>(a, area, shift, m0, m1, n0, acc);
        if (!more) break;
    }
}

// Few rows: a workgroup computes 16 columns for up to 16 MF rows, its waves split the blocks of
// 128 inputs and add up through LDS in wave order.  The weights' bytes bound it: each wave
// keeps kAhead blocks of them in flight, straight into the MFMA's registers (16 rows x 64
// bytes an instruction).  X is the type of x: e4m3 as it is, or what a lane turns to its part of
// a fragment by itself: 32 values of a row, whose block's scale it shares with three lanes.
// 1 x 8192 x 1024 from BF16 takes 5.1 us so and 5.7 with a kernel before it, calls in a row.
constexpr int kFewTile = 16;

struct Fp8Few;  // as X: e4m3

template <class X, int MF>
struct FewInput {
    vec8<X> v[MF][4];
    __device__ __forceinline__ void load(const Fp8Args& a, const char* const (&x)[MF], const uint8_t* const (&)[MF], int kb, int q)
    {
        const int col = kb * kFp8Block + 16 * q;
        if ((kb + 1) * kFp8Block <= a.K) {  // no branch between the loads, which would be a wait too
#pragma unroll
            for (int f = 0; f < MF; ++f)
#pragma unroll
                for (int h = 0; h < 4; ++h)
                    v[f][h] = *reinterpret_cast<const vec8<X>*>(reinterpret_cast<const X*>(x[f]) + col + 64 * (h / 2) + 8 * (h % 2));
            return;
        }
#pragma unroll
        for (int f = 0; f < MF; ++f)
#pragma unroll
            for (int h = 0; h < 4; ++h)
                v[f][h] = load8(reinterpret_cast<const X*>(x[f]), col + 64 * (h / 2) + 8 * (h % 2), a.K);
    }
    __device__ __forceinline__ i32x8 fragment(int f, int& scale) const
    {
        float g[4][8];
        uint32_t top = 0;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            widen<X>(v[f][h], g[h]);
#pragma unroll
            for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(g[h][j]) & 0x7FFFFFFFu);
        }
        top = max(top, (uint32_t)__shfl_xor((int)top, 16));
        top = max(top, (uint32_t)__shfl_xor((int)top, 32));
        const bool bad = top >= 0x7F800000u;
        const int e = fp8_block_exponent(top);
        const float inv = fp8_inverse(e);
        scale = e + 127;
        i32x8 w;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            w[2 * h] = (int)(bad ? kFp8Nan4 : fp8_word(g[h][0] * inv, g[h][1] * inv, g[h][2] * inv, g[h][3] * inv));
            w[2 * h + 1] = (int)(bad ? kFp8Nan4 : fp8_word(g[h][4] * inv, g[h][5] * inv, g[h][6] * inv, g[h][7] * inv));
        }
        return w;
    }
};
template <int MF>
struct FewInput<Fp8Few, MF> {
    i32x4 v[MF][2];
    int s[MF];
    __device__ __forceinline__ void load(const Fp8Args& a, const char* const (&x)[MF], const uint8_t* const (&xs)[MF], int kb, int q)
    {
#pragma unroll
        for (int f = 0; f < MF; ++f) {
            const char* p = x[f] + (int64_t)kb * kFp8Block + q * 16;
            v[f][0] = *reinterpret_cast<const i32x4*>(p);
            v[f][1] = *reinterpret_cast<const i32x4*>(p + 64);
            s[f] = xs[f][(int64_t)kb * a.xs_pitch];
        }
    }
    __device__ __forceinline__ i32x8 fragment(int f, int& scale) const
    {
        scale = s[f];
        return __builtin_shufflevector(v[f][0], v[f][1], 0, 1, 2, 3, 4, 5, 6, 7);
    }
};

template <int WAVES, int MF, int MODE, class X, class T>
__global__ __launch_bounds__(64 * WAVES) void fp8_few_kernel(const Fp8Args a)
{
    constexpr int kAhead = sizeof(FewInput<X, MF>) > 80 ? 2 : 4;
    __shared__ __attribute__((aligned(16))) f32x4 part[WAVES][MF][64];
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6), r = lane & 15, q = lane >> 4;
    const int n0 = blockIdx.x * kFewTile;
    int e = 0;
    int64_t m0 = (int64_t)blockIdx.y * (16 * MF), m1 = a.M;
    if constexpr (MODE != kDense) {
        RowTile t;
        if (!find_tile(a.offsets, a.E, a.M, 16 * MF, blockIdx.y, t)) return;
        e = t.e;
        m0 = t.m0;
        m1 = t.m1;
    }
    const int n = min(n0 + r, a.N - 1);  // columns and rows past the last are read again, and not stored
    const uint8_t* w = a.w + e * a.w_expert + n * a.w_pitch + q * 16;
    const uint8_t* ws = a.ws + e * a.ws_expert + n;
    const char* x[MF];
    const uint8_t* xs[MF];
    bool none[MF];  // kGather: the row has no input, as in fp8_kernel
#pragma unroll
    for (int f = 0; f < MF; ++f) {
        none[f] = false;
        int64_t m = m0 + 16 * f + r;
        m = m < m1 ? m : m1 - 1;
        if constexpr (MODE == kGather) {
            m = a.tokens[m];
            none[f] = m < 0 || m >= a.x_rows;
            if (none[f]) m = 0;
        }
        x[f] = reinterpret_cast<const char*>(a.x) + m * a.x_pitch;
        xs[f] = a.xs + m;
    }
    struct Block {
        i32x4 w[2];
        int ws;
        FewInput<X, MF> x;
    } b[kAhead];
    auto load = [&](Block& c, int kb) {
        const int64_t at = (int64_t)kb * kFp8Block;
        c.w[0] = *reinterpret_cast<const i32x4*>(w + at);
        c.w[1] = *reinterpret_cast<const i32x4*>(w + at + 64);
        c.ws = ws[(int64_t)kb * a.ws_pitch];
        c.x.load(a, x, xs, kb, q);
    };
    f32x4 acc[MF] = {};
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (wave + i * WAVES < a.steps) load(b[i], wave + i * WAVES);
    for (int kb = wave; kb < a.steps; kb += kAhead * WAVES) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int at = kb + i * WAVES;
            if (at >= a.steps) break;
            const i32x8 fw = __builtin_shufflevector(b[i].w[0], b[i].w[1], 0, 1, 2, 3, 4, 5, 6, 7);
            i32x8 fx[MF];
            int scale[MF];
#pragma unroll
            for (int f = 0; f < MF; ++f) {
                fx[f] = b[i].x.fragment(f, scale[f]);
                if (MODE == kGather && none[f]) fx[f] = i32x8{};
            }
            bool far = false;
            if constexpr (fp8_exact<T>) {
                static_assert(MF <= 2, "a word has room for three scales");
                const uint32_t all = (uint32_t)b[i].ws << 24 | (uint32_t)scale[MF - 1] << 16 | (uint32_t)scale[0] << 8;
                far = __any((~fp8_near(all) & 0x80808000u) != 0);
            }
            if (far) {  // a scale that may take values out of BF16: the block's sum is scaled
#pragma unroll
                for (int f = 0; f < MF; ++f) {
                    f32x4 sum = {};
#pragma unroll
                    for (int p = 0; p < 4; ++p)
                        sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp8_to_bf16(fw, p, 1.f), fp8_to_bf16(fx[f], p, 1.f), sum, 0, 0, 0);
#pragma unroll
                    for (int c = 0; c < 4; ++c) acc[f][c] += ldexpf(sum[c], scale[f] + __shfl(b[i].ws, 4 * q + c) - 254);
                }
            } else {
#pragma unroll
                for (int f = 0; f < MF; ++f) {
                    if constexpr (fp8_exact<T>) {
#pragma unroll
                        for (int p = 0; p < 4; ++p)
                            acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp8_to_bf16(fw, p, fp8_scale(b[i].ws)),
                                                                             fp8_to_bf16(fx[f], p, fp8_scale(scale[f])), acc[f], 0, 0, 0);
                    } else
                        acc[f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fw, fx[f], acc[f], 0, 0, 0, b[i].ws, 0, scale[f]);
                }
            }
            if (at + kAhead * WAVES < a.steps) load(b[i], at + kAhead * WAVES);
        }
    }
#pragma unroll
    for (int f = 0; f < MF; ++f) part[wave][f][lane] = acc[f];
    __syncthreads();
    for (int i = threadIdx.x; i < MF * 64; i += 64 * WAVES) {
        f32x4 s = part[0][i / 64][lane];
#pragma unroll
        for (int v = 1; v < WAVES; ++v) s += part[v][i / 64][lane];
        const int64_t m = m0 + 16 * (i / 64) + r;
        if (m >= m1) continue;
        T* out = static_cast<T*>(a.out) + m * a.out_stride;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int at = n0 + 4 * q + c;
            if (at >= a.N) break;
            float v = s[c];
            if constexpr (fp8_exact<T>)
                if (a.add) v += a.add[m * a.add_stride + at];
            out[at] = (T)v;
        }
    }
}

}  // namespace gemm_rs_layer
