// checkpoint.hpp -- an activation kept in 8 bits for the backward pass, and the
// weight gradient computed from it.
//
// Blocks of 32 columns share a power-of-two scale 2^e, e = floor(log2(max|x|)) - 6,
// and hold q = round(x 2^-e) in -127 .. 127.  Powers of two make the scaling exact
// (one rounding, to the integer, which no reciprocal can turn) and q 2^e a value
// with seven significant bits, which BF16 holds exactly: the product below then
// has no rounding of its operands.
#pragma once

#include "common.hpp"

namespace gemm_rs_layer {

constexpr int kCkptNan = 127;
constexpr int kMinExp = -126;

__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// 2^e of a block, NaN for a block marked so
__device__ __forceinline__ float block_scale(int e) { return e == kCkptNan ? __uint_as_float(0x7FC00000u) : pow2(e); }

struct CkptArgs {
    const void* x;   // pack: source
    void* out;       // unpack: target
    int8_t *q, *e;
    int64_t rows, stride;
    int K, chunks;   // columns; 16-column chunks of a padded row
};

constexpr int kCkptThreads = 256;

// Row and chunk of this thread: the workgroup's first chunk is divided by the
// chunks per row once (64 bits), a thread's distance from it in 32 bits.
__device__ __forceinline__ bool ckpt_place(const CkptArgs& a, int64_t& row, int& chunk)
{
    const int64_t base = (int64_t)blockIdx.x * kCkptThreads;
    const int64_t r0 = base / a.chunks;
    const uint32_t c = (uint32_t)(base - r0 * a.chunks) + threadIdx.x;
    row = r0 + c / (uint32_t)a.chunks;
    chunk = (int)(c % (uint32_t)a.chunks);
    return row < a.rows;
}

// A thread quantises 16 columns; the two threads of a block (neighbouring lanes:
// a row has an even number of chunks) exchange their maxima.  Bytes bound this kernel and
// the next: 32768 x 3584 in BF16, 356 MB each, 61 .. 71 us (5.0 .. 5.8 TB/s).
template <class T>
__global__ __launch_bounds__(kCkptThreads) void ckpt_pack_kernel(const CkptArgs a)
{
    int64_t row;
    int chunk;
    const bool in = ckpt_place(a, row, chunk);
    float v[16] = {};
    if (in) {
        const T* src = static_cast<const T*>(a.x) + row * a.stride;
        float lo[8], hi[8];
        widen<T>(load8(src, chunk * 16, a.K), lo);
        widen<T>(load8(src, chunk * 16 + 8, a.K), hi);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] = lo[j];
            v[8 + j] = hi[j];
        }
    }
    uint32_t top = 0;  // bit patterns of magnitudes order like the magnitudes, infinities and NaN last
#pragma unroll
    for (int j = 0; j < 16; ++j) top = max(top, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    top = max(top, (uint32_t)__shfl_xor((int)top, 1));
    const int field = (int)(top >> 23);
    const int e = field == 255 ? kCkptNan : max(field - 127 - 6, kMinExp);
    const float inv = field == 255 ? 0.f : pow2(-e);
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t b = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // limited first, then rounded by adding 1.5 2^23: the low byte of the sum
            // is the integer.  A marked block stores zeros.
            const float s = field == 255 ? 0.f : __builtin_amdgcn_fmed3f(v[k * 4 + j] * inv, -127.f, 127.f);
            b |= (__float_as_uint(s + 12582912.f) & 0xFFu) << (8 * j);
        }
        w[k] = b;
    }
    if (!in) return;
    const int64_t at = (row * a.chunks + chunk) * 16;
    *reinterpret_cast<u32x4*>(a.q + at) = u32x4{w[0], w[1], w[2], w[3]};
    if ((chunk & 1) == 0) a.e[at / 32] = (int8_t)e;
}

__device__ __forceinline__ float byte_value(uint32_t w, int j) { return (float)(int8_t)(w >> (8 * j)); }

template <class T>
__global__ __launch_bounds__(kCkptThreads) void ckpt_unpack_kernel(const CkptArgs a)
{
    int64_t row;
    int chunk;
    if (!ckpt_place(a, row, chunk)) return;
    const int64_t at = (row * a.chunks + chunk) * 16;
    const u32x4 w = *reinterpret_cast<const u32x4*>(a.q + at);
    const float s = block_scale(a.e[at / 32]);
    T* dst = static_cast<T*>(a.out) + row * a.stride;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = byte_value(w[half * 2 + j / 4], j % 4) * s;
        store8(dst, chunk * 16 + half * 8, a.K, f);
    }
}

// ---- weight gradient -----------------------------------------------------------

struct WgradArgs {
    const void* dy;
    const int8_t *q, *e;
    const float* add;
    void* dw;
    int64_t M, dy_stride, add_stride, dw_stride;
    int N, K, Kp;
    int out_f32;
};

template <class T>
struct Mfma;
template <>
struct Mfma<__bf16> {
    typedef bf16x8 frag;
    static __device__ __forceinline__ f32x16 run(frag a, frag b, f32x16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
};
template <>
struct Mfma<_Float16> {
    typedef f16x8 frag;
    static __device__ __forceinline__ f32x16 run(frag a, frag b, f32x16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    }
};

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

// Eight tokens of one column for this lane from a tile stored token-major (16-bit
// elements, `pitch` bytes a row): two transposed reads, each of which takes four
// rows of 16 columns per 16 lanes (lane i addresses row i / 4, columns 4 (i % 4) ..,
// and receives column i of the four rows).
template <class F>
__device__ __forceinline__ F read_column8(const char* p, int pitch)
{
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(p + 4 * pitch));
    const s16x8 v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(F, v);
}

// A lane of a 32 x 32 block of accumulators holds row n (lane % 32), and per group of
// four accumulators four consecutive columns k.  Results leave through LDS so that
// 32 WK / 4 lanes store one row's columns side by side: `area` is the wave's own,
// 32 rows x 32 WK floats, 16-byte chunk c of row r at c ^ r.
template <class T, int WK>
__device__ __forceinline__ void wgrad_store_rows(const WgradArgs& a, char* area, int n0, int k0, const f32x16 (&acc)[WK])
{
    constexpr int kPer = 8 * WK, kRows = 64 / kPer;  // lanes per row, rows per instruction
    typedef float f4 __attribute__((ext_vector_type(4), aligned(4)));
    typedef T t4 __attribute__((ext_vector_type(4), aligned(2)));
    const int lane = threadIdx.x & 63, r = lane & 31, half = lane >> 5;
    __asm__ __volatile__("" ::: "memory");
#pragma unroll
    for (int j = 0; j < WK; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g)
            *reinterpret_cast<f32x4*>(area + (r * kPer + ((8 * j + 2 * g + half) ^ (r & (kPer - 1)))) * 16) =
                f32x4{acc[j][4 * g], acc[j][4 * g + 1], acc[j][4 * g + 2], acc[j][4 * g + 3]};
    // the LDS operations of a wave complete in order
    __asm__ __volatile__("" ::: "memory");
    const int c = lane % kPer, k = k0 + 4 * c;
#pragma unroll 4
    for (int i = 0; i < 32 / kRows; ++i) {
        const int row = i * kRows + lane / kPer, n = n0 + row;
        f32x4 v = *reinterpret_cast<const f32x4*>(area + (row * kPer + (c ^ (row & (kPer - 1)))) * 16);
        if (n >= a.N || k >= a.K) continue;
        if (k + 4 <= a.K) {
            if (a.add) v += *reinterpret_cast<const f4*>(a.add + n * a.add_stride + k);
            if (a.out_f32)
                *reinterpret_cast<f4*>(static_cast<float*>(a.dw) + n * a.dw_stride + k) = v;
            else
                *reinterpret_cast<t4*>(static_cast<T*>(a.dw) + n * a.dw_stride + k) = t4{(T)v[0], (T)v[1], (T)v[2], (T)v[3]};
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e) {
                if (k + e >= a.K) break;
                float x = v[e];
                if (a.add) x += a.add[n * a.add_stride + k + e];
                if (a.out_f32) static_cast<float*>(a.dw)[n * a.dw_stride + k + e] = x;
                else static_cast<T*>(a.dw)[n * a.dw_stride + k + e] = (T)x;
            }
        }
    }
    __asm__ __volatile__("" ::: "memory");
}

constexpr int kWgThreads = 256;

// dw = dy^T x^ for any alignment and stride of dy (wgrad_kernel below takes words):
// 128 x 128 outputs per workgroup, four waves of 64 x 64, 32 tokens a step.  Both operands
// are token-major in memory, the MFMA wants eight tokens of a column in a lane: the tiles
// go into LDS as they are and are read transposed.  The checkpoint is expanded to T between
// its load and LDS.  An odd N or row stride leaves every other row off the words, so rows
// are loaded at two-byte alignment, and no tile is cut: 4096 x 4095 x 1024 takes 360 us (65
// with 4096 columns and the kernel below), 512 x 8191 x 1024 55 (21), and 16384 x 511 x 256,
// eight workgroups, 1404 (23).
constexpr int kWgTile = 128, kWgStep = 32;
constexpr int kWgPitch = kWgTile * 2 + 64;  // rows 16 banks apart: the four rows of a transposed read differ

template <class T>
__global__ __launch_bounds__(kWgThreads) void wgrad_any_kernel(const WgradArgs a)
{
    typedef typename Mfma<T>::frag frag;
    __shared__ __attribute__((aligned(16))) char lds[32 * 1024];
    static_assert(2 * kWgStep * kWgPitch <= (int)sizeof(lds), "stage");
    char *const lds_y = lds, *const lds_x = lds + kWgStep * kWgPitch;
    const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
    const int n0 = blockIdx.y * kWgTile, k0 = blockIdx.x * kWgTile;
    const int wn = (wave >> 1) * 64, wk = (wave & 1) * 64;
    f32x16 acc[2][2] = {};  // [n block][k block]
    // this lane's place in a transposed read
    const int tr = (8 * (lane >> 5) + ((lane & 15) >> 2)) * kWgPitch + (16 * ((lane >> 4) & 1) + 4 * (lane & 3)) * 2;
    for (int64_t m0 = 0; m0 < a.M; m0 += kWgStep) {
        vec8<T> y[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int c = tid + i * kWgThreads, r = c / 16;
            y[i] = vec8<T>{};
            if (m0 + r < a.M) y[i] = load8(static_cast<const T*>(a.dy) + (m0 + r) * a.dy_stride, n0 + (c % 16) * 8, a.N);
        }
        const int xr = tid / 8, xc = k0 + (tid % 8) * 16;
        u32x4 w = {};
        float s = 0.f;
        if (m0 + xr < a.M && xc < a.Kp) {
            const int64_t at = (m0 + xr) * a.Kp + xc;
            w = *reinterpret_cast<const u32x4*>(a.q + at);
            s = block_scale(a.e[at / 32]);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int c = tid + i * kWgThreads;
            *reinterpret_cast<u32x4*>(lds_y + (c / 16) * kWgPitch + (c % 16) * 16) = __builtin_bit_cast(u32x4, y[i]);
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            typedef T t8 __attribute__((ext_vector_type(8)));
            t8 v;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = (T)(byte_value(w[half * 2 + j / 4], j % 4) * s);
            *reinterpret_cast<u32x4*>(lds_x + xr * kWgPitch + (tid % 8) * 32 + half * 16) = __builtin_bit_cast(u32x4, v);
        }
        __syncthreads();
#pragma unroll
        for (int sub = 0; sub < kWgStep / 16; ++sub) {
            frag fy[2], fx[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                fy[i] = read_column8<frag>(lds_y + sub * 16 * kWgPitch + tr + (wn + i * 32) * 2, kWgPitch);
                fx[i] = read_column8<frag>(lds_x + sub * 16 * kWgPitch + tr + (wk + i * 32) * 2, kWgPitch);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) acc[i][j] = Mfma<T>::run(fx[j], fy[i], acc[i][j]);
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) wgrad_store_rows<T, 2>(a, lds + wave * 8192, n0 + wn + i * 32, k0 + wk, acc[i]);
}

// The same for dy in whole words (wgrad_fast): 2 x 2 waves of 32 WN x 32 WK outputs,
// 64 tokens a step, two stages in LDS.
//   - The MFMA wants eight tokens of a column in a lane, memory has a token's columns
//     side by side.  A thread loads 8 tokens x 8 columns of each operand and turns them
//     in registers: dy by half a byte permute per element, the checkpoint for nothing,
//     since its values are converted one by one and paired as they are rounded.  LDS
//     then holds, for every column, 64 tokens in eight 16-byte chunks, and both sides
//     use 16-byte accesses.  (Staging token-major and reading with the transposing
//     LDS loads moves the same bytes in twice the reads, 8 bytes each.)
//   - Chunk c of column r lies at chunk c ^ (r ^ r / 8 & 3) & 7: eight (sixteen)
//     consecutive columns, as a fragment read takes them, lie in different banks, and
//     the blocks of 32 columns alike, so that a lane needs one address per 16 tokens.
//   - A workgroup's work is a list of tiles, then a share of the tiles that do not
//     fill the device a last time: those are cut along the tokens into equal shares
//     (wgrad_join_kernel adds the pieces).
struct WgradPlan {
    int tiles_n, tiles_k;
    int full;          // tiles computed whole, tile t by workgroup t % grid
    int grid;          // workgroups
    int shares;        // workgroups that take a share of the other tiles (0: there are none)
    int dealt;         // neighbouring shares on different XCDs
    int64_t steps;     // of 64 tokens
    float* pieces;     // [shares + cut tiles - 1] partial tiles, that of share s in cut tile t at s + t
};

// Tile t in the order of computation: groups of eight tile rows, column by column, so
// that the 32 tiles an XCD works on at a time share rows of dy and columns of x^.
__device__ __host__ inline void wgrad_tile(const WgradPlan& p, int t, int& tn, int& tk)
{
    const int per = 8 * p.tiles_k, g = t / per, left = p.tiles_n - 8 * g, rows = left < 8 ? left : 8, r = t - g * per;
    tn = 8 * g + r % rows;
    tk = r / rows;
}

// The steps of the cut tiles are numbered through; share s begins at this one.
__device__ __host__ inline int64_t wgrad_share(const WgradPlan& p, int64_t s)
{
    const int64_t rest = (int64_t)p.tiles_n * p.tiles_k - p.full;
    return rest * p.steps * s / p.shares;
}

constexpr int kWgRows = 64;   // tokens per step
constexpr int kWgCol = 128;   // LDS bytes of a column's tokens

// LDS offset of chunk c (8 tokens) of column r
__device__ __forceinline__ int wgrad_at(int r, int c) { return r * kWgCol + ((c ^ r ^ ((r >> 3) & 3)) & 7) * 16; }

// A thread's share of a step: 8 tokens x C columns of dy and of the checkpoint.
template <int C>
struct WgradRegs {
    typedef uint32_t y_t __attribute__((ext_vector_type(C / 2)));
    typedef uint32_t x_t __attribute__((ext_vector_type(C / 4)));
    y_t y[8];
    x_t x[8];
    int e[2];  // scales of tokens 2 (lane % 4) and the next: four lanes share a block of 32 columns
};

template <class T, int C>
struct WgradLoader {
    typedef WgradRegs<C> Regs;
    const WgradArgs& a;
    uint32_t yoff, xoff, eoff, ypitch;
    int eper;
    int64_t end;  // first step past the range
    __amdgpu_buffer_rsrc_t ry, rq, re;

    // tg: which eight of the step's tokens; n, k: the first of the C columns of dy and x
    __device__ __forceinline__ WgradLoader(const WgradArgs& args, int tg, int n, int k, int64_t stop) : a(args), end(stop)
    {
        ypitch = (uint32_t)a.dy_stride * 2u;
        eper = a.Kp / 32;
        yoff = n < a.N ? (uint32_t)(8 * tg) * ypitch + (uint32_t)n * 2u : kOob;
        xoff = k < a.Kp ? (uint32_t)(8 * tg) * (uint32_t)a.Kp + (uint32_t)k : kOob;
        eoff = k < a.Kp ? (uint32_t)(8 * tg + 2 * (threadIdx.x & 3)) * (uint32_t)eper + (uint32_t)(k / 32) : kOob;
    }
    // Resources that begin at the step's first token and end with the last one's row: tokens past M and
    // columns past the row read as zero.
    __device__ __forceinline__ void at(int64_t step)
    {
        const int64_t m = step * kWgRows, left = step < end ? a.M - m : 0;
        const int rows = (int)(left < kWgRows ? left : kWgRows);
        ry = __builtin_amdgcn_make_buffer_rsrc((void*)(static_cast<const T*>(a.dy) + m * a.dy_stride), 0,
                                               rows > 0 ? ((rows - 1) * (int)a.dy_stride + a.N) * 2 : 0, kRsrcFlags);
        rq = __builtin_amdgcn_make_buffer_rsrc((void*)(a.q + m * a.Kp), 0, rows * a.Kp, kRsrcFlags);
        re = __builtin_amdgcn_make_buffer_rsrc((void*)(a.e + m * eper), 0, rows * eper, kRsrcFlags);
    }
    __device__ __forceinline__ void load_y(Regs& r, int i) const
    {
        const uint32_t at = yoff + (uint32_t)i * ypitch;
        if constexpr (C == 8) r.y[i] = __builtin_bit_cast(typename Regs::y_t, __builtin_amdgcn_raw_buffer_load_b128(ry, at, 0, 0));
        else r.y[i] = __builtin_bit_cast(typename Regs::y_t, __builtin_amdgcn_raw_buffer_load_b64(ry, at, 0, 0));
    }
    __device__ __forceinline__ void load_x(Regs& r, int i) const
    {
        const uint32_t at = xoff + (uint32_t)(i * a.Kp);
        if constexpr (C == 8) r.x[i] = __builtin_bit_cast(typename Regs::x_t, __builtin_amdgcn_raw_buffer_load_b64(rq, at, 0, 0));
        else r.x[i] = __builtin_bit_cast(typename Regs::x_t, __builtin_amdgcn_raw_buffer_load_b32(rq, at, 0, 0));
    }
    __device__ __forceinline__ void load_e(Regs& r, int i) const
    {
        r.e[i] = (int8_t)__builtin_amdgcn_raw_buffer_load_b8(re, eoff + (uint32_t)(i * eper), 0, 0);
    }
};

// The eight tokens' scales from the four lanes that hold two each.
template <int C>
__device__ __forceinline__ void wgrad_scales(const WgradRegs<C>& r, float (&sc)[8])
{
    const int s[2] = {(int)__float_as_uint(block_scale(r.e[0])), (int)__float_as_uint(block_scale(r.e[1]))};
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        sc[0 + q] = __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp(s[q], 0x00, 0xF, 0xF, true));
        sc[2 + q] = __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp(s[q], 0x55, 0xF, 0xF, true));
        sc[4 + q] = __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp(s[q], 0xAA, 0xF, 0xF, true));
        sc[6 + q] = __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp(s[q], 0xFF, 0xF, 0xF, true));
    }
}

// Tokens 2 p and 2 p + 1 of column j of the checkpoint as a pair of T.
template <class T, int C>
__device__ __forceinline__ uint32_t wgrad_pair_x(const WgradRegs<C>& r, const float (&sc)[8], int j, int p)
{
    typedef T t2 __attribute__((ext_vector_type(2)));
    const t2 v = {(T)(byte_value(r.x[2 * p][j / 4], j % 4) * sc[2 * p]),
                  (T)(byte_value(r.x[2 * p + 1][j / 4], j % 4) * sc[2 * p + 1])};
    return __builtin_bit_cast(uint32_t, v);
}

// Tokens 2 p and 2 p + 1 of column j of dy.
template <int C>
__device__ __forceinline__ uint32_t wgrad_pair_y(const WgradRegs<C>& r, int j, int p)
{
    return __builtin_amdgcn_perm(r.y[2 * p + 1][j / 2], r.y[2 * p][j / 2], j & 1 ? 0x07060302u : 0x05040100u);
}

template <int WN, int WK>
struct WgradTile {
    static constexpr int kBN = 64 * WN, kBK = 64 * WK;
    static constexpr int kBlocks = WN * WK;           // 32 x 32 blocks of a wave
    static constexpr int kFloats = kBN * kBK;         // of a partial tile
    static constexpr int kStage = (kBN + kBK) * kWgCol;
    static constexpr int kLds = 2 * kStage;
};

// LDS offsets of a thread in each of the two stages: its first column as a
// loader (column j's chunk lies at offset ^ 16 j, j columns on), and its column of the
// wave's first fragment as a reader, for each 16 tokens.
template <class T, int WN, int WK>
struct WgradPlaces {
    typedef WgradTile<WN, WK> Tile;
    typedef typename Mfma<T>::frag frag;
    static constexpr int kX = Tile::kBN * kWgCol;  // the checkpoint's columns after dy's
    static constexpr int kCols = Tile::kBN / 32;   // columns a thread loads

    char* const lds;
    uint32_t put[2], get_y[2][4], get_x[2][4];

    __device__ __forceinline__ explicit WgradPlaces(char* l) : lds(l)
    {
        static_assert(WN == WK, "square tiles");
        const int tg = threadIdx.x / 32, cg = threadIdx.x % 32, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            put[p] = p * Tile::kStage + wgrad_at(kCols * cg, tg);
#pragma unroll
            for (int sub = 0; sub < 4; ++sub) {
                get_y[p][sub] = p * Tile::kStage + wgrad_at((wave >> 1) * 32 * WN + (lane & 31), 2 * sub + (lane >> 5));
                get_x[p][sub] = p * Tile::kStage + wgrad_at((wave & 1) * 32 * WK + (lane & 31), 2 * sub + (lane >> 5));
            }
        }
    }
    // Takes the constancy of these from the compiler, which would give every sum with them a register of its own.
    __device__ __forceinline__ void hide(WgradLoader<T, kCols>& ld)
    {
        __asm__ __volatile__("" : "+v"(put[0]), "+v"(put[1]), "+v"(ld.yoff), "+v"(ld.xoff), "+v"(ld.eoff));
    }
    template <int P>
    __device__ __forceinline__ void write(int j, bool x, const u32x4& v) const
    {
        *reinterpret_cast<u32x4*>(lds + (put[P] ^ (uint32_t)(16 * j)) + j * kWgCol + (x ? kX : 0)) = v;
    }
    // the fragment of block b and 16 tokens `sub` of dy or the checkpoint
    template <int P>
    __device__ __forceinline__ frag read(int sub, int b, bool x) const
    {
        return *reinterpret_cast<const frag*>(lds + (x ? get_x[P][sub] : get_y[P][sub]) + b * 32 * kWgCol + (x ? kX : 0));
    }
    static __device__ __forceinline__ void barrier()
    {
        __asm__ __volatile__("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    }
};

// One tile over the steps s0 .. s1 - 1.  A step runs from barrier to barrier.  At its
// start stage s is written, and the other stage read but for fragments that are already
// in registers, so the whole step can write stage s + 1.  Each of its 4 W^2 MFMAs is
// followed by a share of the step's other work, and fences keep it there: what waited for
// the MFMAs' end, or came in one piece, would find nothing to run beside.
//   MFMA 0 ..   the last 16 tokens of step s - 1, then the first 48 of step s; the
//               fragment reads go 16 tokens ahead
//   columns     of the thread's, of the checkpoint and of dy, a pair of tokens at a time,
//               each written when done
//   the loads   of step s + 2, into the other set of registers: more than a step to
//               arrive
// W = 4, tiles of 256 x 256: one workgroup per CU, one wave per SIMD, whose 256
// accumulators leave no second wave to cover a wait.  What does not fit under an MFMA's 32
// cycles (or under the LDS queue's pace, some 28 cycles per 16-byte instruction of one
// wave) adds to the step, so all of it is spread evenly.
// W = 2, tiles of 128 x 128: two workgroups share a CU.  The loads come first, three to a
// place: 512 x 2048 x 512 takes 11.5 us so, 12.0 with one to a place, 12.5 with all in the
// first.  LDS (16 reads and 8 writes a wave) and the conversion of the checkpoint bound a
// step: 1.3 us for the two workgroups, of which the MFMAs take 0.45.
template <class T, int W>
struct WgradRun : WgradPlaces<T, W, W> {
    typedef WgradPlaces<T, W, W> Places;
    typedef typename Places::frag frag;
    static constexpr int kCols = Places::kCols, kBN = Places::Tile::kBN;

    f32x16 (&acc)[W][W];
    WgradLoader<T, kCols> ld;
    WgradRegs<kCols> r[2];
    frag fy[2][W], fx[2][W];

    __device__ __forceinline__ WgradRun(const WgradArgs& a, char* l, int tn, int tk, int64_t s1, f32x16 (&c)[W][W])
        : Places(l), acc(c),
          ld(a, threadIdx.x / 32, tn * kBN + kCols * (threadIdx.x % 32), tk * kBN + kCols * (threadIdx.x % 32), s1)
    {
    }
    __device__ __forceinline__ void load(WgradRegs<kCols>& g, int i) const  // 0 .. 17
    {
        if (i < 2) ld.load_e(g, i);
        else if (i < 10) ld.load_x(g, i - 2);
        else ld.load_y(g, i - 10);
    }

    // Stage s in buffer P, step s + 1's data in r[P ^ 1].
    template <int P>
    __device__ __forceinline__ void step(int64_t s)
    {
        this->hide(ld);
        WgradRegs<kCols>& g = r[P ^ 1];
        ld.at(s + 2);
        float sc[8];
        wgrad_scales(g, sc);
        u32x4 wx[2], wy;
#pragma unroll
        for (int m = 0; m < 4 * W * W; ++m) {
            const int u = m / (W * W), q = m % (W * W), i = q / W, j = q % W;
            // u = 0: fragments 3 of the step before, read into set 1
            acc[i][j] = Mfma<T>::run(fx[(u + 1) & 1][j], fy[(u + 1) & 1][i], acc[i][j]);
            if constexpr (W == 4) {
                if (q < 12 && q % 3 != 2) {
                    const int f = q / 3 * 2 + q % 3;  // the checkpoint's first: each MFMA row needs all four
                    if (f < 4) fx[u & 1][f] = this->template read<P>(u, f, true);
                    else fy[u & 1][f - 4] = this->template read<P>(u, f - 4, false);
                }
                if (m % 3 == 2 && m / 3 < 18) load(r[P], m / 3);
                const int c = m / 7, k = m % 7;  // column and place in its seven
                if (c < 8) {
                    if (k % 2 == 0) wx[c & 1][k / 2] = wgrad_pair_x<T>(g, sc, c, k / 2);
                    if (k % 2 == 1) wy[k / 2] = wgrad_pair_y(g, c, k / 2);
                    if (k == 5) {
                        wy[3] = wgrad_pair_y(g, c, 3);
                        this->template write<P ^ 1>(c, false, wy);
                    }
                }
                if (c > 0 && k == 1) this->template write<P ^ 1>(c - 1, true, wx[(c - 1) & 1]);
            } else {
                if (q % 2 == 0) fx[u & 1][q / 2] = this->template read<P>(u, q / 2, true);
                else fy[u & 1][q / 2] = this->template read<P>(u, q / 2, false);
#pragma unroll
                for (int l = 3 * m; l < 3 * m + 3 && l < 18; ++l) load(r[P], l);
                wx[0][q] = wgrad_pair_x<T>(g, sc, u, q);
                wy[q] = wgrad_pair_y(g, u, q);
                if (q == 3) {
                    this->template write<P ^ 1>(u, false, wy);
                    this->template write<P ^ 1>(u, true, wx[0]);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        this->barrier();
    }

    __device__ __forceinline__ void run(int64_t s0, int64_t s1)
    {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            ld.at(s0 + p);
#pragma unroll
            for (int i = 0; i < 18; ++i) load(r[p], i);
        }
        float sc[8];
        wgrad_scales(r[0], sc);
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
            u32x4 x, y;
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                x[p] = wgrad_pair_x<T>(r[0], sc, j, p);
                y[p] = wgrad_pair_y(r[0], j, p);
            }
            this->template write<0>(j, false, y);
            this->template write<0>(j, true, x);
        }
        // nothing before the first step: its first MFMAs add zeros
#pragma unroll
        for (int i = 0; i < W; ++i) fy[1][i] = fx[1][i] = frag{};
        this->barrier();
        // in twos: a step past the range multiplies the zeros its loads gave
        for (int64_t s = s0; s < s1; s += 2) {
            step<0>(s);
            step<1>(s + 1);
        }
#pragma unroll
        for (int i = 0; i < W; ++i)
#pragma unroll
            for (int j = 0; j < W; ++j) acc[i][j] = Mfma<T>::run(fx[1][j], fy[1][i], acc[i][j]);
        __syncthreads();
    }
};

template <class T, int WN, int WK>
__global__ __launch_bounds__(kWgThreads, WN == 4 ? 1 : 2) void wgrad_kernel(const WgradArgs a, const WgradPlan p)
{
    typedef WgradTile<WN, WK> Tile;
    extern __shared__ __attribute__((aligned(1024))) char lds[];
    const int wave = uni(threadIdx.x >> 6);
    // workgroups are dealt to the 8 XCDs in turn: those of one XCD take neighbouring tiles, but the tiles of a round
    // that not all take part in, and shares where the plan says so, go over the XCDs in turn
    const int id = (int)blockIdx.x, per = p.grid / 8, me = p.grid % 8 == 0 ? id % 8 * per + id / 8 : id;
    f32x16 acc[WN][WK];
    auto clear = [&]() {
#pragma unroll
        for (int i = 0; i < WN; ++i)
#pragma unroll
            for (int j = 0; j < WK; ++j) acc[i][j] = f32x16{};
    };
    for (int t0 = 0; t0 < p.full; t0 += p.grid) {
        const int t = t0 + (t0 + p.grid <= p.full ? me : id);
        if (t >= p.full) break;
        int tn, tk;
        wgrad_tile(p, t, tn, tk);
        clear();
        WgradRun<T, WN>(a, lds, tn, tk, p.steps, acc).run(0, p.steps);
#pragma unroll
        for (int i = 0; i < WN; ++i)
            wgrad_store_rows<T, WK>(a, lds + wave * (32 * 32 * WK * 4), tn * Tile::kBN + (wave >> 1) * 32 * WN + 32 * i,
                                    tk * Tile::kBK + (wave & 1) * 32 * WK, acc[i]);
        __syncthreads();
    }
    const int share = p.dealt ? id : me;
    if (share >= p.shares) return;
    const int64_t end = wgrad_share(p, share + 1);
    for (int64_t at = wgrad_share(p, share); at < end;) {
        const int64_t t = at / p.steps, stop = (t + 1) * p.steps < end ? (t + 1) * p.steps : end;
        int tn, tk;
        wgrad_tile(p, p.full + (int)t, tn, tk);
        clear();
        WgradRun<T, WN>(a, lds, tn, tk, stop - t * p.steps, acc).run(at - t * p.steps, stop - t * p.steps);
        // In the order of the registers: [block][four accumulators][thread].  From one piece to the next the share, the
        // tile or both go up by one, so their sum tells pieces apart.
        f32x4* out = reinterpret_cast<f32x4*>(p.pieces + (share + t) * Tile::kFloats) + threadIdx.x;
#pragma unroll
        for (int b = 0; b < Tile::kBlocks; ++b)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const f32x16& v = acc[b / WK][b % WK];
                out[(b * 4 + g) * kWgThreads] = f32x4{v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]};
            }
        at = stop;
    }
}

// Adds the pieces of the cut tiles: one workgroup per tile, wave of the tile's workgroup
// and row of its blocks.  Its WAVES waves take equal parts of the pieces, in token order,
// and add up in that order.  The latency of the pieces bounds it: where tiles have many,
// four waves read them at once (16384 x 512 x 256, 32 pieces a tile: 22 us, 32 with one
// wave; 4100 x 300 x 200, 8 pieces: 16.9, 18.5); where they have few, three waves would stand
// idle (6000 x 4000 x 2000, 2 pieces: 121 us, 111 with one wave; 4096 x 4096 x 1024, 4 pieces:
// 61, 58).
template <class T, int WN, int WK, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void wgrad_join_kernel(const WgradArgs a, const WgradPlan p)
{
    typedef WgradTile<WN, WK> Tile;
    constexpr int kArea = 32 * 32 * WK * 4;
    __shared__ __attribute__((aligned(16))) char lds[WAVES * kArea];
    const int t = blockIdx.x, row = blockIdx.y / 4, wave = blockIdx.y % 4;
    const int lane = threadIdx.x & 63, part = uni(threadIdx.x >> 6);
    const int64_t first = t * p.steps, last = first + p.steps, all = ((int64_t)p.tiles_n * p.tiles_k - p.full) * p.steps;
    // from the last share that begins at or before the tile to the last that begins within it
    const int64_t s0 = ((first + 1) * p.shares + all - 1) / all - 1, s1 = (last * p.shares + all - 1) / all;
    const f32x4* in = reinterpret_cast<const f32x4*>(p.pieces) + row * WK * 4 * kWgThreads + wave * 64 + lane;
    constexpr int64_t kPiece = Tile::kFloats / 4;
    constexpr int kAhead = WK == 4 || WAVES > 1 ? 1 : 4;
    f32x4 piece[kAhead][4 * WK];
    auto load = [&](f32x4 (&v)[4 * WK], int64_t s) {
        const f32x4* from = in + (s + t) * kPiece;
#pragma unroll
        for (int g = 0; g < 4 * WK; ++g) v[g] = from[g * kWgThreads];
        __builtin_amdgcn_sched_barrier(0);  // all on their way before one is waited for
    };
    f32x16 acc[WK];
#pragma unroll
    for (int j = 0; j < WK; ++j) acc[j] = f32x16{};
    auto add = [&](const f32x4 (&v)[4 * WK]) {
#pragma unroll
        for (int g = 0; g < 4 * WK; ++g)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[g / 4][4 * (g % 4) + e] += v[g][e];
    };
    const int64_t from = s0 + (s1 - s0) * part / WAVES, to = s0 + (s1 - s0) * (part + 1) / WAVES;
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (from + i < to) load(piece[i], from + i);
    for (int64_t s = from; s < to; s += kAhead) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (s + i < to) {
                add(piece[i]);
                if (s + i + kAhead < to) load(piece[i], s + i + kAhead);
            }
    }
    f32x4* const mine = reinterpret_cast<f32x4*>(lds + part * kArea) + lane;
    if (part > 0)
#pragma unroll
        for (int g = 0; g < 4 * WK; ++g) {
            const f32x16& v = acc[g / 4];
            mine[g * 64] = f32x4{v[4 * (g % 4)], v[4 * (g % 4) + 1], v[4 * (g % 4) + 2], v[4 * (g % 4) + 3]};
        }
    __syncthreads();
    if (part > 0) return;
#pragma unroll
    for (int q = 1; q < WAVES; ++q)
#pragma unroll
        for (int g = 0; g < 4 * WK; ++g) {
            const f32x4 v = mine[(q * 4 * WK + g) * 64];
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[g / 4][4 * (g % 4) + e] += v[e];
        }
    int tn, tk;
    wgrad_tile(p, p.full + t, tn, tk);
    wgrad_store_rows<T, WK>(a, lds, tn * Tile::kBN + (wave >> 1) * 32 * WN + 32 * row,
                            tk * Tile::kBK + (wave & 1) * 32 * WK, acc);
}

}  // namespace gemm_rs_layer
