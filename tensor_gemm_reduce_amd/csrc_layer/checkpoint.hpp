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
// a row has an even number of chunks) exchange their maxima.
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

// dw = dy^T x^: 128 x 128 outputs per workgroup, four waves of 64 x 64, 32 tokens
// a step.  Both operands are token-major in memory, the MFMA wants eight tokens of
// a column in a lane: the tiles go into LDS as they are and are read transposed.
// The checkpoint is expanded to T between its load and LDS.
constexpr int kWgTile = 128, kWgStep = 32, kWgThreads = 256;
constexpr int kWgPitch = kWgTile * 2 + 64;  // rows 16 banks apart: the four rows of a transposed read differ

template <class T>
__global__ __launch_bounds__(kWgThreads) void wgrad_kernel(const WgradArgs a)
{
    typedef typename Mfma<T>::frag frag;
    __shared__ __attribute__((aligned(16))) char lds_y[kWgStep * kWgPitch];
    __shared__ __attribute__((aligned(16))) char lds_x[kWgStep * kWgPitch];
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
    // a lane holds row n, four consecutive k per group of four accumulators
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int n = n0 + wn + i * 32 + (lane & 31);
        if (n >= a.N) continue;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int k = k0 + wk + j * 32 + 8 * (r / 4) + 4 * (lane >> 5) + r % 4;
                if (k >= a.K) continue;
                float v = acc[i][j][r];
                if (a.add) v += a.add[n * a.add_stride + k];
                if (a.out_f32)
                    static_cast<float*>(a.dw)[n * a.dw_stride + k] = v;
                else
                    static_cast<T*>(a.dw)[n * a.dw_stride + k] = (T)v;
            }
    }
}

}  // namespace gemm_rs_layer
