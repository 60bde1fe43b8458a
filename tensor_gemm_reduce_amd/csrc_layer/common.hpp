// common.hpp -- element types, vector loads and reductions shared by the layer
// operators' gfx950 kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gemm_rs_layer {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void_t;

// Third descriptor word of a raw buffer resource on gfx9-family GPUs, and an
// offset past every resource made here: loads there read zero.
constexpr int kRsrcFlags = 0x00020000;
constexpr uint32_t kOob = 0x80000000u;

// Eight elements that may start at any element boundary (gfx950 loads 16 bytes
// from any address; aligned ones are served in fewer requests).
template <class T>
struct Vec8 {
    typedef T type __attribute__((ext_vector_type(8), aligned(sizeof(T))));
};
template <class T>
using vec8 = typename Vec8<T>::type;

// Columns col .. col + 7 of a row that ends at n, zeros past it.
template <class T>
__device__ __forceinline__ vec8<T> load8(const T* row, int col, int n)
{
    vec8<T> v = {};
    if (col + 8 <= n) {
        v = *reinterpret_cast<const vec8<T>*>(row + col);
    } else if (col < n) {
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (col + j < n) v[j] = row[col + j];
    }
    return v;
}

template <class T>
__device__ __forceinline__ void store8(T* row, int col, int n, const float (&f)[8])
{
    if (col + 8 <= n) {
        vec8<T> v;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = (T)f[j];
        *reinterpret_cast<vec8<T>*>(row + col) = v;
    } else if (col < n) {
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (col + j < n) row[col + j] = (T)f[j];
    }
}

template <class T>
__device__ __forceinline__ void widen(const vec8<T>& v, float (&f)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = (float)v[j];
}

__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// Sum over the workgroup, the same bits in every thread.  `slot` (THREADS / 64
// floats) may be reused by another call once a barrier has passed.
template <int THREADS>
__device__ __forceinline__ float block_sum(float v, float* slot)
{
    v = wave_sum(v);
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) s += slot[w];
    return s;
}

__device__ __forceinline__ int uni(int x) { return __builtin_amdgcn_readfirstlane(x); }

}  // namespace gemm_rs_layer
