// block_norm.hpp -- what follows the row-parallel layer: the sum of the ranks'
// partials, the norm after the block, its gate and scale, the residual and the
// norm before the next block, and the gradients of all of them.
#pragma once

#include "common.hpp"

namespace gemm_rs_layer {

constexpr int kMaxParts = 8;

struct NormArgs {
    const void* parts[kMaxParts];
    const void *residual, *post_weight, *gate, *pre_weight;
    void *h, *z, *y;
    float* rstd;
    int64_t part_stride, residual_stride, gate_stride, h_stride, z_stride, y_stride, rows;
    float eps, block_scale, residual_scale;
    int n, nparts, gate_kind;
};

// One workgroup per row; thread t holds the chunks t, t + THREADS, ... of eight
// columns in registers from the first load to the last store, so every input is
// read once and every output written once.  MAXP: 1, or 8 for up to eight parts.
// Bytes bound it from some 1000 rows (4096 x 8192, eight parts, residual and statistics in
// 32 bits 184 us, 5.1 TB/s), one row's latency below: with one chunk per thread (ITEMS = 1)
// all of a row's loads are on their way at once, the weights and the gate too, so that
// nothing is waited for after a sum over the row.  1 x 8192, eight parts, takes 4.3 us so,
// 7.0 with four chunks per thread; 4096 x 8192, one part, 93 and 102; 4096 x 256 8.4 with
// 128 threads, 12.6 with 256.  Rows past 8192 columns take four chunks per thread (us, bytes
// at 5 TB/s in brackets, BF16, one part: 1024 x 8200 40 (17), 1024 x 16384 45 (34), 1024 x
// 32768 83 (67); 1024 x 8192 23 (17)).
template <class T, class R, int THREADS, int ITEMS, int MAXP>
__global__ __launch_bounds__(THREADS) void norm_forward_kernel(const NormArgs a)
{
    __shared__ float slots[2][THREADS / 64];
    constexpr bool kEarly = ITEMS == 1;
    const int64_t row = blockIdx.x;
    const int n = a.n;
    float v[ITEMS][8];

    const R* rrow = static_cast<const R*>(a.residual) + row * a.residual_stride;
    const bool gated = a.gate_kind == GEMM_RS_GATE_CHANNEL || a.gate_kind == GEMM_RS_GATE_FULL;
    const T* gate = static_cast<const T*>(a.gate) + (a.gate_kind == GEMM_RS_GATE_FULL ? row * a.gate_stride : 0);
    vec8<R> early_res = {};
    vec8<T> early_post = {}, early_gate = {}, early_pre = {};
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const int col = (i * THREADS + (int)threadIdx.x) * 8;
        vec8<T> p[MAXP];
#pragma unroll
        for (int k = 0; k < MAXP; ++k)
            if (k < a.nparts) p[k] = load8(static_cast<const T*>(a.parts[k]) + row * a.part_stride, col, n);
        if constexpr (kEarly) {
            if (a.residual) early_res = load8(rrow, col, n);
            if (a.post_weight) early_post = load8(static_cast<const T*>(a.post_weight), col, n);
            if (gated) early_gate = load8(gate, col, n);
            if (a.pre_weight) early_pre = load8(static_cast<const T*>(a.pre_weight), col, n);
        }
        widen<T>(p[0], v[i]);
#pragma unroll
        for (int k = 1; k < MAXP; ++k)
            if (k < a.nparts) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] += (float)p[k][j];
            }
    }

    if (a.y) {
        T* dst = static_cast<T*>(a.y) + row * a.y_stride;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) store8(dst, (i * THREADS + (int)threadIdx.x) * 8, n, v[i]);
    }

    float ry = 1.f;
    if (a.post_weight) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) s += v[i][j] * v[i][j];
        ry = 1.f / sqrtf(block_sum<THREADS>(s, slots[0]) / (float)n + a.eps);
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const vec8<T> w = kEarly ? early_post
                                     : load8(static_cast<const T*>(a.post_weight), (i * THREADS + (int)threadIdx.x) * 8, n);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * ry * (float)w[j];
        }
    }

    float row_scale = a.block_scale;
    if (a.gate_kind == GEMM_RS_GATE_TOKEN) row_scale *= (float)static_cast<const T*>(a.gate)[row];
    R* hrow = static_cast<R*>(a.h) + row * a.h_stride;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const int col = (i * THREADS + (int)threadIdx.x) * 8;
        if (gated) {
            const vec8<T> g = kEarly ? early_gate : load8(gate, col, n);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] *= (float)g[j];
        }
        vec8<R> res = early_res;
        if (!kEarly && a.residual) res = load8(rrow, col, n);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float h = row_scale * v[i][j];
            if (a.residual) h += a.residual_scale * (float)res[j];
            v[i][j] = h;
            s += h * h;
        }
        store8(hrow, col, n, v[i]);
    }

    float rh = 0.f;
    if (a.pre_weight) {
        rh = 1.f / sqrtf(block_sum<THREADS>(s, slots[1]) / (float)n + a.eps);
        T* zrow = static_cast<T*>(a.z) + row * a.z_stride;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int col = (i * THREADS + (int)threadIdx.x) * 8;
            const vec8<T> w = kEarly ? early_pre : load8(static_cast<const T*>(a.pre_weight), col, n);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * rh * (float)w[j];
            store8(zrow, col, n, v[i]);
        }
    }
    if (a.rstd && threadIdx.x == 0) {
        a.rstd[row] = ry;
        a.rstd[a.rows + row] = rh;
    }
}

struct NormGradArgs {
    const void *dz, *dh, *h, *y;
    const float* rstd;
    const void *post_weight, *gate, *pre_weight;
    void *dresidual, *dy, *dgate;
    float* partial;  // [gridDim.x][sums][n]: the pre weight's, post weight's and channel gate's sums
    int64_t dz_stride, dh_stride, h_stride, y_stride, gate_stride, dresidual_stride, dy_stride, dgate_stride, rows;
    float block_scale, residual_scale;
    int n, gate_kind, sums;
};

// What a thread reads of a row: its eight columns of each input.
template <class T, class R>
struct NormGradRow {
    vec8<T> dz, y, gate;
    vec8<R> dh, h;

    __device__ __forceinline__ void load(const NormGradArgs& a, int64_t row, int col)
    {
        dz = y = gate = vec8<T>{};
        dh = h = vec8<R>{};
        if (a.pre_weight) {
            dz = load8(static_cast<const T*>(a.dz) + row * a.dz_stride, col, a.n);
            h = load8(static_cast<const R*>(a.h) + row * a.h_stride, col, a.n);
        }
        if (a.dh) dh = load8(static_cast<const R*>(a.dh) + row * a.dh_stride, col, a.n);
        if (a.post_weight || a.gate) y = load8(static_cast<const T*>(a.y) + row * a.y_stride, col, a.n);
        if (a.gate_kind == GEMM_RS_GATE_FULL) gate = load8(static_cast<const T*>(a.gate) + row * a.gate_stride, col, a.n);
    }
};

// Weights and sums over rows of a thread's eight columns.
template <class T>
struct NormGradColumns {
    vec8<T> pre, post, gate;
    float sum_pre[8], sum_post[8], sum_gate[8];

    __device__ __forceinline__ void load(const NormGradArgs& a, int col)
    {
        pre = post = gate = vec8<T>{};
        if (a.pre_weight) pre = load8(static_cast<const T*>(a.pre_weight), col, a.n);
        if (a.post_weight) post = load8(static_cast<const T*>(a.post_weight), col, a.n);
        if (a.gate_kind == GEMM_RS_GATE_CHANNEL) gate = load8(static_cast<const T*>(a.gate), col, a.n);
    }
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int j = 0; j < 8; ++j) sum_pre[j] = sum_post[j] = sum_gate[j] = 0.f;
    }
    // the workgroup's partial row: [sums][n]
    __device__ __forceinline__ void keep(const NormGradArgs& a, float* part, int col) const
    {
        if (a.pre_weight) {
            store8(part, col, a.n, sum_pre);
            part += a.n;
        }
        if (a.post_weight) {
            store8(part, col, a.n, sum_post);
            part += a.n;
        }
        if (a.gate_kind == GEMM_RS_GATE_CHANNEL) store8(part, col, a.n, sum_gate);
    }
    __device__ __forceinline__ void fetch(const NormGradArgs& a, const float* part, int col)
    {
        if (a.pre_weight) {
            widen<float>(load8(part, col, a.n), sum_pre);
            part += a.n;
        }
        if (a.post_weight) {
            widen<float>(load8(part, col, a.n), sum_post);
            part += a.n;
        }
        if (a.gate_kind == GEMM_RS_GATE_CHANNEL) widen<float>(load8(part, col, a.n), sum_gate);
    }
};

// The arithmetic of one row, in three stages between the sums over the row.  With
// t^ = t r (r = 1 / rms(t)) a norm t^ w passes a gradient d on as r (w d - t^ mean(w d t^)).
template <class T, class R>
struct NormGradMath {
    const NormGradArgs& a;
    float ry, rh, g_row;

    __device__ __forceinline__ NormGradMath(const NormGradArgs& args, int64_t row) : a(args)
    {
        ry = a.post_weight ? a.rstd[row] : 1.f;
        rh = a.pre_weight ? a.rstd[a.rows + row] : 0.f;
        g_row = a.gate_kind == GEMM_RS_GATE_TOKEN ? (float)static_cast<const T*>(a.gate)[row] : 1.f;
    }
    // sum of w d t^ of the next block's norm
    __device__ __forceinline__ float dot_h(const NormGradRow<T, R>& r, const NormGradColumns<T>& c) const
    {
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) s += (float)c.pre[j] * (float)r.dz[j] * ((float)r.h[j] * rh);
        return s;
    }
    // through that norm, the residual's and the gate's gradients; leaves the block norm's w d in d
    __device__ __forceinline__ void middle(const NormGradRow<T, R>& r, NormGradColumns<T>& c, float mean_h, int64_t row, int col,
                                           float (&d)[8], float& dot_y, float& dot_gate) const
    {
        float o[8], dg[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float g = (float)r.dh[j];
            if (a.pre_weight) {
                const float hh = (float)r.h[j] * rh, z = (float)r.dz[j];
                g += rh * ((float)c.pre[j] * z - hh * mean_h);
                c.sum_pre[j] += z * hh;
            }
            o[j] = a.residual_scale * g;
            const float yy = (float)r.y[j] * ry;
            g *= a.block_scale;
            dg[j] = g * (a.post_weight ? yy * (float)c.post[j] : yy);
            dot_gate += dg[j];
            if (a.gate_kind == GEMM_RS_GATE_CHANNEL) {
                c.sum_gate[j] += dg[j];
                g *= (float)c.gate[j];
            }
            if (a.gate_kind == GEMM_RS_GATE_FULL) g *= (float)r.gate[j];
            g *= g_row;
            if (a.post_weight) {
                c.sum_post[j] += g * yy;
                g *= (float)c.post[j];
                dot_y += g * yy;
            }
            d[j] = g;
        }
        if (a.dresidual) store8(static_cast<R*>(a.dresidual) + row * a.dresidual_stride, col, a.n, o);
        if (a.gate_kind == GEMM_RS_GATE_FULL) store8(static_cast<T*>(a.dgate) + row * a.dgate_stride, col, a.n, dg);
    }
    // through the block's own norm
    __device__ __forceinline__ void last(const vec8<T>& y, float mean_y, int64_t row, int col, float (&d)[8]) const
    {
        if (a.post_weight) {
#pragma unroll
            for (int j = 0; j < 8; ++j) d[j] = ry * (d[j] - (float)y[j] * ry * mean_y);
        }
        store8(static_cast<T*>(a.dy) + row * a.dy_stride, col, a.n, d);
    }
};

// Workgroup g takes rows g, g + grid, ..., a thread the same eight columns of each: the
// weights and the sums over rows stay in its registers, and leave as one partial row per
// workgroup (norm_sums_kernel adds them).  Other workgroups' loads cover a row's waits
// (the next row's loads in registers of their own cost more occupancy than they hid:
// 4096 rows of 4096 columns 91 us against 81).  The statistics come from the forward pass,
// so a row needs one or two sums over the workgroup (three with a gate per row).  Bytes
// bound it from some 2000 rows: 4096 x 8192 with post norm and gate, residual in 32 bits,
// 129 us with the sums over rows (4.7 TB/s); below, a row's latency and the second launch.
template <class T, class R, int THREADS>
__global__ __launch_bounds__(THREADS) void norm_backward_kernel(const NormGradArgs a)
{
    __shared__ float slots[2][3][THREADS / 64];
    const float inv_n = 1.f / (float)a.n;
    const int col = (int)threadIdx.x * 8;
    NormGradColumns<T> c;
    c.load(a, col);
    c.clear();
    // `half` alternates, so that a row's sums do not overwrite those of the row before while they are read
    auto compute = [&](const NormGradRow<T, R>& r, int64_t row, int half) {
        const NormGradMath<T, R> m(a, row);
        float mean_h = 0.f, mean_y = 0.f, dot_y = 0.f, dot_gate = 0.f, d[8];
        if (a.pre_weight) mean_h = block_sum<THREADS>(m.dot_h(r, c), slots[half][0]) * inv_n;
        m.middle(r, c, mean_h, row, col, d, dot_y, dot_gate);
        if (a.gate_kind == GEMM_RS_GATE_TOKEN) {
            const float t = block_sum<THREADS>(dot_gate, slots[half][1]);
            if (threadIdx.x == 0) static_cast<T*>(a.dgate)[row] = (T)t;
        }
        if (a.post_weight) mean_y = block_sum<THREADS>(dot_y, slots[half][2]) * inv_n;
        m.last(r.y, mean_y, row, col, d);
    };
    int half = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, half ^= 1) {
        NormGradRow<T, R> r;
        r.load(a, row, col);
        compute(r, row, half);
    }
    c.keep(a, a.partial + (int64_t)blockIdx.x * a.sums * a.n, col);
}

// Rows wider than 8 x 1024: ITEMS chunks of eight columns per thread.  The inputs are read
// again where they are needed again, from cache, and the sums over rows are kept in the
// workgroup's partial row.  Scratch memory bounds it: d and the chunks' inputs pass the 128
// registers of 1024 threads (56 .. 91 of them in scratch with two chunks, 289 .. 369 with
// four; 59% of the waves' cycles are waits).  With the sums over rows, BF16, us (bytes at 5
// TB/s): 1024 x 8200 86 (20), 1024 x 16384 138 (40), 1024 x 20480 391 (50), 1024 x 32768 515
// (81); 1024 x 8192, by the kernel above, 39 (20).
template <class T, class R, int ITEMS>
__global__ __launch_bounds__(1024) void norm_backward_wide_kernel(const NormGradArgs a)
{
    __shared__ float slots[3][1024 / 64];
    const float inv_n = 1.f / (float)a.n;
    float* const part = a.partial + (int64_t)blockIdx.x * a.sums * a.n;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const NormGradMath<T, R> m(a, row);
        float mean_h = 0.f, mean_y = 0.f, dot_h = 0.f, dot_y = 0.f, dot_gate = 0.f, d[ITEMS][8];
        if (a.pre_weight) {
#pragma unroll 1
            for (int col = (int)threadIdx.x * 8; col < a.n; col += 8192) {
                NormGradRow<T, R> r;
                NormGradColumns<T> c;
                r.load(a, row, col);
                c.load(a, col);
                dot_h += m.dot_h(r, c);
            }
            mean_h = block_sum<1024>(dot_h, slots[0]) * inv_n;
        }
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int col = (i * 1024 + (int)threadIdx.x) * 8;
            NormGradRow<T, R> r;
            NormGradColumns<T> c;
            r.load(a, row, col);
            c.load(a, col);
            if (row == blockIdx.x) c.clear();
            else c.fetch(a, part, col);
            m.middle(r, c, mean_h, row, col, d[i], dot_y, dot_gate);
            c.keep(a, part, col);
        }
        if (a.gate_kind == GEMM_RS_GATE_TOKEN) {
            const float t = block_sum<1024>(dot_gate, slots[1]);
            if (threadIdx.x == 0) static_cast<T*>(a.dgate)[row] = (T)t;
        }
        if (a.post_weight) mean_y = block_sum<1024>(dot_y, slots[2]) * inv_n;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int col = (i * 1024 + (int)threadIdx.x) * 8;
            vec8<T> y = {};
            if (a.post_weight) y = load8(static_cast<const T*>(a.y) + row * a.y_stride, col, a.n);
            m.last(y, mean_y, row, col, d[i]);
        }
        __syncthreads();  // the slots are free for the next row
    }
}

// Adds the workgroups' partial sums, in workgroup order within each of SETS strided sets
// and then over the sets.  blockIdx.y is the sum, out[] its target.  Latency bounds it:
// every thread has eight loads in flight.  Measured with the gradients it ends, us (16 /
// 32 sets): 64 groups of 8192 columns 8.4 / 8.8, 1021 of 1000 columns 12.9 / 11.2, 2000 of
// 1000 columns 21 / 18.
struct NormSumsArgs {
    const float* partial;
    float* out[3];
    int n, sums, groups;
};

constexpr int kSumCols = 32;  // columns of a workgroup

template <int SETS>
__global__ __launch_bounds__(kSumCols * SETS) void norm_sums_kernel(const NormSumsArgs a)
{
    __shared__ float part[SETS][kSumCols];
    const int c = threadIdx.x % kSumCols, set = threadIdx.x / kSumCols;
    const int col = blockIdx.x * kSumCols + c;
    const int64_t step = (int64_t)a.sums * a.n;
    float s = 0.f;
    if (col < a.n) {
        const float* p = a.partial + set * step + (int64_t)blockIdx.y * a.n + col;
        // eight loads in flight, added in order; past the last group zeros
        for (int g = set; g < a.groups; g += 8 * SETS) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = g + k * SETS < a.groups ? p[k * SETS * step] : 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) s += v[k];
            p += 8 * SETS * step;
        }
    }
    part[set][c] = s;
    __syncthreads();
    if (set == 0 && col < a.n) {
        s = 0.f;
#pragma unroll
        for (int k = 0; k < SETS; ++k) s += part[k][c];
        a.out[blockIdx.y][col] = s;
    }
}

}  // namespace gemm_rs_layer
