// block_norm.hpp -- what follows the row-parallel layer: the sum of the ranks'
// partials, the norm after the block, its gate and scale, the residual and the
// norm before the next block, and the gradients of all of them.
#pragma once

#include <type_traits>

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
template <class T, class R, int THREADS, int ITEMS, int MAXP>
__global__ __launch_bounds__(THREADS) void norm_forward_kernel(const NormArgs a)
{
    __shared__ float slots[2][THREADS / 64];
    const int64_t row = blockIdx.x;
    const int n = a.n;
    float v[ITEMS][8];

    // every part's chunk in flight at once where the registers hold them (1024
    // threads have 128 each: one chunk's parts at a time)
    constexpr int kAhead = THREADS < 1024 ? ITEMS : 1;
#pragma unroll
    for (int i0 = 0; i0 < ITEMS; i0 += kAhead) {
        vec8<T> p[MAXP][kAhead];
#pragma unroll
        for (int k = 0; k < MAXP; ++k)
            if (k < a.nparts) {
                const T* src = static_cast<const T*>(a.parts[k]) + row * a.part_stride;
#pragma unroll
                for (int i = 0; i < kAhead; ++i) p[k][i] = load8(src, ((i0 + i) * THREADS + (int)threadIdx.x) * 8, n);
            }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            widen<T>(p[0][i], v[i0 + i]);
#pragma unroll
            for (int k = 1; k < MAXP; ++k)
                if (k < a.nparts) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[i0 + i][j] += (float)p[k][i][j];
                }
        }
    }

    const R* rrow = static_cast<const R*>(a.residual) + row * a.residual_stride;
    vec8<R> res[kAhead];  // before the first sum over the row, with the parts
    if (kAhead == ITEMS) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            res[i] = vec8<R>{};
            if (a.residual) res[i] = load8(rrow, (i * THREADS + (int)threadIdx.x) * 8, n);
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
            const vec8<T> w = load8(static_cast<const T*>(a.post_weight), (i * THREADS + (int)threadIdx.x) * 8, n);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * ry * (float)w[j];
        }
    }

    float row_scale = a.block_scale;
    if (a.gate_kind == GEMM_RS_GATE_TOKEN) row_scale *= (float)static_cast<const T*>(a.gate)[row];
    const bool gated = a.gate_kind == GEMM_RS_GATE_CHANNEL || a.gate_kind == GEMM_RS_GATE_FULL;
    const T* gate = static_cast<const T*>(a.gate) + (a.gate_kind == GEMM_RS_GATE_FULL ? row * a.gate_stride : 0);
    R* hrow = static_cast<R*>(a.h) + row * a.h_stride;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const int col = (i * THREADS + (int)threadIdx.x) * 8;
        if (gated) {
            const vec8<T> g = load8(gate, col, n);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] *= (float)g[j];
        }
        if (kAhead < ITEMS) {
            res[0] = vec8<R>{};
            if (a.residual) res[0] = load8(rrow, col, n);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float h = row_scale * v[i][j];
            if (a.residual) h += a.residual_scale * (float)res[kAhead == ITEMS ? i : 0][j];
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
            const vec8<T> w = load8(static_cast<const T*>(a.pre_weight), col, n);
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

// Keeps the loads of a later chunk from being moved up into registers that an
// earlier one still needs.
__device__ __forceinline__ void one_chunk_at_a_time() { __asm__ __volatile__("" ::: "memory"); }

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

// Workgroup g takes rows g, g + grid, ...  With t^ = t r (r = 1 / rms(t)) a norm
// t^ w passes a gradient d on as r (w d - t^ mean(w d t^)); the statistics come
// from the forward pass, so the two means are the only sums over a row (a third
// one is the gradient of a gate per row).  The sums over rows stay in registers
// and leave as one partial row per workgroup (norm_sums_kernel adds them).
// WIDE (rows too wide for that): the inputs are read again where they are needed
// again, from cache, and the sums over rows are kept in the workgroup's partial
// row.
template <class T, class R, int THREADS, int ITEMS, bool WIDE>
__global__ __launch_bounds__(THREADS) void norm_backward_kernel(const NormGradArgs a)
{
    __shared__ float slots[3][THREADS / 64];
    constexpr int kHeld = WIDE ? 1 : ITEMS;
    const int n = a.n;
    const float inv_n = 1.f / (float)n;
    const bool pre = a.pre_weight != nullptr, post = a.post_weight != nullptr;
    const bool channel = a.gate_kind == GEMM_RS_GATE_CHANNEL, full = a.gate_kind == GEMM_RS_GATE_FULL;
    const bool token = a.gate_kind == GEMM_RS_GATE_TOKEN;
    const bool need_y = post || a.gate_kind != GEMM_RS_GATE_NONE;
    const T* const gate = static_cast<const T*>(a.gate);
    float* const part_pre = a.partial + (int64_t)blockIdx.x * a.sums * n;
    float* const part_post = part_pre + (pre ? n : 0);
    float* const part_gate = part_post + (post ? n : 0);
    auto column = [](int i) { return (i * THREADS + (int)threadIdx.x) * 8; };
    auto load_if = [&](bool on, auto* p, int i) {
        auto v = vec8<std::remove_cv_t<std::remove_pointer_t<decltype(p)>>>{};
        if (on) v = load8(p, column(i), n);
        return v;
    };

    float sum_pre[kHeld][8] = {}, sum_post[kHeld][8] = {}, sum_gate[kHeld][8] = {};
    vec8<T> wpre[kHeld], wpost[kHeld], wgate[kHeld];
    if constexpr (!WIDE) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            wpre[i] = load_if(pre, static_cast<const T*>(a.pre_weight), i);
            wpost[i] = load_if(post, static_cast<const T*>(a.post_weight), i);
            wgate[i] = load_if(channel, gate, i);
        }
    }

    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T* const dzrow = static_cast<const T*>(a.dz) + row * a.dz_stride;
        const T* const yrow = static_cast<const T*>(a.y) + row * a.y_stride;
        const R* const hrow = static_cast<const R*>(a.h) + row * a.h_stride;
        const R* const dhrow = static_cast<const R*>(a.dh) + row * a.dh_stride;
        const T* const gaterow = gate + (full ? row * a.gate_stride : 0);
        vec8<T> dz[kHeld], y[kHeld], gf[kHeld];
        vec8<R> dh[kHeld], hv[kHeld];
        if constexpr (!WIDE) {
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                dz[i] = load_if(pre, dzrow, i);
                hv[i] = load_if(pre, hrow, i);
                dh[i] = load_if(a.dh != nullptr, dhrow, i);
                y[i] = load_if(need_y, yrow, i);
                gf[i] = load_if(full, gaterow, i);
            }
        }
        const float ry = post ? a.rstd[row] : 1.f;
        const float rh = pre ? a.rstd[a.rows + row] : 0.f;
        const float g_row = token ? (float)gate[row] : 1.f;

        // through the next block's norm
        float mean_h = 0.f;
        if (pre) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                if constexpr (WIDE) {
                    one_chunk_at_a_time();
                    dz[0] = load_if(true, dzrow, i);
                    hv[0] = load_if(true, hrow, i);
                    wpre[0] = load_if(true, static_cast<const T*>(a.pre_weight), i);
                }
                const int k = WIDE ? 0 : i;
#pragma unroll
                for (int j = 0; j < 8; ++j) s += (float)wpre[k][j] * (float)dz[k][j] * ((float)hv[k][j] * rh);
            }
            mean_h = block_sum<THREADS>(s, slots[0]) * inv_n;
        }
        float d[ITEMS][8];  // the gradient of h, then of u
        float s_tok = 0.f, s_y = 0.f;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int col = column(i), k = WIDE ? 0 : i;
            if constexpr (WIDE) {
                one_chunk_at_a_time();
                dz[0] = load_if(pre, dzrow, i);
                hv[0] = load_if(pre, hrow, i);
                dh[0] = load_if(a.dh != nullptr, dhrow, i);
                y[0] = load_if(need_y, yrow, i);
                gf[0] = load_if(full, gaterow, i);
                wpre[0] = load_if(pre, static_cast<const T*>(a.pre_weight), i);
                wpost[0] = load_if(post, static_cast<const T*>(a.post_weight), i);
                wgate[0] = load_if(channel, gate, i);
                if (row != blockIdx.x) {
                    widen<float>(load_if(pre, part_pre, i), sum_pre[0]);
                    widen<float>(load_if(post, part_post, i), sum_post[0]);
                    widen<float>(load_if(channel, part_gate, i), sum_gate[0]);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum_pre[0][j] = sum_post[0][j] = sum_gate[0][j] = 0.f;
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float g = (float)dh[k][j];
                if (pre) {
                    const float hh = (float)hv[k][j] * rh, z = (float)dz[k][j];
                    g += rh * ((float)wpre[k][j] * z - hh * mean_h);
                    sum_pre[k][j] += z * hh;
                }
                d[i][j] = g;
            }
            if (a.dresidual) {
                float o[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = a.residual_scale * d[i][j];
                store8(static_cast<R*>(a.dresidual) + row * a.dresidual_stride, col, n, o);
            }
            float dg[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float yy = (float)y[k][j] * ry;
                const float u = post ? yy * (float)wpost[k][j] : yy;
                float g = a.block_scale * d[i][j];
                dg[j] = g * u;
                s_tok += dg[j];
                if (channel) {
                    sum_gate[k][j] += dg[j];
                    g *= (float)wgate[k][j];
                }
                if (full) g *= (float)gf[k][j];
                if (token) g *= g_row;
                if (post) {
                    sum_post[k][j] += g * yy;
                    g *= (float)wpost[k][j];
                    s_y += g * yy;
                }
                d[i][j] = g;
            }
            if (full) store8(static_cast<T*>(a.dgate) + row * a.dgate_stride, col, n, dg);
            if constexpr (WIDE) {
                if (pre) store8(part_pre, col, n, sum_pre[0]);
                if (post) store8(part_post, col, n, sum_post[0]);
                if (channel) store8(part_gate, col, n, sum_gate[0]);
            }
        }
        if (token) {
            const float t = block_sum<THREADS>(s_tok, slots[1]);
            if (threadIdx.x == 0) static_cast<T*>(a.dgate)[row] = (T)t;
        }
        // through the block's own norm
        float mean_y = 0.f;
        if (post) mean_y = block_sum<THREADS>(s_y, slots[2]) * inv_n;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int k = WIDE ? 0 : i;
            if (post) {
                if constexpr (WIDE) {
                    one_chunk_at_a_time();
                    y[0] = load_if(true, yrow, i);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) d[i][j] = ry * (d[i][j] - (float)y[k][j] * ry * mean_y);
            }
            store8(static_cast<T*>(a.dy) + row * a.dy_stride, column(i), n, d[i]);
        }
        __syncthreads();  // the slots are free for the next row
    }

    if constexpr (!WIDE) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            if (pre) store8(part_pre, column(i), n, sum_pre[i]);
            if (post) store8(part_post, column(i), n, sum_post[i]);
            if (channel) store8(part_gate, column(i), n, sum_gate[i]);
        }
    }
}

// Adds the workgroups' partial sums, in workgroup order within each of eight
// strided sets and then over the sets.  blockIdx.y is the sum, out[] its target.
struct NormSumsArgs {
    const float* partial;
    float* out[3];
    int n, sums, groups;
};

constexpr int kSumCols = 32, kSumSets = 8;

__global__ __launch_bounds__(kSumCols * kSumSets) void norm_sums_kernel(const NormSumsArgs a)
{
    __shared__ float part[kSumSets][kSumCols];
    const int c = threadIdx.x % kSumCols, set = threadIdx.x / kSumCols;
    const int col = blockIdx.x * kSumCols + c;
    float s = 0.f;
    if (col < a.n)
        for (int g = set; g < a.groups; g += kSumSets)
            s += a.partial[((int64_t)g * a.sums + blockIdx.y) * a.n + col];
    part[set][c] = s;
    __syncthreads();
    if (set == 0 && col < a.n) {
        s = 0.f;
#pragma unroll
        for (int k = 0; k < kSumSets; ++k) s += part[k][c];
        a.out[blockIdx.y][col] = s;
    }
}

}  // namespace gemm_rs_layer
