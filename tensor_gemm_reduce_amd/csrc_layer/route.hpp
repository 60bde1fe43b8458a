// route.hpp -- the router: scores, the choice of k experts for each token, the
// plan of every expert's rows, the gradient of the logits; and a token's rows
// back into one.
//
// A wave takes a token (or 64 / SEG tokens where the experts fit SEG lanes): lane l
// holds experts NV l .. NV l + NV - 1.  Choices have to come out as the formula says, not as
// FP32 rounds it: without a bias and groups scores order as the logits do, which are
// compared as they are; else in 64 bits, where FP32 does not tell.  Either way as unsigned
// keys that order like the values, so that a maximum over the lanes and the lowest lane
// that has it are the choice.  Bytes are few (8192 x 256 logits in FP32: 8 MB, 1.7 us); a
// token's chain of loads, scores and k maxima over the lanes is what takes time (26 us of it; half of the cycles are waits).
#pragma once

#include <type_traits>

#include "common.hpp"

namespace gemm_rs_layer {

constexpr int kPlanIds = 1024;    // choices per workgroup of the plan's kernels, one per thread
constexpr int kRouteTokens = 128; // at most so many tokens per workgroup

// Workgroups count their choices per expert (hist), a second kernel adds the counts up over
// the workgroups before each, and a third gives each choice its row.  One workgroup does
// all by itself.
struct PlanArgs {
    const int32_t* experts;
    int32_t *offsets, *tokens, *slots;
    int32_t* hist;    // [chunks][E]: counts, then the counts before
    int32_t* totals;  // [E]
    int64_t ids;      // T k
    int E, k, chunk, chunks;  // choices per workgroup; workgroups
};

// An unsigned number that orders like v; 1 for a NaN, and never 0.
__device__ __forceinline__ uint32_t route_key(float v)
{
    if (v != v) return 1u;
    const uint32_t b = __float_as_uint(v + 0.f);  // -0 as 0
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t route_key(double v)
{
    if (v != v) return 1u;
    const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
    return b >> 63 ? ~b : b | (uint64_t(1) << 63);
}

// v of another lane of the 16: by the ALU's own exchanges (a shuffle takes the LDS pipe: 8192 x 256 took 35 us with
// shuffles, 31 so).
template <int CTRL, class V>
__device__ __forceinline__ V row_other(V v)
{
    if constexpr (sizeof(V) == 8) {
        const uint64_t b = __builtin_bit_cast(uint64_t, v);
        const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)b, CTRL, 0xF, 0xF, true);
        const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(b >> 32), CTRL, 0xF, 0xF, true);
        return __builtin_bit_cast(V, (uint64_t)hi << 32 | lo);
    } else
        return __builtin_bit_cast(V, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}
// v of lane `at`, the same for all lanes
template <class V>
__device__ __forceinline__ V lane_value(V v, int at)
{
    if constexpr (sizeof(V) == 8) {
        const uint64_t b = __builtin_bit_cast(uint64_t, v);
        const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, at);
        const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), at);
        return __builtin_bit_cast(V, (uint64_t)hi << 32 | lo);
    } else
        return __builtin_bit_cast(V, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), at));
}
// op over the SEG lanes, in every lane
template <int SEG, class V, class OP>
__device__ __forceinline__ V seg_all(V v, OP op)
{
    v = op(v, row_other<0xB1>(v));   // lane ^ 1
    v = op(v, row_other<0x4E>(v));   // lane ^ 2
    v = op(v, row_other<0x141>(v));  // 7 - lane: the other four, which agree
    if constexpr (SEG >= 16) v = op(v, row_other<0x140>(v));  // 15 - lane
    if constexpr (SEG == 32) v = op(v, __shfl_xor(v, 16));
    if constexpr (SEG == 64) v = op(op(lane_value(v, 0), lane_value(v, 16)), op(lane_value(v, 32), lane_value(v, 48)));
    return v;
}
template <int SEG, class V>
__device__ __forceinline__ V seg_max(V v)
{
    return seg_all<SEG>(v, [](V a, V b) { return a > b ? a : b; });
}
template <int SEG>
__device__ __forceinline__ float seg_max(float v)
{
    return seg_all<SEG>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int SEG, class V>
__device__ __forceinline__ V seg_sum(V v)
{
    return seg_all<SEG>(v, [](V a, V b) { return a + b; });
}

__device__ __forceinline__ float route_exp(float v) { return expf(v); }
__device__ __forceinline__ double route_exp(double v) { return exp(v); }

// s = softmax (over the SEG lanes and NV values each) or sigmoid; values of experts that are off are 0.
template <class F, int SEG, int NV>
__device__ __forceinline__ void route_scores(const float (&l)[NV], bool sigmoid, F (&s)[NV])
{
    if (sigmoid) {
#pragma unroll
        for (int i = 0; i < NV; ++i) s[i] = l[i] == -INFINITY ? F(0) : F(1) / (F(1) + route_exp(-(F)l[i]));
        return;
    }
    float top = l[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) top = fmaxf(top, l[i]);
    top = seg_max<SEG>(top);
    if (top == -INFINITY) top = 0.f;  // nothing is on: all zeros
    F sum = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        s[i] = route_exp((F)l[i] - (F)top);
        sum += s[i];
    }
    sum = seg_sum<SEG>(sum);
    const F inv = sum == F(0) ? F(0) : F(1) / sum;
#pragma unroll
    for (int i = 0; i < NV; ++i) s[i] *= inv;
}

struct RouteArgs {
    const void* logits;
    const float* bias;
    float* weights;
    int32_t* experts;
    int64_t T, stride;
    int dtype, E, k, sigmoid, renormalise, groups, keep;
    float scale;
    int tokens;  // per workgroup
    PlanArgs plan;
};

// A lane's logits of token t: experts first, first + step, ..; -inf for those that are not there.  All loads are on their way
// before one is waited for: a token's are a chain of latencies otherwise (8192 x 256: 31 us, 26 so).
template <int NV>
__device__ __forceinline__ void route_load(const void* logits, int dtype, int64_t row, int E, int first, int step, bool live,
                                           float (&l)[NV])
{
    auto load = [&](auto* p) {
        p += row;
        typename std::remove_cv<typename std::remove_reference<decltype(*p)>::type>::type v[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = p[min(first + i * step, E - 1)];
#pragma unroll
        for (int i = 0; i < NV; ++i) l[i] = live && first + i * step < E ? (float)v[i] : -INFINITY;
    };
    if (dtype == 0) load(static_cast<const __bf16*>(logits));
    else if (dtype == 1) load(static_cast<const _Float16*>(logits));
    else load(static_cast<const float*>(logits));
}

// Where the choices of a workgroup go: thread i has choice i of the workgroup's (its expert,
// -1 for none).  Rows count up over the waves' choices in order: a wave finds a choice's
// rank among the same expert's in the wave by comparing indices bit by bit, and the waves'
// counts stand in LDS.  before[e]: the expert's first row of this workgroup.  count:
// [waves][E + 1] 16-bit, and room for E + 1 more words behind it.
__device__ __forceinline__ int plan_rank(int e, bool in, int E, uint16_t* count)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    uint32_t* words = reinterpret_cast<uint32_t*>(count);
    const int pitch = (E + 1) & ~1;
    for (int i = threadIdx.x; i < waves * pitch / 2; i += blockDim.x) words[i] = 0;
    __syncthreads();
    uint64_t same = __ballot(in);
    for (int b = 1; b < E; b <<= 1) {
        const uint64_t m = __ballot((e & b) != 0);
        same &= e & b ? m : ~m;
    }
    const int rank = __popcll(same & ((uint64_t(1) << lane) - 1));
    if (in && rank == 0) count[wave * pitch + e] = (uint16_t)__popcll(same);
    __syncthreads();
    int r = rank;
    if (in)
        for (int w = 0; w < wave; ++w) r += count[w * pitch + e];
    return r;
}

// Exclusive sums over E values v[e] (one per thread, more for small workgroups) in LDS, and the total at E.
__device__ __forceinline__ void scan_experts(int* v, int E, int* part)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    int carry = 0;
    for (int e0 = 0; e0 < E; e0 += blockDim.x) {
        const int e = e0 + threadIdx.x, own = e < E ? v[e] : 0;
        int s = own;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(s, d);
            if (lane >= d) s += o;
        }
        if (lane == 63) part[wave] = s;
        __syncthreads();
        int base = carry, all = 0;
        for (int w = 0; w < waves; ++w) {
            if (w < wave) base += part[w];
            all += part[w];
        }
        carry += all;
        if (e < E) v[e] = base + s - own;
        __syncthreads();
    }
    if (threadIdx.x == 0) v[E] = carry;
    __syncthreads();
}

constexpr int kMaxExperts = 1024;

struct PlanLds {
    uint16_t count[16 * kMaxExperts];
    int before[kMaxExperts + 1];
    int part[16];
};

__device__ __forceinline__ void plan_store(const PlanArgs& a, int64_t id, bool in, int row, int total)
{
    if (id < a.ids) {
        a.slots[id] = in ? row : -1;
        if (in) a.tokens[row] = (int32_t)(id / a.k);
        if (id >= total) a.tokens[id] = -1;
    }
}

// The plan of at most 1024 choices by one workgroup: choice i = thread i.
__device__ __forceinline__ void plan_alone(const PlanArgs& a, PlanLds& s, int e, bool in)
{
    for (int i = threadIdx.x; i < a.E; i += blockDim.x) s.before[i] = 0;
    const int r = plan_rank(e, in, a.E, s.count);
    // the last wave that has an expert knows its number of rows, so each raises the count to its own last rank
    if (in) atomicMax(&s.before[e], r + 1);
    __syncthreads();
    scan_experts(s.before, a.E, s.part);
    for (int i = threadIdx.x; i <= a.E; i += blockDim.x) a.offsets[i] = s.before[i];
    plan_store(a, threadIdx.x, in, in ? s.before[e] + r : 0, s.before[a.E]);
}

// Threads of the router's workgroups, and so choices that one may make: the scores of groups take LDS.
constexpr int route_threads(int nv) { return nv > 4 ? 256 : kPlanIds; }

__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k); }

// What a token's lanes hold after the choice: lane j choice j and its score; the scores' sum; the least distance between a
// choice and the next best expert.
struct Choice {
    int expert;
    float score, sum, gap;
};

// The k largest keys, largest first; the key after the last counts for the distance.  A lane's keys (experts NV lane and on)
// are put in order first, equal ones as they were; then each choice is the largest of the lanes' first keys, the lowest
// lane's of equal ones, which moves up by one.
template <int SEG, int NV, class K>
__device__ __forceinline__ Choice route_choose(K (&key)[NV], const float (&p)[NV], int k)
{
    constexpr bool kGaps = std::is_same<K, uint32_t>::value;
    const int lane = threadIdx.x & 63, sub = lane & (SEG - 1), part = lane / SEG;
    int id[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) id[i] = sub * NV + i;
#pragma unroll
    for (int n = NV; n > 1; --n)
#pragma unroll
        for (int i = 0; i + 1 < n; ++i) {
            const bool swap = key[i + 1] > key[i];
            const K a = swap ? key[i + 1] : key[i], b = swap ? key[i] : key[i + 1];
            const int c = swap ? id[i + 1] : id[i], d = swap ? id[i] : id[i + 1];
            key[i] = a;
            key[i + 1] = b;
            id[i] = c;
            id[i + 1] = d;
        }
    Choice c = {-1, 0.f, 0.f, INFINITY};
    float last = INFINITY;
    for (int j = 0; j < k + (kGaps ? 1 : 0); ++j) {
        const K top = seg_max<SEG>(key[0]);
        if constexpr (kGaps) {
            const float v = key_value(top);
            if (top != 0 && last - v < c.gap) c.gap = last - v;  // NaN's keys are the lowest and have no distance
            last = v;
            if (j == k) break;
        }
        uint64_t m = __ballot(key[0] == top);
        if constexpr (SEG < 64) m = m >> (part * SEG) & ((uint64_t(1) << SEG) - 1);
        const int at = __ffsll((unsigned long long)m) - 1;
        const int e = SEG == 64 ? lane_value(id[0], uni(at)) : __shfl(id[0], part * SEG + at);
        if (sub == j % SEG) c.expert = top != 0 ? e : -1;
        if (sub == at) {
#pragma unroll
            for (int i = 0; i + 1 < NV; ++i) {
                key[i] = key[i + 1];
                id[i] = id[i + 1];
            }
            key[NV - 1] = 0;
        }
    }
    const int from = part * SEG + (c.expert < 0 ? 0 : c.expert / NV);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const float v = __shfl(p[i], from);
        if (c.expert >= 0 && c.expert % NV == i) c.score = v;
    }
    c.sum = seg_sum<SEG>(c.score);
    return c;
}

// Which groups stay, as a mask of lanes: group g's are from g `per` on.  mine: the wave's part of LDS.  gap: the distance of
// the last group that stays from the first that does not.
template <int NV, class F>
__device__ __forceinline__ uint64_t route_groups(const F (&c)[NV], const float (&l)[NV], F* mine, int E, int groups, int keep,
                                                 int& per, F& gap)
{
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < NV; ++i) mine[lane * NV + i] = l[i] == -INFINITY ? (F)-INFINITY : c[i] != c[i] ? (F)-1e30 : c[i];
    __asm__ __volatile__("" ::: "memory");  // the LDS operations of a wave complete in order
    const int size = E / groups;
    per = 64;  // lanes of a group
    while (per * groups > 64) per >>= 1;
    const int group = lane / per;
    F hi = -INFINITY, lo = -INFINITY;
    if (group < groups)
        for (int i = lane % per; i < size; i += per) {
            const F v = mine[group * size + i];
            if (v > hi) {
                lo = hi;
                hi = v;
            } else if (v > lo)
                lo = v;
        }
    for (int d = per / 2; d > 0; d >>= 1) {
        const F oh = __shfl_xor(hi, d), ol = __shfl_xor(lo, d);
        const F third = hi < oh ? hi : oh;  // the smaller of the two largest
        lo = lo > ol ? lo : ol;
        if (third > lo) lo = third;
        if (oh > hi) hi = oh;
    }
    const F total = lo == -INFINITY ? hi : hi + lo;
    int rank = 0;  // how many groups come before this one
    for (int o = 0; o < groups; ++o) {
        const F v = lane_value(total, o * per);
        rank += v > total || (v == total && o < group) ? 1 : 0;
    }
    const bool stays = group < groups && rank < keep;
    const F in = seg_all<64>(stays ? total : (F)INFINITY, [](F a, F b) { return a < b ? a : b; });
    const F out = seg_all<64>(stays || group >= groups ? (F)-INFINITY : total, [](F a, F b) { return a > b ? a : b; });
    // groups that are off are last whatever the others' rounding; sums of two that FP32 does not hold say nothing
    const bool past = group < groups && lo != -INFINITY && (total == INFINITY || total == -INFINITY);
    gap = __any(past) ? (F)0 : out == -INFINITY ? (F)INFINITY : in - out;
    __asm__ __volatile__("" ::: "memory");
    return __ballot(stays);
}

// WIDE: a bias or groups.  The choice is first made in FP32, and stands where all distances in it are more than twice what
// FP32 can be off by: a few roundings of a score (of exp's argument, exp, the sum over the experts, the quotient: some 30 2^-24, so less than
// 2^-18, of the largest) and that of the sum with the bias.  Else, for about a token in a thousand and for equal scores, it is made
// again in 64 bits.
template <int SEG, int NV, bool WIDE>
__global__ __launch_bounds__(route_threads(NV)) void route_kernel(const RouteArgs a)
{
    constexpr int kPer = 64 / SEG;  // tokens of a wave at a time
    constexpr int kThreads = route_threads(NV);
    constexpr bool kGroups = WIDE && SEG == 64;
    __shared__ union {
        PlanLds plan;
        double c[kGroups ? kThreads / 64 : 1][kGroups ? 64 * NV : 1];
    } lds;
    __shared__ int32_t ids[kThreads], hist[kMaxExperts];
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6), waves = kThreads / 64;
    const int sub = lane & (SEG - 1), part = lane / SEG;
    const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
    float bias[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) bias[i] = WIDE && a.bias ? a.bias[min(sub * NV + i, a.E - 1)] : 0.f;
    ids[threadIdx.x] = -1;
    for (int i = threadIdx.x; i < a.E; i += kThreads) hist[i] = 0;
    __syncthreads();
    for (int g = wave * kPer; g < a.tokens; g += waves * kPer) {
        if (t0 + g >= a.T) break;
        const int64_t t = t0 + g + part;
        const bool live = g + part < a.tokens && t < a.T;
        float l[NV], p[NV];
        route_load<NV>(a.logits, a.dtype, (live ? t : a.T - 1) * a.stride, a.E, sub * NV, 1, live, l);
        route_scores<float, SEG, NV>(l, a.sigmoid, p);
        uint32_t key[NV];
        Choice c;
        if constexpr (WIDE) {
            float f[NV], most = 0.f, score = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                f[i] = p[i] + bias[i];
                key[i] = l[i] == -INFINITY ? 0 : route_key(f[i]);
                most = l[i] == -INFINITY ? most : fmaxf(most, fabsf(f[i]));
                score = fmaxf(score, p[i]);
            }
            most = seg_max<SEG>(most);
            score = seg_max<SEG>(score);
            float gap = INFINITY;
            if constexpr (kGroups) if (a.groups > 1) {
                int per;
                const uint64_t kept = route_groups<NV, float>(f, l, reinterpret_cast<float*>(lds.c[wave]), a.E, a.groups, a.keep, per, gap);
                const int size = a.E / a.groups;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int e = lane * NV + i;
                    if (e < a.E && !(kept >> (e / size * per) & 1)) key[i] = 0;
                }
                gap *= 0.5f;  // of sums of two
            }
            c = route_choose<SEG, NV>(key, p, a.k);
            gap = fminf(gap, c.gap);
            const float off = score * 0x1p-18f + most * 0x1p-23f;
            if (__any(live && !(gap > 2.f * off))) {
                double d[NV];
                uint64_t wide[NV];
                route_scores<double, SEG, NV>(l, a.sigmoid, d);
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    d[i] += (double)bias[i];
                    wide[i] = l[i] == -INFINITY ? 0 : route_key(d[i]);
                }
                if constexpr (kGroups) if (a.groups > 1) {
                    int per;
                    double unused;
                    const uint64_t kept = route_groups<NV, double>(d, l, lds.c[wave], a.E, a.groups, a.keep, per, unused);
                    const int size = a.E / a.groups;
#pragma unroll
                    for (int i = 0; i < NV; ++i) {
                        const int e = lane * NV + i;
                        if (e < a.E && !(kept >> (e / size * per) & 1)) wide[i] = 0;
                    }
                }
                c = route_choose<SEG, NV>(wide, p, a.k);
            }
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) key[i] = l[i] == -INFINITY ? 0 : route_key(l[i]);
            c = route_choose<SEG, NV>(key, p, a.k);
        }
        // lane j of the token has choice j (k <= SEG)
        if (live && sub < a.k) {
            const float w = a.renormalise ? c.score / (c.sum + 1e-20f) : c.score;
            a.weights[t * a.k + sub] = a.scale * w;
            a.experts[t * a.k + sub] = c.expert;
            ids[(g + part) * a.k + sub] = c.expert;
            if (a.plan.chunks > 1 && c.expert >= 0) atomicAdd(&hist[c.expert], 1);
        }
    }
    __syncthreads();
    if (a.plan.chunks > 1) {
        for (int i = threadIdx.x; i < a.E; i += kThreads) a.plan.hist[(int64_t)blockIdx.x * a.E + i] = hist[i];
        return;
    }
    const int e = ids[threadIdx.x];
    plan_alone(a.plan, lds.plan, e, e >= 0);
}

// Counts of given choices; all of the plan if one workgroup holds them.
__global__ __launch_bounds__(kPlanIds) void plan_count_kernel(const PlanArgs a)
{
    __shared__ PlanLds s;
    const int64_t id = (int64_t)blockIdx.x * a.chunk + threadIdx.x;
    int e = threadIdx.x < a.chunk && id < a.ids ? a.experts[id] : -1;
    if (e >= a.E) e = -1;
    const bool in = e >= 0;
    if (a.chunks == 1) {
        plan_alone(a, s, e, in);
        return;
    }
    for (int i = threadIdx.x; i < a.E; i += blockDim.x) s.before[i] = 0;
    __syncthreads();
    if (in) atomicAdd(&s.before[e], 1);
    __syncthreads();
    for (int i = threadIdx.x; i < a.E; i += blockDim.x) a.hist[(int64_t)blockIdx.x * a.E + i] = s.before[i];
}

// hist[c][e] becomes the sum over the workgroups before c.  A workgroup takes an expert, a lane a workgroup's count: the
// loads have a line each, but they are few, and only their latency counts.
constexpr int kScanThreads = 256;

__global__ __launch_bounds__(kScanThreads) void plan_scan_kernel(const PlanArgs a)
{
    __shared__ int part[2][kScanThreads / 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, e = blockIdx.x;
    int carry = 0;
    for (int c0 = 0, turn = 0; c0 < a.chunks; c0 += kScanThreads, turn ^= 1) {
        const int c = c0 + threadIdx.x;
        const int own = c < a.chunks ? a.hist[(int64_t)c * a.E + e] : 0;
        int s = own;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(s, d);
            if (lane >= d) s += o;
        }
        if (lane == 63) part[turn][wave] = s;
        __syncthreads();  // one for each turn: the next one writes the other half
        int before = carry;
#pragma unroll
        for (int w = 0; w < kScanThreads / 64; ++w) {
            before += w < wave ? part[turn][w] : 0;
            carry += part[turn][w];
        }
        if (c < a.chunks) a.hist[(int64_t)c * a.E + e] = before + s - own;
    }
    if (threadIdx.x == 0) a.totals[e] = carry;
}

// One thread for each choice of the workgroup's.
__global__ __launch_bounds__(kPlanIds) void plan_place_kernel(const PlanArgs a)
{
    __shared__ PlanLds s;
    for (int i = threadIdx.x; i < a.E; i += blockDim.x) s.before[i] = a.totals[i];
    __syncthreads();
    scan_experts(s.before, a.E, s.part);
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i <= a.E; i += blockDim.x) a.offsets[i] = s.before[i];
    const int64_t id = (int64_t)blockIdx.x * a.chunk + threadIdx.x;
    const bool mine = threadIdx.x < a.chunk && id < a.ids;
    int e = mine ? a.experts[id] : -1;
    if (e >= a.E) e = -1;
    const bool in = e >= 0;
    const int r = plan_rank(e, in, a.E, s.count);
    if (mine) plan_store(a, id, in, in ? s.before[e] + a.hist[(int64_t)blockIdx.x * a.E + e] + r : 0, s.before[a.E]);
}

struct RouteGradArgs {
    const void* logits;
    const int32_t* experts;
    const float* dweights;
    void* dlogits;
    int64_t T, stride, dstride;
    int dtype, E, k, sigmoid, renormalise;
    float scale;
};

// Scores are computed again.  ds is what the weights pass to the scores that were chosen;
// softmax: dl = s (ds - sum ds s), sigmoid: dl = ds s (1 - s).  Where one score is nearly all, what is left are the others'
// parts, which differences of nearly equal numbers lose (a hundredth of 1 - s at a sigmoid's logit of 12, all of it from 17 on):
//   sigmoid      1 - s is 1 / (1 + e^l)
//   softmax      for a score above a half, 1 - s is the sum of the others, and its own term leaves sum ds s
//   renormalise  (dw_i - sum_j dw_j s_j / D) / D is sum_j s_j (dw_i - dw_j) / D^2, and 1e-20 dw_i / D^2
template <int SEG, int NV>
__global__ __launch_bounds__(256) void route_backward_kernel(const RouteGradArgs a)
{
    constexpr int kPer = 64 / SEG;
    const int lane = threadIdx.x & 63, sub = lane & (SEG - 1), part = lane / SEG;
    const int64_t t = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * kPer + part;
    const bool live = t < a.T;
    float l[NV], p[NV], ds[NV];
    route_load<NV>(a.logits, a.dtype, (live ? t : a.T - 1) * a.stride, a.E, sub, 64, live, l);
#pragma unroll
    for (int i = 0; i < NV; ++i) ds[i] = 0.f;
    int e = -1;
    float dw = 0.f;
    if (live && sub < a.k) {
        e = a.experts[t * a.k + sub];
        if (e < 0 || e >= a.E) e = -1;
        else dw = a.scale * a.dweights[t * a.k + sub];
    }
    route_scores<float, SEG, NV>(l, a.sigmoid, p);
    float s = 0.f;  // the score of this lane's choice
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const float v = __shfl(p[i], part * SEG + (e & (SEG - 1)));
        if (e >= 0 && e / 64 == i) s = v;
    }
    auto choice = [&](auto v, int j) {  // choice j's
        if constexpr (SEG == 64) return lane_value(v, j);
        else return __shfl(v, part * SEG + j);
    };
    if (a.renormalise) {
        const float inv = 1.f / (seg_sum<SEG>(s) + 1e-20f);
        float sum = 1e-20f * dw;
        for (int j = 0; j < a.k; ++j) sum += choice(s, j) * (dw - choice(dw, j));
        dw = e < 0 ? 0.f : sum * inv * inv;
    }
    for (int j = 0; j < a.k; ++j) {
        const int ej = choice(e, j);
        const float dj = choice(dw, j);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (ej == i * 64 + sub) ds[i] += dj;
    }
    float rest = 0.f, dot = 0.f, all = 0.f;  // sums of s and ds s without a score above a half, of ds s
    if (!a.sigmoid) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const float d = ds[i] * p[i];
            rest += p[i] > 0.5f ? 0.f : p[i];
            dot += p[i] > 0.5f ? 0.f : d;
            all += p[i] > 0.5f ? d : 0.f;
        }
        rest = seg_sum<SEG>(rest);
        dot = seg_sum<SEG>(dot);
        all = dot + seg_sum<SEG>(all);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int at = i * 64 + sub;
        if (!live || at >= a.E) continue;
        const float d = a.sigmoid      ? ds[i] * (p[i] * (1.f / (1.f + expf(l[i]))))
                        : p[i] > 0.5f ? p[i] * (ds[i] * rest - dot)
                                      : p[i] * (ds[i] - all);
        const int64_t to = t * a.dstride + at;
        if (a.dtype == 0) static_cast<__bf16*>(a.dlogits)[to] = (__bf16)d;
        else if (a.dtype == 1) static_cast<_Float16*>(a.dlogits)[to] = (_Float16)d;
        else static_cast<float*>(a.dlogits)[to] = d;
    }
}

// ---- rows back to tokens -----------------------------------------------------------

struct CombineArgs {
    const void *y, *dout;
    const int32_t* slots;
    const float* weights;
    void *out, *dy;
    float* dweights;
    int64_t T, R, y_stride, out_stride, dout_stride, dy_stride;
    int N, k;
};

constexpr int kCombineThreads = 256;
constexpr int kCombineAhead = 8;  // rows of a token in flight

// A thread sums eight columns of a token's rows; bytes bound it.
template <class T>
__global__ __launch_bounds__(kCombineThreads) void combine_kernel(const CombineArgs a)
{
    const int64_t t = blockIdx.x;
    const int col = (blockIdx.y * kCombineThreads + threadIdx.x) * 8;
    if (col >= a.N) return;
    float acc[8] = {};
    for (int j0 = 0; j0 < a.k; j0 += kCombineAhead) {
        vec8<T> v[kCombineAhead];
        float w[kCombineAhead];
        bool has[kCombineAhead];
#pragma unroll
        for (int j = 0; j < kCombineAhead; ++j) {
            const int64_t at = t * a.k + j0 + j;
            const int slot = j0 + j < a.k ? a.slots[at] : -1;
            has[j] = slot >= 0 && slot < a.R;
            w[j] = has[j] && a.weights ? a.weights[at] : 1.f;
            v[j] = has[j] ? load8(static_cast<const T*>(a.y) + slot * a.y_stride, col, a.N) : vec8<T>{};
        }
#pragma unroll
        for (int j = 0; j < kCombineAhead; ++j)
            if (has[j]) {
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] = __builtin_fmaf(w[j], (float)v[j][i], acc[i]);
            }
    }
    store8(static_cast<T*>(a.out) + t * a.out_stride, col, a.N, acc);
}

// A workgroup takes a token, so that dout is read once for kCombineAhead rows: each is
// multiplied with it (the weight's gradient) and written as the weight times it.
template <class T>
__global__ __launch_bounds__(kCombineThreads) void combine_backward_kernel(const CombineArgs a)
{
    __shared__ float part[kCombineThreads / 64][kCombineAhead];
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int j0 = 0; j0 < a.k; j0 += kCombineAhead) {
        int slot[kCombineAhead];
        float w[kCombineAhead], dot[kCombineAhead];
#pragma unroll
        for (int j = 0; j < kCombineAhead; ++j) {
            const int64_t at = t * a.k + j0 + j;
            slot[j] = j0 + j < a.k ? a.slots[at] : -1;
            if (slot[j] >= a.R) slot[j] = -1;
            w[j] = slot[j] >= 0 && a.weights ? a.weights[at] : 1.f;
            dot[j] = 0.f;
        }
        for (int col = threadIdx.x * 8; col < a.N; col += kCombineThreads * 8) {
            float d[8];
            widen<T>(load8(static_cast<const T*>(a.dout) + t * a.dout_stride, col, a.N), d);
            vec8<T> v[kCombineAhead];
            if (a.dweights)
#pragma unroll
                for (int j = 0; j < kCombineAhead; ++j)
                    if (slot[j] >= 0) v[j] = load8(static_cast<const T*>(a.y) + slot[j] * a.y_stride, col, a.N);
#pragma unroll
            for (int j = 0; j < kCombineAhead; ++j)
                if (slot[j] >= 0) {
                    float f[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (a.dweights) dot[j] = __builtin_fmaf(d[i], (float)v[j][i], dot[j]);
                        f[i] = w[j] * d[i];
                    }
                    store8(static_cast<T*>(a.dy) + slot[j] * a.dy_stride, col, a.N, f);
                }
        }
        if (!a.dweights) continue;
#pragma unroll
        for (int j = 0; j < kCombineAhead; ++j) {
            const float sum = wave_sum(dot[j]);
            if (lane == 0) part[wave][j] = sum;
        }
        __syncthreads();
        const int j = threadIdx.x;
        if (j < kCombineAhead && j0 + j < a.k) {
            float sum = 0.f;
#pragma unroll
            for (int v = 0; v < kCombineThreads / 64; ++v) sum += part[v][j];
            a.dweights[t * a.k + j0 + j] = sum;
        }
        __syncthreads();
    }
}

}  // namespace gemm_rs_layer
