// gfx950 kernels of the routing of tokens to experts: the choice of k experts per token
// with its weights, its backward pass, the plan that sorts the choices by expert, and the
// combination of the experts' rows, forward and backward.
#pragma once

#include "fused.hpp"

namespace tgemm {

enum { DT_F32 = 2 };
enum { SCORE_SOFTMAX = 0, SCORE_SIGMOID = 1 };
enum { GROUP_MAX = 0, GROUP_TOP2 = 1 };

constexpr int kMaxExperts = 1024, kMaxChoices = 64, kMaxExpertGroups = 64;

template <int DT>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
    if constexpr (DT == DT_F32)
        return static_cast<const float*>(p)[i];
    else
        return to_float<DT>(static_cast<const u16*>(p)[i]);
}

// Orders a wave's LDS writes before its other lanes' reads: the hardware completes a
// wave's LDS accesses in order, the compiler is kept from moving them.
__device__ __forceinline__ void wave_lds_sync() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// Reductions over the 64 lanes of a wave, the result in every lane: four rotations within
// rows of 16 lanes and two swaps of rows, all in vector registers (a shuffle through LDS
// takes five times as long).
template <int CTRL>
__device__ __forceinline__ uint32_t row_rotate(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
}
template <int CTRL>
__device__ __forceinline__ float row_rotate(float v) {
    return __uint_as_float(row_rotate<CTRL>(__float_as_uint(v)));
}
template <int CTRL>
__device__ __forceinline__ double row_rotate(double v) {
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    const uint64_t lo = row_rotate<CTRL>((uint32_t)u), hi = row_rotate<CTRL>((uint32_t)(u >> 32));
    return __longlong_as_double((long long)(lo | hi << 32));
}
// The value with odd and even rows of 16 lanes (ROWS 16) or the two halves (ROWS 32) paired
// up: both members of the pair, in every lane.
template <int ROWS>
__device__ __forceinline__ u32x2 swap_rows(uint32_t v) {
    if constexpr (ROWS == 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        return u32x2{r[0], r[1]};
    } else {
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        return u32x2{r[0], r[1]};
    }
}
template <int ROWS, typename OP>
__device__ __forceinline__ float over_rows(float v, OP&& op) {
    const u32x2 r = swap_rows<ROWS>(__float_as_uint(v));
    return op(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
template <int ROWS, typename OP>
__device__ __forceinline__ double over_rows(double v, OP&& op) {
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    const u32x2 lo = swap_rows<ROWS>((uint32_t)u), hi = swap_rows<ROWS>((uint32_t)(u >> 32));
    return op(__longlong_as_double((long long)((uint64_t)lo[0] | (uint64_t)hi[0] << 32)),
              __longlong_as_double((long long)((uint64_t)lo[1] | (uint64_t)hi[1] << 32)));
}
template <typename T, typename OP>
__device__ __forceinline__ T wave_all(T v, OP&& op) {
    v = op(v, row_rotate<0x128>(v));
    v = op(v, row_rotate<0x124>(v));
    v = op(v, row_rotate<0x122>(v));
    v = op(v, row_rotate<0x121>(v));
    v = over_rows<16>(v, op);
    return over_rows<32>(v, op);
}
template <typename T>
__device__ __forceinline__ T wave_max(T v) {
    return wave_all(v, [](T a, T b) { return a > b ? a : b; });
}
template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
    return wave_all(v, [](T a, T b) { return a + b; });
}
__device__ __forceinline__ float lane_value(float v, int lane) {
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), lane));
}
// e^x within two units in the last place: 2^(x log2 e) with the rounding of the product
// carried along.  x above -104 (below, e^x is zero in fp32) and at most 88.
__device__ __forceinline__ float exp_fine(float x) {
    x = fmaxf(x, -104.0f);
    const float h = x * 1.44269504f;
    float r = fmaf(x, 1.44269504f, -h);
    r = fmaf(x, 1.92596299e-8f, r);
    const float e = __builtin_amdgcn_exp2f(h);
    return fmaf(e, r * 0.693147181f, e);
}
__device__ __forceinline__ float logistic_fine(float x) {
    return __builtin_amdgcn_rcpf(1.0f + exp_fine(fminf(-x, 88.0f)));
}
// A float's bits in an order that integers have: for values that are not NaN.
__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t u = __float_as_uint(v);
    return u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
}

// ------------------------------------------------------------------------------------
// Routing.  One wave per token; lane l holds the V experts l V .. l V + V - 1, so that the
// lowest lane with a value holds the lowest index with it.
//   s = softmax(x) or logistic(x), the selection value c = s + bias, or c = x where there
//   is neither a bias nor a choice of groups (s rises with x); with groups, the experts of
//   the topk_groups best groups only (a group's score: its largest c, or the sum of its
//   two largest); then the k largest c, the lowest index first among equals.
//   A logit that is -infinity or NaN, or whose c is, is never chosen; +infinity counts as
//   the largest finite value.
//   w = s of the chosen (the bias only selects), divided by the token's sum of them with
//   `renormalize`, times scale.  Choices past the last candidate: id -1, weight 0.
// SCORED: c comes from the scores.  In fp32 the scores of unlike logits round to equal
// values, and which of two near experts is chosen would depend on the order of a sum: the
// choice is made in fp32 where every comparison that it rests on has a margin of several
// times the scores' error, else the token is done again in fp64.  Not SCORED: the logits
// themselves are compared, exactly.
//   The fp32 choice: a search over the lanes' largest values (one ballot per step) finds a
//   bound that a few more than k values reach; those go to LDS, one per lane, and each
//   counts the ones before it.  Rounds that take one largest value after the other cost
//   three times the instructions (16384 tokens, 256 experts in 8 groups: 52 us so, 27 by the
//   search, whose 588 vector instructions a token are what bounds it); they remain where more than 64 values reach the
//   bound (ties), and in fp64.
struct RouteArgs {
    const void* x;
    const float* bias;
    int32_t* ids;
    float* weights;
    int64_t ldx;
    int32_t tokens, experts, k, scoring, groups, topk_groups, group_score, renormalize;
    float scale;
};

// One token's choice: lane i < k gets the i-th id and its selection score's source (the
// score s, or not SCORED the logit).
template <typename T>
struct Choice {
    int id = -1;
    T value = 0;
};

// The exact rounds: the wave's largest value, its lowest lane, that lane's lowest expert.
// c is used up.
template <typename T, int V>
__device__ __forceinline__ Choice<T> choose_in_rounds(T (&c)[V], const T (&s)[V], int k, int lane) {
    constexpr T kNone = -__builtin_inf();
    Choice<T> r;
    for (int i = 0; i < k; ++i) {
        T m = c[0];
#pragma unroll
        for (int v = 1; v < V; ++v)
            m = c[v] > m ? c[v] : m;
        const T best = wave_max(m);
        if (!(best > kNone))
            break;
        const int from = __builtin_ctzll(__ballot(m == best));
        int at = -1;
        T score = 0;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (at < 0 && c[v] == best) {
                at = v;
                score = s[v];
                if (lane == from)
                    c[v] = kNone;
            }
        const int e = __shfl(lane * V + at, from);
        score = __shfl(score, from);
        if (lane == i) {
            r.id = e;
            r.value = score;
        }
    }
    return r;
}

// The best groups, one at a time; lane g holds group g's score.
__device__ __forceinline__ unsigned long long groups_in_rounds(double score, int topk_groups, int lane) {
    constexpr double kNone = -__builtin_inf();
    unsigned long long kept = 0;
    for (int i = 0; i < topk_groups; ++i) {
        const double m = wave_max(score);
        if (!(m > kNone))
            break;
        const int g = __builtin_ctzll(__ballot(score == m));
        kept |= 1ull << g;
        if (lane == g)
            score = kNone;
    }
    return kept;
}

// Half the margin that an fp32 comparison of selection values needs, relative to |c| + s:
// the exponential, the sum over the experts and the division or addition are together
// within 16 units in the last place (2^-20) for the scores that compete for a choice.
constexpr float kMargin = 3.8147e-6f;   // 2^-18

template <int DT, int V, bool SCORED>
__global__ void __launch_bounds__(256) route_tokens(const RouteArgs p) {
    constexpr float kNone = -__builtin_inff();
    __shared__ double group_c[SCORED ? 4 : 1][SCORED ? 64 * V : 1];
    __shared__ float found_c[4][64], found_s[4][64];
    __shared__ int found_e[4][64];
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * 4 + wave;
    if (t >= p.tokens)
        return;                            // no barrier below: a wave works on its own
    float x[V];
    float top = kNone;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = lane * V + v;
        float a = e < p.experts ? load_logit<DT>(p.x, t * p.ldx + e) : kNone;
        a = a == a ? a : kNone;
        x[v] = (a < __builtin_inff() ? a : 3.402823466e38f) + 0.0f;   // -0 becomes +0
        top = fmaxf(top, x[v]);
    }
    top = wave_max(top);
    const float base = top > kNone ? top : 0.0f;
    const bool softmax = p.scoring == SCORE_SOFTMAX;

    // scores and selection values in fp32
    float s[V], c[V], total = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
        s[v] = c[v] = x[v];
    if (SCORED || (softmax && !p.renormalize)) {
        // masked logits come out as 0 (softmax) or next to it, and are masked again below
        float w[V], bias[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = lane * V + v;
            bias[v] = SCORED && p.bias ? p.bias[e < p.experts ? e : 0] : 0.0f;
        }
        if (softmax) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                w[v] = exp_fine(x[v] - base);
                total += w[v];
            }
            total = wave_sum(total);
        } else {
            total = 1.0f;
#pragma unroll
            for (int v = 0; v < V; ++v)
                w[v] = logistic_fine(x[v]);
        }
        if constexpr (SCORED) {
            const float inv = softmax ? (total > 0.0f ? 1.0f / total : 0.0f) : 1.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                s[v] = w[v] * inv;
                const float cv = s[v] + bias[v];
                c[v] = x[v] > kNone && cv == cv ? cv : kNone;
            }
        }
    }
    bool sure = true;                      // every comparison so far had its margin
    const bool choose_groups = SCORED && p.topk_groups < p.groups;
    const int size = SCORED ? p.experts / p.groups : 1;
    // e / size for e below 1024: the product is at least 1 / 2048 away from a whole number
    const float per_size = 1.0f / (float)size;
    const auto group_of = [&](int e) { return (int)(((float)e + 0.5f) * per_size); };
    if (choose_groups) {
        // lane g scores group g
        float best = kNone, second = kNone;
        const int lanes = size / V;
        if (size % V == 0 && (lanes & (lanes - 1)) == 0) {
            // a group is `lanes` whole lanes, a power of two: its two largest by shuffles
#pragma unroll
            for (int v = 0; v < V; ++v) {
                second = fmaxf(second, fminf(best, c[v]));
                best = fmaxf(best, c[v]);
            }
            for (int d = 1; d < lanes; d *= 2) {
                const float b2 = __shfl_xor(best, d), s2 = __shfl_xor(second, d);
                second = fmaxf(fmaxf(second, s2), fminf(best, b2));
                best = fmaxf(best, b2);
            }
            best = __shfl(best, lane * lanes < 64 ? lane * lanes : 0);
            second = __shfl(second, lane * lanes < 64 ? lane * lanes : 0);
        } else {
            float* row = reinterpret_cast<float*>(group_c[wave]);
#pragma unroll
            for (int v = 0; v < V; ++v)
                row[lane * V + v] = c[v];
            wave_lds_sync();
            if (lane < p.groups)
                for (int i = 0; i < size; ++i) {
                    const float a = row[lane * size + i];
                    second = fmaxf(second, fminf(best, a));
                    best = fmaxf(best, a);
                }
            wave_lds_sync();
        }
        float score = lane < p.groups ? best : kNone;
        if (p.group_score == GROUP_TOP2 && second > kNone)
            score += second;
        score = lane < p.groups ? score : kNone;
        // a group's place: the groups before it
        int place = 0;
        for (int g = 0; g < p.groups; ++g) {
            const float o = lane_value(score, g);
            place += o > score || (o == score && g < lane);
        }
        const bool keep = lane < p.groups && place < p.topk_groups && score > kNone;
        const unsigned long long kept = __ballot(keep);
        // the last group kept and the first one left need a margin between them
        const unsigned long long in = __ballot(lane < p.groups && place == p.topk_groups - 1);
        const unsigned long long out = __ballot(lane < p.groups && place == p.topk_groups);
        const float a = lane_value(score, __builtin_ctzll(in)), b = lane_value(score, __builtin_ctzll(out));
        sure = !(a > kNone) || !(b > kNone) || a - b > 4.0f * kMargin * (fabsf(a) + 2.0f);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = lane * V + v;
            if (e < p.experts && !((kept >> group_of(e)) & 1))
                c[v] = kNone;
        }
    }

    Choice<float> got;
    bool placed = false;
    if (sure) {
        // the largest bound that more than k lanes' largest values reach (all valid ones, if
        // there are fewer), to 16 bits
        float m = c[0];
#pragma unroll
        for (int v = 1; v < V; ++v)
            m = fmaxf(m, c[v]);
        const uint32_t key = ordered(m);
        uint32_t bound = 0;
#pragma unroll
        for (int bit = 31; bit >= 16; --bit) {
            const uint32_t tryit = bound | (1u << bit);
            if (__popcll(__ballot(key >= tryit)) > p.k)
                bound = tryit;
        }
        const uint32_t low = ordered(kNone);
        bound = bound > low ? bound : low + 1;
        // their places in LDS follow the experts' order: those of the lanes before, then the
        // lane's own
        int n = 0, at = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const unsigned long long mask = __ballot(ordered(c[v]) >= bound);
            at = __builtin_amdgcn_mbcnt_lo((uint32_t)mask, at);
            at = __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), at);
            n += __popcll(mask);
        }
        if (n <= 64) {
            placed = true;
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (ordered(c[v]) >= bound) {
                    found_c[wave][at] = c[v];
                    found_s[wave][at] = s[v];
                    found_e[wave][at] = lane * V + v;
                    ++at;
                }
            wave_lds_sync();
            const bool mine = lane < n;
            const float fc = mine ? found_c[wave][lane] : kNone, fs = mine ? found_s[wave][lane] : 0.0f;
            const int fe = mine ? found_e[wave][lane] : -1;
            int place = 0;
#pragma unroll 4
            for (int i = 0; i < n; ++i) {
                const float o = lane_value(fc, i);
                place += i < lane ? o >= fc : o > fc;
            }
            wave_lds_sync();
            if (mine) {
                found_c[wave][place] = fc;
                found_s[wave][place] = fs;
                found_e[wave][place] = fe;
            }
            wave_lds_sync();
            if (lane < n && lane < p.k) {
                got.id = found_e[wave][lane];
                got.value = found_s[wave][lane];
            }
            if constexpr (SCORED) {
                bool near = false;
                if (lane < p.k && lane + 1 < n) {
                    const float a = found_c[wave][lane], b = found_c[wave][lane + 1];
                    const float scale = fabsf(a) + found_s[wave][lane] + found_s[wave][lane + 1];
                    near = !(a - b > 2.0f * kMargin * scale);
                }
                sure = __ballot(near) == 0;
            }
        }
    }
    float w;
    if constexpr (SCORED) {
        if (!sure || !placed) {
            // the token in fp64
            double s64[V], c64[V], sum = 0;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                s64[v] = x[v] > kNone ? (softmax ? exp((double)x[v] - (double)base) : 1.0 / (1.0 + exp(-(double)x[v])))
                                      : 0.0;
                sum += s64[v];
            }
            sum = softmax ? wave_sum(sum) : 1.0;
            const double inv = sum > 0 ? 1.0 / sum : 0.0;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int e = lane * V + v;
                s64[v] *= inv;
                const double cv = s64[v] + (p.bias && e < p.experts ? (double)p.bias[e] : 0.0);
                c64[v] = x[v] > kNone && cv == cv ? cv : -__builtin_inf();
            }
            if (choose_groups) {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    group_c[wave][lane * V + v] = c64[v];
                wave_lds_sync();
                double best = -__builtin_inf(), second = best;
                if (lane < p.groups)
                    for (int i = 0; i < size; ++i) {
                        const double a = group_c[wave][lane * size + i];
                        second = a > best ? best : (a > second ? a : second);
                        best = a > best ? a : best;
                    }
                if (p.group_score == GROUP_TOP2 && second > -__builtin_inf())
                    best += second;
                const unsigned long long kept = groups_in_rounds(best, p.topk_groups, lane);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int e = lane * V + v;
                    if (e < p.experts && !((kept >> group_of(e)) & 1))
                        c64[v] = -__builtin_inf();
                }
            }
            const Choice<double> exact = choose_in_rounds<double, V>(c64, s64, p.k, lane);
            got.id = exact.id;
            got.value = (float)exact.value;
        }
        w = got.id >= 0 ? got.value : 0.0f;
    } else {
        if (!placed)
            got = choose_in_rounds<float, V>(c, s, p.k, lane);
        w = softmax ? exp_fine(got.value - base) / (p.renormalize ? 1.0f : total) : logistic_fine(got.value);
        w = got.id >= 0 ? w : 0.0f;
    }
    if (p.renormalize) {
        const float sum = wave_sum(w);
        w = sum > 0.0f ? w / sum : w;
    }
    if (lane < p.k) {
        p.ids[t * p.k + lane] = got.id;
        p.weights[t * p.k + lane] = w * p.scale;
    }
}

// ------------------------------------------------------------------------------------
// The logits' gradient for fixed choices.  With w'_j the weights before the scale and
// g_j = scale dw_j:
//   softmax                dx_e = s_e ([e chosen] g_e - sum_j g_j s_j)
//   softmax, renormalized  dx_e = [e chosen] w'_e (g_e - sum_j g_j w'_j)
//   logistic               dx_e = [e chosen] g_e s_e (1 - s_e)
//   logistic, renormalized dx_e = [e chosen] w'_e (1 - s_e) (g_e - sum_j g_j w'_j)
// One wave per token, everything in fp32; choices outside the experts are passed over.
// 8192 tokens of 128 experts in bf16: 6.6 us, 275 vector instructions a token.
// ------------------------------------------------------------------------------------
struct RouteGradArgs {
    const void* x;
    const int32_t* ids;
    const float* dw;
    void* dx;
    int64_t ldx, lddx;
    int32_t tokens, experts, k, scoring, renormalize;
    float scale;
};

template <int DT, int V>
__global__ void __launch_bounds__(256) route_grad(const RouteGradArgs p) {
    constexpr float kNone = -__builtin_inff();
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * 4 + wave;
    if (t >= p.tokens)
        return;
    const int my_id = lane < p.k ? p.ids[t * p.k + lane] : -1;
    const float my_dw = lane < p.k ? p.dw[t * p.k + lane] * p.scale : 0.0f;
    float x[V], g[V];
    bool mine[V];
    float top = kNone;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = lane * V + v;
        float a = e < p.experts ? load_logit<DT>(p.x, t * p.ldx + e) : kNone;
        a = a == a ? a : kNone;
        x[v] = a < __builtin_inff() ? a : 3.402823466e38f;
        top = fmaxf(top, x[v]);
        g[v] = 0.0f;
        mine[v] = false;
    }
    for (int i = 0; i < p.k; ++i) {
        const int e = __builtin_amdgcn_readlane(my_id, i);
        const float d = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(my_dw), i));
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (e == lane * V + v) {
                mine[v] = true;
                g[v] += d;
            }
    }
    top = wave_max(top);
    const float base = top > kNone ? top : 0.0f;
    float s[V], total = 0.0f;               // scores; softmax: up to their common divisor
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (x[v] > kNone)
            s[v] = p.scoring == SCORE_SOFTMAX ? exp_fine(x[v] - base) : logistic_fine(x[v]);
        else
            s[v] = 0.0f;
        total += p.renormalize ? (mine[v] ? s[v] : 0.0f) : s[v];
    }
    const bool share = p.renormalize || p.scoring == SCORE_SOFTMAX;
    total = wave_sum(total);
    const float inv = share ? (total > 0.0f ? 1.0f / total : 0.0f) : 1.0f;
    float dot = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
        dot += mine[v] ? g[v] * (s[v] * inv) : 0.0f;
    dot = share ? wave_sum(dot) : 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = lane * V + v;
        if (e >= p.experts)
            continue;
        float d = 0.0f;
        if (mine[v] || (p.scoring == SCORE_SOFTMAX && !p.renormalize))
            d = s[v] * inv * (g[v] - dot);
        if (p.scoring == SCORE_SIGMOID)
            d *= logistic_fine(-x[v]);       // 1 - s
        if constexpr (DT == DT_F32)
            static_cast<float*>(p.dx)[t * p.lddx + e] = d;
        else
            static_cast<u16*>(p.dx)[t * p.lddx + e] = cvt1<DT>(d);
    }
}

// ------------------------------------------------------------------------------------
// The plan: a stable counting sort of the `total` choices (token-major) by expert.
//   offsets[e]  the first row of expert e; order[r] the choice behind row r; slots[c] the
//   row of choice c.  A choice outside the experts has no row (slot -1); order is -1 past
//   the last row.
// Each wave owns a contiguous run of choices, 64 at a time, and its own count per expert
// in LDS; lanes with equal experts find each other by one ballot per bit of the index, so
// ranks follow the order of the choices whatever the schedule.  Up to kPlanChunk choices
// one workgroup does all of it; beyond, plan_count writes the count of each chunk of
// choices and plan_place, one workgroup per chunk, adds up the chunks before its own.
// Bound by latency: 131072 choices of 256 experts 3.8 + 8.6 us, 64 of 64 3.3 us.
// ------------------------------------------------------------------------------------
constexpr int kPlanChunk = 4096, kPlanWaves = 16;   // one workgroup's choices, its waves

struct PlanArgs {
    const int32_t* ids;
    int32_t* offsets;
    int32_t* order;
    int32_t* slots;
    int32_t* counts;       // [chunks][experts] (more than one chunk)
    int64_t total;
    int32_t experts, chunks;
};

// The lanes of this wave whose expert is this lane's (itself included); 0 for lanes
// without one.
__device__ __forceinline__ unsigned long long equal_lanes(int e, int experts) {
    const bool live = e >= 0;
    unsigned long long m = __ballot(live);
    for (int b = 1; b < experts; b *= 2) {
        const unsigned long long set = __ballot(live && (e & b));
        m &= (e & b) ? set : ~set;
    }
    return live ? m : 0ull;
}

__device__ __forceinline__ int plan_expert(const PlanArgs& p, int64_t i) {
    if (i >= p.total)
        return -1;
    const int e = p.ids[i];
    return e >= 0 && e < p.experts ? e : -1;
}

static __global__ void __launch_bounds__(1024) plan_count(const PlanArgs p) {
    __shared__ int count[kMaxExperts];
    const int tid = (int)threadIdx.x;
    int e[kPlanChunk / 1024];
#pragma unroll
    for (int q = 0; q < kPlanChunk / 1024; ++q)
        e[q] = plan_expert(p, (int64_t)blockIdx.x * kPlanChunk + q * 1024 + tid);
    if (tid < p.experts)
        count[tid] = 0;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kPlanChunk / 1024; ++q)
        if (e[q] >= 0)
            atomicAdd(&count[e[q]], 1);    // a sum of ones: the order does not matter
    __syncthreads();
    if (tid < p.experts)
        p.counts[(int64_t)blockIdx.x * p.experts + tid] = count[tid];
}

// CAP: the most experts.
template <int CAP>
__global__ void __launch_bounds__(kPlanWaves * 64) plan_place(const PlanArgs p) {
    __shared__ int waves[kPlanWaves * CAP];        // [kPlanWaves][experts]
    __shared__ int first_row[CAP];                 // this chunk's first row of each expert
    __shared__ int scan[kPlanWaves];
    static_assert(CAP <= kPlanWaves * 64, "one thread per expert");
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t chunk0 = (int64_t)blockIdx.x * kPlanChunk;
    const int64_t left = p.total - chunk0;
    const int n = left < kPlanChunk ? (int)left : kPlanChunk;
    // this wave's run of choices: whole groups of 64
    const int per_wave = ((n + kPlanWaves * 64 - 1) / (kPlanWaves * 64)) * 64;
    const int w0 = wave * per_wave, w1 = w0 + per_wave < n ? w0 + per_wave : n;
    constexpr int R = kPlanChunk / (kPlanWaves * 64);   // a lane's choices, at most
    int mine[R];
#pragma unroll
    for (int q = 0; q < R; ++q) {
        const int i = w0 + 64 * q + lane;
        mine[q] = i < w1 ? plan_expert(p, chunk0 + i) : -1;
    }
    for (int i = tid; i < kPlanWaves * p.experts; i += kPlanWaves * 64)
        waves[i] = 0;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < R; ++q)
        if (mine[q] >= 0)
            atomicAdd(&waves[wave * p.experts + mine[q]], 1);
    __syncthreads();
    // each expert's choices: in all, before this chunk, and before each wave of it
    int all = 0, before = 0;
    if (tid < p.experts) {
        int here = 0;
        for (int w = 0; w < kPlanWaves; ++w) {
            const int c = waves[w * p.experts + tid];
            waves[w * p.experts + tid] = here;
            here += c;
        }
        all = here;
        if (p.chunks > 1) {
            all = 0;
#pragma unroll 16
            for (int b = 0; b < p.chunks; ++b) {
                const int c = p.counts[(int64_t)b * p.experts + tid];
                before += b < (int)blockIdx.x ? c : 0;
                all += c;
            }
        }
    }
    // exclusive scan of `all` over the experts
    int sum = all;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int o = __shfl_up(sum, d);
        sum += lane >= d ? o : 0;
    }
    if (lane == 63)
        scan[wave] = sum;
    __syncthreads();
    int base = 0, rows = 0;
    for (int w = 0; w < kPlanWaves; ++w) {
        base += w < wave ? scan[w] : 0;
        rows += scan[w];
    }
    if (tid < p.experts) {
        first_row[tid] = base + sum - all + before;
        if (blockIdx.x == 0)
            p.offsets[tid] = base + sum - all;
    }
    if (blockIdx.x == 0 && tid == 0)
        p.offsets[p.experts] = rows;
    __syncthreads();
    // the rows, 64 choices at a time; the wave's count of an expert moves on by the lanes
    // that hold it (a wave's LDS accesses complete in order)
#pragma unroll
    for (int q = 0; q < R; ++q) {
        const int i = w0 + 64 * q + lane, e = mine[q];
        if (w0 + 64 * q >= w1)
            break;
        const unsigned long long same = equal_lanes(e, p.experts);
        int r = -1;
        if (e >= 0) {
            const int at = waves[wave * p.experts + e];
            r = first_row[e] + at + __popcll(same & ((1ull << lane) - 1));
            if (lane == 63 - __builtin_clzll(same))
                waves[wave * p.experts + e] = at + __popcll(same);
            p.order[r] = (int)(chunk0 + i);
        }
        wave_lds_sync();
        if (i < w1)
            p.slots[chunk0 + i] = r;
    }
    // no choice behind the rows past the last expert's
    for (int i = tid; i < n; i += kPlanWaves * 64)
        if (chunk0 + i >= rows)
            p.order[chunk0 + i] = -1;
}

// ------------------------------------------------------------------------------------
// The combination: Y[t] = residual[t] + sum_j w[t,j] O[slot[t,j]], summed in fp32 in the
// order of j and rounded once.  A thread owns eight columns of a token; the k rows' loads
// are independent of each other.  Bound by memory: 4096 tokens of 8 rows of 2048 in 29 us,
// 5.7 TB/s.
// ------------------------------------------------------------------------------------
struct CombineArgs {
    const u16* O;
    const int32_t* slots;
    const float* weights;      // null: all one
    const u16* residual;       // null: none; may be Y itself
    u16* Y;
    int32_t tokens, k, width, rows, ldo, ldr, ldy, vec;
};

template <int DT>
__global__ void __launch_bounds__(256) combine_rows(const CombineArgs p) {
    const int runs = (p.width + 7) / 8;
    const int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t t = q / runs;
    if (t >= p.tokens)
        return;
    const int n = (int)(q - t * runs) * 8, left = p.width - n;
    auto sum = [&](auto wholec) {
        constexpr bool WHOLE = decltype(wholec)::value;
        float y[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (p.residual)
            unpack8<DT>(load8_raw<WHOLE>(p.residual + t * p.ldr + n, left), y);
        // four choices' loads at a time
        for (int j0 = 0; j0 < p.k; j0 += 4) {
            u32x4 o_raw[4];
            float w[4];
            bool live[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int64_t c = t * p.k + (j0 + q < p.k ? j0 + q : p.k - 1);
                const int slot = p.slots[c];
                live[q] = j0 + q < p.k && slot >= 0 && slot < p.rows;
                w[q] = p.weights ? p.weights[c] : 1.0f;
                if (live[q])
                    o_raw[q] = load8_raw<WHOLE>(p.O + (int64_t)slot * p.ldo + n, left);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (live[q]) {
                    float o[8];
                    unpack8<DT>(o_raw[q], o);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        y[e] = fmaf(w[q], o[e], y[e]);
                }
        }
        store8<DT>(p.Y + t * p.ldy + n, WHOLE, left, y);
    };
    if (p.vec && left >= 8)
        sum(std::true_type{});
    else
        sum(std::false_type{});
}

// Its backward pass: dO[slot[t,j]] = w[t,j] dY[t] and dw[t,j] = <dY[t], O[slot[t,j]]>, one
// wave per choice (the waves of a token read the same dY row, from cache), the inner
// product in fp32.  A choice without a row has dw 0.  1998 choices of 1024 in 6.3 us.
struct CombineGradArgs {
    const u16* dY;
    const u16* O;              // null: dw is not wanted
    const int32_t* slots;
    const float* weights;      // null: all one
    u16* dO;                   // null: not wanted
    float* dw;
    int64_t choices;
    int32_t k, width, rows, lddy, ldo, lddo, vec;
};

template <int DT>
__global__ void __launch_bounds__(256) combine_grad(const CombineGradArgs p) {
    const int lane = (int)threadIdx.x & 63;
    const int64_t c = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (c >= p.choices)
        return;
    const int slot = p.slots[c];
    const bool live = slot >= 0 && slot < p.rows;
    const int64_t t = c / p.k;
    float dot = 0.0f;
    if (live) {
        const float w = p.weights ? p.weights[c] : 1.0f;
        auto run = [&](auto wholec, int n) {
            constexpr bool WHOLE = decltype(wholec)::value;
            const int left = p.width - n;
            float dy[8], o[8];
            u32x4 o_raw{};
            const u32x4 dy_raw = load8_raw<WHOLE>(p.dY + t * p.lddy + n, left);
            if (p.dw)
                o_raw = load8_raw<WHOLE>(p.O + (int64_t)slot * p.ldo + n, left);
            unpack8<DT>(dy_raw, dy);
            if (p.dw) {
                unpack8<DT>(o_raw, o);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    dot = fmaf(dy[e], o[e], dot);
            }
            if (p.dO) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    dy[e] *= w;
                store8<DT>(p.dO + (int64_t)slot * p.lddo + n, WHOLE, left, dy);
            }
        };
        for (int n = lane * 8; n < p.width; n += 512) {
            if (p.vec && n + 8 <= p.width)
                run(std::true_type{}, n);
            else
                run(std::false_type{}, n);
        }
    }
    if (p.dw) {
        dot = wave_sum(dot);
        if (lane == 0)
            p.dw[c] = dot;
    }
}

}  // namespace tgemm
