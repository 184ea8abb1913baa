// gfx950 kernels of the products with an epilogue (gemm_fused) and of the products over
// ragged groups of rows (gemm_grouped), forward and backward.
//
//   z[s,n] = sum_k a(s,k) b_g(n,k) + bias_g[n]          s a row of group g
//   C[s,n] = act(z[s,n]) + residual[s,n]                 or, gated, with h = N / 2,
//   C[s,n] = act(z[s,n]) * z[s,n+h] + residual[s,n]      n < h
//
// A plain product is one group of all rows.  Groups are runs of rows of C (and of A, or of
// an index into A) between consecutive offsets, which lie in device memory: the host does
// not know them, launches the most tiles that any offsets could need, and each workgroup
// finds its tile by a prefix sum over the groups' tile counts.  Everything up to the one
// rounding of C (and of z, where it is kept for the backward pass) is fp32.
#pragma once

#include "kernels.hpp"

namespace tgemm {

enum { ACT_NONE = 0, ACT_RELU, ACT_GELU, ACT_GELU_TANH, ACT_SILU };

// One call, as the kernels see it.  Sizes fit 32 bits; rows times a leading dimension may
// not, and is computed in 64.
struct FusedArgs {
    const u16* A;
    const u16* B;
    u16* C;
    const u16* bias;       // [N] per group, or null
    const u16* residual;   // rows of C's width, or null; may be C itself
    u16* preact;           // rows of N, or null
    const int32_t* offsets;    // [groups + 1], or null: one group of all rows
    const int32_t* row_index;  // row s of the product is row row_index[s] / row_div of A
    int64_t stride_b, stride_c, stride_bias;   // elements between groups
    int32_t rows;          // rows of C (the offsets stay within them)
    int32_t a_rows;        // rows of A
    int32_t N, K, lda, ldb, ldc, ldr, ldp;
    int32_t groups, row_div, act, gated;
    int32_t vec;           // VEC_*: tensors that take 16-byte accesses at multiples of 8
};
enum { VEC_C = 1, VEC_RES = 2, VEC_PRE = 4, VEC_BIAS = 8 };

__device__ __forceinline__ int clamp_row(int v, int rows) { return v < 0 ? 0 : (v > rows ? rows : v); }

// Rows [lo, hi) of group g; offsets out of order or past the rows give an empty or a
// shortened group, never an access outside the tensors.
__device__ __forceinline__ void group_rows(const FusedArgs& p, int g, int& lo, int& hi) {
    if (!p.offsets) {
        lo = 0;
        hi = p.rows;
        return;
    }
    lo = clamp_row(p.offsets[g], p.rows);
    hi = clamp_row(p.offsets[g + 1], p.rows);
    if (hi < lo)
        hi = lo;
}

// The A row behind row s of the product; -1 (read as zeros) where the index points
// outside A.
__device__ __forceinline__ int a_row_of(const FusedArgs& p, int s) {
    if (!p.row_index)
        return s;
    const int v = p.row_index[s];
    const int r = p.row_div == 1 ? v : v / p.row_div;
    return v >= 0 && r < p.a_rows ? r : -1;
}

// The tile of workgroup `wg` when every group is cut into tiles of BM rows, each with
// grid_n column tiles: its group, first row, end row and column tile.  False past the
// last tile.  The order is tile_of's over all groups' row tiles, so that the row tiles of
// one group, which share its B, run on one XCD at the same time.  Every wave computes the
// same prefix sum over the groups, 64 at a time.
template <int BM>
__device__ __forceinline__ bool find_tile(const FusedArgs& p, int wg, int grid_n, int group_m, int& g,
                                          int& row0, int& row_end, int& tn) {
    int tm;
    if (!p.offsets) {
        const int gm = (p.rows + BM - 1) / BM;
        if (wg >= gm * grid_n)
            return false;
        tile_of(wg, gm, grid_n, group_m, tm, tn);
        g = 0;
        row0 = tm * BM;
        row_end = p.rows;
        return true;
    }
    const int lane = (int)threadIdx.x & 63;
    // all groups' tiles
    int total = 0;
    for (int g0 = 0; g0 < p.groups; g0 += 64) {
        int lo = 0, hi = 0;
        if (g0 + lane < p.groups)
            group_rows(p, g0 + lane, lo, hi);
        int t = (hi - lo + BM - 1) / BM;
#pragma unroll
        for (int d = 1; d < 64; d *= 2)
            t += __shfl_xor(t, d);
        total += t;
    }
    total = __builtin_amdgcn_readfirstlane(total);
    if (wg >= total * grid_n)
        return false;
    tile_of(wg, total, grid_n, group_m, tm, tn);
    int before = 0;
    for (int g0 = 0; g0 < p.groups; g0 += 64) {
        int lo = 0, hi = 0;
        if (g0 + lane < p.groups)
            group_rows(p, g0 + lane, lo, hi);
        const int t = (hi - lo + BM - 1) / BM;
        int sum = t;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int o = __shfl_up(sum, d);
            sum += lane >= d ? o : 0;
        }
        const unsigned long long past = __ballot(before + sum > tm);
        if (past) {
            const int at = __builtin_ctzll(past);
            g = g0 + at;
            const int first = before + __builtin_amdgcn_readlane(sum - t, at);
            row0 = __builtin_amdgcn_readlane(lo, at) + (tm - first) * BM;
            row_end = __builtin_amdgcn_readlane(hi, at);
            return true;
        }
        before += __builtin_amdgcn_readlane(sum, 63);
    }
    return false;
}

// ------------------------------------------------------------------------------------
// Activations in fp32, with the hardware's exp2 and reciprocal (one unit in the last
// place each): their results are rounded to 16 bits, whose half step is 2^-12 at best.
// ------------------------------------------------------------------------------------
__device__ __forceinline__ float logistic(float x) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * x));
}

// Phi(-a) for a >= 0 as 2^Q(a): log2 Phi(-a) is close to a parabola, and Q, of degree 7,
// was fitted to it on [0, 6] for the least absolute error (3.3e-6 in the exponential,
// 6.5e-6 evaluated in fp32).  Beyond 6, where Phi(-a) < 1e-9, Q falls on (its leading
// coefficient is negative): 2e-3 relative at 8.3.  One transcendental instead of the two
// of erfc's usual forms: the 8192^3 product with GELU takes 729 us so and 749 with erfc_pos.
__device__ __forceinline__ float normal_tail(float a) {
    float q = fmaf(a, -1.8348411e-6f, 6.159888e-5f);
    q = fmaf(a, q, -9.3052925e-4f);
    q = fmaf(a, q, 8.507907e-3f);
    q = fmaf(a, q, -5.3960098e-2f);
    q = fmaf(a, q, -0.45846437f);
    q = fmaf(a, q, -1.1512511f);
    q = fmaf(a, q, -0.9999953f);
    return __builtin_amdgcn_exp2f(q);
}

// erfc(u) for u >= 0 as exp(-u^2) t P(t), t = 1 / (1 + 0.43 u), the form of Hastings
// ("Approximations for Digital Computers", 1955): P, of degree 7, was fitted to
// exp(u^2) erfc(u) / t on [0, 12] for the least relative error, 1.8e-7.  For the slopes,
// whose column sums are kept in fp32.
__device__ __forceinline__ float erfc_pos(float u, float& gauss) {
    const float t = __builtin_amdgcn_rcpf(fmaf(0.43f, u, 1.0f));
    gauss = __builtin_amdgcn_exp2f(-1.44269504f * u * u);
    float q = fmaf(t, 0.07092017f, -0.29907167f);
    q = fmaf(t, q, 0.3647995f);
    q = fmaf(t, q, -0.06887345f);
    q = fmaf(t, q, 0.23823461f);
    q = fmaf(t, q, 0.20746253f);
    q = fmaf(t, q, 0.24398948f);
    q = fmaf(t, q, 0.24253866f);
    return t * q * gauss;
}

constexpr float kGeluTanh = 1.59576912f;    // 2 sqrt(2 / pi): (1 + tanh(u / 2)) / 2 = logistic(u)

__device__ __forceinline__ float activate(int act, float x) {
    switch (act) {
    case ACT_RELU: return x > 0.0f ? x : (x != x ? x : 0.0f);
    case ACT_GELU: {
        // x Phi(x) = max(x, 0) - |x| Phi(-|x|)
        // a NaN comes through the tail; an infinity leaves 1e30 * 0 of the second term
        const float a = fabsf(x);
        return fmaf(-fminf(a, 1e30f), normal_tail(a), fmaxf(x, 0.0f));
    }
    case ACT_GELU_TANH: return x * logistic(kGeluTanh * (x + 0.044715f * x * x * x));
    case ACT_SILU: return x * logistic(x);
    default: return x;
    }
}

// Value and slope of an activation.
__device__ __forceinline__ void activate_slope(int act, float x, float& value, float& slope) {
    switch (act) {
    case ACT_RELU:
        value = x > 0.0f ? x : (x != x ? x : 0.0f);
        slope = x > 0.0f ? 1.0f : 0.0f;
        break;
    case ACT_GELU: {
        // Phi(x) = 1/2 +- (1/2 - erfc(|x| / sqrt(2)) / 2); x in the density is kept finite
        float gauss;                       // exp(-x^2 / 2)
        const float tail = erfc_pos(0.70710678f * fabsf(x), gauss);
        const float phi = 0.5f + copysignf(fmaf(-0.5f, tail, 0.5f), x);
        value = x * phi;
        slope = fmaf(__builtin_amdgcn_fmed3f(x, -100.0f, 100.0f) * 0.39894228f, gauss, phi);
        break;
    }
    case ACT_GELU_TANH: {
        const float p = logistic(kGeluTanh * (x + 0.044715f * x * x * x));
        value = x * p;
        slope = p + value * (1.0f - p) * kGeluTanh * (1.0f + 0.134145f * x * x);
        break;
    }
    case ACT_SILU: {
        const float p = logistic(x);
        value = x * p;
        slope = p + value * (1.0f - p);
        break;
    }
    default:
        value = x;
        slope = 1.0f;
    }
}

// ------------------------------------------------------------------------------------
// Runs of eight 16-bit values: one 16-byte access where the tensor allows it and all
// eight lie inside, else one by one.
// ------------------------------------------------------------------------------------
template <int DT>
__device__ __forceinline__ float to_float(u16 h) {
    if constexpr (DT == DT_F16)
        return (float)__builtin_bit_cast(_Float16, h);
    else
        return __uint_as_float((uint32_t)h << 16);
}

template <int DT>
__device__ __forceinline__ void unpack8(u32x4 v, float (&x)[8]) {
    const u16x8 h = __builtin_bit_cast(u16x8, v);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        x[e] = to_float<DT>(h[e]);
}

// WHOLE: the caller has branched on the tensor's alignment and the run lying inside, so that
// several loads go out together.
template <bool WHOLE>
__device__ __forceinline__ u32x4 load8_raw(const u16* p, int left) {
    if constexpr (WHOLE)
        return *reinterpret_cast<const u32x4*>(p);
    u16x8 h;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        h[e] = e < left ? p[e] : (u16)0;
    return __builtin_bit_cast(u32x4, h);
}

template <int DT>
__device__ __forceinline__ void load8(const u16* p, bool vec, int left, float (&x)[8]) {
    unpack8<DT>(vec && left >= 8 ? load8_raw<true>(p, left) : load8_raw<false>(p, left), x);
}

// STREAM: with the non-temporal hint, for z, which nothing reads before the backward pass.
// (On C the hint takes 4 % off the experts' products of 1024 k by themselves, and costs the
// combination that reads C next as much: it finds less of it in the last-level cache.)
template <int DT, bool STREAM = false>
__device__ __forceinline__ void store8(u16* p, bool vec, int left, const float* x) {
    const u32x4 v{pack2<DT>(x[0], x[1]), pack2<DT>(x[2], x[3]), pack2<DT>(x[4], x[5]),
                  pack2<DT>(x[6], x[7])};
    if (vec && left >= 8) {
        if constexpr (STREAM)
            __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(p));
        else
            *reinterpret_cast<u32x4*>(p) = v;
    } else {
        const u16x8 h = __builtin_bit_cast(u16x8, v);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < left)
                p[e] = h[e];
    }
}

// The bias of eight columns n .. n+7 of group g (and, gated, of the eight h on).
template <int DT>
__device__ __forceinline__ void load_bias(const FusedArgs& p, int g, int n, int width, float (&bz)[8],
                                          float (&bu)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
        bz[e] = bu[e] = 0.0f;
    if (p.bias && n < width) {
        const u16* b = p.bias + g * p.stride_bias + n;
        load8<DT>(b, p.vec & VEC_BIAS, width - n, bz);
        if (p.gated)
            load8<DT>(b + width, p.vec & VEC_BIAS, width - n, bu);
    }
}

// An activation over a run of values: one uniform branch for all of them.
template <int COUNT>
__device__ __forceinline__ void activate_all(int act, float* z) {
    switch (act) {
    case ACT_RELU:
#pragma unroll
        for (int e = 0; e < COUNT; ++e)
            z[e] = activate(ACT_RELU, z[e]);
        break;
    case ACT_GELU:
#pragma unroll
        for (int e = 0; e < COUNT; ++e)
            z[e] = activate(ACT_GELU, z[e]);
        break;
    case ACT_GELU_TANH:
#pragma unroll
        for (int e = 0; e < COUNT; ++e)
            z[e] = activate(ACT_GELU_TANH, z[e]);
        break;
    case ACT_SILU:
#pragma unroll
        for (int e = 0; e < COUNT; ++e)
            z[e] = activate(ACT_SILU, z[e]);
        break;
    default: break;
    }
}

// The epilogue of Q runs of eight columns n .. n+7 (n < width, C's) of the rows s, s + STEP,
// .. below `end`: z holds the products there and, gated, u the products h columns on; bz and
// bu their bias.  The runs go through each stage together, so that their memory accesses
// and their chains of arithmetic overlap.
template <int DT, int Q, int STEP, bool GATED>
__device__ __forceinline__ void finish_runs(const FusedArgs& p, int s, int end, int n, int width, float (&z)[Q * 8],
                                            float (&u)[GATED ? Q * 8 : 1], const float (&bz)[8],
                                            const float (&bu)[8]) {
    const int left = width - n;
    u32x4 raw[Q];                          // the residual, where it is read whole
    const bool whole = p.residual && (p.vec & VEC_RES) && left >= 8;
    if (whole) {
#pragma unroll
        for (int q = 0; q < Q; ++q)
            if (s + q * STEP < end)
                raw[q] = *reinterpret_cast<const u32x4*>(p.residual + (int64_t)(s + q * STEP) * p.ldr + n);
    }
    if (p.bias) {
#pragma unroll
        for (int e = 0; e < Q * 8; ++e) {
            z[e] += bz[e & 7];
            if constexpr (GATED)
                u[e] += bu[e & 7];
        }
    }
    if (p.preact) {
#pragma unroll
        for (int q = 0; q < Q; ++q)
            if (s + q * STEP < end) {
                u16* to = p.preact + (int64_t)(s + q * STEP) * p.ldp + n;
                store8<DT, true>(to, p.vec & VEC_PRE, left, z + q * 8);
                if constexpr (GATED)
                    store8<DT, true>(to + width, p.vec & VEC_PRE, left, u + q * 8);
            }
    }
    activate_all<Q * 8>(p.act, z);
    if constexpr (GATED) {
#pragma unroll
        for (int e = 0; e < Q * 8; ++e)
            z[e] *= u[e];
    }
    if (whole) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            float r[8];
            unpack8<DT>(raw[q], r);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                z[q * 8 + e] += r[e];
        }
    } else if (p.residual) {
#pragma unroll
        for (int q = 0; q < Q; ++q)
            if (s + q * STEP < end) {
                float r[8];
                load8<DT>(p.residual + (int64_t)(s + q * STEP) * p.ldr + n, false, left, r);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    z[q * 8 + e] += r[e];
            }
    }
#pragma unroll
    for (int q = 0; q < Q; ++q)
        if (s + q * STEP < end)
            store8<DT>(p.C + (int64_t)(s + q * STEP) * p.ldc + n, p.vec & VEC_C, left, z + q * 8);
}

// The B row (column of the product) of column c of column tile tn, whose tile is BN wide;
// -1 past the end.  Gated, 32-column blocks take turns between the two halves of N, so
// that a lane that holds a gate value also holds, one block on, the value it multiplies.
template <int BN>
__device__ __forceinline__ int b_row_of(const FusedArgs& p, int tn, int c) {
    if (!p.gated) {
        const int n = tn * BN + c;
        return n < p.N ? n : -1;
    }
    const int h = p.N >> 1, n = tn * (BN / 2) + (c >> 6) * 32 + (c & 31);
    return n < h ? n + ((c >> 5) & 1) * h : -1;
}

// ------------------------------------------------------------------------------------
// The generic kernel: any alignment, size and layout.  64 x 64 tile, K step 64, four
// waves of one 32 x 32 MFMA block each; C through an fp32 tile in the same LDS.
//   Elements are loaded singly, a wave's 64 lanes along the contiguous dimension (whole
// 128-byte pieces): 32 loads per lane and step, those of the next step in flight beside the
// MFMAs.  An operand whose k is not the contiguous dimension is turned in registers: a
// lane's 16 k of one column go to LDS in two 16-byte writes.
//   Bound by the single-element loads: 316 TFLOP/s at 4096 x 4096 x 4097 (bf16, [N,K]; 115
// with steps of 16 and nothing in flight), 23 us for 1000 x 1000 x 1001 (66), 80 us for
// 4 x 8192 x 4097 (275); the sum over 4096 rows to 4097 x 4096 512 us (268 TFLOP/s).
// ------------------------------------------------------------------------------------
constexpr int kGenericStep = 64, kGenericRow = kGenericStep + 8;   // k per step; LDS row (odd 16-byte pieces)

// Element `at` (in: it lies in the rows) of sixteen rows, the i-th held by lane i of `mine`
// (< 0: a row of zeros).  Called by whole waves.  One element to a register: held as 16-bit
// values they are packed in pairs where they are loaded, which waits for every second load.
__device__ __forceinline__ void load_rows(uint32_t (&v)[16], const u16* base, int64_t ld, int mine, int64_t at, bool in) {
    int row[16];           // read while all lanes are active
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        row[i] = __builtin_amdgcn_readlane(mine, i);
        v[i] = 0;
    }
    if (in) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (row[i] >= 0)
                v[i] = base[row[i] * ld + at];
    }
}

// Lane l's values are k = 16 wave + i of column l.
__device__ __forceinline__ void put_turned(u16* lds, int lane, int wave, const uint32_t (&v)[16]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        u32x4 w;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            w[q] = v[8 * h + 2 * q] | v[8 * h + 2 * q + 1] << 16;
        *reinterpret_cast<u32x4*>(lds + lane * kGenericRow + wave * 16 + 8 * h) = w;
    }
}

// Lane l's values are k = l of rows 16 wave + i.
__device__ __forceinline__ void put_rows(u16* lds, int lane, int wave, const uint32_t (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
        lds[(wave * 16 + i) * kGenericRow + lane] = (u16)v[i];
}

template <int DT>
__device__ __forceinline__ void generic_step(f32x16& acc, const u16* left, const u16* right, int lane, int wm, int wn) {
#pragma unroll
    for (int s = 0; s < kGenericStep / 16; ++s) {
        const int at = (lane & 31) * kGenericRow + 16 * s + (lane >> 5) * 8;
        const u32x4 lf = *reinterpret_cast<const u32x4*>(left + wm * 32 * kGenericRow + at);
        const u32x4 rf = *reinterpret_cast<const u32x4*>(right + wn * 32 * kGenericRow + at);
        acc = mfma_32x32x16<DT>(rf, lf, acc);
    }
}

template <int DT, int LAYOUT>
__global__ void __launch_bounds__(256) fused_generic(const FusedArgs p, int grid_n) {
    __shared__ __attribute__((aligned(16))) u16 lds[2 * 64 * kGenericRow];
    u16 *const As = lds, *const Bs = lds + 64 * kGenericRow;
    float* const Cs = reinterpret_cast<float*>(lds);        // [64][68]
    static_assert(64 * 68 * sizeof(float) <= sizeof(lds), "C staging fits the operands' stage");
    int g, row0, row_end, tn;
    if (!find_tile<64>(p, (int)blockIdx.x, grid_n, 8, g, row0, row_end, tn))
        return;
    const u16* B = p.B + (int64_t)g * p.stride_b;
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave >> 1, wn = wave & 1;
    f32x16 acc = f32x16{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
    // lane i < 16: the A row and the B row that the wave loads i-th; B [K,N]: the lane's column
    const int slot = wave * 16 + (lane & 15);
    const int a_row = row0 + slot < row_end ? a_row_of(p, row0 + slot) : -1;
    const int b_row = b_row_of<64>(p, tn, LAYOUT == LAYOUT_NK ? slot : lane);
    uint32_t av[16], bv[16];
    auto load = [&](int k0) {
        load_rows(av, p.A, p.lda, a_row, (int64_t)k0 + lane, lane < p.K - k0);
        if constexpr (LAYOUT == LAYOUT_NK) {
            load_rows(bv, B, p.ldb, b_row, (int64_t)k0 + lane, lane < p.K - k0);
        } else {
            const int k = k0 + slot;
            load_rows(bv, B, p.ldb, slot < p.K - k0 ? k : -1, b_row, b_row >= 0);
        }
    };
    load(0);
    for (int k0 = 0; k0 < p.K; k0 += kGenericStep) {
        put_rows(As, lane, wave, av);
        if constexpr (LAYOUT == LAYOUT_NK)
            put_rows(Bs, lane, wave, bv);
        else
            put_turned(Bs, lane, wave, bv);
        __syncthreads();
        if (k0 + kGenericStep < p.K)
            load(k0 + kGenericStep);
        generic_step<DT>(acc, As, Bs, lane, wm, wn);
        __syncthreads();
    }
#pragma unroll
    for (int v = 0; v < 16; ++v)
        Cs[(wm * 32 + (lane & 31)) * 68 + wn * 32 + 8 * (v >> 2) + 4 * (lane >> 5) + (v & 3)] = acc[v];
    __syncthreads();
    const int width = p.gated ? p.N >> 1 : p.N, runs = p.gated ? 4 : 8;
    for (int q = tid; q < 64 * runs; q += 256) {
        const int r = q / runs, c = (q % runs) * 8;
        const int n = tn * (runs * 8) + c;
        if (row0 + r < row_end && n < width) {
            float z[8], u[8], bz[8], bu[8], none[1];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                z[e] = Cs[r * 68 + c + e];
                u[e] = p.gated ? Cs[r * 68 + c + 32 + e] : 0.0f;
            }
            load_bias<DT>(p, g, n, width, bz, bu);
            if (p.gated)
                finish_runs<DT, 1, 1, true>(p, row0 + r, row_end, n, width, z, u, bz, bu);
            else
                finish_runs<DT, 1, 1, false>(p, row0 + r, row_end, n, width, z, none, bz, bu);
        }
    }
}

// ------------------------------------------------------------------------------------
// Products that sum over a group's rows (the gradient of B): for every group
//   D_g[i,j] = sum_{s in g} left(s,i) right(s,j)
// with left and right rows of A- and C-sized tensors, either of which may go through the
// row index.  An empty group's D is zero.
// ------------------------------------------------------------------------------------
struct SumArgs {
    const u16* left;
    const u16* right;
    u16* D;
    const int32_t* offsets;
    const int32_t* row_index;
    int64_t stride_d;
    int32_t rows, a_rows, groups, row_div;
    int32_t I, J, ldl, ldr, ldd;
    int32_t index_left, index_right;   // which of the two goes through the row index
    int32_t vec;                       // D takes 16-byte stores at multiples of 8
    float* partial;                    // parts > 1: [parts][groups][I][J] sums of row ranges
    int32_t parts;
};

__device__ __forceinline__ void group_rows(const SumArgs& p, int g, int& lo, int& hi) {
    lo = p.offsets ? clamp_row(p.offsets[g], p.rows) : 0;
    hi = p.offsets ? clamp_row(p.offsets[g + 1], p.rows) : p.rows;
    if (hi < lo)
        hi = lo;
}

// Row s of an operand; -1 where the index points outside it.
__device__ __forceinline__ int sum_row(const SumArgs& p, bool indexed, int s) {
    if (!indexed)
        return s;
    const int v = p.row_index[s], r = p.row_div == 1 ? v : v / p.row_div;
    return v >= 0 && r < p.a_rows ? r : -1;
}

template <int DT>
__global__ void __launch_bounds__(256) sum_generic(const SumArgs p, int grid_i, int grid_j) {
    __shared__ __attribute__((aligned(16))) u16 Ls[64 * kGenericRow];
    __shared__ __attribute__((aligned(16))) u16 Rs[64 * kGenericRow];
    const int per = grid_i * grid_j, g = (int)blockIdx.x / per;
    int ti, tj;
    tile_of((int)blockIdx.x % per, grid_i, grid_j, 8, ti, tj);
    int lo, hi;
    group_rows(p, g, lo, hi);
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave >> 1, wn = wave & 1;
    const int ci = ti * 64 + lane, cj = tj * 64 + lane;
    f32x16 acc = f32x16{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
    uint32_t lv[16], rv[16];
    auto load = [&](int s0) {
        // lane i < 16: the row that the wave loads i-th
        const int slot = wave * 16 + (lane & 15);
        const bool in = slot < hi - s0;
        load_rows(lv, p.left, p.ldl, in ? sum_row(p, p.index_left, s0 + slot) : -1, ci, ci < p.I);
        load_rows(rv, p.right, p.ldr, in ? sum_row(p, p.index_right, s0 + slot) : -1, cj, cj < p.J);
    };
    if (lo < hi)
        load(lo);
    for (int s0 = lo; s0 < hi; s0 += kGenericStep) {
        put_turned(Ls, lane, wave, lv);
        put_turned(Rs, lane, wave, rv);
        __syncthreads();
        if (s0 + kGenericStep < hi)
            load(s0 + kGenericStep);
        generic_step<DT>(acc, Ls, Rs, lane, wm, wn);
        __syncthreads();
    }
    const int i = ti * 64 + wm * 32 + (lane & 31);
    if (i < p.I) {
        u16* row = p.D + (int64_t)g * p.stride_d + (int64_t)i * p.ldd;
#pragma unroll
        for (int v = 0; v < 16; ++v) {
            const int j = tj * 64 + wn * 32 + 8 * (v >> 2) + 4 * (lane >> 5) + (v & 3);
            if (j < p.J)
                row[j] = cvt1<DT>(acc[v]);
        }
    }
}

// ------------------------------------------------------------------------------------
// The epilogue's backward pass:  dZ = dC act'(Z), or gated dZ = [dC up act'(gate),
// dC act(gate)], rounded once to the operands' type for the two products that follow, and
// the column sums of the unrounded dZ (dbias).  One workgroup takes kSliceRows rows of a
// group and 512 columns of dC: 64 lanes of eight columns, four rows at a time.  The column
// sums of a slice go to a workspace row of their own and are added in slice order by
// bias_sum, so the result does not depend on the launch order.
// Bound by memory: 16-byte accesses, each value read and written once; 4096 x 8192 in 49-56
// us (202 MB, 4 TB/s).
// ------------------------------------------------------------------------------------
constexpr int kSliceRows = 16;

struct SlopeArgs {
    const u16* dC;
    const u16* Z;          // null: act none, not gated
    u16* dZ;               // null: dZ is not wanted (it equals dC)
    float* sums;           // [slices][N], or null
    int32_t slices;        // rows of the workspace: no group's slices reach past them
    const int32_t* offsets;
    int32_t rows, groups, N, lddc, ldz, lddz, act, gated;
    int32_t vec;           // dC, Z, dZ all take 16-byte accesses
};

__device__ __forceinline__ void group_rows(const SlopeArgs& p, int g, int& lo, int& hi) {
    lo = p.offsets ? clamp_row(p.offsets[g], p.rows) : 0;
    hi = p.offsets ? clamp_row(p.offsets[g + 1], p.rows) : p.rows;
    if (hi < lo)
        hi = lo;
}

// Slices of kSliceRows rows of groups before group g (the workspace rows of group g start
// there).  Called by whole waves.
__device__ __forceinline__ int slices_before(const SlopeArgs& p, int g) {
    int n = 0;
    for (int i = (int)threadIdx.x & 63; i < g; i += 64) {
        int lo, hi;
        group_rows(p, i, lo, hi);
        n += (hi - lo + kSliceRows - 1) / kSliceRows;
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2)
        n += __shfl_xor(n, d);
    return n;
}

template <int DT, bool GATED>
__global__ void __launch_bounds__(256) slope_rows(const SlopeArgs p) {
    __shared__ __attribute__((aligned(16))) float red[4][GATED ? 2 : 1][512];
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int width = GATED ? p.N >> 1 : p.N;
    // the slice: group, first row, end row
    int slice = (int)blockIdx.x, lo = 0, hi = 0;
    if (!p.offsets) {
        lo = slice * kSliceRows;
        hi = p.rows;
    } else {
        int before = 0;
        bool found = false;
        for (int g0 = 0; g0 < p.groups && !found; g0 += 64) {
            int l = 0, h = 0;
            if (g0 + lane < p.groups)
                group_rows(p, g0 + lane, l, h);
            const int t = (h - l + kSliceRows - 1) / kSliceRows;
            int sum = t;
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                const int o = __shfl_up(sum, d);
                sum += lane >= d ? o : 0;
            }
            const unsigned long long past = __ballot(before + sum > slice);
            if (past) {
                const int at = __builtin_ctzll(past);
                const int first = before + __builtin_amdgcn_readlane(sum - t, at);
                lo = __builtin_amdgcn_readlane(l, at) + (slice - first) * kSliceRows;
                hi = __builtin_amdgcn_readlane(h, at);
                found = true;
            }
            before += __builtin_amdgcn_readlane(sum, 63);
        }
        if (!found)
            return;                       // the whole workgroup: no slice of this number
    }
    hi = hi < lo + kSliceRows ? hi : lo + kSliceRows;
    const int n = ((int)blockIdx.y * 64 + lane) * 8, left = width - n;
    float s0[8] = {0, 0, 0, 0, 0, 0, 0, 0}, s1[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    // a wave's four rows: all loads before the arithmetic
    auto rows = [&](auto wholec) {
        constexpr bool WHOLE = decltype(wholec)::value;
        constexpr int R = kSliceRows / 4;
        u32x4 dy_raw[R], z_raw[R], u_raw[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            // a row past the slice reads the last one's values and is not used
            const int64_t r = lo + wave * R + i < hi ? lo + wave * R + i : hi - 1;
            dy_raw[i] = load8_raw<WHOLE>(p.dC + r * p.lddc + n, left);
            if (p.Z)
                z_raw[i] = load8_raw<WHOLE>(p.Z + r * p.ldz + n, left);
            if constexpr (GATED)
                u_raw[i] = load8_raw<WHOLE>(p.Z + r * p.ldz + width + n, left);
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int r = lo + wave * R + i;
            if (r >= hi)
                break;
            float dy[8], z[8], u[8];
            unpack8<DT>(dy_raw[i], dy);
            if (p.Z)
                unpack8<DT>(z_raw[i], z);
            if constexpr (GATED)
                unpack8<DT>(u_raw[i], u);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float value = 0.0f, slope = 1.0f;
                if (p.Z)
                    activate_slope(p.act, z[e], value, slope);
                z[e] = dy[e] * slope;
                if constexpr (GATED) {
                    z[e] *= u[e];
                    u[e] = dy[e] * value;
                    s1[e] += u[e];
                }
                s0[e] += z[e];
            }
            if (p.dZ) {
                u16* q = p.dZ + (int64_t)r * p.lddz + n;
                store8<DT>(q, WHOLE, left, z);
                if constexpr (GATED)
                    store8<DT>(q + width, WHOLE, left, u);
            }
        }
    };
    if (p.vec && left >= 8)
        rows(std::true_type{});
    else if (left > 0)
        rows(std::false_type{});
    if (!p.sums)
        return;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        red[wave][0][lane * 8 + e] = s0[e];
        if constexpr (GATED)
            red[wave][1][lane * 8 + e] = s1[e];
    }
    __syncthreads();
    for (int q = tid; q < (GATED ? 1024 : 512); q += 256) {
        const int half = q >> 9, c = q & 511, col = (int)blockIdx.y * 512 + c;
        if (col < width)
            p.sums[(int64_t)slice * p.N + half * width + col] =
                (red[0][half][c] + red[1][half][c]) + (red[2][half][c] + red[3][half][c]);
    }
}

}  // namespace tgemm
