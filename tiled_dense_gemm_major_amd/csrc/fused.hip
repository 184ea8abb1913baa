// libtgemm: products with an epilogue and products over groups of rows, forward and
// backward (C ABI): argument checks, the choice of a kernel and the launches.
// Declarations and conventions are in include/tgemm.h.
#include "tgemm.h"

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "fused_launch.hpp"

namespace tgemm {

// dbias of group blockIdx.y: the slices' sums in order, sixteen runs of slices side by side.
__global__ void __launch_bounds__(1024) bias_sum(const SlopeArgs p, float* __restrict__ dbias) {
    __shared__ float red[16][64];
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    const int g = (int)blockIdx.y, n = (int)blockIdx.x * 64 + lane;
    int lo, hi;
    group_rows(p, g, lo, hi);
    const int first = slices_before(p, g), count = (hi - lo + kSliceRows - 1) / kSliceRows;
    const int b = first + (int)((int64_t)wave * count / 16);
    int e = first + (int)((int64_t)(wave + 1) * count / 16);
    e = e < p.slices ? e : p.slices;       // groups that overlap (offsets out of order) have more
    float t = 0.0f;
    if (n < p.N) {
#pragma unroll 8
        for (int i = b; i < e; ++i)
            t += p.sums[(int64_t)i * p.N + n];
    }
    red[wave][lane] = t;
    __syncthreads();
    if (wave == 0 && n < p.N) {
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < 16; ++w)
            sum += red[w][lane];
        dbias[(int64_t)g * p.N + n] = sum;
    }
}

}  // namespace tgemm

namespace {

using tgemm::u16;
using tgemm_fused::FusedArgs;
using tgemm_fused::SlopeArgs;
using tgemm_fused::SumArgs;

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
// Rows, N and K: a tile that starts inside ends below 2^31, so that the kernels' 32-bit
// indexes past a tensor's end compare as such.
constexpr int64_t kMaxSize = (int64_t(1) << 31) - 512;
constexpr int64_t kMaxStride = int64_t(1) << 40;   // elements between groups

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Elements spanned by `rows` rows of `cols` elements, `ld` apart.
int64_t span(int64_t rows, int64_t cols, int64_t ld) {
    return rows > 0 && cols > 0 ? (rows - 1) * ld + cols : 0;
}

bool al16(const void* p) { return (uintptr_t)p % 16 == 0; }

// A tensor's bytes, for the aliasing rules.
struct Extent {
    const void* p;
    int64_t bytes;
};

bool overlaps(const Extent& a, const Extent& b) {
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    return a.p && b.p && a.bytes > 0 && b.bytes > 0 && x < y + (uintptr_t)b.bytes &&
           y < x + (uintptr_t)a.bytes;
}

// One call as the caller described it: a plain product is one group of all rows.
struct Layer {
    int dtype;
    int64_t groups, rows, n, k;
    const int32_t* offsets;
    const int32_t* row_index;
    int64_t row_div;
    const void* A;
    int64_t a_rows, lda;
    const void* B;
    int64_t ldb, stride_b;
    int b_layout;
    int activation, gated;

    int64_t width() const { return gated ? n / 2 : n; }
    int64_t b_rows() const { return b_layout == TGEMM_B_NK ? n : k; }
    int64_t b_cols() const { return b_layout == TGEMM_B_NK ? k : n; }
    Extent a() const { return {A, 2 * span(a_rows, k, lda)}; }
    Extent b() const { return {B, 2 * ((groups - 1) * stride_b + span(b_rows(), b_cols(), ldb))}; }
};

int check_layer(const Layer& l) {
    if (l.dtype != TGEMM_F16 && l.dtype != TGEMM_BF16)
        return TGEMM_ERR_INVALID_VALUE;
    if (l.b_layout != TGEMM_B_NK && l.b_layout != TGEMM_B_KN)
        return TGEMM_ERR_INVALID_VALUE;
    if (l.activation < TGEMM_ACT_NONE || l.activation > TGEMM_ACT_SILU || (l.gated != 0 && l.gated != 1))
        return TGEMM_ERR_INVALID_VALUE;
    if (l.groups < 1 || l.rows < 0 || l.n < 0 || l.k < 0 || l.a_rows < 0 || l.row_div < 1)
        return TGEMM_ERR_INVALID_VALUE;
    if (l.gated && l.n % 2 != 0)
        return TGEMM_ERR_INVALID_VALUE;
    if (l.groups > 65535 || l.rows > kMaxSize || l.n > kMaxSize || l.k > kMaxSize ||
        l.a_rows > kMaxDim || l.row_div > kMaxDim)
        return TGEMM_ERR_UNSUPPORTED;
    if (l.lda < 1 || l.lda < l.k || l.ldb < 1 || l.ldb < l.b_cols() || l.stride_b < 0)
        return TGEMM_ERR_INVALID_VALUE;
    if (l.lda > kMaxDim || l.ldb > kMaxDim || l.stride_b > kMaxStride)
        return TGEMM_ERR_UNSUPPORTED;
    if (!l.row_index && l.a_rows < l.rows)
        return TGEMM_ERR_INVALID_VALUE;
    if (l.groups > 1 && !l.offsets)
        return TGEMM_ERR_NULL_POINTER;
    if ((uintptr_t)l.offsets % 4 || (uintptr_t)l.row_index % 4 || ((uintptr_t)l.A & 1) ||
        ((uintptr_t)l.B & 1))
        return TGEMM_ERR_ALIGNMENT;
    return TGEMM_OK;
}

int check_ld(int64_t ld, int64_t cols) {
    return ld < 1 || ld < cols ? TGEMM_ERR_INVALID_VALUE : (ld > kMaxDim ? TGEMM_ERR_UNSUPPORTED : TGEMM_OK);
}

int status(hipError_t e) { return e == hipSuccess ? TGEMM_OK : TGEMM_ERR_LAUNCH; }

// An upper bound on the tiles of bm rows that the groups can need: each group adds at
// most one partial tile to the whole ones.
int64_t most_tiles(const Layer& l, int64_t bm) {
    if (!l.offsets)
        return cdiv(l.rows, bm);
    return l.rows / bm + (l.groups < l.rows ? l.groups : l.rows);
}

// The tiled kernels move 16-byte pieces of A and B through buffers whose offsets stay below
// 2^31 bytes: one group's B, the rows of an A tile, or all of A through a row index.
constexpr int64_t kMaxBufferBytes = int64_t(1) << 31;

bool tiles_fit(const Layer& l) {
    const bool kn = l.b_layout == TGEMM_B_KN;
    return al16(l.A) && al16(l.B) && l.lda % 8 == 0 && l.ldb % 8 == 0 && (l.groups == 1 || l.stride_b % 8 == 0) &&
           l.k % 8 == 0 && (!kn || l.width() % 8 == 0) && l.lda <= (int64_t(1) << 21) &&
           2 * span(l.b_rows(), l.b_cols(), l.ldb) <= kMaxBufferBytes &&
           (!l.row_index || 2 * span(l.a_rows, l.k, l.lda) <= kMaxBufferBytes);
}

// The form of a product over rows: the least estimated time.  A form's compute time is its
// rounds of workgroups on the 256 compute units times its K steps times the time of a step,
// measured at K = 4096 with bf16 operands in cache (us per 64 k, alone on a unit and with
// as many neighbours as fit); its memory time is the operands' and C's bytes at the rate
// that it streams B with (the stream forms read 5.5 TB/s, the tiled ones 4.6 with one row
// tile per group, the quad kernel 5.1).
tgemm_fused::Form choose_rows(const Layer& l) {
    struct Cost {
        int per_unit;                 // workgroups that share a compute unit
        double alone, shared, fixed;  // us per step in either case; us per launch
        double rate;                  // TB/s
    };
    static const Cost kCost[tgemm_fused::FORMS] = {
        {1, 1.34, 1.34, 9, 5.1}, {1, 1.10, 1.10, 8, 5.0}, {2, 0.80, 0.97, 6, 4.6}, {1, 0.60, 0.60, 6, 4.6}, {2, 0.39, 0.68, 5, 4.6},
        {3, 0.26, 0.58, 5, 4.6}, {1, 0.24, 0.24, 5, 4.6}, {2, 0.16, 0.30, 4, 5.5}, {4, 0.22, 0.55, 4, 5.6},
        {2, 0.18, 0.32, 4, 5.4}, {1, 0.24, 0.24, 4, 5.0}};
    // groups that have rows, if each row fell into any group alike
    const double live = l.groups == 1 ? 1.0 : l.groups * (1.0 - exp(-(double)l.rows / l.groups));
    const double avg = l.rows / live, steps = (double)cdiv(l.k, 64);
    const double bytes = 2.0 * (live * l.n * l.k + (double)l.rows * l.k + (double)l.rows * l.width());
    int best = 1;
    double least = 0;
    for (int f = 0; f < tgemm_fused::FORMS; ++f) {
        if (!tgemm_fused::form_takes((tgemm_fused::Form)f, l.b_layout))
            continue;
        const Cost& c = kCost[f];
        const tgemm_fused::Tile t = tgemm_fused::kTiles[f];
        const double row_tiles = l.groups == 1 ? (double)cdiv(l.rows, t.m)
                                               : live * (avg / t.m + 0.4 > 1.0 ? avg / t.m + 0.4 : 1.0);
        const double tiles = row_tiles * (double)cdiv(l.width(), t.n / (l.gated ? 2 : 1));
        const double slots = 256.0 * c.per_unit, full = floor(tiles / slots), rest = tiles - full * slots;
        const double compute = steps * (full * c.shared + (rest > 256 ? c.shared : (rest > 0 ? c.alone : 0)));
        const double memory = bytes / (c.rate * 1e6);
        const double cost = (compute > memory ? compute : memory) + c.fixed;
        if (f == 0 || cost < least) {
            best = f;
            least = cost;
        }
    }
    return (tgemm_fused::Form)best;
}

// The product over rows of groups, with its epilogue.
int launch_rows(const Layer& l, const FusedArgs& p, hipStream_t s) {
    if (tiles_fit(l)) {
        const tgemm_fused::Form form = choose_rows(l);
        const int64_t tm = most_tiles(l, tgemm_fused::kTiles[form].m);
        const int64_t tn = cdiv(l.width(), tgemm_fused::kTiles[form].n / (l.gated ? 2 : 1));
        if (tm * tn > kMaxDim)
            return TGEMM_ERR_UNSUPPORTED;
        (void)hipGetLastError();
        if (form >= tgemm_fused::FORM_STREAM16)
            return status(tgemm_fused::rows_stream(l.dtype, l.b_layout, form, p, tm, (int)tn, s));
        if (form <= tgemm_fused::FORM_QUAD192)
            return status(l.b_layout == TGEMM_B_NK ? tgemm_fused::rows_quad_nk(l.dtype, form, p, tm, (int)tn, s)
                                                   : tgemm_fused::rows_quad_kn(l.dtype, form, p, tm, (int)tn, s));
        return status(l.b_layout == TGEMM_B_NK ? tgemm_fused::rows_tiled_nk(l.dtype, form, p, tm, (int)tn, s)
                                               : tgemm_fused::rows_tiled_kn(l.dtype, form, p, tm, (int)tn, s));
    }
    const int64_t grid_n = l.gated ? cdiv(l.n / 2, 32) : cdiv(l.n, 64);
    const int64_t grid = most_tiles(l, 64) * grid_n;
    if (grid > kMaxDim)
        return TGEMM_ERR_UNSUPPORTED;
    (void)hipGetLastError();
#define GENERIC_ROWS(DT, L)                                                                \
    hipLaunchKernelGGL((tgemm::fused_generic<DT, L>), dim3((unsigned)grid), dim3(256), 0, s, p, (int)grid_n)
    if (l.dtype == TGEMM_F16) {
        if (l.b_layout == TGEMM_B_NK)
            GENERIC_ROWS(0, 0);
        else
            GENERIC_ROWS(0, 1);
    } else {
        if (l.b_layout == TGEMM_B_NK)
            GENERIC_ROWS(1, 0);
        else
            GENERIC_ROWS(1, 1);
    }
#undef GENERIC_ROWS
    return status(hipGetLastError());
}

FusedArgs row_args(const Layer& l, void* C, int64_t ldc) {
    FusedArgs p{};
    p.A = static_cast<const u16*>(l.A);
    p.B = static_cast<const u16*>(l.B);
    p.C = static_cast<u16*>(C);
    p.offsets = l.offsets;
    p.row_index = l.row_index;
    p.stride_b = l.stride_b;
    p.rows = (int)l.rows;
    p.a_rows = (int)l.a_rows;
    p.N = (int)l.n;
    p.K = (int)l.k;
    p.lda = (int)l.lda;
    p.ldb = (int)l.ldb;
    p.ldc = (int)ldc;
    p.groups = (int)l.groups;
    p.row_div = (int)l.row_div;
    p.act = l.activation;
    p.gated = l.gated;
    p.vec = al16(C) && ldc % 8 == 0 ? tgemm::VEC_C : 0;
    return p;
}

int forward(const Layer& l, void* C, int64_t ldc, const tgemm_epilogue& e, void* stream) {
    int rc = check_layer(l);
    if (rc == TGEMM_OK)
        rc = check_ld(ldc, l.width());
    if (rc == TGEMM_OK && e.residual)
        rc = check_ld(e.ldr, l.width());
    if (rc == TGEMM_OK && e.preact)
        rc = check_ld(e.ldp, l.n);
    if (rc == TGEMM_OK && e.bias && (e.bias_stride < 0 || e.bias_stride > kMaxStride))
        rc = TGEMM_ERR_INVALID_VALUE;
    if (rc != TGEMM_OK)
        return rc;
    if (l.rows == 0 || l.width() == 0)
        return TGEMM_OK;
    if (!C || (l.k > 0 && (!l.A || !l.B)))
        return TGEMM_ERR_NULL_POINTER;
    if (((uintptr_t)C | (uintptr_t)e.bias | (uintptr_t)e.residual | (uintptr_t)e.preact) & 1)
        return TGEMM_ERR_ALIGNMENT;
    const Extent c{C, 2 * span(l.rows, l.width(), ldc)}, z{e.preact, 2 * span(l.rows, l.n, e.ldp)},
        res{e.residual, 2 * span(l.rows, l.width(), e.ldr)},
        bias{e.bias, 2 * ((l.groups - 1) * e.bias_stride + l.n)},
        off{l.offsets, 4 * (l.groups + 1)}, idx{l.row_index, 4 * l.rows};
    const bool in_place = e.residual == C && e.ldr == ldc;   // each value read before it is written
    if (overlaps(c, l.a()) || overlaps(c, l.b()) || overlaps(c, bias) || overlaps(c, z) ||
        (overlaps(c, res) && !in_place) || overlaps(z, l.a()) || overlaps(z, l.b()) ||
        overlaps(z, bias) || overlaps(z, res) || overlaps(c, off) || overlaps(c, idx) ||
        overlaps(z, off) || overlaps(z, idx))
        return TGEMM_ERR_ALIASING;
    FusedArgs p = row_args(l, C, ldc);
    p.bias = static_cast<const u16*>(e.bias);
    p.residual = static_cast<const u16*>(e.residual);
    p.preact = static_cast<u16*>(e.preact);
    p.stride_bias = e.bias_stride;
    p.ldr = (int)e.ldr;
    p.ldp = (int)e.ldp;
    const bool halves = !l.gated || l.width() % 8 == 0;      // the second half is aligned too
    if (al16(e.residual) && e.ldr % 8 == 0)
        p.vec |= tgemm::VEC_RES;
    if (al16(e.preact) && e.ldp % 8 == 0 && halves)
        p.vec |= tgemm::VEC_PRE;
    if (al16(e.bias) && (l.groups == 1 || e.bias_stride % 8 == 0) && halves)
        p.vec |= tgemm::VEC_BIAS;
    return launch_rows(l, p, static_cast<hipStream_t>(stream));
}

// Workspace rows of the bias gradient: one per slice of a group's rows.
int64_t most_slices(int64_t groups, int64_t rows) {
    return rows / tgemm::kSliceRows + (groups < rows ? groups : rows);
}

struct Gradients {
    const void* dC;
    int64_t lddc;
    const void* Z;
    int64_t ldz;
    void* dZ;
    int64_t lddz;
    void* dA;
    int64_t ldda;
    void* dB;
    int64_t lddb, stride_db;
    float* dbias;
    void* workspace;
    int64_t workspace_bytes;
};

// The form of a sum over rows, by the same estimate: rounds of workgroups times steps of 64
// rows times the time of a step; and the number of ranges that a group's rows are cut into
// where the 128 x 128 tiles leave compute units idle (fp32 partial tiles, written and read
// once: 8192 rows to 1024 x 1024 77 us whole).  Parts of 256 rows or more, at most 16, and
// at most kMaxPartialBytes of them.
struct SumPlan {
    tgemm_fused::SumForm form;
    int parts;
};
constexpr int64_t kMaxPartialBytes = int64_t(64) << 20;

SumPlan choose_sum(int64_t groups, int64_t rows, int64_t I, int64_t J, bool quad, bool split) {
    struct Cost {
        int per_unit;
        double alone, shared, fixed;
    };
    static const Cost kCost[tgemm_fused::SUM_FORMS] = {
        {1, 1.43, 1.43, 8}, {1, 1.75, 1.75, 9}, {2, 0.72, 1.05, 6}, {2, 0.5, 0.55, 5}};
    const double steps = (double)cdiv(cdiv(rows, groups), 64);
    const auto cost_of = [&](int f, int64_t parts) {
        const int t = tgemm_fused::kSumTiles[f];
        const double tiles = (double)(groups * cdiv(I, t) * cdiv(J, t) * parts);
        const Cost& c = kCost[f];
        const double slots = 256.0 * c.per_unit, full = floor(tiles / slots), rest = tiles - full * slots;
        return ceil(steps / parts) * (full * c.shared + (rest > 256 ? c.shared : (rest > 0 ? c.alone : 0))) +
               c.fixed * (full + (rest > 0));
    };
    SumPlan best{tgemm_fused::SUM_256, 1};
    double least = cost_of(tgemm_fused::SUM_256, 1);
    for (int f = 0; f < tgemm_fused::SUM_FORMS; ++f)
        if (f != tgemm_fused::SUM_256 && (f != tgemm_fused::SUM_QUAD || quad) && cost_of(f, 1) < least) {
            best.form = (tgemm_fused::SumForm)f;
            least = cost_of(f, 1);
        }
    const int64_t tiles = groups * cdiv(I, 128) * cdiv(J, 128);
    if (split && tiles > 0 && tiles < 256)
        for (int64_t parts = 2; parts <= 16 && parts * tiles <= 512 && steps / parts >= 4; ++parts) {
            const double bytes = 4.0 * parts * groups * I * J;
            if (bytes > (double)kMaxPartialBytes)
                break;
            const double cost = cost_of(tgemm_fused::SUM_128, parts) + 4 + 2 * bytes / 4.6e6;
            if (cost < least) {
                best = {tgemm_fused::SUM_128, (int)parts};
                least = cost;
            }
        }
    return best;
}

int64_t partial_bytes(const SumPlan& plan, int64_t groups, int64_t I, int64_t J) {
    return plan.parts > 1 ? 4 * plan.parts * groups * I * J : 0;
}

// `partial`: workspace for the parts' sums, 16-byte aligned, or null.
int launch_sum(const Layer& l, SumArgs p, float* partial, int64_t bytes, hipStream_t s) {
    const auto through = [&](bool indexed, int64_t cols, int64_t ld) {
        return ld <= (int64_t(1) << 23) && cols % 8 == 0 && ld % 8 == 0 &&
               (!indexed || 2 * span(p.a_rows, cols, ld) <= kMaxBufferBytes);
    };
    if (al16(p.left) && al16(p.right) && through(p.index_left, p.I, p.ldl) && through(p.index_right, p.J, p.ldr)) {
        if (l.groups * cdiv(p.I, 64) * cdiv(p.J, 64) > kMaxDim)
            return TGEMM_ERR_UNSUPPORTED;
        const bool quad = !p.row_index && p.vec && 2 * span(p.rows, p.I, p.ldl) <= kMaxBufferBytes &&
                          2 * span(p.rows, p.J, p.ldr) <= kMaxBufferBytes;
        SumPlan plan = choose_sum(l.groups, l.rows, p.I, p.J, quad, partial != nullptr);
        if (partial_bytes(plan, l.groups, p.I, p.J) > bytes)
            plan = choose_sum(l.groups, l.rows, p.I, p.J, quad, false);
        p.partial = partial;
        p.parts = plan.parts;
        (void)hipGetLastError();
        return status(plan.form == tgemm_fused::SUM_QUAD ? tgemm_fused::sum_quad(l.dtype, p, s)
                                                         : tgemm_fused::sum_tiled(l.dtype, plan.form, p, s));
    }
    p.parts = 1;
    const int64_t gi = cdiv(p.I, 64), gj = cdiv(p.J, 64);
    if (l.groups * gi * gj > kMaxDim)
        return TGEMM_ERR_UNSUPPORTED;
    (void)hipGetLastError();
    if (l.dtype == TGEMM_F16)
        hipLaunchKernelGGL((tgemm::sum_generic<0>), dim3((unsigned)(l.groups * gi * gj)), dim3(256), 0, s, p,
                           (int)gi, (int)gj);
    else
        hipLaunchKernelGGL((tgemm::sum_generic<1>), dim3((unsigned)(l.groups * gi * gj)), dim3(256), 0, s, p,
                           (int)gi, (int)gj);
    return status(hipGetLastError());
}

int backward(const Layer& l, const Gradients& d, void* stream) {
    int rc = check_layer(l);
    const bool slope = l.activation != TGEMM_ACT_NONE || l.gated;
    const bool need_dz = slope && (d.dA || d.dB);
    if (rc == TGEMM_OK)
        rc = check_ld(d.lddc, l.width());
    if (rc == TGEMM_OK && slope)
        rc = check_ld(d.ldz, l.n);
    if (rc == TGEMM_OK && need_dz)
        rc = check_ld(d.lddz, l.n);
    if (rc == TGEMM_OK && d.dA)
        rc = check_ld(d.ldda, l.k);
    if (rc == TGEMM_OK && d.dB)
        rc = check_ld(d.lddb, l.b_cols());
    if (rc == TGEMM_OK && (d.workspace_bytes < 0 || (d.dB && d.stride_db < 0)))
        rc = TGEMM_ERR_INVALID_VALUE;
    if (rc == TGEMM_OK && d.dB && d.stride_db > kMaxStride)
        rc = TGEMM_ERR_UNSUPPORTED;
    if (rc == TGEMM_OK && d.dB && l.groups > 1 && d.stride_db < span(l.b_rows(), l.b_cols(), d.lddb))
        rc = TGEMM_ERR_INVALID_VALUE;
    if (rc != TGEMM_OK)
        return rc;
    if (!d.dA && !d.dB && !d.dbias)
        return TGEMM_OK;
    const bool rows = l.rows > 0;
    if (rows && l.n > 0 && (!d.dC || (slope && !d.Z) || (need_dz && !d.dZ)))
        return TGEMM_ERR_NULL_POINTER;
    if (rows && l.k > 0 && ((d.dA && l.n > 0 && !l.B) || (d.dB && l.n > 0 && !l.A)))
        return TGEMM_ERR_NULL_POINTER;
    if (((uintptr_t)d.dC | (uintptr_t)d.Z | (uintptr_t)d.dZ | (uintptr_t)d.dA | (uintptr_t)d.dB) & 1)
        return TGEMM_ERR_ALIGNMENT;
    if ((uintptr_t)d.dbias % 4)
        return TGEMM_ERR_ALIGNMENT;
    // the workspace: the bias's sums, then (as much as is there) the parts of dB's
    const int64_t sums_bytes = d.dbias ? 4 * most_slices(l.groups, l.rows) * l.n : 0;
    if (sums_bytes > 0 && (!d.workspace || d.workspace_bytes < sums_bytes))
        return TGEMM_ERR_WORKSPACE;
    if (!al16(d.workspace))
        return TGEMM_ERR_ALIGNMENT;
    const int64_t parts_at = cdiv(sums_bytes, 16) * 16;
    const bool lent = d.workspace && d.dB && d.workspace_bytes > parts_at;
    float* parts = lent ? static_cast<float*>(d.workspace) + parts_at / 4 : nullptr;
    const Extent in[] = {{d.dC, 2 * span(l.rows, l.width(), d.lddc)},
                         {slope ? d.Z : nullptr, 2 * span(l.rows, l.n, d.ldz)},
                         l.a(),
                         l.b(),
                         {l.offsets, 4 * (l.groups + 1)},
                         {l.row_index, 4 * l.rows}};
    const Extent out[] = {
        {need_dz ? d.dZ : nullptr, 2 * span(l.rows, l.n, d.lddz)},
        {d.dA, 2 * span(l.rows, l.k, d.ldda)},
        {d.dB, 2 * ((l.groups - 1) * d.stride_db + span(l.b_rows(), l.b_cols(), d.lddb))},
        {d.dbias, 4 * l.groups * l.n},
        {d.workspace, lent ? d.workspace_bytes : sums_bytes}};
    for (int i = 0; i < 5; ++i) {
        for (int j = 0; j < 6; ++j) {
            // dZ may take Z's place: each value is read before it is written
            if (i == 0 && j == 1 && d.dZ == d.Z && d.lddz == d.ldz)
                continue;
            if (overlaps(out[i], in[j]))
                return TGEMM_ERR_ALIASING;
        }
        for (int j = 0; j < i; ++j)
            if (overlaps(out[i], out[j]))
                return TGEMM_ERR_ALIASING;
    }

    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (l.n > 0 && (need_dz || d.dbias)) {
        SlopeArgs p{};
        p.dC = static_cast<const u16*>(d.dC);
        p.Z = slope ? static_cast<const u16*>(d.Z) : nullptr;
        p.dZ = need_dz ? static_cast<u16*>(d.dZ) : nullptr;
        p.sums = d.dbias ? static_cast<float*>(d.workspace) : nullptr;
        p.offsets = l.offsets;
        p.rows = (int)l.rows;
        p.groups = (int)l.groups;
        p.N = (int)l.n;
        p.lddc = (int)d.lddc;
        p.ldz = (int)d.ldz;
        p.lddz = (int)d.lddz;
        p.act = l.activation;
        p.gated = l.gated;
        p.vec = al16(d.dC) && d.lddc % 8 == 0 && (!p.Z || (al16(d.Z) && d.ldz % 8 == 0)) &&
                (!p.dZ || (al16(d.dZ) && d.lddz % 8 == 0)) && l.width() % 8 == 0;
        const int64_t slices = l.offsets ? most_slices(l.groups, l.rows) : cdiv(l.rows, tgemm::kSliceRows);
        p.slices = (int)slices;
        const int64_t columns = cdiv(l.width(), 512);
        if (columns > 65535)
            return TGEMM_ERR_UNSUPPORTED;
        (void)hipGetLastError();
        if (slices > 0) {
            const dim3 grid((unsigned)slices, (unsigned)columns);
#define SLOPE(DT, G) hipLaunchKernelGGL((tgemm::slope_rows<DT, G>), grid, dim3(256), 0, s, p)
            if (l.dtype == TGEMM_F16) {
                if (l.gated)
                    SLOPE(0, true);
                else
                    SLOPE(0, false);
            } else {
                if (l.gated)
                    SLOPE(1, true);
                else
                    SLOPE(1, false);
            }
#undef SLOPE
            rc = status(hipGetLastError());
            if (rc != TGEMM_OK)
                return rc;
        }
        if (d.dbias) {
            hipLaunchKernelGGL(tgemm::bias_sum, dim3((unsigned)cdiv(l.n, 64), (unsigned)l.groups), dim3(1024),
                               0, s, p, d.dbias);
            rc = status(hipGetLastError());
            if (rc != TGEMM_OK)
                return rc;
        }
    }
    const void* dz = slope ? d.dZ : d.dC;
    const int64_t lddz = slope ? d.lddz : d.lddc;
    if (d.dA && rows && l.k > 0) {
        // dA = dZ b^T: the same groups, summed over n, with B's storage read the other way
        Layer t = l;
        t.n = l.k;
        t.k = l.n;
        t.row_index = nullptr;
        t.row_div = 1;
        t.A = dz;
        t.a_rows = l.rows;
        t.lda = lddz;
        t.b_layout = l.b_layout == TGEMM_B_NK ? TGEMM_B_KN : TGEMM_B_NK;
        t.activation = TGEMM_ACT_NONE;
        t.gated = 0;
        rc = launch_rows(t, row_args(t, d.dA, d.ldda), s);
        if (rc != TGEMM_OK)
            return rc;
    }
    if (d.dB && l.n > 0 && l.k > 0) {
        SumArgs p{};
        const bool nk = l.b_layout == TGEMM_B_NK;            // dB [N,K]: dZ on the left
        const u16* a = static_cast<const u16*>(l.A);
        const u16* z = static_cast<const u16*>(dz);
        p.left = nk ? z : a;
        p.right = nk ? a : z;
        p.D = static_cast<u16*>(d.dB);
        p.offsets = l.offsets;
        p.row_index = l.row_index;
        p.stride_d = d.stride_db;
        p.rows = (int)l.rows;
        p.a_rows = (int)l.a_rows;
        p.groups = (int)l.groups;
        p.row_div = (int)l.row_div;
        p.I = (int)(nk ? l.n : l.k);
        p.J = (int)(nk ? l.k : l.n);
        p.ldl = (int)(nk ? lddz : l.lda);
        p.ldr = (int)(nk ? l.lda : lddz);
        p.ldd = (int)d.lddb;
        p.index_left = l.row_index && !nk;
        p.index_right = l.row_index && nk;
        p.vec = al16(d.dB) && d.lddb % 8 == 0 && (l.groups == 1 || d.stride_db % 8 == 0);
        rc = launch_sum(l, p, parts, lent ? d.workspace_bytes - parts_at : 0, s);
    }
    return rc;
}

const tgemm_epilogue kNoEpilogue{};

}  // namespace

extern "C" {

int gemm_fused(int dtype, int64_t m, int64_t n, int64_t k, const void* A, int64_t lda, const void* B,
               int64_t ldb, int b_layout, void* C, int64_t ldc, const tgemm_epilogue* epilogue, void* stream) {
    const tgemm_epilogue& e = epilogue ? *epilogue : kNoEpilogue;
    return forward(Layer{dtype, 1, m, n, k, nullptr, nullptr, 1, A, m, lda, B, ldb, 0, b_layout, e.activation,
                         e.gated},
                   C, ldc, e, stream);
}

int gemm_grouped(int dtype, int64_t groups, int64_t rows, int64_t n, int64_t k, const int32_t* offsets,
                 const int32_t* row_index, int64_t row_div, const void* A, int64_t a_rows, int64_t lda,
                 const void* B, int64_t ldb, int64_t stride_b, int b_layout, void* C, int64_t ldc,
                 const tgemm_epilogue* epilogue, void* stream) {
    if (rows > 0 && !offsets)
        return TGEMM_ERR_NULL_POINTER;
    const tgemm_epilogue& e = epilogue ? *epilogue : kNoEpilogue;
    return forward(Layer{dtype, groups, rows, n, k, offsets, row_index, row_div, A, a_rows, lda, B, ldb, stride_b,
                         b_layout, e.activation, e.gated},
                   C, ldc, e, stream);
}

int gemm_backward_workspace_size(int64_t groups, int64_t rows, int64_t n, int64_t k, int dbias, int64_t* bytes) {
    if (!bytes)
        return TGEMM_ERR_NULL_POINTER;
    if (groups < 1 || rows < 0 || n < 0 || k < 0 || (dbias != 0 && dbias != 1))
        return TGEMM_ERR_INVALID_VALUE;
    if (groups > 65535 || rows > kMaxSize || n > kMaxSize || k > kMaxSize)
        return TGEMM_ERR_UNSUPPORTED;
    const int64_t sums = dbias ? cdiv(4 * most_slices(groups, rows) * n, 16) * 16 : 0;
    // the parts' sums, for whichever of the forms a call may choose from
    int64_t parts = 0;
    if (rows > 0 && n > 0 && k > 0)
        for (int quad = 0; quad < 2; ++quad) {
            const int64_t b = partial_bytes(choose_sum(groups, rows, n, k, quad != 0, true), groups, n, k);
            parts = b > parts ? b : parts;
        }
    *bytes = sums + parts;
    return TGEMM_OK;
}

int gemm_fused_backward(int dtype, int64_t m, int64_t n, int64_t k, const void* dC, int64_t lddc, const void* A,
                        int64_t lda, const void* B, int64_t ldb, int b_layout, int activation, int gated,
                        const void* preact, int64_t ldp, void* dZ, int64_t lddz, void* dA, int64_t ldda, void* dB,
                        int64_t lddb, float* dbias, void* workspace, int64_t workspace_bytes, void* stream) {
    return backward(Layer{dtype, 1, m, n, k, nullptr, nullptr, 1, A, m, lda, B, ldb, 0, b_layout, activation, gated},
                    Gradients{dC, lddc, preact, ldp, dZ, lddz, dA, ldda, dB, lddb, 0, dbias, workspace,
                              workspace_bytes},
                    stream);
}

int gemm_grouped_backward(int dtype, int64_t groups, int64_t rows, int64_t n, int64_t k, const int32_t* offsets,
                          const int32_t* row_index, int64_t row_div, const void* dC, int64_t lddc, const void* A,
                          int64_t a_rows, int64_t lda, const void* B, int64_t ldb, int64_t stride_b, int b_layout,
                          int activation, int gated, const void* preact, int64_t ldp, void* dZ, int64_t lddz,
                          void* dA, int64_t ldda, void* dB, int64_t lddb, int64_t stride_db, float* dbias,
                          void* workspace, int64_t workspace_bytes, void* stream) {
    if (!offsets && (rows > 0 || groups > 1))
        return TGEMM_ERR_NULL_POINTER;
    return backward(Layer{dtype, groups, rows, n, k, offsets, row_index, row_div, A, a_rows, lda, B, ldb, stride_b,
                          b_layout, activation, gated},
                    Gradients{dC, lddc, preact, ldp, dZ, lddz, dA, ldda, dB, lddb, stride_db, dbias, workspace,
                              workspace_bytes},
                    stream);
}

}  // extern "C"
