// The tiled kernels of the fused and grouped products for aligned operands: MFMA tiles fed
// by direct-to-LDS loads.
#pragma once

#include "fused.hpp"

namespace tgemm {

// Keeps the compiler from moving a wave's LDS reads above its LDS writes of other lanes'
// values; the hardware completes a wave's LDS accesses in order.
__device__ __forceinline__ void wave_lds_order() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// ------------------------------------------------------------------------------------
// Operand tiles of 64 k, staged by 1 KiB direct-to-LDS loads (64 lanes x 16 bytes, lane l
// landing at byte 16 l), LD loads per wave.
//   KRows: R rows of 64 k (128 bytes each, 8 rows per load).  Chunk c of row r sits at
//     c ^ swz(r): the row-wise operand reads of 32 lanes are free of bank conflicts.
//   KCols: 64 k rows of R columns (2 R bytes each, 512 / R rows per load), read by the
//     transposing LDS read: four k rows of 16 columns per 16 lanes, so that lanes 0-31 read
//     4 rows x 64 bytes.  The rows are a whole number of 256-byte bank windows apart (R >=
//     128; half of one, R = 64), so chunk c of row k sits at c ^ kc_swz(k), which puts the
//     four pieces into four different quarters of the window.
// Offsets are bytes below 2^31; a lane whose row, column or k lies outside reads at
// kOutOfRange, which the buffer's range check turns into zeros.
// ------------------------------------------------------------------------------------
constexpr int kTileK = 64;

template <int R, int NW>
struct KRows {
    static constexpr int LD = R / 8 / NW;
    static_assert(LD >= 2 && LD % 2 == 0, "whole load pairs per wave");
    uint32_t off[LD];
    int kc[2];                               // this lane's k in a load (by the load's parity)
    // byte_of(r): the byte offset of tile row r, or kOutOfRange
    template <typename F>
    __device__ __forceinline__ void init(int wave, int lane, F&& byte_of) {
#pragma unroll
        for (int q = 0; q < 2; ++q)
            kc[q] = ((lane & 7) ^ swz<8>(8 * q + (lane >> 3))) * 8;
#pragma unroll
        for (int i = 0; i < LD; ++i) {
            const uint32_t o = byte_of(8 * (wave * LD + i) + (lane >> 3));
            off[i] = o == kOutOfRange ? o : o + (uint32_t)kc[i & 1] * 2u;
        }
    }
    __device__ __forceinline__ void load(rsrc4_t r, uint32_t lds, int wave, int k0, int K) const {
        const uint32_t v0 = k0 + kc[0] < K ? 0u : kOutOfRange, v1 = k0 + kc[1] < K ? 0u : kOutOfRange;
#pragma unroll
        for (int i = 0; i < LD; ++i)
            dma16_at(r, lds + (uint32_t)((wave * LD + i) * 1024), off[i] | (i & 1 ? v1 : v0), (uint32_t)k0 * 2u);
    }
};

template <int R>
__device__ __forceinline__ int kc_swz(int k) {
    return R >= 128 ? 4 * (k & 3) : 4 * ((k >> 1) & 1);
}

template <int R, int NW>
struct KCols {
    static constexpr int LD = R / 8 / NW, CH = R / 8, KPL = 64 / CH;
    static_assert(R == 64 || R == 128 || R == 256, "tile columns");
    static_assert(LD >= 1, "whole loads per wave");
    // the k row of this lane in load i, and the tile column of its chunk
    static __device__ __forceinline__ int k_of(int wave, int lane, int i) { return (wave * LD + i) * KPL + lane / CH; }
    static __device__ __forceinline__ int col_of(int wave, int lane, int i) {
        return ((lane % CH) ^ kc_swz<R>(k_of(wave, lane, i))) * 8;
    }
};

// One MFMA operand (8 consecutive k of one column) from a KCols tile: two transposing
// reads, k rows 4 apart.  `at`: the lane's element offset for column block j.
template <int R>
__device__ __forceinline__ int kc_at(int lane, int col0, int j) {
    const int g = lane >> 4, sl = lane & 15;
    const int kl = 8 * (g >> 1) + (sl >> 2), c = col0 + 32 * j + 16 * (g & 1) + 4 * (sl & 3);
    return kl * R + (((c >> 3) ^ kc_swz<R>(kl)) << 3) + (c & 7);
}
template <int R>
__device__ __forceinline__ u32x4 read_kcols(const u16* p0) {
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p0));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p0 + 4 * R));
    const u32x2 l2 = __builtin_bit_cast(u32x2, lo);
    const u32x2 h2 = __builtin_bit_cast(u32x2, hi);
    return u32x4{l2[0], l2[1], h2[0], h2[1]};
}

// ------------------------------------------------------------------------------------
// The epilogue of a wave's block of PASSES x 32 rows and WTN tile columns.  put(i, stage)
// writes the i-th 32 rows to the wave's LDS stage as fp32 (row stride WTN + 4 floats);
// they come back as runs of eight columns of one row per lane, so that bias, residual,
// stored z and C move in 16-byte pieces of whole row segments.  m0: the block's first row;
// n0: its first column of C.
// ------------------------------------------------------------------------------------
template <int DT, int WTN, int PASSES, bool GATED, typename PUT>
__device__ __forceinline__ void rows_epilogue_as(const FusedArgs& p, int g, float* stage, int lane, int m0,
                                                 int row_end, int n0, PUT&& put) {
    constexpr int SRF = WTN + 4, RUNS = WTN / (GATED ? 16 : 8), RPI = 64 / RUNS, Q = 32 / RPI;
    const int c = (lane % RUNS) * 8, n = n0 + c, width = p.gated ? p.N >> 1 : p.N;
    const int zc = GATED ? (c >> 5) * 64 + (c & 31) : c;
    float bz[8], bu[8];
    load_bias<DT>(p, g, n, width, bz, bu);
    static_for<0, PASSES>([&](auto ic) {
        const int m = m0 + decltype(ic)::value * 32 + lane / RUNS;
        wave_lds_order();
        put(ic, stage);
        wave_lds_order();
        float z[Q * 8], u[GATED ? Q * 8 : 1];
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const float* src = stage + (q * RPI + lane / RUNS) * SRF + zc;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                z[q * 8 + e] = src[e];
                if constexpr (GATED)
                    u[q * 8 + e] = src[32 + e];
            }
        }
        if (n < width)
            finish_runs<DT, Q, RPI, GATED>(p, m, row_end, n, width, z, u, bz, bu);
    });
}

template <int DT, int WTN, int PASSES, typename PUT>
__device__ __forceinline__ void rows_epilogue(const FusedArgs& p, int g, float* stage, int lane, int m0, int row_end,
                                              int n0, PUT&& put) {
    if (p.gated)
        rows_epilogue_as<DT, WTN, PASSES, true>(p, g, stage, lane, m0, row_end, n0, put);
    else
        rows_epilogue_as<DT, WTN, PASSES, false>(p, g, stage, lane, m0, row_end, n0, put);
}

// ------------------------------------------------------------------------------------
// The tiled kernel over rows of groups: A rows [M,K] (through the row index, if any), B
// [N,K] or [K,N].  WM x WN waves of (BM/WM) x (BN/WN), MFMA 32x32x16, ST stages.
//   A step's four sub-steps of 16 k run the MFMAs of operands read one sub-step before; in
//   the last, after half of its MFMAs, each wave waits until its loads of tile t+1 have
//   landed (those of up to ST-2 later tiles stay in flight) and meets the others, which
//   have then also read all of tile t; the loads of tile t+ST go into the stage that tile
//   leaves, and the first operands of tile t+1 are read beside the other half.  (Reading a
//   sub-step's operands right before its MFMAs leaves the matrix cores waiting for the LDS
//   half of the time where a SIMD holds one wave: 1300 cycles a step of 128 x 128 x 64
//   instead of the 512 of its MFMAs; more stages do not help.)
//   Loads past the last tile read nothing (zeros), so that every step has the same number
//   of loads in flight.
//   For products whose 256-wide tiles would leave units idle: 1024 x 4096 x 4096 takes 43 us
//   by 128 x 128 (four stages) and 65 by the quad tiles, 1001 x 2048 x 1024 10.5 by 64 x 128
//   and 25; at 800 x 8192 x 4096 both take 69.  Bound by the load path.
// ------------------------------------------------------------------------------------
template <int DT, int LAYOUT, int BM, int BN, int WM, int WN, int ST, int OCC>
__global__ void __attribute__((amdgpu_flat_work_group_size(WM * WN * 64, WM * WN * 64),
                               amdgpu_waves_per_eu(OCC, OCC)))
fused_tiled(const FusedArgs p, int grid_n, int group_m) {
    constexpr int NW = WM * WN, WTM = BM / WM, WTN = BN / WN, TM = WTM / 32, TN = WTN / 32;
    constexpr int SLOT_A = BM * kTileK, STAGE = (BM + BN) * kTileK;   // elements
    constexpr int SRF = WTN + 4;                                      // staged row in floats
    static_assert(WTN % 64 == 0, "gate and up blocks of a pair in one wave");
    static_assert(NW * 32 * SRF * 4 <= ST * STAGE * 2, "C staging fits the ring");
    __shared__ __attribute__((aligned(1024))) u16 lds[ST * STAGE];
    int g, row0, row_end, tn;
    if (!find_tile<BM>(p, (int)blockIdx.x, grid_n, group_m, g, row0, row_end, tn))
        return;
    g = __builtin_amdgcn_readfirstlane(g);
    row0 = __builtin_amdgcn_readfirstlane(row0);
    row_end = __builtin_amdgcn_readfirstlane(row_end);
    const int tid = (int)threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN, half = lane >> 5, lr = lane & 31;
    const int K = p.K, nk = (K + kTileK - 1) / kTileK;

    // A: rows of the tile from its first row on, or the whole of A through the row index
    KRows<BM, NW> la;
    const u16* a0 = p.row_index ? p.A : p.A + (int64_t)row0 * p.lda;
    const int a_rows = p.row_index ? p.a_rows : (row_end - row0 < BM ? row_end - row0 : BM);
    const rsrc4_t ra = make_rsrc4(a0, span_bytes(a_rows, K, p.lda));
    la.init(wave, lane, [&](int r) -> uint32_t {
        if (row0 + r >= row_end)
            return kOutOfRange;
        const int s = p.row_index ? a_row_of(p, row0 + r) : r;
        return s < 0 ? kOutOfRange : (uint32_t)s * (uint32_t)p.lda * 2u;
    });
    const u16* b0 = p.B + (int64_t)g * p.stride_b;
    const rsrc4_t rb = LAYOUT == LAYOUT_NK ? make_rsrc4(b0, span_bytes(p.N, K, p.ldb))
                                           : make_rsrc4(b0, span_bytes(K, p.N, p.ldb));
    using BC = KCols<BN, NW>;
    KRows<BN, NW> lb;
    uint32_t bo[BC::LD];
    if constexpr (LAYOUT == LAYOUT_NK) {
        lb.init(wave, lane, [&](int r) -> uint32_t {
            const int n = b_row_of<BN>(p, tn, r);
            return n < 0 ? kOutOfRange : (uint32_t)n * (uint32_t)p.ldb * 2u;
        });
    } else {
#pragma unroll
        for (int i = 0; i < BC::LD; ++i) {
            const int n = b_row_of<BN>(p, tn, BC::col_of(wave, lane, i));
            bo[i] = n < 0 ? kOutOfRange
                          : ((uint32_t)BC::k_of(wave, lane, i) * (uint32_t)p.ldb + (uint32_t)n) * 2u;
        }
    }
    const uint32_t lds0 = lds_addr(lds);
    auto load = [&](int t, int slot) {
        const int k0 = t * kTileK;
        const uint32_t at = lds0 + (uint32_t)(slot * STAGE * 2);
        la.load(ra, at, wave, k0, K);
        if constexpr (LAYOUT == LAYOUT_NK) {
            lb.load(rb, at + SLOT_A * 2, wave, k0, K);
        } else {
#pragma unroll
            for (int i = 0; i < BC::LD; ++i)
                dma16_at(rb, at + SLOT_A * 2 + (uint32_t)((wave * BC::LD + i) * 1024),
                         k0 + BC::k_of(wave, lane, i) < K ? bo[i] : kOutOfRange,
                         (uint32_t)(k0 < K ? k0 : 0) * (uint32_t)p.ldb * 2u);
        }
    };
    constexpr int LOADS = KRows<BM, NW>::LD + BN / 8 / NW;

    f32x16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
            acc[i][j] = f32x16{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
    const int xr = swz<8>(lr);
    int kb[TN];
    if constexpr (LAYOUT == LAYOUT_KN) {
#pragma unroll
        for (int j = 0; j < TN; ++j)
            kb[j] = kc_at<BN>(lane, wn * WTN, j);
    }
    u32x4 fa[2][TM], fb[2][TN];
    auto read = [&](int slot, int s, auto bufc) {       // the operands of sub-step s
        constexpr int buf = decltype(bufc)::value;
        const u16* as = lds + slot * STAGE + (wm * WTM + lr) * kTileK;
        const u16* bs = lds + slot * STAGE + SLOT_A;
        const int ko = (((2 * s) | half) ^ xr) * 8;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            if constexpr (LAYOUT == LAYOUT_NK)
                fb[buf][j] = *reinterpret_cast<const u32x4*>(bs + (wn * WTN + 32 * j + lr) * kTileK + ko);
            else
                fb[buf][j] = read_kcols<BN>(bs + kb[j] + 16 * s * BN);
        }
#pragma unroll
        for (int i = 0; i < TM; ++i)
            fa[buf][i] = *reinterpret_cast<const u32x4*>(as + 32 * i * kTileK + ko);
        __builtin_amdgcn_sched_barrier(0);
    };
    auto multiply = [&](auto bufc, auto fromc, auto toc) {   // blocks [from, to) of the wave's
        constexpr int buf = decltype(bufc)::value;
        static_for<decltype(fromc)::value, decltype(toc)::value>([&](auto jc) {
            constexpr int i = decltype(jc)::value / TN, j = decltype(jc)::value % TN;
            acc[i][j] = mfma_32x32x16<DT>(fb[buf][j], fa[buf][i], acc[i][j]);
        });
        __builtin_amdgcn_sched_barrier(0);
    };
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    using IH = std::integral_constant<int, TM * TN / 2>;
    using IE = std::integral_constant<int, TM * TN>;
#pragma unroll
    for (int t = 0; t < ST; ++t)
        load(t, t);
    wait_vm_then_sync<(ST - 1) * LOADS>();
    read(0, 0, I0{});
    int slot = 0;
    for (int t = 0; t < nk; ++t) {
        const int next = slot + 1 == ST ? 0 : slot + 1;
        read(slot, 1, I1{});
        multiply(I0{}, I0{}, IE{});
        read(slot, 2, I0{});
        multiply(I1{}, I0{}, IE{});
        read(slot, 3, I1{});
        multiply(I0{}, I0{}, IE{});
        multiply(I1{}, I0{}, IH{});
        wait_vm_then_sync<(ST - 2) * LOADS>();
        __builtin_amdgcn_sched_barrier(0);
        load(t + ST, slot);
        read(next, 0, I0{});
        multiply(I1{}, IH{}, IE{});
        slot = next;
    }
    wait_vm_then_sync<0>();            // no load writes LDS any more, no wave reads it

    rows_epilogue<DT, WTN, TM>(
        p, g, reinterpret_cast<float*>(lds) + wave * 32 * SRF, lane, row0 + wm * WTM, row_end,
        tn * (p.gated ? BN / 2 : BN) + wn * (p.gated ? WTN / 2 : WTN), [&](auto ic, float* stage) {
            constexpr int i = decltype(ic)::value;
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    *reinterpret_cast<f32x4*>(stage + lr * SRF + 32 * j + 8 * v + 4 * half) =
                        f32x4{acc[i][j][4 * v], acc[i][j][4 * v + 1], acc[i][j][4 * v + 2], acc[i][j][4 * v + 3]};
        });
}

// ------------------------------------------------------------------------------------
// The quad kernel over rows of groups: BMT x 256 tiles (BMT 256 or 192), one wave per SIMD
// with a quadrant each, the library's main loop (quad_body) on a tile of a group.
// ------------------------------------------------------------------------------------
template <int DT, int BMT>
struct QuadRows {
    static constexpr bool kActive = true;
    const FusedArgs& p;
    int g, row0, row_end, tn;

    __device__ __forceinline__ int rows() const { return row_end - row0 < BMT ? row_end - row0 : BMT; }
    __device__ __forceinline__ int a_rows() const { return p.row_index ? p.a_rows : rows(); }
    __device__ __forceinline__ int a_row(int r) const { return p.row_index ? a_row_of(p, row0 + r) : r; }
    __device__ __forceinline__ int b_row(int c) const { return b_row_of<256>(p, tn, c); }

    template <int MF, int TM, int TN, typename ACC>
    __device__ __forceinline__ void finish(const ACC& acc, u16* lds, int wave, int lane) const {
        constexpr int SRF = 128 + 4;
        const int wm = wave >> 1, wn = wave & 1, lr = lane % MF, kq = lane / MF;
        rows_epilogue<DT, 128, TM * MF / 32>(
            p, g, reinterpret_cast<float*>(lds) + wave * 32 * SRF, lane, row0 + wm * (TM * MF), row_end,
            tn * (p.gated ? 128 : 256) + wn * (p.gated ? 64 : 128), [&](auto ic, float* stage) {
                constexpr int i0 = decltype(ic)::value * 32 / MF;
#pragma unroll
                for (int i = 0; i < 32 / MF; ++i)
#pragma unroll
                    for (int j = 0; j < TN; ++j)
#pragma unroll
                        for (int v = 0; v < (MF == 16 ? 1 : 4); ++v)
                            *reinterpret_cast<f32x4*>(stage + (i * MF + lr) * SRF + MF * j +
                                                      (MF == 16 ? 4 * kq : 8 * v + 4 * kq)) =
                                f32x4{acc[i0 + i][j][4 * v], acc[i0 + i][j][4 * v + 1], acc[i0 + i][j][4 * v + 2],
                                      acc[i0 + i][j][4 * v + 3]};
            });
    }
};

template <int DT, int MF, int LAYOUT, bool OFFS, int BMT>
__global__ void __attribute__((amdgpu_flat_work_group_size(256, 256), amdgpu_waves_per_eu(1, 1)))
fused_quad(const FusedArgs p, int grid_n, int group_m) {
    int g, row0, row_end, tn;
    if (!find_tile<BMT>(p, (int)blockIdx.x, grid_n, group_m, g, row0, row_end, tn))
        return;
    g = __builtin_amdgcn_readfirstlane(g);
    row0 = __builtin_amdgcn_readfirstlane(row0);
    row_end = __builtin_amdgcn_readfirstlane(row_end);
    const QuadRows<DT, BMT> hook{p, g, row0, row_end, tn};
    quad_body<DT, MF, (MF == 16 ? 2 : 1), (MF == 16 ? 56 : 40), (MF == 16 ? 40 : 12), 1, 2, OFFS, LAYOUT, BMT,
              LAYOUT_MK, 0>(p.row_index ? p.A : p.A + (int64_t)row0 * p.lda, p.B + (int64_t)g * p.stride_b, nullptr,
                            hook.rows(), p.N, p.K, p.lda, p.ldb, 0, 0, tn, 0, 0, nullptr, 0, 0, 0, false, hook);
}

// The quad kernel of the sums over a group's rows, without a row index: 8192 x 4096 over
// 4096 rows 196 us (1400 TFLOP/s), against 232 by sum_tiled's 256 x 256.
template <int DT, bool OFFS>
__global__ void __attribute__((amdgpu_flat_work_group_size(256, 256), amdgpu_waves_per_eu(1, 1)))
sum_quad(const SumArgs p, int grid_i, int grid_j) {
    const int per = grid_i * grid_j, g = (int)blockIdx.x / per;
    int ti, tj, lo, hi;
    tile_of((int)blockIdx.x % per, grid_i, grid_j, 4, ti, tj);
    group_rows(p, g, lo, hi);
    lo = __builtin_amdgcn_readfirstlane(lo);
    hi = __builtin_amdgcn_readfirstlane(hi);
    quad_body<DT, 32, 1, 40, 12, 1, 2, OFFS, LAYOUT_KN, 256, LAYOUT_KM, 0>(
        p.left + (int64_t)lo * p.ldl, p.right + (int64_t)lo * p.ldr, p.D + (int64_t)g * p.stride_d, p.I, p.J, hi - lo,
        p.ldl, p.ldr, p.ldd, ti, tj, 0, 0, nullptr, 0, 0, 0);
}

// ------------------------------------------------------------------------------------
// The tiled kernel of the sums over a group's rows (sum_generic's products): both operands
// have the summed row as their row index, so both are KCols tiles, read by transposing
// reads.  With a row index, each tile's 64 indices come by a direct-to-LDS load of their own
// into a ring of four, four tiles before the tile whose loads need them (so that they are
// there by the wait for an older tile).
//   Through the index, 16 experts of 512 rows to 2048 x 2048 each take 97 us (256 x 256
// tiles; 708 TFLOP/s), without it 87: 14.7 % of its LDS cycles are bank conflicts, and a
// tile has 8 steps.
//   parts > 1 (few tiles, many rows): the rows of a group are cut into as many ranges, one
// workgroup each, whose fp32 tiles go to the workspace; sum_parts adds them in order.
// ------------------------------------------------------------------------------------
__device__ __forceinline__ void dma4_at(rsrc4_t r, uint32_t lds_byte, uint32_t voff) {
    const uint32_t m0v = __builtin_amdgcn_readfirstlane(lds_byte);
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds"
                 ::"v"(voff), "s"(r), "s"(m0v)
                 : "memory", "m0");
}

template <int DT, int BI, int BJ, int WI, int WJ, int ST, int OCC>
__global__ void __attribute__((amdgpu_flat_work_group_size(WI * WJ * 64, WI * WJ * 64),
                               amdgpu_waves_per_eu(OCC, OCC)))
sum_tiled(const SumArgs p, int grid_i, int grid_j) {
    constexpr int NW = WI * WJ, WTI = BI / WI, WTJ = BJ / WJ, TI = WTI / 32, TJ = WTJ / 32;
    constexpr int SLOT_L = BI * kTileK, STAGE = (BI + BJ) * kTileK;
    constexpr int SRS = WTJ + 8;                        // staged row in elements
    static_assert(NW * 32 * SRS <= ST * STAGE, "D staging fits the ring");
    __shared__ __attribute__((aligned(1024))) u16 lds[ST * STAGE];
    __shared__ __attribute__((aligned(256))) int32_t idx[NW][4][64];
    const int per = grid_i * grid_j, gp = (int)blockIdx.x / per, g = gp % p.groups, part = gp / p.groups;
    int ti, tj, lo, hi;
    tile_of((int)blockIdx.x % per, grid_i, grid_j, 4, ti, tj);
    group_rows(p, g, lo, hi);
    if (p.parts > 1) {                                  // whole tiles of 64 rows to each part
        const int tiles = (hi - lo + kTileK - 1) / kTileK, first = lo;
        lo = first + (int)((int64_t)part * tiles / p.parts) * kTileK;
        const int end = first + (int)((int64_t)(part + 1) * tiles / p.parts) * kTileK;
        hi = end < hi ? end : hi;
    }
    lo = __builtin_amdgcn_readfirstlane(lo);
    hi = __builtin_amdgcn_readfirstlane(hi);
    const int tid = (int)threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wi = wave / WJ, wj = wave % WJ, half = lane >> 5, lr = lane & 31;
    const int K = hi - lo, nk = (K + kTileK - 1) / kTileK;
    using LC = KCols<BI, NW>;
    using RC = KCols<BJ, NW>;
    const bool indexed = p.row_index != nullptr;
    constexpr int LOADS = LC::LD + RC::LD;

    const uint32_t lds0 = lds_addr(lds), idx0 = lds_addr(&idx[wave][0][0]);
    const rsrc4_t rx = make_rsrc4(p.row_index + (indexed ? lo : 0), indexed ? (uint32_t)K * 4u : 0u);
    auto load_idx = [&](int t) {
        if (indexed)
            dma4_at(rx, idx0 + (uint32_t)((t & 3) * 256), (uint32_t)(t * kTileK + lane) * 4u);
    };
    auto load = [&](int t, int slot) {
        const int k0 = t * kTileK;
        const uint32_t at = lds0 + (uint32_t)(slot * STAGE * 2);
        auto operand = [&](auto cols, const u16* base, int ld, int limit, int col0, bool via, uint32_t lds_at) {
            using C = decltype(cols);
            // plain rows: a buffer over the tile's own rows, so the tail reads as zeros
            const int rows = K - k0 < kTileK ? (K - k0 > 0 ? K - k0 : 0) : kTileK;
            const rsrc4_t r = via ? make_rsrc4(base, span_bytes(p.a_rows, limit, ld))
                                  : make_rsrc4(base + (int64_t)(lo + (rows > 0 ? k0 : 0)) * ld,
                                               span_bytes(rows, limit, ld));
#pragma unroll
            for (int i = 0; i < C::LD; ++i) {
                const int kk = C::k_of(wave, lane, i), n = col0 + C::col_of(wave, lane, i);
                int row = kk;
                bool ok = n < limit && kk < rows;
                if (via) {
                    const int v = idx[wave][t & 3][kk];
                    row = p.row_div == 1 ? v : v / p.row_div;
                    ok = ok && v >= 0 && row < p.a_rows;
                }
                dma16_at(r, lds_at + (uint32_t)((wave * C::LD + i) * 1024),
                         ok ? ((uint32_t)row * (uint32_t)ld + (uint32_t)n) * 2u : kOutOfRange, 0u);
            }
        };
        operand(LC{}, p.left, p.ldl, p.I, ti * BI, p.index_left, at);
        operand(RC{}, p.right, p.ldr, p.J, tj * BJ, p.index_right, at + SLOT_L * 2);
    };

    f32x16 acc[TI][TJ];
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j)
            acc[i][j] = f32x16{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
    int la[TI], ra[TJ];
#pragma unroll
    for (int i = 0; i < TI; ++i)
        la[i] = kc_at<BI>(lane, wi * WTI, i);
#pragma unroll
    for (int j = 0; j < TJ; ++j)
        ra[j] = kc_at<BJ>(lane, wj * WTJ, j);
    // a wave reads the indices that it loaded itself: its own wait is enough
#pragma unroll
    for (int t = 0; t < 4; ++t)
        load_idx(t);
    wait_vm<0>();
    const auto send = [&](int t, int slot) {      // tile t, and the indices of tile t + 4
        load(t, slot);
        if (indexed) {
            wave_lds_order();                     // the indices of tile t are read
            load_idx(t + 4);
        }
    };
    u32x4 fl[2][TI], fr[2][TJ];
    auto read = [&](int slot, int s, auto bufc) {
        constexpr int buf = decltype(bufc)::value;
        const u16* ls = lds + slot * STAGE;
        const u16* rs = ls + SLOT_L;
#pragma unroll
        for (int j = 0; j < TJ; ++j)
            fr[buf][j] = read_kcols<BJ>(rs + ra[j] + 16 * s * BJ);
#pragma unroll
        for (int i = 0; i < TI; ++i)
            fl[buf][i] = read_kcols<BI>(ls + la[i] + 16 * s * BI);
        __builtin_amdgcn_sched_barrier(0);
    };
    auto multiply = [&](auto bufc, auto fromc, auto toc) {
        constexpr int buf = decltype(bufc)::value;
        static_for<decltype(fromc)::value, decltype(toc)::value>([&](auto jc) {
            constexpr int i = decltype(jc)::value / TJ, j = decltype(jc)::value % TJ;
            acc[i][j] = mfma_32x32x16<DT>(fr[buf][j], fl[buf][i], acc[i][j]);
        });
        __builtin_amdgcn_sched_barrier(0);
    };
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    using IH = std::integral_constant<int, TI * TJ / 2>;
    using IE = std::integral_constant<int, TI * TJ>;
    static_assert(ST <= 4, "the indices of the first tiles are there, and at most three later tiles in flight");
#pragma unroll
    for (int t = 0; t < ST; ++t)
        send(t, t);
    // Loads complete in order: with a row index each tile's are followed by one of indices.
    // The indices that tile u needs were sent after tile u - 4, so the wait for tile t+1 in
    // step t, which sends tile t + ST <= t + 4, covers them.
    if (indexed)
        wait_vm_then_sync<(ST - 1) * (LOADS + 1)>();
    else
        wait_vm_then_sync<(ST - 1) * LOADS>();
    read(0, 0, I0{});
    int slot = 0;
    for (int t = 0; t < nk; ++t) {
        const int next = slot + 1 == ST ? 0 : slot + 1;
        read(slot, 1, I1{});
        multiply(I0{}, I0{}, IE{});
        read(slot, 2, I0{});
        multiply(I1{}, I0{}, IE{});
        read(slot, 3, I1{});
        multiply(I0{}, I0{}, IE{});
        multiply(I1{}, I0{}, IH{});
        if (indexed)
            wait_vm_then_sync<(ST - 2) * (LOADS + 1)>();
        else
            wait_vm_then_sync<(ST - 2) * LOADS>();
        __builtin_amdgcn_sched_barrier(0);
        send(t + ST, slot);
        read(next, 0, I0{});
        multiply(I1{}, IH{}, IE{});
        slot = next;
    }
    wait_vm_then_sync<0>();
    if (p.parts > 1) {
        // a lane's four consecutive columns of one row are one 16-byte store
        float* P = p.partial + (int64_t)gp * p.I * p.J;
#pragma unroll
        for (int i = 0; i < TI; ++i) {
            const int row = ti * BI + wi * WTI + 32 * i + lr;
#pragma unroll
            for (int j = 0; j < TJ; ++j)
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const int col = tj * BJ + wj * WTJ + 32 * j + 8 * v + 4 * half;
                    if (row < p.I && col < p.J)         // J is a multiple of 8
                        *reinterpret_cast<f32x4*>(P + (int64_t)row * p.J + col) =
                            f32x4{acc[i][j][4 * v], acc[i][j][4 * v + 1], acc[i][j][4 * v + 2],
                                  acc[i][j][4 * v + 3]};
                }
        }
        return;
    }
    // D: 32 rows at a time through LDS, 16 bytes per lane of whole row segments
    u16* stage = lds + wave * 32 * SRS;
    constexpr int RUNS = WTJ / 8, RPI = 64 / RUNS;
    const int j0 = tj * BJ + wj * WTJ + (lane % RUNS) * 8;
    u16* D = p.D + (int64_t)g * p.stride_d;
#pragma unroll
    for (int i = 0; i < TI; ++i) {
        wave_lds_order();
#pragma unroll
        for (int j = 0; j < TJ; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                *reinterpret_cast<u32x2*>(stage + lr * SRS + 32 * j + 8 * v + 4 * half) =
                    u32x2{pack2<DT>(acc[i][j][4 * v], acc[i][j][4 * v + 1]),
                          pack2<DT>(acc[i][j][4 * v + 2], acc[i][j][4 * v + 3])};
        wave_lds_order();
#pragma unroll
        for (int q = 0; q < 32 / RPI; ++q) {
            const int r = q * RPI + lane / RUNS, row = ti * BI + wi * WTI + 32 * i + r;
            const u32x4 v = *reinterpret_cast<const u32x4*>(stage + r * SRS + (lane % RUNS) * 8);
            if (row < p.I && j0 < p.J) {
                u16* q0 = D + (int64_t)row * p.ldd + j0;
                if (p.vec && j0 + 8 <= p.J) {
                    *reinterpret_cast<u32x4*>(q0) = v;
                } else {
                    const u16x8 h = __builtin_bit_cast(u16x8, v);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (j0 + e < p.J)
                            q0[e] = h[e];
                }
            }
        }
    }
}

// The parts' sums in order, eight columns of one row per thread, rounded once: with it the
// sum over 8192 rows to 1024 x 1024 takes 37 us (79 whole), over 16384 to 512 x 512 27 (154).
template <int DT>
__global__ void __launch_bounds__(256) sum_parts(const SumArgs p) {
    const int64_t runs = p.J / 8, q = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t plane = (int64_t)p.groups * p.I * p.J;
    if (q >= (int64_t)p.groups * p.I * runs)
        return;
    const int64_t row = q / runs;                       // group * I + i
    const int j = (int)(q - row * runs) * 8;
    const float* src = p.partial + row * p.J + j;
    float t[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 4
    for (int part = 0; part < p.parts; ++part) {
        const f32x4 a = *reinterpret_cast<const f32x4*>(src + part * plane);
        const f32x4 b = *reinterpret_cast<const f32x4*>(src + part * plane + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            t[e] += a[e];
            t[4 + e] += b[e];
        }
    }
    const int g = (int)(row / p.I), i = (int)(row - (int64_t)g * p.I);
    store8<DT>(p.D + (int64_t)g * p.stride_d + (int64_t)i * p.ldd + j, p.vec, 8, t);
}

}  // namespace tgemm
