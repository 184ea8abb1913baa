// The streaming kernel of the fused and grouped products: few rows per group, B [N,K].
#pragma once

#include "fused_tile.hpp"

namespace tgemm {

// The end of the streaming kernels: red[wave][row][column] (rows of NB + 4 floats) holds the
// waves' partial sums; added in wave order, they go through the epilogue as runs of eight
// columns.
template <int DT, int BM, int NB, int NW>
__device__ __forceinline__ void stream_epilogue(const FusedArgs& p, int g, const float* red, int tid, int row0,
                                                int row_end, int tn) {
    constexpr int SR = NB + 4;
    const int width = p.gated ? p.N >> 1 : p.N;
    auto emit = [&](auto gatedc) {
        constexpr bool GATED = decltype(gatedc)::value;
        constexpr int RUNS = NB / (GATED ? 16 : 8);
        for (int q = tid; q < BM * RUNS; q += NW * 64) {
            const int m = q / RUNS, c = (q % RUNS) * 8;
            const int n = tn * (GATED ? NB / 2 : NB) + c;
            if (row0 + m >= row_end || n >= width)
                continue;
            const int zc = GATED ? (c >> 4) * 32 + (c & 15) : c;
            float z[8] = {}, u[GATED ? 8 : 1] = {}, bz[8], bu[8];
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float* src = red + (w * BM + m) * SR + zc;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    z[e] += src[e];
                    if constexpr (GATED)
                        u[e] += src[16 + e];
                }
            }
            load_bias<DT>(p, g, n, width, bz, bu);
            finish_runs<DT, 1, 1, GATED>(p, row0 + m, row_end, n, width, z, u, bz, bu);
        }
    };
    if (p.gated)
        emit(std::true_type{});
    else
        emit(std::false_type{});
}

// ------------------------------------------------------------------------------------
// With few rows a product is one pass over B.  A workgroup takes 16 MT rows of a group and
// NB = 16 NT columns; its NW waves split K into contiguous runs of 64-wide chunks, each
// keeping an MT x NT block of 16x16x32 MFMA accumulators.
//   A wave fills a ring of S chunks of its own by 1 KiB direct-to-LDS loads of whole
//   128-byte row segments (8 rows each), S - 1 chunks ahead, and waits for its own loads
//   only: no barrier until the end.  (Loading MFMA operands straight into registers reads
//   16 rows x 16 bytes per quarter wave, and the load path, which takes one line at a
//   time, then holds the stream at 4 TB/s.)
//   LIVE: the A loads that a tile of few rows needs (8 rows each); the LDS rows of the
//   others are zeroed once.
//   At the end the waves' partial blocks are added in LDS in wave order (deterministic) and
//   go through the epilogue as runs of eight columns.
//   Gated, 16-column blocks take turns between the halves of N.
// Rows, columns and k outside read as zeros through the buffers' range check.
// Bound by B's stream: 4 x 8192 x 4096 gated in 12.4 us (67 MB, 5.4 TB/s), 64 rows over 64
// experts of 2048 x 2048 in 56 us (294 MB, 5.3 TB/s); from about 128 rows of one group the
// tiled kernels are faster (128 x 8192 x 4096: 31.6 us here, 25.2 tiled).
// ------------------------------------------------------------------------------------
template <int DT, int MT, int NT, int NW, int S, int OCC>
__global__ void __attribute__((amdgpu_flat_work_group_size(NW * 64, NW * 64), amdgpu_waves_per_eu(OCC)))
fused_stream(const FusedArgs p, int grid_n) {
    constexpr int BM = 16 * MT, NB = 16 * NT, SR = NB + 4;   // SR: staged row in floats
    constexpr int LA = BM / 8, LB = NB / 8;                  // 1 KiB loads per chunk
    constexpr int SLOT = (BM + NB) * kTileK;                 // elements of one chunk: A, then B
    constexpr int RED = NW * BM * SR * 2;                    // elements of the reduction
    static_assert(NT % 2 == 0, "gate and up blocks of a pair in one workgroup");
    __shared__ __attribute__((aligned(1024))) u16 lds[NW * S * SLOT > RED ? NW * S * SLOT : RED];
    int g, row0, row_end, tn;
    if (!find_tile<BM>(p, (int)blockIdx.x, grid_n, 1, g, row0, row_end, tn))
        return;
    g = __builtin_amdgcn_readfirstlane(g);
    row0 = __builtin_amdgcn_readfirstlane(row0);
    row_end = __builtin_amdgcn_readfirstlane(row_end);
    const int tid = (int)threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, kq = lane >> 4, K = p.K;
    const int width = p.gated ? p.N >> 1 : p.N;

    const u16* a0 = p.row_index ? p.A : p.A + (int64_t)row0 * p.lda;
    const int live_rows = row_end - row0 < BM ? row_end - row0 : BM;
    const rsrc4_t ra = make_rsrc4(a0, span_bytes(p.row_index ? p.a_rows : live_rows, K, p.lda));
    const rsrc4_t rb = make_rsrc4(p.B + (int64_t)g * p.stride_b, span_bytes(p.N, K, p.ldb));
    // load i: rows 8 i + lane / 8, the 16-byte chunk that the row's swizzle puts at lane % 8
    const int lrow = lane >> 3;
    int kc[2];
#pragma unroll
    for (int q = 0; q < 2; ++q)
        kc[q] = ((lane & 7) ^ swz<8>(8 * q + lrow)) * 8;
    uint32_t ao[LA], bo[LB];
#pragma unroll
    for (int i = 0; i < LA; ++i) {
        const int m = 8 * i + lrow;
        const int s = m >= live_rows ? -1 : (p.row_index ? a_row_of(p, row0 + m) : m);
        ao[i] = s < 0 ? kOutOfRange : ((uint32_t)s * (uint32_t)p.lda + (uint32_t)kc[i & 1]) * 2u;
    }
#pragma unroll
    for (int i = 0; i < LB; ++i) {
        const int c = 8 * i + lrow, up = (c >> 4) & 1;
        const int n = p.gated ? tn * (NB / 2) + (c >> 5) * 16 + (c & 15) : tn * NB + c;
        bo[i] = n < width ? ((uint32_t)(n + (p.gated && up ? width : 0)) * (uint32_t)p.ldb + (uint32_t)kc[i & 1]) * 2u
                          : kOutOfRange;
    }
    const int chunks = (K + kTileK - 1) / kTileK;
    const int lo = (int)((int64_t)wave * chunks / NW), hi = (int)((int64_t)(wave + 1) * chunks / NW);
    u16* ring = lds + wave * S * SLOT;
    const uint32_t ring0 = lds_addr(ring);
    f32x4 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
            acc[i][j] = f32x4{0, 0, 0, 0};
    auto walk = [&](auto livec) {
        constexpr int LIVE = decltype(livec)::value;
        auto load = [&](int t, int slot) {
            const int k0 = t * kTileK;
            const uint32_t at = ring0 + (uint32_t)(slot * SLOT * 2), ko = (uint32_t)k0 * 2u;
            const uint32_t v0 = t < hi && k0 + kc[0] < K ? 0u : kOutOfRange;
            const uint32_t v1 = t < hi && k0 + kc[1] < K ? 0u : kOutOfRange;
#pragma unroll
            for (int i = 0; i < LB; ++i)
                dma16_at(rb, at + (uint32_t)(BM * kTileK * 2 + i * 1024), bo[i] | (i & 1 ? v1 : v0), ko);
#pragma unroll
            for (int i = 0; i < LIVE; ++i)
                dma16_at(ra, at + (uint32_t)(i * 1024), ao[i] | (i & 1 ? v1 : v0), ko);
        };
        if constexpr (LIVE < LA) {
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int i = LIVE; i < LA; ++i)
                    *reinterpret_cast<u32x4*>(ring + s * SLOT + i * 512 + lane * 8) = u32x4{0u, 0u, 0u, 0u};
        }
#pragma unroll
        for (int s = 0; s < S - 1; ++s)
            load(lo + s, s);
        int slot = 0;
        for (int t = lo; t < hi; ++t) {
            // the slot that chunk t-1 left: this wave has read it
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            load(t + S - 1, slot == 0 ? S - 1 : slot - 1);
            wait_vm<(S - 1) * (LB + LIVE)>();
            const u16* as = ring + slot * SLOT + r * kTileK;
            const u16* bs = as + BM * kTileK;
            u32x4 fa[2][MT], fb[2][NT];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int ko = ((4 * s + kq) ^ swz<8>(r)) * 8;
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    fb[s][j] = *reinterpret_cast<const u32x4*>(bs + 16 * j * kTileK + ko);
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    fa[s][i] = *reinterpret_cast<const u32x4*>(as + 16 * i * kTileK + ko);
            }
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        acc[i][j] = mfma_16x16x32<DT>(fb[s][j], fa[s][i], acc[i][j]);
            slot = slot + 1 == S ? 0 : slot + 1;
        }
    };
    if (live_rows > BM / 2)
        walk(std::integral_constant<int, LA>{});
    else
        walk(std::integral_constant<int, LA / 2>{});
    wait_vm_then_sync<0>();
    // acc[i][j]: row 16 i + l % 16, columns 16 j + 4 (l / 16) .. +3
    float* red = reinterpret_cast<float*>(lds);
    float* mine = red + wave * BM * SR;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
            *reinterpret_cast<f32x4*>(mine + (16 * i + r) * SR + 16 * j + kq * 4) = acc[i][j];
    __syncthreads();
    stream_epilogue<DT, BM, NB, NW>(p, g, red, tid, row0, row_end, tn);
}

// The same for B [K,N]: a chunk's 64 k rows of the workgroup's 32 columns (64 bytes each, 16
// rows per load) lie in LDS as they come -- the four rows of a transposing read are 64 bytes
// apart and fill the 64 banks -- and 32x32x16 MFMAs take MT x 32 rows.  Adjacent column
// blocks, which share each 128-byte line of B, run on one XCD.  8 x 8192 x 4096 in 22 us (3
// TB/s) against 26 of the tiled kernel, 64 x 4096 x 4096 in 15.7 against 25.
template <int DT, int MT, int NW, int S, int OCC>
__global__ void __attribute__((amdgpu_flat_work_group_size(NW * 64, NW * 64), amdgpu_waves_per_eu(OCC)))
fused_stream_kn(const FusedArgs p, int grid_n) {
    constexpr int BM = 32 * MT, NB = 32, SR = NB + 4;
    constexpr int LA = BM / 8, LB = 4;
    constexpr int SLOT = (BM + NB) * kTileK;
    constexpr int RED = NW * BM * SR * 2;
    __shared__ __attribute__((aligned(1024))) u16 lds[NW * S * SLOT > RED ? NW * S * SLOT : RED];
    int g, row0, row_end, tn;
    if (!find_tile<BM>(p, (int)blockIdx.x, grid_n, 1, g, row0, row_end, tn))
        return;
    g = __builtin_amdgcn_readfirstlane(g);
    row0 = __builtin_amdgcn_readfirstlane(row0);
    row_end = __builtin_amdgcn_readfirstlane(row_end);
    const int tid = (int)threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lr = lane & 31, half = lane >> 5, K = p.K;
    const int width = p.gated ? p.N >> 1 : p.N;
    const u16* a0 = p.row_index ? p.A : p.A + (int64_t)row0 * p.lda;
    const int live_rows = row_end - row0 < BM ? row_end - row0 : BM;
    const rsrc4_t ra = make_rsrc4(a0, span_bytes(p.row_index ? p.a_rows : live_rows, K, p.lda));
    const rsrc4_t rb = make_rsrc4(p.B + (int64_t)g * p.stride_b, span_bytes(K, p.N, p.ldb));
    const int lrow = lane >> 3;
    int kc[2];
#pragma unroll
    for (int q = 0; q < 2; ++q)
        kc[q] = ((lane & 7) ^ swz<8>(8 * q + lrow)) * 8;
    uint32_t ao[LA], bo[LB];
#pragma unroll
    for (int i = 0; i < LA; ++i) {
        const int m = 8 * i + lrow;
        const int s = m >= live_rows ? -1 : (p.row_index ? a_row_of(p, row0 + m) : m);
        ao[i] = s < 0 ? kOutOfRange : ((uint32_t)s * (uint32_t)p.lda + (uint32_t)kc[i & 1]) * 2u;
    }
    const int bk = lane >> 2, bc = (lane & 3) * 8;
    const int bn = p.gated ? tn * (NB / 2) + (bc & 15) : tn * NB + bc;
#pragma unroll
    for (int i = 0; i < LB; ++i)
        bo[i] = bn < width ? ((uint32_t)(16 * i + bk) * (uint32_t)p.ldb +
                              (uint32_t)(bn + (p.gated && bc >= 16 ? width : 0))) * 2u
                           : kOutOfRange;
    const int chunks = (K + kTileK - 1) / kTileK;
    const int lo = (int)((int64_t)wave * chunks / NW), hi = (int)((int64_t)(wave + 1) * chunks / NW);
    u16* ring = lds + wave * S * SLOT;
    const uint32_t ring0 = lds_addr(ring);
    f32x16 acc[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
        acc[i] = f32x16{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
    const int g4 = lane >> 4, sl = lane & 15;
    const int btr = (8 * (g4 >> 1) + (sl >> 2)) * NB + 16 * (g4 & 1) + 4 * (sl & 3);
    auto walk = [&](auto livec) {
        constexpr int LIVE = decltype(livec)::value;
        auto load = [&](int t, int slot) {
            const int k0 = t < hi ? t * kTileK : 0;
            const uint32_t at = ring0 + (uint32_t)(slot * SLOT * 2);
            const bool in = t < hi;
#pragma unroll
            for (int i = 0; i < LB; ++i)
                dma16_at(rb, at + (uint32_t)(BM * kTileK * 2 + i * 1024),
                         in && k0 + 16 * i + bk < K ? bo[i] : kOutOfRange, (uint32_t)k0 * (uint32_t)p.ldb * 2u);
            const uint32_t v0 = in && k0 + kc[0] < K ? 0u : kOutOfRange;
            const uint32_t v1 = in && k0 + kc[1] < K ? 0u : kOutOfRange;
#pragma unroll
            for (int i = 0; i < LIVE; ++i)
                dma16_at(ra, at + (uint32_t)(i * 1024), ao[i] | (i & 1 ? v1 : v0), (uint32_t)k0 * 2u);
        };
        if constexpr (LIVE < LA) {
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int i = LIVE; i < LA; ++i)
                    *reinterpret_cast<u32x4*>(ring + s * SLOT + i * 512 + lane * 8) = u32x4{0u, 0u, 0u, 0u};
        }
#pragma unroll
        for (int s = 0; s < S - 1; ++s)
            load(lo + s, s);
        int slot = 0;
        for (int t = lo; t < hi; ++t) {
            wave_lds_order();              // this wave has read the slot that chunk t-1 left
            load(t + S - 1, slot == 0 ? S - 1 : slot - 1);
            wait_vm<(S - 1) * (LB + LIVE)>();
            const u16* as = ring + slot * SLOT;
            const u16* bs = as + BM * kTileK;
            u32x4 fa[4][MT], fb[4];
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                fb[s] = read_kcols<NB>(bs + btr + 16 * s * NB);
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    fa[s][i] = *reinterpret_cast<const u32x4*>(as + (32 * i + lr) * kTileK +
                                                               (((2 * s) | half) ^ swz<8>(lr)) * 8);
            }
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    acc[i] = mfma_32x32x16<DT>(fb[s], fa[s][i], acc[i]);
            slot = slot + 1 == S ? 0 : slot + 1;
        }
    };
    if (live_rows > BM / 2)
        walk(std::integral_constant<int, LA>{});
    else if (live_rows > 8)
        walk(std::integral_constant<int, LA / 2>{});
    else
        walk(std::integral_constant<int, 1>{});
    wait_vm_then_sync<0>();
    float* red = reinterpret_cast<float*>(lds);
    float* mine = red + wave * BM * SR;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v)
            *reinterpret_cast<f32x4*>(mine + (32 * i + lr) * SR + 8 * v + 4 * half) =
                f32x4{acc[i][4 * v], acc[i][4 * v + 1], acc[i][4 * v + 2], acc[i][4 * v + 3]};
    __syncthreads();
    stream_epilogue<DT, BM, NB, NW>(p, g, red, tid, row0, row_end, tn);
}

}  // namespace tgemm
