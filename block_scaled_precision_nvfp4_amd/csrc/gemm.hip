// gemm.hip -- block-scaled GEMM C[M][N] = alpha * A[M][K] * B[N][K]^T on gfx950 MFMA.
//
// NVFP4 operands (E2M1 codes, one E4M3 scale per 16 K-elements, fp32 tensor scale).  The
// gfx950 block-scaled MFMA takes one power-of-two (E8M0) scale per 32 K-elements, which
// can express neither an E4M3 mantissa nor a 16-element block.  Each element is therefore
// dequantized in registers to f16 -- E2M1 value times E4M3 scale has at most 6 significant
// bits and lies in [2^-10, 2688], so the f16 value is exact -- and contracted with the
// f16 MFMA v_mfma_f32_32x32x16_f16.  Dequantization per pair of codes is one
// v_cvt_scalef32_pk_f16_fp4 (hardware E2M1 -> f16; its scale operand contributes only its
// exponent, here 2^8) and one packed f16 multiply by the block scale, held as the f16
// whose bit pattern is (E4M3 byte << 7): for every E4M3 code, normal or subnormal, that
// f16 equals the E4M3 value times 2^-8, so the product is exactly code * scale.  The
// tensor scales enter once, in the epilogue: alpha = 1 / (S_a * S_b).  An operand may
// instead carry one outer scale per row (row-scaled NVFP4); the epilogue then takes
// alpha(m, n) from a per-tile table of row and column factors (see tile_factors).
//
// MXFP8 operands (E4M3 codes, one E8M0 scale per 32 K-elements) map one-to-one onto the
// scaled MFMA v_mfma_scale_f32_32x32x64_f8f6f4.  Its K layout: in lane (row, g), bytes
// 0-15 of the 32-byte operand are K-elements 16g..16g+15 of the step and bytes 16-31 are
// K-elements 32+16g..32+16g+15; the scale of K-block 0 (elements 0-31) comes from lanes
// 0-31, that of K-block 1 from lanes 32-63.
//
// Tiling: a workgroup computes a 256 x 256 tile of C with 4 waves of 128 x 128 (4 x 4 MFMA
// tiles of 32 x 32, 256 fp32 accumulators per lane).  Each K slice (128 elements for NVFP4, 64
// for MXFP8) of both operands is 64 bytes of codes per row, moved from memory straight into a
// ring of 4 LDS stages by LDS DMA, three slices ahead of its use, with one barrier per slice.
// Scales: 16-byte records of a row's scale bytes where scale rows lie 16 bytes apart (NVFP4 K a
// multiple of 256; MXFP8 also at an offset inside the record, or per-slice bytes otherwise),
// and for NVFP4 with any other K (or K-grouped) per-slice records of 3 aligned dwords per row.
// MXFP8 codes may come in the slab layout, where each slice of a tile's rows is one contiguous
// block.  Plain NVFP4 launches with per-tensor scales run persistently (gemm_nvp_kernel),
// carrying the LDS ring from one tile to the next.  The buffer loads' range check zero-fills
// rows beyond M or N, and an out-of-range offset the K tail.  16-byte chunks are XOR-swizzled
// by row.  Inside a slice the operands of the next MFMA step are read from LDS (and, for
// NVFP4, dequantized) while the current step's MFMAs issue.  Workgroups are renumbered so that
// each of the 8 XCDs (which take workgroups round-robin) works on a contiguous band of output
// tiles and reuses operand rows from its own L2.
#include "gemm_tile.hpp"
#include "launch.hpp"

namespace bsq {

// ---------------------------------------------------------------- grouped launches
//
// A grouped launch runs one GEMM per group g, the groups given by boundaries offs[g] ..
// offs[g+1] on the device (clamped to [0, extent]):
//   M-grouped (the per-expert GEMMs of a mixture-of-experts layer, fprop and dgrad): the
//     group's rows of A [extent][K] and of C [extent][N], against B_g [N][K], the g-th of
//     the stacked B [groups][N][K];
//   K-grouped (wgrad): C_g [M][N], the g-th of the stacked C [groups][M][N], contracts
//     columns offs[g] .. offs[g+1] of A [M][extent] and B [N][extent] (rows of length
//     extent); the boundaries must be multiples of 32 (a group whose are not is computed as
//     empty, C_g = 0).
// Workgroups are dealt to the groups in order, each group taking a multiple of 8 of them so
// that its tiles see the same XCD phase as a plain launch; a workgroup past its group's tiles
// exits at once.  Everything a group needs -- its operand and output bases, its tensor scales
// and its extent -- is folded into the GemmArgs, and the tile code runs unchanged.
struct GroupArgs {
    const int64_t* offs;   // groups + 1 boundaries (device)
    int64_t groups;
    int64_t extent;        // rows of A and C (M-grouped) or K (K-grouped)
};

__device__ __forceinline__ void group_bounds(const GroupArgs& q, int64_t grp, int64_t& o0, int64_t& o1) {
    int64_t a = q.offs[grp], b = q.offs[grp + 1];
    a = a < 0 ? 0 : (a > q.extent ? q.extent : a);
    b = b < a ? a : (b > q.extent ? q.extent : b);
    o0 = a;
    o1 = b;
}

__device__ __forceinline__ int64_t shfl64(int64_t v, int src) {
    const int lo = __shfl((int)(uint32_t)v, src), hi = __shfl((int)(uint32_t)((uint64_t)v >> 32), src);
    return (int64_t)(((uint64_t)(uint32_t)hi << 32) | (uint32_t)lo);
}

// A wave-uniform 64-bit value moved to scalar registers (buffer resources built from it must
// be scalar).
__device__ __forceinline__ int64_t uniform64(int64_t v) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)v >> 32));
    return (int64_t)(((uint64_t)hi << 32) | lo);
}

// M-grouped: the group of workgroup bid and its index within the group's share (each wave
// scans the boundaries itself, 64 groups at a time, with a wave prefix sum of the shares).
// The loop runs to the end with a uniform trip count and the results pass through
// readfirstlane, so that they stay in scalar registers.
__device__ __forceinline__ bool group_of_m(const GroupArgs& q, int64_t nbn, int64_t bid, int64_t& grp,
                                           int64_t& local) {
    const int lane = threadIdx.x & 63;
    int64_t before = 0, found = -1, loc = 0;
    for (int64_t c0 = 0; c0 < q.groups; c0 += 64) {
        const int64_t gi = c0 + lane;
        int64_t t = 0;
        if (gi < q.groups) {
            int64_t o0, o1;
            group_bounds(q, gi, o0, o1);
            t = (((o1 - o0 + GBM - 1) / GBM) * nbn + 7) & ~(int64_t)7;
        }
        int64_t incl = t;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int64_t v = shfl64(incl, lane >= o ? lane - o : lane);
            if (lane >= o) incl += v;
        }
        const int64_t start = before + incl - t;
        const uint64_t hit = __ballot(t > 0 && bid >= start && bid < start + t);
        if (found < 0 && hit != 0) {
            const int l = __builtin_ctzll(hit);
            found = uniform64(c0 + l);
            loc = uniform64(bid - shfl64(start, l));
        }
        before = uniform64(before + shfl64(incl, 63));
    }
    grp = found;
    local = loc;
    return found >= 0;
}

// The GEMM of K-group grp folded into g: its K range, operand and output bases and tensor
// scales.
template <int FMT, int OUT_F32>
__device__ __forceinline__ void k_group_args(GemmArgs& g, const GroupArgs& q, int64_t grp) {
    using F = Fmt<FMT>;
    constexpr int ES = OUT_F32 ? 4 : 2;
    int64_t o0, o1;
    group_bounds(q, grp, o0, o1);
    if (o0 % 32 != 0 || (o1 - o0) % 32 != 0) o1 = o0 = 0;
    g.K = o1 - o0;
    // a slab operand's group is addressed from its band (mx_gslab_codes); a row-major one
    // from the group's first code byte of each row
    if (!(g.slab & 1)) g.a_codes += o0 / F::EPB;
    if (!(g.slab & 2)) g.b_codes += o0 / F::EPB;
    g.k0 = o0;
    g.a_scales += o0 / F::BLK;
    g.b_scales += o0 / F::BLK;
    g.c = (uint8_t*)g.c + grp * g.M * g.N * ES;
    if constexpr (F::NV) {
        g.a_s_enc += grp;
        g.b_s_enc += grp;
    }
}

// Fold group bookkeeping into g; bid becomes the workgroup's index within its group's tiles.
// Returns false for a workgroup with no tile.
template <int FMT, int OUT_F32, int GM>
__device__ __forceinline__ bool enter_group(GemmArgs& g, const GroupArgs& q, int64_t& bid) {
    using F = Fmt<FMT>;
    constexpr int ES = OUT_F32 ? 4 : 2;
    const int64_t rb = g.ld / F::EPB, sb = g.ld / F::BLK;
    const int64_t nbn = (g.N + GBN - 1) / GBN;
    int64_t grp, local, o0, o1;
    if constexpr (GM == 1) {
        if (!group_of_m(q, nbn, bid, grp, local)) return false;
        group_bounds(q, grp, o0, o1);
        g.M = o1 - o0;
        g.a_codes += o0 * rb;
        g.a_scales += o0 * sb;
        g.b_codes += grp * g.N * rb;
        g.b_scales += grp * g.N * sb;
        g.c = (uint8_t*)g.c + o0 * g.N * ES;
        if constexpr (F::NV) {
            g.a_s_enc += g.a_rows ? o0 : grp;
            g.b_s_enc += g.b_rows ? grp * g.N : grp;
        }
    } else {
        const int64_t nbm = (g.M + GBM - 1) / GBM;
        const int64_t share = (nbm * nbn + 7) & ~(int64_t)7;
        grp = bid / share;
        local = bid - grp * share;
        if (grp >= q.groups) return false;
        k_group_args<FMT, OUT_F32>(g, q, grp);
    }
    bid = local;
    return bid < ((g.M + GBM - 1) / GBM) * nbn;
}

// One output tile per workgroup.  GM 0: a plain launch; 1: M-grouped; 2: K-grouped; 3:
// K-grouped MXFP8 with slab-layout operands.
template <int FMT, int OUT_F32, int GM>
__global__ __launch_bounds__(Fmt<FMT>::THREADS, 1) void gemm_kernel(GemmArgs g, GroupArgs q) {
    using F = Fmt<FMT>;
    // static LDS (up to 152 KiB of gfx950's 160 KiB): no per-kernel attribute to raise at run time
    __shared__ __attribute__((aligned(16))) uint8_t lds[F::LDS];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int64_t bid = blockIdx.x;
    if constexpr (GM != 0) {
        if (!enter_group<FMT, OUT_F32, GM>(g, q, bid)) return;   // uniform
    }
    int64_t tm, tn;
    tile_of((g.M + GBM - 1) / GBM, (g.N + GBN - 1) / GBN, bid, tm, tn);
    const int64_t m0 = tm * GBM, n0 = tn * GBN;
    constexpr int TN = F::TN;
    const int wm = (wave / F::WAVES_N) * 128, wn = (wave % F::WAVES_N) * 32 * TN;

    floatx16 acc[4][TN];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

    const int64_t nk = (g.K + F::BK - 1) / F::BK;
    // Uniform output factor of the LDS-DMA NVFP4 kernel with per-tensor scales on both
    // operands, alpha = fp32(1 / (S_a S_b)) with the product and quotient in binary64 (as in
    // tile_factors); computed before the main loop so that the epilogue does not wait for the
    // scale loads.
    float alpha_pt = 1.0f;
    if constexpr (FMT == 2 || FMT == 3) {
        if (!g.a_rows && !g.b_rows) alpha_pt = (float)(1.0 / ((double)g.a_s_enc[0] * (double)g.b_s_enc[0]));
#if __HIP_DEVICE_COMPILE__
        asm volatile("" : "+v"(alpha_pt));
#endif
    }
    const int frow = lane & 31, kh = lane >> 5;
    if constexpr (FMT == 1) {
        // scale records need rows 16 bytes apart; aligned ones also K a multiple of 512 and
        // 16-byte aligned scale tensors
        const bool rows16 = (g.ld / 32) % 16 == 0;
        const bool recs = rows16 && g.K % (MX_GROUP * 64) == 0 &&
                          (((uintptr_t)g.a_scales | (uintptr_t)g.b_scales) % 16) == 0;
        if constexpr (GM == 3) {
            // K-grouped slab operands (a kernel of its own: with the other main loops in one
            // function the register allocation spills): group starts are multiples of 32, not
            // of a slice, so offset records for the scales (their rows are 16 bytes apart: the
            // API asks for K % 512 == 0 here) and band-wide addressing for the codes
            if (g.slab == 3) mx_main_loop<MX_GSLAB, 3>(g, m0, n0, nk, lds, wm, wn, lane, acc);
            else if (g.slab == 2) mx_main_loop<MX_GSLAB, 2>(g, m0, n0, nk, lds, wm, wn, lane, acc);
            else mx_main_loop<MX_GSLAB, 1>(g, m0, n0, nk, lds, wm, wn, lane, acc);
        } else if (recs && g.slab == 3) mx_main_loop<MX_SLAB, 3>(g, m0, n0, nk, lds, wm, wn, lane, acc);
        else if (recs && g.slab == 2) mx_main_loop<MX_SLAB, 2>(g, m0, n0, nk, lds, wm, wn, lane, acc);
        else if (recs && g.slab == 1) mx_main_loop<MX_SLAB, 1>(g, m0, n0, nk, lds, wm, wn, lane, acc);
        else if (recs) mx_main_loop<MX_RECS>(g, m0, n0, nk, lds, wm, wn, lane, acc);
        else if (rows16) mx_main_loop<MX_OFFRECS>(g, m0, n0, nk, lds, wm, wn, lane, acc);
        else mx_main_loop<MX_SLOTS>(g, m0, n0, nk, lds, wm, wn, lane, acc);
    } else if constexpr (FMT == 2) {
        nvw_main_loop<TN>(g, m0, n0, nk, lds, wm, wn, lane, acc);
    } else {
        nvs_main_loop<TN>(g, m0, n0, nk, lds, wm, wn, lane, acc);
    }
    (void)alpha_pt;

    static_assert(F::LDS - FACT_BYTES >= 4 * 128 * (128 * 2 + 16) && F::LDS - FACT_BYTES >= 4 * 64 * (128 * 4 + 16),
                  "factor tables overlap the epilogue staging");
    // NVFP4 output factors (MXFP8 needs none: its scales are inside the MFMA)
    float* fa = (float*)(lds + F::LDS - FACT_BYTES);
    float* fb = fa + 256;
    __syncthreads();   // every wave is done with the operand buffers (and its DMAs)
    constexpr int ES = OUT_F32 ? 4 : 2;
    // staged epilogue: every column of the tile inside C (rows past M are skipped there)
    const bool staged = n0 + GBN <= g.N && (g.N * ES) % 16 == 0;   // uniform
    const int64_t m_end = g.M - m0;
    if constexpr (FMT == 2 || FMT == 3) {
        // per-tensor scales on both operands: one uniform factor, no tables
        if (staged && !g.a_rows && !g.b_rows) {
            store_tile_lds<OUT_F32, true>(g, lds, m0, n0, wm, wn, wave, lane, nullptr, nullptr, alpha_pt, m_end, acc);
            return;
        }
    }
    if constexpr (F::NV) {
        tile_factors<FMT>(g, m0, n0, fa, fb);
        __syncthreads();
    }
    if (staged) {
        store_tile_lds<OUT_F32, F::NV>(g, lds, m0, n0, wm, wn, wave, lane, fa, fb, 1.0f, m_end, acc);
        return;
    }
    // the accumulators hold C^T tiles (see nvw_mfma): lane (frow, kh), register r of tile (i, j)
    // is row 32i + frow, column 32j + within
    static_for<0, 4 * TN>([&](auto t_c) {
        constexpr int i = decltype(t_c)::value / TN, j = decltype(t_c)::value % TN;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int within = 8 * (r >> 2) + 4 * kh + (r & 3);
            const int lrow = wm + 32 * i + frow;
            const int lcol = wn + 32 * j + within;
            const int64_t row = m0 + lrow, col = n0 + lcol;
            if (row < g.M && col < g.N) {
                const float v = F::NV ? acc[i][j][r] * (fa[lrow] * fb[lcol]) : acc[i][j][r];
                if (OUT_F32) {
                    // two 16-bit halves: one 32-bit store per accumulator here changes the
                    // MXFP8 kernel's register allocation so that its main loop spills ~220
                    // registers per lane
                    const uint32_t b = __float_as_uint(v);
                    uint16_t* p = (uint16_t*)((float*)g.c + row * g.N + col);
                    p[0] = (uint16_t)(b & 0xFFFFu);
                    p[1] = (uint16_t)(b >> 16);
                }
                else ((uint16_t*)g.c)[row * g.N + col] = (uint16_t)f32_to_bf16_rne(v);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    });
}

// ---------------------------------------------------------------- persistent NVFP4 kernel
//
// Plain NVFP4 launches with a per-tensor scale on B and on A (or, with bf16 output, one per row of A), on
// nvp_tiles.
template <bool OUT_F32>
constexpr int nvp_stores() { return OUT_F32 ? 64 : 32; }   // 128 rows x 256 or 512 bytes / (64 x 16)

// One tile's accumulators (C^T layout, see nvw_mfma) times alpha, to C.  The tile at (m0, n0)
// is 256 x 64 TN (2 x 2 waves of 128 x 32 TN); `stage` is 32 KiB of LDS no other wave touches
// until the next barrier.  A pass stages 32 rows (one accumulator row group i) by JS x 32
// columns of the wave's block in the wave's 8 KiB, row-major with the 16-byte chunk index
// XORed with the row, then each lane stores CPL chunks.  Every lane takes part in every pass.
// With rowf, row r of the tile takes the factor rowf[r] instead of alpha (a row-scaled A).
template <bool OUT_F32, int TN>
__device__ __forceinline__ void nvp_store(const GemmArgs& g, int64_t m0, int64_t n0, int wm, int wn, int wave,
                                          int lane, float alpha, const floatx16 (&acc)[4][TN], uint8_t* stage,
                                          const float* rowf = nullptr) {
    constexpr int ES = OUT_F32 ? 4 : 2;
    constexpr int JS = 8 / ES < TN ? 8 / ES : TN;   // 32-column groups per pass (8 KiB / 32 rows / 32 / ES)
    constexpr int RB = 32 * JS * ES;                // staged bytes per row
    constexpr int CPR = RB / 16;                    // 16-byte chunks per row (a power of 2)
    constexpr int CPL = 32 * CPR / 64;              // chunks per lane per pass
    static_assert(32 * RB <= 8192 && (CPR & (CPR - 1)) == 0 && CPL * 64 == 32 * CPR, "pass shape");
    uint8_t* reg = stage + wave * 8192;
    const int frow = lane & 31, kh = lane >> 5;
    const __amdgpu_buffer_rsrc_t rs =
        make_rsrc((const uint8_t*)g.c + m0 * g.N * ES, tile_rows(g.M - m0, GBM) * g.N * ES);
    const uint32_t pitch = (uint32_t)(g.N * ES);
    const int64_t cleft = g.N - n0 - wn;   // columns of C from the block's first one on
    const uint32_t cbase = (uint32_t)(n0 + wn) * ES;
    static_for<0, 4 * (TN / JS)>([&](auto p_c) {
        constexpr int I = decltype(p_c)::value / (TN / JS), J0 = (decltype(p_c)::value % (TN / JS)) * JS;
        const float f = rowf ? rowf[wm + 32 * I + frow] : alpha;   // the lane's row in this pass
#pragma unroll
        for (int jj = 0; jj < JS; ++jj)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int j = J0 + jj;
                const float x = acc_read(acc[I][j][4 * q]) * f, y = acc_read(acc[I][j][4 * q + 1]) * f;
                const float z = acc_read(acc[I][j][4 * q + 2]) * f, w = acc_read(acc[I][j][4 * q + 3]) * f;
                const int col = 32 * jj + 8 * q + 4 * kh;   // first of the 4 columns, within the pass
                uint8_t* dst = reg + frow * RB + (((col * ES / 16) ^ (frow & (CPR - 1))) << 4) + (col * ES) % 16;
                if constexpr (OUT_F32) *(float4*)dst = make_float4(x, y, z, w);
                else *(uint2*)dst = make_uint2(bf16x2_rne(x, y), bf16x2_rne(z, w));
            }
#pragma unroll
        for (int k = 0; k < CPL; ++k) {
            const int t = 64 * k + lane, r = t / CPR, c = t % CPR;
            const uint4 v = *(const uint4*)(reg + r * RB + ((c ^ (r & (CPR - 1))) << 4));
            const int col = 32 * J0 + c * (16 / ES);   // first column of the chunk in the block
            const uint32_t off = col < cleft ? (uint32_t)(wm + 32 * I + r) * pitch + cbase + (uint32_t)(col * ES) : OOB;
            __builtin_amdgcn_raw_buffer_store_b128(u32x4s{v.x, v.y, v.z, v.w}, rs, (int)off, 0, 0);
        }
    });
}

// AROWS: A is row-scaled (one tensor scale per row of A, B per-tensor): each tile's rows take
// fp32(1 / (S_a[m] S_b)) (product and quotient in binary64, as tile_factors), the row's scale
// loaded at the top of the tile and the factors put in LDS between the last slice and the
// stores.
template <bool OUT_F32, bool AROWS = false>
__global__ __launch_bounds__(256, 1) void gemm_nvp_kernel(GemmArgs g, int64_t t_full, int64_t halves) {
    constexpr int TN = 4;
    __shared__ __attribute__((aligned(16))) uint8_t lds[Fmt<2>::LDS];
    __shared__ float rowf[AROWS ? GBM : 1];   // a row-scaled A's factors of the tile being stored
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = (wave >> 1) * 128, wn = (wave & 1) * 128;
    const int64_t nbm = (g.M + GBM - 1) / GBM, nbn = (g.N + GBN - 1) / GBN;
    const int64_t P = gridDim.x;
    const int items = (int)((t_full - 1 - (int64_t)blockIdx.x) / P) + 1;   // t_full >= P
    const int nk = (int)(g.K / 128);   // even, >= 4
    // alpha = fp32(1 / (S_a S_b)), product and quotient in binary64 (as in tile_factors)
    const double sbd = (double)g.b_s_enc[0];
    float alpha = AROWS ? 1.0f : (float)(1.0 / ((double)g.a_s_enc[0] * sbd));
#if __HIP_DEVICE_COMPILE__
    asm volatile("" : "+v"(alpha));
#endif
    // thread t's row of the tile (t < 256 = GBM): its A tensor scale and output factor
    auto row_scale = [&](int64_t tm0) { return g.a_s_enc[tm0 + threadIdx.x < g.M ? tm0 + threadIdx.x : g.M - 1]; };
    auto put_factors = [&](int64_t tm0, float sa) {
        rowf[threadIdx.x] = tm0 + threadIdx.x < g.M ? (float)(1.0 / ((double)sa * sbd)) : 1.0f;
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    };
    [[maybe_unused]] float sa_row = 0.0f;
    nvp_tiles<nvp_stores<OUT_F32>()>(
        g, nbm, nbn, P, items, lds, wm, wn, lane,
        [&](int64_t m0) {
            if constexpr (AROWS) sa_row = row_scale(m0);   // used by the stores at the tile's end
        },
        [&](int64_t m0, int64_t n0, const floatx16 (&acc)[4][TN], uint8_t* stage) {
            if constexpr (AROWS) {
                put_factors(m0, sa_row);
                nvp_store<OUT_F32, TN>(g, m0, n0, wm, wn, wave, lane, alpha, acc, stage, rowf);
            } else {
                nvp_store<OUT_F32, TN>(g, m0, n0, wm, wn, wave, lane, alpha, acc, stage);
            }
        });

    // The last, partial round of tiles (t_full .. t_full + halves / 2), each split into two
    // 256 x 128 halves, one per workgroup: 4 waves of 128 x 64 (TN = 2) with the full tile's
    // DMA plan (the B rows past 128 read nothing).  A half costs a little more than half a tile
    // (6 dequantization VALU per MFMA against 4.4), against a whole tile for the workgroups of
    // a partial round that is left whole.
    if ((int64_t)blockIdx.x < halves) {
        __syncthreads();   // every wave is done with the ring
        uint32_t tm, tn;
        tile_of32((uint32_t)nbm, (uint32_t)nbn, (uint32_t)t_full + blockIdx.x / 2, tm, tn);
        const int64_t hm0 = (int64_t)tm * GBM, hn0 = (int64_t)tn * GBN + 128 * (blockIdx.x & 1);
        if (hn0 < g.N) {   // uniform
            const int hwm = (wave >> 1) * 128, hwn = (wave & 1) * 64;
            floatx16 hacc[4][2];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int r = 0; r < 16; ++r) hacc[i][j][r] = 0.0f;
            nvw_main_loop<2, 4>(g, hm0, hn0, nk, lds, hwm, hwn, lane, hacc, 128);
            lds_barrier();   // every wave is done with the ring
            if constexpr (AROWS) {
                put_factors(hm0, row_scale(hm0));
                nvp_store<OUT_F32, 2>(g, hm0, hn0, hwm, hwn, wave, lane, alpha, hacc, lds, rowf);
            } else {
                nvp_store<OUT_F32, 2>(g, hm0, hn0, hwm, hwn, wave, lane, alpha, hacc, lds);
            }
        }
    }
}

template <int FMT, int OUT, int GM>
static int launch_one(const GemmArgs& g, const GroupArgs& q, int64_t tiles, hipStream_t s) {
    if (tiles <= 0) return 0;
    hipLaunchKernelGGL((gemm_kernel<FMT, OUT, GM>), dim3((unsigned)tiles), dim3(Fmt<FMT>::THREADS), 0, s, g, q);
    return (int)hipGetLastError();
}

// Slab-layout MXFP8 codes are read only by the aligned-record main loop and, in K-grouped
// launches, by the offset-record loop with band-wide code addressing; any other path would
// address them as row-major.  The C ABI admits slab operands only where those loops apply;
// this check keeps every launch path to the same rule.
static bool slab_ok(const GemmArgs& g, int fmt, int mode) {
    if (g.slab == 0) return true;
    if (fmt != 1 || g.K % (MX_GROUP * 64) != 0) return false;
    if ((((uintptr_t)g.a_scales | (uintptr_t)g.b_scales) % 16) != 0) return false;
    if (mode == 2) return (int64_t)GBM * g.K <= 0x7FFFFFFF;   // K-grouped: a band within one resource
    if (mode == 1 && (g.slab & 1)) return false;    // M-grouped: group bands cut the token operand
    return true;
}

// Workgroups of a persistent NVFP4 launch over `tiles` output tiles, or 0 where that kernel does
// not apply: a per-tensor scale on B and on A (or one per row of A, bf16 output only: with fp32
// output that variant spills), K a multiple of 256 and at least 512, N a
// multiple of 8 (every 16-byte chunk of a row of C lies inside C or outside it), C 16-byte aligned, a
// tile's rows of C within a 2^31-byte resource, and the global slice count of a workgroup
// within int range.
static int64_t persistent_workgroups(const GemmArgs& g, int c_dtype, int64_t tiles) {
    if (tiles >= ((int64_t)1 << 31) || g.N >= ((int64_t)1 << 34)) return 0;   // 32-bit tile arithmetic
    const int64_t es = c_dtype == 1 ? 4 : 2;
    if (g.b_rows || (g.a_rows && c_dtype == 1) || g.K % 256 != 0 || g.K < 512 || g.N % 8 != 0) return 0;
    if ((uintptr_t)g.c % 16 != 0 || (int64_t)GBM * g.N * es > 0x7FFFFFFF) return 0;
    int dev = 0, cus = 0;
    if (hipGetDevice(&dev) != hipSuccess ||
        hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus < 8)
        return 0;
    const int64_t p = tiles <= cus ? tiles : (int64_t)(cus / 8) * 8;
    if (((tiles + p - 1) / p) * (g.K / 128) >= ((int64_t)1 << 30)) return 0;
    return p;
}

template <int GM>
static int launch_fmt(int fmt, int c_dtype, const GemmArgs& g, const GroupArgs& q, int64_t tiles, hipStream_t s) {
    if constexpr (GM == 0) {
        if (fmt == 0) {
            const int64_t p = persistent_workgroups(g, c_dtype, tiles);
            if (p > 0) {
                // a last round that would leave at least half the workgroups idle is split into
                // half tiles, one per workgroup
                const int64_t r = tiles % p;
                const int64_t t_full = (r != 0 && 2 * r <= p) ? tiles - r : tiles;
                const int64_t halves = t_full < tiles ? 2 * r : 0;
                const dim3 grid((unsigned)p), block(256);
                if (g.a_rows) {   // bf16 output (persistent_workgroups)
                    hipLaunchKernelGGL((gemm_nvp_kernel<false, true>), grid, block, 0, s, g, t_full, halves);
                } else if (c_dtype == 1) {
                    hipLaunchKernelGGL((gemm_nvp_kernel<true>), grid, block, 0, s, g, t_full, halves);
                } else {
                    hipLaunchKernelGGL((gemm_nvp_kernel<false>), grid, block, 0, s, g, t_full, halves);
                }
                return (int)hipGetLastError();
            }
        }
    }
    // NVFP4: the LDS DMA kernel with scale records when every K handled is a multiple of 256
    // (known on the host unless K varies per group), with per-slice scale records otherwise
    if constexpr (GM != 2) {
        if (fmt == 0 && g.K % 256 == 0)
            return c_dtype == 1 ? launch_one<2, 1, GM>(g, q, tiles, s) : launch_one<2, 0, GM>(g, q, tiles, s);
    }
    if (fmt == 0) return c_dtype == 1 ? launch_one<3, 1, GM>(g, q, tiles, s) : launch_one<3, 0, GM>(g, q, tiles, s);
    return c_dtype == 1 ? launch_one<1, 1, GM>(g, q, tiles, s) : launch_one<1, 0, GM>(g, q, tiles, s);
}

int launch_blockscaled_gemm(int fmt, int64_t M, int64_t N, int64_t K, const uint8_t* a_codes,
                            const uint8_t* a_scales, const float* a_s_enc, const uint8_t* b_codes,
                            const uint8_t* b_scales, const float* b_s_enc, int a_rows, int b_rows, void* c,
                            int c_dtype, void* hip_stream, int slab) {
    if (M == 0 || N == 0) return 0;
    GemmArgs g{M, N, K, a_codes, a_scales, a_s_enc, b_codes, b_scales, b_s_enc, c, a_rows, b_rows, K, slab};
    if (!slab_ok(g, fmt, 0)) return (int)hipErrorInvalidValue;
    const int64_t tiles = ((M + GBM - 1) / GBM) * ((N + GBN - 1) / GBN);
    return launch_fmt<0>(fmt, c_dtype, g, GroupArgs{nullptr, 0, 0}, tiles, (hipStream_t)hip_stream);
}

int64_t grouped_gemm_workgroups(int mode, int64_t groups, int64_t M, int64_t N) {
    const int64_t nbm = (M + GBM - 1) / GBM, nbn = (N + GBN - 1) / GBN;
    if (mode == 1) return nbn * (nbm + groups) + 7 * groups;   // >= the sum of the groups' shares
    return groups * ((nbm * nbn + 7) & ~(int64_t)7);
}

int launch_blockscaled_grouped_gemm(int fmt, int mode, int64_t groups, const int64_t* offsets, int64_t M, int64_t N,
                                    int64_t K, const uint8_t* a_codes, const uint8_t* a_scales, const float* a_s_enc,
                                    const uint8_t* b_codes, const uint8_t* b_scales, const float* b_s_enc,
                                    int a_rows, int b_rows, void* c, int c_dtype, void* hip_stream, int slab) {
    if (groups == 0 || M == 0 || N == 0) return 0;
    GemmArgs g{M, N, K, a_codes, a_scales, a_s_enc, b_codes, b_scales, b_s_enc, c, a_rows, b_rows, K, slab};
    const GroupArgs q{offsets, groups, mode == 1 ? M : K};
    if (!slab_ok(g, fmt, mode)) return (int)hipErrorInvalidValue;
    const int64_t tiles = grouped_gemm_workgroups(mode, groups, M, N);
    hipStream_t s = (hipStream_t)hip_stream;
    if (mode == 1) return launch_fmt<1>(fmt, c_dtype, g, q, tiles, s);
    if (g.slab != 0)   // MXFP8 (slab_ok): the K-grouped kernel for slab-layout operands
        return c_dtype == 1 ? launch_one<1, 1, 3>(g, q, tiles, s) : launch_one<1, 0, 3>(g, q, tiles, s);
    return launch_fmt<2>(fmt, c_dtype, g, q, tiles, s);
}

}  // namespace bsq
