// gated_small.hip -- the gated feed-forward products (gated.hip states them) for sizes whose 256 x 256 tiles
// would leave most of the chip idle.
//
// A workgroup computes 64 x 64 of the product: its 4 waves each take the whole tile over a quarter of the K
// slices, straight from memory to registers in the MFMA's layout, and their sums are joined in LDS, where
// the elementwise part finds them row-major.  Such a problem is bound by latency: a wave asks for its
// next slice before it computes the current one, and no wave waits for another before the join.
#include "gated.hpp"
#include "launch.hpp"

namespace bsq {

constexpr int ST = 64;              // rows and B rows of a tile
constexpr int SWAVES = 4;
constexpr int SRS = ST * 4 + 16;    // bytes between rows in LDS
constexpr int small_k(bool nv) { return nv ? 128 : 64; }   // K elements of a slice

typedef unsigned int u32x2s __attribute__((ext_vector_type(2)));

// One fragment's 32 rows of a slice: 128 elements of NVFP4 (lane (row, kh): 64 of them and 4 scales) or 64 of
// MXFP8 (an MFMA step).
template <bool NV>
struct SmallFrag {
    u32x4s c[2];
    uint32_t s[NV ? 2 : 1];
};

// Where a fragment's rows lie.  Rows and K past the operand read as zero.
struct SmallRows {
    __amdgpu_buffer_rsrc_t codes, scales;
    uint32_t row;         // the lane's row in the resources
    uint32_t slab_rows;   // slab layout: rows of the band; 0 otherwise
};

// 32 rows from r0 on of an operand of R rows.
template <bool NV>
__device__ __forceinline__ SmallRows small_rows(const uint8_t* codes, const uint8_t* scales, int64_t r0, int64_t R,
                                                int64_t K, bool slab, int lane) {
    const int64_t rb = NV ? K / 2 : K, sb = NV ? K / 16 : K / 32, n = tile_rows(R - r0, 32);
    SmallRows q;
    const int64_t band = slab ? r0 & ~(int64_t)255 : r0, bn = slab ? tile_rows(R - band, 256) : n;
    q.codes = make_rsrc(codes + band * rb, (R > r0 ? bn : 0) * rb);
    q.scales = make_rsrc(scales + r0 * sb, n * sb);
    q.row = (uint32_t)(lane & 31);
    q.slab_rows = slab ? (uint32_t)bn : 0u;
    if (slab) q.row += (uint32_t)(r0 - band);
    return q;
}

template <bool NV>
__device__ __forceinline__ void small_load(const SmallRows& q, uint32_t K, uint32_t k0, int lane, SmallFrag<NV>& f) {
    const uint32_t kh = (uint32_t)lane >> 5, srow = (uint32_t)(lane & 31);
    if constexpr (NV) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {   // 32 elements and their two scales
            const uint32_t k = k0 + 64 * kh + 32 * h;
            f.c[h] = __builtin_amdgcn_raw_buffer_load_b128(q.codes, (int)(k < K ? q.row * (K / 2) + k / 2 : OOB), 0, 0);
            f.s[h] = __builtin_amdgcn_raw_buffer_load_b16(q.scales, (int)(k < K ? srow * (K / 16) + k / 16 : OOB), 0, 0);
        }
    } else {
#pragma unroll
        for (int b = 0; b < 2; ++b) {   // elements 16 kh .. and 32 + 16 kh ..; the scale of block kh
            const uint32_t k = k0 + 32 * b + 16 * kh;
            const uint32_t at = q.slab_rows ? (k / 64) * (q.slab_rows * 64) + q.row * 64 + k % 64 : q.row * K + k;
            // in the slab layout a row past the band would be another slab's
            const bool in = k < K && (!q.slab_rows || q.row < q.slab_rows);
            f.c[b] = __builtin_amdgcn_raw_buffer_load_b128(q.codes, (int)(in ? at : OOB), 0, 0);
        }
        const uint32_t k = k0 + 32 * kh;
        f.s[0] = __builtin_amdgcn_raw_buffer_load_b8(q.scales, (int)(k < K ? srow * (K / 32) + k / 32 : OOB), 0, 0);
    }
}

template <bool NV>
__device__ __forceinline__ void small_use(const SmallFrag<NV> (&a)[2], const SmallFrag<NV> (&b)[2], floatx16 (&acc)[2][2]) {
    if constexpr (NV) {
        static_for<0, 8>([&](auto s_c) {
            constexpr int S = decltype(s_c)::value;
            half8_t av[2], bv[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                av[i] = nv_dequant(a[i].c[S / 4][S % 4], nv_scale(a[i].s[0] | a[i].s[1] << 16, S >> 1));
                bv[i] = nv_dequant(b[i].c[S / 4][S % 4], nv_scale(b[i].s[0] | b[i].s[1] << 16, S >> 1));
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(bv[j], av[i], acc[i][j], 0, 0, 0);
        });
    } else {
        intx8 av[2], bv[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                av[i][e] = (int)a[i].c[0][e];
                av[i][4 + e] = (int)a[i].c[1][e];
                bv[i][e] = (int)b[i].c[0][e];
                bv[i][4 + e] = (int)b[i].c[1][e];
            }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(bv[j], av[i], acc[i][j], 0, 0, 0,
                                                                             (int)b[j].s[0], 0, (int)a[i].s[0]);
    }
}

// The tile's product, joined: sums(row, column) is a part's float in LDS.  ar, br: the two fragments of A and B.
template <bool NV>
__device__ __forceinline__ void small_product(const SmallRows (&ar)[2], const SmallRows (&br)[2], int64_t K, uint8_t* lds,
                                              int wave, int lane) {
    constexpr int SK = small_k(NV);
    floatx16 acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
    SmallFrag<NV> a[2][2], b[2][2];   // [slice parity][fragment]
    auto load = [&](int64_t s, auto p_c) {
        constexpr int P = decltype(p_c)::value;
        const uint32_t k0 = (uint32_t)(s * SK);   // past K: nothing is read
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            small_load<NV>(ar[i], (uint32_t)K, k0, lane, a[P][i]);
            small_load<NV>(br[i], (uint32_t)K, k0, lane, b[P][i]);
        }
    };
    const int64_t slices = (K + SK - 1) / SK;
    using P0 = std::integral_constant<int, 0>;
    using P1 = std::integral_constant<int, 1>;
    if (wave < slices) load(wave, P0{});
    for (int64_t s = wave; s < slices; s += 2 * SWAVES) {
        load(s + SWAVES, P1{});
        small_use<NV>(a[0], b[0], acc);
        if (s + SWAVES >= slices) break;
        load(s + 2 * SWAVES, P0{});
        small_use<NV>(a[1], b[1], acc);
    }
    const int frow = lane & 31, kh = lane >> 5;
    uint8_t* mine = lds + wave * ST * SRS;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *(float4*)(mine + (32 * i + frow) * SRS + 4 * (32 * j + 8 * q + 4 * kh)) =
                    make_float4(acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]);
    __syncthreads();
}

// Eight columns' sums over the parts.
__device__ __forceinline__ void small_sum(const uint8_t* lds, int row, int col, float (&v)[8]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float4 s = *(const float4*)(lds + row * SRS + 4 * col + 16 * h);
#pragma unroll
        for (int w = 1; w < SWAVES; ++w) {
            const float4 t = *(const float4*)(lds + (w * ST + row) * SRS + 4 * col + 16 * h);
            s.x += t.x; s.y += t.y; s.z += t.z; s.w += t.w;
        }
        v[4 * h] = s.x; v[4 * h + 1] = s.y; v[4 * h + 2] = s.z; v[4 * h + 3] = s.w;
    }
}

// Eight bf16 values to a row that has `left` elements from p on.
__device__ __forceinline__ void small_store(uint16_t* p, int64_t left, u32x4s v) {
    if (left >= 8) {
        store_any(p, v);
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < left) p[e] = (uint16_t)(v[e / 2] >> (16 * (e & 1)));
}

__device__ __forceinline__ u32x4s small_load8(const uint16_t* p, int64_t left) {
    if (left >= 8) return load_any(p);
    u32x4s v = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < left) v[e / 2] |= (uint32_t)p[e] << (16 * (e & 1));
    return v;
}

__device__ __forceinline__ u32x4s small_pack(const float (&v)[8]) {
    return u32x4s{bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]), bf16x2_rne(v[4], v[5]), bf16x2_rne(v[6], v[7])};
}

// The tile of this workgroup, column blocks first; workgroups go to the 8 XCDs in turn, so each XCD is given a
// contiguous range of tiles.
__device__ __forceinline__ void small_tile(int64_t nbn, int64_t& tm, int64_t& tn) {
    const uint32_t t8 = gridDim.x & ~7u, id = blockIdx.x;
    const int64_t t = id < t8 ? (id & 7u) * (t8 >> 3) + (id >> 3) : id;
    tm = t / nbn;
    tn = t % nbn;
}

// Forward: 64 tokens by 32 columns of h; the B fragments are 32 rows of gate and 32 of up.  A thread takes
// 8 columns of a row.  Output factors as gated_factors has them.
template <bool NV>
__global__ __launch_bounds__(64 * SWAVES, 2) void gated_small_kernel(GatedArgs g) {
    __shared__ __attribute__((aligned(16))) uint8_t lds[SWAVES * ST * SRS];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int64_t nbn = (g.N + ST / 2 - 1) / (ST / 2);
    int64_t tm, tn;
    small_tile(nbn, tm, tn);
    const int64_t m0 = tm * ST, n0 = tn * (ST / 2);
    const SmallRows ar[2] = {small_rows<NV>(g.a_codes, g.a_scales, m0, g.M, g.K, g.slab & 1, lane),
                             small_rows<NV>(g.a_codes, g.a_scales, m0 + 32, g.M, g.K, g.slab & 1, lane)};
    const SmallRows br[2] = {small_rows<NV>(g.b_codes, g.b_scales, n0, g.N, g.K, g.slab & 2, lane),
                             small_rows<NV>(g.u_codes, g.u_scales, n0, g.N, g.K, g.slab & 2, lane)};
    const int row = threadIdx.x >> 2, col = 8 * (threadIdx.x & 3);
    const int64_t m = m0 + row, n = n0 + col, left = g.N - n;
    const bool in = m < g.M && left > 0;
    [[maybe_unused]] double sa = 1.0, sg[8], su[8];
    if constexpr (NV) {   // fetched before the product
        if (in) {
            sa = (double)g.a_s_enc[g.a_rows ? m : 0];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int64_t c = g.b_rows ? (e < left ? n + e : n) : 0;
                sg[e] = (double)g.b_s_enc[c];
                su[e] = (double)g.u_s_enc[c];
            }
        }
    }
    small_product<NV>(ar, br, g.K, lds, wave, lane);
    if (!in) return;
    float gv[8], uv[8], hv[8];
    small_sum(lds, row, col, gv);
    small_sum(lds, row, 32 + col, uv);
    if constexpr (NV) {
        const float fr = g.a_rows ? (float)(1.0 / sa) : 1.0f;
        const double s1 = g.a_rows ? 1.0 : sa;
        float fg = 0.0f, fu = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (e == 0 || g.b_rows) {
                fg = (float)(1.0 / (s1 * sg[e]));
                fu = (float)(1.0 / (s1 * su[e]));
            }
            gv[e] *= fr * fg;
            uv[e] *= fr * fu;
        }
    }
    with_act(g.act, [&](auto act_c) {
#pragma unroll
        for (int e = 0; e < 8; ++e) hv[e] = act_value<decltype(act_c)::value>(gv[e]) * uv[e];
    });
    small_store((uint16_t*)g.c + m * g.N + n, left, small_pack(hv));
    if (g.gate_up) {
        small_store(g.gate_up + m * 2 * g.N + n, left, small_pack(gv));
        small_store(g.gate_up + m * 2 * g.N + g.N + n, left, small_pack(uv));
    }
}

// Backward: 64 x 64 of dh; a thread takes 16 columns of a row, their gate and up fetched before the product.
// Output factors as tile_factors has them.
template <bool NV>
__global__ __launch_bounds__(64 * SWAVES, 2) void gated_backward_small_kernel(GatedBackArgs g) {
    __shared__ __attribute__((aligned(16))) uint8_t lds[SWAVES * ST * SRS];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int64_t nbn = (g.N + ST - 1) / ST;
    int64_t tm, tn;
    small_tile(nbn, tm, tn);
    const int64_t m0 = tm * ST, n0 = tn * ST;
    SmallRows ar[2], br[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        ar[i] = small_rows<NV>(g.a_codes, g.a_scales, m0 + 32 * i, g.M, g.K, g.slab & 1, lane);
        br[i] = small_rows<NV>(g.b_codes, g.b_scales, n0 + 32 * i, g.N, g.K, g.slab & 2, lane);
    }
    const int row = threadIdx.x >> 2;
    const int64_t m = m0 + row, at = m * 2 * g.N;
    u32x4s gate[2], up[2];
    int64_t n[2], left[2];
    [[maybe_unused]] double sa = 1.0, sb[2][8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        n[h] = n0 + 8 * (threadIdx.x & 3) + 32 * h;
        left[h] = m < g.M ? g.N - n[h] : 0;
        gate[h] = up[h] = u32x4s{0, 0, 0, 0};
        if (left[h] > 0) {
            gate[h] = small_load8(g.gate_up + at + n[h], left[h]);
            up[h] = small_load8(g.gate_up + at + g.N + n[h], left[h]);
        }
        if constexpr (NV) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                sb[h][e] = 1.0;
                if (e < left[h]) sb[h][e] = (double)g.b_s_enc[g.b_rows ? n[h] + e : 0];
            }
        }
    }
    if constexpr (NV) sa = (double)g.a_s_enc[g.a_rows ? (m < g.M ? m : g.M - 1) : 0];
    small_product<NV>(ar, br, g.K, lds, wave, lane);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (left[h] <= 0) continue;
        float dh[8];
        small_sum(lds, row, (int)(n[h] - n0), dh);
        if constexpr (NV) {
            float f = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (g.a_rows && g.b_rows) f = (float)(1.0 / sa) * (float)(1.0 / sb[h][e]);
                else if (e == 0 || g.b_rows) f = (float)(1.0 / (sa * sb[h][e]));
                dh[e] *= f;
            }
        }
        u32x4s dg, du;
        with_act(g.act, [&](auto act_c) { gated_grads<decltype(act_c)::value>(dh, gate[h], up[h], dg, du); });
        small_store((uint16_t*)g.c + at + n[h], left[h], dg);
        small_store((uint16_t*)g.c + at + g.N + n[h], left[h], du);
    }
}

int launch_gated_small(int fmt, const GatedArgs& g, void* hip_stream) {
    const int64_t tiles = ((g.M + ST - 1) / ST) * ((g.N + ST / 2 - 1) / (ST / 2));
    const dim3 grid((unsigned)tiles), block(64 * SWAVES);
    if (fmt == 0) hipLaunchKernelGGL((gated_small_kernel<true>), grid, block, 0, (hipStream_t)hip_stream, g);
    else hipLaunchKernelGGL((gated_small_kernel<false>), grid, block, 0, (hipStream_t)hip_stream, g);
    return (int)hipGetLastError();
}

int launch_gated_backward_small(int fmt, const GatedBackArgs& g, void* hip_stream) {
    const int64_t tiles = ((g.M + ST - 1) / ST) * ((g.N + ST - 1) / ST);
    const dim3 grid((unsigned)tiles), block(64 * SWAVES);
    if (fmt == 0) hipLaunchKernelGGL((gated_backward_small_kernel<true>), grid, block, 0, (hipStream_t)hip_stream, g);
    else hipLaunchKernelGGL((gated_backward_small_kernel<false>), grid, block, 0, (hipStream_t)hip_stream, g);
    return (int)hipGetLastError();
}

}  // namespace bsq
