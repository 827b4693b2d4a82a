// matvec.hip -- products of a few bf16 tokens with NVFP4 weights: y[m][n] = sum_k x[m][k] W[n][k], and the
// gated pair h = act(x Wg^T) (x Wu^T), the form of a linear layer and of a gated feed-forward block
// that serves single tokens.
//
// Bound by reading the weights, 9/16 byte each, which have no reuse beyond the tokens of the call.
// A weight E2M1 * E4M3 has at most 6 significant bits and lies in [2^-10, 2688], so it is exact in
// bf16; x is bf16 as it comes; the bf16 MFMA multiplies exactly and accumulates in binary32.  The only
// roundings are those sums, one division by the tensor (or row) scale and the output's.
#include "activation.hpp"
#include "launch.hpp"

namespace bsq {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef float floatx2 __attribute__((ext_vector_type(2)));

constexpr int MV_ROWS = 16;     // weight rows of a workgroup (of gate and of up when gated)
constexpr int MV_CHUNK = 128;   // K elements that a wave takes at a time
constexpr int MV_WAVES = 8;

struct MvOperand {
    const uint8_t* codes;
    const uint8_t* scales;
    const float* s_enc;
};

struct MvArgs {
    const uint16_t* x;
    int64_t ldx;          // elements between tokens
    int64_t M, N, K;
    MvOperand w[2];       // the weights; gate and up
    int rows;             // the scales are one per row
    void* y;              // [M][N], bf16 or fp32
    int y_f32;
};

// Bytes of the weight row `n`'s codes of one lane's 32 elements and their two block scales, as
// binary32; what lies past K is 0.
struct MvPiece {
    uint4 codes;
    float s0, s1;
};

__device__ __forceinline__ float e4m3_value(uint32_t b) { return __builtin_amdgcn_cvt_f32_fp8((int)b, 0); }

__device__ __forceinline__ MvPiece mv_load(const MvOperand& w, int64_t n, int64_t N, int64_t K, int64_t k) {
    MvPiece p{make_uint4(0, 0, 0, 0), 0.0f, 0.0f};
    if (n < N && k < K) {
        const uint8_t* c = w.codes + n * (K / 2) + k / 2;   // rows are 8-byte aligned (K % 16 == 0)
        const uint8_t* s = w.scales + n * (K / 16) + k / 16;
        const uint2 lo = *(const uint2*)c;
        p.codes.x = lo.x;
        p.codes.y = lo.y;
        p.s0 = e4m3_value(s[0]);
        if (k + 16 < K) {
            const uint2 hi = *(const uint2*)(c + 8);
            p.codes.z = hi.x;
            p.codes.w = hi.y;
            p.s1 = e4m3_value(s[1]);
        }
    }
    return p;
}

// Eight codes times their block's scale, in bf16 (exact).
__device__ __forceinline__ bf16x8_t mv_dequant(uint32_t w, float s) {
    bf16x8_t r;
    static_for<0, 4>([&](auto i_c) {
        constexpr int I = decltype(i_c)::value;
        const floatx2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, I);
        r[2 * I] = (__bf16)(v[0] * s);
        r[2 * I + 1] = (__bf16)(v[1] * s);
    });
    return r;
}

// MFMA operand layout (v_mfma_f32_16x16x32_bf16): lane l holds row l % 16 of A (tokens) and of B (weight
// rows), 8 elements each; accumulator r of lane l is token 4 (l / 16) + r, weight row l % 16.  The order
// of K inside a chunk is free as long as both operands use the same: lane group g = l / 16 takes the
// chunk's elements 32g .. 32g+31, which are 16 consecutive code bytes, in 4 MFMA steps of 8.
template <int MT, bool GATED, int ACT>
__global__ __launch_bounds__(64 * MV_WAVES) void matvec_kernel(MvArgs a) {
    constexpr int NW = GATED ? 2 : 1;
    __shared__ float red[MV_WAVES][NW][MT * 16][MV_ROWS + 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r16 = lane & 15, g = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * MV_ROWS, m0 = (int64_t)blockIdx.y * (16 * MT);
    floatx4 acc[NW][MT];
#pragma unroll
    for (int o = 0; o < NW; ++o)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[o][t] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t c0 = (int64_t)wave * MV_CHUNK; c0 < a.K; c0 += MV_WAVES * MV_CHUNK) {
        const int64_t k = c0 + 32 * g;
        MvPiece p[NW];
#pragma unroll
        for (int o = 0; o < NW; ++o) p[o] = mv_load(a.w[o], n0 + r16, a.N, a.K, k);
        uint4 xv[MT][4];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const int64_t m = m0 + 16 * t + r16;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                xv[t][j] = (m < a.M && k + 8 * j < a.K) ? *(const uint4*)(a.x + m * a.ldx + k + 8 * j)
                                                        : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int o = 0; o < NW; ++o) {
            const bf16x8_t b[4] = {mv_dequant(p[o].codes.x, p[o].s0), mv_dequant(p[o].codes.y, p[o].s0),
                                   mv_dequant(p[o].codes.z, p[o].s1), mv_dequant(p[o].codes.w, p[o].s1)};
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[o][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, xv[t][j]), b[j],
                                                                         acc[o][t], 0, 0, 0);
        }
    }
#pragma unroll
    for (int o = 0; o < NW; ++o)
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) red[wave][o][16 * t + 4 * g + r][r16] = acc[o][t][r];
    __syncthreads();
    for (int i = threadIdx.x; i < MT * 16 * MV_ROWS; i += 64 * MV_WAVES) {
        const int mt = i / MV_ROWS, nt = i % MV_ROWS;
        const int64_t m = m0 + mt, n = n0 + nt;
        if (m >= a.M || n >= a.N) continue;
        float v[NW];
#pragma unroll
        for (int o = 0; o < NW; ++o) {
            float s = 0.0f;
            for (int w = 0; w < MV_WAVES; ++w) s += red[w][o][mt][nt];
            v[o] = s / a.w[o].s_enc[a.rows ? n : 0];
        }
        float y = v[0];
        if constexpr (GATED) y = act_value<ACT>(v[0]) * v[NW - 1];
        if (a.y_f32) ((float*)a.y)[m * a.N + n] = y;
        else ((uint16_t*)a.y)[m * a.N + n] = (uint16_t)bf16x2_rne(y, 0.0f);
    }
}

template <bool GATED, int ACT>
static int launch_mv(const MvArgs& a, hipStream_t s) {
    const unsigned nb = (unsigned)((a.N + MV_ROWS - 1) / MV_ROWS);
    const dim3 block(64 * MV_WAVES);
    if (a.M <= 16) {
        hipLaunchKernelGGL((matvec_kernel<1, GATED, ACT>), dim3(nb, 1), block, 0, s, a);
    } else {
        hipLaunchKernelGGL((matvec_kernel<2, GATED, ACT>), dim3(nb, (unsigned)((a.M + 31) / 32)), block, 0, s, a);
    }
    return (int)hipGetLastError();
}

int launch_nvfp4_matvec(int act, const void* x, int64_t ldx, int64_t M, int64_t N, int64_t K, const uint8_t* w_codes,
                        const uint8_t* w_scales, const float* w_s_enc, const uint8_t* up_codes,
                        const uint8_t* up_scales, const float* up_s_enc, int rows, void* y, int y_f32,
                        void* hip_stream) {
    if (M == 0 || N == 0) return 0;
    const MvArgs a{(const uint16_t*)x, ldx, M, N, K, {{w_codes, w_scales, w_s_enc}, {up_codes, up_scales, up_s_enc}},
                   rows, y, y_f32};
    hipStream_t s = (hipStream_t)hip_stream;
    if (act < 0) return launch_mv<false, 0>(a, s);
    if (act == 0) return launch_mv<true, 0>(a, s);
    if (act == 1) return launch_mv<true, 1>(a, s);
    return launch_mv<true, 2>(a, s);
}

}  // namespace bsq
