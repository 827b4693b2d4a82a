// matvec.hip -- products of a few bf16 tokens with NVFP4 weights: y[m][n] = sum_k x[m][k] W[n][k], and the
// gated pair h = act(x Wg^T) (x Wu^T), the form of a linear layer and of a gated feed-forward block
// that serves single tokens.
//
// Bound by reading the weights, 9/16 byte each, which have no reuse beyond the tokens of the call: what
// matters is how many bytes are in flight.  A wave takes 16 weight rows by 256 elements at a time, whole
// 128-byte lines of each row, two such chunks loaded before the first is used, and 16 waves share a CU
// (72 KiB of weights in flight); K is split over the 4 to 16 waves of a workgroup and joined in LDS.
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
constexpr int MV_CHUNK = 256;   // K elements that a wave takes at a time
constexpr int MV_WAVES = 16;    // at most

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

// One lane's 64 elements of a weight row: their codes and the bytes of their 4 block scales.
struct MvPiece {
    uint4 lo, hi;
    uint32_t scales;
};
struct __attribute__((packed, aligned(8))) MvCodes16 { uint32_t w[4]; };   // rows are 8-byte aligned (K % 16 == 0)
struct __attribute__((packed, aligned(1))) MvScales4 { uint32_t w; };

// The piece of row n from element k on.  FULL: all of it lies inside K; otherwise what lies past K is 0.
template <bool FULL>
__device__ __forceinline__ MvPiece mv_load(const MvOperand& w, int64_t n, int64_t K, int64_t k) {
    const uint8_t* c = w.codes + n * (K / 2) + k / 2;
    const uint8_t* s = w.scales + n * (K / 16) + k / 16;
    if constexpr (FULL) {
        const MvCodes16 a = *(const MvCodes16*)c, b = *(const MvCodes16*)(c + 16);
        return {make_uint4(a.w[0], a.w[1], a.w[2], a.w[3]), make_uint4(b.w[0], b.w[1], b.w[2], b.w[3]),
                ((const MvScales4*)s)->w};
    }
    uint2 v[4];
    uint32_t sc = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        v[b] = make_uint2(0, 0);
        if (k + 16 * b < K) {
            v[b] = *(const uint2*)(c + 8 * b);
            sc |= (uint32_t)s[b] << (8 * b);
        }
    }
    return {make_uint4(v[0].x, v[0].y, v[1].x, v[1].y), make_uint4(v[2].x, v[2].y, v[3].x, v[3].y), sc};
}

// Eight elements of token row x from k on (zeros past K unless FULL).
template <bool FULL>
__device__ __forceinline__ bf16x8_t mv_token(const uint16_t* x, int64_t K, int64_t k) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (FULL || k < K) v = *(const uint4*)(x + k);
    return __builtin_bit_cast(bf16x8_t, v);
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

template <int I>
__device__ __forceinline__ uint32_t mv_word(const MvPiece& p) {
    const uint4& q = I < 4 ? p.lo : p.hi;
    if constexpr (I % 4 == 0) return q.x;
    else if constexpr (I % 4 == 1) return q.y;
    else if constexpr (I % 4 == 2) return q.z;
    else return q.w;
}

// MFMA operand layout (v_mfma_f32_16x16x32_bf16): lane l holds row l % 16 of A (tokens) and of B (weight
// rows), 8 elements each; accumulator r of lane l is token 4 (l / 16) + r, weight row l % 16.  The order
// of K inside a chunk is free as long as both operands use the same: lane group g = l / 16 takes the
// chunk's elements 64g .. 64g+63, which are 32 consecutive code bytes, in 8 MFMA steps of 8.
template <bool FULL, int MT, int NW>
__device__ __forceinline__ void mv_step(const MvPiece (&p)[NW], const uint16_t* const (&x)[MT], int64_t K, int64_t k,
                                        floatx4 (&acc)[NW][MT]) {
    static_for<0, 8>([&](auto j_c) {
        constexpr int J = decltype(j_c)::value;
        bf16x8_t xv[MT];
#pragma unroll
        for (int t = 0; t < MT; ++t) xv[t] = mv_token<FULL>(x[t], K, k + 8 * J);
#pragma unroll
        for (int o = 0; o < NW; ++o) {
            const bf16x8_t b = mv_dequant(mv_word<J>(p[o]), __builtin_amdgcn_cvt_f32_fp8((int)p[o].scales, J / 2));
#pragma unroll
            for (int t = 0; t < MT; ++t)
                acc[o][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv[t], b, acc[o][t], 0, 0, 0);
        }
    });
}

// A workgroup: 16 MT tokens by 16 weight rows, its waves dealt the chunks of K in turn.  Lanes of rows past
// N and of tokens past M repeat the last one (their outputs are not stored).
template <int MT, bool GATED, int ACT>
__global__ __launch_bounds__(64 * MV_WAVES) void matvec_kernel(MvArgs a) {
    constexpr int NW = GATED ? 2 : 1;
    constexpr int WAVES = MT * NW > 2 ? MV_WAVES / 2 : MV_WAVES;   // at most (launch_mv)
    __shared__ float red[WAVES][NW][MT * 16][MV_ROWS + 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int r16 = lane & 15, g = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * MV_ROWS, m0 = (int64_t)blockIdx.y * (16 * MT);
    const int64_t row = n0 + r16 < a.N ? n0 + r16 : a.N - 1;
    const uint16_t* x[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int64_t m = m0 + 16 * t + r16;
        x[t] = a.x + (m < a.M ? m : a.M - 1) * a.ldx;
    }
    floatx4 acc[NW][MT];
#pragma unroll
    for (int o = 0; o < NW; ++o)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[o][t] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    const int64_t step = (int64_t)waves * MV_CHUNK;
    int64_t c = (int64_t)wave * MV_CHUNK;
    for (; c + step + MV_CHUNK <= a.K; c += 2 * step) {   // two whole chunks, both loaded first
        const int64_t k = c + 64 * g;
        MvPiece p[2][NW];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int o = 0; o < NW; ++o) p[u][o] = mv_load<true>(a.w[o], row, a.K, k + u * step);
        mv_step<true>(p[0], x, a.K, k, acc);
        mv_step<true>(p[1], x, a.K, k + step, acc);
    }
    for (; c < a.K; c += step) {
        const int64_t k = c + 64 * g;
        MvPiece p[NW];
        if (c + MV_CHUNK <= a.K) {
#pragma unroll
            for (int o = 0; o < NW; ++o) p[o] = mv_load<true>(a.w[o], row, a.K, k);
            mv_step<true>(p, x, a.K, k, acc);
        } else {
#pragma unroll
            for (int o = 0; o < NW; ++o) p[o] = mv_load<false>(a.w[o], row, a.K, k);
            mv_step<false>(p, x, a.K, k, acc);
        }
    }
#pragma unroll
    for (int o = 0; o < NW; ++o)
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) red[wave][o][16 * t + 4 * g + r][r16] = acc[o][t][r];
    __syncthreads();
    for (int i = threadIdx.x; i < MT * 16 * MV_ROWS; i += blockDim.x) {
        const int mt = i / MV_ROWS, nt = i % MV_ROWS;
        const int64_t m = m0 + mt, n = n0 + nt;
        if (m >= a.M || n >= a.N) continue;
        float v[NW];
#pragma unroll
        for (int o = 0; o < NW; ++o) {
            float s = 0.0f;
            for (int w = 0; w < waves; ++w) s += red[w][o][mt][nt];
            v[o] = s / a.w[o].s_enc[a.rows ? n : 0];
        }
        float y = v[0];
        if constexpr (GATED) y = act_value<ACT>(v[0]) * v[NW - 1];
        if (a.y_f32) ((float*)a.y)[m * a.N + n] = y;
        else ((uint16_t*)a.y)[m * a.N + n] = (uint16_t)bf16x2_rne(y, 0.0f);
    }
}

// Waves of a workgroup: as many as let every workgroup of the launch be resident at once (16 waves on each
// of 256 CUs), at least 4, and no more than there are chunks of K.
template <int MT, bool GATED, int ACT>
static int launch_mt(const MvArgs& a, hipStream_t s) {
    const unsigned nb = (unsigned)((a.N + MV_ROWS - 1) / MV_ROWS), mb = (unsigned)((a.M + 16 * MT - 1) / (16 * MT));
    const int64_t chunks = (a.K + MV_CHUNK - 1) / MV_CHUNK;
    int waves = MT * (GATED ? 2 : 1) > 2 ? MV_WAVES / 2 : MV_WAVES;
    while (waves > 4 && (int64_t)waves * nb * mb > 256 * 16) waves /= 2;
    while (waves > 1 && waves / 2 >= chunks) waves /= 2;
    hipLaunchKernelGGL((matvec_kernel<MT, GATED, ACT>), dim3(nb, mb), dim3(64 * waves), 0, s, a);
    return (int)hipGetLastError();
}

template <bool GATED, int ACT>
static int launch_mv(const MvArgs& a, hipStream_t s) {
    if (a.M <= 16) return launch_mt<1, GATED, ACT>(a, s);
    if (a.M <= 32) return launch_mt<2, GATED, ACT>(a, s);
    return launch_mt<4, GATED, ACT>(a, s);
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
