// matvec.hip -- products of a few bf16 tokens with NVFP4 weights: y[m][n] = sum_k x[m][k] W[n][k], and the
// gated pair h = act(x Wg^T) (x Wu^T), the form of a linear layer and of a gated feed-forward block
// that serves single tokens.
//
// Bound by reading the weights, 9/16 byte each, which have no reuse beyond the tokens of the call: what
// matters is how many bytes are in flight.  A wave takes 16 weight rows by 256 elements at a time (a
// chunk), whole 128-byte lines of each row, and loads the next chunks before it uses the current one.  K
// is split over the waves of a workgroup and joined in LDS.
//
// x is bf16 as it comes, and so is every weight: E2M1 * 2^-7, or E2M1 * E4M3, which has at most 6
// significant bits and lies in [2^-10, 2688].  The bf16 MFMA multiplies exactly and accumulates in
// binary32.  The only roundings are those sums, a block's scale where it is applied to a block's sum, one
// division by the tensor (or row) scale and the output's.
//
// us in a graph, weights rotating through 800 MB (the same weights again and again, in part from the caches, in
// brackets); a large copy on this card moves 4.7 TB/s:
//   1 token    4096 x 4096 5.1 (4.3), 4096 x 14336 9.5 (8.4), 16384 x 16384 33.7 (30.3): 3.5 and 4.5 TB/s of
//              weights in the last two; gated 14336 x 4096 16.0 (15.2), 4.1 TB/s
//   4 tokens   4096 x 4096 6.8 (6.0), 4096 x 14336 14.1 (12.3)
//   8          4096 x 4096 7.7 (6.5), 4096 x 14336 15.4 (13.9), gated 14336 x 4096 22.4 (19.3)
//   16         4096 x 4096 8.6 (7.6), 4096 x 14336 17.5 (16.3), gated 14336 x 4096 23.9 (21.1)
//   64         4096 x 4096 13.0 (11.7), gated 14336 x 8192 62 (56)
// The smallest, 1 x 256 x 256, takes 2.2.  What is left for one token is the way in and out: the launch, the
// first trip to memory, the join.  Several are held back by one workgroup of 8 waves per CU (its tokens take
// 132 KiB of LDS from 16 on) that meets at a barrier after every chunk.
#include "activation.hpp"
#include "launch.hpp"

namespace bsq {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef float floatx2 __attribute__((ext_vector_type(2)));

constexpr int MV_ROWS = 16;     // weight rows of a wave (of gate and of up when gated)
constexpr int MV_CHUNK = 256;   // K elements that a wave takes at a time
constexpr int MV_CUS = 256;

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
    int act;
    int wr;               // 16-row blocks of a workgroup; its waves are wr times as many as parts of K
};

// One lane's 64 elements of a weight row: their codes and the bytes of their 4 block scales.
struct MvPiece {
    uint4 lo, hi;
    uint32_t scales;
};

// How a lane's pieces lie in its row.
constexpr int MV_ALIGNED = 0;   // K a multiple of 64: a piece lies inside K or outside
constexpr int MV_SHIFTED = 1;   // any other K above 64: the row's last 64 elements stand in for a piece that K ends in
constexpr int MV_BLOCKS = 2;    // K below 64: each 16-element block is loaded for itself

// A wave's 16 rows of a weight.  Rows past N read as zero codes (the buffer's range) and the last row's scales.
struct MvRsrc {
    __amdgpu_buffer_rsrc_t codes, scales;
    const uint8_t* row_scales;   // of the lane's row
};

__device__ __forceinline__ MvRsrc mv_rsrc(const MvOperand& w, int64_t n0, int64_t N, int64_t K, int r16) {
    const int64_t rows = N - n0 < MV_ROWS ? N - n0 : MV_ROWS;   // K < 2^24: below 2^27 bytes
    const int n = rows < 0 ? 0 : (int)rows;
    const int64_t row = n0 + r16 < N ? n0 + r16 : N - 1;
    return {__builtin_amdgcn_make_buffer_rsrc((void*)(w.codes + n0 * (K / 2)), (short)0, n * (int)(K / 2), 0x00020000),
            __builtin_amdgcn_make_buffer_rsrc((void*)(w.scales + n0 * (K / 16)), (short)0, n * (int)(K / 16), 0x00020000),
            w.scales + row * (K / 16)};
}

constexpr uint32_t MV_OOB = 0x80000000u;   // an offset beyond every resource

typedef unsigned int mv_u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int mv_u32x2 __attribute__((ext_vector_type(2)));
struct __attribute__((packed, aligned(1))) MvScales4 { uint32_t w; };

// The piece of row r from element k on.  What lies past K is 0, with MV_SHIFTED after mv_fix.
template <int LOAD>
__device__ __forceinline__ MvPiece mv_load(const MvRsrc& w, uint32_t r, uint32_t K, uint32_t k) {
    if constexpr (LOAD == MV_BLOCKS) {
        mv_u32x2 v[4];
        uint32_t sc[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const uint32_t kb = k + 16 * b;
            v[b] = __builtin_amdgcn_raw_buffer_load_b64(w.codes, (int)(kb < K ? r * (K / 2) + kb / 2 : MV_OOB), 0, 0);
            sc[b] = __builtin_amdgcn_raw_buffer_load_b8(w.scales, (int)(kb < K ? r * (K / 16) + kb / 16 : MV_OOB), 0, 0);
        }
        return {make_uint4(v[0].x, v[0].y, v[1].x, v[1].y), make_uint4(v[2].x, v[2].y, v[3].x, v[3].y),
                sc[0] | sc[1] << 8 | sc[2] << 16 | sc[3] << 24};
    }
    uint32_t c, s;
    if constexpr (LOAD == MV_SHIFTED) {
        const uint32_t kk = k < K - 64 ? k : K - 64;
        c = r * (K / 2) + kk / 2;
        s = ((const MvScales4*)(w.row_scales + kk / 16))->w;
    } else {
        c = k < K ? r * (K / 2) + k / 2 : MV_OOB;
        s = __builtin_amdgcn_raw_buffer_load_b32(w.scales, (int)(k < K ? r * (K / 16) + k / 16 : MV_OOB), 0, 0);
    }
    const mv_u32x4 lo = __builtin_amdgcn_raw_buffer_load_b128(w.codes, (int)c, 0, 0);
    const mv_u32x4 hi = __builtin_amdgcn_raw_buffer_load_b128(w.codes, (int)c, 16, 0);
    return {make_uint4(lo.x, lo.y, lo.z, lo.w), make_uint4(hi.x, hi.y, hi.z, hi.w), s};
}

// MV_SHIFTED: moves what was loaded for the piece at k to its place and clears what lies past K (a block
// whose scale is 0 counts as zeros).  Only a chunk that K ends in, or past, needs it.
__device__ __forceinline__ void mv_fix(MvPiece& p, uint32_t K, uint32_t k) {
    const uint32_t by = k > K - 64 ? (k - (K - 64)) / 16 : 0;   // blocks
    p.scales = by >= 4 ? 0u : p.scales >> (8 * by);
    if (by & 1) {
        p.lo = make_uint4(p.lo.z, p.lo.w, p.hi.x, p.hi.y);
        p.hi = make_uint4(p.hi.z, p.hi.w, 0u, 0u);
    }
    if (by & 2) p.lo = p.hi;
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
// rows), 8 elements each; accumulator r of lane l is row 4 (l / 16) + r of A, weight row l % 16.  The
// order of K inside a chunk is free as long as both operands use the same: lane group g = l / 16 takes
// the chunk's elements 64g .. 64g+63, which are 32 consecutive code bytes and the blocks 4g .. 4g+3, in 8
// MFMA steps of 8.

// The workgroup's outputs from the sums of its parts of K.  sum(o, q, b, m, n): operand o's sum of part q,
// row block b, token m, row n of the block.  s0: the tensor scales of this thread's first output.
template <bool GATED, class S>
__device__ __forceinline__ void mv_join(const MvArgs& a, int parts, int tokens, int64_t m0,
                                        const float (&s0)[GATED ? 2 : 1], S&& sum) {
    constexpr int NW = GATED ? 2 : 1;
    for (int i = threadIdx.x; i < tokens * MV_ROWS * a.wr; i += blockDim.x) {
        const int nt = i % MV_ROWS, b = i / MV_ROWS % a.wr, mt = i / MV_ROWS / a.wr;
        const int64_t m = m0 + mt, n = ((int64_t)blockIdx.x * a.wr + b) * MV_ROWS + nt;
        if (n >= a.N) continue;
        float v[NW];
#pragma unroll
        for (int o = 0; o < NW; ++o) {
            float s = 0.0f;
            for (int q = 0; q < parts; ++q) s += sum(o, q, b, mt, nt);
            v[o] = s / (i == (int)threadIdx.x ? s0[o] : a.w[o].s_enc[a.rows ? n : 0]);
        }
        float y = v[0];
        if constexpr (GATED)
            y = (a.act == 0 ? act_value<0>(v[0]) : a.act == 1 ? act_value<1>(v[0]) : act_value<2>(v[0])) * v[NW - 1];
        if (a.y_f32) ((float*)a.y)[m * a.N + n] = y;
        else ((uint16_t*)a.y)[m * a.N + n] = (uint16_t)bf16x2_rne(y, 0.0f);
    }
}

// Those tensor scales, fetched at the start: at the end they would cost a trip to memory.
template <int NW>
__device__ __forceinline__ void mv_scales(const MvArgs& a, float (&s0)[NW]) {
    const int64_t n = ((int64_t)blockIdx.x * a.wr + threadIdx.x / MV_ROWS % a.wr) * MV_ROWS + threadIdx.x % MV_ROWS;
#pragma unroll
    for (int o = 0; o < NW; ++o) s0[o] = a.w[o].s_enc[a.rows ? (n < a.N ? n : a.N - 1) : 0];
}

// ---------------------------------------------------------------- one token

// One chunk of x: A's row i holds the chunk's block i and zeros elsewhere, so the product's row i is block
// i's sum, over weights without their scale, and accumulator r of lane group g is block 4g + r, whose scale
// is byte r of the lane's own.  That leaves half a VALU operation per weight and six per chunk for the scales.
// The weights of a block's sum are code * 2^-7 (exact in bf16), at most 6/128 each, so that 16 of them times
// finite tokens stay below the largest token; its scale takes the 2^7 back (at most 448 * 128).
// Lane (i, g) holds x where i / 4 = g, in the steps 2 (i % 4) and 2 (i % 4) + 1.
struct MvOneX {
    bf16x8_t v[2];
    __device__ __forceinline__ void load(const __amdgpu_buffer_rsrc_t& x, int r16, int g, uint32_t K, uint32_t k) {
        const uint32_t e = k + 16 * (r16 & 3);
#pragma unroll
        for (int h = 0; h < 2; ++h)
            v[h] = __builtin_bit_cast(bf16x8_t, __builtin_amdgcn_raw_buffer_load_b128(
                       x, (int)(r16 >> 2 == g && e + 8 * h < K ? 2 * e + 16 * h : MV_OOB), 0, 0));
    }
};

constexpr float MV_CODE_SCALE = 128.0f;

__device__ __forceinline__ bf16x8_t mv_codes(uint32_t w) {
    bf16x8_t r;
    static_for<0, 4>([&](auto i_c) {
        constexpr int I = decltype(i_c)::value;
        const bf16x2_t v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f / MV_CODE_SCALE, I);
        r[2 * I] = v[0];
        r[2 * I + 1] = v[1];
    });
    return r;
}

template <int NW>
__device__ __forceinline__ void mv_use_one(const MvPiece (&p)[NW], const MvOneX& x, int r16, floatx4 (&acc)[NW]) {
    const floatx4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
    const bf16x8_t none = {};
    floatx4 d[NW];
    static_for<0, 8>([&](auto j_c) {
        constexpr int J = decltype(j_c)::value;
        const bf16x8_t xv = (r16 & 3) == J / 2 ? x.v[J & 1] : none;
#pragma unroll
        for (int o = 0; o < NW; ++o)
            d[o] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv, mv_codes(mv_word<J>(p[o])), J == 0 ? zero : d[o], 0, 0, 0);
    });
#pragma unroll
    for (int o = 0; o < NW; ++o) {
        const floatx2 lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(p[o].scales, MV_CODE_SCALE, false);
        const floatx2 hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(p[o].scales, MV_CODE_SCALE, true);
        acc[o][0] = __builtin_fmaf(d[o][0], lo[0], acc[o][0]);
        acc[o][1] = __builtin_fmaf(d[o][1], lo[1], acc[o][1]);
        acc[o][2] = __builtin_fmaf(d[o][2], hi[0], acc[o][2]);
        acc[o][3] = __builtin_fmaf(d[o][3], hi[1], acc[o][3]);
    }
}

constexpr int MV_ONE_WAVES = 16;

// A workgroup: one token (blockIdx.y) by 16 weight rows, K dealt in chunks to its waves.
template <bool GATED, int LOAD>
__global__ __launch_bounds__(64 * MV_ONE_WAVES) void matvec_kernel(MvArgs a) {
    constexpr int NW = GATED ? 2 : 1, D = 4 / NW;   // chunks in flight
    __shared__ float red[MV_ONE_WAVES][NW][4][MV_ROWS + 1];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int parts = (int)(blockDim.x >> 6);
    const int r16 = lane & 15, g = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * MV_ROWS, m0 = blockIdx.y;
    const uint32_t K = (uint32_t)a.K;
    const int chunks = (int)((K + MV_CHUNK - 1) / MV_CHUNK);
    const __amdgpu_buffer_rsrc_t xr =
        __builtin_amdgcn_make_buffer_rsrc((void*)(a.x + m0 * a.ldx), (short)0, (int)(2 * K), 0x00020000);
    MvRsrc w[NW];
    floatx4 acc[NW];
#pragma unroll
    for (int o = 0; o < NW; ++o) {
        w[o] = mv_rsrc(a.w[o], n0, a.N, a.K, r16);
        acc[o] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    float s0[NW];
    mv_scales(a, s0);
    MvPiece p[D][NW];
    MvOneX x[D];
    auto load = [&](int c, int d) {
        const uint32_t k = (uint32_t)c * MV_CHUNK + 64 * g;
        x[d].load(xr, r16, g, K, k);
#pragma unroll
        for (int o = 0; o < NW; ++o) p[d][o] = mv_load<LOAD>(w[o], (uint32_t)r16, K, k);
    };
    auto use = [&](int c, int d) {
        if constexpr (LOAD == MV_SHIFTED) {
            if ((uint32_t)(c + 1) * MV_CHUNK > K)   // uniform
#pragma unroll
                for (int o = 0; o < NW; ++o) mv_fix(p[d][o], K, (uint32_t)c * MV_CHUNK + 64 * g);
        }
        mv_use_one(p[d], x[d], r16, acc);
    };
    int c = wave, left = chunks > wave ? (chunks - wave - 1) / parts + 1 : 0;   // this wave's next chunk, and how many
    if (left >= 2 * D) {   // a chunk is loaded as another is used, without a branch in between
#pragma unroll
        for (int d = 0; d < D; ++d) load(c + d * parts, d);
        for (; left >= 2 * D; left -= D, c += D * parts)
            static_for<0, D>([&](auto d_c) {
                constexpr int U = decltype(d_c)::value;
                use(c + U * parts, U);
                load(c + (U + D) * parts, U);
            });
#pragma unroll
        for (int d = 0; d < D; ++d) use(c + d * parts, d);
        left -= D;
        c += D * parts;
    }
    while (left > 0)   // up to D chunks, all loaded first
        static_for<0, D>([&](auto n_c) {
            constexpr int N = D - decltype(n_c)::value;
            if (left >= N) {
#pragma unroll
                for (int d = 0; d < N; ++d) load(c + d * parts, d);
#pragma unroll
                for (int d = 0; d < N; ++d) use(c + d * parts, d);
                left -= N;
                c += N * parts;
            }
        });
#pragma unroll
    for (int o = 0; o < NW; ++o) red[wave][o][g][r16] = (acc[o][0] + acc[o][1]) + (acc[o][2] + acc[o][3]);
    __syncthreads();
    mv_join<GATED>(a, parts, 1, m0, s0, [&](int o, int q, int, int, int n) {
        const float (&f)[4][MV_ROWS + 1] = red[q][o];
        return (f[0][n] + f[1][n]) + (f[2][n] + f[3][n]);
    });
}

// ---------------------------------------------------------------- several tokens

// Up to T tokens.  A's rows are the tokens, and the weights take their block scales first (two VALU
// operations per weight).  The waves of a workgroup are wr row blocks times `parts` parts of K that go
// through K in step, a chunk of each part at a time; a step's tokens come through LDS, where the wr waves
// of a part share them, double-buffered: a wave that reads them from memory in the MFMA's layout
// touches 64 lines per load.  Tokens and weights are asked for two steps ahead.
constexpr int MV_XPITCH = 2 * MV_CHUNK + 16;   // bytes between tokens in LDS: 16 tokens' reads cover all banks
constexpr int mv_parts(int t) { return t == 4 ? 16 : 128 / t; }   // at most
constexpr int mv_waves(int t) { return t == 4 ? 16 : 8; }        // at most
constexpr int mv_min_wr(int t) { return t <= 16 ? 1 : t / 16; }   // so that a thread carries T / 2 wr <= 8 vectors

template <int T, bool GATED, int LOAD>
__global__ __launch_bounds__(64 * mv_waves(T)) void matvec_tokens_kernel(MvArgs a) {
    constexpr int NW = GATED ? 2 : 1, MT = (T + 15) / 16, XV = T == 4 ? 2 : 8, RS = MV_ROWS + 1;
    constexpr int XBUF = mv_parts(T) * T * MV_XPITCH;
    static_assert(mv_waves(T) * NW * T * RS * 4 <= 2 * XBUF, "the join takes the tokens' place");
    __shared__ __attribute__((aligned(16))) uint8_t lds[2 * XBUF];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int parts = (int)(blockDim.x >> 6) / a.wr, wr = wave % a.wr, part = wave / a.wr;
    const int r16 = lane & 15, g = lane >> 4;
    const int64_t n0 = ((int64_t)blockIdx.x * a.wr + wr) * MV_ROWS, m0 = (int64_t)blockIdx.y * T;
    const int tokens = (int)(a.M - m0 < T ? a.M - m0 : T);
    const uint32_t K = (uint32_t)a.K;
    const int steps = (int)((K + MV_CHUNK * parts - 1) / (MV_CHUNK * parts));
    MvRsrc w[NW];
#pragma unroll
    for (int o = 0; o < NW; ++o) w[o] = mv_rsrc(a.w[o], n0, a.N, a.K, r16);
    float s0[NW];
    mv_scales(a, s0);
    floatx4 acc[NW][MT];
#pragma unroll
    for (int o = 0; o < NW; ++o)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[o][t] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    // step s takes the chunks s parts .. s parts + parts - 1, one for each part; the waves of a part fetch its
    // tokens, 32 threads a token
    const int tip = (int)threadIdx.x - part * 64 * a.wr, xe = 8 * (tip & 31);
    const uint16_t* xsrc = a.x + (m0 + (tip >> 5)) * a.ldx + part * MV_CHUNK + xe;
    uint8_t* xdst = lds + (part * T + (tip >> 5)) * MV_XPITCH + 2 * xe;
    mv_u32x4 xv[2][XV];   // of an even and of an odd step
    auto load_x = [&](int s, mv_u32x4 (&v)[XV]) {
        const bool in = (uint32_t)(s * parts + part) * MV_CHUNK + xe < K;
#pragma unroll
        for (int u = 0; u < XV; ++u) {
            v[u] = mv_u32x4{0, 0, 0, 0};
            if (in && (tip >> 5) + 2 * a.wr * u < tokens)
                v[u] = *(const mv_u32x4*)(xsrc + (int64_t)(2 * a.wr * u) * a.ldx + (int64_t)s * parts * MV_CHUNK);
        }
    };
    auto put_x = [&](int s, const mv_u32x4 (&v)[XV]) {
#pragma unroll
        for (int u = 0; u < XV; ++u)
            if ((tip >> 5) + 2 * a.wr * u < tokens) *(mv_u32x4*)(xdst + (s & 1) * XBUF + 2 * a.wr * u * MV_XPITCH) = v[u];
    };
    MvPiece p[2][NW];
    auto load_w = [&](int s, MvPiece (&d)[NW]) {
        const uint32_t k = (uint32_t)(s * parts + part) * MV_CHUNK + 64 * g;
#pragma unroll
        for (int o = 0; o < NW; ++o) d[o] = mv_load<LOAD>(w[o], (uint32_t)r16, K, k);
    };
    const uint8_t* xrow[MT];   // lanes of tokens past M repeat the last one (their outputs are not stored)
#pragma unroll
    for (int t = 0; t < MT; ++t)
        xrow[t] = lds + (part * T + (16 * t + r16 < tokens ? 16 * t + r16 : tokens - 1)) * MV_XPITCH + 128 * g;
    auto use = [&](int s, MvPiece (&d)[NW]) {
        if constexpr (LOAD == MV_SHIFTED) {
            if ((uint32_t)(s * parts + part + 1) * MV_CHUNK > K)   // uniform
#pragma unroll
                for (int o = 0; o < NW; ++o) mv_fix(d[o], K, (uint32_t)(s * parts + part) * MV_CHUNK + 64 * g);
        }
        static_for<0, 8>([&](auto j_c) {
            constexpr int J = decltype(j_c)::value;
            bf16x8_t xf[MT];
#pragma unroll
            for (int t = 0; t < MT; ++t) xf[t] = *(const bf16x8_t*)(xrow[t] + (s & 1) * XBUF + 16 * J);
#pragma unroll
            for (int o = 0; o < NW; ++o) {
                const bf16x8_t b = mv_dequant(mv_word<J>(d[o]), __builtin_amdgcn_cvt_f32_fp8((int)d[o].scales, J / 2));
#pragma unroll
                for (int t = 0; t < MT; ++t)
                    acc[o][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[t], b, acc[o][t], 0, 0, 0);
            }
        });
    };
    // past K nothing is read, and zeros go where nobody looks
    auto step = [&](int s, MvPiece (&w0)[NW], mv_u32x4 (&x0)[XV], const mv_u32x4 (&x1)[XV]) {
        load_x(s + 2, x0);
        use(s, w0);
        load_w(s + 2, w0);
        if (s > 0) put_x(s + 1, x1);   // where step s - 1's tokens were
        __syncthreads();               // they are there, and step s's are done with
    };
    if (steps > 0) {
        load_x(0, xv[0]);
        load_x(1, xv[1]);
        load_w(0, p[0]);
        load_w(1, p[1]);
        put_x(0, xv[0]);
        put_x(1, xv[1]);
        __syncthreads();
    }
    for (int s = 0; s < steps; s += 2) {
        step(s, p[0], xv[0], xv[1]);
        if (s + 1 < steps) step(s + 1, p[1], xv[1], xv[0]);
    }
    float* red = (float*)lds;   // [wave][NW][T][RS]
#pragma unroll
    for (int o = 0; o < NW; ++o)
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int m = 16 * t + 4 * g + r;
                if (m < tokens) red[((wave * NW + o) * T + m) * RS + r16] = acc[o][t][r];
            }
    __syncthreads();
    mv_join<GATED>(a, parts, tokens, m0, s0, [&](int o, int q, int b, int m, int n) {
        return red[(((q * a.wr + b) * NW + o) * T + m) * RS + n];
    });
}

// ---------------------------------------------------------------- launches

// One token: as many waves share K as let every workgroup be resident at once (16 waves on each CU), at least
// 4 and no more than there are chunks.
template <bool GATED, int LOAD>
static int launch_one(MvArgs a, hipStream_t s) {
    const int64_t blocks = (a.N + MV_ROWS - 1) / MV_ROWS, chunks = (a.K + MV_CHUNK - 1) / MV_CHUNK;
    int parts = MV_ONE_WAVES;
    while (parts > 4 && parts * blocks * a.M > MV_CUS * MV_ONE_WAVES) parts /= 2;
    while (parts > 1 && parts / 2 >= chunks) parts /= 2;
    a.wr = 1;
    hipLaunchKernelGGL((matvec_kernel<GATED, LOAD>), dim3((unsigned)blocks, (unsigned)a.M), dim3(64 * parts), 0, s, a);
    return (int)hipGetLastError();
}

// Several: row blocks share a workgroup, and with it the tokens, until there is one workgroup for each CU;
// the other waves share K.
template <int T>
static int64_t tokens_workgroups(const MvArgs& a) {
    return ((a.N + MV_ROWS * mv_min_wr(T) - 1) / (MV_ROWS * mv_min_wr(T))) * ((a.M + T - 1) / T);
}

template <int T, bool GATED, int LOAD>
static int launch_tokens(MvArgs a, hipStream_t s) {
    const int64_t blocks = (a.N + MV_ROWS - 1) / MV_ROWS, mb = (a.M + T - 1) / T;
    const int64_t chunks = (a.K + MV_CHUNK - 1) / MV_CHUNK;
    a.wr = mv_min_wr(T);
    while (a.wr < 4 && a.wr * MV_CUS < blocks * mb) a.wr *= 2;
    int parts = mv_waves(T) / a.wr < mv_parts(T) ? mv_waves(T) / a.wr : mv_parts(T);
    while (parts > 1 && parts / 2 >= chunks) parts /= 2;
    hipLaunchKernelGGL((matvec_tokens_kernel<T, GATED, LOAD>), dim3((unsigned)((blocks + a.wr - 1) / a.wr), (unsigned)mb),
                       dim3(64 * a.wr * parts), 0, s, a);
    return (int)hipGetLastError();
}

// Tiles of as many tokens as leave three CUs in four a workgroup: a larger one reads and dequantizes a weight
// fewer times, a smaller one splits into more workgroups.  us with tiles of 16 / 32 / 64, weights rotating:
// 64 x 14336 x 8192 gated 142 / 88 / 61, 64 x 14336 x 4096 54 / 34 / 25; 64 x 6151 x 4112 31 / 21 / 28, 64 x
// 4096 x 4096 15 / 13 / 24, 32 x 14336 x 4096 28 / 19 / 21; 32 x 4096 x 4096 11 / 13 / 20, 33 x 1000 x
// 16384 17 / 31 / 63.
template <bool GATED, int LOAD>
static int launch_mv(const MvArgs& a, hipStream_t s) {
    if (a.M == 1) return launch_one<GATED, LOAD>(a, s);
    if (a.M <= 4) return launch_tokens<4, GATED, LOAD>(a, s);
    if (a.M > 4096 || (a.M > 32 && 4 * tokens_workgroups<64>(a) >= 3 * MV_CUS)) return launch_tokens<64, GATED, LOAD>(a, s);
    if (a.M > 16 && 4 * tokens_workgroups<32>(a) >= 3 * MV_CUS) return launch_tokens<32, GATED, LOAD>(a, s);
    return launch_tokens<16, GATED, LOAD>(a, s);
}

int launch_nvfp4_matvec(int act, const void* x, int64_t ldx, int64_t M, int64_t N, int64_t K, const uint8_t* w_codes,
                        const uint8_t* w_scales, const float* w_s_enc, const uint8_t* up_codes,
                        const uint8_t* up_scales, const float* up_s_enc, int rows, void* y, int y_f32,
                        void* hip_stream) {
    if (M == 0 || N == 0) return 0;
    const MvArgs a{(const uint16_t*)x, ldx, M, N, K, {{w_codes, w_scales, w_s_enc}, {up_codes, up_scales, up_s_enc}},
                   rows, y, y_f32, act, 1};
    hipStream_t s = (hipStream_t)hip_stream;
    if (K < 64) return act < 0 ? launch_tokens<64, false, MV_BLOCKS>(a, s) : launch_tokens<64, true, MV_BLOCKS>(a, s);
    if (K % 64 == 0) return act < 0 ? launch_mv<false, MV_ALIGNED>(a, s) : launch_mv<true, MV_ALIGNED>(a, s);
    return act < 0 ? launch_mv<false, MV_SHIFTED>(a, s) : launch_mv<true, MV_SHIFTED>(a, s);
}

}  // namespace bsq
