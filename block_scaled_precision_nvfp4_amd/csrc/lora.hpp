// lora.hpp -- what the adapters' kernels (lora.hip) and the product of tokens with NVFP4 weights (matvec.hip) share.
#pragma once

#include "device_common.hpp"

namespace bsq {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

struct LoraArgs {
    int64_t M, N, K;
    int r;                      // a multiple of 8
    int64_t L;                  // adapters
    const uint16_t* x;
    int64_t ldx;
    const int32_t* adapters;    // [M]; outside [0, L): none
    const uint16_t* a;          // [L][r][K]
    const uint16_t* b;          // [L][N][r]
    const float* scales;        // [L], or none
    float* t;                   // the down products: [M][r], or fragments of three bf16 parts (lora.hip)
    const void* y;
    int64_t ldy;
    void* out;
    int64_t ldo;
};

__host__ __device__ constexpr int lora_steps(int r) { return (r + 31) / 32; }

// A value as three bf16 parts that add up to it: 8 bits of the significand each, cut, not rounded, so that a large value
// does not become infinite.  Exact from 2^-110 on; below, what lies under bf16's smallest value is cut off, less than 2^-133
// (the matrix instruction takes subnormal parts as they are).  An infinity or NaN goes into the first part alone.
__device__ __forceinline__ void lora_split(float v, uint16_t (&part)[3]) {
    const uint32_t u = __float_as_uint(v);
    const bool fin = (u & 0x7F800000u) != 0x7F800000u;
    const uint32_t hi = (u & 0xFFFF0000u) | (!fin && (u & 0x7FFFFFu) ? 0x400000u : 0u);
    const float r1 = v - __uint_as_float(hi);
    const uint32_t mid = __float_as_uint(r1) & 0xFFFF0000u;
    const float r2 = r1 - __uint_as_float(mid);
    part[0] = (uint16_t)(hi >> 16);
    part[1] = (uint16_t)(fin ? mid >> 16 : 0u);
    part[2] = (uint16_t)(fin ? __float_as_uint(r2) >> 16 : 0u);
}

// Few tokens: a wave takes a token's products with RQ rows of its adapter's A, U pieces of 512 elements at a time, all
// their loads in flight at once: t[m][q] as fp32.  Unit `unit` of lora_few_units, 64 lanes.
//
// us of a whole call, 4096 x 4096, its tokens taken so and in tiles (lora_down_kernel, lora_up_kernel), rank 16 and rank 64:
//   64 tokens of one adapter   6.7 and 11.4,  11.1 and 11.6     64 of 64, mixed     9.6 and 46,  19 and 58
//   128 of one                 7.8 and 11.8,  14.0 and 12.2     128 of 128, mixed    12 and 47,  31 and 66
//   128 of 8 in runs           7.8 and 13.1,  14.9 and 15.5     128 of 8, mixed     7.9 and 16,  15 and 20
//   256 of one                12.1 and 11.9,  22.2 and 12.3     256 of 256, mixed    21 and 49,  54 and 82
//   256 of 8, mixed             12 and 16,    25 and 25     96 of one          7.3 and 11.7,  12.8 and 12.1
// So of one adapter tiles pay from between 64 and 96 tokens on with rank 64, from some 256 with rank 16; of mixed ones from 256
// or later.  The limit is below the first of these and looks at neither ranks nor adapters.
constexpr int LORA_FEW = 64;   // tokens at most

__host__ __device__ inline int64_t lora_few_units(int64_t M, int r, int rq) { return M * ((r + rq - 1) / rq); }
// a wave for every product while that leaves the chip room: the shortest way through K
__host__ __device__ inline int lora_few_rows(int64_t M, int r) { return M * r <= 2048 ? 1 : 4; }

template <int RQ, int U>
__device__ __forceinline__ void lora_down_few_rows(const LoraArgs& a, int64_t unit) {
    const int lane = threadIdx.x & 63, blocks = (a.r + RQ - 1) / RQ, K = (int)a.K;
    const int64_t m = unit / blocks;
    const int q0 = (int)(unit % blocks) * RQ;
    if (m >= a.M) return;
    const int id = a.adapters[m];
    if (id < 0 || id >= a.L) return;
    const uint16_t* x = a.x + m * a.ldx;
    const uint16_t* w = a.a + ((int64_t)id * a.r + q0) * a.K;   // r is a multiple of RQ
    float acc[RQ] = {};
    for (int k0 = 8 * lane; k0 < K; k0 += 512 * U) {
        uint4 xv[U], wv[RQ][U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool in = k0 + 512 * u < K;
            xv[u] = make_uint4(0, 0, 0, 0);
            if (in) xv[u] = *(const uint4*)(x + k0 + 512 * u);
#pragma unroll
            for (int q = 0; q < RQ; ++q) {
                wv[q][u] = make_uint4(0, 0, 0, 0);
                if (in) wv[q][u] = *(const uint4*)(w + (int64_t)q * a.K + k0 + 512 * u);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float f[8];
            unpack_bf16x8(xv[u], f);
#pragma unroll
            for (int q = 0; q < RQ; ++q) {
                float v[8];
                unpack_bf16x8(wv[q][u], v);
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[q] = __builtin_fmaf(f[e], v[e], acc[q]);
            }
        }
    }
#pragma unroll
    for (int q = 0; q < RQ; ++q) {
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) acc[q] += __shfl_xor(acc[q], o);
        if (lane == 0) a.t[m * a.r + q0 + q] = acc[q];
    }
}

__device__ __forceinline__ void lora_down_few(const LoraArgs& a, int rq, int64_t unit) {
    if (rq == 1) lora_down_few_rows<1, 4>(a, unit);
    else lora_down_few_rows<4, 2>(a, unit);
}

// In lora.hip: the down products of up to LORA_FEW tokens and of more, and the up products onto y.
int launch_lora_down_few(const LoraArgs& a, hipStream_t s);
int launch_lora_down_many(const LoraArgs& a, hipStream_t s);
int launch_lora_up(const LoraArgs& a, int y_f32, int out_f32, hipStream_t s);

}  // namespace bsq
