// lora.hip -- low-rank adapters beside a projection, each token with its own: out[m] = y[m] + s_a (x[m] A_a^T) B_a^T with a
// the token's adapter, A [L][r][K], B [L][N][r].
//
// Two kernels: the down products t[m] = x[m] A_a^T into the caller's workspace (fp32), then the up products
// onto y, or beside NVFP4 weights inside the epilogue of their product (matvec.hip).  Tokens go in tiles of
// 16, the rows of a matrix instruction; a tile's adapters are taken one after another, each over all 16 rows,
// and a row keeps the result of its own.  Rows do not mix, so a NaN stays with its token, or its adapter's tokens.
#include "launch.hpp"
#include "lora.hpp"

namespace bsq {

typedef float floatx4 __attribute__((ext_vector_type(4)));

constexpr int LORA_TOKENS = 16;
constexpr int LORA_DOWN_WAVES = 16;    // share K

// The ids of a tile's adapters: lane i holds token i % 16's, -1 for none.
__device__ __forceinline__ int lora_ids(const LoraArgs& a, int64_t m0) {
    const int64_t m = m0 + (threadIdx.x & 15);
    const int id = m < a.M ? a.adapters[m] : -1;
    return id >= 0 && id < a.L ? id : -1;
}

// Calls body(adapter) for the tile's adapters number first, first + step, ... in the order of their first tokens.
template <class F>
__device__ __forceinline__ void for_adapters(int ids, int first, int step, F&& body) {
    uint64_t left = __ballot(ids >= 0) & 0xFFFFu;
    for (int n = 0; left != 0; ++n) {
        const int id = __builtin_amdgcn_readlane(ids, __builtin_ctzll(left));
        left &= ~__ballot(ids == id);
        if (n >= first && (n - first) % step == 0) body(id);
    }
}

// t[m][rank] of a tile: blockIdx.x tile, .y which of its adapters, .z 16 NR ranks.  The waves share K, 64
// elements of every row at a time (whole 128-byte lines), and are joined in LDS.
template <int NR>
__global__ __launch_bounds__(64 * LORA_DOWN_WAVES) void lora_down_kernel(LoraArgs a) {
    __shared__ float red[LORA_DOWN_WAVES][NR][LORA_TOKENS][16 + 1];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int waves = (int)(blockDim.x >> 6), r16 = lane & 15, g = lane >> 4;
    const int64_t m0 = (int64_t)blockIdx.x * LORA_TOKENS, rank0 = (int64_t)blockIdx.z * 16 * NR;
    const int ids = lora_ids(a, m0);
    const int64_t mx = m0 + r16 < a.M ? m0 + r16 : a.M - 1;   // rows past the end repeat the last one
    const uint16_t* x = a.x + mx * a.ldx;
    for_adapters(ids, blockIdx.y, gridDim.y, [&](int id) {
        floatx4 acc[NR];
        const uint16_t* w[NR];
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            acc[n] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
            const int64_t rank = rank0 + 16 * n + r16;
            w[n] = a.a + ((int64_t)id * a.r + (rank < a.r ? rank : a.r - 1)) * a.K;
        }
        for (int64_t k0 = (int64_t)wave * 64; k0 < a.K; k0 += 64 * waves) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t k = k0 + 16 * g + 8 * h;
                bf16x8_t xv = {}, wv[NR] = {};
                if (k < a.K) {
                    xv = *(const bf16x8_t*)(x + k);
#pragma unroll
                    for (int n = 0; n < NR; ++n) wv[n] = *(const bf16x8_t*)(w[n] + k);
                }
#pragma unroll
                for (int n = 0; n < NR; ++n) acc[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv, wv[n], acc[n], 0, 0, 0);
            }
        }
        __syncthreads();   // the adapter before this one has been added up
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) red[wave][n][4 * g + i][r16] = acc[n][i];
        __syncthreads();
        for (int i = threadIdx.x; i < LORA_TOKENS * 16 * NR; i += blockDim.x) {
            const int m = i / (16 * NR), n = i / 16 % NR, q = i % 16;
            const int64_t rank = rank0 + 16 * n + q;
            if (rank >= a.r || m0 + m >= a.M) continue;
            const int mine = a.adapters[m0 + m];
            if (mine != id) continue;
            float s = 0.0f;
            for (int v = 0; v < waves; ++v) s += red[v][n][m][q];
            a.t[(m0 + m) * a.r + rank] = s;
        }
    });
}

// The up products of a tile by 64 columns per wave.  B's rows take the matrix instruction's rows, so that a lane
// ends with 16 adjacent columns of one token: row 4 g + i of block b stands for column 16 g + 4 b + i.  t goes in as
// three bf16 parts that add up to it exactly.
constexpr int LORA_UP_WAVES = 4, LORA_COLS = 64;

template <bool F32>
__global__ __launch_bounds__(64 * LORA_UP_WAVES) void lora_up_kernel(LoraArgs a) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int r16 = lane & 15, g = lane >> 4;
    const int64_t cols = (a.N + LORA_COLS * LORA_UP_WAVES - 1) / (LORA_COLS * LORA_UP_WAVES);
    const int64_t m0 = blockIdx.x / cols * LORA_TOKENS, n0 = (blockIdx.x % cols * LORA_UP_WAVES + wave) * LORA_COLS;
    if (n0 >= a.N) return;
    const int ids = lora_ids(a, m0);   // lane's token r16
    const int64_t m = m0 + r16;
    const float* t = a.t + (m < a.M ? m : a.M - 1) * a.r;
    const int64_t c0 = n0 + 16 * g;
    float add[16] = {};
    float scale = 0.0f;
    for_adapters(ids, 0, 1, [&](int id) {
        floatx4 acc[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) acc[b] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int q0 = 0; q0 < a.r; q0 += 32) {
            const int q = q0 + 8 * g;
            bf16x8_t part[3] = {};
            if (q < a.r && ids == id) lora_split8(t + q, part);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int64_t n = n0 + 16 * (r16 >> 2) + 4 * b + (r16 & 3);
                bf16x8_t w = {};
                if (q < a.r && n < a.N) w = *(const bf16x8_t*)(a.b + ((int64_t)id * a.N + n) * a.r + q);
#pragma unroll
                for (int p = 2; p >= 0; --p) acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, part[p], acc[b], 0, 0, 0);
            }
        }
        if (ids == id) {
            scale = a.scales ? a.scales[id] : 1.0f;
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) add[4 * b + i] = acc[b][i];
        }
    });
    if (m >= a.M || (ids < 0 && a.out == a.y)) return;
    for (int i = 0; i < 16; ++i) {
        const int64_t n = c0 + i;
        if (n >= a.N) break;
        if constexpr (F32) {
            const float y = ((const float*)a.y)[m * a.ldy + n];
            ((float*)a.out)[m * a.ldo + n] = ids < 0 ? y : __builtin_fmaf(scale, add[i], y);
        } else {
            const uint16_t y = ((const uint16_t*)a.y)[m * a.ldy + n];
            ((uint16_t*)a.out)[m * a.ldo + n] =
                ids < 0 ? y : (uint16_t)bf16x2_rne(__builtin_fmaf(scale, add[i], __uint_as_float((uint32_t)y << 16)), 0.0f);
        }
    }
}

int launch_lora_down(const LoraArgs& a, hipStream_t s) {
    if (a.M == 0 || a.r == 0) return 0;
    const int64_t tiles = (a.M + LORA_TOKENS - 1) / LORA_TOKENS;
    const unsigned many = tiles <= 16 ? (unsigned)(a.M < LORA_TOKENS ? a.M : LORA_TOKENS) : 1u;
    if (a.r <= 16)
        hipLaunchKernelGGL(lora_down_kernel<1>, dim3((unsigned)tiles, many, 1), dim3(64 * LORA_DOWN_WAVES), 0, s, a);
    else
        hipLaunchKernelGGL(lora_down_kernel<4>, dim3((unsigned)tiles, many, (unsigned)((a.r + 63) / 64)),
                           dim3(64 * LORA_DOWN_WAVES), 0, s, a);
    return (int)hipGetLastError();
}

int64_t lora_up_groups(int64_t M, int64_t N) {
    return ((M + LORA_TOKENS - 1) / LORA_TOKENS) * ((N + LORA_COLS * LORA_UP_WAVES - 1) / (LORA_COLS * LORA_UP_WAVES));
}

int launch_lora_add(int f32, int64_t M, int64_t N, int64_t K, int64_t r, int64_t L, const void* x, int64_t ldx,
                    const int32_t* adapters, const void* lora_a, const void* lora_b, const float* scales, const void* y,
                    int64_t ldy, void* out, int64_t ldo, float* workspace, void* hip_stream) {
    if (M == 0 || N == 0) return 0;
    hipStream_t s = (hipStream_t)hip_stream;
    const LoraArgs a{M, N, K, (int)r, L, (const uint16_t*)x, ldx, adapters, (const uint16_t*)lora_a, (const uint16_t*)lora_b,
                     scales, workspace, y, ldy, out, ldo};
    const int e = launch_lora_down(a, s);
    if (e) return e;
    const dim3 grid((unsigned)lora_up_groups(M, N)), block(64 * LORA_UP_WAVES);
    if (f32) hipLaunchKernelGGL(lora_up_kernel<true>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(lora_up_kernel<false>, grid, block, 0, s, a);
    return (int)hipGetLastError();
}

}  // namespace bsq
