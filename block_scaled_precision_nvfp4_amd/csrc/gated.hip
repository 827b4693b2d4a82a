// gated.hip -- the two matrix products around the activation of a gated feed-forward block, on quantized
// operands, each with its elementwise part in the epilogue:
//
//   forward   g = A Wg^T, u = A Wu^T, h = act(g) u; g and u kept in bf16 for the backward pass if asked
//   backward  dh = dY Wd^T; d_gate = dh u act'(g), d_up = dh act(g)
//
// The products are the 256 x 256 tiles of gemm_tile.hpp.  The forward's B operand interleaves the two
// weights, 64 rows of gate and 64 of up per wave, so that one pass over A feeds both and g and u of an
// output land in the same lane (GatedDma).  h comes from the unrounded fp32 g and u, and dh is never
// rounded nor stored: the roundings are the fp32 sums, the scale factors, a few fp32 operations of the
// activation and one bf16 rounding per output.
#include "activation.hpp"
#include "gemm_tile.hpp"
#include "launch.hpp"

namespace bsq {

// Calls body(std::integral_constant<int, ACT>) for the run-time act.
template <class F>
__device__ __forceinline__ void with_act(int act, F&& body) {
    if (act == 0) body(std::integral_constant<int, 0>{});
    else if (act == 1) body(std::integral_constant<int, 1>{});
    else body(std::integral_constant<int, 2>{});
}

// The tile's K loop.  MODE and SL (MXFP8): where scales and codes come from, as in the main loop; each
// kernel holds one of the loops (several in one function cost it its register allocation).
template <int FMT, int MODE, int SL, class G>
__device__ __forceinline__ void tile_product(const G& g, int64_t m0, int64_t n0, uint8_t* lds, int wm, int wn,
                                             int lane, floatx16 (&acc)[4][4]) {
    using F = Fmt<FMT>;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
    const int64_t nk = (g.K + F::BK - 1) / F::BK;
    if constexpr (FMT == 1) mx_main_loop<MODE, SL, true>(g, m0, n0, nk, lds, wm, wn, lane, acc);
    else if constexpr (FMT == 2) nvw_main_loop<4>(g, m0, n0, nk, lds, wm, wn, lane, acc);
    else nvs_main_loop<4>(g, m0, n0, nk, lds, wm, wn, lane, acc);
}

// ---------------------------------------------------------------- forward

// Output factors of a gated tile, g(m, n) = sum fa[m] fb[n] (and u with the up rows of fb): with a
// per-tensor A, fa = 1 and fb = fp32(1 / (S_a S_b)), product and quotient in binary64; with a row-scaled A,
// fa[m] = fp32(1 / S_a[m]) and fb = fp32(1 / S_b).
__device__ __forceinline__ void gated_factors(const GatedArgs& g, int64_t m0, int64_t n0, float* fa, float* fb) {
    const int t = threadIdx.x;   // 256 threads: one A row and one B row each
    const int64_t m = m0 + t, n = n0 + 64 * (t >> 7) + (t & 63);
    const float* sb = t & 64 ? g.u_s_enc : g.b_s_enc;
    const double sbv = g.b_rows ? (n < g.N ? (double)sb[n] : 1.0) : (double)sb[0];
    fa[t] = g.a_rows && m < g.M ? (float)(1.0 / (double)g.a_s_enc[m]) : 1.0f;
    fb[t] = (float)(1.0 / (g.a_rows ? sbv : sbv * (double)g.a_s_enc[0]));
}

// One tile per workgroup: 256 rows of A by 128 columns of h.  Epilogue in two passes of 64 rows per
// wave: g, u and h are formed where the accumulators are and staged in the wave's own LDS region as
// three row-major blocks of 64 columns, then stored in 16-byte chunks (single elements where the rows
// of h do not keep 16-byte chunks apart).
template <int FMT, int MODE = 0, int SL = 0>
__global__ __launch_bounds__(256, 1) void gated_kernel(GatedArgs g) {
    using F = Fmt<FMT>;
    constexpr int RS = 3 * 128 + 16;   // staged bytes of a row: h, gate, up
    static_assert(4 * 64 * RS <= F::LDS - FACT_BYTES, "epilogue staging");
    __shared__ __attribute__((aligned(16))) uint8_t lds[F::LDS];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = (wave >> 1) * 128, wn = (wave & 1) * 128;
    int64_t tm, tn;
    tile_of((g.M + GBM - 1) / GBM, (g.N + GBN / 2 - 1) / (GBN / 2), blockIdx.x, tm, tn);
    const int64_t m0 = tm * GBM, n0 = tn * (GBN / 2);
    floatx16 acc[4][4];
    tile_product<FMT, MODE, SL>(g, m0, n0, lds, wm, wn, lane, acc);
    float* fa = (float*)(lds + F::LDS - FACT_BYTES);
    float* fb = fa + 256;
    __syncthreads();   // every wave is done with the operand buffers (and its DMAs)
    if constexpr (F::NV) {
        gated_factors(g, m0, n0, fa, fb);
        __syncthreads();
    }
    const int frow = lane & 31, kh = lane >> 5;
    uint8_t* reg = lds + wave * 64 * RS;
    const int64_t c0 = n0 + wn / 2;   // the wave's first column of h
    const bool save = g.gate_up != nullptr, chunks = g.N % 8 == 0;   // uniform
    with_act(g.act, [&](auto act_c) {
        constexpr int ACT = decltype(act_c)::value;
        static_for<0, 2>([&](auto h_c) {
            constexpr int H = decltype(h_c)::value;
            static_for<0, 4>([&](auto t_c) {
                constexpr int IL = decltype(t_c)::value / 2, I = 2 * H + IL, J = decltype(t_c)::value % 2;
                [[maybe_unused]] const float fr = F::NV ? fa[wm + 32 * I + frow] : 1.0f;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int col = 32 * J + 8 * q + 4 * kh;
                    float hv[4], gv[4], uv[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        gv[r] = acc[I][J][4 * q + r];
                        uv[r] = acc[I][J + 2][4 * q + r];
                        if constexpr (F::NV) {
                            gv[r] *= fr * fb[wn + col + r];
                            uv[r] *= fr * fb[wn + 64 + col + r];
                        }
                        hv[r] = act_value<ACT>(gv[r]) * uv[r];
                    }
                    uint8_t* dst = reg + (32 * IL + frow) * RS + 2 * col;
                    *(uint2*)dst = make_uint2(bf16x2_rne(hv[0], hv[1]), bf16x2_rne(hv[2], hv[3]));
                    if (save) {
                        *(uint2*)(dst + 128) = make_uint2(bf16x2_rne(gv[0], gv[1]), bf16x2_rne(gv[2], gv[3]));
                        *(uint2*)(dst + 256) = make_uint2(bf16x2_rne(uv[0], uv[1]), bf16x2_rne(uv[2], uv[3]));
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            });
            asm volatile("" ::: "memory");
            // a wave reads back only what it wrote, in order
            const int64_t r0 = m0 + wm + 64 * H;
            for (int o = 0; o < (save ? 3 : 1); ++o) {
                uint16_t* out = o == 0 ? (uint16_t*)g.c : g.gate_up + (o == 2 ? g.N : 0);
                const int64_t pitch = o == 0 ? g.N : 2 * g.N;
                if (chunks) {
#pragma unroll
                    for (int p = 0; p < 8; ++p) {
                        const int row = 8 * p + (lane >> 3), c = lane & 7;
                        const uint4 v = *(const uint4*)(reg + row * RS + 128 * o + 16 * c);
                        if (r0 + row < g.M && c0 + 8 * c < g.N) *(uint4*)(out + (r0 + row) * pitch + c0 + 8 * c) = v;
                    }
                } else {
                    for (int row = 0; row < 64; ++row)
                        if (r0 + row < g.M && c0 + lane < g.N)
                            out[(r0 + row) * pitch + c0 + lane] = *(const uint16_t*)(reg + row * RS + 128 * o + 2 * lane);
                }
            }
            asm volatile("" ::: "memory");
        });
    });
}

// ---------------------------------------------------------------- backward

struct GatedBackArgs : GemmArgs {   // c: the gradient of [gate, up], [M][2N] bf16
    const uint16_t* gate_up;        // [M][2N] bf16
    int act;
};

// One tile per workgroup: 256 x 256 of dh.  Epilogue in two passes of 64 rows per wave: dh goes through the
// wave's own LDS region in fp32, then each lane takes 8 columns of a row, reads their gate and up (16
// bytes each) and writes both gradients.
template <int FMT, int MODE = 0, int SL = 0>
__global__ __launch_bounds__(256, 1) void gated_backward_kernel(GatedBackArgs g) {
    using F = Fmt<FMT>;
    constexpr int RS = 128 * 4 + 16;
    static_assert(4 * 64 * RS <= F::LDS - FACT_BYTES, "epilogue staging");
    __shared__ __attribute__((aligned(16))) uint8_t lds[F::LDS];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = (wave >> 1) * 128, wn = (wave & 1) * 128;
    int64_t tm, tn;
    tile_of((g.M + GBM - 1) / GBM, (g.N + GBN - 1) / GBN, blockIdx.x, tm, tn);
    const int64_t m0 = tm * GBM, n0 = tn * GBN;
    floatx16 acc[4][4];
    tile_product<FMT, MODE, SL>((const GemmArgs&)g, m0, n0, lds, wm, wn, lane, acc);
    float* fa = (float*)(lds + F::LDS - FACT_BYTES);
    float* fb = fa + 256;
    __syncthreads();   // every wave is done with the operand buffers (and its DMAs)
    if constexpr (F::NV) {
        tile_factors<FMT>(g, m0, n0, fa, fb);
        __syncthreads();
    }
    const int frow = lane & 31, kh = lane >> 5;
    uint8_t* reg = lds + wave * 64 * RS;
    const bool chunks = g.N % 8 == 0;   // uniform
    with_act(g.act, [&](auto act_c) {
        constexpr int ACT = decltype(act_c)::value;
        static_for<0, 2>([&](auto h_c) {
            constexpr int H = decltype(h_c)::value;
            static_for<0, 8>([&](auto t_c) {
                constexpr int IL = decltype(t_c)::value / 4, I = 2 * H + IL, J = decltype(t_c)::value % 4;
                [[maybe_unused]] const float fr = F::NV ? fa[wm + 32 * I + frow] : 1.0f;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int col = 32 * J + 8 * q + 4 * kh;
                    float4 v = make_float4(acc[I][J][4 * q], acc[I][J][4 * q + 1], acc[I][J][4 * q + 2],
                                           acc[I][J][4 * q + 3]);
                    if constexpr (F::NV) {
                        const float* f = fb + wn + col;
                        v.x *= fr * f[0]; v.y *= fr * f[1]; v.z *= fr * f[2]; v.w *= fr * f[3];
                    }
                    *(float4*)(reg + (32 * IL + frow) * RS + 4 * col) = v;
                }
                __builtin_amdgcn_sched_barrier(0);
            });
            asm volatile("" ::: "memory");
            const int64_t r0 = m0 + wm + 64 * H, c0 = n0 + wn;
            uint16_t* out = (uint16_t*)g.c;
            if (chunks) {
#pragma unroll 4
                for (int p = 0; p < 16; ++p) {
                    const int row = 4 * p + (lane >> 4), c = 8 * (lane & 15);
                    if (r0 + row >= g.M || c0 + c >= g.N) continue;
                    const int64_t at = (r0 + row) * 2 * g.N + c0 + c;
                    float gv[8], uv[8], dh[8];
                    unpack_bf16x8(*(const uint4*)(g.gate_up + at), gv);
                    unpack_bf16x8(*(const uint4*)(g.gate_up + at + g.N), uv);
                    *(float4*)dh = *(const float4*)(reg + row * RS + 4 * c);
                    *(float4*)(dh + 4) = *(const float4*)(reg + row * RS + 4 * c + 16);
                    uint32_t dg[4], du[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const ActGrad a = act_grad<ACT>(gv[2 * e]), b = act_grad<ACT>(gv[2 * e + 1]);
                        dg[e] = bf16x2_rne(dh[2 * e] * uv[2 * e] * a.df, dh[2 * e + 1] * uv[2 * e + 1] * b.df);
                        du[e] = bf16x2_rne(dh[2 * e] * a.f, dh[2 * e + 1] * b.f);
                    }
                    *(uint4*)(out + at) = make_uint4(dg[0], dg[1], dg[2], dg[3]);
                    *(uint4*)(out + at + g.N) = make_uint4(du[0], du[1], du[2], du[3]);
                }
            } else {
                for (int e = lane; e < 64 * 128; e += 64) {
                    const int row = e >> 7, c = e & 127;
                    if (r0 + row >= g.M || c0 + c >= g.N) continue;
                    const int64_t at = (r0 + row) * 2 * g.N + c0 + c;
                    const float gv = __uint_as_float((uint32_t)g.gate_up[at] << 16);
                    const float uv = __uint_as_float((uint32_t)g.gate_up[at + g.N] << 16);
                    const float dh = *(const float*)(reg + row * RS + 4 * c);
                    const ActGrad a = act_grad<ACT>(gv);
                    out[at] = (uint16_t)bf16x2_rne(dh * uv * a.df, 0.0f);
                    out[at + g.N] = (uint16_t)bf16x2_rne(dh * a.f, 0.0f);
                }
            }
            asm volatile("" ::: "memory");
        });
    });
}

// ---------------------------------------------------------------- launches

// Calls launch(FMT, MODE, SL as integral constants) for the operands' format.  NVFP4: aligned scale records
// where K is a multiple of 256, per-slice records otherwise.  MXFP8: aligned records where K is a
// multiple of 512 (the C ABI asks for 16-byte aligned scale tensors, and for that K with a slab
// operand), per-slice slots otherwise.
template <class F>
static int with_loop(int fmt, int64_t K, int slab, F&& launch) {
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    using I2 = std::integral_constant<int, 2>;
    using I3 = std::integral_constant<int, 3>;
    using Slab = std::integral_constant<int, MX_SLAB>;
    if (fmt == 0 && K % 256 == 0) launch(I2{}, I0{}, I0{});
    else if (fmt == 0) launch(I3{}, I0{}, I0{});
    else if (K % (MX_GROUP * 64) != 0) launch(I1{}, std::integral_constant<int, MX_SLOTS>{}, I0{});
    else if (slab == 0) launch(I1{}, std::integral_constant<int, MX_RECS>{}, I0{});
    else if (slab == 1) launch(I1{}, Slab{}, I1{});
    else if (slab == 2) launch(I1{}, Slab{}, I2{});
    else launch(I1{}, Slab{}, I3{});
    return (int)hipGetLastError();
}

int64_t gated_tiles(int64_t M, int64_t N) { return ((M + GBM - 1) / GBM) * ((N + GBN / 2 - 1) / (GBN / 2)); }

int launch_gated_gemm(int fmt, int act, int64_t M, int64_t N, int64_t K, const uint8_t* a_codes,
                      const uint8_t* a_scales, const float* a_s_enc, const uint8_t* gate_codes,
                      const uint8_t* gate_scales, const float* gate_s_enc, const uint8_t* up_codes,
                      const uint8_t* up_scales, const float* up_s_enc, int a_rows, int b_rows, int slab, void* h,
                      void* gate_up, void* hip_stream) {
    GatedArgs g;
    (GemmArgs&)g = GemmArgs{M, N, K, a_codes, a_scales, a_s_enc, gate_codes, gate_scales, gate_s_enc, h, a_rows,
                            b_rows, K, slab, 0};
    g.u_codes = up_codes;
    g.u_scales = up_scales;
    g.u_s_enc = up_s_enc;
    g.gate_up = (uint16_t*)gate_up;
    g.act = act;
    return with_loop(fmt, K, slab, [&](auto f, auto mode, auto sl) {
        hipLaunchKernelGGL((gated_kernel<decltype(f)::value, decltype(mode)::value, decltype(sl)::value>),
                           dim3((unsigned)gated_tiles(M, N)), dim3(256), 0, (hipStream_t)hip_stream, g);
    });
}

int launch_gated_gemm_backward(int fmt, int act, int64_t M, int64_t N, int64_t K, const uint8_t* dy_codes,
                               const uint8_t* dy_scales, const float* dy_s_enc, const uint8_t* w_codes,
                               const uint8_t* w_scales, const float* w_s_enc, int a_rows, int b_rows, int slab,
                               const void* gate_up, void* d_gate_up, void* hip_stream) {
    GatedBackArgs g;
    (GemmArgs&)g = GemmArgs{M, N, K, dy_codes, dy_scales, dy_s_enc, w_codes, w_scales, w_s_enc, d_gate_up, a_rows,
                            b_rows, K, slab, 0};
    g.gate_up = (const uint16_t*)gate_up;
    g.act = act;
    const int64_t tiles = ((M + GBM - 1) / GBM) * ((N + GBN - 1) / GBN);
    return with_loop(fmt, K, slab, [&](auto f, auto mode, auto sl) {
        hipLaunchKernelGGL((gated_backward_kernel<decltype(f)::value, decltype(mode)::value, decltype(sl)::value>),
                           dim3((unsigned)tiles), dim3(256), 0, (hipStream_t)hip_stream, g);
    });
}

}  // namespace bsq
