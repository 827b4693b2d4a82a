// gated.hpp -- what the gated feed-forward products' kernels share (gated.hip: 256 x 256 tiles; gated_small.hip:
// 64 x 64 tiles).
#pragma once

#include "activation.hpp"
#include "gemm_tile.hpp"

namespace bsq {

// Cache policy of a buffer access whose data is not used again soon (non-temporal): gate, up and their gradients
// leave L2 to the operands (16384 x 14336 x 4096 backward: 1034 -> 989 us).
constexpr int STREAM = 2;

// Eight bf16 values at any multiple of an element (rows of tensors whose width is no multiple of 8).
struct __attribute__((packed, aligned(2))) Bf16x8Any { uint32_t w[4]; };

__device__ __forceinline__ u32x4s load_any(const uint16_t* p) {
    const Bf16x8Any v = *(const Bf16x8Any*)p;
    return u32x4s{v.w[0], v.w[1], v.w[2], v.w[3]};
}
__device__ __forceinline__ void store_any(uint16_t* p, u32x4s v) { *(Bf16x8Any*)p = Bf16x8Any{{v.x, v.y, v.z, v.w}}; }

// Calls body(std::integral_constant<int, ACT>) for the run-time act.
template <class F>
__device__ __forceinline__ void with_act(int act, F&& body) {
    if (act == 0) body(std::integral_constant<int, 0>{});
    else if (act == 1) body(std::integral_constant<int, 1>{});
    else body(std::integral_constant<int, 2>{});
}

struct GatedBackArgs : GemmArgs {   // c: the gradient of [gate, up], [M][2N] bf16
    const uint16_t* gate_up;        // [M][2N] bf16
    int act;
};

// Both gradients of 8 columns of a row (bf16 pairs) from dh and their gate and up.
template <int ACT>
__device__ __forceinline__ void gated_grads(const float (&dh)[8], u32x4s gate, u32x4s up, u32x4s& dg, u32x4s& du) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const ActGrad a = act_grad<ACT>(bf16_lo(gate[e])), b = act_grad<ACT>(bf16_hi(gate[e]));
        dg[e] = bf16x2_rne(dh[2 * e] * bf16_lo(up[e]) * a.df, dh[2 * e + 1] * bf16_hi(up[e]) * b.df);
        du[e] = bf16x2_rne(dh[2 * e] * a.f, dh[2 * e + 1] * b.f);
    }
}

// gated_small.hip: the same products where the large tiles leave most of the chip idle.
int launch_gated_small(int fmt, const GatedArgs& g, void* hip_stream);
int launch_gated_backward_small(int fmt, const GatedBackArgs& g, void* hip_stream);

}  // namespace bsq
