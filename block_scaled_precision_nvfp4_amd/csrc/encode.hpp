// encode.hpp -- the block encoders that the casts and the gathers into quantized operands share: maxima over
// groups of lanes, the MXFP8 rowwise encoder of 8 elements and the NVFP4 encoder of a 16-block.
#pragma once

#include "device_common.hpp"

namespace bsq {

// Maximum of m over aligned groups of 2^lg lanes (1 <= lg <= 6, uniform), returned to every lane
// of the group, without LDS traffic: DPP quad moves (lane ^ 1, lane ^ 2), the half-row and row
// mirrors (which, once quads agree, pair each quad with the other quad of its 8 and each 8 with
// the other 8 of its row of 16), then v_permlane16_swap and v_permlane32_swap across rows.
// Every lane of the wave must be active.
template <int CTRL>
__device__ __forceinline__ float dpp_max_step(float m) {
    const int b = __builtin_bit_cast(int, m);
    return __builtin_fmaxf(m, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(b, b, CTRL, 0xF, 0xF, false)));
}

__device__ __forceinline__ float group_max_dpp(float m, int lg) {
    m = dpp_max_step<0xB1>(m);                 // quad_perm [1, 0, 3, 2]
    if (lg >= 2) m = dpp_max_step<0x4E>(m);    // quad_perm [2, 3, 0, 1]
    if (lg >= 3) m = dpp_max_step<0x141>(m);   // row_half_mirror
    if (lg >= 4) m = dpp_max_step<0x140>(m);   // row_mirror
    if (lg >= 5) {
        const uint32_t b = __builtin_bit_cast(uint32_t, m);
        const auto r = __builtin_amdgcn_permlane16_swap(b, b, false, false);
        m = __builtin_fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
    }
    if (lg >= 6) {
        const uint32_t b = __builtin_bit_cast(uint32_t, m);
        const auto r = __builtin_amdgcn_permlane32_swap(b, b, false, false);
        m = __builtin_fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
    }
    return m;
}

// Maximum of v over the wave, returned to every lane (DPP and lane swaps: no LDS round trips).
__device__ __forceinline__ float wave_max(float v) { return group_max_dpp(v, 6); }

// max(m, m of lane ^ 1), the other half of a 16-block, by a DPP quad move (a lane whose
// partner is inactive keeps its own m).
__device__ __forceinline__ float pair_max(float m) {
    const int b = __builtin_bit_cast(int, m);
    return __builtin_fmaxf(m, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(b, b, 0xB1, 0xF, 0xF, false)));
}

// ---------------------------------------------------------------- MXFP8

// Scale byte of a 32-block with amax m: X = floor(log2 m) - 8 clamped at -127, byte X+127;
// for a normal binary32 m that is max(exponent_field - 8, 0), and 0 for subnormal or zero m.
__device__ __forceinline__ uint32_t mx_scale_byte(float m) {
    const int e = (int)(__float_as_uint(m) >> 23);
    return (uint32_t)(e > 8 ? e - 8 : 0);
}

// 2^-X for scale byte b (X = b - 127): binary32 with exponent field 254 - b (b <= 246).
__device__ __forceinline__ float mx_inv_scale(uint32_t b) { return __uint_as_float((254u - b) << 23); }

// Two 16-bit lanes of a 32-bit word, unsigned or signed: packed minima and maxima
// (v_pk_max_u16, v_pk_min_u16, v_pk_min_i16).
typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));
typedef short i16x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pk_max_u16(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, a), __builtin_bit_cast(u16x2_t, b)));
}
__device__ __forceinline__ uint32_t pk_min_u16(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_min(__builtin_bit_cast(u16x2_t, a), __builtin_bit_cast(u16x2_t, b)));
}
__device__ __forceinline__ uint32_t pk_min_i16(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_min(__builtin_bit_cast(i16x2_t, a), __builtin_bit_cast(i16x2_t, b)));
}

// Four E4M3 codes (bytes 0..3: a.lo, a.hi, b.lo, b.hi) of bf16 pairs a and b divided by the
// binary32 power of two s, rounded to nearest even (v_cvt_scalef32_pk_fp8_bf16: exact for a
// normal s and quotients below 464 in magnitude; larger ones give the NaN code, so callers clamp).
__device__ __forceinline__ uint32_t fp8x4_scaled(uint32_t a, uint32_t b, float s) {
    typedef short s16x2_t __attribute__((ext_vector_type(2)));
    // the first conversion replaces the low word of a's own register; the second the high one
    s16x2_t o = __builtin_bit_cast(s16x2_t, a);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(o, __builtin_bit_cast(bf16x2_t, a), s, false);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(o, __builtin_bit_cast(bf16x2_t, b), s, true);
    return __builtin_bit_cast(uint32_t, o);
}

// Packed MXFP8 rowwise encode of an 8-element unit w[0..3] (bf16 pairs of one row) whose 32-block
// spans the 4 lanes of an aligned quad: the same codes and scale byte as the binary32 form.  The
// block amax is a 16-bit unsigned maximum over magnitude bits (within the unit, across its two
// halves, then across the quad by DPP); the clamp to 448 * 2^X and the scaled conversion are the
// columnwise encoder's.  Returns false, for every lane of the wave, when some block of the wave
// has scale byte 0 (amax exponent field <= 8, all-zero blocks included): the caller then takes the
// binary32 form.  The lanes of a quad are all active or all inactive (an inactive lane adds
// nothing: DPP reads from it return 0 and the ballot skips it).
__device__ __forceinline__ uint32_t mx_quad_amax(const uint32_t w[4]) {   // the block's amax, in both halves
    uint32_t M = pk_max_u16(pk_max_u16(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                            pk_max_u16(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
    M = pk_max_u16(M, __builtin_amdgcn_alignbit(M, M, 16));   // the unit's, in both halves
    M = pk_max_u16(M, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)M, 0xB1, 0xF, 0xF, false));   // lane ^ 1
    return pk_max_u16(M, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)M, 0x4E, 0xF, 0xF, false));   // lane ^ 2
}

constexpr uint32_t MX_PACKED_LEAST = 0x480u;   // the least amax (bf16 bits) that the packed encoder takes

__device__ __forceinline__ void mx_encode_packed(const uint32_t w[4], uint32_t M, uint32_t& lo, uint32_t& hi, uint32_t& sb) {
    const uint32_t T = (M & 0x7F807F80u) | 0x00600060u, T2 = T | 0x80008000u;
    sb = ((M >> 7) & 0xFFu) - 8u;
    const float s = __uint_as_float(sb << 23);
    uint32_t z[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) z[i] = pk_min_u16(pk_min_i16(w[i], T), T2);
    lo = fp8x4_scaled(z[0], z[1], s);
    hi = fp8x4_scaled(z[2], z[3], s);
}

__device__ __forceinline__ bool mx_row_unit_packed(const uint32_t w[4], uint32_t& lo, uint32_t& hi, uint32_t& sb) {
    const uint32_t M = mx_quad_amax(w);
    if (__builtin_amdgcn_ballot_w64((M & 0xFFFFu) < MX_PACKED_LEAST) != 0) return false;   // wave-uniform
    mx_encode_packed(w, M, lo, hi, sb);
    return true;
}

// ---------------------------------------------------------------- NVFP4

// Encode one 16-block's worth of values held by this thread (N = 8 or 16 values) whose
// largest magnitude vmax (over the block) is known.  Writes the packed codes (N/2 bytes as
// N/8 words) into w[] and returns the scale code.  first_index: output-layout index of v[0];
// consecutive values are consecutive indices.  enc_tab: the workgroup's multiplier table for
// S, or null (then the multiplier is divided out here).  QUARTER: v holds the butterfly's
// outputs h, four times the transform's values (exactly); the block is then encoded from
// h * fl(enc / 4), which equals fl((h / 4) * enc) whenever enc / 4 is exact (one rounding of
// the same product), and otherwise from (h / 4) * enc.
template <int N, bool SR, bool QUARTER>
__device__ __forceinline__ uint32_t encode_block(float* v, float vmax, float S, const float* enc_tab,
                                                 uint64_t first_index, uint64_t seed, uint32_t stream, uint32_t dir,
                                                 uint32_t* w) {
    const uint32_t sb = block_scale_code(QUARTER ? vmax * 0.25f : vmax, S);
#pragma unroll
    for (int i = 0; i < N / 8; ++i) w[i] = 0u;
    if (sb != 0u) {
        float enc = enc_tab ? enc_tab[sb] : S / e4m3_decode_nonneg(sb);
        if (QUARTER) {
            const float e4 = enc * 0.25f;
            if (e4 * 4.0f == enc) {
                enc = e4;
            } else {
#pragma unroll
                for (int j = 0; j < N; ++j) v[j] *= 0.25f;
            }
        }
        if (SR) {
#pragma unroll
            for (int g = 0; g < N / 4; ++g) {
                const u32x4 rw = sr_words((first_index >> 2) + g, seed, stream, dir);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = 4 * g + e;
                    const uint32_t c = e2m1_encode_sr(v[j] * enc, word_of(rw, e));
                    w[j >> 3] |= c << (4 * (j & 7));
                }
            }
        } else {
            static_for<0, N / 8>([&](auto g_c) {
                constexpr int g = decltype(g_c)::value;
                uint32_t x = 0;
                x = e2m1_pack2_rne<0>(x, v[8 * g + 0] * enc, v[8 * g + 1] * enc);
                x = e2m1_pack2_rne<1>(x, v[8 * g + 2] * enc, v[8 * g + 3] * enc);
                x = e2m1_pack2_rne<2>(x, v[8 * g + 4] * enc, v[8 * g + 5] * enc);
                x = e2m1_pack2_rne<3>(x, v[8 * g + 6] * enc, v[8 * g + 7] * enc);
                w[g] = x;
            });
        }
    }
    return sb;
}

}  // namespace bsq
