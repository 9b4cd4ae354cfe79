// ep_wave.h -- wave64 reductions and bf16 conversions shared by the router,
// the experts' products and the gradients.
#pragma once

#include "ep_device.h"

namespace ep {

// One data-parallel-primitive step: the value of another lane by the control
// CTRL, `old` where that lane does not exist.
template <int CTRL>
__device__ __forceinline__ float dpp(float v, float old) {
    return __int_as_float(
        __builtin_amdgcn_update_dpp(__float_as_int(old), __float_as_int(v), CTRL, 0xf, 0xf, false));
}
constexpr int kRowShr1 = 0x111, kRowShr2 = 0x112, kRowShr4 = 0x114, kRowShr8 = 0x118;
constexpr int kRowBcast15 = 0x142, kRowBcast31 = 0x143;

__device__ __forceinline__ float read_lane_f(float v, int src) {
    return __int_as_float(read_lane(__float_as_int(v), src));
}

// Maximum and sum over the wave's 64 lanes, the same value in every lane: a
// scan inside each row of 16 lanes, then the rows' totals; the sum's order is
// fixed.
__device__ __forceinline__ float wave_max(float v) {
    v = fmaxf(v, dpp<kRowShr1>(v, v));
    v = fmaxf(v, dpp<kRowShr2>(v, v));
    v = fmaxf(v, dpp<kRowShr4>(v, v));
    v = fmaxf(v, dpp<kRowShr8>(v, v));
    v = fmaxf(v, dpp<kRowBcast15>(v, v));
    v = fmaxf(v, dpp<kRowBcast31>(v, v));
    return read_lane_f(v, 63);
}
__device__ __forceinline__ float wave_sum(float v) {
    v += dpp<kRowShr1>(v, 0.0f);
    v += dpp<kRowShr2>(v, 0.0f);
    v += dpp<kRowShr4>(v, 0.0f);
    v += dpp<kRowShr8>(v, 0.0f);
    v += dpp<kRowBcast15>(v, 0.0f);
    v += dpp<kRowBcast31>(v, 0.0f);
    return read_lane_f(v, 63);
}

__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        const int lane = lane_id();
        const int lo = shfl(__double2loint(v), lane ^ d), hi = shfl(__double2hiint(v), lane ^ d);
        v = fmax(v, __hiloint2double(hi, lo));
    }
    return v;
}

__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// Round to nearest even, NaN kept quiet.
__device__ __forceinline__ uint32_t to_bf16(float f) {
    const uint32_t u = __float_as_uint(f);
    if ((u & 0x7fffffffu) > 0x7f800000u) return ((u >> 16) | 0x40u) & 0xffffu;
    return (u + 0x7fffu + ((u >> 16) & 1u)) >> 16;
}
// Two values to a packed pair (one conversion instruction on CDNA4), rounded
// as above.
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const bf16x2 r = __builtin_convertvector((f32x2){a, b}, bf16x2);
    return __builtin_bit_cast(uint32_t, r);
}

}  // namespace ep
