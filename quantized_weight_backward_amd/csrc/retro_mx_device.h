// retro_mx_device.h - device pieces shared by the microscaled 4-bit kernels
// and the expert layer: float loads and stores, the block scale, and the
// addresses of a microscaled matrix (layout: retro_mx.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace retro {
namespace mx {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

constexpr int kStep = 256;       // elements of a codes/scales step along K
constexpr int kStepBytes = 128;  // its code bytes in a row
constexpr int kStepScales = 8;   // its scale bytes in a row

// 256-element steps of a row
__host__ __device__ inline int64_t steps_of(int64_t K) { return (K + kStep - 1) / kStep; }

// 2^(e - 127) for a scale byte e below 255 (2^-127 is subnormal).
__device__ __forceinline__ float scale_value(uint32_t e) { return __uint_as_float(e ? e << 23 : 0x00400000u); }

// The scale byte of a block from the largest magnitude's bits: the exponent
// field of amax less 2 (a subnormal amax, field 0, gives 0, as does amax = 0);
// an infinity or NaN, whose bits are the largest of all, gives 255.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
    const uint32_t field = amax_bits >> 23;
    return field == 255u ? 255u : field > 2u ? field - 2u : 0u;
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(_Float16 v) { return float(v); }
__device__ __forceinline__ float to_f32(__bf16 v) { return float(v); }

template <typename T> __device__ __forceinline__ T from_f32(float v) { return T(v); }

// Two values to a byte of E2M1 codes, a in the low nibble: v / scale rounded to
// nearest even, saturated to 6. The conversion takes only the scale's exponent.
template <int BYTE>
__device__ __forceinline__ uint32_t to_fp4(uint32_t old, float a, float b, float scale) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, a, b, scale, BYTE);
}

// The value of the lane whose number differs in one bit.
template <int BIT>
__device__ __forceinline__ uint32_t swap_lanes(uint32_t v) {
    if constexpr (BIT == 1) return uint32_t(__builtin_amdgcn_mov_dpp(int(v), 0xB1, 0xf, 0xf, true));  // 1 0 3 2
    if constexpr (BIT == 2) return uint32_t(__builtin_amdgcn_mov_dpp(int(v), 0x4E, 0xf, 0xf, true));  // 2 3 0 1
    if constexpr (BIT == 4) {
        // eights mirrored, then each four mirrored back
        const int m = __builtin_amdgcn_mov_dpp(int(v), 0x141, 0xf, 0xf, true);
        return uint32_t(__builtin_amdgcn_mov_dpp(m, 0x1B, 0xf, 0xf, true));
    }
}

// The largest of 16 neighbouring lanes' values, in all of them: exchanges in
// pairs, in fours, and of the halves' mirror images.
__device__ __forceinline__ uint32_t max16(uint32_t v) {
    v = max(v, swap_lanes<1>(v));
    v = max(v, swap_lanes<2>(v));
    v = max(v, uint32_t(__builtin_amdgcn_mov_dpp(int(v), 0x141, 0xf, 0xf, true)));  // half rows mirrored
    v = max(v, uint32_t(__builtin_amdgcn_mov_dpp(int(v), 0x140, 0xf, 0xf, true)));  // rows mirrored
    return v;
}

// 16 bytes of elements at whatever alignment they have: memory accesses take any.
template <typename TX>
struct Wide {
    static constexpr int kPer = 16 / sizeof(TX);
    typedef TX vec __attribute__((ext_vector_type(16 / sizeof(TX)), aligned(sizeof(TX))));
};

// 8 elements of a row, the first `left` of them (zeros past them).
template <typename TX>
__device__ __forceinline__ void load8(const TX* x, int64_t left, float v[8]) {
    constexpr int kPer = Wide<TX>::kPer;
    if (left >= 8) {
#pragma unroll
        for (int j = 0; j < 8 / kPer; ++j) {
            const auto w = reinterpret_cast<const typename Wide<TX>::vec*>(x)[j];
#pragma unroll
            for (int i = 0; i < kPer; ++i) v[j * kPer + i] = to_f32(w[i]);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < left ? to_f32(x[i]) : 0.f;
}

// A quarter of a block of 32: four neighbouring lanes, each with its 8 elements,
// agree on the scale byte `e`; returns the lane's 8 codes.
__device__ __forceinline__ uint32_t quantize8(const float v[8], uint32_t& e) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i]));
    m = max(m, swap_lanes<1>(m));
    m = max(m, swap_lanes<2>(m));
    e = scale_byte(m);
    const float s = scale_value(e);
    uint32_t q = to_fp4<0>(0, v[0], v[1], s);
    q = to_fp4<1>(q, v[2], v[3], s);
    q = to_fp4<2>(q, v[4], v[5], s);
    return to_fp4<3>(q, v[6], v[7], s);
}

}  // namespace mx
}  // namespace retro
