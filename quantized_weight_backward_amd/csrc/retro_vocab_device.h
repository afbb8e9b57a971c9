// retro_vocab_device.h - device pieces shared by the kernels of retro_vocab.h.
#pragma once

#include <type_traits>

#include "retro_mx_device.h"

namespace retro {
namespace vocab {

// 8 elements to a row's place of which `left` elements are in it.
template <typename TY>
__device__ __forceinline__ void store8(TY* to, int64_t left, const float e[8]) {
    constexpr int kPer = mx::Wide<TY>::kPer;
    if (left >= 8) {
#pragma unroll
        for (int j = 0; j < 8 / kPer; ++j) {
            typename mx::Wide<TY>::vec v;
#pragma unroll
            for (int i = 0; i < kPer; ++i) v[i] = mx::from_f32<TY>(e[j * kPer + i]);
            reinterpret_cast<typename mx::Wide<TY>::vec*>(to)[j] = v;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left) to[i] = mx::from_f32<TY>(e[i]);
}

// 8 elements as 16 bytes of E, at a 16-byte aligned place.
template <typename E>
__device__ __forceinline__ void store_part(uint16_t* to, const float e[8]) {
    typedef E vec __attribute__((ext_vector_type(8)));
    vec v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = E(e[i]);
    *reinterpret_cast<vec*>(to) = v;
}

// What E leaves of v; nothing of an infinity or NaN, which the first part is.
template <typename E>
__device__ __forceinline__ float rest_of(float v) {
    const float r = v - float(E(v));
    return __builtin_isfinite(r) ? r : 0.f;
}

// 8 elements as one or two parts that add up to them, each in a plane of its own.
template <typename E, int PARTS>
__device__ __forceinline__ void store_parts(uint16_t* to, int64_t plane, float e[8]) {
    store_part<E>(to, e);
    if constexpr (PARTS == 2) {
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = rest_of<E>(e[i]);
        store_part<E>(to + plane, e);
    }
}

// The power of two that puts a largest magnitude, given by its bits, into
// 2^13 .. 2^14: F16 then holds what is 2^28 below it with all its 11 bits, and
// products of two such rows stay far inside F32. 1 where that is no number, 2^126 where it
// would be more: its inverse is a normal number.
__device__ __forceinline__ int scale_log2(uint32_t top) {
    const int field = int(top >> 23);
    return field == 255 ? 0 : min(126, 140 - field);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }
__device__ __forceinline__ float scale_of(uint32_t top) { return pow2(scale_log2(top)); }
__device__ __forceinline__ float unscale_of(uint32_t top) { return pow2(-scale_log2(top)); }

// The largest of a wave's values, in all its lanes.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = mx::max16(v);
    v = max(v, uint32_t(__shfl_xor(int(v), 16)));
    return max(v, uint32_t(__shfl_xor(int(v), 32)));
}

// Token t's id or target, -1 where it is none.
__device__ __forceinline__ int token_at(const void* ids, bool wide, int64_t t, int64_t N) {
    const int64_t v = wide ? static_cast<const int64_t*>(ids)[t] : int64_t(static_cast<const int32_t*>(ids)[t]);
    return v >= 0 && v < N ? int(v) : -1;
}

}  // namespace vocab
}  // namespace retro
