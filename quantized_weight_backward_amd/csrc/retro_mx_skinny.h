// retro_mx_skinny.h - the product of a few rows of A with a microscaled B: B is
// read once, straight into registers, by all CUs.
#pragma once

#include "retro_mx_device.h"

namespace retro {
namespace mx {

__device__ __forceinline__ f32x4 mfma16(const i32x4& a, const i32x4& b, const f32x4& c, int ea, int eb) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(i32x8{a[0], a[1], a[2], a[3], 0, 0, 0, 0},
                                                            i32x8{b[0], b[1], b[2], b[3], 0, 0, 0, 0}, c, 4, 4, 0, ea,
                                                            0, eb);
}

constexpr int kSkinnyWaves = 8;
constexpr int kSkinnyRows = 16;  // rows of B a workgroup

// A step's 256 elements of 16 rows: lane (r, q) holds blocks q and 4 + q of row
// r, and the words of the row's scale bytes 0-3 and 4-7 (one 64-byte and one
// 8-byte piece of a row an instruction).
struct StepRows {
    i32x4 code[2];
    u32x2 scale;
};

__device__ __forceinline__ void load_rows(StepRows& s, const uint8_t* codes, const uint8_t* scales, int q) {
    s.code[0] = *reinterpret_cast<const i32x4*>(codes + q * 16);
    s.code[1] = *reinterpret_cast<const i32x4*>(codes + 64 + q * 16);
    s.scale = *reinterpret_cast<const u32x2*>(scales);
}

// 16 rows of B times up to 16 TB rows of A, the steps of K dealt to the waves in
// turn (U at a time, so that 2 U loads of B a lane are in flight); the waves'
// sums are added in LDS in the order of the waves. The reading of B bounds it:
// T = 16, N = 4096, K = 14336 in 10.5 us traced, 3.0 TB/s. `first` is the
// launch's first workgroup of all.
template <typename TY, int TB, int U>
__global__ __launch_bounds__(kSkinnyWaves * 64, 4) void product_skinny_kernel(
    const uint8_t* __restrict__ ac, const uint8_t* __restrict__ as, const uint8_t* __restrict__ bc,
    const uint8_t* __restrict__ bs, TY* __restrict__ Y, int64_t ldy, int steps, int64_t N, int T,
    uint32_t first) {
    __shared__ float part[kSkinnyWaves][TB * 16][kSkinnyRows + 4];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
    const int r = lane & 15, q = lane >> 4;
    const int64_t n0 = int64_t(first + blockIdx.x) * kSkinnyRows, n = min(n0 + r, N - 1);
    const uint8_t* b_row = bc + n * steps * kStepBytes;
    const uint8_t* a_row[TB];
    int t[TB];
#pragma unroll
    for (int i = 0; i < TB; ++i) {
        t[i] = min(i * 16 + r, T - 1);
        a_row[i] = ac + int64_t(t[i]) * steps * kStepBytes;
    }
    f32x4 acc[TB] = {};
    for (int s0 = wave; s0 < steps; s0 += kSkinnyWaves * U) {
        StepRows b[U], a[U][TB];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = s0 + u * kSkinnyWaves;
            if (s < steps) {
                load_rows(b[u], b_row + s * kStepBytes, bs + (s * N + n) * kStepScales, q);
#pragma unroll
                for (int i = 0; i < TB; ++i)
                    load_rows(a[u][i], a_row[i] + s * kStepBytes, as + (int64_t(s) * T + t[i]) * kStepScales, q);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (s0 + u * kSkinnyWaves < steps)
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int i = 0; i < TB; ++i)
                        acc[i] = mfma16(b[u].code[k], a[u][i].code[k], acc[i], int(b[u].scale[k] >> (8 * q)),
                                        int(a[u][i].scale[k] >> (8 * q)));
    }
#pragma unroll
    for (int i = 0; i < TB; ++i) *reinterpret_cast<f32x4*>(&part[wave][i * 16 + r][4 * q]) = acc[i];
    __syncthreads();
    for (int o = threadIdx.x; o < TB * 256; o += kSkinnyWaves * 64) {
        const int tt = o / 16, c = o % 16;
        if (tt >= T || n0 + c >= N) continue;
        float y = 0.f;
#pragma unroll
        for (int w = 0; w < kSkinnyWaves; ++w) y += part[w][tt][c];
        Y[tt * ldy + n0 + c] = from_f32<TY>(y);
    }
}

// The same for T rows of A given as floats: the workgroup quantises them into
// LDS first (retro_mx_quantize's rule), while its first loads of B are on their
// way. For few elements only, since every workgroup does it. T = 1, N = 14336,
// K = 4096 in 9.0 us, 3.5 TB/s of B with the launch (8.0 traced, 6.1 at a copy's rate).
template <typename TX, int U>
__global__ __launch_bounds__(kSkinnyWaves * 64, 4) void linear_skinny_kernel(
    const TX* __restrict__ X, int64_t ldx, const uint8_t* __restrict__ bc, const uint8_t* __restrict__ bs,
    TX* __restrict__ Y, int64_t ldy, int K, int steps, int64_t N, int T, uint32_t first) {
    __shared__ float part[kSkinnyWaves][16][kSkinnyRows + 4];
    extern __shared__ __align__(16) uint8_t x_codes[];  // T x steps x 128, then the scales, T x steps x 8
    uint8_t* x_scales = x_codes + T * steps * kStepBytes;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
    const int r = lane & 15, q = lane >> 4;
    const int64_t n0 = int64_t(first + blockIdx.x) * kSkinnyRows, n = min(n0 + r, N - 1);
    const uint8_t* b_row = bc + n * steps * kStepBytes;
    StepRows b[U];
    auto load_b = [&](int s0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = s0 + u * kSkinnyWaves;
            if (s < steps) load_rows(b[u], b_row + s * kStepBytes, bs + (s * N + n) * kStepScales, q);
        }
    };
    load_b(wave);
    const int units = steps * (kStep / 8);  // of 8 elements, a multiple of 32
    for (int u = threadIdx.x; u < T * units; u += kSkinnyWaves * 64) {
        const int row = u / units, at = u - row * units, k = at * 8;
        const TX* x = X + row * ldx + k;
        float v[8];
        load8(x, K - k, v);
        uint32_t e;
        const uint32_t codes = quantize8(v, e);
        *reinterpret_cast<uint32_t*>(x_codes + u * 4) = codes;
        if ((at & 3) == 0) x_scales[u / 4] = uint8_t(e);
    }
    __syncthreads();
    const int t = min(r, T - 1);
    f32x4 acc = {};
    for (int s0 = wave; s0 < steps; s0 += kSkinnyWaves * U) {
        if (s0 != wave) load_b(s0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = s0 + u * kSkinnyWaves;
            if (s >= steps) continue;
            StepRows a;
            load_rows(a, x_codes + (t * steps + s) * kStepBytes, x_scales + (t * steps + s) * kStepScales, q);
#pragma unroll
            for (int k = 0; k < 2; ++k)
                acc = mfma16(b[u].code[k], a.code[k], acc, int(b[u].scale[k] >> (8 * q)), int(a.scale[k] >> (8 * q)));
        }
    }
    *reinterpret_cast<f32x4*>(&part[wave][r][4 * q]) = acc;
    __syncthreads();
    if (threadIdx.x < 256) {
        const int tt = threadIdx.x / 16, c = threadIdx.x % 16;
        if (tt < T && n0 + c < N) {
            float y = 0.f;
#pragma unroll
            for (int w = 0; w < kSkinnyWaves; ++w) y += part[w][tt][c];
            Y[tt * ldy + n0 + c] = from_f32<TX>(y);
        }
    }
}

}  // namespace mx
}  // namespace retro
