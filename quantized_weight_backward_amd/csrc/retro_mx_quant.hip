// retro_mx_quant.hip - quantisation to microscaled 4-bit matrices and packed
// MXFP4 / NVFP4 blocks, and their decode (retro_mx.h).
#include "retro_mx_device.h"
#include "retro_mx_host.h"

namespace retro {
namespace mx {
namespace {

constexpr int kThreads = 256;

// Rows: a thread takes 8 elements of a row, four neighbouring threads share a
// block of 32 and exchange its largest magnitude.
template <typename TX>
__global__ __launch_bounds__(kThreads) void quantize_rows_kernel(const TX* __restrict__ X, int64_t ldx, uint32_t rows,
                                                                 int64_t all_rows, uint32_t K, uint32_t units,
                                                                 uint8_t* __restrict__ codes,
                                                                 uint8_t* __restrict__ scales) {
    const uint32_t u = blockIdx.x * kThreads + threadIdx.x;
    const uint32_t row = u / units, k = (u - row * units) * 8;
    if (row >= rows) return;  // whole blocks: units is a multiple of 32
    float v[8];
    load8(X + int64_t(row) * ldx + k, int64_t(K) - k, v);
    uint32_t e;
    const uint32_t q = quantize8(v, e);
    *reinterpret_cast<uint32_t*>(codes + int64_t(row) * units * 4 + k / 2) = q;
    if ((k & 31) == 0)
        scales[(int64_t(k / kStep) * all_rows + row) * kStepScales + (k % kStep) / 32] = uint8_t(e);
}

// Columns: a thread takes the block of 32 rows of one column.
template <typename TX>
__global__ __launch_bounds__(kThreads) void quantize_cols_kernel(const TX* __restrict__ X, int64_t ldx, int64_t rows,
                                                                 uint32_t cols, uint32_t col_groups, uint32_t steps,
                                                                 int64_t block0, uint8_t* __restrict__ codes,
                                                                 uint8_t* __restrict__ scales) {
    const int64_t tb = block0 + blockIdx.x / col_groups;  // block of 32 rows
    const uint32_t c = (blockIdx.x % col_groups) * kThreads + threadIdx.x;
    if (c >= cols) return;
    const TX* x = X + tb * 32 * ldx + c;
    const int n = int(min(int64_t(32), rows - tb * 32));  // may be negative: a padded block
    float v[32];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        v[i] = i < n ? to_f32(x[int64_t(i) * ldx]) : 0.f;
        m = max(m, abs_bits(v[i]));
    }
    const uint32_t e = scale_byte(m);
    const float s = scale_value(e);
    u32x4 q;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t w = to_fp4<0>(0, v[8 * i], v[8 * i + 1], s);
        w = to_fp4<1>(w, v[8 * i + 2], v[8 * i + 3], s);
        w = to_fp4<2>(w, v[8 * i + 4], v[8 * i + 5], s);
        q[i] = to_fp4<3>(w, v[8 * i + 6], v[8 * i + 7], s);
    }
    *reinterpret_cast<u32x4*>(codes + int64_t(c) * steps * kStepBytes + tb * 16) = q;
    scales[(tb / 8 * cols + c) * kStepScales + tb % 8] = uint8_t(e);
}

// Packed MXFP4 blocks: a thread a block.
template <typename TX>
__global__ __launch_bounds__(kThreads) void quantize_mxfp4_kernel(const TX* __restrict__ X, int64_t ldx, uint32_t rows,
                                                                  uint32_t blocks, uint8_t* __restrict__ W) {
    const uint32_t u = blockIdx.x * kThreads + threadIdx.x;
    const uint32_t row = u / blocks, b = u - row * blocks;
    if (row >= rows) return;
    const TX* x = X + int64_t(row) * ldx + int64_t(b) * 32;
    float v[32];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        v[i] = to_f32(x[i]);
        m = max(m, abs_bits(v[i]));
    }
    const uint32_t e = scale_byte(m);
    const float s = scale_value(e);
    uint8_t* w = W + (int64_t(row) * blocks + b) * 17;
    w[0] = uint8_t(e);
#pragma unroll
    for (int i = 0; i < 16; ++i) w[1 + i] = uint8_t(to_fp4<0>(0, v[i], v[16 + i], s));
}

// The E4M3 scale of a sub-block nearest to amax / 6. The quotient in F32 is
// never on the middle of two E4M3 values unless amax / 6 is: 6 times such a
// middle is exact, so another amax is at least 2^-24 of it away, more than the
// half ulp that the division rounds by.
__device__ __forceinline__ uint32_t e4m3_scale(uint32_t amax_bits) {
    if (amax_bits >= 0x7f800000u) return 0x7fu;
    const float v = fminf(__uint_as_float(amax_bits) / 6.0f, 448.0f);
    return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(v, v, 0, false)) & 0xffu;
}

// |v| / S to the nearest E2M1 code: |v| against S times the middles of the
// grid, products of at most 7 bits and therefore exact, where the quotient
// would round. A middle itself goes to the even code.
__device__ __forceinline__ uint32_t nvfp4_code(float v, float S) {
    const float a = fabsf(v);
    uint32_t c = uint32_t(a > 0.25f * S) + uint32_t(a >= 0.75f * S) + uint32_t(a > 1.25f * S) +
                 uint32_t(a >= 1.75f * S) + uint32_t(a > 2.5f * S) + uint32_t(a >= 3.5f * S) +
                 uint32_t(a > 5.0f * S);
    c = S > 0.f ? c : 0u;
    return c | (__float_as_uint(v) >> 31 << 3);
}

// Packed NVFP4 blocks: a thread a sub-block of 16.
template <typename TX>
__global__ __launch_bounds__(kThreads) void quantize_nvfp4_kernel(const TX* __restrict__ X, int64_t ldx, uint32_t rows,
                                                                  uint32_t subs, uint8_t* __restrict__ W) {
    const uint32_t u = blockIdx.x * kThreads + threadIdx.x;
    const uint32_t row = u / subs, b = u - row * subs;
    if (row >= rows) return;
    const TX* x = X + int64_t(row) * ldx + int64_t(b) * 16;
    float v[16];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        v[i] = to_f32(x[i]);
        m = max(m, abs_bits(v[i]));
    }
    const uint32_t e = e4m3_scale(m);
    const float S = __builtin_amdgcn_cvt_f32_fp8(int(e), 0);
    uint8_t* w = W + (int64_t(row) * subs + (b & ~3u)) / 4 * 36;
    w[b & 3] = uint8_t(e);
    uint32_t lo = 0, hi = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        lo |= (nvfp4_code(v[i], S) | nvfp4_code(v[8 + i], S) << 4) << (8 * i);
        hi |= (nvfp4_code(v[4 + i], S) | nvfp4_code(v[12 + i], S) << 4) << (8 * i);
    }
    // rows of 36-byte blocks are 4-byte aligned
    uint32_t* d = reinterpret_cast<uint32_t*>(w + 4 + 8 * (b & 3));
    d[0] = lo;
    d[1] = hi;
}

// Values of a microscaled matrix: a thread 8 elements of a row.
template <typename TY>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(const uint8_t* __restrict__ codes,
                                                              const uint8_t* __restrict__ scales, uint32_t rows,
                                                              int64_t all_rows, uint32_t K, uint32_t units,
                                                              uint32_t row_code_bytes, TY* __restrict__ Y,
                                                              int64_t ldy) {
    const uint32_t u = blockIdx.x * kThreads + threadIdx.x;
    const uint32_t row = u / units, k = (u - row * units) * 8;
    if (row >= rows) return;
    const uint32_t q = *reinterpret_cast<const uint32_t*>(codes + int64_t(row) * row_code_bytes + k / 2);
    const uint32_t e = scales[(int64_t(k / kStep) * all_rows + row) * kStepScales + (k % kStep) / 32];
    const float s = e == 255u ? __uint_as_float(0x7fc00000u) : scale_value(e);
    f32x2 v[4];
    v[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 0);
    v[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 1);
    v[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 2);
    v[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 3);
    TY* y = Y + int64_t(row) * ldy + k;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (k + i < K) y[i] = from_f32<TY>(v[i / 2][i % 2] * s);
}

// Packed MXFP4 blocks to a microscaled matrix: a thread a block of 32 (past K:
// zeros). The nibbles change from (j, j + 16) to neighbours.
__global__ __launch_bounds__(kThreads) void from_blocks_kernel(const uint8_t* __restrict__ W, uint32_t rows,
                                                               int64_t all_rows, uint32_t blocks,
                                                               uint32_t padded_blocks, uint8_t* __restrict__ codes,
                                                               uint8_t* __restrict__ scales) {
    const uint32_t u = blockIdx.x * kThreads + threadIdx.x;
    const uint32_t row = u / padded_blocks, b = u - row * padded_blocks;
    if (row >= rows) return;
    uint32_t q[4] = {0, 0, 0, 0}, e = 0;
    if (b < blocks) {
        const uint8_t* w = W + (int64_t(row) * blocks + b) * 17;
        e = w[0];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t p = w[1 + 2 * i], n = w[2 + 2 * i];
            q[i / 4] |= ((p & 15u) | (n & 15u) << 4) << (8 * (i % 4));
            q[2 + i / 4] |= ((p >> 4) | (n >> 4) << 4) << (8 * (i % 4));
        }
    }
    u32x4 o = {q[0], q[1], q[2], q[3]};
    *reinterpret_cast<u32x4*>(codes + (int64_t(row) * padded_blocks + b) * 16) = o;
    scales[(int64_t(b / 8) * all_rows + row) * kStepScales + b % 8] = uint8_t(e);
}

// Rows in launches of at most kMaxBlocks workgroups: f(first row, rows, blocks).
template <typename F>
int in_row_ranges(int64_t rows, int64_t units, F&& f) {
    const int64_t most = std::max<int64_t>(1, kMaxBlocks * kThreads / units);
    for (int64_t r = 0; r < rows; r += most) {
        const int64_t n = std::min(most, rows - r);
        host::clear_last_error();
        f(r, uint32_t(n), uint32_t(host::cdiv(n * units, kThreads)));
        const int rc = host::launch_status();
        if (rc != RETRO_OK) return rc;
    }
    return RETRO_OK;
}

template <typename TX>
int launch_cols(const TX* X, int64_t ldx, int64_t rows, int64_t cols, uint8_t* codes, uint8_t* scales,
                hipStream_t st) {
    const int64_t steps = steps_of(rows), groups = host::cdiv(cols, kThreads);
    const int64_t most = std::max<int64_t>(1, kMaxBlocks / groups);
    for (int64_t b = 0; b < steps * 8; b += most) {
        const int64_t n = std::min(most, steps * 8 - b);
        host::clear_last_error();
        quantize_cols_kernel<TX><<<dim3(uint32_t(n * groups)), dim3(kThreads), 0, st>>>(
            X, ldx, rows, uint32_t(cols), uint32_t(groups), uint32_t(steps), b, codes, scales);
        const int rc = host::launch_status();
        if (rc != RETRO_OK) return rc;
    }
    return RETRO_OK;
}

}  // namespace

int launch_quantize_rows(int xtype, const void* X, int64_t ldx, int64_t rows, int64_t K, void* codes, void* scales,
                         hipStream_t st) {
    return with_float(xtype, [&](auto* tag) {
        using TX = std::remove_pointer_t<decltype(tag)>;
        const int64_t units = steps_of(K) * (kStep / 8);
        return in_row_ranges(rows, units, [&](int64_t r, uint32_t n, uint32_t blocks) {
            quantize_rows_kernel<TX><<<dim3(blocks), dim3(kThreads), 0, st>>>(
                static_cast<const TX*>(X) + r * ldx, ldx, n, rows, uint32_t(K), uint32_t(units),
                static_cast<uint8_t*>(codes) + r * units * 4, static_cast<uint8_t*>(scales) + r * kStepScales);
        });
    });
}

}  // namespace mx
}  // namespace retro

using namespace retro;
using namespace retro::mx;

extern "C" {

int64_t retro_mx_code_bytes(int64_t rows, int64_t K) {
    if (!dim_ok(rows) || !dim_ok(K)) return -1;
    return code_bytes(rows, K);
}

int64_t retro_mx_scale_bytes(int64_t rows, int64_t K) {
    if (!dim_ok(rows) || !dim_ok(K)) return -1;
    return scale_bytes(rows, K);
}

int retro_quantize(int type, int xtype, const void* X, int64_t ldx, void* W, int64_t K, int64_t N, void* stream) {
    const int size = float_bytes(xtype);
    if (!size || (type != RETRO_MXFP4 && type != RETRO_NVFP4)) return RETRO_E_TYPE;
    if (!dim_ok(K) || !dim_ok(N) || K % (type == RETRO_MXFP4 ? 32 : 64)) return RETRO_E_SHAPE;
    const int64_t xb = span_bytes(N, K, ldx, size);
    if (xb < 0) return RETRO_E_SHAPE;
    if (K == 0 || N == 0) return RETRO_OK;
    if (!X || !W) return RETRO_E_NULL;
    if (!aligned(W, 16) || !aligned(X, size)) return RETRO_E_ALIGN;
    if (overlap({X, xb}, {W, N * host::row_bytes_of(type, K)})) return RETRO_E_ALIAS;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    return with_float(xtype, [&](auto* tag) {
        using TX = std::remove_pointer_t<decltype(tag)>;
        const int64_t units = type == RETRO_MXFP4 ? K / 32 : K / 16, rb = host::row_bytes_of(type, K);
        return in_row_ranges(N, units, [&](int64_t r, uint32_t n, uint32_t blocks) {
            const TX* x = static_cast<const TX*>(X) + r * ldx;
            uint8_t* w = static_cast<uint8_t*>(W) + r * rb;
            if (type == RETRO_MXFP4)
                quantize_mxfp4_kernel<TX><<<dim3(blocks), dim3(kThreads), 0, st>>>(x, ldx, n, uint32_t(units), w);
            else
                quantize_nvfp4_kernel<TX><<<dim3(blocks), dim3(kThreads), 0, st>>>(x, ldx, n, uint32_t(units), w);
        });
    });
}

int retro_mx_quantize(int xtype, const void* X, int64_t ldx, int64_t rows, int64_t cols, void* row_codes,
                      void* row_scales, void* col_codes, void* col_scales, void* stream) {
    const int size = float_bytes(xtype);
    if (!size) return RETRO_E_TYPE;
    if (!dim_ok(rows) || !dim_ok(cols)) return RETRO_E_SHAPE;
    const int64_t xb = span_bytes(rows, cols, ldx, size);
    if (xb < 0) return RETRO_E_SHAPE;
    if (rows == 0 || cols == 0) return RETRO_OK;
    if (!X || !row_codes != !row_scales || !col_codes != !col_scales || (!row_codes && !col_codes))
        return RETRO_E_NULL;
    if (!aligned(X, size) || !aligned(row_codes, 16) || !aligned(row_scales, 16) || !aligned(col_codes, 16) ||
        !aligned(col_scales, 16))
        return RETRO_E_ALIGN;
    const Span spans[5] = {{X, xb},
                           {row_codes, code_bytes(rows, cols)},
                           {row_scales, scale_bytes(rows, cols)},
                           {col_codes, code_bytes(cols, rows)},
                           {col_scales, scale_bytes(cols, rows)}};
    for (int i = 0; i < 5; ++i)
        for (int j = 0; j < i; ++j)
            if (overlap(spans[i], spans[j])) return RETRO_E_ALIAS;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (row_codes) {
        const int rc = launch_quantize_rows(xtype, X, ldx, rows, cols, row_codes, row_scales, st);
        if (rc != RETRO_OK) return rc;
    }
    if (!col_codes) return RETRO_OK;
    return with_float(xtype, [&](auto* tag) {
        using TX = std::remove_pointer_t<decltype(tag)>;
        return launch_cols(static_cast<const TX*>(X), ldx, rows, cols, static_cast<uint8_t*>(col_codes),
                           static_cast<uint8_t*>(col_scales), st);
    });
}

int retro_mx_dequantize(int ytype, const void* codes, const void* scales, void* Y, int64_t ldy, int64_t K,
                        int64_t rows, void* stream) {
    const int size = float_bytes(ytype);
    if (!size) return RETRO_E_TYPE;
    if (!dim_ok(rows) || !dim_ok(K)) return RETRO_E_SHAPE;
    const int64_t yb = span_bytes(rows, K, ldy, size);
    if (yb < 0) return RETRO_E_SHAPE;
    if (K == 0 || rows == 0) return RETRO_OK;
    if (!codes || !scales || !Y) return RETRO_E_NULL;
    if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(Y, size)) return RETRO_E_ALIGN;
    if (overlap({Y, yb}, {codes, code_bytes(rows, K)}) || overlap({Y, yb}, {scales, scale_bytes(rows, K)}))
        return RETRO_E_ALIAS;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    return with_float(ytype, [&](auto* tag) {
        using TY = std::remove_pointer_t<decltype(tag)>;
        const int64_t units = host::cdiv(K, 8), rb = steps_of(K) * kStepBytes;
        return in_row_ranges(rows, units, [&](int64_t r, uint32_t n, uint32_t blocks) {
            dequantize_kernel<TY><<<dim3(blocks), dim3(kThreads), 0, st>>>(
                static_cast<const uint8_t*>(codes) + r * rb, static_cast<const uint8_t*>(scales) + r * kStepScales, n,
                rows, uint32_t(K), uint32_t(units), uint32_t(rb), static_cast<TY*>(Y) + r * ldy, ldy);
        });
    });
}

int retro_mx_from_blocks(const void* W, void* codes, void* scales, int64_t K, int64_t N, void* stream) {
    if (!dim_ok(K) || !dim_ok(N) || K % 32) return RETRO_E_SHAPE;
    if (K == 0 || N == 0) return RETRO_OK;
    if (!W || !codes || !scales) return RETRO_E_NULL;
    if (!aligned(W, 16) || !aligned(codes, 16) || !aligned(scales, 16)) return RETRO_E_ALIGN;
    const Span w{W, N * host::row_bytes_of(RETRO_MXFP4, K)}, c{codes, code_bytes(N, K)}, s{scales, scale_bytes(N, K)};
    if (overlap(w, c) || overlap(w, s) || overlap(c, s)) return RETRO_E_ALIAS;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const int64_t padded = steps_of(K) * 8;
    return in_row_ranges(N, padded, [&](int64_t r, uint32_t n, uint32_t blocks) {
        from_blocks_kernel<<<dim3(blocks), dim3(kThreads), 0, st>>>(
            static_cast<const uint8_t*>(W) + r * (K / 32) * 17, n, N, uint32_t(K / 32), uint32_t(padded),
            static_cast<uint8_t*>(codes) + r * padded * 16, static_cast<uint8_t*>(scales) + r * kStepScales);
    });
}

}  // extern "C"
