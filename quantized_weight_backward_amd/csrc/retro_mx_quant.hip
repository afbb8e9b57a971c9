// retro_mx_quant.hip - quantisation to microscaled 4-bit matrices and packed
// MXFP4 / NVFP4 blocks, and their decode (retro_mx.h).
#include "retro_mx_device.h"
#include "retro_mx_host.h"

namespace retro {
namespace mx {
namespace {

constexpr int kThreads = 256;

// All of these read X once and write 17 bytes for 32 elements, with a few integer
// operations and half a conversion instruction an element: memory bounds them.

// Rows: a thread takes 8 elements of a row, four neighbouring threads share a
// block of 32 and exchange its largest magnitude. 4096 x 14336 BF16: 28 us, 5.3
// TB/s; 16 x 14336: 2.4 us traced, a launch.
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

constexpr int kTileRows = 256, kTileCols = 128;  // a workgroup's part of X
constexpr int kTileWaves = 8;                    // each 32 rows
constexpr int kColPitch = kStepBytes + 16;

// Two neighbouring elements of a row, at whatever alignment the row has.
template <typename TX>
struct __attribute__((packed, aligned(sizeof(TX)))) Pair {
    TX a, b;
};

// 32 rows of two columns in a lane. F32 values are held as such, 16-bit ones as
// loaded, two to a register: magnitudes compare as integers, and the conversions
// take 16-bit pairs.
template <typename TX>
struct Columns {
    float v[2][32];
    __device__ __forceinline__ void set(int i, Pair<TX> p) {
        v[0][i] = p.a;
        v[1][i] = p.b;
    }
    __device__ __forceinline__ void largest(uint32_t m[2]) const {
        m[0] = m[1] = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            m[0] = max(m[0], abs_bits(v[0][i]));
            m[1] = max(m[1], abs_bits(v[1][i]));
        }
    }
    // The larger of row i's two magnitudes, in an order that of_row undoes.
    __device__ __forceinline__ uint32_t row(int i) const { return max(abs_bits(v[0][i]), abs_bits(v[1][i])); }
    static __device__ __forceinline__ uint32_t of_row(uint32_t m) { return m; }
    // Codes of rows i and i + 1 of column j, and of row i's two columns, as a byte.
    template <int BYTE>
    __device__ __forceinline__ uint32_t down(uint32_t old, int j, int i, float s) const {
        return to_fp4<BYTE>(old, v[j][i], v[j][i + 1], s);
    }
    template <int BYTE>
    __device__ __forceinline__ uint32_t across(uint32_t old, int i, float s) const {
        return to_fp4<BYTE>(old, v[0][i], v[1][i], s);
    }
};

__device__ __forceinline__ float half_of(uint32_t bits, const __bf16*) { return __uint_as_float(bits << 16); }
__device__ __forceinline__ float half_of(uint32_t bits, const _Float16*) {
    return float(__builtin_bit_cast(_Float16, uint16_t(bits)));
}
template <int BYTE>
__device__ __forceinline__ uint32_t pair_to_fp4(uint32_t old, uint32_t two, float s, const __bf16*) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, __builtin_bit_cast(bf16x2, two), s, BYTE);
}
template <int BYTE>
__device__ __forceinline__ uint32_t pair_to_fp4(uint32_t old, uint32_t two, float s, const _Float16*) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(old, __builtin_bit_cast(f16x2, two), s, BYTE);
}

template <typename TX>
struct Columns16 {
    uint32_t x[32];
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    __device__ __forceinline__ void set(int i, Pair<TX> p) { x[i] = __builtin_bit_cast(uint32_t, p); }
    __device__ __forceinline__ void largest(uint32_t m[2]) const {
        u16x2 both = {0, 0};
#pragma unroll
        for (int i = 0; i < 32; ++i)
            both = __builtin_elementwise_max(both, __builtin_bit_cast(u16x2, x[i] & 0x7fff7fffu));
        m[0] = __float_as_uint(half_of(both[0], static_cast<const TX*>(nullptr)));
        m[1] = __float_as_uint(half_of(both[1], static_cast<const TX*>(nullptr)));
    }
    __device__ __forceinline__ uint32_t row(int i) const { return max(x[i] & 0x7fffu, (x[i] >> 16) & 0x7fffu); }
    static __device__ __forceinline__ uint32_t of_row(uint32_t m) {
        return __float_as_uint(half_of(m, static_cast<const TX*>(nullptr)));
    }
    template <int BYTE>
    __device__ __forceinline__ uint32_t down(uint32_t old, int j, int i, float s) const {
        const uint32_t two = __builtin_amdgcn_perm(x[i + 1], x[i], j ? 0x07060302u : 0x05040100u);
        return pair_to_fp4<BYTE>(old, two, s, static_cast<const TX*>(nullptr));
    }
    template <int BYTE>
    __device__ __forceinline__ uint32_t across(uint32_t old, int i, float s) const {
        return pair_to_fp4<BYTE>(old, x[i], s, static_cast<const TX*>(nullptr));
    }
};
template <> struct Columns<__bf16> : Columns16<__bf16> {};
template <> struct Columns<_Float16> : Columns16<_Float16> {};

// Lane I's value of each 16 lanes, in all of them.
template <int I>
__device__ __forceinline__ uint32_t from16(uint32_t v) {
    return uint32_t(__builtin_amdgcn_mov_dpp(int(v), 0x150 + I, 0xf, 0xf, true));
}

// Rows 4 G .. 4 G + 3 of `c`, a byte each, and the lanes' scale words of 16 rows.
template <int G, typename TX>
__device__ __forceinline__ uint32_t across4(const Columns<TX>& c, uint32_t scales) {
    constexpr int L = 4 * G % 16;
    uint32_t w = c.template across<0>(0, 4 * G, __uint_as_float(from16<L>(scales)));
    w = c.template across<1>(w, 4 * G + 1, __uint_as_float(from16<L + 1>(scales)));
    w = c.template across<2>(w, 4 * G + 2, __uint_as_float(from16<L + 2>(scales)));
    return c.template across<3>(w, 4 * G + 3, __uint_as_float(from16<L + 3>(scales)));
}

// Columns, or columns and rows from one reading of X. A wave takes 32 rows, a
// lane two neighbouring columns of them: a column's block lies in one lane, a
// row's in 16 lanes, of which lane j keeps the scales of rows j and 16 + j. 256
// rows make whole 128-byte steps of the columns' codes, which are gathered in LDS
// and written as such (and 64-byte pieces of the rows'). 2048 x 17408 BF16: columns
// 15.6 us (5.8 TB/s), both 21.7 us (5.0 TB/s; two readings take 34).
template <typename TX, bool ROWS>
__global__ __launch_bounds__(kTileWaves * 64, 4) void quantize_tile_kernel(
    const TX* __restrict__ X, int64_t ldx, int64_t rows, uint32_t cols, uint32_t groups, int64_t tile0, uint32_t col0,
    uint32_t row_steps, uint32_t col_steps, uint8_t* __restrict__ row_codes, uint8_t* __restrict__ row_scales,
    uint8_t* __restrict__ col_codes, uint8_t* __restrict__ col_scales) {
    __shared__ __align__(16) uint8_t by_col[kTileCols * kColPitch];
    __shared__ __align__(16) uint8_t col_e[kTileCols * kStepScales];
    __shared__ __align__(16) uint32_t by_row[ROWS ? kTileRows / 4 * 64 : 4];  // four rows' bytes a word
    __shared__ __align__(16) uint8_t row_e[ROWS ? kTileRows * 4 : 16];
    const int64_t tile = tile0 + blockIdx.x / groups;  // of 256 rows
    const uint32_t c0 = col0 + (blockIdx.x % groups) * kTileCols;
    const int wave = threadIdx.x / 64, lane = threadIdx.x % 64;
    const int64_t r0 = tile * kTileRows + wave * 32;
    const uint32_t c = c0 + 2 * lane;
    const int n = int(min(max(rows - r0, int64_t(0)), int64_t(32)));
    Columns<TX> v;
    const TX* x = X + r0 * ldx + c;
    if (n == 32 && c0 + kTileCols <= cols) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v.set(i, *reinterpret_cast<const Pair<TX>*>(x + i * ldx));
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            Pair<TX> p = {TX(0.f), TX(0.f)};
            if (i < n && c < cols) p.a = x[i * ldx];
            if (i < n && c + 1 < cols) p.b = x[i * ldx + 1];
            v.set(i, p);
        }
    }
    uint32_t m[2];
    v.largest(m);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint32_t e = scale_byte(m[j]);
        const float s = scale_value(e);
        u32x4 q;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t w = v.template down<0>(0, j, 8 * i, s);
            w = v.template down<1>(w, j, 8 * i + 2, s);
            w = v.template down<2>(w, j, 8 * i + 4, s);
            q[i] = v.template down<3>(w, j, 8 * i + 6, s);
        }
        *reinterpret_cast<u32x4*>(by_col + (2 * lane + j) * kColPitch + wave * 16) = q;
        col_e[(2 * lane + j) * kStepScales + wave] = uint8_t(e);
    }
    if constexpr (ROWS) {
        uint32_t scales[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t mine = 0;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const uint32_t of_row = max16(v.row(16 * half + i));
                mine = (lane & 15) == i ? of_row : mine;
            }
            const uint32_t e = scale_byte(Columns<TX>::of_row(mine));
            scales[half] = __float_as_uint(scale_value(e));
            row_e[(wave * 32 + 16 * half + (lane & 15)) * 4 + lane / 16] = uint8_t(e);
        }
        uint32_t* w = by_row + wave * 8 * 64 + lane;
        w[0 * 64] = across4<0>(v, scales[0]);
        w[1 * 64] = across4<1>(v, scales[0]);
        w[2 * 64] = across4<2>(v, scales[0]);
        w[3 * 64] = across4<3>(v, scales[0]);
        w[4 * 64] = across4<4>(v, scales[1]);
        w[5 * 64] = across4<5>(v, scales[1]);
        w[6 * 64] = across4<6>(v, scales[1]);
        w[7 * 64] = across4<7>(v, scales[1]);
    }
    __syncthreads();
    for (int o = threadIdx.x; o < kTileCols * 8; o += kTileWaves * 64) {
        const uint32_t cc = o / 8, part = o % 8;
        if (c0 + cc < cols)
            *reinterpret_cast<u32x4*>(col_codes + (int64_t(c0 + cc) * col_steps + tile) * kStepBytes + part * 16) =
                *reinterpret_cast<const u32x4*>(by_col + cc * kColPitch + part * 16);
    }
    if (threadIdx.x < kTileCols && c0 + threadIdx.x < cols)
        *reinterpret_cast<u32x2*>(col_scales + (tile * cols + c0 + threadIdx.x) * kStepScales) =
            *reinterpret_cast<const u32x2*>(col_e + threadIdx.x * kStepScales);
    if constexpr (ROWS) {
        const int64_t t0 = tile * kTileRows;
        for (int o = threadIdx.x; o < kTileRows / 4 * 16; o += kTileWaves * 64) {
            // words of four lanes, a byte a row: transposed to a word of each row
            const int four = o / 16, part = o % 16;
            const u32x4 w = *reinterpret_cast<const u32x4*>(by_row + four * 64 + part * 4);
            const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u);
            const uint32_t b = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u);
            const uint32_t d = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u);
            const uint32_t e = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
            const uint32_t out[4] = {
                __builtin_amdgcn_perm(b, a, 0x05040100u), __builtin_amdgcn_perm(b, a, 0x07060302u),
                __builtin_amdgcn_perm(e, d, 0x05040100u), __builtin_amdgcn_perm(e, d, 0x07060302u)};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (t0 + 4 * four + j < rows)
                    *reinterpret_cast<uint32_t*>(row_codes + (t0 + 4 * four + j) * row_steps * kStepBytes + c0 / 2 +
                                                 part * 4) = out[j];
        }
        if (threadIdx.x < kTileRows && t0 + threadIdx.x < rows)
            *reinterpret_cast<uint32_t*>(row_scales + (int64_t(c0 / kStep) * rows + t0 + threadIdx.x) * kStepScales +
                                         (c0 % kStep) / 32) =
                *reinterpret_cast<const uint32_t*>(row_e + threadIdx.x * 4);
    }
}

// 16 bytes of neighbouring elements of a row.
template <typename TX, int PER>
__device__ __forceinline__ void load_few(const TX* x, float v[PER]) {
    const auto w = *reinterpret_cast<const typename Wide<TX>::vec*>(x);
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] = to_f32(w[i]);
}

// Words at any byte address.
struct __attribute__((packed)) AnyWord {
    uint32_t w;
};

// Packed MXFP4 blocks: a lane takes 16 bytes of X, 8 (F32) or 4 lanes a block.
// A lane of the first half of a block has the low nibbles of its bytes, the lane
// half a block on their high ones. 17408 x 5120 F32: 71 us, 5.7 TB/s (74 traced).
template <typename TX>
__global__ __launch_bounds__(kThreads) void quantize_mxfp4_kernel(const TX* __restrict__ X, int64_t ldx, uint32_t rows,
                                                                  uint32_t units, uint8_t* __restrict__ W) {
    constexpr int PER = 16 / sizeof(TX), kLanes = 32 / PER;
    const uint32_t u = blockIdx.x * kThreads + threadIdx.x;
    const uint32_t row = u / units, at = u - row * units;
    if (row >= rows) return;  // whole blocks: units is a multiple of kLanes
    float v[PER];
    load_few<TX, PER>(X + int64_t(row) * ldx + int64_t(at) * PER, v);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) m = max(m, abs_bits(v[i]));
    m = max(m, swap_lanes<1>(m));
    if (kLanes > 2) m = max(m, swap_lanes<2>(m));
    if (kLanes > 4) m = max(m, swap_lanes<4>(m));
    const uint32_t e = scale_byte(m), lane = at % kLanes;
    const float s = scale_value(e);
    uint8_t* w = W + (int64_t(row) * (units / kLanes) + at / kLanes) * 17;
    if (lane == 0) w[0] = uint8_t(e);
#pragma unroll
    for (int i = 0; i < PER; i += 4) {
        // one code a byte, with the other half's in the nibble above
        uint32_t mine = 0;
        mine = to_fp4<0>(mine, v[i], 0.f, s);
        mine = to_fp4<1>(mine, v[i + 1], 0.f, s);
        mine = to_fp4<2>(mine, v[i + 2], 0.f, s);
        mine = to_fp4<3>(mine, v[i + 3], 0.f, s);
        const uint32_t other = swap_lanes<kLanes / 2>(mine);
        if (lane < kLanes / 2)
            reinterpret_cast<AnyWord*>(w + 1 + lane * PER + i)->w = mine | other << 4;
    }
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
// would round; a middle itself goes to the even code. Three comparisons find the
// code's bits from the top.
__device__ __forceinline__ uint32_t nvfp4_code(float v, float S) {
    const float a = fabsf(v);
    const bool b2 = a >= 1.75f * S;
    const bool b1 = a >= (b2 ? 3.5f : 0.75f) * S;
    const float last = b2 ? (b1 ? 5.0f : 2.5f) : (b1 ? 1.25f : 0.25f);
    const bool b0 = a > last * S;
    const uint32_t c = S > 0.f ? uint32_t(b2) * 4 + uint32_t(b1) * 2 + uint32_t(b0) : 0u;
    return c | (__float_as_uint(v) >> 31 << 3);
}

// Packed NVFP4 blocks: a lane takes 16 bytes of X, 4 (F32) or 2 lanes a
// sub-block of 16, nibbles as above. 17408 x 5120 F32: 89 us, 4.6 TB/s, in calls one
// after another, 107 traced one launch at a time (the exact comparisons keep the
// vector units busy as long as memory takes).
template <typename TX>
__global__ __launch_bounds__(kThreads) void quantize_nvfp4_kernel(const TX* __restrict__ X, int64_t ldx, uint32_t rows,
                                                                  uint32_t units, uint8_t* __restrict__ W) {
    constexpr int PER = 16 / sizeof(TX), kLanes = 16 / PER;
    const uint32_t u = blockIdx.x * kThreads + threadIdx.x;
    const uint32_t row = u / units, at = u - row * units;
    if (row >= rows) return;
    float v[PER];
    load_few<TX, PER>(X + int64_t(row) * ldx + int64_t(at) * PER, v);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) m = max(m, abs_bits(v[i]));
    m = max(m, swap_lanes<1>(m));
    if (kLanes > 2) m = max(m, swap_lanes<2>(m));
    if (kLanes > 4) m = max(m, swap_lanes<4>(m));
    const uint32_t e = e4m3_scale(m), lane = at % kLanes, sub = at / kLanes;
    const float S = __builtin_amdgcn_cvt_f32_fp8(int(e), 0);
    uint8_t* w = W + (int64_t(row) * (units / (4 * kLanes)) + sub / 4) * 36;
    if (lane == 0) w[sub & 3] = uint8_t(e);
    // rows of 36-byte blocks are 4-byte aligned
    uint32_t* d = reinterpret_cast<uint32_t*>(w + 4 + 8 * (sub & 3) + lane * PER);
#pragma unroll
    for (int i = 0; i < PER; i += 4) {
        const uint32_t mine = nvfp4_code(v[i], S) | nvfp4_code(v[i + 1], S) << 8 | nvfp4_code(v[i + 2], S) << 16 |
                              nvfp4_code(v[i + 3], S) << 24;
        const uint32_t other = swap_lanes<kLanes / 2>(mine);
        if (lane < kLanes / 2) d[i / 4] = mine | other << 4;
    }
}

// Values of a microscaled matrix: a thread 8 elements of a row. 4096 x 14336 to
// BF16: 26 us, 5.7 TB/s.
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
    constexpr int kPer = Wide<TY>::kPer;
    if (k + 8 <= K) {
#pragma unroll
        for (int j = 0; j < 8 / kPer; ++j) {
            typename Wide<TY>::vec o;
#pragma unroll
            for (int i = 0; i < kPer; ++i) o[i] = from_f32<TY>(v[(j * kPer + i) / 2][i % 2] * s);
            reinterpret_cast<typename Wide<TY>::vec*>(y)[j] = o;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (k + i < K) y[i] = from_f32<TY>(v[i / 2][i % 2] * s);
}

// Packed MXFP4 blocks to a microscaled matrix: a thread a block of 32 (past K:
// zeros). The nibbles change from (j, j + 16) to neighbours. The 17-byte blocks are
// read by bytes, which the caches gather: 17408 x 5120 in 17.5 us, 5.4 TB/s of the 95
// MB read and written.
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

template <bool ROWS, typename TX>
int launch_tiles(const TX* X, int64_t ldx, int64_t rows, int64_t cols, uint8_t* row_codes, uint8_t* row_scales,
                 uint8_t* col_codes, uint8_t* col_scales, hipStream_t st) {
    // with rows wanted the columns' padding is written too
    const int64_t tiles = steps_of(rows), all = ROWS ? steps_of(cols) * 2 : host::cdiv(cols, kTileCols);
    for (int64_t g = 0; g < all; g += kMaxBlocks) {
        const int64_t groups = std::min(all - g, kMaxBlocks), most = kMaxBlocks / groups;
        for (int64_t b = 0; b < tiles; b += most) {
            const int64_t n = std::min(most, tiles - b);
            host::clear_last_error();
            quantize_tile_kernel<TX, ROWS><<<dim3(uint32_t(n * groups)), dim3(kTileWaves * 64), 0, st>>>(
                X, ldx, rows, uint32_t(cols), uint32_t(groups), b, uint32_t(g * kTileCols), uint32_t(steps_of(cols)),
                uint32_t(tiles), row_codes, row_scales, col_codes, col_scales);
            const int rc = host::launch_status();
            if (rc != RETRO_OK) return rc;
        }
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
        const int64_t units = K / (16 / int64_t(sizeof(TX))), rb = host::row_bytes_of(type, K);
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
    if (!col_codes) return launch_quantize_rows(xtype, X, ldx, rows, cols, row_codes, row_scales, st);
    return with_float(xtype, [&](auto* tag) {
        using TX = std::remove_pointer_t<decltype(tag)>;
        const TX* x = static_cast<const TX*>(X);
        uint8_t *rc = static_cast<uint8_t*>(row_codes), *rs = static_cast<uint8_t*>(row_scales),
                *cc = static_cast<uint8_t*>(col_codes), *cs = static_cast<uint8_t*>(col_scales);
        return row_codes ? launch_tiles<true>(x, ldx, rows, cols, rc, rs, cc, cs, st)
                         : launch_tiles<false>(x, ldx, rows, cols, rc, rs, cc, cs, st);
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
