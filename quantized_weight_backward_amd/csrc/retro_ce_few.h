// retro_ce_few.h - the logits of up to 64 tokens through a packed head, read once as it
// is: codes become F16 in registers, and the matrix cores multiply them as they are.
//
//   l[t][n] = sum over sub-blocks b of 32: a[n][b] sum_k q[n][k] x[t][k] + c[n][b] sum_k x[t][k]
//
// A code q has at most 8 bits and x (scaled by a power of two, in one F16 part or two)
// 11 a part, so their products are exact; the F32 sum of a sub-block is scaled by its
// a and c as the format defines them. Tokens are the rows of a 16 x 16 block, rows of the
// head its columns: a lane decodes 8 codes of the row whose scale it applies to the four
// results that it gets.
//
// What bounds it is memory where few tokens are given: Q4_K 131072 x 4096 and 16 tokens
// take 93 us for 302 MB (Q8_0 139 for 570), against 252 us with the weights decoded to
// F32 in front of F32 matrix instructions. Half of that is decoding: 16 VALU instructions
// for the 8 codes and four results of a lane.
#pragma once

#include "retro_ce_kernel.h"
#include "retro_kernels.h"

namespace retro {
namespace ce {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32x2b __attribute__((ext_vector_type(2), aligned(1)));
typedef _Float16 f16x2v __attribute__((ext_vector_type(2)));
using mx::f32x4;
using mx::u32x4;

// Two F16 of 1024 + the bytes lo and hi of w.
template <int LO, int HI>
__device__ __forceinline__ f16x2v bytes_above_1024(uint32_t w) {
    return __builtin_bit_cast(f16x2v, __builtin_amdgcn_perm(0x64646464u, w, 0x04000400u | (HI << 16) | LO));
}

// Eight unsigned bytes less `less` as F16.
__device__ __forceinline__ f16x8 bytes_to_f16(uint32_t w0, uint32_t w1, float less) {
    const _Float16 s = _Float16(-1024.f - less);
    const f16x2v off = {s, s};
    const f16x2v v0 = bytes_above_1024<0, 1>(w0) + off, v1 = bytes_above_1024<2, 3>(w0) + off;
    const f16x2v v2 = bytes_above_1024<0, 1>(w1) + off, v3 = bytes_above_1024<2, 3>(w1) + off;
    return f16x8{v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
}

// Codes 8g .. 8g + 7 of a sub-block of 32, its factor and its offset.
struct Codes {
    f16x8 q, q2;  // q2: a second product's, where a code times its scale has more bits than one holds
    float a, c;
};

template <int TYPE>
constexpr bool kFewType = kNibbleLayout<TYPE> || TYPE == kQ8_0 || TYPE == kQ4_K || TYPE == kQ5_K || TYPE == kQ6_K;
// Whose scales pass what F32 holds above a sum of scaled x: the token's factor goes first.
template <int TYPE>
constexpr bool kFactorFirst = TYPE == kMXFP4;
template <int TYPE>
constexpr bool kOffset = kHasOffset<TYPE> || TYPE == kQ4_K || TYPE == kQ5_K;

// What a lane needs of 256 elements of a row, as they lie there: loaded a chunk before it
// is decoded, so that memory answers while the chunk before is multiplied.
template <int TYPE, bool SUPER = TYPE == kQ4_K || TYPE == kQ5_K || TYPE == kQ6_K>
struct Raw {
    u32x2b w[8];
    uint32_t h[8], qh[8];
};
template <int TYPE>
struct Raw<TYPE, true> {
    u32x4 h;
    u32x2 w[4], qh[2];
    uint32_t d;
};

// Of chunk `chunk`; blocks past the row's `last` are the last again.
template <int TYPE>
__device__ __forceinline__ void load_raw(Raw<TYPE>& r, const uint8_t* row, int chunk, int last, int g) {
    if constexpr (TYPE == kQ8_0 || kNibbleLayout<TYPE>) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint8_t* blk = row + min(chunk * 8 + i, last) * Format<TYPE>::kBytes;
            if constexpr (TYPE == kQ8_0) {
                r.w[i] = *reinterpret_cast<const u32x2*>(blk + 2 + 8 * g);
                r.h[i] = *reinterpret_cast<const uint16_t*>(blk);
            } else {
                r.w[i] = *reinterpret_cast<const u32x2b*>(blk + kHeader<TYPE> + 8 * (g & 1));
                const uint16_t* h = reinterpret_cast<const uint16_t*>(blk);
                if constexpr (TYPE == kMXFP4)
                    r.h[i] = blk[0];
                else if constexpr (kHasOffset<TYPE>)
                    r.h[i] = uint32_t(h[0]) | (uint32_t(h[1]) << 16);
                else
                    r.h[i] = h[0];
                if constexpr (kHasFifth<TYPE>) {
                    constexpr int at = kHasOffset<TYPE> ? 2 : 1;
                    r.qh[i] = uint32_t(h[at]) | (uint32_t(h[at + 1]) << 16);
                }
            }
        }
    } else if constexpr (TYPE == kQ4_K || TYPE == kQ5_K) {
        const uint8_t* sb = row + int64_t(chunk) * Format<TYPE>::kBytes;
        r.h = *reinterpret_cast<const u32x4*>(sb);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r.w[i] = *reinterpret_cast<const u32x2*>(sb + (TYPE == kQ5_K ? 48 : 16) + 32 * i + 8 * g);
        if constexpr (TYPE == kQ5_K) r.qh[0] = *reinterpret_cast<const u32x2*>(sb + 16 + 8 * g);
    } else {
        // Q6_K: 4 bits of two sub-blocks a byte, 2 of four; 16 scales; d
        const uint8_t* sb = row + int64_t(chunk) * 210;
#pragma unroll
        for (int i = 0; i < 4; ++i) r.w[i] = *reinterpret_cast<const u32x2*>(sb + 32 * i + 8 * g);
#pragma unroll
        for (int i = 0; i < 2; ++i) r.qh[i] = *reinterpret_cast<const u32x2*>(sb + 128 + 32 * i + 8 * g);
        // the scales of this lane's halves of two sub-blocks in a word: bytes 8 (g / 2) and 16 above
        const u32x2 s0 = *reinterpret_cast<const u32x2*>(sb + 192), s1 = *reinterpret_cast<const u32x2*>(sb + 200);
        r.h = u32x4{s0[0], s0[1], s1[0], s1[1]};
        r.d = *reinterpret_cast<const uint16_t*>(sb + 208);
    }
}

// Sub-block i (of 32) of a chunk of 256.
template <int TYPE>
__device__ __forceinline__ Codes codes_of(const Raw<TYPE>& raw, int i, int g) {
    Codes r;
    r.c = 0.f;
    if constexpr (TYPE == kQ8_0) {
        r.a = half_to_f32(uint16_t(raw.h[i]));
        r.q = bytes_to_f16(raw.w[i][0] ^ 0x80808080u, raw.w[i][1] ^ 0x80808080u, 128.f);
    } else if constexpr (kNibbleLayout<TYPE>) {
        // low nibbles of the code bytes, then high ones
        const int sh = g >= 2 ? 4 : 0;
        uint32_t w0 = (raw.w[i][0] >> sh) & 0x0F0F0F0Fu, w1 = (raw.w[i][1] >> sh) & 0x0F0F0F0Fu;
        if constexpr (TYPE == kMXFP4) {
            // two codes to a byte, which the conversion takes
            r.a = mx_scale(raw.h[i]);
            const uint32_t p0 = w0 | (w0 >> 4), p1 = w1 | (w1 >> 4);
            const f16x2v v0 = __builtin_bit_cast(f16x2v, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(p0, 1.f, 0));
            const f16x2v v1 = __builtin_bit_cast(f16x2v, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(p0, 1.f, 2));
            const f16x2v v2 = __builtin_bit_cast(f16x2v, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(p1, 1.f, 0));
            const f16x2v v3 = __builtin_bit_cast(f16x2v, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(p1, 1.f, 2));
            r.q = f16x8{v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
        } else {
            r.a = half_to_f32(uint16_t(raw.h[i]));
            if constexpr (kHasOffset<TYPE>) r.c = half_to_f32(uint16_t(raw.h[i] >> 16));
            if constexpr (kHasFifth<TYPE>) {
                w0 |= fifth_bits(raw.qh[i], 8 * g);
                w1 |= fifth_bits(raw.qh[i], 8 * g + 4);
            }
            r.q = bytes_to_f16(w0, w1, kHasOffset<TYPE> ? 0.f : kHasFifth<TYPE> ? 16.f : 8.f);
        }
    } else if constexpr (TYPE == kQ4_K || TYPE == kQ5_K) {
        float m;
        q4_k_coeffs(raw.h[0], raw.h[1], raw.h[2], raw.h[3], i, r.a, m);
        r.c = -m;
        const u32x2 w = raw.w[i / 2];
        uint32_t w0 = (w[0] >> (4 * (i & 1))) & 0x0F0F0F0Fu, w1 = (w[1] >> (4 * (i & 1))) & 0x0F0F0F0Fu;
        if constexpr (TYPE == kQ5_K) {
            w0 |= ((raw.qh[0][0] >> i) & 0x01010101u) << 4;
            w1 |= ((raw.qh[0][1] >> i) & 0x01010101u) << 4;
        }
        r.q = bytes_to_f16(w0, w1, 0.f);
    } else {
        // Q6_K: a scale covers 16 codes, half of the sub-block's lanes. (q - 32) times it
        // has up to 13 bits: its four low bits and the rest make products of their own.
        const int half = i >> 2, p = i & 3;
        const u32x2 ql = raw.w[2 * half + (p & 1)], qh = raw.qh[half];
        const int sc = static_cast<int8_t>(raw.h[i / 2] >> (16 * (i & 1) + 8 * (g >> 1)));
        r.a = half_to_f32(uint16_t(raw.d));
        const int sh = 4 * (p >> 1);
        const f16x8 q = bytes_to_f16(((ql[0] >> sh) & 0x0F0F0F0Fu) | (((qh[0] >> (2 * p)) & 0x03030303u) << 4),
                                     ((ql[1] >> sh) & 0x0F0F0F0Fu) | (((qh[1] >> (2 * p)) & 0x03030303u) << 4), 32.f);
        r.q = q * _Float16(float(sc & 15));
        r.q2 = q * _Float16(float(sc & ~15));
    }
    return r;
}

struct FewArgs {
    const uint8_t* W;  // of this piece
    int64_t ldw, rows, N, n0;
    int K, T;
    const uint16_t* x;  // planes in steps of 64 rows, K in whole 256s
    int64_t plane;      // elements
    const float* factor;
    const void* targets;
    bool wide_targets;
    // kStats
    float2* part;
    int64_t part0;
    float* at_target;
    // kProb: d, rows of tokens
    const float* lse;
    float* out;
};

// Blocks of 16 rows of the head a wave, which share the reads of x: with one, 142 us
// where two took 114 to 121 (Q4_K 131072 x 4096, 16 tokens, rows not yet through LDS).
constexpr int kFewBlocks = 2;
constexpr int kFewRows = 16 * kFewBlocks;  // of the head a wave
constexpr int kFewK = 256;  // of x in LDS

__device__ __forceinline__ f32x4 mfma16(const f16x8& a, const f16x8& b, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// A wave's rows of 256 elements go from memory to LDS in pieces of 16 bytes, side by side:
// a lane needs bytes here and there of 16 rows, which asked of memory take a cache line
// each time (16 tokens through 131072 x 4096: Q8_0 313 us against 139, Q4_0 307 and 116,
// Q4_K 109 and 93). The last piece ends with the row's.
template <int TYPE>
struct Staged {
    static constexpr int kBytes = kFewK / Format<TYPE>::kBlock * Format<TYPE>::kBytes;
    static constexpr int kPitch = (kBytes + 15) / 16 * 16 + (kBytes % 64 == 0 ? 16 : 0);
    static constexpr int kPieces = (kBytes + 15) / 16;
    static constexpr int kLoads = (kFewRows * kPieces + 63) / 64;  // a lane
    static constexpr int kLds = kFewRows * kPitch;                 // a wave
};
// Beside 64 tokens in two parts, 128 KB, LDS has no room for it.
template <int TB, int PX>
constexpr bool kStaged = TB * PX <= 4;
// Waves that share the chunks of x in LDS. Four, of which several workgroups fit, while x
// is small; with 64 tokens four are one workgroup a CU (Q8_0 327 us, Q4_K 323), eight as
// well (197 and 199).
template <int TB, int PX>
constexpr int kFewWaves = TB * PX >= 4 ? 8 : 4;
template <int TYPE, int TB, int PX>
constexpr int few_waves_a_simd() {
    constexpr int waves = kFewWaves<TB, PX>;
    const int lds = 2 * kFewK / 64 * 16 * TB * PX * 128 + (kStaged<TB, PX> ? waves * Staged<TYPE>::kLds : 0);
    const int fit = 160 * 1024 / lds * waves / 4;
    return fit < 4 ? fit : 4;
}
typedef uint32_t u32x4b __attribute__((ext_vector_type(4), aligned(1)));
template <int TYPE>
using LdsPiece = uint32_t __attribute__((ext_vector_type(4), aligned(Staged<TYPE>::kBytes % 16 == 0 ? 16 : 2)));

// Up to 16 TB tokens, x in PX parts.
template <int TYPE, int TB, int PX, Kind KIND>
__global__ __launch_bounds__((kFewWaves<TB, PX> * 64), (few_waves_a_simd<TYPE, TB, PX>())) void few_kernel(const FewArgs g) {
    constexpr int kWaves = kFewWaves<TB, PX>;
    constexpr int kRows = kFewK / 64 * 16 * TB * PX;  // of 128 bytes in LDS: step, part, token
    constexpr int kCopies = kRows * 128 / (1024 * kWaves);
    __shared__ __align__(1024) uint8_t lds0[kRows * 128];
    __shared__ __align__(1024) uint8_t lds1[kRows * 128];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
    const int r = lane & 15, gr = lane >> 4;
    const int64_t run = int64_t(blockIdx.x) * kWaves + wave, row0 = run * kFewRows;

    // x's rows of a chunk: row (step, part, token) of 128 bytes, its 16-byte blocks
    // permuted by XOR with (row / 2) % 8
    const __amdgpu_buffer_rsrc_t x = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(g.x), 0,
                                                                       int(uint32_t(PX * g.plane * 2)), 0x00020000);
    auto copy = [&](uint8_t* lds, int chunk) {
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
            const int at = (i * kWaves + wave) * 8;
            const uint32_t row = at + (lane >> 3);
            const uint32_t token = row % (16 * TB), part = row / (16 * TB) % PX, step = row / (16 * TB * PX);
            const uint32_t from = uint32_t(part * g.plane * 2) + (step * 64 + token) * 128 +
                                  ((lane & 7) ^ ((row >> 1) & 7)) * 16;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(x, lds + at * 128, 16, from, uint32_t(chunk) * (kFewK / 64 * 64 * 128),
                                                     0, 0);
        }
    };
    const uint8_t* w[kFewBlocks];
#pragma unroll
    for (int i = 0; i < kFewBlocks; ++i) w[i] = g.W + min(row0 + i * 16 + r, g.rows - 1) * g.ldw;
    f32x4 acc[kFewBlocks][TB] = {};
    auto factor_of = [&](int t, int i) {
        const int token = 16 * t + 4 * gr + i;
        return token < g.T ? g.factor[token] : 0.f;
    };
    float factor[TB][4];
    if constexpr (kFactorFirst<TYPE>)
#pragma unroll
        for (int t = 0; t < TB; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) factor[t][i] = factor_of(t, i);
    const f16x8 ones = {1, 1, 1, 1, 1, 1, 1, 1};
    const int last = g.K / Format<TYPE>::kBlock - 1;
    auto load = [&](Raw<TYPE>* raw, int chunk) __attribute__((always_inline)) {
#pragma unroll
        for (int n = 0; n < kFewBlocks; ++n) load_raw<TYPE>(raw[n], w[n], chunk, last, gr);
    };
    auto sub_blocks = [&](const uint8_t* lds, const Raw<TYPE>* raw, int chunk, auto whole) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kFewK / 32; ++i) {
            if (!decltype(whole)::value && chunk * kFewK + i * 32 >= g.K) break;
            f16x8 xs[TB][PX];
#pragma unroll
            for (int t = 0; t < TB; ++t)
#pragma unroll
                for (int p = 0; p < PX; ++p) {
                    const int row = ((i / 2) * PX + p) * (16 * TB) + t * 16 + r, block = (i % 2) * 4 + gr;
                    xs[t][p] = *reinterpret_cast<const f16x8*>(lds + row * 128 + ((block ^ ((row >> 1) & 7)) * 16));
                }
            f32x4 sum[TB];
            if constexpr (kOffset<TYPE>)
#pragma unroll
                for (int t = 0; t < TB; ++t) {
                    sum[t] = mfma16(xs[t][0], ones, f32x4{0, 0, 0, 0});
                    if constexpr (PX == 2) sum[t] = mfma16(xs[t][1], ones, sum[t]);
                }
#pragma unroll
            for (int n = 0; n < kFewBlocks; ++n) {
                const Codes c = codes_of<TYPE>(raw[n], i, gr);
#pragma unroll
                for (int t = 0; t < TB; ++t) {
                    f32x4 v = {0, 0, 0, 0};
#pragma unroll
                    for (int p = PX - 1; p >= 0; --p) {
                        v = mfma16(xs[t][p], c.q, v);
                        if constexpr (TYPE == kQ6_K) v = mfma16(xs[t][p], c.q2, v);
                    }
#pragma unroll
                    for (int i4 = 0; i4 < 4; ++i4) {
                        const float by = kFactorFirst<TYPE> ? v[i4] * factor[t][i4] : v[i4];
                        acc[n][t][i4] = fmaf(c.a, by, acc[n][t][i4]);
                        if constexpr (kOffset<TYPE>) acc[n][t][i4] = fmaf(c.c, sum[t][i4], acc[n][t][i4]);
                    }
                }
            }
        }
    };
    auto any = [&](const uint8_t* lds, const Raw<TYPE>* raw, int chunk) __attribute__((always_inline)) {
        if (Format<TYPE>::kBlock == kFewK || (chunk + 1) * kFewK <= g.K)
            sub_blocks(lds, raw, chunk, std::true_type{});
        else
            sub_blocks(lds, raw, chunk, std::false_type{});
    };

    const int chunks = (g.K + kFewK - 1) / kFewK;
    copy(lds0, 0);
    if constexpr (kStaged<TB, PX>) {
        typedef Staged<TYPE> Z;
        __shared__ __align__(16) uint8_t staged[kWaves][Z::kLds];
        uint8_t* mine = staged[wave];
        const int64_t base = min(row0, g.rows - 1);
        const uint8_t* from = g.W + base * g.ldw;
        const int below = int(min(g.rows - 1 - base, int64_t(kFewRows - 1)));
        uint32_t at[Z::kLoads], to[Z::kLoads];
#pragma unroll
        for (int i = 0; i < Z::kLoads; ++i) {
            const int piece = min(i * 64 + lane, kFewRows * Z::kPieces - 1), row = piece / Z::kPieces;
            const int byte = min(piece % Z::kPieces * 16, Z::kBytes - 16);
            at[i] = uint32_t(min(row, below)) * uint32_t(g.ldw) + byte;
            to[i] = row * Z::kPitch + byte;
        }
        u32x4 pieces[Z::kLoads];
        auto whole = [&](int chunk) { return (chunk + 1) * kFewK <= g.K; };
        auto fetch = [&](int chunk) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < Z::kLoads; ++i)
                pieces[i] = *reinterpret_cast<const u32x4b*>(from + int64_t(chunk) * Z::kBytes + at[i]);
        };
        auto step = [&](const uint8_t* lds, uint8_t* next, int chunk) __attribute__((always_inline)) {
            copies_done_for_all<0>();
            const bool here = whole(chunk);
            if (here)
#pragma unroll
                for (int i = 0; i < Z::kLoads; ++i) *reinterpret_cast<LdsPiece<TYPE>*>(mine + to[i]) = pieces[i];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            if (chunk + 1 < chunks) {
                copy(next, chunk + 1);
                if (whole(chunk + 1)) fetch(chunk + 1);
            }
            Raw<TYPE> raw[kFewBlocks];
            if (here) {
#pragma unroll
                for (int n = 0; n < kFewBlocks; ++n) load_raw<TYPE>(raw[n], mine + (n * 16 + r) * Z::kPitch, 0, 7, gr);
                sub_blocks(lds, raw, chunk, std::true_type{});
            } else if (Format<TYPE>::kBlock < kFewK) {  // the last blocks of a row
                load(raw, chunk);
                sub_blocks(lds, raw, chunk, std::false_type{});
            }
        };
        if (whole(0)) fetch(0);
        for (int c = 0; c < chunks; c += 2) {
            step(lds0, lds1, c);
            if (c + 1 >= chunks) break;
            step(lds1, lds0, c + 1);
        }
    } else {
        Raw<TYPE> raw0[kFewBlocks], raw1[kFewBlocks];
        load(raw0, 0);
        for (int c = 0; c < chunks; c += 2) {
            copies_done_for_all<0>();
            if (c + 1 < chunks) {
                copy(lds1, c + 1);
                load(raw1, c + 1);
            }
            any(lds0, raw0, c);
            if (c + 1 >= chunks) break;
            copies_done_for_all<0>();
            if (c + 2 < chunks) {
                copy(lds0, c + 2);
                load(raw0, c + 2);
            }
            any(lds1, raw1, c + 1);
        }
    }

    // A lane: tokens 16 t + 4 gr + i, rows row0 + 16 n + r.
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int token = 16 * t + 4 * gr + i;
            const bool live = token < g.T;
            const float f = kFactorFirst<TYPE> ? 1.f : factor_of(t, i);
            const int64_t target = live ? vocab::token_at(g.targets, g.wide_targets, token, g.N) : -1;
            float l[kFewBlocks];
#pragma unroll
            for (int n = 0; n < kFewBlocks; ++n) l[n] = acc[n][t][i] * f;
            if constexpr (KIND == kStats) {
                float top = -__builtin_inff();
#pragma unroll
                for (int n = 0; n < kFewBlocks; ++n) {
                    const int64_t row = row0 + n * 16 + r;
                    if (row >= g.rows) l[n] = -__builtin_inff();
                    if (live && target == g.n0 + row && row < g.rows) g.at_target[token] = l[n];
                    top = fmaxf(top, l[n]);
                }
#pragma unroll
                for (int d = 1; d < 16; d *= 2) top = fmaxf(top, __shfl_xor(top, d));
                const float from = top == -__builtin_inff() ? 0.f : top;
                float sum = 0.f;
#pragma unroll
                for (int n = 0; n < kFewBlocks; ++n) sum += exp_of(l[n] - from);
#pragma unroll
                for (int d = 1; d < 16; d *= 2) sum += __shfl_xor(sum, d);
                if (live && r == 0 && row0 < g.rows) g.part[(g.part0 + run) * g.T + token] = make_float2(top, sum);
            } else {
                const float lse = target >= 0 ? g.lse[token] : 0.f;
#pragma unroll
                for (int n = 0; n < kFewBlocks; ++n) {
                    const int64_t row = row0 + n * 16 + r;
                    if (!live || row >= g.rows) continue;
                    g.out[token * g.rows + row] =
                        target >= 0 ? exp_of(l[n] - lse) - (g.n0 + row == target ? 1.f : 0.f) : 0.f;
                }
            }
        }
}

}  // namespace ce
}  // namespace retro
