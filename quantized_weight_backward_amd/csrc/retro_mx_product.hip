// retro_mx_product.hip - Y = A B^T of two microscaled matrices on the scaled
// matrix cores, and the product with A quantised in the call (retro_mx.h).
#include "retro_mx_device.h"
#include "retro_mx_host.h"
#include "retro_mx_skinny.h"
#include "retro_mx_tile.h"

namespace retro {
namespace mx {
namespace {

// Y[t][n] = sum over blocks b of 2^(ea + eb - 254) * (sum of 32 E2M1 products).
// v_mfma_scale_f32_32x32x64_f8f6f4 takes, per lane, a row's block of 32 codes
// (16 bytes: lane % 32 the row, lane / 32 one of two blocks) and that block's
// scale byte, and adds both blocks' scaled sums. Which of a row's blocks meet in
// one instruction is free as long as A and B agree: in a step of 256 elements
// lane half h takes blocks 4h .. 4h + 3 in turn, so one 32-bit word holds its
// four scale bytes.

// Simple form: a wave a 32 x 32 tile of Y, operands straight from memory.
template <typename TY>
__global__ __launch_bounds__(64) void product_simple_kernel(const uint8_t* __restrict__ ac,
                                                            const uint8_t* __restrict__ as,
                                                            const uint8_t* __restrict__ bc,
                                                            const uint8_t* __restrict__ bs, TY* __restrict__ Y,
                                                            int64_t ldy, int64_t steps, int64_t N, int64_t T,
                                                            int64_t tiles_n, int64_t tile0) {
    const int lane = threadIdx.x, r = lane & 31, h = lane >> 5;
    const int64_t tile = tile0 + blockIdx.x, t0 = tile / tiles_n * 32, n0 = tile % tiles_n * 32;
    const int64_t ra = min(t0 + r, T - 1), rb = min(n0 + r, N - 1);
    const uint8_t* pa = ac + ra * steps * kStepBytes + h * 64;
    const uint8_t* pb = bc + rb * steps * kStepBytes + h * 64;
    const uint8_t* sa = as + ra * kStepScales + h * 4;
    const uint8_t* sb = bs + rb * kStepScales + h * 4;
    f32x16 acc = {};
    for (int64_t c = 0; c < steps; ++c) {
        const int ea = *reinterpret_cast<const int*>(sa + c * T * kStepScales);
        const int eb = *reinterpret_cast<const int*>(sb + c * N * kStepScales);
        i32x8 a[4] = {}, b[4] = {};
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const i32x4 va = *reinterpret_cast<const i32x4*>(pa + c * kStepBytes + s * 16);
            const i32x4 vb = *reinterpret_cast<const i32x4*>(pb + c * kStepBytes + s * 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[s][i] = va[i];
                b[s][i] = vb[i];
            }
        }
        acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a[0], b[0], acc, 4, 4, 0, ea, 0, eb);
        acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a[1], b[1], acc, 4, 4, 1, ea, 1, eb);
        acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a[2], b[2], acc, 4, 4, 2, ea, 2, eb);
        acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a[3], b[3], acc, 4, 4, 3, ea, 3, eb);
    }
    if (n0 + r >= N) return;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int64_t t = t0 + (i / 4) * 8 + h * 4 + i % 4;
        if (t < T) Y[t * ldy + n0 + r] = from_f32<TY>(acc[i]);
    }
}

using Tile256x256 = Tile<2, 4, 4, 2>;
using Tile256x192 = Tile<4, 2, 2, 3>;
using Tile128x128 = Tile<2, 2, 2, 2>;
using Tile64x128 = Tile<2, 2, 1, 2>;
using Tile64x64 = Tile<2, 2, 1, 1>;
using Tile64x64K4 = Tile<2, 2, 1, 1, 4>;
using Tile32x64K4 = Tile<1, 2, 1, 1, 4>;

struct Args {
    const uint8_t *ac, *as, *bc, *bs;
    int64_t ldy, K, N, T;
    hipStream_t st;
};

template <typename TY>
int launch_simple(const Args& p, TY* Y) {
    const int64_t tiles_n = host::cdiv(p.N, 32), tiles_t = host::cdiv(p.T, 32);
    return in_block_ranges(tiles_n * tiles_t, [&](int64_t first, uint32_t blocks) {
        product_simple_kernel<TY><<<dim3(blocks), dim3(64), 0, p.st>>>(p.ac, p.as, p.bc, p.bs, Y, p.ldy, steps_of(p.K),
                                                                       p.N, p.T, tiles_n, first);
    });
}

template <class Z, typename TY>
int launch_tile(const Args& p, TY* Y) {
    const int64_t tiles_n = host::cdiv(p.N, Z::kRowsN), tiles_t = host::cdiv(p.T, Z::kRowsT);
    const double row = double(steps_of(p.K)) * (kStepBytes + kStepScales);
    const int group = host::group_height(tiles_t, tiles_n, Z::kPerCU, double(p.T) * row, double(p.N) * row);
    host::clear_last_error();
    product_tile_kernel<TY, Z><<<dim3(uint32_t(tiles_n * tiles_t)), dim3(Z::kThreads), 0, p.st>>>(
        p.ac, p.as, p.bc, p.bs, Y, p.ldy, uint32_t(steps_of(p.K)), p.N, p.T, uint32_t(tiles_n), uint32_t(tiles_t),
        uint32_t(group));
    return host::launch_status();
}

// Whether all of a tile kernel's workgroups fit one launch.
template <class Z>
bool one_launch(int64_t N, int64_t T) {
    return host::cdiv(T, Z::kRowsT) * host::cdiv(N, Z::kRowsN) <= kMaxThreads / Z::kThreads;
}

// The tiles address 256 rows of codes, all rows' scales of a step and five rows
// of Y with 32-bit offsets.
bool tiles_apply(int size, int64_t ldy, int64_t K, int64_t N, int64_t T) {
    return K > 0 && steps_of(K) * kStepBytes * 256 < (int64_t(1) << 32) &&
           steps_of(K) * std::max(N, T) * kStepScales < (int64_t(1) << 32) &&
           (ldy * 5 + 32) * size < (int64_t(1) << 32);
}

// Rows of A the skinny kernel takes.
constexpr int64_t kSkinnyMaxT = 32;
bool skinny_applies(int64_t K, int64_t T) { return K > 0 && T <= kSkinnyMaxT; }

template <int TB, int U, typename TY>
int launch_skinny_blocks(const Args& p, TY* Y) {
    return in_block_ranges(host::cdiv(p.N, kSkinnyRows), [&](int64_t first, uint32_t blocks) {
        product_skinny_kernel<TY, TB, U><<<dim3(blocks), dim3(kSkinnyWaves * 64), 0, p.st>>>(
            p.ac, p.as, p.bc, p.bs, Y, p.ldy, int(steps_of(p.K)), p.N, int(p.T), uint32_t(first));
    });
}

template <typename TY>
int launch_skinny(const Args& p, TY* Y) {
    return p.T <= 16 ? launch_skinny_blocks<1, 4>(p, Y) : launch_skinny_blocks<2, 2>(p, Y);
}

// A linear layer quantises x in the product's own kernel where that is few
// elements a workgroup. N = 14336, K = 4096: 12.5 us for 4 rows, 17.3 for 8, against
// 14.7 in two launches.
constexpr int64_t kFusedElements = 16384;
bool fuse_linear(int64_t K, int64_t T) {
    return T <= 16 && T * steps_of(K) * kStep <= kFusedElements;
}

template <typename TX>
int launch_linear_skinny(const Args& p, const TX* X, int64_t ldx, TX* Y) {
    const int64_t steps = steps_of(p.K);
    return in_block_ranges(host::cdiv(p.N, kSkinnyRows), [&](int64_t first, uint32_t blocks) {
        linear_skinny_kernel<TX, 4>
            <<<dim3(blocks), dim3(kSkinnyWaves * 64), size_t(p.T * steps * (kStepBytes + kStepScales)), p.st>>>(
                X, ldx, p.bc, p.bs, Y, p.ldy, int(p.K), int(steps), p.N, int(p.T), uint32_t(first));
    });
}

int choose(int size, int64_t ldy, int64_t K, int64_t N, int64_t T) {
    auto tiles = [&](int64_t t, int64_t n) { return host::cdiv(T, t) * host::cdiv(N, n); };
    // Few rows of A and of B: 16 rows of B a workgroup put more CUs to work than
    // tiles do. T = 16, N = 4096, K = 14336: 10.0 us against 14.7 for 32 x 64
    // tiles; N = 14336, K = 4096: 10.8 against 9.2. T = 32: 13.8 against 15.6 and
    // 14.6 against 9.7.
    if (skinny_applies(K, T) && tiles(32, 64) < 128) return RETRO_MX_VARIANT_SKINNY;
    // Time of a round of workgroups over the CUs, in us: a start and end and a time
    // for each 256 elements of K, with one workgroup a CU and with as many as fit.
    // Fitted to T x N x K = 4096 x 14336 x 4096, 4096 x 5120 x 4096, 8192^3, 17408 x
    // 5120 x 2048, 2048 x 5120 x 17408 and 64 .. 1024 x 4096 x 4096 and 14336. The
    // last round has as many a CU as it needs, of which the first cost least beside
    // one another (512 x 4096 x 4096: two of four a CU 12.0 us, one 11.0, four 19.1),
    // or, at one a CU, as many CUs (the fewer, the higher their clock): 2048 x 5120 x
    // 17408 takes 97 us as 216 tiles of 256 x 192 and 112 as 160 of 256 x 256, 8192^3
    // 309 and 276.
    struct Cost {
        int variant, rows_t, rows_n, per_cu;
        double one, one_step, full, full_step;
    };
    const double f32 = size == 4 ? 4 : 0;  // twice the bytes to write, with nothing beside
    const Cost costs[] = {
        {RETRO_MX_VARIANT_TILE_256x256, 256, 256, Tile256x256::kPerCU, 7 + f32, 1.4, 7 + f32, 1.9},
        {RETRO_MX_VARIANT_TILE_256x192, 256, 192, Tile256x192::kPerCU, 3 + f32, 1.1, 5 + f32, 1.55},
        {RETRO_MX_VARIANT_TILE_128x128, 128, 128, Tile128x128::kPerCU, 3, 0.8, 5, 1.07},
        {RETRO_MX_VARIANT_TILE_64x128, 64, 128, Tile64x128::kPerCU, 2.5, 0.6, 4, 0.95},
        {RETRO_MX_VARIANT_TILE_64x64, 64, 64, Tile64x64::kPerCU, 2, 0.47, 4.5, 0.92},
        {RETRO_MX_VARIANT_TILE_64x64_K4, 64, 64, Tile64x64K4::kPerCU, 2.5, 0.3, 2.5, 0.3},
        {RETRO_MX_VARIANT_TILE_32x64_K4, 32, 64, Tile32x64K4::kPerCU, 2.5, 0.23, 2.5, 0.23},
    };
    const double steps = double(steps_of(K));
    int best = 0;
    double least = 0;
    for (const Cost& c : costs) {
        if (!product_applies(c.variant, size, ldy, K, N, T)) continue;
        const int64_t n = tiles(c.rows_t, c.rows_n), round = int64_t(host::kNumCUs) * c.per_cu;
        const int64_t rest = host::cdiv(n % round, host::kNumCUs);
        const double one = c.one + c.one_step * steps, full = c.full + c.full_step * steps;
        double cost = double(n / round) * full;
        const double of = c.per_cu > 1 ? double(rest - 1) / (c.per_cu - 1) : 1;
        const double filled = c.per_cu > 1 ? of * of : double(n % round) / double(round);
        if (rest) cost += one + (full - one) * filled;
        if (!best || cost < least) {
            best = c.variant;
            least = cost;
        }
    }
    return best ? best : skinny_applies(K, T) ? RETRO_MX_VARIANT_SKINNY : RETRO_MX_VARIANT_SIMPLE;
}

}  // namespace

bool product_applies(int variant, int size, int64_t ldy, int64_t K, int64_t N, int64_t T) {
    switch (variant) {
        case RETRO_MX_VARIANT_AUTO:
        case RETRO_MX_VARIANT_SIMPLE: return true;
        case RETRO_MX_VARIANT_TILE_256x256: return tiles_apply(size, ldy, K, N, T) && one_launch<Tile256x256>(N, T);
        case RETRO_MX_VARIANT_TILE_256x192: return tiles_apply(size, ldy, K, N, T) && one_launch<Tile256x192>(N, T);
        case RETRO_MX_VARIANT_TILE_64x128: return tiles_apply(size, ldy, K, N, T) && one_launch<Tile64x128>(N, T);
        case RETRO_MX_VARIANT_TILE_128x128: return tiles_apply(size, ldy, K, N, T) && one_launch<Tile128x128>(N, T);
        case RETRO_MX_VARIANT_TILE_64x64: return tiles_apply(size, ldy, K, N, T) && one_launch<Tile64x64>(N, T);
        case RETRO_MX_VARIANT_TILE_64x64_K4: return tiles_apply(size, ldy, K, N, T) && one_launch<Tile64x64K4>(N, T);
        case RETRO_MX_VARIANT_TILE_32x64_K4: return tiles_apply(size, ldy, K, N, T) && one_launch<Tile32x64K4>(N, T);
        case RETRO_MX_VARIANT_SKINNY: return skinny_applies(K, T);
        default: return false;
    }
}

int launch_product(int variant, int ytype, const void* ac, const void* as, const void* bc, const void* bs, void* Y,
                   int64_t ldy, int64_t K, int64_t N, int64_t T, hipStream_t st) {
    const Args p{static_cast<const uint8_t*>(ac), static_cast<const uint8_t*>(as), static_cast<const uint8_t*>(bc),
                 static_cast<const uint8_t*>(bs), ldy, K, N, T, st};
    if (variant == RETRO_MX_VARIANT_AUTO) variant = choose(float_bytes(ytype), ldy, K, N, T);
    return with_float(ytype, [&](auto* tag) {
        using TY = std::remove_pointer_t<decltype(tag)>;
        TY* y = static_cast<TY*>(Y);
        switch (variant) {
            case RETRO_MX_VARIANT_TILE_256x256: return launch_tile<Tile256x256>(p, y);
            case RETRO_MX_VARIANT_TILE_256x192: return launch_tile<Tile256x192>(p, y);
            case RETRO_MX_VARIANT_TILE_64x128: return launch_tile<Tile64x128>(p, y);
            case RETRO_MX_VARIANT_TILE_128x128: return launch_tile<Tile128x128>(p, y);
            case RETRO_MX_VARIANT_TILE_64x64: return launch_tile<Tile64x64>(p, y);
            case RETRO_MX_VARIANT_SKINNY: return launch_skinny(p, y);
            case RETRO_MX_VARIANT_TILE_64x64_K4: return launch_tile<Tile64x64K4>(p, y);
            case RETRO_MX_VARIANT_TILE_32x64_K4: return launch_tile<Tile32x64K4>(p, y);
            default: return launch_simple(p, y);
        }
    });
}

}  // namespace mx
}  // namespace retro

using namespace retro;
using namespace retro::mx;

namespace {

// Sizes that both products take: fewer than 2^30 tiles of 32 x 32 in Y.
bool product_dims(int64_t K, int64_t N, int64_t T) {
    return dim_ok(K) && dim_ok(N) && dim_ok(T) && host::cdiv(N, 32) * host::cdiv(T, 32) < host::kGridLimit;
}

// The shape and operand checks of both products.
int check_product(int ytype, const void* bc, const void* bs, const void* Y, int64_t ldy, int64_t K, int64_t N,
                  int64_t T, int64_t& y_bytes) {
    const int size = float_bytes(ytype);
    if (!size) return RETRO_E_TYPE;
    if (!product_dims(K, N, T)) return RETRO_E_SHAPE;
    y_bytes = span_bytes(T, N, ldy, size);
    if (y_bytes < 0) return RETRO_E_SHAPE;
    if (N == 0 || T == 0) return RETRO_OK;
    if (!Y || (K && (!bc || !bs))) return RETRO_E_NULL;
    if (!aligned(bc, 16) || !aligned(bs, 16) || !aligned(Y, size)) return RETRO_E_ALIGN;
    if (overlap({Y, y_bytes}, {bc, code_bytes(N, K)}) || overlap({Y, y_bytes}, {bs, scale_bytes(N, K)}))
        return RETRO_E_ALIAS;
    return RETRO_OK;
}

int64_t linear_workspace(int64_t K, int64_t T) {
    // codes, then scales on a 16-byte boundary (code rows are multiples of 128)
    return code_bytes(T, K) + scale_bytes(T, K);
}

}  // namespace

extern "C" {

int retro_mx_mul_mat(int ytype, const void* a_codes, const void* a_scales, const void* b_codes, const void* b_scales,
                     void* Y, int64_t ldy, int64_t K, int64_t N, int64_t T, void* stream) {
    return retro_mx_mul_mat_variant(RETRO_MX_VARIANT_AUTO, ytype, a_codes, a_scales, b_codes, b_scales, Y, ldy, K, N,
                                    T, stream);
}

int retro_mx_mul_mat_choice(int ytype, int64_t ldy, int64_t K, int64_t N, int64_t T) {
    const int size = float_bytes(ytype);
    if (!size) return RETRO_E_TYPE;
    if (!product_dims(K, N, T) || span_bytes(T, N, ldy, size) < 0) return RETRO_E_SHAPE;
    return choose(size, ldy, K, N, T);
}

int retro_mx_mul_mat_variant(int variant, int ytype, const void* a_codes, const void* a_scales, const void* b_codes,
                             const void* b_scales, void* Y, int64_t ldy, int64_t K, int64_t N, int64_t T,
                             void* stream) {
    int64_t yb = 0;
    const int rc = check_product(ytype, b_codes, b_scales, Y, ldy, K, N, T, yb);
    if (rc != RETRO_OK || N == 0 || T == 0) return rc;
    if (K && (!a_codes || !a_scales)) return RETRO_E_NULL;
    if (!aligned(a_codes, 16) || !aligned(a_scales, 16)) return RETRO_E_ALIGN;
    if (overlap({Y, yb}, {a_codes, code_bytes(T, K)}) || overlap({Y, yb}, {a_scales, scale_bytes(T, K)}))
        return RETRO_E_ALIAS;
    if (!product_applies(variant, float_bytes(ytype), ldy, K, N, T)) return RETRO_E_VARIANT;
    return launch_product(variant, ytype, a_codes, a_scales, b_codes, b_scales, Y, ldy, K, N, T,
                          static_cast<hipStream_t>(stream));
}

int64_t retro_mx_linear_workspace_size(int xtype, int64_t K, int64_t N, int64_t T) {
    if (!float_bytes(xtype)) return RETRO_E_TYPE;
    if (!product_dims(K, N, T)) return RETRO_E_SHAPE;
    return N == 0 || fuse_linear(K, T) ? 0 : linear_workspace(K, T);
}

int retro_mx_linear(int xtype, const void* X, int64_t ldx, const void* b_codes, const void* b_scales, void* Y,
                    int64_t ldy, int64_t K, int64_t N, int64_t T, void* workspace, int64_t workspace_bytes,
                    void* stream) {
    int64_t yb = 0;
    int rc = check_product(xtype, b_codes, b_scales, Y, ldy, K, N, T, yb);
    if (rc != RETRO_OK) return rc;
    const int64_t xb = span_bytes(T, K, ldx, float_bytes(xtype));
    if (xb < 0) return RETRO_E_SHAPE;
    if (N == 0 || T == 0) return RETRO_OK;
    if (K && !X) return RETRO_E_NULL;
    if (!aligned(X, float_bytes(xtype))) return RETRO_E_ALIGN;
    if (overlap({Y, yb}, {X, xb})) return RETRO_E_ALIAS;
    const int64_t need = retro_mx_linear_workspace_size(xtype, K, N, T);
    const Span w{workspace, need};
    if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 16) || overlap(w, {X, xb}) ||
                 overlap(w, {Y, yb}) || overlap(w, {b_codes, code_bytes(N, K)}) ||
                 overlap(w, {b_scales, scale_bytes(N, K)})))
        return RETRO_E_WORKSPACE;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (K && fuse_linear(K, T))
        return with_float(xtype, [&](auto* tag) {
            using TX = std::remove_pointer_t<decltype(tag)>;
            const Args p{nullptr, nullptr, static_cast<const uint8_t*>(b_codes),
                         static_cast<const uint8_t*>(b_scales), ldy, K, N, T, st};
            return launch_linear_skinny(p, static_cast<const TX*>(X), ldx, static_cast<TX*>(Y));
        });
    uint8_t* codes = static_cast<uint8_t*>(workspace);
    uint8_t* scales = codes + code_bytes(T, K);
    if (K) {
        rc = launch_quantize_rows(xtype, X, ldx, T, K, codes, scales, st);
        if (rc != RETRO_OK) return rc;
    }
    return launch_product(RETRO_MX_VARIANT_AUTO, xtype, codes, scales, b_codes, b_scales, Y, ldy, K, N, T, st);
}

}  // extern "C"
