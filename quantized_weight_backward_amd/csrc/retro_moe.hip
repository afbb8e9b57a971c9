// retro_moe.hip - a mixture-of-experts layer for a few tokens over microscaled
// 4-bit experts (retro_mx.h).
//
// A layer for T tokens reads the chosen experts' weights once and little else,
// so their bytes bound it; T <= 64 tokens leave at most 64 columns an expert.
// Launches:
//   router   logits, and x in bf16 parts with zeros up to whole 256-element steps
//   choose   top-k of each token
//   gate_up  a workgroup: 16 features of one chosen expert, all its tokens
//   down     a workgroup: 16 outputs, all chosen experts, all tokens
// Weights are decoded exactly to bf16 (E2M1 times a power of two) and meet x
// and h on v_mfma_f32_16x16x32_bf16 with F32 sums. x and h are cut into bf16
// parts that add up to them: one for a BF16 x, two for F16 (11 bits), three for
// F32 (24 bits); h, which is computed in F32, into two (16 bits, below a BF16
// or F16 result's own rounding) or three.
#include "retro_mx_device.h"
#include "retro_mx_host.h"

namespace retro {
namespace mx {
namespace {

struct Layer {
    int T, E, k;
    int64_t D, F;
    int64_t steps_d, steps_f;    // 256-element steps
    const uint8_t *guc, *gus, *dc, *ds;
    float* logits;               // T x E
    int* ids;                    // T x k, expert of each pair
    float* share;                // T x k
    __bf16* xp;                  // parts x T x Dp
    __bf16* hp;                  // parts x (T * k) x Fp
};

// v as bf16 parts that add up to it (up to the last part's rounding). What does
// not fit is left whole in the first part: inf - inf would be NaN.
template <int P>
__device__ __forceinline__ void cut(float v, __bf16 part[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
        part[i] = __bf16(v);
        const float got = float(part[i]);
        v = abs_bits(got) < 0x7f800000u ? v - got : 0.f;
    }
}

constexpr int kRouterWaves = 4;

// logits: a wave one expert and one token. Workgroups past the experts cut x.
template <typename TX, typename TR, int PX>
__global__ __launch_bounds__(kRouterWaves * 64) void moe_router_kernel(Layer L, const TX* __restrict__ X, int64_t ldx,
                                                                       const TR* __restrict__ R, int64_t ldr,
                                                                       int expert_groups) {
    const int t = blockIdx.y;
    const TX* x = X + int64_t(t) * ldx;
    if (int(blockIdx.x) < expert_groups) {
        const int e = blockIdx.x * kRouterWaves + threadIdx.x / 64, lane = threadIdx.x % 64;
        if (e >= L.E) return;
        const TR* r = R + int64_t(e) * ldr;
        float s = 0.f;
        for (int64_t d = lane; d < L.D; d += 64) s = fmaf(to_f32(x[d]), to_f32(r[d]), s);
#pragma unroll
        for (int m = 32; m; m >>= 1) s += __shfl_xor(s, m);
        if (lane == 0) L.logits[t * L.E + e] = s;
        return;
    }
    const int64_t Dp = L.steps_d * kStep;
    const int64_t d = int64_t(blockIdx.x - expert_groups) * (kRouterWaves * 64) + threadIdx.x;
    if (d >= Dp) return;
    __bf16 part[PX];
    cut<PX>(d < L.D ? to_f32(x[d]) : 0.f, part);
#pragma unroll
    for (int i = 0; i < PX; ++i) L.xp[(int64_t(i) * L.T + t) * Dp + d] = part[i];
}

// Larger logits first, equal ones by index, NaN last: a 64-bit key.
__device__ __forceinline__ uint64_t key_of(float v, int e) {
    uint32_t b = __float_as_uint(v + 0.f);  // -0 as +0
    b = (b & 0x7fffffffu) > 0x7f800000u ? 0u : (b & 0x80000000u) ? ~b : b | 0x80000000u;
    return uint64_t(b) << 32 | uint32_t(~e);
}

// A wave a token; lane l holds experts l, 64 + l, 128 + l, 192 + l.
__global__ __launch_bounds__(64) void moe_choose_kernel(Layer L, int renormalize) {
    const int t = blockIdx.x, lane = threadIdx.x;
    uint64_t key[4];
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int e = 64 * i + lane;
        v[i] = e < L.E ? L.logits[t * L.E + e] : -__builtin_inff();
        key[i] = e < L.E ? key_of(v[i], e) : 0;
    }
    float top = 0.f, chosen_sum = 0.f, mine = 0.f;
    for (int j = 0; j < L.k; ++j) {
        uint64_t best = key[0];
#pragma unroll
        for (int i = 1; i < 4; ++i) best = key[i] > best ? key[i] : best;
#pragma unroll
        for (int m = 32; m; m >>= 1) {
            const uint64_t o = __shfl_xor((unsigned long long)best, m);
            best = o > best ? o : best;
        }
        const int e = int(~uint32_t(best));
        float l = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float got = __shfl(v[i], e & 63);
            if (e >> 6 == i) l = got;
            if (key[i] == best) key[i] = 0;
        }
        if (j == 0) top = l;
        const float p = expf(l - top);
        chosen_sum += p;
        if (lane == j) {
            mine = p;
            L.ids[t * L.k + j] = e;
        }
    }
    float sum = chosen_sum;
    if (!renormalize) {
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (64 * i + lane < L.E) sum += expf(v[i] - top);
#pragma unroll
        for (int m = 32; m; m >>= 1) sum += __shfl_xor(sum, m);
    }
    if (lane < L.k) L.share[t * L.k + lane] = mine / sum;
}

// The chosen experts in order of index, as a bit set in LDS.
__device__ __forceinline__ void chosen_set(const Layer& L, uint64_t set[4]) {
    if (threadIdx.x < 4) set[threadIdx.x] = 0;
    __syncthreads();
    for (int p = threadIdx.x; p < L.T * L.k; p += blockDim.x) {
        const int e = L.ids[p];
        atomicOr(reinterpret_cast<unsigned long long*>(&set[e >> 6]), 1ull << (e & 63));
    }
    __syncthreads();
}

__device__ __forceinline__ int count_set(const uint64_t set[4]) {
    return __popcll(set[0]) + __popcll(set[1]) + __popcll(set[2]) + __popcll(set[3]);
}

// The expert of rank n among the chosen ones (n below their number).
__device__ __forceinline__ int expert_of_rank(const uint64_t set[4], int n) {
    for (int w = 0; w < 4; ++w) {
        uint64_t b = set[w];
        const int c = __popcll(b);
        if (n < c) {
            for (; n > 0; --n) b &= b - 1;
            return 64 * w + __ffsll((unsigned long long)b) - 1;
        }
        n -= c;
    }
    return 0;
}

// The pairs of one expert, in order, by one wave; returns their number.
__device__ __forceinline__ int pairs_of(const Layer& L, int e, int16_t* list) {
    const int lane = threadIdx.x & 63;
    int n = 0;
    for (int p0 = 0; p0 < L.T * L.k; p0 += 64) {
        const bool hit = p0 + lane < L.T * L.k && L.ids[p0 + lane] == e;
        const uint64_t m = __ballot(hit);
        if (hit) list[n + __popcll(m & ((1ull << lane) - 1))] = int16_t(p0 + lane);
        n += __popcll(m);
    }
    return n;
}

// 32 codes of a row's block (16 bytes) times their scale, as bf16: four
// operands of 8 elements.
__device__ __forceinline__ void decode_block(const u32x4& q, uint32_t e, bf16x8 w[4]) {
    const float s = e == 255u ? __uint_as_float(0x7fc00000u) : scale_value(e);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[i], s, 0);
        const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[i], s, 1);
        const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[i], s, 2);
        const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[i], s, 3);
        w[i] = bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
    }
}

constexpr int kGateWaves = 8;

// 16 features of one chosen expert: rows f0 .. f0 + 15 of gate and up times x of
// the expert's tokens, 16 tokens at a time. The waves share the 128-element
// pieces of D; their sums are added in LDS in the order of the waves.
template <int PX, int PH>
__global__ __launch_bounds__(kGateWaves * 64) void moe_gate_up_kernel(Layer L) {
    __shared__ uint64_t set[4];
    __shared__ int16_t list[RETRO_MOE_MAX_T];
    __shared__ int n_pairs;
    __shared__ float part[kGateWaves][2][16][17];
    chosen_set(L, set);
    if (int(blockIdx.y) >= count_set(set)) return;
    const int e = expert_of_rank(set, blockIdx.y);
    const int wave = threadIdx.x / 64, lane = threadIdx.x % 64, r = lane & 15, g = lane >> 4;
    if (wave == 0) {
        const int n = pairs_of(L, e, list);
        if (lane == 0) n_pairs = n;
    }
    __syncthreads();
    const int64_t rows = int64_t(L.E) * 2 * L.F, Dp = L.steps_d * kStep, Fp = L.steps_f * kStep;
    const int64_t f0 = int64_t(blockIdx.x) * 16, f = min(f0 + r, L.F - 1);
    const int64_t row[2] = {int64_t(e) * 2 * L.F + f, int64_t(e) * 2 * L.F + L.F + f};
    for (int p0 = 0; p0 < n_pairs; p0 += 16) {
        const int pair = list[min(p0 + r, n_pairs - 1)];
        const __bf16* x = L.xp + int64_t(pair / L.k) * Dp;
        f32x4 acc[2] = {};
        // past F only the zeros that pad h are left to write
        for (int64_t b = f0 < L.F ? int64_t(wave) * 4 + g : L.steps_d * 8; b < L.steps_d * 8; b += kGateWaves * 4) {
            bf16x8 v[PX][4];
#pragma unroll
            for (int p = 0; p < PX; ++p)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[p][i] = *reinterpret_cast<const bf16x8*>(x + int64_t(p) * L.T * Dp + b * 32 + i * 8);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const u32x4 q = *reinterpret_cast<const u32x4*>(L.guc + row[m] * L.steps_d * kStepBytes + b * 16);
                const uint32_t s = L.gus[(b / 8 * rows + row[m]) * kStepScales + b % 8];
                bf16x8 w[4];
                decode_block(q, s, w);
#pragma unroll
                for (int p = PX - 1; p >= 0; --p)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[i], v[p][i], acc[m], 0, 0, 0);
            }
        }
        __syncthreads();  // the last round's sums are read
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) part[wave][m][4 * g + i][r] = acc[m][i];
        __syncthreads();
        const int ff = threadIdx.x & 15, c = threadIdx.x >> 4;
        if (c < 16 && p0 + c < n_pairs) {
            float gate = 0.f, up = 0.f;
#pragma unroll
            for (int w = 0; w < kGateWaves; ++w) {
                gate += part[w][0][ff][c];
                up += part[w][1][ff][c];
            }
            const float h = f0 + ff < L.F ? gate / (1.f + expf(-gate)) * up : 0.f;
            __bf16 cutp[PH];
            cut<PH>(h, cutp);
#pragma unroll
            for (int p = 0; p < PH; ++p)
                L.hp[(int64_t(p) * L.T * L.k + list[p0 + c]) * Fp + f0 + ff] = cutp[p];
        }
    }
}

constexpr int kDownWaves = 16;
constexpr int kDownRows = 16;

// 16 outputs d: rows of every chosen expert's down matrix times h of its
// tokens. A wave takes (expert, part of F) items in turn and leaves each pair's
// 16 sums in LDS; then one thread adds up a token's pairs in order.
template <typename TY, int PH>
__global__ __launch_bounds__(kDownWaves * 64) void moe_down_kernel(Layer L, TY* __restrict__ Y, int64_t ldy,
                                                                   int max_parts) {
    __shared__ uint64_t set[4];
    __shared__ int16_t lists[kDownWaves][RETRO_MOE_MAX_T];
    extern __shared__ float sums[];  // parts x pairs x 16
    chosen_set(L, set);
    const int n_chosen = count_set(set), pairs = L.T * L.k;
    const int parts = max(1, min(max_parts, (3 * kDownWaves + n_chosen - 1) / n_chosen));
    const int wave = threadIdx.x / 64, lane = threadIdx.x % 64, r = lane & 15, g = lane >> 4;
    const int64_t rows = int64_t(L.E) * L.D, Fp = L.steps_f * kStep;
    const int64_t d0 = int64_t(blockIdx.x) * kDownRows, d = min(d0 + r, L.D - 1);
    const int64_t chunks = L.steps_f * 2;  // 128-element pieces of F
    for (int item = wave; item < n_chosen * parts; item += kDownWaves) {
        const int e = expert_of_rank(set, item / parts), part = item % parts;
        const int n = pairs_of(L, e, lists[wave]);
        const int64_t c0 = chunks * part / parts, c1 = chunks * (part + 1) / parts;
        const int64_t row = int64_t(e) * L.D + d;
        for (int p0 = 0; p0 < n; p0 += 16) {
            const int pair = lists[wave][min(p0 + r, n - 1)];
            const __bf16* h = L.hp + int64_t(pair) * Fp;
            f32x4 acc = {};
            for (int64_t c = c0; c < c1; ++c) {
                const int64_t b = c * 4 + g;
                const u32x4 q = *reinterpret_cast<const u32x4*>(L.dc + row * L.steps_f * kStepBytes + b * 16);
                const uint32_t s = L.ds[(b / 8 * rows + row) * kStepScales + b % 8];
                bf16x8 w[4];
                decode_block(q, s, w);
#pragma unroll
                for (int p = PH - 1; p >= 0; --p)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const bf16x8 v = *reinterpret_cast<const bf16x8*>(h + int64_t(p) * pairs * Fp + b * 32 + i * 8);
                        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[i], v, acc, 0, 0, 0);
                    }
            }
            if (p0 + r < n)
#pragma unroll
                for (int i = 0; i < 4; ++i) sums[(part * pairs + pair) * 16 + 4 * g + i] = acc[i];
        }
    }
    __syncthreads();
    for (int o = threadIdx.x; o < L.T * 16; o += kDownWaves * 64) {
        const int t = o / 16, dd = o % 16;
        if (d0 + dd >= L.D) continue;
        float y = 0.f;
        for (int j = 0; j < L.k; ++j) {
            float s = 0.f;
            for (int p = 0; p < parts; ++p) s += sums[(p * pairs + t * L.k + j) * 16 + dd];
            y = fmaf(L.share[t * L.k + j], s, y);
        }
        Y[int64_t(t) * ldy + d0 + dd] = from_f32<TY>(y);
    }
}

// bf16 parts of x and h for a type of x.
constexpr int x_parts(int type) { return type == RETRO_BF16 ? 1 : type == RETRO_F16 ? 2 : 3; }
constexpr int h_parts(int type) { return type == RETRO_F32 ? 3 : 2; }
template <typename TX> constexpr int type_of();
template <> constexpr int type_of<float>() { return RETRO_F32; }
template <> constexpr int type_of<_Float16>() { return RETRO_F16; }
template <> constexpr int type_of<__bf16>() { return RETRO_BF16; }

// The workspace's pieces, each on a 256-byte boundary.
struct Pieces {
    int64_t logits, ids, share, xp, hp, all;
};

Pieces pieces(int xtype, int64_t T, int64_t D, int64_t F, int64_t E, int64_t k) {
    Pieces p{};
    int64_t at = 0;
    auto put = [&](int64_t& where, int64_t bytes) {
        where = at;
        at += host::cdiv(bytes, 256) * 256;
    };
    put(p.logits, T * E * 4);
    put(p.ids, T * k * 4);
    put(p.share, T * k * 4);
    put(p.xp, x_parts(xtype) * T * steps_of(D) * kStep * 2);
    put(p.hp, h_parts(xtype) * T * k * steps_of(F) * kStep * 2);
    p.all = at;
    return p;
}

// LDS for the pairs' sums of the down kernel.
constexpr int64_t kSumBytes = 128 * 1024;

template <typename TX, typename TR>
int launch_layer(Layer L, const TX* X, int64_t ldx, const TR* R, int64_t ldr, TX* Y, int64_t ldy, int renormalize,
                 hipStream_t st) {
    constexpr int PX = x_parts(type_of<TX>()), PH = h_parts(type_of<TX>());
    const int groups = int(host::cdiv(L.E, kRouterWaves));
    const int64_t cuts = host::cdiv(L.steps_d * kStep, kRouterWaves * 64);
    host::clear_last_error();
    moe_router_kernel<TX, TR, PX>
        <<<dim3(uint32_t(groups + cuts), L.T), dim3(kRouterWaves * 64), 0, st>>>(L, X, ldx, R, ldr, groups);
    moe_choose_kernel<<<dim3(L.T), dim3(64), 0, st>>>(L, renormalize);
    const int most = std::min(L.E, L.T * L.k);
    moe_gate_up_kernel<PX, PH>
        <<<dim3(uint32_t(L.steps_f * (kStep / 16)), most), dim3(kGateWaves * 64), 0, st>>>(L);
    const int64_t pair_bytes = int64_t(L.T) * L.k * 16 * 4;
    const int parts = int(std::max<int64_t>(1, std::min<int64_t>(L.steps_f * 2, kSumBytes / pair_bytes)));
    moe_down_kernel<TX, PH>
        <<<dim3(uint32_t(host::cdiv(L.D, kDownRows))), dim3(kDownWaves * 64), size_t(parts * pair_bytes), st>>>(
            L, Y, ldy, parts);
    return host::launch_status();
}

}  // namespace
}  // namespace mx
}  // namespace retro

using namespace retro;
using namespace retro::mx;

namespace {

int check_layer(int xtype, int64_t T, int64_t D, int64_t F, int64_t E, int64_t k) {
    if (!float_bytes(xtype)) return RETRO_E_TYPE;
    if (T < 0 || T > RETRO_MOE_MAX_T || E < 1 || E > RETRO_MOE_MAX_E || k < 1 || k > RETRO_MOE_MAX_TOP_K || k > E ||
        D < 1 || F < 1 || D >= host::kDimLimit / (2 * RETRO_MOE_MAX_E) || F >= host::kDimLimit / (2 * RETRO_MOE_MAX_E))
        return RETRO_E_SHAPE;
    return RETRO_OK;
}

}  // namespace

extern "C" {

int64_t retro_moe_workspace_size(int xtype, int64_t T, int64_t D, int64_t F, int64_t E, int64_t top_k) {
    const int rc = check_layer(xtype, T, D, F, E, top_k);
    if (rc != RETRO_OK) return rc;
    return T == 0 ? 0 : pieces(xtype, T, D, F, E, top_k).all;
}

int retro_moe(int xtype, const void* X, int64_t ldx, int rtype, const void* R, int64_t ldr, const void* gate_up_codes,
              const void* gate_up_scales, const void* down_codes, const void* down_scales, void* Y, int64_t ldy,
              int64_t T, int64_t D, int64_t F, int64_t E, int64_t top_k, int renormalize, void* workspace,
              int64_t workspace_bytes, void* stream) {
    int rc = check_layer(xtype, T, D, F, E, top_k);
    if (rc != RETRO_OK) return rc;
    if (rtype != RETRO_F32 && rtype != xtype) return RETRO_E_TYPE;
    const int size = float_bytes(xtype), rsize = float_bytes(rtype);
    const Span x{X, span_bytes(T, D, ldx, size)}, y{Y, span_bytes(T, D, ldy, size)},
        r{R, span_bytes(E, D, ldr, rsize)};
    if (x.n < 0 || y.n < 0 || r.n < 0) return RETRO_E_SHAPE;
    if (T == 0) return RETRO_OK;
    if (!X || !R || !gate_up_codes || !gate_up_scales || !down_codes || !down_scales || !Y) return RETRO_E_NULL;
    if (!aligned(X, size) || !aligned(Y, size) || !aligned(R, rsize) || !aligned(gate_up_codes, 16) ||
        !aligned(gate_up_scales, 16) || !aligned(down_codes, 16) || !aligned(down_scales, 16))
        return RETRO_E_ALIGN;
    const Span in[6] = {x,
                        r,
                        {gate_up_codes, code_bytes(E * 2 * F, D)},
                        {gate_up_scales, scale_bytes(E * 2 * F, D)},
                        {down_codes, code_bytes(E * D, F)},
                        {down_scales, scale_bytes(E * D, F)}};
    for (const Span& s : in)
        if (mx::overlap(y, s)) return RETRO_E_ALIAS;
    const Pieces p = pieces(xtype, T, D, F, E, top_k);
    const Span w{workspace, p.all};
    bool fits = workspace && workspace_bytes >= p.all && aligned(workspace, 16) && !mx::overlap(w, y);
    for (const Span& s : in) fits = fits && !mx::overlap(w, s);
    if (!fits) return RETRO_E_WORKSPACE;
    char* base = static_cast<char*>(workspace);
    Layer L{};
    L.T = int(T);
    L.E = int(E);
    L.k = int(top_k);
    L.D = D;
    L.F = F;
    L.steps_d = steps_of(D);
    L.steps_f = steps_of(F);
    L.guc = static_cast<const uint8_t*>(gate_up_codes);
    L.gus = static_cast<const uint8_t*>(gate_up_scales);
    L.dc = static_cast<const uint8_t*>(down_codes);
    L.ds = static_cast<const uint8_t*>(down_scales);
    L.logits = reinterpret_cast<float*>(base + p.logits);
    L.ids = reinterpret_cast<int*>(base + p.ids);
    L.share = reinterpret_cast<float*>(base + p.share);
    L.xp = reinterpret_cast<__bf16*>(base + p.xp);
    L.hp = reinterpret_cast<__bf16*>(base + p.hp);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    return with_float(xtype, [&](auto* tag) {
        using TX = std::remove_pointer_t<decltype(tag)>;
        const TX* xs = static_cast<const TX*>(X);
        if (rtype == RETRO_F32)
            return launch_layer(L, xs, ldx, static_cast<const float*>(R), ldr, static_cast<TX*>(Y), ldy, renormalize,
                                st);
        return launch_layer(L, xs, ldx, static_cast<const TX*>(R), ldr, static_cast<TX*>(Y), ldy, renormalize, st);
    });
}

}  // extern "C"
