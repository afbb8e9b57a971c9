// retro_moe.hip - a mixture-of-experts layer for a few tokens over microscaled
// 4-bit experts (retro_mx.h).
//
// A layer for T tokens reads the chosen experts' weights once and little else,
// so their bytes bound it; T <= 64 tokens leave at most 64 columns an expert.
// Launches:
//   router   logits, and x in bf16 parts with zeros up to whole 256-element steps
//   choose   top-k of each token, the list of chosen experts and their pairs
//   gate_up  a workgroup: some features of one chosen expert, 16 of its tokens
//   down     a workgroup: some outputs of all tokens, over all chosen experts or
//            a part of them
//   join     adds the parts
// Weights are decoded exactly to bf16 (E2M1 times a power of two) and meet x
// and h on v_mfma_f32_16x16x32_bf16 with F32 sums. x is cut into bf16 parts that
// add up to it: one for a BF16 x, two for F16 (11 bits), three for F32 (24 bits).
// h, which is computed in F32, is rounded to three parts for F32 and to two (16
// bits) for BF16 and F16, which round y to 8 or 11 bits: with three the error
// against 64 bits is the same to four digits (1.6e-3 of y in BF16; 0.1 to 0.2% of
// its last bits differ from those of an F32 h, 0.3% with two), and the layers below
// take 21.6, 66 and 190 us instead of 16.6, 63 and 179.
//
// Measured (BF16; calls one after another from a graph, weights in turn past the
// caches; in brackets router, choose, gate_up, down and join traced one launch at
// a time, which takes longer: they do not add up to the call): 1 token, 4 of 32
// experts, D = 2048, F = 1024: 16.2 us (3.0, in gate_up, 6.9, 6.9, none: launches and
// the latencies of each, 13 MB of weights are 2.6 us). 16 tokens, 8 of 64 experts, F =
// 1000: 63 us (4.0, 4.6, 32, 20, 4.8) for 185 MB, 2.9 TB/s. 32 tokens, 2 of 8
// experts, D = 4096, F = 14336: 172 to 180 us (5.3, 6.7, 106, 66, 5.4) for 749 MB, 4.2
// to 4.4 TB/s, where a plain read reaches 5.2; traced, gate_up reads at 4.7 and down
// at 3.8.
#include "retro_mx_device.h"
#include "retro_mx_host.h"

namespace retro {
namespace mx {
namespace {

// A pair is a token's j-th choice, number t * k + j.
struct Layer {
    int T, E, k;
    int64_t D, F;
    int64_t steps_d, steps_f;  // 256-element steps
    const uint8_t *guc, *gus, *dc, *ds;
    float* logits;   // T x E
    float* share;    // T x k
    int* lists;      // number of tiles (up to 16 pairs of an expert), then of each: expert, first place, pairs
    int16_t* order;  // the pairs, by expert
    __bf16* xp;      // parts x T x Dp
    __bf16* hp;      // parts x (T * k) x Fp: share times h
    float* sums;     // splits x T x D
};

// v as bf16 parts that add up to it (up to the last part's rounding). An infinity
// or NaN is left whole in the first part (inf - inf would be NaN), and a value
// that would round up to an infinity is cut short.
template <int P>
__device__ __forceinline__ void cut(float v, __bf16 part[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
        float got = float(__bf16(v));
        if (abs_bits(got) == 0x7f800000u) got = __uint_as_float(__float_as_uint(v) & 0xffff0000u);
        part[i] = __bf16(got);
        v = abs_bits(got) < 0x7f800000u ? v - got : 0.f;
    }
}

constexpr int kRouterWaves = 4;

// 8 elements on a 16-byte boundary.
template <typename T>
__device__ __forceinline__ void load8_aligned(const T* x, float v[8]) {
    typedef T vec __attribute__((ext_vector_type(16 / sizeof(T))));
    constexpr int kPer = 16 / sizeof(T);
#pragma unroll
    for (int j = 0; j < 8 / kPer; ++j) {
        const vec w = reinterpret_cast<const vec*>(x)[j];
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[j * kPer + i] = to_f32(w[i]);
    }
}

// logits: a wave one expert and TOKENS tokens, 8 elements a lane at a time; whole
// steps of 512 elements without branches where all rows are `aligned` to 16
// bytes. Workgroups past the experts cut x.
template <typename TX, typename TR, int PX, int TOKENS>
__global__ __launch_bounds__(kRouterWaves * 64) void moe_router_kernel(Layer L, const TX* __restrict__ X, int64_t ldx,
                                                                       const TR* __restrict__ R, int64_t ldr,
                                                                       int expert_groups, bool aligned) {
    const int lane = threadIdx.x % 64, t0 = blockIdx.y * TOKENS, n = min(TOKENS, L.T - t0);
    if (int(blockIdx.x) < expert_groups) {
        const int e = blockIdx.x * kRouterWaves + threadIdx.x / 64;
        if (e >= L.E) return;
        const TR* r = R + int64_t(e) * ldr + lane * 8;
        const TX* x[TOKENS];
#pragma unroll
        for (int t = 0; t < TOKENS; ++t) x[t] = X + int64_t(min(t0 + t, L.T - 1)) * ldx + lane * 8;
        float s[TOKENS] = {};
        int64_t d = 0;
        if (aligned)
#pragma unroll 4
            for (; d + 512 <= L.D; d += 512) {
                float a[8];
                load8_aligned(r + d, a);
#pragma unroll
                for (int t = 0; t < TOKENS; ++t) {
                    float v[8];
                    load8_aligned(x[t] + d, v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) s[t] = fmaf(v[i], a[i], s[t]);
                }
            }
        for (; d < L.D; d += 512) {
            float a[8];
            load8(r + d, L.D - d - lane * 8, a);
#pragma unroll
            for (int t = 0; t < TOKENS; ++t) {
                float v[8];
                load8(x[t] + d, L.D - d - lane * 8, v);
#pragma unroll
                for (int i = 0; i < 8; ++i) s[t] = fmaf(v[i], a[i], s[t]);
            }
        }
#pragma unroll
        for (int t = 0; t < TOKENS; ++t) {
#pragma unroll
            for (int m = 32; m; m >>= 1) s[t] += __shfl_xor(s[t], m);
            if (lane == 0 && t < n) L.logits[(t0 + t) * L.E + e] = s[t];
        }
        return;
    }
    const int64_t Dp = L.steps_d * kStep;
    const int64_t d = (int64_t(blockIdx.x - expert_groups) * (kRouterWaves * 64) + threadIdx.x) * 8;
    if (d >= Dp) return;
    for (int t = t0; t < t0 + n; ++t) {
        float x[8];
        load8(X + int64_t(t) * ldx + d, L.D - d, x);
        bf16x8 out[PX];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            __bf16 part[PX];
            cut<PX>(x[j], part);
#pragma unroll
            for (int i = 0; i < PX; ++i) out[i][j] = part[i];
        }
#pragma unroll
        for (int i = 0; i < PX; ++i)
            *reinterpret_cast<bf16x8*>(L.xp + (int64_t(i) * L.T + t) * Dp + d) = out[i];
    }
}

// A key that grows with the logit: 0 stands for none, 1 for NaN, -0 is +0.
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t b = __float_as_uint(v + 0.f);
    return (b & 0x7fffffffu) > 0x7f800000u ? 1u : (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) {
    return __uint_as_float(k == 1u ? 0x7fc00000u : (k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}

// The largest of a wave's values, uniform.
__device__ __forceinline__ uint32_t max_of_wave(uint32_t v) {
    v = max16(v);
    const uint32_t a = __builtin_amdgcn_readlane(int(v), 0), b = __builtin_amdgcn_readlane(int(v), 16),
                   c = __builtin_amdgcn_readlane(int(v), 32), d = __builtin_amdgcn_readlane(int(v), 48);
    return max(max(a, b), max(c, d));
}

// Tiles of T tokens' pairs: each chosen expert's in sixteens.
constexpr int kMaxTiles = RETRO_MOE_MAX_E + RETRO_MOE_MAX_T * RETRO_MOE_MAX_TOP_K / 16;
__host__ __device__ inline int most_tiles(int64_t T, int64_t E, int64_t k) {
    const int64_t pairs = T * k, chosen = pairs < E ? pairs : E;
    return int(chosen + pairs / 16);
}

// The chosen experts and their pairs, in LDS.
struct Lists {
    int16_t ids[RETRO_MOE_MAX_T * RETRO_MOE_MAX_TOP_K];    // expert of each pair
    float share[RETRO_MOE_MAX_T * RETRO_MOE_MAX_TOP_K];    // and its share
    int16_t order[RETRO_MOE_MAX_T * RETRO_MOE_MAX_TOP_K];  // the pairs by expert
    unsigned long long tokens[RETRO_MOE_MAX_E];  // of each expert, a bit each
    int place[RETRO_MOE_MAX_E];
    int entry[3 * kMaxTiles];  // of each tile: expert, first place, pairs
    int wave_tiles[4], wave_pairs[4], n_tiles;
};

// Top-k of one token by a wave, lane l holding experts l, 64 + l, ... below 64 WORDS.
template <int WORDS>
__device__ __forceinline__ void choose_token(const Layer& L, int t, int renormalize, Lists& s) {
    const int lane = threadIdx.x % 64;
    uint32_t key[WORDS];
    float v[WORDS];
#pragma unroll
    for (int i = 0; i < WORDS; ++i) {
        const int e = 64 * i + lane;
        v[i] = e < L.E ? L.logits[t * L.E + e] : 0.f;
        key[i] = e < L.E ? key_of(v[i]) : 0u;
    }
    uint32_t mine = 0, top = 0;  // lane j: the key of choice j
    int expert = 0;
    for (int j = 0; j < L.k; ++j) {
        // the largest key, at its lowest expert
        uint32_t best = key[0];
#pragma unroll
        for (int i = 1; i < WORDS; ++i) best = max(best, key[i]);
        best = max_of_wave(best);
        if (j == 0) top = best;
        int e = -1;
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
            const uint64_t m = __ballot(key[i] == best);
            if (e < 0 && m) {
                const int at = __ffsll((unsigned long long)m) - 1;
                e = 64 * i + at;
                if (lane == at) key[i] = 0;
            }
        }
        if (lane == j) {
            mine = best;
            expert = e;
        }
    }
    const float first = of_key(top);
    const float p = lane < L.k ? expf(of_key(mine) - first) : 0.f;
    float sum = p;
    if (!renormalize) {
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < WORDS; ++i)
            if (64 * i + lane < L.E) sum += expf(v[i] - first);
    }
#pragma unroll
    for (int m = 32; m; m >>= 1) sum += __shfl_xor(sum, m);
    if (lane < L.k) {
        s.ids[t * L.k + lane] = int16_t(expert);
        s.share[t * L.k + lane] = p / sum;
    }
}

// Top-k of all tokens by a workgroup of at least 4 waves, a wave a token at a
// time; then the lists by expert, an expert's pairs in the order of their tokens
// (which tile a pair is in decides the order of its sums).
__device__ __forceinline__ void choose(const Layer& L, int renormalize, Lists& s) {
    const int waves = blockDim.x / 64, wave = threadIdx.x / 64, lane = threadIdx.x % 64;
    for (int e = threadIdx.x; e < RETRO_MOE_MAX_E; e += blockDim.x) s.tokens[e] = 0;
    for (int t = wave; t < L.T; t += waves) {
        if (L.E <= 64)
            choose_token<1>(L, t, renormalize, s);
        else if (L.E <= 128)
            choose_token<2>(L, t, renormalize, s);
        else
            choose_token<4>(L, t, renormalize, s);
    }
    __syncthreads();
    const int pairs = L.T * L.k;
    if (L.T == 1) {  // every choice is an expert of its own
        if (int(threadIdx.x) < pairs) {
            s.entry[3 * threadIdx.x] = s.ids[threadIdx.x];
            s.entry[3 * threadIdx.x + 1] = threadIdx.x;
            s.entry[3 * threadIdx.x + 2] = 1;
            s.order[threadIdx.x] = int16_t(threadIdx.x);
        }
        if (threadIdx.x == 0) s.n_tiles = pairs;
        __syncthreads();
        return;
    }
    for (int p = threadIdx.x; p < pairs; p += blockDim.x) atomicOr(&s.tokens[s.ids[p]], 1ull << (p / L.k));
    __syncthreads();
    // where each expert's tiles and pairs begin
    const int e = threadIdx.x;
    int n = 0, first = 0, tile = 0;
    if (e < RETRO_MOE_MAX_E) {
        n = __popcll(s.tokens[e]);
        int run_pairs = n, run_tiles = (n + 15) / 16;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int p = __shfl_up(run_pairs, d), q = __shfl_up(run_tiles, d);
            if (lane >= d) {
                run_pairs += p;
                run_tiles += q;
            }
        }
        first = run_pairs - n;
        tile = run_tiles - (n + 15) / 16;
        if (lane == 63) {
            s.wave_pairs[wave] = run_pairs;
            s.wave_tiles[wave] = run_tiles;
        }
    }
    __syncthreads();
    if (e < RETRO_MOE_MAX_E) {
        for (int w = 0; w < wave; ++w) {
            first += s.wave_pairs[w];
            tile += s.wave_tiles[w];
        }
        s.place[e] = first;
        for (int i = 0; i < n; i += 16, ++tile) {
            s.entry[3 * tile] = e;
            s.entry[3 * tile + 1] = first + i;
            s.entry[3 * tile + 2] = min(16, n - i);
        }
        if (e == RETRO_MOE_MAX_E - 1) s.n_tiles = tile;
    }
    __syncthreads();
    for (int p = threadIdx.x; p < pairs; p += blockDim.x) {
        const int id = s.ids[p];
        s.order[s.place[id] + __popcll(s.tokens[id] & ((1ull << (p / L.k)) - 1))] = int16_t(p);
    }
    __syncthreads();
}

// The lists for the launches that follow.
__device__ __forceinline__ void write_lists(const Layer& L, const Lists& s) {
    if (threadIdx.x == 0) L.lists[0] = s.n_tiles;
    for (int i = threadIdx.x; i < 3 * s.n_tiles; i += blockDim.x) L.lists[1 + i] = s.entry[i];
    for (int p = threadIdx.x; p < L.T * L.k; p += blockDim.x) {
        L.order[p] = s.order[p];
        L.share[p] = s.share[p];
    }
}

constexpr int kChooseWaves = 16;

__global__ __launch_bounds__(kChooseWaves * 64) void moe_choose_kernel(Layer L, int renormalize) {
    __shared__ Lists lists;
    choose(L, renormalize, lists);
    write_lists(L, lists);
}

// A lane's part of a 256-element step of 16 rows: lane (r, g) holds blocks g and
// 4 + g of row r and the row's eight scale bytes, so that a wave reads whole
// 128-byte pieces of the rows.
struct Step {
    u32x4 code[2];
    u32x2 scale;
};

__device__ __forceinline__ void load_step(Step& s, const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                          int64_t row, int64_t steps, int64_t step, int g) {
    const uint8_t* c = codes + (row * steps + step) * kStepBytes + g * 16;
    s.code[0] = *reinterpret_cast<const u32x4*>(c);
    s.code[1] = *reinterpret_cast<const u32x4*>(c + 64);
    s.scale = *reinterpret_cast<const u32x2*>(scales + (step * rows + row) * kStepScales);
}

// A block times the scale byte at the bottom of `scale`, as bf16: four operands
// of 8 elements.
__device__ __forceinline__ void decode(const u32x4& code, uint32_t scale, bf16x8 w[4]) {
    const uint32_t e = scale & 0xffu;
    const float s = e == 255u ? __uint_as_float(0x7fc00000u) : scale_value(e);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t q = code[i];
        const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 0);
        const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 1);
        const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 2);
        const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 3);
        w[i] = bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
    }
}

// 32 elements of a row of x or h, as four operands.
__device__ __forceinline__ void load_block(bf16x8 v[4], const __bf16* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const bf16x8*>(p + i * 8);
}

// use(c) for c = first, first + by, ... below end, each loaded while the one
// before is used.
template <typename Loaded, typename Load, typename Use>
__device__ __forceinline__ void in_pairs(int first, int end, int by, Load&& load, Use&& use) {
    if (first >= end) return;
    Loaded a, b;
    load(a, first);
    for (int c = first;; c += 2 * by) {
        if (c + by >= end) {
            use(a);
            return;
        }
        load(b, c + by);
        use(a);
        if (c + 2 * by >= end) {
            use(b);
            return;
        }
        load(a, c + 2 * by);
        use(b);
    }
}

constexpr int kGateWaves = 4;

// 16 features of one chosen expert: their rows of gate and of up times x of a tile
// of its tokens. D's steps are dealt to the waves in turn, whose sums are added in
// LDS in their order. A wave loads a step while it works on the one before.
//
// For a token or a few (OWN_LISTS) every workgroup chooses the experts itself,
// which takes it about a microsecond where a launch of its own takes several.
template <int PX, int PH, bool OWN_LISTS>
__global__ __launch_bounds__(kGateWaves * 64, PX == 1 ? 3 : 2) void moe_gate_up_kernel(Layer L, int renormalize) {
    __shared__ float part[kGateWaves][2][16][17];
    const int* entry = L.lists + 1 + blockIdx.y * 3;
    const int16_t* order = L.order;
    const float* share = L.share;
    if constexpr (OWN_LISTS) {
        __shared__ Lists own;
        choose(L, renormalize, own);
        if (blockIdx.x == 0 && blockIdx.y == 0) write_lists(L, own);
        if (int(blockIdx.y) >= own.n_tiles) return;
        entry = own.entry + blockIdx.y * 3;
        order = own.order;
        share = own.share;
    } else {
        if (int(blockIdx.y) >= L.lists[0]) return;
    }
    const int e = entry[0], first = entry[1], n = entry[2];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
    const int r = lane & 15, g = lane >> 4;
    const int64_t rows = int64_t(L.E) * 2 * L.F, Dp = L.steps_d * kStep, Fp = L.steps_f * kStep;
    const int64_t f0 = int64_t(blockIdx.x) * 16;
    const int64_t row = int64_t(e) * 2 * L.F + min(f0 + r, L.F - 1);  // of gate; F further on of up
    // past F only the zeros that pad h are written
    const int steps = f0 < L.F ? int(L.steps_d) : 0;
    // lanes of columns past the pairs load nothing; their sums are dropped
    const bool used = r < n;
    const int pair = order[first + (used ? r : 0)];
    const __bf16* x = L.xp + int64_t(pair / L.k) * Dp + g * 32;
    f32x4 acc[2] = {};
    struct Loaded {
        Step w[2];
        bf16x8 v[2][PX][4];
    };
    auto load = [&](Loaded& l, int c) {
#pragma unroll
        for (int m = 0; m < 2; ++m) load_step(l.w[m], L.guc, L.gus, rows, row + m * L.F, L.steps_d, c, g);
        if (used)
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int p = 0; p < PX; ++p)
                    load_block(l.v[b][p], x + int64_t(p) * L.T * Dp + c * kStep + b * 128);
    };
    auto use = [&](const Loaded& l) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                bf16x8 o[4];
                decode(l.w[m].code[b], l.w[m].scale[b] >> (8 * g), o);
#pragma unroll
                for (int p = PX - 1; p >= 0; --p)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(o[i], l.v[b][p][i], acc[m], 0, 0, 0);
            }
    };
    in_pairs<Loaded>(wave, steps, kGateWaves, load, use);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[wave][m][4 * g + i][r] = acc[m][i];
    __syncthreads();
    static_assert(kGateWaves * 64 == 16 * 16, "an output a thread");
    const int f = threadIdx.x % 16, c = threadIdx.x / 16;
    if (c >= n) return;
    float gate = 0.f, up = 0.f;
#pragma unroll
    for (int w = 0; w < kGateWaves; ++w) {
        gate += part[w][0][f][c];
        up += part[w][1][f][c];
    }
    const int pr = order[first + c];
    const float h = f0 + f < L.F ? gate / (1.f + expf(-gate)) * up * share[pr] : 0.f;
    __bf16 cutp[PH];
    cut<PH>(h, cutp);
#pragma unroll
    for (int p = 0; p < PH; ++p) L.hp[(int64_t(p) * L.T * L.k + pr) * Fp + f0 + f] = cutp[p];
}

// 16 (or 4) bytes a lane from offset at + `more` (uniform) of the `bytes` at p into
// LDS, lane after lane.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, uint32_t(min(bytes, int64_t(0xffffffffu))),
                                             0x00020000);
}
__device__ __forceinline__ void copy16(uint8_t* lds, const void* p, int64_t bytes, uint32_t at, uint32_t more) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer(p, bytes), lds, 16, at, more, 0, 0);
}
__device__ __forceinline__ void copy4(uint8_t* lds, const void* p, int64_t bytes, uint32_t at, uint32_t more) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer(p, bytes), lds, 4, at, more, 0, 0);
}

// All but a wave's last N copies into LDS have landed, its reads are done, and
// so for every wave.
template <int N>
__device__ __forceinline__ void stage_ready() {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4) << 14 | 0x70);  // vmcnt(N) lgkmcnt(0)
    asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// For larger layers a workgroup of WAVES waves multiplies 32 WAVES rows of weights
// with a tile through a ring of stages in LDS, each a piece of 128 elements: rows,
// their scales, and the tile's x or h. Read straight into the operands' lanes each
// 16 bytes are a cache access of their own (a lane holds another row than its
// neighbour): 38 to 40 accesses a load instruction, of which x or h had two for
// each of the rows'. A copy of 64 or 256 contiguous bytes takes one for each 64, 15
// to 16 an instruction, and x or h is copied once for all waves. 32 tokens, 2 of 8
// experts, D = 4096, F = 14336: down 36 to 8 million accesses, 93 to 64 us; gate_up
// 48 to 16 million, 117 to 107 us, its bytes at 4.7 TB/s (traced).
// The two halves of a stage's rows are two ranges of the matrix's; a wave
// multiplies 16 of each. Rows of 64 bytes lie permuted by XOR with (row / 4) % 4,
// x's or h's of 256 bytes by XOR with the row, so that neighbouring lanes' reads
// meet all banks.
template <int P, int WAVES>
struct Ring {
    static constexpr int kRange = 16 * WAVES, kRows = 2 * kRange;
    static constexpr int kIn = kRows * 64, kScales = kIn + P * 4096, kBytes = kScales + kRows * 4;
    static constexpr int kCopiesOfIn = (P * 4 + WAVES - 1) / WAVES;
    static constexpr int kCopies = 2 + kCopiesOfIn + 1;  // of a wave, a piece

    const uint8_t *codes, *scales;
    const __bf16* in;  // P x `in_rows` x `in_pitch` elements
    int64_t rows, second;  // of the matrix; between the two ranges
    uint32_t pitch, part;  // bytes of a row of codes, of a part of `in`
    int wave, lane;
    int last0, last1;  // the ranges' last rows: past them they are copied again
    uint32_t code_at[2], scale_at, in_at[kCopiesOfIn];

    // n0 and n1: rows that there are in the two ranges (one at least in the first)
    __device__ __forceinline__ Ring(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t second, int n0,
                                    int n1, int64_t steps, const __bf16* in, int64_t in_rows)
        : codes(codes), scales(scales), in(in), rows(rows), second(n1 > 0 ? second : 0),
          pitch(uint32_t(steps) * kStepBytes), part(uint32_t(in_rows * steps * (kStep * 2))) {
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
        lane = threadIdx.x % 64;
        last0 = min(n0, kRange) - 1;
        last1 = n1 > 0 ? min(n1, kRange) - 1 : last0;
#pragma unroll
        for (int j = 0; j < 2; ++j)
            code_at[j] = min(wave * 16 + lane / 4, j ? last1 : last0) * pitch + ((lane % 4) ^ (lane / 16)) * 16;
        scale_at = min(scale_copy() % (WAVES / 4) * 64 + lane, scale_range() ? last1 : last0) * kStepScales;
    }

    // A wave copies 64 rows' scales (two waves the same): which, and of which range.
    __device__ __forceinline__ int scale_copy() const { return wave % (WAVES / 2); }
    __device__ __forceinline__ int scale_range() const { return scale_copy() / (WAVES / 4); }

    // Row `at(i)` of `in` is the tile's row i, i < 16.
    template <typename At>
    __device__ __forceinline__ void set_tile(At&& at) {
#pragma unroll
        for (int j = 0; j < kCopiesOfIn; ++j) {
            const int row = (j * WAVES + wave) % (P * 4) % 4 * 4 + lane / 16;
            in_at[j] = uint32_t(at(row)) * (pitch * 4) + ((lane % 16) ^ row) * 16;
        }
    }

    // Piece c of rows row0 and on.
    __device__ __forceinline__ void copy(uint8_t* stage, int64_t row0, int c) const {
#pragma unroll
        for (int j = 0; j < 2; ++j)
            copy16(stage + (j * kRange + wave * 16) * 64, codes + (row0 + j * second) * pitch,
                   int64_t((j ? last1 : last0) + 1) * pitch, code_at[j], c * 64);
#pragma unroll
        for (int j = 0; j < kCopiesOfIn; ++j) {
            const int at = (j * WAVES + wave) % (P * 4);
            copy16(stage + kIn + at * 1024, in, int64_t(P) * part, in_at[j], at / 4 * part + c * 256);
        }
        copy4(stage + kScales + scale_copy() * 256,
              scales + (c / 2 * rows + row0 + (scale_range() ? second : 0)) * kStepScales,
              int64_t((scale_range() ? last1 : last0) + 1) * kStepScales, scale_at, c % 2 * 4);
    }

    // acc[m] += the wave's 16 rows of range m times the tile.
    __device__ __forceinline__ void multiply(const uint8_t* stage, f32x4 acc[2]) const {
        const int r = lane & 15, g = lane >> 4;
        bf16x8 v[P][4];
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[p][i] =
                    *reinterpret_cast<const bf16x8*>(stage + kIn + p * 4096 + r * 256 + (((g * 4 + i) ^ r) * 16));
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const int row = m * kRange + wave * 16 + r;
            const u32x4 q = *reinterpret_cast<const u32x4*>(stage + row * 64 + ((g ^ ((r >> 2) & 3)) * 16));
            bf16x8 o[4];
            decode(q, stage[kScales + row * 4 + g], o);
#pragma unroll
            for (int p = P - 1; p >= 0; --p)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(o[i], v[p][i], acc[m], 0, 0, 0);
        }
    }
};

// `pieces` pieces through the stages l: copy(stage) takes the next piece, the last
// again past the end, and use(stage) the next that was copied. Whole rounds
// without a way out in between: so the compiler sees that a stage was refilled
// S - 1 steps ago, and waits for no later copy.
template <int S, int COPIES, typename Copy, typename Use>
__device__ __forceinline__ void through_ring(uint8_t* l0, uint8_t* l1, uint8_t* l2, uint8_t* l3, int pieces,
                                             Copy&& copy, Use&& use) {
    auto step = [&](const uint8_t* cur, uint8_t* refill) {
        stage_ready<(S - 2) * COPIES>();
        copy(refill);
        use(cur);
    };
    copy(l0);
    copy(l1);
    if constexpr (S > 3) copy(l2);
    for (; pieces >= S; pieces -= S) {
        step(l0, S > 3 ? l3 : l2);
        step(l1, l0);
        step(l2, l1);
        if constexpr (S > 3) step(l3, l2);
    }
    if (pieces > 0) step(l0, S > 3 ? l3 : l2);
    if (pieces > 1) step(l1, l0);
    if (S > 3 && pieces > 2) step(l2, l1);
    stage_ready<0>();
}

constexpr int kRingWavesUp = 4;

// 64 features of one tile through the ring: their rows of gate are its first
// range, of up its second.
template <int PX, int PH, bool OWN_LISTS>
__global__ __launch_bounds__(kRingWavesUp * 64, PX < 3 ? 3 : 2) void moe_gate_up_ring_kernel(Layer L, int renormalize) {
    using R = Ring<PX, kRingWavesUp>;
    __shared__ __align__(256) uint8_t l0[R::kBytes], l1[R::kBytes], l2[R::kBytes];
    const int* entry = L.lists + 1 + blockIdx.y * 3;
    const int16_t* order = L.order;
    const float* share = L.share;
    if constexpr (OWN_LISTS) {
        __shared__ Lists own;
        choose(L, renormalize, own);
        if (blockIdx.x == 0 && blockIdx.y == 0) write_lists(L, own);
        if (int(blockIdx.y) >= own.n_tiles) return;
        entry = own.entry + blockIdx.y * 3;
        order = own.order;
        share = own.share;
    } else {
        if (int(blockIdx.y) >= L.lists[0]) return;
    }
    const int e = __builtin_amdgcn_readfirstlane(entry[0]), first = __builtin_amdgcn_readfirstlane(entry[1]);
    const int n = __builtin_amdgcn_readfirstlane(entry[2]);
    const int64_t f0 = int64_t(blockIdx.x) * R::kRange, Fp = L.steps_f * kStep;
    f32x4 acc[2] = {};
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), r = threadIdx.x & 15, g = threadIdx.x / 16 % 4;
    if (f0 < L.F) {  // past F only the zeros that pad h are written
        const int there = int(min(int64_t(R::kRange), L.F - f0));
        R ring(L.guc, L.gus, int64_t(L.E) * 2 * L.F, L.F, there, there, L.steps_d, L.xp, L.T);
        ring.set_tile([&](int i) { return order[first + min(i, n - 1)] / L.k; });
        const int64_t row0 = int64_t(e) * 2 * L.F + f0;
        const int pieces = int(L.steps_d) * 2;
        int next = 0;
        through_ring<3, R::kCopies>(
            l0, l1, l2, nullptr, pieces,
            [&](uint8_t* stage) {
                ring.copy(stage, row0, next);
                next = min(next + 1, pieces - 1);
            },
            [&](const uint8_t* stage) { ring.multiply(stage, acc); });
    }
    if (r >= n) return;
    const int pair = order[first + r];
    const float by = share[pair];
    const int64_t f = f0 + wave * 16 + 4 * g;
    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
    bf16x4 out[PH];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float gate = acc[0][i], h = f + i < L.F ? gate / (1.f + expf(-gate)) * acc[1][i] * by : 0.f;
        __bf16 part[PH];
        cut<PH>(h, part);
#pragma unroll
        for (int p = 0; p < PH; ++p) out[p][i] = part[p];
    }
#pragma unroll
    for (int p = 0; p < PH; ++p)
        *reinterpret_cast<bf16x4*>(L.hp + (int64_t(p) * L.T * L.k + pair) * Fp + f) = out[p];
}

// 16 RF outputs of all tokens. The tiles' rows, one tile after another, are one
// list of 128-element pieces, of which every wave of the gridDim.y workgroups of
// these outputs takes an equal run. Within a tile the columns are its pairs, whose
// h holds the share; at its end the wave adds its sums to those of the pairs'
// tokens in LDS, and at the end of the kernel the waves' are added in their order.
// One workgroup writes Y; the sums of several are added by the join.
template <typename TY, int PH, int RF, int WAVES>
__global__ __launch_bounds__(WAVES * 64, WAVES == 16 ? 4 : 2) void moe_down_kernel(Layer L, TY* __restrict__ Y,
                                                                                   int64_t ldy) {
    constexpr int kWide = 16 * RF + 4;
    extern __shared__ __align__(16) float sums[];  // wave x token x kWide, then the lists
    int* entry = reinterpret_cast<int*>(sums + WAVES * L.T * kWide);
    const int n_tiles = L.lists[0], most = most_tiles(L.T, L.E, L.k);
    int16_t* order = reinterpret_cast<int16_t*>(entry + 3 * most);
    // all that may be there: what lies past the chosen ones is not used
    for (int i = threadIdx.x; i < 3 * most; i += WAVES * 64) entry[i] = L.lists[1 + i];
    for (int i = threadIdx.x; i < L.T * L.k; i += WAVES * 64) order[i] = L.order[i];
    for (int i = threadIdx.x; i < WAVES * L.T * kWide; i += WAVES * 64) sums[i] = 0.f;
    __syncthreads();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
    const int r = lane & 15, g = lane >> 4;
    float* mine = sums + wave * L.T * kWide;
    const int64_t rows = int64_t(L.E) * L.D, Fp = L.steps_f * kStep, part_of_h = int64_t(L.T) * L.k * Fp;
    const int64_t d0 = int64_t(blockIdx.x) * (16 * RF);
    const int pieces = int(L.steps_f) * 2;
    const int64_t all = int64_t(n_tiles) * pieces;
    const int share = blockIdx.y * WAVES + wave, shares = gridDim.y * WAVES;
    const int64_t lo = all * share / shares, hi = all * (share + 1) / shares;
    for (int64_t at = lo; at < hi;) {
        const int i = __builtin_amdgcn_readfirstlane(int(at / pieces)), c0 = int(at - int64_t(i) * pieces);
        const int c1 = int(min(int64_t(pieces), c0 + hi - at));
        at += c1 - c0;
        const int e = __builtin_amdgcn_readfirstlane(entry[3 * i]);
        const int first = __builtin_amdgcn_readfirstlane(entry[3 * i + 1]);
        const int n = __builtin_amdgcn_readfirstlane(entry[3 * i + 2]);
        const uint8_t *code[RF], *scale[RF];
#pragma unroll
        for (int m = 0; m < RF; ++m) {
            const int64_t row = int64_t(e) * L.D + min(d0 + 16 * m + r, L.D - 1);
            code[m] = L.dc + row * L.steps_f * kStepBytes + g * 16;
            scale[m] = L.ds + row * kStepScales;
        }
        const int pair = order[first + min(r, n - 1)];
        const __bf16* h = L.hp + pair * Fp + g * 32;
        f32x4 acc[RF] = {};
        struct Loaded {
            u32x4 code[RF];
            uint32_t scale[RF];
            bf16x8 v[PH][4];
        };
        auto load = [&](Loaded& l, int c) {
#pragma unroll
            for (int m = 0; m < RF; ++m) {
                l.code[m] = *reinterpret_cast<const u32x4*>(code[m] + c * 64);
                l.scale[m] = *reinterpret_cast<const uint32_t*>(scale[m] + c / 2 * rows * kStepScales + c % 2 * 4);
            }
#pragma unroll
            for (int p = 0; p < PH; ++p) load_block(l.v[p], h + p * part_of_h + c * 128);
        };
        auto use = [&](const Loaded& l) {
#pragma unroll
            for (int m = 0; m < RF; ++m) {
                bf16x8 o[4];
                decode(l.code[m], l.scale[m] >> (8 * g), o);
#pragma unroll
                for (int p = PH - 1; p >= 0; --p)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(o[q], l.v[p][q], acc[m], 0, 0, 0);
            }
        };
        in_pairs<Loaded>(c0, c1, 1, load, use);
        // a token has an expert once, so no two lanes add to one place
        if (r < n)
#pragma unroll
            for (int m = 0; m < RF; ++m) {
                f32x4* to = reinterpret_cast<f32x4*>(mine + pair / L.k * kWide + 16 * m + 4 * g);
                *to = *to + acc[m];
            }
    }
    __syncthreads();
    for (int o = threadIdx.x; o < L.T * 16 * RF; o += WAVES * 64) {
        const int t = o / (16 * RF), c = o % (16 * RF);
        if (d0 + c >= L.D) continue;
        float y = 0.f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) y += sums[(w * L.T + t) * kWide + c];
        if (gridDim.y == 1)
            Y[int64_t(t) * ldy + d0 + c] = from_f32<TY>(y);
        else
            L.sums[(int64_t(blockIdx.y) * L.T + t) * L.D + d0 + c] = y;
    }
}

// The same product through the ring, 256 outputs a workgroup, whose waves take
// its run of pieces together.
constexpr int kRingWaves = 8, kRingRows = 256;

template <typename TY, int PH, int S>
__global__ __launch_bounds__(kRingWaves * 64, 2) void moe_down_ring_kernel(Layer L, TY* __restrict__ Y, int64_t ldy) {
    using R = Ring<PH, kRingWaves>;
    static_assert(R::kRows == kRingRows, "outputs of a workgroup");
    constexpr int kWide = 32 + 4;
    __shared__ __align__(256) uint8_t l0[R::kBytes], l1[R::kBytes], l2[R::kBytes], l3[S > 3 ? R::kBytes : 16];
    extern __shared__ __align__(16) float sums[];  // wave x token x kWide, then the lists
    int* entry = reinterpret_cast<int*>(sums + kRingWaves * L.T * kWide);
    const int n_tiles = L.lists[0], most = most_tiles(L.T, L.E, L.k);
    int16_t* order = reinterpret_cast<int16_t*>(entry + 3 * most);
    for (int i = threadIdx.x; i < 3 * most; i += kRingWaves * 64) entry[i] = L.lists[1 + i];
    for (int i = threadIdx.x; i < L.T * L.k; i += kRingWaves * 64) order[i] = L.order[i];
    for (int i = threadIdx.x; i < kRingWaves * L.T * kWide; i += kRingWaves * 64) sums[i] = 0.f;
    __syncthreads();
    const int64_t d0 = int64_t(blockIdx.x) * kRingRows;
    const int pieces = int(L.steps_f) * 2;
    const int64_t all = int64_t(n_tiles) * pieces;
    const int lo = int(all * blockIdx.y / gridDim.y), hi = int(all * (blockIdx.y + 1) / gridDim.y);
    const int there = int(min(int64_t(kRingRows), L.D - d0));
    R ring(L.dc, L.ds, int64_t(L.E) * L.D, R::kRange, there, there - R::kRange, L.steps_f, L.hp, int64_t(L.T) * L.k);
    const int r = ring.lane & 15, g = ring.lane >> 4;
    float* mine = sums + ring.wave * L.T * kWide;
    if (lo < hi) {
        int tile = lo / pieces, column = lo % pieces, copied = lo;  // the next copy's piece
        int64_t row0 = 0;
        auto start_tile = [&]() {
            const int e = __builtin_amdgcn_readfirstlane(entry[3 * tile]);
            const int first = __builtin_amdgcn_readfirstlane(entry[3 * tile + 1]);
            const int n = __builtin_amdgcn_readfirstlane(entry[3 * tile + 2]);
            row0 = int64_t(e) * L.D + d0;
            ring.set_tile([&](int i) { return order[first + min(i, n - 1)]; });
        };
        start_tile();
        f32x4 acc[2] = {};
        int used = tile, left = min(pieces - column, hi - lo), more = hi - lo;  // of the tile in use, of all
        through_ring<S, R::kCopies>(
            l0, l1, l2, l3, hi - lo,
            [&](uint8_t* stage) {
                ring.copy(stage, row0, column);
                if (++copied < hi && ++column == pieces) {
                    column = 0;
                    ++tile;
                    start_tile();
                }
            },
            [&](const uint8_t* stage) {
                ring.multiply(stage, acc);
                --more;
                if (--left) return;
                // the end of a tile, or of the run
                const int first = entry[3 * used + 1], n = entry[3 * used + 2];
                if (r < n) {
                    float* to = mine + order[first + r] / L.k * kWide + 4 * g;
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        f32x4* at = reinterpret_cast<f32x4*>(to + 16 * m);
                        *at = *at + acc[m];
                    }
                }
                acc[0] = acc[1] = f32x4{};
                ++used;
                left = min(pieces, more);
            });
    }
    // a wave's own sums: 16 outputs of each range
    for (int o = ring.lane; o < L.T * 32; o += 64) {
        const int t = o / 32, c = o % 32;
        const int64_t d = d0 + c / 16 * R::kRange + ring.wave * 16 + c % 16;
        if (d >= L.D) continue;
        const float y = mine[t * kWide + c];
        if (gridDim.y == 1)
            Y[int64_t(t) * ldy + d] = from_f32<TY>(y);
        else
            L.sums[(int64_t(blockIdx.y) * L.T + t) * L.D + d] = y;
    }
}

constexpr int kJoinThreads = 256;

// The workgroups' sums, in their order: an output a thread, 16 loads in flight.
template <typename TY>
__global__ __launch_bounds__(kJoinThreads) void moe_join_kernel(Layer L, TY* __restrict__ Y, int64_t ldy, int splits) {
    const int64_t d = int64_t(blockIdx.x) * kJoinThreads + threadIdx.x, stride = int64_t(L.T) * L.D;
    if (d >= L.D) return;
    const float* p = L.sums + int64_t(blockIdx.y) * L.D + d;
    float y = 0.f;
#pragma unroll 16
    for (int i = 0; i < splits; ++i) y += p[i * stride];
    Y[int64_t(blockIdx.y) * ldy + d] = from_f32<TY>(y);
}

// bf16 parts of x and h for a type of x.
constexpr int x_parts(int type) { return type == RETRO_BF16 ? 1 : type == RETRO_F16 ? 2 : 3; }
constexpr int h_parts(int type) { return type == RETRO_F32 ? 3 : 2; }
template <typename TX> constexpr int type_of();
template <> constexpr int type_of<float>() { return RETRO_F32; }
template <> constexpr int type_of<_Float16>() { return RETRO_F16; }
template <> constexpr int type_of<__bf16>() { return RETRO_BF16; }

// The down kernel's shape: outputs of a workgroup, waves, and workgroups that
// share the pieces.
struct Down {
    bool ring;
    int rows, waves, splits;
    int64_t blocks(int64_t D) const { return host::cdiv(D, rows); }
    int64_t lds(int64_t T, int64_t E, int64_t k) const {
        const int64_t wide = ring ? 32 + 4 : rows + 4;
        return waves * T * wide * 4 + 12 * most_tiles(T, E, k) + 2 * T * k;
    }
};

Down down_shape(int xtype, int64_t T, int64_t D, int64_t F, int64_t E, int64_t k) {
    const int64_t items = std::min(E, T * k) * steps_of(F) * 2;
    // Few pieces, as for single tokens: one workgroup of 16 waves, no parts to add
    // (1 token, 4 of 32 experts, D = 2048, F = 1024, 32 pieces: the layer in 16.4 us
    // against 18.8; 2 of 8, D = 4096, F = 4096, 64: 24.7 against 25.9; 8 of 64, F = 2048,
    // 128: 31.5 against 27.1).
    if (T <= 16 && items <= 64) return {false, 16, 16, 1};
    // The staged kernel addresses h with 32 bits, and holds four or (many tokens)
    // three stages beside the tokens' sums; those of F32 fit up to 32 tokens (2 of 8,
    // D = 4096, F = 14336: the layer in 217 us with 32 and 272 with 33).
    const int parts = h_parts(xtype);
    const bool fits = parts * T * k * steps_of(F) * 512 < (int64_t(1) << 32) && (parts < 3 || T <= 32);
    const int rows = fits ? kRingRows : 32;
    // as many workgroups as CUs, each at least four pieces (sixteen: 1 token, 4 of 16
    // experts, D = 2048, F = 5120 in 37.7 us instead of 29.9)
    const int64_t slabs = host::cdiv(D, rows);
    return {fits, rows, 8, int(std::max<int64_t>(1, std::min(host::cdiv(host::kNumCUs, slabs), items / 4)))};
}

// The workspace's pieces, each on a 256-byte boundary.
struct Pieces {
    int64_t logits, share, lists, order, xp, hp, sums, all;
};

Pieces pieces(int xtype, int64_t T, int64_t D, int64_t F, int64_t E, int64_t k) {
    Pieces p{};
    int64_t at = 0;
    auto put = [&](int64_t& where, int64_t bytes) {
        where = at;
        at += host::cdiv(bytes, 256) * 256;
    };
    put(p.logits, T * E * 4);
    put(p.share, T * k * 4);
    put(p.lists, (1 + 3 * most_tiles(T, E, k)) * 4);
    put(p.order, T * k * 2);
    put(p.xp, x_parts(xtype) * T * steps_of(D) * kStep * 2);
    put(p.hp, h_parts(xtype) * T * k * steps_of(F) * kStep * 2);
    const Down s = down_shape(xtype, T, D, F, E, k);
    put(p.sums, s.splits > 1 ? s.splits * T * D * 4 : 0);
    p.all = at;
    return p;
}

template <typename TX, typename TR>
int launch_layer(const Layer& L, const TX* X, int64_t ldx, const TR* R, int64_t ldr, TX* Y, int64_t ldy,
                 int renormalize, hipStream_t st) {
    constexpr int PX = x_parts(type_of<TX>()), PH = h_parts(type_of<TX>());
    const int groups = int(host::cdiv(L.E, kRouterWaves));
    const int64_t cuts = host::cdiv(L.steps_d * kStep, kRouterWaves * 64 * 8);
    const int tiles = most_tiles(L.T, L.E, L.k);
    const bool aligned = mx::aligned(X, 16) && mx::aligned(R, 16) && ldx * int64_t(sizeof(TX)) % 16 == 0 &&
                         ldr * int64_t(sizeof(TR)) % 16 == 0;
    host::clear_last_error();
    // a token a wave while that leaves CUs to fill (32 tokens, 8 experts, D = 4096: 4.8
    // us against 8.4 with four), else four, which read R a fourth as often
    auto router = [&](auto kernel, int tokens) {
        kernel<<<dim3(uint32_t(groups + cuts), uint32_t(host::cdiv(L.T, tokens))), dim3(kRouterWaves * 64), 0, st>>>(
            L, X, ldx, R, ldr, groups, aligned);
    };
    if (L.E * L.T <= 8 * host::kNumCUs)
        router(moe_router_kernel<TX, TR, PX, 1>, 1);
    else
        router(moe_router_kernel<TX, TR, PX, 4>, 4);
    const bool own_lists = L.T <= kGateWaves;
    if (!own_lists) moe_choose_kernel<<<dim3(1), dim3(kChooseWaves * 64), 0, st>>>(L, renormalize);
    // 64 features a workgroup through the ring where that makes one a CU (1 token, 2
    // of 8 experts, D = 4096, F = 8192, 256 of them: 44 us against 46 for the layer; F =
    // 14336: 50 against 55; F = 4096, 128: 30 against 25, all with one set of weights, part
    // of which the last cache holds; 32 tokens, F = 14336: 177 against 208, with 128
    // features 182). Else 16, four times as many workgroups.
    const int64_t ring_slabs = L.steps_f * (kStep / (16 * kRingWavesUp));
    if (ring_slabs * tiles >= host::kNumCUs) {
        auto gate_up = [&](void (*kernel)(Layer, int)) {
            kernel<<<dim3(uint32_t(ring_slabs), tiles), dim3(kRingWavesUp * 64), 0, st>>>(L, renormalize);
        };
        own_lists ? gate_up(moe_gate_up_ring_kernel<PX, PH, true>) : gate_up(moe_gate_up_ring_kernel<PX, PH, false>);
    } else {
        auto gate_up = [&](void (*kernel)(Layer, int)) {
            kernel<<<dim3(uint32_t(L.steps_f * (kStep / 16)), tiles), dim3(kGateWaves * 64), 0, st>>>(L, renormalize);
        };
        own_lists ? gate_up(moe_gate_up_kernel<PX, PH, true>) : gate_up(moe_gate_up_kernel<PX, PH, false>);
    }
    const Down s = down_shape(type_of<TX>(), L.T, L.D, L.F, L.E, L.k);
    auto down = [&](void (*kernel)(Layer, TX*, int64_t)) {
        kernel<<<dim3(uint32_t(s.blocks(L.D)), s.splits), dim3(s.waves * 64),
                 size_t(s.lds(L.T, L.E, L.k)), st>>>(L, Y, ldy);
    };
    if (s.waves == 16)
        down(moe_down_kernel<TX, PH, 1, 16>);
    else if (!s.ring)
        down(moe_down_kernel<TX, PH, 2, 8>);
    else if (L.T <= 32)
        down(moe_down_ring_kernel<TX, PH, 4>);
    else if constexpr (PH < 3)
        down(moe_down_ring_kernel<TX, PH, 3>);
    if (s.splits > 1)
        moe_join_kernel<<<dim3(uint32_t(host::cdiv(L.D, kJoinThreads)), L.T), dim3(kJoinThreads), 0, st>>>(L, Y, ldy,
                                                                                                        s.splits);
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
    L.share = reinterpret_cast<float*>(base + p.share);
    L.lists = reinterpret_cast<int*>(base + p.lists);
    L.order = reinterpret_cast<int16_t*>(base + p.order);
    L.xp = reinterpret_cast<__bf16*>(base + p.xp);
    L.hp = reinterpret_cast<__bf16*>(base + p.hp);
    L.sums = reinterpret_cast<float*>(base + p.sums);
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
