// retro_ce_kernel.h - the matrix products of the cross entropy over a
// vocabulary: C[i][j] = sum_k A[i][k] B[j][k] of 16-bit rows, with what becomes
// of C done in the registers that hold it, so that no logits are kept.
//
//   kStats  A rows of the head, B tokens: per 32 BT rows of the head and token the
//           largest logit and the sum of exp(l - largest), and the target's logit
//   kProb   the same logits again: d = exp(l - lse) - [target], written as 16-bit
//           operands of the gradients' products: rows of tokens, and of the head
//           times dloss
//   kSum    C itself, in F32 (added to what is there) or rounded to the result's type
//
// Tokens are the columns of a matrix-core block: a lane then holds rows of the head of
// one token, whose maximum and sum need two exchanges, with the three other lanes of it.
//
// The power that the matrix cores draw bounds the large tiles: 4096 x 131072 x 4096 in
// BF16 takes 3.37 ms as kStats (1.31 PFLOP/s), 3.41 as dW and dX and 3.62 as kProb, which
// writes 2.1 GB besides; a library product of that size, its result written and nothing
// more, takes 2.9 to 3.2. Eight waves of 128 x 64 results: four of 128 x 128 ran at 1.17
// PFLOP/s, and three steps of A in LDS with two of B at 1.27. Few tokens are bound by the
// head's reading: one through 32768 x 2048, 134 MB, takes 22 us.
#pragma once

#include <type_traits>

#include "retro_vocab_device.h"

namespace retro {
namespace ce {

using mx::f32x4;
using mx::i32x4;
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

enum Kind { kStats, kProb, kSum };

constexpr int kStepBytes = 128;  // 64 elements of a row

// c += a b, 16 x 16 results of 32 k. 32 x 32 of 16 k move twice the results through the
// registers for the same work, which costs power, and power is what bounds the clock:
// alone, on random operands, they run at 1.86 PFLOP/s, these at 2.13. Written as
// assembly so that a result stays in its registers: the compiler moves results of this
// size from one set to another, runs out of them and spills in the loop. The wait states
// are for operands that a vector instruction has just written. That no result is moved or
// read too early is the compiler's doing, and read from the built code by a test
// (tests/test_vocab_products_build.py).
__device__ __forceinline__ void mfma(__bf16, const i32x4& a, const i32x4& b, f32x4& c) {
    asm volatile("s_nop 1\n\tv_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+v"(c) : "v"(a), "v"(b));
}
__device__ __forceinline__ void mfma(_Float16, const i32x4& a, const i32x4& b, f32x4& c) {
    asm volatile("s_nop 1\n\tv_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+v"(c) : "v"(a), "v"(b));
}
// Results of products issued before can be read after it: of 8 passes, 11 wait states
// after the last. The compiler sees each result written anew.
template <int N>
__device__ __forceinline__ void results_ready(f32x4 (&c)[N], bool first) {
    if (first) asm volatile("s_nop 15\n\ts_nop 3" : "+v"(c[0]));
#pragma unroll
    for (int j = 0; j < N; ++j) asm volatile("" : "+v"(c[j]));
}

// exp(x) for x <= 0 or so: off by |x| 2^-24 and a step, of a value that falls with x.
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896340736f); }

// Rows of 16-bit elements in one or two parts. A row's elements lie in steps of 64 (128
// bytes), `stride` apart: 128 bytes for rows as they are in a tensor, or the whole
// column of that step's 64 elements of all rows. What is made for the products is laid
// out so: a tile's step is then one run of memory. Rows of 64 KB side by side, 256 of
// them read at one place, took a sixth longer (4096 x 131072 x 4096 4.2 ms against 3.6).
struct Operand {
    const uint8_t* p;
    int64_t pitch, stride;  // bytes between rows, between steps of a row
    int64_t plane, bytes;   // bytes from the first part to the second, and of one
    int64_t rows;
};

struct Args {
    Operand a, b;
    uint32_t steps;       // of 64 elements in a row
    uint32_t pairs;       // products of parts: (1, 1), or the first two or three of `order`
    uint32_t order;       // part of A in bit 2p, part of B in bit 2p + 1 of product p
    uint32_t tiles_a, tiles_b, group, splits;
    // kStats, kProb: token factors and targets
    const float* factor;   // what a token's sums are multiplied with (NULL: 1)
    const uint32_t* top;   // and, with factor, W's scale
    const void* targets;
    bool wide_targets;
    int64_t N, n0;         // rows of the head in all, and before A's first
    // kStats
    float2* part;          // [runs of 32 BT rows][T]
    int64_t part0;         // first run
    float* at_target;      // [T]
    // kProb
    const float* lse;
    const float* weight;   // a token's factor in `across` (NULL: no `across`); 0 where it is not learnt from
    float by;              // factor of `along`
    uint16_t *along, *across;            // rows of tokens; rows of the head; both in steps
    int64_t along_stride, along_plane, along_cols;     // elements; columns written, whole 64s
    int64_t across_stride, across_plane, across_cols;
    // kSum
    void* out;
    int64_t ldo, split_stride;           // elements
    const float* out_factor;             // (NULL: 1)
    int64_t cols;                        // of C that are written
};

// Workgroup of WA x WB waves, each BA x BB blocks of 32 x 32, and S steps' tiles in LDS.
// Two steps suffice where the products take as long as a copy; tiles of few tokens are
// bound by the head's copies, and hold more of them in flight.
template <int WA_, int WB_, int BA_, int BB_, int S_ = 2>
struct Tile {
    static constexpr int WA = WA_, WB = WB_, BA = BA_, BB = BB_, S = S_;
    static constexpr int kWaves = WA * WB;
    static constexpr int kRowsA = 32 * WA * BA, kRowsB = 32 * WB * BB;
    static constexpr int kBytes = (kRowsA + kRowsB) * kStepBytes;  // LDS of one step
    static constexpr int kCopies = kBytes / (1024 * kWaves);       // 1 KB copies a wave and step
    static constexpr int kFit = 160 * 1024 / (S * kBytes), kPerCU = kFit < 4 ? kFit : 4;
    static constexpr int kThreads = kWaves * 64;
    static constexpr int kPerSimd = kWaves * kPerCU / 4 < 8 ? (kWaves * kPerCU + 3) / 4 : 8;
    static_assert(kRowsA * kStepBytes % (1024 * kWaves) == 0 && kRowsB * kStepBytes % (1024 * kWaves) == 0,
                  "a copy lies in one operand");
};

// One step's tiles from memory into LDS, without registers: a wave's copy moves 8
// pieces of 128 bytes, which become 8 rows of LDS.
//   A and, but in kSum, B: a row is a row of the operand, its 64 elements along k. The
//     16-byte blocks of row r land permuted by XOR with (r / 2) % 8, so that the 16 lanes
//     of a read of one block from neighbouring rows meet all banks once.
//   B in kSum, whose k runs over the operand's rows: LDS row 64 c + k holds columns
//     64 c .. 64 c + 63 of row k, permuted by XOR with twice (k / 2) % 4, so that the four
//     rows of a transposing read lie in banks of their own.
// What lies past the operand reads as zeros (the buffer's bound).
// The lane's bytes from its wave's first row of a copy. What else differs between a
// wave's copies of an operand is uniform and part of the buffer's address, so that one
// register serves all of them.
__device__ __forceinline__ uint32_t lane_bytes(uint32_t pitch, bool columns, int wave, int lane) {
    const uint32_t r = lane >> 3, slot = lane & 7;
    return (wave * 8 + r) * pitch + (slot ^ (columns ? (r >> 1) << 1 : (wave & 1) * 4 + (r >> 1))) * 16;
}

// Where an operand's tile of a step begins, and the bytes from there to its end.
struct Cursor {
    const uint8_t* p;
    int64_t left;
    // What lies `further` on, nothing of it where that is past the end.
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(int64_t further) const {
        const int64_t n = left - further;
        const int32_t high = int32_t(n >> 32);
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p + further), 0,
                                                 int(high < 0 ? 0u : high > 0 ? 0xffffffffu : uint32_t(n)), 0x00020000);
    }
};

// All but every wave's last N copies into LDS have landed, its reads are done, and
// every wave is here. A wave's counters cover its own work only, so the wait comes
// before the barrier.
template <int N>
__device__ __forceinline__ void copies_done_for_all() {
    static_assert(N < 64, "what the counter holds");
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (N == 0)
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    else {
        __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4) << 14 | 0x70);  // vmcnt(N) lgkmcnt(0)
        asm volatile("s_barrier" ::: "memory");
    }
    __builtin_amdgcn_sched_barrier(0);
}

// What the wave's lanes wrote to LDS before is what they read after.
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// A transposing read of LDS: see `across`.
__device__ __forceinline__ s16x4 column4(const uint8_t* lds) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) s16x4*)(const_cast<uint8_t*>(lds)));
}

// The parts of v as element `at` of w: d in the bits that the result has (8 or 11, two parts
// for F32), whose rounding is that of the result's own size; two parts of it double a product.
template <typename E, int PARTS>
__device__ __forceinline__ void put_parts(float v, int at, u16x4 (&w)[PARTS]) {
    w[0][at] = __builtin_bit_cast(uint16_t, E(v));
    if constexpr (PARTS == 2) w[1][at] = __builtin_bit_cast(uint16_t, E(vocab::rest_of<E>(v)));
}

// 8 elements to a place of any alignment of which `left` lie in the row.
__device__ __forceinline__ void put8(uint16_t* to, int64_t left, const u16x8& w) {
    typedef uint16_t any __attribute__((ext_vector_type(8), aligned(2)));
    if (left >= 8) {
        *reinterpret_cast<any*>(to) = w;
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left) to[i] = w[i];
}

template <typename E, class Z, Kind KIND, typename TO, int PARTS>
__global__ __launch_bounds__(Z::kThreads, Z::kPerSimd) void product_kernel(const Args g) {
    constexpr int WB = Z::WB, BA = Z::BA, BB = Z::BB;
    constexpr int NA = 2 * BA, NB = 2 * BB;  // 16 x 16 blocks
    // arrays of their own: the compiler sees which a copy goes to
    __shared__ __align__(1024) uint8_t lds0[Z::kBytes];
    __shared__ __align__(1024) uint8_t lds1[Z::kBytes];
    __shared__ __align__(1024) uint8_t lds2[Z::S > 2 ? Z::kBytes : 1];
    __shared__ __align__(1024) uint8_t lds3[Z::S > 3 ? Z::kBytes : 1];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
    const int r = lane & 15, h = lane >> 4, wa = wave / WB, wb = wave % WB;

    // Workgroups go to the 8 XCDs in turn; each XCD takes a contiguous range of
    // tiles, in groups of `group` tiles of B by all of A, so that the workgroups
    // that share its L2 at one time form a block of tiles.
    const uint32_t tiles = g.tiles_a * g.tiles_b, all = tiles * g.splits, per = all / 8, more = all % 8;
    const uint32_t x = blockIdx.x % 8;
    uint32_t id = x * per + min(x, more) + blockIdx.x / 8;
    const uint32_t split = id / tiles;
    id -= split * tiles;
    const uint32_t gr = id / (g.group * g.tiles_a), in = id - gr * g.group * g.tiles_a;
    const uint32_t high = min(g.group, g.tiles_b - gr * g.group);
    const int64_t b0 = int64_t(gr * g.group + in % high) * Z::kRowsB, a0 = int64_t(in / high) * Z::kRowsA;

    constexpr bool kColumns = KIND == kSum;
    // Steps of this split; step s is k = s % steps of product s / steps.
    const uint32_t total = g.steps * g.pairs;
    const uint32_t begin = uint32_t(uint64_t(total) * split / g.splits);
    const uint32_t end = uint32_t(uint64_t(total) * (split + 1) / g.splits);
    // Tiles of few tokens begin at steps of their own: rows a power of two apart, all
    // read at one place, would come from few memory channels.
    const uint32_t turn = Z::S > 2 && !kColumns ? uint32_t(a0 / Z::kRowsA * 5 % g.steps) : 0;
    // The step to be copied next: its cursors move on by a step, and begin anew with a
    // product of parts.
    Cursor at_a, at_b;
    uint32_t next = begin, next_k = 0;
    const int64_t step_a = g.a.stride, step_b = kColumns ? 64 * g.b.pitch : g.b.stride;
    const int64_t tile_a = a0 * g.a.pitch, tile_b = kColumns ? b0 / 64 * g.b.stride : b0 * g.b.pitch;
    auto seek = [&]() {
        const uint32_t p = (next >= g.steps) + (next >= 2 * g.steps);
        next_k = next - p * g.steps;
        const uint32_t k = Z::S > 2 && !kColumns ? (next_k + turn < g.steps ? next_k + turn : next_k + turn - g.steps) : next_k;
        const int64_t from_a = tile_a + k * step_a, from_b = tile_b + k * step_b;
        at_a = {g.a.p + ((g.order >> (2 * p)) & 1 ? g.a.plane : 0) + from_a, g.a.bytes - from_a};
        at_b = {g.b.p + ((g.order >> (2 * p + 1)) & 1 ? g.b.plane : 0) + from_b, g.b.bytes - from_b};
    };
    // To the step after it, or nowhere from the last one.
    auto advance = [&]() {
        if (next + 1 >= end) return;
        ++next;
        ++next_k;
        if (next_k == g.steps || (Z::S > 2 && !kColumns && next_k + turn == g.steps)) {
            seek();
        } else {
            at_a.p += step_a;
            at_a.left -= step_a;
            at_b.p += step_b;
            at_b.left -= step_b;
        }
    };
    // A wave's i-th copy of an operand is kTurn rows further on than the one before.
    constexpr int kTurn = 8 * Z::kWaves, kCopiesA = Z::kRowsA / kTurn;
    static_assert(Z::kWaves % 2 == 0 && kTurn <= 64, "a wave's copies are permuted alike");
    const uint32_t lane_a = lane_bytes(uint32_t(g.a.pitch), false, wave, lane);
    const uint32_t lane_b = lane_bytes(uint32_t(g.b.pitch), kColumns, wave, lane);
    auto part = [&](uint8_t* lds, int i) {
        uint8_t* to = lds + (i * Z::kWaves + wave) * 8 * kStepBytes;
        const int row = (i < kCopiesA ? i : i - kCopiesA) * kTurn;
        if (i < kCopiesA)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(at_a.resource(row * g.a.pitch), to, 16, lane_a, 0, 0, 0);
        else
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                at_b.resource(kColumns ? row / 64 * g.b.stride + row % 64 * g.b.pitch : row * g.b.pitch), to, 16, lane_b, 0,
                0, 0);
    };
    auto copy = [&](uint8_t* lds) {
#pragma unroll
        for (int i = 0; i < Z::kCopies; ++i) part(lds, i);
        advance();
    };

    // LDS offsets of the lane's elements of its first row, k 0 .. 31 and 32 .. 63
    uint32_t off[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) off[s] = r * kStepBytes + (((4 * s + h) ^ ((r >> 1) & 7)) * 16);
    const uint32_t base_a = wa * BA * 32 * kStepBytes, base_b = (Z::kRowsA + wb * BB * 32) * kStepBytes;
    // Of columns: 16 lanes read 4 rows of k by 16 columns and get a column's four each.
    // Lane l of them reads 4 elements of row l / 4 of the four, the second read's four
    // rows follow the first's.
    uint32_t across[2][NB];
    if constexpr (kColumns)
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                const uint32_t k = 8 * h + 4 * half + r / 4, col = wb * BB * 32 + j * 16 + r % 4 * 4, c = col % 64;
                across[half][j] = (Z::kRowsA + col / 64 * 64 + k) * kStepBytes +
                                  (((c / 8) ^ ((k >> 1 & 3) << 1)) * 16) + c % 8 * 2;
            }
    i32x4 fa[NA], fb[2][NB];
    // The wave's i-th 16 rows of A and of B, half s of a step.
    auto read_a = [&](const uint8_t* lds, int s, int i) {
        fa[i] = *reinterpret_cast<const i32x4*>(lds + base_a + off[s] + i * 16 * kStepBytes);
    };
    auto read_b = [&](const uint8_t* lds, int s, int j) {
        if constexpr (kColumns) {
            const s16x4 v0 = column4(lds + across[0][j] + s * 32 * kStepBytes);
            const s16x4 v1 = column4(lds + across[1][j] + s * 32 * kStepBytes);
            fb[s][j] = __builtin_bit_cast(i32x4, s16x8{v0[0], v0[1], v0[2], v0[3], v1[0], v1[1], v1[2], v1[3]});
        } else {
            fb[s][j] = *reinterpret_cast<const i32x4*>(lds + base_b + off[s] + j * 16 * kStepBytes);
        }
    };
    f32x4 acc[NA][NB] = {};

    // One step from `cur`, whose copies are done and whose first half is in registers:
    // its products, and among them the reads of its second half, and then of the next
    // step's first. A's registers hold one half: 16 rows' are read again as soon as their
    // products are issued. A quarter into the second half's products everyone has read
    // all of cur and the next step's copies are in `nxt`; from there on cur is refilled
    // with the step S after its own. A product occupies the matrix core for 16 cycles, in
    // which what stands between it and the next is issued; all reads or copies before the
    // products kept the matrix core waiting. Past the last step the last one is copied
    // again, so that the loop has no branches.
    auto run = [&](uint8_t* cur, const uint8_t* nxt) {
        auto half = [&](auto which) {
            constexpr int B = decltype(which)::value;
            constexpr int kProducts = NA * NB, kSync = kProducts / 4, kFrom = B ? kSync : 0;
#pragma unroll
            for (int m = 0; m < kProducts; ++m) {
                if (B == 1 && m == kSync) {
                    __builtin_amdgcn_s_setprio(0);
                    copies_done_for_all<(Z::S - 2) * Z::kCopies>();
                }
                mfma(E(), fa[m / NB], fb[B][m % NB], acc[m / NB][m % NB]);
                const uint8_t* from = B ? nxt : cur;
#pragma unroll
                for (int i = 0; i < NA; ++i)
                    if (m == (i * NB + NB > kFrom + i ? i * NB + NB - 1 : kFrom + i)) read_a(from, 1 - B, i);
#pragma unroll
                for (int j = 0; j < NB; ++j)
                    if (m == (kFrom + 1 + 2 * j < kProducts ? kFrom + 1 + 2 * j : kProducts - 1)) read_b(from, 1 - B, j);
                if constexpr (B == 1)
#pragma unroll
                    for (int i = 0; i < Z::kCopies; ++i)
                        if (m == kSync + (i + 1) * (kProducts - 1 - kSync) / Z::kCopies) part(cur, i);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        __builtin_amdgcn_s_setprio(1);
        half(std::integral_constant<int, 0>{});
        half(std::integral_constant<int, 1>{});
        advance();
    };
    if (begin < end) {
        seek();
        copy(lds0);
        copy(lds1);
        if constexpr (Z::S > 2) copy(lds2);
        if constexpr (Z::S > 3) copy(lds3);
        copies_done_for_all<(Z::S - 1) * Z::kCopies>();
#pragma unroll
        for (int i = 0; i < NA; ++i) read_a(lds0, 0, i);
#pragma unroll
        for (int j = 0; j < NB; ++j) read_b(lds0, 0, j);
        uint32_t s = begin;
        for (; s + Z::S <= end; s += Z::S) {
            run(lds0, lds1);
            run(lds1, Z::S > 2 ? lds2 : lds0);
            if constexpr (Z::S > 2) run(lds2, Z::S > 3 ? lds3 : lds0);
            if constexpr (Z::S > 3) run(lds3, lds0);
        }
        if (s < end) run(lds0, lds1);
        if (Z::S > 2 && s + 1 < end) run(lds1, Z::S > 2 ? lds2 : lds0);
        if (Z::S > 3 && s + 2 < end) run(lds2, lds3);
        copies_done_for_all<0>();  // the copies past the end are done before LDS is given up
    }
#pragma unroll
    for (int i = 0; i < NA; ++i) results_ready(acc[i], i == 0);

    // Element v of a block: row 4 h + v of A, row r of B.
    const int64_t aw = a0 + wa * BA * 32, bw = b0 + wb * BB * 32;
    // The wave's own part of LDS, in which 16-bit results change places so that a lane
    // stores 16 bytes of a row and a row's lanes whole lines.
    constexpr int kStage = Z::kBytes / ((Z::kWaves + 1) / 2);
    uint16_t* stage = reinterpret_cast<uint16_t*>((wave % 2 ? lds1 : lds0) + wave / 2 * kStage);
    if constexpr (KIND == kSum) {
        TO* out = static_cast<TO*>(g.out) + split * g.split_stride;
        const float f = g.out_factor ? *g.out_factor : 1.f;
        if constexpr (sizeof(TO) == 2) {
            constexpr int kPitch = BB * 32 + 8;
            static_assert(32 * kPitch * 2 <= kStage, "a block row fits");
#pragma unroll
            for (int i = 0; i < BA; ++i) {
#pragma unroll
                for (int v = 0; v < 8; ++v)
#pragma unroll
                    for (int j = 0; j < NB; ++j) {
                        const float c = acc[2 * i + v / 4][j][v % 4];
                        stage[(v / 4 * 16 + 4 * h + v % 4) * kPitch + j * 16 + r] =
                            __builtin_bit_cast(uint16_t, mx::from_f32<TO>(g.out_factor ? c * f : c));
                    }
                wave_fence();
                constexpr int kLanes = BB * 4, kRows = 64 / kLanes;  // lanes of a row, rows a store
#pragma unroll
                for (int p = 0; p < 32 / kRows; ++p) {
                    const int at = p * kRows + lane / kLanes, col = lane % kLanes * 8;
                    const u16x8 w = *reinterpret_cast<const u16x8*>(stage + at * kPitch + col);
                    const int64_t row = aw + i * 32 + at, left = g.cols - (bw + col);
                    if (row < g.a.rows) put8(reinterpret_cast<uint16_t*>(out + row * g.ldo + bw + col), left, w);
                }
                wave_fence();
            }
        } else {
#pragma unroll
            for (int i = 0; i < NA; ++i)
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const int64_t row = aw + i * 16 + 4 * h + v;
                    if (row >= g.a.rows) continue;
#pragma unroll
                    for (int j = 0; j < NB; ++j) {
                        const int64_t col = bw + j * 16 + r;
                        if (col >= g.cols) continue;
                        TO* to = out + row * g.ldo + col;
                        const float c = g.out_factor ? acc[i][j][v] * f : acc[i][j][v];
                        if constexpr (PARTS)  // of kSum: add
                            *to = *to + c;
                        else
                            *to = c;
                    }
                }
        }
        return;
    }

    const float by_top = g.factor ? vocab::unscale_of(*g.top) : 1.f;
    auto scaled = [&](int j, int64_t t) {
        if (!g.factor || t >= g.b.rows) return;
        const float f = g.factor[t] * by_top;  // first: either alone may be far from a logit's size
#pragma unroll
        for (int i = 0; i < NA; ++i)
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[i][j][v] = acc[i][j][v] * f;
    };
    // the target as a row of this lane's, were it one
    auto target_of = [&](int token) { return int64_t(token) - g.n0 - aw - 4 * h; };

    if constexpr (KIND == kStats) {
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const int64_t t = bw + j * 16 + r;
            if (t >= g.b.rows) continue;  // all lanes of a token alike
            scaled(j, t);
            const int64_t target = target_of(vocab::token_at(g.targets, g.wide_targets, t, g.N));
            if (aw + BA * 32 > g.a.rows)
#pragma unroll
                for (int i = 0; i < NA; ++i)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        if (aw + 4 * h + i * 16 + v >= g.a.rows) acc[i][j][v] = -__builtin_inff();
            if (target >= 0 && target < BA * 32)
#pragma unroll
                for (int i = 0; i < NA; ++i)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        if (target == i * 16 + v) g.at_target[t] = acc[i][j][v];
            float top = -__builtin_inff();
#pragma unroll
            for (int i = 0; i < NA; ++i)
#pragma unroll
                for (int v = 0; v < 4; ++v) top = fmaxf(top, acc[i][j][v]);
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const float from = top == -__builtin_inff() ? 0.f : top;
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < NA; ++i)
#pragma unroll
                for (int v = 0; v < 4; ++v) sum += exp_of(acc[i][j][v] - from);
            sum += __shfl_xor(sum, 16);
            sum += __shfl_xor(sum, 32);
            if (h == 0) g.part[(g.part0 + (a0 / 32 + wa * BA) / BA) * g.b.rows + t] = make_float2(top, sum);
        }
    }
    if constexpr (KIND == kProb) {
        float weight[NB];
        bool learnt[NB];
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            // logits become d; the padding past the last token and the last row is zeros
            const int64_t t = bw + j * 16 + r;
            const int token = t < g.b.rows ? vocab::token_at(g.targets, g.wide_targets, t, g.N) : -1;
            learnt[j] = token >= 0;
            weight[j] = learnt[j] && g.weight ? g.weight[t] : 0.f;
            const float lse = learnt[j] ? g.lse[t] : 0.f;
            const int64_t target = target_of(token);
            scaled(j, t);
#pragma unroll
            for (int i = 0; i < NA; ++i)
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[i][j][v] = learnt[j] ? exp_of(acc[i][j][v] - lse) : 0.f;
            if (target >= 0 && target < BA * 32)
#pragma unroll
                for (int i = 0; i < NA; ++i)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        if (target == i * 16 + v) acc[i][j][v] -= 1.f;
            if (aw + BA * 32 > g.a.rows)
#pragma unroll
                for (int i = 0; i < NA; ++i)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        if (aw + 4 * h + i * 16 + v >= g.a.rows) acc[i][j][v] = 0.f;
        }
        if (g.along) {
            // rows of tokens: a lane has four neighbouring elements of its token's row
            constexpr int kBlocks = PARTS == 2 && BA > 1 ? BA / 2 : BA;  // of 32 rows of the head at a time
            constexpr int kPitch = kBlocks * 32 + 8, kLanes = kBlocks * 4, kRows = 64 / kLanes, kPlane = 32 * kPitch;
            static_assert(PARTS * kPlane * 2 <= kStage, "32 tokens' rows fit");
#pragma unroll
            for (int j = 0; j < BB; ++j)
#pragma unroll
                for (int i0 = 0; i0 < BA; i0 += kBlocks) {
#pragma unroll
                    for (int i = 0; i < 2 * kBlocks; ++i)
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            u16x4 w[PARTS];
#pragma unroll
                            for (int v = 0; v < 4; ++v) put_parts<E, PARTS>(acc[2 * i0 + i][2 * j + q][v] * g.by, v, w);
#pragma unroll
                            for (int part = 0; part < PARTS; ++part)
                                *reinterpret_cast<u16x4*>(stage + part * kPlane + (q * 16 + r) * kPitch + i * 16 + 4 * h) =
                                    w[part];
                        }
                    wave_fence();
#pragma unroll
                    for (int p = 0; p < 32 / kRows; ++p) {
                        const int at = p * kRows + lane / kLanes, col = lane % kLanes * 8;
                        const int64_t t = bw + j * 32 + at, row = aw + i0 * 32 + col;
                        if (t < g.b.rows && row < g.along_cols)
#pragma unroll
                            for (int part = 0; part < PARTS; ++part)
                                *reinterpret_cast<u16x8*>(g.along + part * g.along_plane + row / 64 * g.along_stride +
                                                          t * 64 + row % 64) =
                                    *reinterpret_cast<const u16x8*>(stage + part * kPlane + at * kPitch + col);
                    }
                    wave_fence();
                }
        }
        if (g.across) {
            constexpr int kPitch = BB * 32 + 8, kLanes = BB * 4, kRows = 64 / kLanes, kPlane = 32 * kPitch;
            static_assert(PARTS * kPlane * 2 <= kStage, "32 rows of the head fit");
#pragma unroll
            for (int i = 0; i < BA; ++i) {
#pragma unroll
                for (int v = 0; v < 8; ++v)
#pragma unroll
                    for (int j = 0; j < NB; ++j) {
                        u16x4 w[PARTS];
                        put_parts<E, PARTS>(learnt[j] ? acc[2 * i + v / 4][j][v % 4] * weight[j] : 0.f, 0, w);
#pragma unroll
                        for (int part = 0; part < PARTS; ++part)
                            stage[part * kPlane + (v / 4 * 16 + 4 * h + v % 4) * kPitch + j * 16 + r] = w[part][0];
                    }
                wave_fence();
#pragma unroll
                for (int p = 0; p < 32 / kRows; ++p) {
                    const int at = p * kRows + lane / kLanes, col = lane % kLanes * 8;
                    const int64_t row = aw + i * 32 + at, t = bw + col;
                    if (row < g.a.rows && t < g.across_cols)
#pragma unroll
                        for (int part = 0; part < PARTS; ++part)
                            *reinterpret_cast<u16x8*>(g.across + part * g.across_plane + t / 64 * g.across_stride +
                                                      row * 64 + t % 64) =
                                *reinterpret_cast<const u16x8*>(stage + part * kPlane + at * kPitch + col);
                }
                wave_fence();
            }
        }
    }
}

}  // namespace ce
}  // namespace retro
