// retro_mx_tile.h - the tiled product of two microscaled matrices: operand
// tiles copied to LDS while the matrix cores work on the tiles before them.
//
// What bounds the 256 x 256 tile (eight waves of 128 x 64, the choice for large
// products): power. On random operands the scaled products alone run at 5.8 PFLOP/s
// at a clock of 1.5 GHz, on zeros at 8.2. 8192^3 takes 270 us (4.1 PFLOP/s); with
// nothing but its products and barriers 203 to 220, its LDS reads alone 121 and
// its copies alone 152 (the three share the clock, and LDS: of its 128 bytes a
// cycle the reads take 75%, the copies 25% at the products' full rate). Four waves of
// 128 x 128 read a third less but hide less: 297 us as scheduled by the compiler,
// 273 with the reads and copies placed among the products by hand, and 8% slower than
// eight waves at K = 4096. Stages of 128 elements, three or four deep, copy 64
// bytes of a row at a time: 201 us for the copies instead of 152.
// 4096 x 14336 x 4096: 144 to 155 us (3.1 to 3.3 PFLOP/s) in calls one after another,
// 172 traced one launch at a time; three and a half rounds of tiles.
#pragma once

#include <type_traits>

#include "retro_mx_device.h"

namespace retro {
namespace mx {

__device__ __forceinline__ i32x8 operand(const i32x4& v) { return i32x8{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }

template <int BYTE>
__device__ __forceinline__ f32x16 mfma32(const i32x4& a, const i32x4& b, const f32x16& c, int ea, int eb) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(a), operand(b), c, 4, 4, BYTE, ea, BYTE, eb);
}

// Workgroup of WT x WN waves, each BT x BN blocks of 32 x 32 outputs, so a tile
// of (32 WT BT) x (32 WN BN). A step is 256 elements of K: 128 code bytes a row.
// KG such groups of waves take the steps of K in turn and add their sums at the
// end: for few tiles, where a CU would wait on one step's copies after another.
template <int WT_, int WN_, int BT_, int BN_, int KG_ = 1>
struct Tile {
    static constexpr int WT = WT_, WN = WN_, BT = BT_, BN = BN_, KG = KG_;
    static constexpr int kWaves = WT * WN;  // of a group
    static constexpr int kRowsT = 32 * WT * BT, kRowsN = 32 * WN * BN;
    static constexpr int kBytes = (kRowsT + kRowsN) * kStepBytes;  // LDS of one step
    static constexpr int kCopies = kBytes / (1024 * kWaves);       // 1 KB copies a wave and step
    // workgroups a CU, by their two steps of LDS
    static constexpr int kFit = 160 * 1024 / (2 * kBytes * KG), kPerCU = kFit < 4 ? kFit : 4;
    static constexpr int kThreads = kWaves * KG * 64;
    static constexpr int kPerSimd = kWaves * KG * kPerCU / 4 < 8 ? (kWaves * KG * kPerCU + 3) / 4 : 8;
    static_assert(kRowsT * kStepBytes % (1024 * kWaves) == 0 && kRowsN * kStepBytes % (1024 * kWaves) == 0,
                  "a copy lies in one operand");
};

// One step's tiles from memory into LDS, without registers: a wave's copy
// moves 8 rows of 128 bytes. The 16-byte blocks of row r land in LDS permuted by
// XOR with (r / 2) % 8, so that the 16 lanes of a read of one block from
// neighbouring rows meet all banks once. Rows past the matrix read as zeros (the
// buffer's bound, against which the lane's offset is checked: the row is in it).
template <class Z>
__device__ __forceinline__ void copy_step(__amdgpu_buffer_rsrc_t a, __amdgpu_buffer_rsrc_t b, uint8_t* lds,
                                          uint32_t pitch, uint32_t step, int wave, int lane) {
    const uint32_t r = lane >> 3, slot = lane & 7;
#pragma unroll
    for (int i = 0; i < Z::kCopies; ++i) {
        const int at = (i * Z::kWaves + wave) * 8;  // first row of this copy
        const bool of_a = i * Z::kWaves * 8 < Z::kRowsT;
        const uint32_t row = at - (of_a ? 0 : Z::kRowsT);
        const uint32_t swz = ((row + r) >> 1) & 7;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(of_a ? a : b, lds + at * kStepBytes, 16,
                                                 (row + r) * pitch + ((slot ^ swz) * 16), step * kStepBytes, 0, 0);
    }
}

// Every wave's copies into LDS have landed, its reads are done, and every wave is
// here. A wave's counters cover its own work only, so the wait comes before the
// barrier.
__device__ __forceinline__ void copies_done_for_all() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

template <typename TY, class Z>
__global__ __launch_bounds__(Z::kThreads, Z::kPerSimd) void product_tile_kernel(
    const uint8_t* __restrict__ ac, const uint8_t* __restrict__ as, const uint8_t* __restrict__ bc,
    const uint8_t* __restrict__ bs, TY* __restrict__ Y, int64_t ldy, uint32_t steps, int64_t N, int64_t T,
    uint32_t tiles_n, uint32_t tiles_t, uint32_t group) {
    constexpr int WN = Z::WN, BT = Z::BT, BN = Z::BN;
    __shared__ __align__(1024) uint8_t all0[Z::KG * Z::kBytes];
    __shared__ __align__(1024) uint8_t all1[Z::KG * Z::kBytes];
    const int wave_of_all = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
    const int wave = wave_of_all % Z::kWaves, kg = wave_of_all / Z::kWaves;
    uint8_t *lds0 = all0 + kg * Z::kBytes, *lds1 = all1 + kg * Z::kBytes;
    const int r = lane & 31, h = lane >> 5, wt = wave / WN, wn = wave % WN;

    // Workgroups go to the 8 XCDs in turn; each XCD takes a contiguous range of
    // tiles, in groups of `group` tile rows by all tile columns, so that the
    // workgroups that share its L2 at one time form a block of tiles.
    const uint32_t all = tiles_n * tiles_t, per = all / 8, more = all % 8;
    const uint32_t x = blockIdx.x % 8, id = x * per + min(x, more) + blockIdx.x / 8;
    const uint32_t g = id / (group * tiles_n), in = id - g * group * tiles_n;
    const uint32_t high = min(group, tiles_t - g * group);
    const uint32_t tt = g * group + in % high, tn = in / high;
    const int64_t t0 = int64_t(tt) * Z::kRowsT, n0 = int64_t(tn) * Z::kRowsN;

    const uint32_t pitch = steps * kStepBytes;
    const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(ac + t0 * pitch), 0, uint32_t(min(int64_t(Z::kRowsT), T - t0) * pitch), 0x00020000);
    const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(bc + n0 * pitch), 0, uint32_t(min(int64_t(Z::kRowsN), N - n0) * pitch), 0x00020000);

    // scale words of the wave's rows; rows past the matrix take its last row's
    uint32_t sa[BT], sb[BN];
#pragma unroll
    for (int i = 0; i < BT; ++i) sa[i] = uint32_t(min(t0 + (wt * BT + i) * 32 + r, T - 1)) * kStepScales + h * 4;
#pragma unroll
    for (int i = 0; i < BN; ++i) sb[i] = uint32_t(min(n0 + (wn * BN + i) * 32 + r, N - 1)) * kStepScales + h * 4;
    auto load_scales = [&](int (&da)[BT], int (&db)[BN], uint32_t step) {
        const uint8_t *pa = as + int64_t(step) * T * kStepScales, *pb = bs + int64_t(step) * N * kStepScales;
#pragma unroll
        for (int i = 0; i < BT; ++i) da[i] = *reinterpret_cast<const int*>(pa + sa[i]);
#pragma unroll
        for (int i = 0; i < BN; ++i) db[i] = *reinterpret_cast<const int*>(pb + sb[i]);
    };

    // LDS offsets of the lane's block s of its first rows
    uint32_t off[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) off[s] = r * kStepBytes + (((4 * h + s) ^ ((r >> 1) & 7)) * 16);
    const uint32_t base_a = wt * BT * 32 * kStepBytes, base_b = (Z::kRowsT + wn * BN * 32) * kStepBytes;

    i32x4 fa[2][BT], fb[2][BN];
    auto read = [&](const uint8_t* lds, int s, i32x4 (&a)[BT], i32x4 (&b)[BN]) {
#pragma unroll
        for (int i = 0; i < BT; ++i) a[i] = *reinterpret_cast<const i32x4*>(lds + base_a + off[s] + i * 32 * kStepBytes);
#pragma unroll
        for (int i = 0; i < BN; ++i) b[i] = *reinterpret_cast<const i32x4*>(lds + base_b + off[s] + i * 32 * kStepBytes);
    };
    f32x16 acc[BT][BN] = {};

    // One step from `cur` (its copies done, block 0 in registers): the reads of
    // block s + 1 are issued ahead of block s's products; before the last
    // block's, everyone has read all of cur and the next step's copies are in
    // `nxt`, so cur is refilled with the step after that. Past the last step the
    // last one is copied again, so that the loop has no branches. `live` is false
    // where the last round has no step left for this group.
    int ea[2][BT], eb[2][BN];
    auto run = [&](uint8_t* cur, const uint8_t* nxt, uint32_t round, int (&ca)[BT], int (&cb)[BN], bool live) {
        auto block = [&](auto which) {
            constexpr int B = decltype(which)::value;
            if (!live) return;
#pragma unroll
            for (int i = 0; i < BT; ++i)
#pragma unroll
                for (int j = 0; j < BN; ++j)
                    acc[i][j] = mfma32<B>(fa[B % 2][i], fb[B % 2][j], acc[i][j], ca[i], cb[j]);
        };
        const uint32_t after = min((round + 2) * Z::KG + kg, steps - 1);
        read(cur, 1, fa[1], fb[1]);
        __builtin_amdgcn_sched_barrier(0);
        block(std::integral_constant<int, 0>{});
        read(cur, 2, fa[0], fb[0]);
        __builtin_amdgcn_sched_barrier(0);
        block(std::integral_constant<int, 1>{});
        read(cur, 3, fa[1], fb[1]);
        __builtin_amdgcn_sched_barrier(0);
        block(std::integral_constant<int, 2>{});
        copies_done_for_all();
        read(nxt, 0, fa[0], fb[0]);
        copy_step<Z>(ra, rb, cur, pitch, after, wave, lane);
        __builtin_amdgcn_sched_barrier(0);
        block(std::integral_constant<int, 3>{});
        load_scales(ca, cb, after);
    };

    const uint32_t first = min(uint32_t(kg), steps - 1), second = min(uint32_t(Z::KG + kg), steps - 1);
    copy_step<Z>(ra, rb, lds0, pitch, first, wave, lane);
    load_scales(ea[0], eb[0], first);
    copies_done_for_all();
    copy_step<Z>(ra, rb, lds1, pitch, second, wave, lane);
    load_scales(ea[1], eb[1], second);
    read(lds0, 0, fa[0], fb[0]);
    const uint32_t whole_rounds = steps / Z::KG;
    uint32_t round = 0;
    for (; round + 2 <= whole_rounds; round += 2) {
        run(lds0, lds1, round, ea[0], eb[0], true);
        run(lds1, lds0, round + 1, ea[1], eb[1], true);
    }
    if (Z::KG == 1) {
        if (round < whole_rounds) run(lds0, lds1, round, ea[0], eb[0], true);
    } else {
        if (round * Z::KG < steps) run(lds0, lds1, round, ea[0], eb[0], round * Z::KG + kg < steps);
        if ((round + 1) * Z::KG < steps) run(lds1, lds0, round + 1, ea[1], eb[1], (round + 1) * Z::KG + kg < steps);
    }
    copies_done_for_all();  // the copies past the end are done before LDS is given up or used again

    if constexpr (Z::KG > 1) {
        // the groups' sums, added in the order of the groups by the first
        static_assert((Z::KG - 1) * Z::kRowsT * Z::kRowsN * 4 <= Z::KG * Z::kBytes, "the sums fit");
        float* sums = reinterpret_cast<float*>(all0) + (kg - 1) * Z::kRowsT * Z::kRowsN;
        const int mine = wave * BT * BN * 16 * 64 + lane;
        if (kg > 0)
#pragma unroll
            for (int i = 0; i < BT; ++i)
#pragma unroll
                for (int j = 0; j < BN; ++j)
#pragma unroll
                    for (int v = 0; v < 16; ++v) sums[mine + ((i * BN + j) * 16 + v) * 64] = acc[i][j][v];
        __syncthreads();
        if (kg > 0) return;
        for (int k = 0; k < Z::KG - 1; ++k)
#pragma unroll
            for (int i = 0; i < BT; ++i)
#pragma unroll
                for (int j = 0; j < BN; ++j)
#pragma unroll
                    for (int v = 0; v < 16; ++v)
                        acc[i][j][v] += reinterpret_cast<const float*>(
                            all0)[k * Z::kRowsT * Z::kRowsN + mine + ((i * BN + j) * 16 + v) * 64];
    }

    // A register holds one row for 32 lanes: 32 neighbouring outputs a store.
    // Row addresses are uniform; the lane adds its 32-bit offset. The stores go
    // past the L2, which the operands need: 17408 x 5120 x 2048 to F32 in 144 us
    // against 162, 8192^3 in 278 against 292.
    const int64_t tw = t0 + wt * BT * 32, nw = n0 + wn * BN * 32;
    const uint32_t lane_at = (uint32_t(h) * 4 * uint32_t(ldy) + r) * uint32_t(sizeof(TY));
    const bool whole = tw + BT * 32 <= T && nw + BN * 32 <= N;
#pragma unroll
    for (int i = 0; i < BT; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
            const int64_t t = tw + i * 32 + (v / 4) * 8 + v % 4;
            char* row = reinterpret_cast<char*>(Y + t * ldy + nw) + lane_at;
#pragma unroll
            for (int j = 0; j < BN; ++j)
                if (whole || (t + h * 4 < T && nw + j * 32 + r < N))
                    __builtin_nontemporal_store(from_f32<TY>(acc[i][j][v]),
                                                reinterpret_cast<TY*>(row + j * 32 * sizeof(TY)));
        }
}

}  // namespace mx
}  // namespace retro
