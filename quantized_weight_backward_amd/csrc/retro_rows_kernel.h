// retro_rows_kernel.h - kernels over rows of one weight type: embedding lookup,
// and the rows of a table as 16-bit planes for the matrix cores.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "retro_kernels.h"
#include "retro_vocab_device.h"

namespace retro {
namespace vocab {

// Elements k .. k + 7 of a row, zeros past K (k a multiple of 8).
template <int TYPE>
__device__ __forceinline__ void row8(const uint8_t* row, int k, int K, int wide, float e[8]) {
    float a[4], b[4];
    skinny_load4<TYPE>(row, k, K, wide, a);
    if (k + 4 < K || Format<TYPE>::kBlock == 1)  // packed rows end with a block
        skinny_load4<TYPE>(row, k + 4, K, wide, b);
    else
        b[0] = b[1] = b[2] = b[3] = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        e[i] = a[i];
        e[4 + i] = b[i];
    }
}

// y[t] = scale * W[ids[t]]: a thread 8 elements. Memory bounds it: 16384 rows of 4096 in
// BF16 take 49 us, 5.4 TB/s read and written; a single token takes its launch.
template <int TYPE, typename TY, typename TI>
__global__ __launch_bounds__(256) void embed_kernel(const uint8_t* __restrict__ W, int64_t ldw,
                                                    const TI* __restrict__ ids, TY* __restrict__ Y, int64_t ldy,
                                                    float scale, int K, int64_t N, int64_t T, int wide, uint32_t per,
                                                    int64_t first) {
    const int64_t at = (first + blockIdx.x) * 256 + threadIdx.x;
    const int64_t t = at >> 32 ? at / per : int64_t(uint32_t(at) / per);
    if (t >= T) return;
    const int k = int(at - t * per) * 8;
    const int64_t id = ids[t];
    float e[8] = {};
    if (id >= 0 && id < N) {
        row8<TYPE>(W + id * ldw, k, K, wide, e);
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] *= scale;
    }
    store8(Y + t * ldy + k, K - k, e);
}

// Rows as planes (PlaneArgs): a thread 8 elements of a row. Rows past the last up to
// whole 64s are zeros. Bound by what it writes: 32768 rows of Q8_0 4096 in two parts
// 132 us, 5.1 TB/s with the reads.
template <int TYPE, int PARTS>
__global__ __launch_bounds__(256) void planes_kernel(const uint8_t* __restrict__ W, int64_t ldw, int64_t rows, int K,
                                                     uint16_t* __restrict__ out, int64_t plane,
                                                     const uint32_t* __restrict__ top, int wide, uint32_t per,
                                                     int64_t first) {
    const int64_t at = (first + blockIdx.x) * 256 + threadIdx.x;
    const int64_t r = at >> 32 ? at / per : int64_t(uint32_t(at) / per), all = (rows + 63) / 64 * 64;
    if (r >= all) return;
    const int k = int(at - r * per) * 8;
    float e[8] = {};
    if (k < K && r < rows) row8<TYPE>(W + r * ldw, k, K, wide, e);
    uint16_t* to = out + (k / 64 * all + r) * 64 + k % 64;
    if constexpr (PARTS == 0) {
        typedef typename std::conditional<TYPE == kBF16, __bf16, _Float16>::type E;
        store_part<E>(to, e);
    } else {
        const float s = scale_of(*top);
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] *= s;
        store_parts<_Float16, PARTS>(to, plane, e);
    }
}

// The largest finite magnitude's bits of a table: of the values themselves, since a
// block's scale says nothing of them where its codes are small or zero. An infinity or NaN
// is its own row's logit and says nothing of the others. Q8_0 131072 x 4096 223 us, 2.5 TB/s:
// bound by decoding (the scales alone took 98).
template <int TYPE>
__global__ __launch_bounds__(256) void top_kernel(const uint8_t* __restrict__ W, int64_t ldw, int64_t rows, int K,
                                                  uint32_t* __restrict__ top, int wide, uint32_t per) {
    // four groups of 8 in flight a thread
    uint32_t m = 0;
    const int64_t all = rows * per, step = int64_t(gridDim.x) * 256;
    for (int64_t at = int64_t(blockIdx.x) * 256 + threadIdx.x; at < all; at += 4 * step) {
        float e[4][8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t i = min(at + j * step, all - 1);  // the last group again past the end
            const int64_t r = i >> 32 ? i / per : int64_t(uint32_t(i) / per);
            row8<TYPE>(W + r * ldw, int(i - r * per) * 8, K, wide, e[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t bits = mx::abs_bits(e[j][i]);
                m = max(m, bits < 0x7f800000u ? bits : 0u);
            }
    }
    __shared__ uint32_t tops[4];
    m = wave_max(m);
    if (threadIdx.x % 64 == 0) tops[threadIdx.x / 64] = m;
    __syncthreads();
    m = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
    // a maximum is the same in whatever order. One address takes one atomic at a time:
    // those of 2048 workgroups took longer than the reads.
    if (threadIdx.x == 0 && m > __hip_atomic_load(top, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)) atomicMax(top, m);
}

}  // namespace vocab
}  // namespace retro
