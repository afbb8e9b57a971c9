// retro_mx_host.h - host-side checks shared by the entry points of
// retro_mx.h. No device code.
#pragma once

#include <algorithm>

#include "retro_host.h"
#include "retro_mx.h"

namespace retro {
namespace mx {

// Workgroups (of at most 512 threads) of one launch, whose threads have to stay
// below 2^32; larger work is cut into several launches.
constexpr int64_t kMaxBlocks = int64_t(1) << 22;
constexpr int64_t kMaxThreads = (int64_t(1) << 32) - 1;

// f(first, blocks) for each launch of `blocks` workgroups.
template <typename F>
int in_block_ranges(int64_t blocks, F&& f) {
    for (int64_t b = 0; b < blocks; b += kMaxBlocks) {
        host::clear_last_error();
        f(b, uint32_t(std::min(kMaxBlocks, blocks - b)));
        const int rc = host::launch_status();
        if (rc != RETRO_OK) return rc;
    }
    return RETRO_OK;
}

inline int float_bytes(int type) {
    return type == RETRO_F32 ? 4 : type == RETRO_F16 || type == RETRO_BF16 ? 2 : 0;
}

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

inline bool dim_ok(int64_t n) { return n >= 0 && n < host::kDimLimit; }

// Bytes from the first to the last element of rows x cols floats ld apart; -1
// beyond the limit (or for ld < cols). An empty tensor spans nothing.
inline int64_t span_bytes(int64_t rows, int64_t cols, int64_t ld, int size) {
    if (ld < cols) return -1;
    if (rows == 0 || cols == 0) return 0;
    if (rows > 1 && ld > (host::kByteLimit / size - cols) / (rows - 1)) return -1;
    return ((rows - 1) * ld + cols) * size;
}

inline int64_t code_bytes(int64_t rows, int64_t K) { return rows * host::cdiv(K, 256) * 128; }
inline int64_t scale_bytes(int64_t rows, int64_t K) { return rows * host::cdiv(K, 256) * 8; }

struct Span {
    const void* p;
    int64_t n;
};

inline bool overlap(const Span& a, const Span& b) {
    if (a.n <= 0 || b.n <= 0 || !a.p || !b.p) return false;
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
    return pa < pb + uint64_t(b.n) && pb < pa + uint64_t(a.n);
}

// Calls f with a null pointer of the C++ type of a float type.
template <typename F>
int with_float(int type, F&& f) {
    switch (type) {
        case RETRO_F32: return f(static_cast<float*>(nullptr));
        case RETRO_F16: return f(static_cast<_Float16*>(nullptr));
        case RETRO_BF16: return f(static_cast<__bf16*>(nullptr));
        default: return RETRO_E_TYPE;
    }
}

// Launches shared between files (arguments checked by the caller).
int launch_quantize_rows(int xtype, const void* X, int64_t ldx, int64_t rows, int64_t K, void* codes, void* scales,
                         hipStream_t st);
int launch_product(int variant, int ytype, const void* ac, const void* as, const void* bc, const void* bs, void* Y,
                   int64_t ldy, int64_t K, int64_t N, int64_t T, hipStream_t st);
// Whether a variant takes a shape and row stride of Y (of elements of `size` bytes).
bool product_applies(int variant, int size, int64_t ldy, int64_t K, int64_t N, int64_t T);

}  // namespace mx
}  // namespace retro
