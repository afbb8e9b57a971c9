// retro_vocab_host.h - launches over the rows of one weight type that the
// operators of retro_vocab.h share, defined in retro_unit.hip (one object per
// type). Arguments are checked by the caller. No device code.
#pragma once

#include "retro_mx_host.h"
#include "retro_vocab.h"

namespace retro {
namespace ce {
struct FewArgs;
}
namespace vocab {

// The 16-byte pieces of 16-bit rows that a matrix-core step takes: K in whole 64s.
constexpr int64_t kStepK = 64;
inline int64_t padded(int64_t K) { return K > 0 ? host::cdiv(K, kStepK) * kStepK : kStepK; }

// Bytes that the address of every row has to be a multiple of (retro_api.hip).
int row_alignment(int type);

struct EmbedArgs {
    const uint8_t* W;
    int64_t ldw;      // bytes
    const void* ids;  // RETRO_I32 or RETRO_I64
    bool wide_ids;
    void* Y;
    int64_t ldy;  // elements
    float scale;
    int64_t K, N, T;
};

// Rows of W as 16-bit planes in steps of 64 elements: element k of row r at
// (k / 64 * padded(rows) + r) * 64 + k % 64, zeros past K and past the rows.
struct PlaneArgs {
    const uint8_t* W;  // the first row
    int64_t ldw;       // bytes
    int64_t rows, K;
    uint16_t* out;
    int64_t plane;        // elements from the first part's plane to the second's
    const uint32_t* top;  // bits of the table's largest finite magnitude (parts > 0)
    int parts;            // 0: W's own 16-bit elements; 1, 2: F16 parts scaled by top's power of two
};

template <int TYPE>
int launch_embed(int ytype, const EmbedArgs& a, hipStream_t st);
template <int TYPE>
int launch_planes(const PlaneArgs& a, hipStream_t st);
// *top = the larger of *top and the largest finite magnitude's bits of `rows` rows.
template <int TYPE>
int launch_top(const uint8_t* W, int64_t ldw, int64_t rows, int64_t K, uint32_t* top, hipStream_t st);

// The logits of up to 64 tokens through packed rows, in one launch (retro_ce_few.h).
// The weight types that it takes:
inline bool few_type(int type) {
    return type == RETRO_Q4_0 || type == RETRO_Q4_1 || type == RETRO_Q5_0 || type == RETRO_Q5_1 || type == RETRO_Q8_0 ||
           type == RETRO_MXFP4 || type == RETRO_Q4_K || type == RETRO_Q5_K || type == RETRO_Q6_K;
}
// Runs of the head's rows that it gives statistics of.
inline int64_t few_runs(int64_t rows) { return host::cdiv(rows, 32); }
template <int TYPE>
int launch_few(bool prob, int parts, const ce::FewArgs& a, hipStream_t st);

// Calls f with a std::integral_constant of a weight type.
template <typename F>
int with_type(int type, F&& f) {
    switch (type) {
#define RETRO_TYPE(t) \
    case t: return f(std::integral_constant<int, t>{})
        RETRO_TYPE(RETRO_F32);
        RETRO_TYPE(RETRO_F16);
        RETRO_TYPE(RETRO_BF16);
        RETRO_TYPE(RETRO_Q4_0);
        RETRO_TYPE(RETRO_Q4_1);
        RETRO_TYPE(RETRO_Q5_0);
        RETRO_TYPE(RETRO_Q5_1);
        RETRO_TYPE(RETRO_Q8_0);
        RETRO_TYPE(RETRO_Q2_K);
        RETRO_TYPE(RETRO_Q3_K);
        RETRO_TYPE(RETRO_Q4_K);
        RETRO_TYPE(RETRO_Q5_K);
        RETRO_TYPE(RETRO_Q6_K);
        RETRO_TYPE(RETRO_MXFP4);
        RETRO_TYPE(RETRO_NVFP4);
#undef RETRO_TYPE
        default: return RETRO_E_TYPE;
    }
}

}  // namespace vocab
}  // namespace retro
