// retro_ce.hip - softmax cross entropy through a resident head and its gradients
// (retro_vocab.h), in pieces of the head.
#include <algorithm>

#include "retro_ce_few.h"
#include "retro_ce_kernel.h"
#include "retro_vocab_host.h"

namespace retro {
namespace ce {
namespace {

using host::cdiv;
using mx::Span;

// ---------------------------------------------------------------- rows of tokens

// x as the matrix cores take it, in steps of 64 elements (element k of row t at
// (k / 64 * gridDim.x + t) * 64 + k % 64), zeros past K and past the last token, in x's
// own 16-bit type (PARTS 0) or as F16 parts scaled by a power of two of the row's own,
// whose inverse goes to factor[t]. Memory bounds it, or its launch. With a mask (the gradients' products) the rows of
// tokens that are not learnt from are zeros, whatever they hold. A workgroup a row.
template <typename TX, int PARTS>
__global__ __launch_bounds__(256) void token_rows_kernel(const TX* __restrict__ X, int64_t ldx, int64_t K,
                                                         const void* __restrict__ targets, bool wide_targets, int64_t N,
                                                         bool mask, uint16_t* __restrict__ out, int64_t padded_k,
                                                         int64_t T, float* __restrict__ factor) {
    const int64_t t = blockIdx.x;
    const bool live = t < T && (!mask || vocab::token_at(targets, wide_targets, t, N) >= 0);
    const TX* x = X + t * ldx;
    float s = 1.f;
    if constexpr (PARTS > 0) {
        __shared__ uint32_t tops[4];
        uint32_t m = 0;
        if (live)
            for (int64_t k = threadIdx.x * 8; k < K; k += 256 * 8) {
                float e[8];
                mx::load8(x + k, K - k, e);
#pragma unroll
                for (int i = 0; i < 8; ++i) m = max(m, mx::abs_bits(e[i]));
            }
        m = vocab::wave_max(m);
        if (threadIdx.x % 64 == 0) tops[threadIdx.x / 64] = m;
        __syncthreads();
        m = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
        s = vocab::scale_of(m);
        if (threadIdx.x == 0 && t < T) factor[t] = vocab::unscale_of(m);
    }
    for (int64_t k = threadIdx.x * 8; k < padded_k; k += 256 * 8) {
        float e[8] = {};
        if (live) mx::load8(x + k, K - k, e);
        uint16_t* to = out + (k / 64 * gridDim.x + t) * 64 + k % 64;
        if constexpr (PARTS == 0) {
            vocab::store_part<TX>(to, e);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] *= s;
            vocab::store_parts<_Float16, PARTS>(to, padded_k * gridDim.x, e);
        }
    }
}

// ---------------------------------------------------------------- what follows the products

// lse and loss from the runs' largest logits and sums, joined in an order that the
// sizes alone give. TT tokens a workgroup, 256 / TT threads each, four runs in flight.
template <int TT>
__global__ __launch_bounds__(256) void combine_kernel(const float2* __restrict__ part, int64_t runs, int64_t T,
                                                      const void* __restrict__ targets, bool wide_targets, int64_t N,
                                                      const float* __restrict__ at_target, float* __restrict__ loss,
                                                      float* __restrict__ lse) {
    constexpr int kPer = 256 / TT;
    __shared__ float2 held[kPer][TT];
    const int tt = threadIdx.x % TT, p = threadIdx.x / TT;
    const int64_t t = int64_t(blockIdx.x) * TT + tt;
    const float none = -__builtin_inff();
    float top = none, sum = 0.f;
    auto join = [&](float2 v) {
        const float m = fmaxf(top, v.x), from = m == none ? 0.f : m;
        sum = sum * exp_of(top - from) + v.y * exp_of(v.x - from);
        top = m;
    };
    if (t < T)
        for (int64_t i = p; i < runs; i += 4 * kPer) {
            float2 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = i + j * kPer < runs ? part[(i + j * kPer) * T + t] : make_float2(none, 0.f);
#pragma unroll
            for (int j = 0; j < 4; ++j) join(v[j]);
        }
    for (int d = kPer / 2; d > 0; d /= 2) {
        held[p][tt] = make_float2(top, sum);
        __syncthreads();
        if (p < d) join(held[p + d][tt]);
        __syncthreads();
    }
    if (p || t >= T) return;
    // the loss from differences: a small one beside a large logit has its digits below lse's
    const float over = sum == 0.f ? 0.f : logf(sum);
    lse[t] = top + over;
    loss[t] = vocab::token_at(targets, wide_targets, t, N) >= 0 ? top - at_target[t] + over : 0.f;
}

// Each token's factor in d^T: dloss and x's own, 0 where it is not learnt from, all
// scaled by one power of two whose inverse goes to *unscale. One workgroup.
__global__ __launch_bounds__(1024) void weights_kernel(const float* __restrict__ dloss, const float* __restrict__ factor,
                                                       const void* __restrict__ targets, bool wide_targets, int64_t N,
                                                       int64_t T, float* __restrict__ weight,
                                                       float* __restrict__ unscale) {
    __shared__ uint32_t tops[16];
    auto weight_of = [&](int64_t t) {
        if (vocab::token_at(targets, wide_targets, t, N) < 0) return 0.f;
        return factor ? dloss[t] * factor[t] : dloss[t];
    };
    uint32_t m = 0;
    for (int64_t t = threadIdx.x; t < T; t += 1024) m = max(m, mx::abs_bits(weight_of(t)));
    m = vocab::wave_max(m);
    if (threadIdx.x % 64 == 0) tops[threadIdx.x / 64] = m;
    __syncthreads();
    for (int i = 0; i < 16; ++i) m = max(m, tops[i]);
    const float s = vocab::scale_of(m);
    for (int64_t t = threadIdx.x; t < T; t += 1024) weight[t] = weight_of(t) * s;
    if (threadIdx.x == 0) *unscale = vocab::unscale_of(m);
}

// dX from the F32 sums of all splits, added in their order: times dloss and what the
// operands were scaled with; zeros where a token is not learnt from.
template <typename TX>
__global__ __launch_bounds__(256) void dx_kernel(const float* __restrict__ sums, int64_t splits, int64_t split_stride,
                                                 int64_t K, int64_t T, const float* __restrict__ dloss, float by,
                                                 const uint32_t* __restrict__ top, const void* __restrict__ targets,
                                                 bool wide_targets, int64_t N, TX* __restrict__ dX, int64_t lddx,
                                                 uint32_t per, int64_t first) {
    const int64_t at = (first + blockIdx.x) * 256 + threadIdx.x;
    const int64_t t = at >> 32 ? at / per : int64_t(uint32_t(at) / per);
    if (t >= T) return;
    const int64_t k = (at - t * per) * 8;
    float e[8] = {};
    if (vocab::token_at(targets, wide_targets, t, N) >= 0) {
        const float f = by * (top ? vocab::unscale_of(*top) : 1.f), d = dloss[t];
        const float* from = sums + t * K + k;
        mx::load8(from, K - k, e);
        for (int64_t s = 1; s < splits; ++s) {
            float more[8];
            mx::load8(from + s * split_stride, K - k, more);
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] += more[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = e[i] * f * d;
    }
    vocab::store8(dX + t * lddx + k, K - k, e);
}

__global__ __launch_bounds__(256) void zero_kernel(uint32_t* p, int64_t n) {
    const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (i < n) p[i] = 0;
}

template <typename TY>
__global__ __launch_bounds__(256) void zero_rows_kernel(TY* p, int64_t ld, int64_t cols, int64_t rows) {
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
        for (int64_t c = threadIdx.x; c < cols; c += 256) p[r * ld + c] = TY(0.f);
}

// ---------------------------------------------------------------- few tokens through packed blocks

constexpr int kRun = 4096;  // logits a workgroup of the two kernels below

// x in F32, rows together.
template <typename TX>
__global__ __launch_bounds__(256) void widen_kernel(const TX* __restrict__ X, int64_t ldx, int64_t K,
                                                    const void* __restrict__ targets, bool wide_targets, int64_t N,
                                                    bool mask, float* __restrict__ out) {
    const int64_t t = blockIdx.x;
    const bool live = !mask || vocab::token_at(targets, wide_targets, t, N) >= 0;
    for (int64_t k = threadIdx.x; k < K; k += 256) out[t * K + k] = live ? mx::to_f32(X[t * ldx + k]) : 0.f;
}

// Largest logit and sum of a run of a token's logits (grid: runs, T).
__global__ __launch_bounds__(256) void run_stats_kernel(const float* __restrict__ l, int64_t rows, int64_t T,
                                                        const void* __restrict__ targets, bool wide_targets, int64_t N,
                                                        int64_t n0, float2* __restrict__ part, int64_t part0,
                                                        float* __restrict__ at_target) {
    __shared__ float tops[4], sums[4];
    const int64_t t = blockIdx.y, at = int64_t(blockIdx.x) * kRun, target = vocab::token_at(targets, wide_targets, t, N);
    const float none = -__builtin_inff();
    float v[kRun / 256], top = none, sum = 0.f;
#pragma unroll
    for (int i = 0; i < kRun / 256; ++i) {
        const int64_t n = at + i * 256 + threadIdx.x;
        v[i] = n < rows ? l[t * rows + n] : none;
        top = fmaxf(top, v[i]);
        if (n < rows && n + n0 == target) at_target[t] = v[i];
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) top = fmaxf(top, __shfl_xor(top, d));
    if (threadIdx.x % 64 == 0) tops[threadIdx.x / 64] = top;
    __syncthreads();
    top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
    const float from = top == none ? 0.f : top;
#pragma unroll
    for (int i = 0; i < kRun / 256; ++i) sum += exp_of(v[i] - from);
#pragma unroll
    for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d);
    if (threadIdx.x % 64 == 0) sums[threadIdx.x / 64] = sum;
    __syncthreads();
    if (threadIdx.x == 0) part[(part0 + blockIdx.x) * T + t] = make_float2(top, sums[0] + sums[1] + sums[2] + sums[3]);
}

// The logits become d.
__global__ __launch_bounds__(256) void run_prob_kernel(float* __restrict__ l, int64_t rows,
                                                       const void* __restrict__ targets, bool wide_targets, int64_t N,
                                                       int64_t n0, const float* __restrict__ lse) {
    const int64_t t = blockIdx.y, at = int64_t(blockIdx.x) * kRun, target = vocab::token_at(targets, wide_targets, t, N);
    const float from = target >= 0 ? lse[t] : 0.f;
#pragma unroll
    for (int i = 0; i < kRun / 256; ++i) {
        const int64_t n = at + i * 256 + threadIdx.x;
        if (n >= rows) break;
        l[t * rows + n] = target >= 0 ? exp_of(l[t * rows + n] - from) - (n + n0 == target ? 1.f : 0.f) : 0.f;
    }
}

// ---------------------------------------------------------------- plans

using Big = Tile<2, 4, 4, 2>;     // 256 x 256
using Mid = Tile<2, 2, 2, 2>;     // 128 x 128
using Rows64 = Tile<4, 1, 1, 2, 3>;   // 128 rows of A by 64 of B
using Half64 = Tile<2, 1, 1, 2, 4>;   // 64 by 64
using Rows32 = Tile<4, 1, 1, 1, 4>;   // 128 by 32
using Cols64 = Tile<1, 4, 2, 1, 3>;   // 64 rows of A by 128 of B
using Cols32 = Tile<1, 4, 1, 1, 4>;

struct Call {
    int type, xtype;
    const uint8_t* W;
    int64_t ldw;
    const void* X;
    int64_t ldx;
    bool wide_targets;
    const void* targets;
    int64_t K, N, T;
    hipStream_t st;
};

bool is_float(int type) { return mx::float_bytes(type) != 0; }

// F16 parts that a type's values take: one holds the 8 and 11 bits of the 16-bit
// floats, the 2 of MXFP4 and the 6 of NVFP4, each under its scale.
int parts_of(int type) {
    return type == RETRO_F16 || type == RETRO_BF16 || type == RETRO_MXFP4 || type == RETRO_NVFP4 ? 1 : 2;
}

// And in dX of a BF16 x, where a value's 11 bits leave the sum's 8 as they are: an error
// of 2^-12 of each weight, beside d's; two parts double the product. (Not in the logits
// that d is made of: d = p - 1 of a confident token is a small difference, off by what its
// logits and lse are. Logits of one part, beside an lse of two, put an error of 1e-3 into
// d, several times 1 - p.) Beside an F32 dW, for which d has two parts, W has them too.
int sum_parts_of(int type, int xtype, bool weight_grad) {
    return xtype == RETRO_BF16 && !(weight_grad && type == RETRO_F32) ? 1 : parts_of(type);
}

// Both operands in one 16-bit type, which the matrix cores take as they are.
bool is_narrow(int type, int xtype) { return type == xtype && type != RETRO_F32; }

// Whether the head's rows can be copied to LDS where they are: 16-byte pieces, whole
// steps, and 256 rows within 32 bits.
bool is_direct(int type, int xtype, int64_t ldw, int64_t K) {
    return is_narrow(type, xtype) && K > 0 && K % vocab::kStepK == 0 && ldw % 16 == 0 && ldw < (1 << 24);
}

// Few tokens through packed blocks: decoded in registers, each block read once; making
// planes would write and read 4 bytes and more for every element. Of the types that
// few_kernel does not take the logits are the library's F32 products.
constexpr int64_t kFewT = 64;
bool is_few(int type, int64_t ldw, int64_t K, int64_t T) {
    return !is_float(type) && T <= kFewT && K > 0 && ldw == host::row_bytes_of(type, K);
}

// Rows of the head in one piece, a multiple of 256 and never 0.
int64_t piece_rows(int64_t N, int64_t most) {
    return std::max<int64_t>(256, std::min(cdiv(N, 256) * 256, most / 256 * 256));
}
// planes of at most 2^27 elements
int64_t plane_piece(int64_t K, int64_t N) { return piece_rows(N, std::min<int64_t>((1 << 27) / vocab::padded(K), 32768)); }
// d of at most 2^27 elements a plane, where that leaves 4096 rows for the sums over them
int64_t grad_piece(int64_t K, int64_t N, int64_t T) {
    return std::min(plane_piece(K, N), piece_rows(N, std::max<int64_t>((1 << 27) / std::max<int64_t>(T, 1), 4096)));
}
int64_t few_piece(int64_t N, int64_t T) { return piece_rows(N, (1 << 24) / std::max<int64_t>(T, 1)); }
// Elements of a token's row that few_kernel reads.
int64_t few_padded(int64_t K) { return cdiv(K, kFewK) * kFewK; }

// Parts of the workspace, each on a 256-byte boundary.
struct Bump {
    int64_t at = 0;
    int64_t take(int64_t bytes) {
        const int64_t here = at;
        at += cdiv(bytes, 256) * 256;
        return here;
    }
};

template <class Z>
int64_t runs_of(int64_t rows) { return cdiv(rows, Z::kRowsA) * Z::WA; }

// Tile of a number of the head's rows and of tokens: 256 x 256 where they leave few CUs
// idle.
enum Shape { kBig, kMid, kSmall64, kHalf64, kSmall32 };
Shape shape_of(int64_t rows, int64_t tokens) {
    if (tokens <= 32) return kSmall32;
    if (tokens <= 64) return cdiv(rows, 128) >= 2 * host::kNumCUs ? kSmall64 : kHalf64;
    if (tokens <= 128) return kMid;
    return cdiv(rows, 256) * cdiv(tokens, 256) >= 128 ? kBig : kMid;
}

// Rows of the head in whole rounds of 256 x 256 tiles over the CUs, where what is left
// would fill less than half of another: it goes to smaller tiles in a launch of its
// own. 50001 x 2048 and 1021 tokens: 784 tiles, three rounds and 16, 243 us in one launch
// and 219 in two.
int64_t rows_of_rounds(int64_t rows, int64_t tokens) {
    if (shape_of(rows, tokens) != kBig) return rows;
    const int64_t across = cdiv(tokens, 256), tiles = cdiv(rows, 256) * across, over = tiles % host::kNumCUs;
    if (tiles < host::kNumCUs || over == 0 || over >= host::kNumCUs / 2) return rows;
    const int64_t most = (tiles - over) / across * 256;
    return most ? most : rows;
}
Shape shape_of_rest(int64_t rows, int64_t tokens) {
    return cdiv(rows, 128) * cdiv(tokens, 128) >= host::kNumCUs ? kMid : kHalf64;
}

int64_t runs_in(Shape shape, int64_t rows) {
    switch (shape) {
        case kBig: return runs_of<Big>(rows);
        case kMid: return runs_of<Mid>(rows);
        case kSmall64: return runs_of<Rows64>(rows);
        case kHalf64: return runs_of<Half64>(rows);
        default: return runs_of<Rows32>(rows);
    }
}
int64_t logits_runs(int64_t rows, int64_t tokens) {
    const int64_t most = rows_of_rounds(rows, tokens), rest = rows - most;
    return runs_in(shape_of(rows, tokens), most) + (rest ? runs_in(shape_of_rest(rest, tokens), rest) : 0);
}

struct Forward {
    int64_t x, factor, top, planes, part, at_target, few_x, few_l, bytes, piece;
};

int64_t plane_bytes(int parts, int64_t rows, int64_t cols) { return 2 * std::max(parts, 1) * rows * cols; }

Forward forward_plan(int type, int64_t ldw, int xtype, int64_t K, int64_t N, int64_t T) {
    Forward p = {};
    Bump b;
    p.at_target = b.take(4 * T);
    if (is_few(type, ldw, K, T)) {
        if (vocab::few_type(type)) {  // 2^24 rows are 2^17 workgroups
            p.piece = piece_rows(N, 1 << 24);
            p.part = b.take(8 * T * cdiv(N, p.piece) * vocab::few_runs(p.piece));
            p.factor = b.take(4 * T);
            p.x = b.take(plane_bytes(parts_of(xtype), vocab::padded(T), few_padded(K)));
        } else {
            p.piece = few_piece(N, T);
            p.part = b.take(8 * T * (cdiv(N, p.piece) * cdiv(p.piece, kRun)));
            p.few_x = b.take(4 * T * K);
            p.few_l = b.take(4 * T * p.piece);
        }
        p.bytes = b.at;
        return p;
    }
    const bool narrow = is_narrow(type, xtype), direct = is_direct(type, xtype, ldw, K);
    // of a head read in place, at most 2^22 tiles of 128 x 128
    p.piece = direct ? piece_rows(N, std::min<int64_t>(1 << 24, (1 << 29) / cdiv(T, 128))) : plane_piece(K, N);
    p.x = b.take(plane_bytes(narrow ? 1 : parts_of(xtype), vocab::padded(T), vocab::padded(K)));
    p.factor = b.take(4 * T);
    p.top = b.take(4);
    p.planes = direct ? 0 : b.take(plane_bytes(narrow ? 1 : parts_of(type), p.piece, vocab::padded(K)));
    const int64_t whole = N / p.piece, rest = N % p.piece;
    p.part = b.take(8 * T * (whole * logits_runs(p.piece, T) + (rest ? logits_runs(rest, T) : 0)));
    p.bytes = b.at;
    return p;
}

struct Backward {
    int64_t x, factor, weight, unscale, top, planes, along, across, sums, few_x, few_l, few_ws, bytes;
    int64_t piece, splits;
    Shape shape;
};

// Tile and splits of dX's product, whose rows of the head are cut into splits so that
// every CU has work: one workgroup of 256 x 256 each, two of the smaller tiles, which is
// what fits at once (as many as fit and a rest took 178 us for the step of 64 tokens
// through 32768 x 4096, one round 169).
void sum_plan(int64_t K, int64_t T, int64_t steps, Backward& p) {
    const int64_t big = cdiv(T, 256) * cdiv(K, 256);
    int64_t tiles, want;
    if (T <= 32) {
        p.shape = kSmall32;
        tiles = cdiv(K, 128);
        want = 512;
    } else if (T <= 64) {
        p.shape = kSmall64;
        tiles = cdiv(K, 128);
        want = 512;
    } else if (T <= 128) {
        p.shape = kMid;
        tiles = cdiv(T, 128) * cdiv(K, 128);
        want = 512;
    } else {
        p.shape = kBig;
        tiles = big;
        want = 256;
    }
    p.splits = std::max<int64_t>(1, std::min<int64_t>({want / tiles, steps / 4, 64}));
}

Backward backward_plan(int type, int64_t ldw, int xtype, bool weight_grad, bool x_grad, int64_t K, int64_t N, int64_t T) {
    Backward p = {};
    Bump b;
    if (is_few(type, ldw, K, T)) {
        p.piece = few_piece(N, T);
        p.splits = cdiv(N, p.piece);
        if (vocab::few_type(type)) {
            p.factor = b.take(4 * T);
            p.x = b.take(plane_bytes(parts_of(xtype), vocab::padded(T), few_padded(K)));
        } else {
            p.few_x = b.take(4 * T * K);
        }
        p.few_l = b.take(4 * T * p.piece);
        p.sums = b.take(4 * p.splits * T * K);
        p.few_ws = b.take(host::kSplitWorkspaceMax);
        p.bytes = b.at;
        return p;
    }
    const bool narrow = is_narrow(type, xtype), direct = is_direct(type, xtype, ldw, K);
    const int64_t Kp = vocab::padded(K), Tp = vocab::padded(T);
    const int px = narrow ? 1 : parts_of(xtype), pw = narrow ? 1 : parts_of(type);
    const int pd = xtype == RETRO_F32 || (weight_grad && type == RETRO_F32) ? 2 : 1;
    p.piece = grad_piece(K, N, T);
    p.x = b.take(plane_bytes(px, Tp, Kp));
    p.factor = b.take(4 * T);
    p.top = b.take(4);
    p.unscale = b.take(4);
    p.planes = direct ? 0 : b.take(plane_bytes(pw, p.piece, Kp));
    if (weight_grad) {
        p.weight = b.take(4 * T);
        p.across = b.take(plane_bytes(pd, p.piece, Tp));
    }
    if (x_grad) {
        p.along = b.take(plane_bytes(pd, T, p.piece));
        sum_plan(K, T, p.piece / vocab::kStepK, p);
        p.sums = b.take(4 * p.splits * T * K);
    }
    p.bytes = b.at;
    return p;
}

// Products of parts: hi hi, hi lo, lo hi; lo lo is below the parts' own rounding.
void set_pairs(Args& g, int parts_a, int parts_b) {
    g.order = 0;
    g.pairs = 1;
    if (parts_a == 2) g.order |= 1u << (2 * g.pairs++);
    if (parts_b == 2) g.order |= 2u << (2 * g.pairs++);
}

template <typename E, class Z, Kind KIND, typename TO, int PARTS>
int launch(Args g, hipStream_t st) {
    g.tiles_a = uint32_t(cdiv(g.a.rows, Z::kRowsA));
    const int64_t cols = KIND == kSum ? g.cols : g.b.rows;
    g.tiles_b = uint32_t(cdiv(cols, Z::kRowsB));
    g.group = uint32_t(host::group_height(g.tiles_b, g.tiles_a, Z::kPerCU, double(cols), double(g.a.rows)));
    host::clear_last_error();
    product_kernel<E, Z, KIND, TO, PARTS>
        <<<dim3(g.tiles_a * g.tiles_b * g.splits), dim3(Z::kThreads), 0, st>>>(g);
    return host::launch_status();
}

template <typename E, Kind KIND, int PARTS>
int launch_shape(Shape shape, const Args& g, hipStream_t st) {
    switch (shape) {
        case kBig: return launch<E, Big, KIND, float, PARTS>(g, st);
        case kMid: return launch<E, Mid, KIND, float, PARTS>(g, st);
        case kSmall64: return launch<E, Rows64, KIND, float, PARTS>(g, st);
        case kHalf64: return launch<E, Half64, KIND, float, PARTS>(g, st);
        default: return launch<E, Rows32, KIND, float, PARTS>(g, st);
    }
}

#define RETRO_TRY(e)                     \
    do {                                 \
        const int rc_ = (e);             \
        if (rc_ != RETRO_OK) return rc_; \
    } while (0)

template <typename E, Kind KIND, int PARTS>
int launch_logits(Args g, hipStream_t st) {
    // the padding of `across`, to whole 64s of tokens, lies in the tiles
    const int64_t tokens = g.across ? std::max<int64_t>(g.b.rows, 33) : g.b.rows;
    const Shape shape = shape_of(g.a.rows, tokens);
    const int64_t most = rows_of_rounds(g.a.rows, tokens), rest = g.a.rows - most;
    g.a.rows = most;
    RETRO_TRY((launch_shape<E, KIND, PARTS>(shape, g, st)));
    if (!rest) return RETRO_OK;
    g.a.rows = rest;
    g.a.p += most * g.a.pitch;
    g.n0 += most;
    g.part0 += runs_in(shape, most);
    g.a.bytes -= most * g.a.pitch;
    if (g.along) g.along += most / vocab::kStepK * g.along_stride;
    g.along_cols -= most;
    if (g.across) g.across += most * vocab::kStepK;
    return launch_shape<E, KIND, PARTS>(shape_of_rest(rest, tokens), g, st);
}

template <typename E, bool ADD>
int launch_dx(Shape shape, const Args& g, hipStream_t st) {
    switch (shape) {
        case kBig: return launch<E, Big, kSum, float, ADD>(g, st);
        case kMid: return launch<E, Mid, kSum, float, ADD>(g, st);
        case kSmall64: return launch<E, Cols64, kSum, float, ADD>(g, st);
        default: return launch<E, Cols32, kSum, float, ADD>(g, st);
    }
}

template <typename E, typename TW>
int launch_dw(const Args& g, hipStream_t st) {
    if (cdiv(g.a.rows, 256) * cdiv(g.cols, 256) >= 128) return launch<E, Big, kSum, TW, 0>(g, st);
    return launch<E, Mid, kSum, TW, 0>(g, st);
}

int zero(void* p, int64_t words, hipStream_t st) {
    host::clear_last_error();
    zero_kernel<<<dim3(uint32_t(cdiv(words, 256))), dim3(256), 0, st>>>(static_cast<uint32_t*>(p), words);
    return host::launch_status();
}

int token_rows(const Call& c, int parts, bool mask, uint8_t* out, int64_t padded_k, float* factor) {
    return mx::with_float(c.xtype, [&](auto* tag) {
        using TX = std::remove_pointer_t<decltype(tag)>;
        auto kernel = parts == 2 ? token_rows_kernel<TX, 2> : token_rows_kernel<TX, 1>;
        if constexpr (sizeof(TX) == 2)
            if (parts == 0) kernel = token_rows_kernel<TX, 0>;
        host::clear_last_error();
        kernel<<<dim3(uint32_t(vocab::padded(c.T))), dim3(256), 0, c.st>>>(
            static_cast<const TX*>(c.X), c.ldx, c.K, c.targets, c.wide_targets, c.N, mask,
            reinterpret_cast<uint16_t*>(out), padded_k, c.T, factor);
        return host::launch_status();
    });
}

// Operands in steps, of rows of K elements (K in whole 64s).
Operand in_steps(const uint8_t* p, int64_t rows, int64_t all_rows, int64_t K) {
    return {p, vocab::kStepK * 2, all_rows * vocab::kStepK * 2, all_rows * K * 2, all_rows * K * 2, rows};
}

// Rows n0 .. n0 + rows of the head as an operand: in place, or as planes.
int head_rows(const Call& c, int64_t n0, int64_t rows, int parts, uint8_t* planes, const uint32_t* top, Operand& o) {
    if (is_direct(c.type, c.xtype, c.ldw, c.K)) {
        o = {c.W + n0 * c.ldw, c.ldw, vocab::kStepK * 2, 0, (rows - 1) * c.ldw + c.K * 2, rows};
        return RETRO_OK;
    }
    o = in_steps(planes, rows, vocab::padded(rows), vocab::padded(c.K));
    vocab::PlaneArgs a{c.W + n0 * c.ldw, c.ldw, rows, c.K, reinterpret_cast<uint16_t*>(planes), o.plane / 2, top,
                       is_narrow(c.type, c.xtype) ? 0 : parts};
    return vocab::with_type(c.type, [&](auto type) { return vocab::launch_planes<decltype(type)::value>(a, c.st); });
}

int head_top(const Call& c, uint32_t* top) {
    const int rc = zero(top, 1, c.st);
    if (rc != RETRO_OK || c.N == 0 || c.K == 0) return rc;
    return vocab::with_type(
        c.type, [&](auto type) { return vocab::launch_top<decltype(type)::value>(c.W, c.ldw, c.N, c.K, top, c.st); });
}

// The products' element type: BF16 only where both operands are.
template <typename F>
int with_element(const Call& c, F&& f) {
    return is_narrow(c.type, c.xtype) && c.type == RETRO_BF16 ? f(__bf16()) : f(_Float16());
}

int widen(const Call& c, bool mask, float* out) {
    return mx::with_float(c.xtype, [&](auto* tag) {
        using TX = std::remove_pointer_t<decltype(tag)>;
        host::clear_last_error();
        widen_kernel<TX><<<dim3(uint32_t(c.T)), dim3(256), 0, c.st>>>(static_cast<const TX*>(c.X), c.ldx, c.K, c.targets,
                                                                      c.wide_targets, c.N, mask, out);
        return host::launch_status();
    });
}

// What few_kernel takes of a call, but rows and results.
FewArgs few_args(const Call& c, const uint8_t* x, const float* factor) {
    FewArgs a = {};
    a.ldw = c.ldw;
    a.N = c.N;
    a.K = int(c.K);
    a.T = int(c.T);
    a.x = reinterpret_cast<const uint16_t*>(x);
    a.plane = vocab::padded(c.T) * few_padded(c.K);
    a.factor = factor;
    a.targets = c.targets;
    a.wide_targets = c.wide_targets;
    return a;
}

int few(const Call& c, FewArgs& a, int64_t n0, int64_t rows, bool prob) {
    a.W = c.W + n0 * c.ldw;
    a.n0 = n0;
    a.rows = rows;
    return vocab::with_type(c.type, [&](auto type) {
        return vocab::launch_few<decltype(type)::value>(prob, parts_of(c.xtype), a, c.st);
    });
}

int forward(const Call& c, float* loss, float* lse, uint8_t* ws) {
    const Forward p = forward_plan(c.type, c.ldw, c.xtype, c.K, c.N, c.T);
    float* at_target = reinterpret_cast<float*>(ws + p.at_target);
    float2* part = reinterpret_cast<float2*>(ws + p.part);
    int64_t runs = 0;
    if (c.N > 0 && is_few(c.type, c.ldw, c.K, c.T) && vocab::few_type(c.type)) {
        float* factor = reinterpret_cast<float*>(ws + p.factor);
        RETRO_TRY(token_rows(c, parts_of(c.xtype), false, ws + p.x, few_padded(c.K), factor));
        FewArgs a = few_args(c, ws + p.x, factor);
        a.part = part;
        a.at_target = at_target;
        for (int64_t n0 = 0; n0 < c.N; n0 += p.piece) {
            const int64_t rows = std::min(p.piece, c.N - n0);
            a.part0 = runs;
            RETRO_TRY(few(c, a, n0, rows, false));
            runs += vocab::few_runs(rows);
        }
    } else if (c.N > 0 && is_few(c.type, c.ldw, c.K, c.T)) {
        float *x = reinterpret_cast<float*>(ws + p.few_x), *l = reinterpret_cast<float*>(ws + p.few_l);
        RETRO_TRY(widen(c, false, x));
        for (int64_t n0 = 0; n0 < c.N; n0 += p.piece) {
            const int64_t rows = std::min(p.piece, c.N - n0), n = cdiv(rows, kRun);
            RETRO_TRY(retro_mul_mat(c.type, c.W + n0 * c.ldw, x, l, c.K, rows, c.T, c.st));
            host::clear_last_error();
            run_stats_kernel<<<dim3(uint32_t(n), uint32_t(c.T)), dim3(256), 0, c.st>>>(
                l, rows, c.T, c.targets, c.wide_targets, c.N, n0, part, runs, at_target);
            RETRO_TRY(host::launch_status());
            runs += n;
        }
    } else if (c.N > 0) {
        const bool narrow = is_narrow(c.type, c.xtype);
        float* factor = narrow ? nullptr : reinterpret_cast<float*>(ws + p.factor);
        uint32_t* top = narrow ? nullptr : reinterpret_cast<uint32_t*>(ws + p.top);
        if (!narrow) RETRO_TRY(head_top(c, top));
        Args g = {};
        g.b = in_steps(ws + p.x, c.T, vocab::padded(c.T), vocab::padded(c.K));
        // x in place where its rows are whole steps on 16-byte boundaries
        if (narrow && c.K > 0 && c.K % vocab::kStepK == 0 && c.ldx % 8 == 0 && c.ldx < (1 << 23) && mx::aligned(c.X, 16))
            g.b = {static_cast<const uint8_t*>(c.X), c.ldx * 2, vocab::kStepK * 2, 0, ((c.T - 1) * c.ldx + c.K) * 2, c.T};
        else
            RETRO_TRY(token_rows(c, narrow ? 0 : parts_of(c.xtype), false, ws + p.x, vocab::padded(c.K), factor));
        g.steps = uint32_t(vocab::padded(c.K) / vocab::kStepK);
        g.splits = 1;
        set_pairs(g, narrow ? 1 : parts_of(c.type), narrow ? 1 : parts_of(c.xtype));
        g.factor = factor;
        g.top = top;
        g.targets = c.targets;
        g.wide_targets = c.wide_targets;
        g.N = c.N;
        g.part = part;
        g.at_target = at_target;
        for (g.n0 = 0; g.n0 < c.N; g.n0 += p.piece) {
            const int64_t rows = std::min(p.piece, c.N - g.n0);
            RETRO_TRY(head_rows(c, g.n0, rows, parts_of(c.type), ws + p.planes, top, g.a));
            g.part0 = runs;
            RETRO_TRY(with_element(c, [&](auto e) { return launch_logits<decltype(e), kStats, 1>(g, c.st); }));
            runs += logits_runs(rows, c.T);
        }
    }
    host::clear_last_error();
    // neighbouring tokens' runs lie side by side: eight together where there are workgroups enough
    auto combine = c.T > 512 ? combine_kernel<8> : combine_kernel<1>;
    combine<<<dim3(uint32_t(cdiv(c.T, c.T > 512 ? 8 : 1))), dim3(256), 0, c.st>>>(
        part, runs, c.T, c.targets, c.wide_targets, c.N, at_target, loss, lse);
    return host::launch_status();
}

int finish_dx(const Call& c, const float* sums, int64_t splits, float by, const uint32_t* top, const float* dloss,
              void* dX, int64_t lddx) {
    const uint32_t per = uint32_t(cdiv(c.K, 8));
    return mx::with_float(c.xtype, [&](auto* tag) {
        using TX = std::remove_pointer_t<decltype(tag)>;
        return mx::in_block_ranges(cdiv(c.T * per, 256), [&](int64_t first, uint32_t blocks) {
            dx_kernel<TX><<<dim3(blocks), dim3(256), 0, c.st>>>(sums, splits, c.T * c.K, c.K, c.T, dloss, by, top,
                                                                c.targets, c.wide_targets, c.N, static_cast<TX*>(dX),
                                                                lddx, per, first);
        });
    });
}

int backward(const Call& c, const float* lse, const float* dloss, void* dX, int64_t lddx, void* dW, int64_t lddw,
             uint8_t* ws) {
    const Backward p = backward_plan(c.type, c.ldw, c.xtype, dW != nullptr, dX != nullptr, c.K, c.N, c.T);
    float* sums = reinterpret_cast<float*>(ws + p.sums);
    if (is_few(c.type, c.ldw, c.K, c.T)) {
        float *x = reinterpret_cast<float*>(ws + p.few_x), *l = reinterpret_cast<float*>(ws + p.few_l);
        const bool fused = vocab::few_type(c.type);
        float* factor = reinterpret_cast<float*>(ws + p.factor);
        if (fused)
            RETRO_TRY(token_rows(c, parts_of(c.xtype), true, ws + p.x, few_padded(c.K), factor));
        else
            RETRO_TRY(widen(c, true, x));
        FewArgs a = few_args(c, ws + p.x, factor);
        a.lse = lse;
        a.out = l;
        RETRO_TRY(zero(ws + p.few_ws, host::kSplitCountBytes / 4, c.st));
        int64_t done = 0;
        for (int64_t n0 = 0; n0 < c.N; n0 += p.piece, ++done) {
            const int64_t rows = std::min(p.piece, c.N - n0);
            const uint8_t* W = c.W + n0 * c.ldw;
            if (fused) {
                RETRO_TRY(few(c, a, n0, rows, true));
            } else {
                RETRO_TRY(retro_mul_mat(c.type, W, x, l, c.K, rows, c.T, c.st));
                host::clear_last_error();
                run_prob_kernel<<<dim3(uint32_t(cdiv(rows, kRun)), uint32_t(c.T)), dim3(256), 0, c.st>>>(
                    l, rows, c.targets, c.wide_targets, c.N, n0, lse);
                RETRO_TRY(host::launch_status());
            }
            RETRO_TRY(retro_out_prod_ws(RETRO_VARIANT_AUTO, c.type, W, l, sums + done * c.T * c.K, c.K, rows, c.T,
                                        ws + p.few_ws, host::kSplitWorkspaceMax, c.st));
        }
        return finish_dx(c, sums, done, 1.f, nullptr, dloss, dX, lddx);
    }

    const bool narrow = is_narrow(c.type, c.xtype);
    float* factor = narrow ? nullptr : reinterpret_cast<float*>(ws + p.factor);
    uint32_t* top = narrow ? nullptr : reinterpret_cast<uint32_t*>(ws + p.top);
    float *weight = reinterpret_cast<float*>(ws + p.weight), *unscale = reinterpret_cast<float*>(ws + p.unscale);
    const int px = narrow ? 1 : parts_of(c.xtype), pw = narrow ? 1 : parts_of(c.type);
    const int pd = c.xtype == RETRO_F32 || (dW && c.type == RETRO_F32) ? 2 : 1;
    const int64_t Kp = vocab::padded(c.K), Tp = vocab::padded(c.T);
    if (!narrow) RETRO_TRY(head_top(c, top));
    RETRO_TRY(token_rows(c, narrow ? 0 : px, true, ws + p.x, Kp, factor));
    if (dW) {
        host::clear_last_error();
        weights_kernel<<<dim3(1), dim3(1024), 0, c.st>>>(dloss, factor, c.targets, c.wide_targets, c.N, c.T, weight,
                                                         unscale);
        RETRO_TRY(host::launch_status());
    }
    // F16's d, at most 1, is scaled so that what is 2^28 below it keeps its bits
    const bool f16 = !(narrow && c.type == RETRO_BF16);
    const float by = f16 ? 0x1p14f : 1.f;

    Args g = {};
    const Operand x = g.b = in_steps(ws + p.x, c.T, Tp, Kp);
    g.steps = uint32_t(Kp / vocab::kStepK);
    g.splits = 1;
    set_pairs(g, pw, px);
    g.factor = factor;
    g.top = top;
    g.targets = c.targets;
    g.wide_targets = c.wide_targets;
    g.N = c.N;
    g.lse = lse;
    g.weight = dW ? weight : nullptr;
    g.by = by;
    g.along = dX ? reinterpret_cast<uint16_t*>(ws + p.along) : nullptr;
    g.across = dW ? reinterpret_cast<uint16_t*>(ws + p.across) : nullptr;
    for (g.n0 = 0; g.n0 < c.N; g.n0 += p.piece) {
        const int64_t rows = std::min(p.piece, c.N - g.n0), rows_p = vocab::padded(rows);
        RETRO_TRY(head_rows(c, g.n0, rows, pw, ws + p.planes, top, g.a));
        g.along_stride = c.T * vocab::kStepK;
        g.along_cols = rows_p;
        g.along_plane = c.T * rows_p;
        g.across_stride = rows * vocab::kStepK;
        g.across_cols = Tp;
        g.across_plane = rows * Tp;
        RETRO_TRY(with_element(c, [&](auto e) {
            if constexpr (std::is_same<decltype(e), _Float16>::value)
                if (pd == 2) return launch_logits<_Float16, kProb, 2>(g, c.st);
            return launch_logits<decltype(e), kProb, 1>(g, c.st);
        }));
        if (dX) {
            // sums[t][k] (+)= sum_n d[t][n] W[n][k]
            Args s = {};
            s.a = in_steps(ws + p.along, c.T, c.T, rows_p);
            s.b = g.a;
            s.steps = uint32_t(rows_p / vocab::kStepK);
            s.splits = uint32_t(p.splits);
            set_pairs(s, c.xtype == RETRO_F32 ? 2 : 1, narrow ? 1 : sum_parts_of(c.type, c.xtype, dW != nullptr));
            s.out = sums;
            s.ldo = c.K;
            s.split_stride = c.T * c.K;
            s.cols = c.K;
            RETRO_TRY(with_element(c, [&](auto e) {
                return g.n0 ? launch_dx<decltype(e), true>(p.shape, s, c.st)
                            : launch_dx<decltype(e), false>(p.shape, s, c.st);
            }));
        }
        if (dW) {
            Args s = {};
            // dW[n][k] = sum_t d[t][n] x[t][k]
            s.a = in_steps(ws + p.across, rows, rows, Tp);
            s.b = x;
            s.steps = uint32_t(Tp / vocab::kStepK);
            s.splits = 1;
            set_pairs(s, c.type == RETRO_F32 ? 2 : 1, px);
            s.ldo = lddw;
            s.cols = c.K;
            s.out_factor = unscale;
            RETRO_TRY(mx::with_float(c.type, [&](auto* tag) {
                using TW = std::remove_pointer_t<decltype(tag)>;
                s.out = static_cast<TW*>(dW) + g.n0 * lddw;
                if constexpr (std::is_same<TW, __bf16>::value)
                    if (narrow) return launch_dw<__bf16, TW>(s, c.st);
                return launch_dw<_Float16, TW>(s, c.st);
            }));
        }
    }
    return dX ? finish_dx(c, sums, p.splits, 1.f / by, top, dloss, dX, lddx) : RETRO_OK;
}

int64_t head_bytes(int type, int64_t ldw, int64_t K, int64_t N) {
    return N > 0 ? (N - 1) * ldw + host::row_bytes_of(type, K) : 0;
}

int id_bytes(int type) { return type == RETRO_I32 ? 4 : type == RETRO_I64 ? 8 : 0; }

constexpr int64_t kMaxK = int64_t(1) << 22, kMaxT = int64_t(1) << 22;

// Types, sizes and spans that both calls share.
int check_sizes(int type, int64_t ldw, int xtype, int64_t K, int64_t N, int64_t T) {
    host::Geometry geo;
    if (!host::geometry(type, geo) || !is_float(xtype)) return RETRO_E_TYPE;
    if (K < 0 || K >= kMaxK || K % geo.block || !mx::dim_ok(N) || T < 0 || T >= kMaxT) return RETRO_E_SHAPE;
    if (ldw < host::row_bytes_of(type, K) || (N > 1 && ldw > host::kByteLimit / (N - 1) - kMaxK * 4)) return RETRO_E_SHAPE;
    return RETRO_OK;
}

int check_operands(const Call& c, const void* loss, const void* lse, int64_t& x_bytes) {
    const int size = mx::float_bytes(c.xtype);
    x_bytes = mx::span_bytes(c.T, c.K, c.ldx, size);
    if (x_bytes < 0) return RETRO_E_SHAPE;
    if (c.T == 0) return RETRO_OK;
    if (!c.targets || !loss || !lse || (c.K > 0 && (!c.X || (c.N > 0 && !c.W)))) return RETRO_E_NULL;
    if (!mx::aligned(c.W, 16) || !mx::aligned(c.X, size) || !mx::aligned(c.targets, c.wide_targets ? 8 : 4) ||
        !mx::aligned(loss, 4) || !mx::aligned(lse, 4) || c.ldw % vocab::row_alignment(c.type))
        return RETRO_E_ALIGN;
    return RETRO_OK;
}

}  // namespace
}  // namespace ce
}  // namespace retro

using namespace retro;
using namespace retro::ce;

extern "C" {

int64_t retro_cross_entropy_workspace_size(int type, int64_t ldw, int xtype, int64_t K, int64_t N, int64_t T) {
    const int rc = check_sizes(type, ldw, xtype, K, N, T);
    if (rc != RETRO_OK) return rc;
    return T == 0 ? 0 : forward_plan(type, ldw, xtype, K, N, T).bytes;
}

int retro_cross_entropy(int type, const void* W, int64_t ldw, int xtype, const void* X, int64_t ldx, int idtype,
                        const void* targets, float* loss, float* lse, int64_t K, int64_t N, int64_t T, void* workspace,
                        int64_t workspace_bytes, void* stream) {
    RETRO_TRY(check_sizes(type, ldw, xtype, K, N, T));
    if (!id_bytes(idtype)) return RETRO_E_TYPE;
    const Call c{type,    xtype, static_cast<const uint8_t*>(W), ldw, X, ldx, idtype == RETRO_I64,
                 targets, K,     N,                              T,   static_cast<hipStream_t>(stream)};
    int64_t xb = 0;
    RETRO_TRY(check_operands(c, loss, lse, xb));
    if (T == 0) return RETRO_OK;
    const Span w{W, head_bytes(type, ldw, K, N)}, x{X, xb}, y{targets, T * id_bytes(idtype)};
    const Span outs[] = {{loss, 4 * T}, {lse, 4 * T}};
    const int64_t need = forward_plan(type, ldw, xtype, K, N, T).bytes;
    const Span s{workspace, need};
    if (!workspace || workspace_bytes < need || !mx::aligned(workspace, 16)) return RETRO_E_WORKSPACE;
    for (const Span& in : {w, x, y, outs[0], outs[1]})
        if (mx::overlap(s, in)) return RETRO_E_WORKSPACE;
    for (const Span& o : outs)
        for (const Span& in : {w, x, y})
            if (mx::overlap(o, in)) return RETRO_E_ALIAS;
    if (mx::overlap(outs[0], outs[1])) return RETRO_E_ALIAS;
    return forward(c, loss, lse, static_cast<uint8_t*>(workspace));
}

int64_t retro_cross_entropy_backward_workspace_size(int type, int64_t ldw, int xtype, int weight_grad, int64_t K,
                                                    int64_t N, int64_t T) {
    const int rc = check_sizes(type, ldw, xtype, K, N, T);
    if (rc != RETRO_OK) return rc;
    if (weight_grad && !is_float(type)) return RETRO_E_TYPE;
    return T == 0 || N == 0 || K == 0 ? 0 : backward_plan(type, ldw, xtype, weight_grad != 0, true, K, N, T).bytes;
}

int retro_cross_entropy_backward(int type, const void* W, int64_t ldw, int xtype, const void* X, int64_t ldx, int idtype,
                                 const void* targets, const float* lse, const float* dloss, void* dX, int64_t lddx,
                                 void* dW, int64_t lddw, int64_t K, int64_t N, int64_t T, void* workspace,
                                 int64_t workspace_bytes, void* stream) {
    RETRO_TRY(check_sizes(type, ldw, xtype, K, N, T));
    if (!id_bytes(idtype) || (dW && !is_float(type))) return RETRO_E_TYPE;
    const Call c{type,    xtype, static_cast<const uint8_t*>(W), ldw, X, ldx, idtype == RETRO_I64,
                 targets, K,     N,                              T,   static_cast<hipStream_t>(stream)};
    int64_t xb = 0;
    // dX and dW of no tokens: dW is still written
    RETRO_TRY(check_operands(c, dloss, lse, xb));
    const int xs = mx::float_bytes(xtype), ws = std::max(1, mx::float_bytes(type));
    const int64_t dxb = dX ? mx::span_bytes(T, K, lddx, xs) : 0, dwb = dW ? mx::span_bytes(N, K, lddw, ws) : 0;
    if (dxb < 0 || dwb < 0) return RETRO_E_SHAPE;
    if (K == 0 || (T == 0 && (N == 0 || !dW))) return RETRO_OK;
    if (!dX && !dW && T > 0) return RETRO_E_NULL;
    if (!mx::aligned(dX, xs) || !mx::aligned(dW, ws)) return RETRO_E_ALIGN;
    const Span ins[] = {{W, head_bytes(type, ldw, K, N)}, {X, xb}, {targets, T * id_bytes(idtype)}, {lse, 4 * T}, {dloss, 4 * T}};
    const Span outs[] = {{dX, dxb}, {dW, dwb}};
    for (const Span& o : outs)
        for (const Span& in : ins)
            if (mx::overlap(o, in)) return RETRO_E_ALIAS;
    if (mx::overlap(outs[0], outs[1])) return RETRO_E_ALIAS;
    const hipStream_t st = c.st;
    if (T == 0 || N == 0) {  // an empty sum
        const bool of_w = T == 0;
        return mx::with_float(of_w ? type : xtype, [&](auto* tag) {
            using TY = std::remove_pointer_t<decltype(tag)>;
            TY* p = static_cast<TY*>(of_w ? dW : dX);
            if (!p) return int(RETRO_OK);
            const int64_t rows = of_w ? N : T;
            host::clear_last_error();
            zero_rows_kernel<TY><<<dim3(uint32_t(std::min<int64_t>(rows, 65536))), dim3(256), 0, st>>>(
                p, of_w ? lddw : lddx, K, rows);
            return host::launch_status();
        });
    }
    const int64_t need = backward_plan(type, ldw, xtype, dW != nullptr, true, K, N, T).bytes;
    const Span s{workspace, need};
    if (!workspace || workspace_bytes < need || !mx::aligned(workspace, 16)) return RETRO_E_WORKSPACE;
    for (const Span& in : ins)
        if (mx::overlap(s, in)) return RETRO_E_WORKSPACE;
    for (const Span& o : outs)
        if (mx::overlap(s, o)) return RETRO_E_WORKSPACE;
    return backward(c, lse, dloss, dX, lddx, dW, lddw, static_cast<uint8_t*>(workspace));
}

}  // extern "C"
