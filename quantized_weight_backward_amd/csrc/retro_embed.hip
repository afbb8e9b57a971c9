// retro_embed.hip - embedding lookup and its gradient (retro_vocab.h).
#include <algorithm>

#include "retro_vocab_device.h"
#include "retro_vocab_host.h"

namespace retro {
namespace vocab {
namespace {

using host::cdiv;
using mx::Span;

// The gradient. Tokens are sorted by id, stably, so that the tokens of an id lie side
// by side in rising order: a radix sort from the low digit up, of `bits` bits a pass.
// An id that is none sorts last, as N. The sorted list is cut into runs; a wave adds
// up a run's rows, 512 columns of them, and writes the row of each id that lies in the
// run alone. Of an id that goes on in other runs it writes its part, and a second
// launch joins the parts: a frequent id is not one wave's work.
//
// What bounds it is the table being written. All of it is cleared beside the sort, in
// the same launches, so that the sort costs no time of its own and only rows of tokens
// are written after it. 16384 tokens of 4096 BF16 columns into 131072 F32
// rows: 435 us, of which 344 in the launch that clears 2.15 GB and sorts (6.2 TB/s), 88
// in the rows' sums, 6 in joining them.

constexpr int kMaxBits = 9, kMaxDigits = 1 << kMaxBits;
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
// Tokens that one workgroup sorts in LDS. 12000 of 1000 rows take 41 us so and 46 in the
// larger sort's launches; 16384 take 51 and 48 there, and beside a table of 131072 x 4096
// being cleared 435 and 470. The rule is one of tokens alone: small tables give up 3 us.
constexpr int kSmallT = 16384;
constexpr int kBlockItems = 2048;  // of a workgroup of a larger sort's pass
constexpr int kBlockThreads = 256, kBlockWaves = kBlockThreads / 64;
// Tokens of a run. Shorter ones are more waves, which few tokens of few columns need (777
// of 1000 columns into 32000 rows: 59 us in runs of 64, 33 in runs of 16; 16384 of 512:
// 115 and 93), longer ones fewer parts to join; at 16384 tokens of 4096 columns, 2048
// waves in runs of 64, either takes as long.
constexpr int kMaxRun = 64;
int run_for(int64_t K, int64_t T) { return cdiv(T, kMaxRun) * cdiv(K, 512) < 2048 ? 16 : kMaxRun; }

// Passes and bits of each for keys 0 .. N.
struct Radix {
    int passes, bits;
};
Radix radix_of(int64_t N) {
    int bits = 1;
    while ((N >> bits) > 0) ++bits;
    const int passes = int(cdiv(bits, kMaxBits));
    return {passes, int(cdiv(bits, passes))};
}

__device__ __forceinline__ uint32_t key_of(const void* ids, bool wide, int64_t t, int64_t N) {
    const int id = token_at(ids, wide, t, N);
    return id < 0 ? uint32_t(N) : uint32_t(id);
}

// What the wave's lanes wrote to LDS before is what they read after.
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Zeros over rows of `row` bytes `pitch` apart, 16 bytes a step: a workgroup kFill steps
// a thread, side by side, from its own first one on. A row is whole 2s.
constexpr int kFill = 16;
struct Fill {
    uint8_t* p;
    int64_t pitch, row, per, begin, end;  // per: steps of a row
};
template <int THREADS>
__device__ __forceinline__ void fill(const Fill& f, int64_t block) {
    typedef uint32_t words __attribute__((ext_vector_type(4), aligned(2)));
    const int64_t first = f.begin + block * (kFill * THREADS);
    const bool one = f.per >= f.end;  // row
    if (one && first + kFill * THREADS < f.end) {
        words* to = reinterpret_cast<words*>(f.p) + first + threadIdx.x;
#pragma unroll
        for (int j = 0; j < kFill; ++j) to[j * THREADS] = words{0, 0, 0, 0};
        return;
    }
    for (int j = 0; j < kFill; ++j) {
        const int64_t at = first + j * THREADS + threadIdx.x;
        if (at >= f.end) return;
        const int64_t r = one ? 0 : at / f.per, b = (at - r * f.per) * 16;
        uint8_t* to = f.p + r * f.pitch + b;
        if (b + 16 <= f.row) {
            *reinterpret_cast<words*>(to) = words{0, 0, 0, 0};
        } else {
            for (int64_t i = 0; i < f.row - b; i += 2) *reinterpret_cast<uint16_t*>(to + i) = 0;
        }
    }
}

// The lane's place among the lanes of its wave that have its digit (live lanes only),
// and their number. All lanes of the wave are here.
__device__ __forceinline__ uint32_t match(uint32_t digit, int bits, bool live, uint32_t& count) {
    uint64_t same = __ballot(live);
    for (int b = 0; b < bits; ++b) {
        const bool one = (digit >> b) & 1;
        const uint64_t ones = __ballot(one);
        same &= one ? ones : ~ones;
    }
    count = uint32_t(__popcll(same));
    return uint32_t(__popcll(same & ((uint64_t(1) << (threadIdx.x % 64)) - 1)));
}

// Exclusive sums over `n` (at most the workgroup's threads) values, one a thread.
template <int THREADS>
__device__ __forceinline__ uint32_t scan(uint32_t v, uint32_t* waves) {
    uint32_t in = v;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint32_t below = __shfl_up(in, d);
        if (int(threadIdx.x % 64) >= d) in += below;
    }
    if (threadIdx.x % 64 == 63) waves[threadIdx.x / 64] = in;
    __syncthreads();
    uint32_t before = 0;
    for (int w = 0; w < THREADS / 64; ++w) before += w < int(threadIdx.x / 64) ? waves[w] : 0;
    __syncthreads();
    return before + in - v;
}

// Up to kSmallT tokens, PER a thread: all passes in one workgroup, the other workgroups
// fill. Wave w takes items w * per .., 64 at a time, and keeps a count a digit: an item's
// place is its digit's first, the counts of the waves before, its wave's count so far,
// and the lanes before it.
template <int PER>
__global__ __launch_bounds__(kSortThreads) void sort_small_kernel(const void* __restrict__ ids, bool wide, int64_t N,
                                                                 int T, int passes, int bits, uint32_t* __restrict__ keys,
                                                                 uint32_t* __restrict__ order, Fill f) {
    if (blockIdx.x > 0) {
        fill<kSortThreads>(f, blockIdx.x - 1);
        return;
    }
    __shared__ uint32_t key[PER * kSortThreads];
    __shared__ uint16_t from[PER * kSortThreads];
    __shared__ uint16_t count[kSortWaves][kMaxDigits];
    __shared__ uint32_t waves[kSortWaves];
    const int wave = threadIdx.x / 64, lane = threadIdx.x % 64, rounds = (T + kSortThreads - 1) / kSortThreads;
    uint32_t k[PER], at[PER], place[PER];
    auto item = [&](int i) { return (wave * rounds + i) * 64 + lane; };
    for (int i = 0; i < PER; ++i) {
        const bool live = i < rounds && item(i) < T;
        k[i] = live ? key_of(ids, wide, item(i), N) : 0;
        at[i] = uint32_t(item(i));
    }
    for (int p = 0; p < passes; ++p) {
        for (int d = threadIdx.x; d < kSortWaves * kMaxDigits; d += kSortThreads) (&count[0][0])[d] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (i >= rounds) break;
            const bool live = item(i) < T;
            const uint32_t digit = (k[i] >> (p * bits)) & ((1u << bits) - 1);
            uint32_t same;
            const uint32_t mine = match(digit, bits, live, same);
            const uint32_t before = count[wave][digit];
            place[i] = before + mine;
            wave_fence();
            if (live && mine == 0) count[wave][digit] = uint16_t(before + same);
            wave_fence();
        }
        __syncthreads();
        // counts become the places of each wave's first item of a digit
        uint32_t all = 0;
        if (threadIdx.x < kMaxDigits)
            for (int w = 0; w < kSortWaves; ++w) all += count[w][threadIdx.x];
        uint32_t first = scan<kSortThreads>(all, waves);
        if (threadIdx.x < kMaxDigits)
            for (int w = 0; w < kSortWaves; ++w) {
                const uint32_t n = count[w][threadIdx.x];
                count[w][threadIdx.x] = uint16_t(first);
                first += n;
            }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (i >= rounds || item(i) >= T) break;
            const uint32_t to = count[wave][(k[i] >> (p * bits)) & ((1u << bits) - 1)] + place[i];
            key[to] = k[i];
            from[to] = uint16_t(at[i]);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (i >= rounds || item(i) >= T) break;
            k[i] = key[item(i)];
            at[i] = from[item(i)];
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (i >= rounds || item(i) >= T) break;
        keys[item(i)] = k[i];
        order[item(i)] = at[i];
    }
}

// A pass of a larger sort: a workgroup kBlockItems items, a wave a quarter of them in
// rows of 64; the workgroups past `blocks` fill. With `totals` NULL the digits of each workgroup are counted, into
// counts[digit][workgroup]; then counts holds the items of the digit in workgroups
// before, totals the digits' numbers, and the items are moved.
__global__ __launch_bounds__(kBlockThreads) void sort_pass_kernel(
    const void* __restrict__ ids, bool wide, int64_t N, const uint32_t* __restrict__ keys_in,
    const uint32_t* __restrict__ order_in, int64_t T, int shift, int bits, uint32_t blocks,
    uint32_t* __restrict__ counts, const uint32_t* __restrict__ totals, uint32_t* __restrict__ keys,
    uint32_t* __restrict__ order, Fill f) {
    if (blockIdx.x >= blocks) {
        fill<kBlockThreads>(f, blockIdx.x - blocks);
        return;
    }
    constexpr int kRounds = kBlockItems / kBlockThreads;
    __shared__ uint32_t count[kBlockWaves][kMaxDigits];
    __shared__ uint32_t waves[kBlockWaves];
    const int wave = threadIdx.x / 64, lane = threadIdx.x % 64, digits = 1 << bits;
    const int64_t first = int64_t(blockIdx.x) * kBlockItems + wave * (kBlockItems / kBlockWaves) + lane;
    for (int d = threadIdx.x; d < kBlockWaves * kMaxDigits; d += kBlockThreads) (&count[0][0])[d] = 0;
    __syncthreads();
    uint32_t k[kRounds], place[kRounds];
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
        const int64_t t = first + i * 64;
        const bool live = t < T;
        k[i] = !live ? 0 : keys_in ? keys_in[t] : key_of(ids, wide, t, N);
        const uint32_t digit = (k[i] >> shift) & (digits - 1);
        uint32_t same;
        const uint32_t mine = match(digit, bits, live, same);
        const uint32_t before = count[wave][digit];
        place[i] = before + mine;
        wave_fence();
        if (live && mine == 0) count[wave][digit] = before + same;
        wave_fence();
    }
    __syncthreads();
    if (!totals) {
        for (int d = threadIdx.x; d < digits; d += kBlockThreads) {
            uint32_t all = 0;
            for (int w = 0; w < kBlockWaves; ++w) all += count[w][d];
            counts[int64_t(d) * blocks + blockIdx.x] = all;
        }
        return;
    }
    uint32_t before = 0;  // of the digits below
    for (int d0 = 0; d0 < digits; d0 += kBlockThreads) {
        const int d = d0 + threadIdx.x;
        const uint32_t n = d < digits ? totals[d] : 0, below = scan<kBlockThreads>(n, waves);
        if (d < digits) {
            uint32_t to = before + below + counts[int64_t(d) * blocks + blockIdx.x];
            for (int w = 0; w < kBlockWaves; ++w) {
                const uint32_t of = count[w][d];
                count[w][d] = to;
                to += of;
            }
        }
        __shared__ uint32_t last;
        if (threadIdx.x == kBlockThreads - 1) last = below + n;
        __syncthreads();
        before += last;
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
        const int64_t t = first + i * 64;
        if (t >= T) break;
        const uint32_t to = count[wave][(k[i] >> shift) & (digits - 1)] + place[i];
        keys[to] = k[i];
        order[to] = order_in ? order_in[t] : uint32_t(t);
    }
}

// counts of one digit (a workgroup each): those of the workgroups before, and their sum.
__global__ __launch_bounds__(256) void sort_scan_kernel(uint32_t* __restrict__ counts, uint32_t blocks,
                                                        uint32_t* __restrict__ totals) {
    __shared__ uint32_t waves[4], last;
    uint32_t* c = counts + int64_t(blockIdx.x) * blocks;
    uint32_t before = 0;
    for (uint32_t b0 = 0; b0 < blocks; b0 += 256) {
        const uint32_t b = b0 + threadIdx.x, n = b < blocks ? c[b] : 0, below = scan<256>(n, waves);
        if (b < blocks) c[b] = before + below;
        if (threadIdx.x == 255) last = below + n;
        __syncthreads();
        before += last;
        __syncthreads();
    }
    if (threadIdx.x == 0) totals[blockIdx.x] = before;
}

// A wave's view of the sorted list from one place on: its lanes hold the next 64 keys
// and tokens, in one round of loads.
struct Window {
    uint32_t key, token;
};
__device__ __forceinline__ Window window_at(const uint32_t* __restrict__ keys, const uint32_t* __restrict__ order,
                                            uint32_t from, uint32_t T) {
    const uint32_t i = from + threadIdx.x % 64;
    return i < T ? Window{keys[i], order[i]} : Window{~0u, 0};
}

// The first place in [low, high) whose key is `key` or above, 64 probes a round.
__device__ __forceinline__ uint32_t first_of(const uint32_t* __restrict__ keys, uint32_t low, uint32_t high, uint32_t key) {
    while (high - low > 0) {
        const uint32_t step = (high - low + 63) / 64, i = low + threadIdx.x % 64 * step;
        const uint64_t below = __ballot(i < high && keys[i] < key);  // some first lanes
        if (!below) return low;
        const uint32_t n = uint32_t(__popcll(below));
        high = min(high, low + n * step);
        low += (n - 1) * step + 1;
    }
    return low;
}

// A wave's row or run, uniform, and its 512 columns: waves are dealt `chunks` to a row.
// Lanes past the columns stay, with nothing to load or store: the tokens that they hold
// are read by the others.
struct Place {
    int64_t row, k;
};
__device__ __forceinline__ Place place_of(int64_t first_block, uint32_t chunks) {
    const int64_t at = (first_block + blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int64_t row = at >> 32 ? at / chunks : int64_t(uint32_t(at) / chunks);
    return {row, (at - row * chunks) * 512 + threadIdx.x % 64 * 8};
}

template <typename TW, bool ADD>
__device__ __forceinline__ void write_row(TW* to, int64_t left, float scale, const float sum[8]) {
    float e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = sum[i] * scale;
    if constexpr (ADD) {
        float old[8];
        mx::load8(to, left, old);
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] += old[i];
    }
    store8(to, left, e);
}

// The sums of run c. Of an id that lies in other runs too, the part that begins with
// the run goes to slot 2c, one that begins inside it to slot 2c + 1.
template <typename TY, typename TW, bool ADD>
__global__ __launch_bounds__(256) void runs_kernel(const TY* __restrict__ dY, int64_t ldy, float scale,
                                                   TW* __restrict__ dW, int64_t ldw, int64_t K, uint32_t T, int64_t N,
                                                   uint32_t run, const uint32_t* __restrict__ keys,
                                                   const uint32_t* __restrict__ order, float* __restrict__ parts,
                                                   int64_t pitch, uint32_t chunks, int64_t first_block) {
    const Place at = place_of(first_block, chunks);
    if (at.row * run >= T) return;
    const uint32_t begin = uint32_t(at.row) * run, n = min(T - begin, run);
    const Window w = window_at(keys, order, begin, T);
    const uint32_t none = ~0u, head = uint32_t(__builtin_amdgcn_readfirstlane(int(w.key)));
    const uint32_t tail = uint32_t(__builtin_amdgcn_readlane(int(w.key), n - 1));
    const uint32_t before = begin > 0 && keys[begin - 1] == head ? head : none;      // an id that began in a run before
    const uint32_t after = begin + n < T && keys[begin + n] == tail ? tail : none;   // one that goes on
    const TY* from = dY + at.k;
    const int64_t left = K - at.k;
    auto key_at = [&](uint32_t i) { return uint32_t(__builtin_amdgcn_readlane(int(w.key), i)); };
    float e[8] = {};
    uint32_t first = 0;
    for (uint32_t i0 = 0; i0 < n; i0 += 8) {
        // eight rows in flight; past the run the last one again, not added
        float v[8][8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            mx::load8(from + int64_t(uint32_t(__builtin_amdgcn_readlane(int(w.token), min(i0 + j, n - 1)))) * ldy, left, v[j]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t i = i0 + j;
            if (i >= n) break;
            const uint32_t key = key_at(i);
            if (key >= N) return;  // the tokens of no id are the last
#pragma unroll
            for (int c = 0; c < 8; ++c) e[c] += v[j][c];
            if (i + 1 < n && key_at(i + 1) == key) continue;
            if ((key == before && first == 0) || key == after)
                store8(parts + (2 * at.row + (first ? 1 : 0)) * pitch + at.k, pitch - at.k, e);
            else
                write_row<TW, ADD>(dW + key * ldw + at.k, left, scale, e);
            first = i + 1;
#pragma unroll
            for (int c = 0; c < 8; ++c) e[c] = 0.f;
        }
    }
}

// The rows of ids that lie in several runs, by the run in which they begin.
template <typename TW, bool ADD>
__global__ __launch_bounds__(256) void join_kernel(float scale, TW* __restrict__ dW, int64_t ldw, int64_t K, uint32_t T,
                                                   int64_t N, uint32_t run, const uint32_t* __restrict__ keys,
                                                   const float* __restrict__ parts, int64_t pitch, uint32_t chunks,
                                                   int64_t first_block) {
    const Place at = place_of(first_block, chunks);
    if ((at.row + 1) * run >= T) return;  // nothing goes on after the last run
    const uint32_t begin = uint32_t(at.row) * run, next = begin + run, key = keys[next - 1];
    if (key >= N || keys[next] != key) return;
    const bool inside = keys[begin] != key;  // it begins inside this run
    if (!inside && begin > 0 && keys[begin - 1] == key) return;
    const uint32_t last = (first_of(keys, next, T, key + 1) - 1) / run - uint32_t(at.row);
    const float* from = parts + 2 * at.row * pitch + at.k;
    float e[8];
    mx::load8(from + (inside ? pitch : 0), pitch - at.k, e);
    for (uint32_t c = 1; c <= last; c += 8) {
        float v[8][8];
#pragma unroll
        for (int j = 0; j < 8; ++j) mx::load8(from + 2 * int64_t(min(c + j, last)) * pitch, pitch - at.k, v[j]);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c + j <= last)
#pragma unroll
                for (int i = 0; i < 8; ++i) e[i] += v[j][i];
    }
    write_row<TW, ADD>(dW + key * ldw + at.k, K - at.k, scale, e);
}

struct Plan {
    Radix radix;
    int64_t keys[2], order[2], counts, totals, parts, bytes;
    int64_t blocks, run;
};

Plan plan_of(int64_t K, int64_t N, int64_t T) {
    Plan p = {};
    p.radix = radix_of(N);
    p.blocks = cdiv(T, kBlockItems);
    auto take = [&](int64_t bytes) {
        const int64_t here = p.bytes;
        p.bytes += cdiv(bytes, 256) * 256;
        return here;
    };
    for (int i = 0; i < (T > kSmallT ? 2 : 1); ++i) {
        p.keys[i] = take(4 * T);
        p.order[i] = take(4 * T);
    }
    if (T > kSmallT) {
        p.counts = take(4 * p.blocks << p.radix.bits);
        p.totals = take(4 << p.radix.bits);
    }
    p.run = run_for(K, T);
    p.parts = take(4 * 2 * cdiv(T, p.run) * cdiv(K, 8) * 8);
    return p;
}

#define RETRO_TRY(e)                     \
    do {                                 \
        const int rc_ = (e);             \
        if (rc_ != RETRO_OK) return rc_; \
    } while (0)

// Sorted keys and tokens end in plane `out` of the workspace; `f`, where it has
// steps, is filled in shares beside the sort's launches.
int sort(const Plan& p, const void* ids, bool wide, int64_t N, int64_t T, uint8_t* ws, int& out, Fill f, hipStream_t st) {
    auto words = [&](int64_t at) { return reinterpret_cast<uint32_t*>(ws + at); };
    auto fillers = [](const Fill& f, int threads) { return cdiv(f.end - f.begin, kFill * threads); };
    out = 0;
    host::clear_last_error();
    if (T <= kSmallT) {
        // a thread that can hold 16 items takes 4 us longer over 8
        auto kernel = T <= 8 * kSortThreads ? sort_small_kernel<8> : sort_small_kernel<16>;
        kernel<<<dim3(uint32_t(1 + fillers(f, kSortThreads))), dim3(kSortThreads), 0, st>>>(
            ids, wide, N, int(T), p.radix.passes, p.radix.bits, words(p.keys[0]), words(p.order[0]), f);
        return host::launch_status();
    }
    const uint32_t blocks = uint32_t(p.blocks);
    const int64_t steps = f.end, shares = 2 * p.radix.passes;
    for (int i = 0; i < p.radix.passes; ++i) {
        const uint32_t *keys_in = i ? words(p.keys[out]) : nullptr, *order_in = i ? words(p.order[out]) : nullptr;
        const int to = i ? 1 - out : 0, shift = i * p.radix.bits;
        uint32_t *counts = words(p.counts), *totals = words(p.totals);
        auto pass = [&](int share, const uint32_t* of, uint32_t* keys, uint32_t* order) {
            f.begin = steps * share / shares;
            f.end = steps * (share + 1) / shares;
            sort_pass_kernel<<<dim3(uint32_t(blocks + fillers(f, kBlockThreads))), dim3(kBlockThreads), 0, st>>>(
                ids, wide, N, keys_in, order_in, T, shift, p.radix.bits, blocks, counts, of, keys, order, f);
        };
        pass(2 * i, nullptr, nullptr, nullptr);
        sort_scan_kernel<<<dim3(1u << p.radix.bits), dim3(256), 0, st>>>(counts, blocks, totals);
        pass(2 * i + 1, totals, words(p.keys[to]), words(p.order[to]));
        out = to;
    }
    return host::launch_status();
}

constexpr int64_t kMaxK = int64_t(1) << 22, kMaxT = int64_t(1) << 28;

int id_bytes(int type) { return type == RETRO_I32 ? 4 : type == RETRO_I64 ? 8 : 0; }

}  // namespace
}  // namespace vocab
}  // namespace retro

using namespace retro;
using namespace retro::vocab;

extern "C" {

int retro_embedding(int type, const void* W, int64_t ldw, int idtype, const void* ids, float scale, int ytype, void* Y,
                    int64_t ldy, int64_t K, int64_t N, int64_t T, void* stream) {
    host::Geometry geo;
    const int size = mx::float_bytes(ytype), idsize = id_bytes(idtype);
    if (!host::geometry(type, geo) || !size || !idsize) return RETRO_E_TYPE;
    if (K < 0 || K >= kMaxK || K % geo.block || !mx::dim_ok(N) || !mx::dim_ok(T)) return RETRO_E_SHAPE;
    const int64_t row = host::row_bytes_of(type, K), yb = mx::span_bytes(T, K, ldy, size);
    if (yb < 0 || ldw < row || (N > 1 && ldw > (host::kByteLimit - row) / (N - 1))) return RETRO_E_SHAPE;
    if (T == 0 || K == 0) return RETRO_OK;
    if (!ids || !Y || (N > 0 && !W)) return RETRO_E_NULL;
    if (!mx::aligned(W, 16) || !mx::aligned(Y, size) || !mx::aligned(ids, idsize) || ldw % row_alignment(type))
        return RETRO_E_ALIGN;
    const Span y{Y, yb};
    if (mx::overlap(y, {W, N > 0 ? (N - 1) * ldw + row : 0}) || mx::overlap(y, {ids, T * idsize})) return RETRO_E_ALIAS;
    const EmbedArgs a{static_cast<const uint8_t*>(W), ldw, ids, idtype == RETRO_I64, Y, ldy, scale, K, N, T};
    return with_type(type, [&](auto t) { return launch_embed<decltype(t)::value>(ytype, a, static_cast<hipStream_t>(stream)); });
}

int64_t retro_embedding_backward_workspace_size(int64_t K, int64_t N, int64_t T) {
    if (K < 0 || K >= kMaxK || !mx::dim_ok(N) || T < 0 || T >= kMaxT) return RETRO_E_SHAPE;
    return K == 0 || N == 0 ? 0 : plan_of(K, N, T).bytes;
}

int retro_embedding_backward(int idtype, const void* ids, int ytype, const void* dY, int64_t ldy, float scale, int wtype,
                             void* dW, int64_t ldw, int accumulate, int64_t K, int64_t N, int64_t T, void* workspace,
                             int64_t workspace_bytes, void* stream) {
    const int ys = mx::float_bytes(ytype), wsize = mx::float_bytes(wtype), idsize = id_bytes(idtype);
    if (!ys || !wsize || !idsize) return RETRO_E_TYPE;
    const int64_t need = retro_embedding_backward_workspace_size(K, N, T);
    if (need < 0) return int(need);
    const int64_t yb = mx::span_bytes(T, K, ldy, ys), wb = mx::span_bytes(N, K, ldw, wsize);
    if (yb < 0 || wb < 0) return RETRO_E_SHAPE;
    if (N == 0 || K == 0 || (T == 0 && accumulate)) return RETRO_OK;
    if (!dW || (T > 0 && (!ids || !dY))) return RETRO_E_NULL;
    if (!mx::aligned(dW, wsize) || !mx::aligned(dY, ys) || !mx::aligned(ids, idsize)) return RETRO_E_ALIGN;
    const Span w{dW, wb}, y{dY, yb}, i{ids, T * idsize}, s{workspace, need};
    if (mx::overlap(w, y) || mx::overlap(w, i)) return RETRO_E_ALIAS;
    if (need && (!workspace || workspace_bytes < need || !mx::aligned(workspace, 16) || mx::overlap(s, w) ||
                 mx::overlap(s, y) || mx::overlap(s, i)))
        return RETRO_E_WORKSPACE;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const Plan p = plan_of(K, N, T);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    float* parts = reinterpret_cast<float*>(ws + p.parts);
    int out = 0;
    Fill f = {};
    if (!accumulate) {
        f.p = static_cast<uint8_t*>(dW);
        f.pitch = ldw * wsize;
        f.row = K * wsize;
        int64_t rows = N;
        if (f.pitch == f.row) {  // one long row
            f.row *= N;
            rows = 1;
        }
        f.per = cdiv(f.row, 16);
        f.end = rows * f.per;
    }
    RETRO_TRY(sort(p, ids, idtype == RETRO_I64, N, T, ws, out, f, st));
    if (T == 0) return RETRO_OK;
    const uint32_t *keys = reinterpret_cast<uint32_t*>(ws + p.keys[out]),
                   *order = reinterpret_cast<uint32_t*>(ws + p.order[out]);
    const uint32_t chunks = uint32_t(cdiv(K, 512));
    const int64_t pitch = cdiv(K, 8) * 8;
    return mx::with_float(ytype, [&](auto* ytag) {
        using TY = std::remove_pointer_t<decltype(ytag)>;
        const TY* dy = static_cast<const TY*>(dY);
        return mx::with_float(wtype, [&](auto* wtag) {
            using TW = std::remove_pointer_t<decltype(wtag)>;
            TW* w = static_cast<TW*>(dW);
            const int64_t waves = cdiv(T, p.run) * chunks;
            const uint32_t run = uint32_t(p.run), t = uint32_t(T);
            RETRO_TRY(mx::in_block_ranges(cdiv(waves, 4), [&](int64_t first, uint32_t blocks) {
                auto kernel = accumulate ? runs_kernel<TY, TW, true> : runs_kernel<TY, TW, false>;
                kernel<<<dim3(blocks), dim3(256), 0, st>>>(dy, ldy, scale, w, ldw, K, t, N, run, keys, order, parts, pitch,
                                                           chunks, first);
            }));
            if (T <= p.run) return int(RETRO_OK);  // one run
            return mx::in_block_ranges(cdiv(waves, 4), [&](int64_t first, uint32_t blocks) {
                auto kernel = accumulate ? join_kernel<TW, true> : join_kernel<TW, false>;
                kernel<<<dim3(blocks), dim3(256), 0, st>>>(scale, w, ldw, K, t, N, run, keys, parts, pitch, chunks, first);
            });
        });
    });
}

}  // extern "C"
