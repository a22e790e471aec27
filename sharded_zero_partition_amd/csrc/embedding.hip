// embedding.hip -- rows of a table by tokens, and the table's gradient (gfx950).
//
// Both are bound by HBM: a lookup reads and writes each row once (8192 rows of 5120 bf16:
// 168 MB in 25 us), a gradient reads dy once and writes the table once.
//
// The gradient adds up rows of dy that have the same token.  Atomic adds would
// take an order of their own each time; here the tokens are sorted (stable, so a
// row's summands come as the tokens do), the sorted list is cut into tiles of
// equal length, and one wave sums a tile's rows of dy for 512 columns.  Tokens
// are as uneven as text is (the most frequent one has several per cent), and
// equal tiles make the waves' work equal.  A run of equal tokens inside a tile
// is a finished row; one that crosses tiles leaves a partial sum for each, which
// a last kernel adds in order.  Rows that no token names are zeros from the start.
// dy and finished rows pass by the caches (8192 tokens, 50257 x 5120 bf16, from HBM: 132 us
// instead of 138; as fast where dy was just written).
//   8192 tokens, 50257 x 5120 bf16: sorting under the fill 89 to 99 us, sums 22 to 27, joining 6
//   32768 tokens, 1600 fp16 columns added to fp32: sorting 25 us, sums 39, joining 11
#include <type_traits>

#include "octets.hpp"
#include "timed_launch.hpp"

#pragma clang fp contract(off)

namespace zp {
namespace {

constexpr int kThreads = 256;

// ---------------------------------------------------------------------------
// lookup
// ---------------------------------------------------------------------------

// Row of the table that token i names, or -1.
template <typename I>
__device__ __forceinline__ int64_t named_row(const void* tokens, int64_t i, int64_t first, int64_t rows) {
    const int64_t t = ((Global<const I>*)tokens)[i];
    const uint64_t r = uint64_t(t) - uint64_t(first);   // right for every t that is not below
    return t >= first && r < uint64_t(rows) ? int64_t(r) : -1;
}

struct LookupArgs {
    EmbedLaunch e;
    Divisor per_row;   // octets of a row
    int64_t octets;
};

template <int DI, int DO, typename I>
__global__ __launch_bounds__(kThreads) void lookup_kernel(const LookupArgs a) {
    const int64_t base = int64_t(blockIdx.x) * (kThreads * kRowOctets);
    int64_t row;
    uint32_t rest;
    divide(base, a.per_row, &row, &rest);
    int64_t i[kRowOctets], col[kRowOctets], left[kRowOctets], r[kRowOctets];
#pragma unroll
    for (int u = 0; u < kRowOctets; ++u) {
        const uint32_t k = threadIdx.x + u * kThreads;
        const uint32_t q = divide(rest + k, a.per_row);
        i[u] = row + q;
        col[u] = int64_t(rest + k - q * a.per_row.g) * kOctet;
        left[u] = base + k < a.octets ? a.e.cols - col[u] : 0;
        r[u] = left[u] > 0 ? named_row<I>(a.e.tokens, i[u], a.e.first, a.e.rows) : -1;
    }
    Octet<DI> x[kRowOctets];
#pragma unroll
    for (int u = 0; u < kRowOctets; ++u)
        x[u] = load_octet<DI>(place<DI>(a.e.in, r[u], a.e.s_in, col[u]), r[u] < 0 ? 0 : left[u]);
#pragma unroll
    for (int u = 0; u < kRowOctets; ++u) {
        Octet<DO> y;
#pragma unroll
        for (int k = 0; k < kOctet; ++k) y.set(k, r[u] < 0 ? 0.0f : x[u].get(k) * a.e.scale);
        store_octet<DO, true>(place<DO>(a.e.out, i[u], a.e.s_out, col[u]), left[u], y);
    }
}

// ---------------------------------------------------------------------------
// sorting: (row, place) pairs, rows ascending, places ascending in a row; tokens
// that name no row count as row `rows` and come last
// ---------------------------------------------------------------------------

// Zeros into the whole table, by the blocks of the first sorting launch that come after
// the sorting ones: sorting waits for memory, a fill is nothing but memory, which it writes
// at 6 TB/s.  (The gradient of 8192 tokens of 50257 x 5120 bf16 takes 125 us; 142 where the
// launch that sums filled only the rows that no token names.)
constexpr int kFillRows = 16;   // of a block
struct Fill {
    char* out;
    int64_t pitch, rows, cols;   // bytes; cols in 16-bit units, whatever the type; rows: 0 if nothing is filled
    Divisor per_row;             // 16-byte pieces of a row
    int32_t before;              // blocks of the launch that sort
    int64_t blocks() const { return (rows + kFillRows - 1) / kFillRows; }
};
template <int kBlock>
__device__ __forceinline__ void fill(const Fill& f) {
    const int64_t r0 = (int64_t(blockIdx.x) - f.before) * kFillRows;
    const int64_t r1 = r0 + kFillRows < f.rows ? r0 + kFillRows : f.rows;
    Octet<ZERO_DTYPE_FP16> zero;
    zero.zero();
    if (f.per_row.g < kBlock) {   // short rows: all of them at once
        const uint32_t all = uint32_t(r1 - r0) * f.per_row.g;
        for (uint32_t x = threadIdx.x; x < all; x += kBlock) {
            const uint32_t r = divide(x, f.per_row);
            const int64_t c = int64_t(x - r * f.per_row.g) * kOctet;
            store_octet<ZERO_DTYPE_FP16, true>(f.out + (r0 + r) * f.pitch + 2 * c, f.cols - c, zero);
        }
        return;
    }
    for (int64_t r = r0; r < r1; ++r)
        for (int64_t c = int64_t(threadIdx.x) * kOctet; c < f.cols; c += kBlock * kOctet)
            store_octet<ZERO_DTYPE_FP16, true>(f.out + r * f.pitch + 2 * c, f.cols - c, zero);
}

struct SortArgs {
    const void* tokens;
    int64_t n, first, rows;
    uint32_t* key;      // sorted rows
    uint32_t* order;    // and their places
    Fill fill;          // of the first launch
};

template <typename I>
__device__ __forceinline__ uint32_t key_of(const SortArgs& a, int64_t i) {
    const int64_t r = named_row<I>(a.tokens, i, a.first, a.rows);
    return r < 0 ? uint32_t(a.rows) : uint32_t(r);
}

// Few tokens: each one's place is how many keys are smaller, or equal and before
// it.  16 threads count for a token, 32 tokens a block: n^2 comparisons, but one
// launch where digit by digit takes four that wait for each other.  The whole gradient by
// ranks / by digits, us:
//   50257 x 64 added to fp32      2048 tokens 18.6 / 34.8, 8192 27.4 / 36.8, 12288 37.3 / 38.9, 16384 47.6 / 42.2
//   50257 x 1600 added to fp32    2048 20.4 / 37.0, 8192 37.4 / 45.7, 12288 56.8 / 54.2, 16384 74.1 / 63.9
//   50257 x 5120 bf16, written    2048 113 / 132, 8192 132 / 152, 12288 144 / 164, 16384 173 / 174
// They cross between 8192 and 16384.
constexpr int64_t kRankMost = 8192;
constexpr int kRankThreads = 512, kRankShare = 16, kRankTokens = kRankThreads / kRankShare;
template <typename I>
__global__ __launch_bounds__(kRankThreads) void rank_kernel(const SortArgs a) {
    __shared__ u32x4 keys[kRankMost / 4];
    if (int(blockIdx.x) >= a.fill.before) return fill<kRankThreads>(a.fill);
    const int n = int(a.n), tid = int(threadIdx.x), fours = (n + 3) / 4;
    uint32_t* flat = reinterpret_cast<uint32_t*>(keys);
    constexpr int ahead = 8;
    for (int j0 = tid; j0 < 4 * fours; j0 += ahead * kRankThreads) {
        uint32_t k[ahead];
#pragma unroll
        for (int u = 0; u < ahead; ++u) k[u] = j0 + u * kRankThreads < n ? key_of<I>(a, j0 + u * kRankThreads) : 0xFFFFFFFFu;   // above all keys
#pragma unroll
        for (int u = 0; u < ahead; ++u)
            if (j0 + u * kRankThreads < 4 * fours) flat[j0 + u * kRankThreads] = k[u];
    }
    __syncthreads();
    const int first = int(blockIdx.x) * kRankTokens, i = first + tid / kRankShare, part = tid % kRankShare;
    const uint32_t mine = i < n ? flat[i] : 0;
    int rank = 0;
    // fours before the block's tokens (first is one's start), its own, and those after
    const int lo = first / 4, hi = min(lo + kRankTokens / 4, fours);
    const auto count = [&](int j, auto f) {
        const u32x4 k = keys[j];
#pragma unroll
        for (int q = 0; q < 4; ++q) rank += f(k[q], 4 * j + q) ? 1 : 0;
    };
#pragma unroll 4
    for (int j = part; j < lo; j += kRankShare) count(j, [&](uint32_t k, int) { return k <= mine; });
    for (int j = lo + part; j < hi; j += kRankShare) count(j, [&](uint32_t k, int at) { return k < mine || (k == mine && at < i); });
#pragma unroll 4
    for (int j = hi + part; j < fours; j += kRankShare) count(j, [&](uint32_t k, int) { return k < mine; });
#pragma unroll
    for (int h = 1; h < kRankShare; h *= 2) rank += __shfl_xor(rank, h);
    if (part == 0 && i < n) {
        a.key[rank] = mine;
        a.order[rank] = uint32_t(i);
    }
}

// Many: digits of at most 9 bits, lowest first.  A block counts the digits of its
// part of the list; then each block, knowing all counts, puts its elements where
// the lower digits, the earlier blocks, its earlier waves and its wave's earlier
// elements leave off.
constexpr int kDigitBits = 9;
constexpr int kMaxDigits = 1 << kDigitBits;
constexpr int kSortWaves = kThreads / 64;
constexpr int64_t kMaxSortBlocks = 256;
struct DigitArgs {
    SortArgs s;
    const uint32_t* in_key;     // not in the first pass, which takes the tokens
    const uint32_t* in_order;
    uint32_t* count;            // blocks x digits
    int64_t part;               // elements of a block, a multiple of 4 kThreads
    int32_t blocks, shift, digits;   // digits: a power of two
};

// Four elements of a lane, 64 apart; those from hi on are no elements.  One branch-free
// batch of loads.
constexpr int kSortAhead = 4;
template <typename I, bool kFirst>
__device__ __forceinline__ void digit_load(const DigitArgs& a, int64_t i0, int64_t hi, uint32_t k[kSortAhead]) {
#pragma unroll
    for (int u = 0; u < kSortAhead; ++u) {
        const int64_t i = i0 + 64 * u < hi ? i0 + 64 * u : hi - 1;   // hi > i0 of the wave's first lane
        if constexpr (kFirst) k[u] = key_of<I>(a.s, i);
        else k[u] = ((Global<const uint32_t>*)a.in_key)[i];
    }
}

template <typename I, bool kFirst>
__global__ __launch_bounds__(kThreads) void digit_count_kernel(const DigitArgs a) {
    __shared__ uint32_t count[kMaxDigits];
    if (kFirst && int(blockIdx.x) >= a.s.fill.before) return fill<kThreads>(a.s.fill);
    for (int d = threadIdx.x; d < a.digits; d += kThreads) count[d] = 0;
    __syncthreads();
    const int wave = int(threadIdx.x) >> 6, lane = int(threadIdx.x) & 63;
    const int64_t quarter = a.part / kSortWaves, lo = int64_t(blockIdx.x) * a.part + wave * quarter;
    const int64_t hi = lo + quarter < a.s.n ? lo + quarter : a.s.n;
    for (int64_t i0 = lo; i0 < hi; i0 += 64 * kSortAhead) {
        uint32_t k[kSortAhead];
        digit_load<I, kFirst>(a, i0 + lane, hi, k);
#pragma unroll
        for (int u = 0; u < kSortAhead; ++u)
            if (i0 + 64 * u + lane < hi) atomicAdd(&count[(k[u] >> a.shift) & (a.digits - 1)], 1u);
    }
    __syncthreads();
    for (int d = threadIdx.x; d < a.digits; d += kThreads) a.count[int64_t(blockIdx.x) * a.digits + d] = count[d];
}

template <typename I, bool kFirst>
__global__ __launch_bounds__(kThreads) void digit_move_kernel(const DigitArgs a) {
    __shared__ uint32_t next[kSortWaves][kMaxDigits];   // where a wave's next element with the digit goes
    __shared__ uint32_t total[kMaxDigits];
    const int tid = int(threadIdx.x), wave = tid >> 6, lane = tid & 63;
    const int64_t quarter = a.part / kSortWaves;
    const int64_t lo = int64_t(blockIdx.x) * a.part + wave * quarter;
    const int64_t hi = lo + quarter < a.s.n ? lo + quarter : a.s.n;
    for (int d = tid; d < a.digits; d += kThreads)
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) next[w][d] = 0;
    __syncthreads();
    // each wave's counts, for the waves after it
    for (int64_t i0 = lo; i0 < hi; i0 += 64 * kSortAhead) {
        uint32_t k[kSortAhead];
        digit_load<I, kFirst>(a, i0 + lane, hi, k);
#pragma unroll
        for (int u = 0; u < kSortAhead; ++u)
            if (i0 + 64 * u + lane < hi)
                for (int w = wave + 1; w < kSortWaves; ++w) atomicAdd(&next[w][(k[u] >> a.shift) & (a.digits - 1)], 1u);
    }
    // the earlier blocks' counts, and all blocks'
    for (int d = tid; d < a.digits; d += kThreads) {
        uint32_t before = 0, all = 0;
        constexpr int ahead = 16;   // loads at once
        for (int b0 = 0; b0 < a.blocks; b0 += ahead) {
            uint32_t c[ahead];
#pragma unroll
            for (int j = 0; j < ahead; ++j) c[j] = a.count[int64_t(min(b0 + j, a.blocks - 1)) * a.digits + d];
#pragma unroll
            for (int j = 0; j < ahead; ++j) {
                before += b0 + j < int(blockIdx.x) ? c[j] : 0;
                all += b0 + j < a.blocks ? c[j] : 0;
            }
        }
        total[d] = all;
        next[0][d] = before;   // nothing is counted there
    }
    __syncthreads();
    // sums of the lower digits, by one wave: 64 digits at a time
    if (wave == 0) {
        uint32_t below = 0;
        for (int d0 = 0; d0 < a.digits; d0 += 64) {
            const int d = d0 + lane;
            const uint32_t own = d < a.digits ? total[d] : 0;
            uint32_t x = own;
#pragma unroll
            for (int h = 1; h < 64; h *= 2) {
                const uint32_t y = __shfl_up(x, h);
                if (lane >= h) x += y;
            }
            if (d < a.digits) total[d] = below + x - own;
            below += __shfl(x, 63);
        }
    }
    __syncthreads();
    for (int d = tid; d < a.digits; d += kThreads) {
        const uint32_t first = total[d] + next[0][d];
#pragma unroll
        for (int w = 1; w < kSortWaves; ++w) next[w][d] += first;
        next[0][d] = first;
    }
    __syncthreads();
    for (int64_t i0 = lo; i0 < hi; i0 += 64 * kSortAhead) {   // wave-uniform bounds
        uint32_t k[kSortAhead], o[kSortAhead];
        digit_load<I, kFirst>(a, i0 + lane, hi, k);
#pragma unroll
        for (int u = 0; u < kSortAhead; ++u) {
            const int64_t i = i0 + 64 * u + lane;
            if constexpr (kFirst) o[u] = uint32_t(i);
            else o[u] = ((Global<const uint32_t>*)a.in_order)[i < hi ? i : hi - 1];
        }
#pragma unroll
        for (int u = 0; u < kSortAhead; ++u) {
            const bool there = i0 + 64 * u + lane < hi;
            const uint32_t d = (k[u] >> a.shift) & (a.digits - 1);
            // lanes with the same digit
            uint64_t same = __ballot(there);
            for (int bit = 1; bit < a.digits; bit *= 2) {
                const uint64_t with = __ballot((d & bit) != 0);
                same &= (d & bit) ? with : ~with;
            }
            uint32_t to = 0;
            const int before = __popcll(same & ((uint64_t(1) << lane) - 1));
            if (there) to = next[wave][d] + before;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            if (there && (same >> lane) == 1) next[wave][d] += before + 1;   // the last of them
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            if (there && int64_t(to) < a.s.n) {   // always, unless tokens changed between the passes, which read them again
                a.s.key[to] = k[u];
                a.s.order[to] = o[u];
            }
        }
    }
}

// ---------------------------------------------------------------------------
// sums
// ---------------------------------------------------------------------------

constexpr int kChunk = 64 * kOctet;   // columns of a wave
constexpr int kAhead = 4;             // rows of dy loaded at once: few registers, more waves (16: 81 us where 4 take 71)

struct SumArgs {
    EmbedLaunch e;
    const uint32_t* key;      // n sorted rows
    const uint32_t* order;
    float* part;              // [tiles][2][chunks * kChunk]: of the run that enters a tile, and of the one that leaves it
    int64_t tiles;
    int32_t tile;             // length: 8, 16, 32 or a multiple of 64
    int32_t chunks;
};

__device__ __forceinline__ uint32_t uniform(uint32_t x) { return uint32_t(__builtin_amdgcn_readfirstlane(int(x))); }

template <int DO>
__device__ __forceinline__ void finish_row(const EmbedLaunch& e, uint32_t row, int64_t col, int64_t left,
                                           const float acc[kOctet]) {
    if (left <= 0) return;
    char* at = place<DO>(e.out, row, e.s_out, col);
    Octet<DO> y;
    if (e.accumulate) {
        y = load_octet<DO>(at, left);
#pragma unroll
        for (int k = 0; k < kOctet; ++k) y.set(k, y.get(k) + e.scale * acc[k]);
    } else {
#pragma unroll
        for (int k = 0; k < kOctet; ++k) y.set(k, e.scale * acc[k]);
    }
    store_octet<DO, true>(at, left, y);
}

// The 512 columns of tile t of the sorted list.
template <int DI, int DO>
__device__ __forceinline__ void sum_tile(const SumArgs& a, int64_t t, int chunk) {
    const int lane = int(threadIdx.x) & 63;
    const int64_t col = int64_t(chunk) * kChunk + lane * kOctet, left = a.e.cols - col;
    const int64_t lo = t * a.tile, hi = lo + a.tile < a.e.n ? lo + a.tile : a.e.n;
    const uint32_t none = uint32_t(a.e.rows);
    float acc[kOctet] = {};
    uint32_t run = uniform(a.key[lo]);   // the row that acc is of
    bool enters = lo > 0 && uniform(a.key[lo > 0 ? lo - 1 : 0]) == run;
    float* mine = a.part + t * 2 * a.chunks * kChunk + col;

    const auto flush = [&](bool leaves) {
        if (run >= none) return;
        if (enters || leaves) {
            float* at = mine + (enters ? 0 : a.chunks * kChunk);
            ((Global<f32x4>*)at)[0] = f32x4{acc[0], acc[1], acc[2], acc[3]};
            ((Global<f32x4>*)at)[1] = f32x4{acc[4], acc[5], acc[6], acc[7]};
        } else {
            finish_row<DO>(a.e, run, col, left, acc);
        }
    };
    for (int64_t p0 = lo; p0 < hi; p0 += 64) {
        const int64_t p = p0 + lane;
        const uint32_t keys = p < hi ? a.key[p] : none, places = p < hi ? a.order[p] : 0;
        const int m = int(hi - p0 < 64 ? hi - p0 : 64);
        constexpr int ahead = kAhead;
        for (int j0 = 0; j0 < m; j0 += ahead) {
            Octet<DI> x[ahead];
#pragma unroll
            for (int j = 0; j < ahead; ++j) {
                x[j].zero();
                const uint32_t r = uint32_t(__builtin_amdgcn_readlane(int(keys), j0 + j));   // none behind hi
                const uint32_t i = uint32_t(__builtin_amdgcn_readlane(int(places), j0 + j));
                // (i is below n unless tokens changed while they were sorted: places that nothing wrote)
                if (r < none && i < a.e.n) x[j] = load_octet<DI, true>(place<DI>(a.e.in, i, a.e.s_in, col), left);
            }
#pragma unroll
            for (int j = 0; j < ahead; ++j) {
                if (j0 + j >= m) break;
                const uint32_t r = uint32_t(__builtin_amdgcn_readlane(int(keys), j0 + j));
                if (r != run) {
                    flush(false);
                    run = r;
                    enters = false;
#pragma unroll
                    for (int k = 0; k < kOctet; ++k) acc[k] = 0.0f;
                }
#pragma unroll
                for (int k = 0; k < kOctet; ++k) acc[k] += x[j].get(k);
            }
        }
    }
    flush(hi < a.e.n && uniform(a.key[hi < a.e.n ? hi : 0]) == run);
}

template <int DI, int DO>
__global__ __launch_bounds__(kThreads) void tile_sum_kernel(const SumArgs a) {
    const int64_t w = int64_t(blockIdx.x) * (kThreads / 64) + (int(threadIdx.x) >> 6);
    const int64_t t = w / a.chunks;
    if (t < a.tiles) sum_tile<DI, DO>(a, t, int(w - t * a.chunks));
}

// Adds up the partial sums of the runs that cross tiles, 512 columns of them.  A wave looks
// at one tile's end; a run that leaves the tile and began in it is the wave's own if it
// crosses few tiles, and else the block's, whose four waves have a quarter of its tiles each.
constexpr int kJoinWaves = kThreads / 64, kJoinOwn = 8;
struct Run {
    int64_t first, count;   // tiles
    uint32_t row;
};
// The run that leaves tile t and began in it; count 0: there is none.
__device__ __forceinline__ Run run_from(const SumArgs& a, int64_t t) {
    const int lane = int(threadIdx.x) & 63;
    const int64_t end = (t + 1) * a.tile, lo = t * a.tile;   // end is below n
    const uint32_t after = a.key[end], before = a.key[end - 1], at = a.key[lo], earlier = a.key[lo > 0 ? lo - 1 : 0];
    Run r = {t, 0, uniform(after)};
    if (r.row >= uint32_t(a.e.rows) || uniform(before) != r.row) return r;
    if (lo > 0 && uniform(at) == r.row && uniform(earlier) == r.row) return r;   // began earlier
    // the last tile that the run enters
    int64_t last = t + 1;
    for (;;) {
        const int64_t p = (last + 1 + lane) * a.tile;
        const uint64_t on = __ballot(p < a.e.n && a.key[p < a.e.n ? p : 0] == r.row && a.key[p < a.e.n ? p - 1 : 0] == r.row);
        const int c = on == ~uint64_t(0) ? 64 : __ffsll((unsigned long long)~on) - 1;
        last += c;
        if (c < 64) break;
    }
    r.count = last - t + 1;
    return r;
}
// The sum of the run's parts `begin` .. `stop` - 1, in order.
__device__ __forceinline__ void add_parts(const SumArgs& a, const Run& r, int64_t begin, int64_t stop, int64_t col, f32x4 acc[2]) {
    const int64_t half = int64_t(a.chunks) * kChunk;
    constexpr int ahead = 8;
    for (int64_t u = begin; u < stop; u += ahead) {
        f32x4 x[ahead][2];
#pragma unroll
        for (int j = 0; j < ahead; ++j) {
            const int64_t v = u + j < stop ? u + j : stop - 1;
            // (it leaves its first tile, wherever it began there, and enters the others)
            const float* p = a.part + ((r.first + v) * 2 + (v == 0 ? 1 : 0)) * half + col;
            x[j][0] = ((Global<const f32x4>*)p)[0];
            x[j][1] = ((Global<const f32x4>*)p)[1];
        }
#pragma unroll
        for (int j = 0; j < ahead; ++j)
            if (u + j < stop) {
                acc[0] += x[j][0];
                acc[1] += x[j][1];
            }
    }
}
template <int DO>
__device__ __forceinline__ void put_run(const SumArgs& a, const Run& r, int64_t col, const f32x4 acc[2]) {
    const float all[kOctet] = {acc[0].x, acc[0].y, acc[0].z, acc[0].w, acc[1].x, acc[1].y, acc[1].z, acc[1].w};
    finish_row<DO>(a.e, r.row, col, a.e.cols - col, all);
}
template <int DO>
__global__ __launch_bounds__(kThreads) void join_kernel(const SumArgs a) {
    __shared__ f32x4 sums[kJoinWaves - 1][2][64];
    __shared__ Run runs[kJoinWaves];
    const int lane = int(threadIdx.x) & 63, wave = int(uniform(threadIdx.x >> 6));
    const int64_t four = int64_t(blockIdx.x) / a.chunks, t = four * kJoinWaves + wave;
    const int64_t col = (int64_t(blockIdx.x) - four * a.chunks) * kChunk + lane * kOctet;
    Run own = {t, 0, 0};
    if (t < a.tiles - 1) own = run_from(a, t);
    if (lane == 0) runs[wave] = own;
    if (own.count > 0 && own.count <= kJoinOwn) {
        f32x4 acc[2] = {};
        add_parts(a, own, 0, own.count, col, acc);
        put_run<DO>(a, own, col, acc);
    }
    __syncthreads();
    for (int i = 0; i < kJoinWaves; ++i) {
        const Run r = runs[i];
        if (r.count <= kJoinOwn) continue;   // the same for all waves
        const int64_t share = (r.count + kJoinWaves - 1) / kJoinWaves, begin = wave * share;
        f32x4 acc[2] = {};
        add_parts(a, r, begin, begin + share < r.count ? begin + share : r.count, col, acc);
        if (wave > 0) {
            sums[wave - 1][0][lane] = acc[0];
            sums[wave - 1][1][lane] = acc[1];
        }
        __syncthreads();
        if (wave == 0) {
            for (int w = 1; w < kJoinWaves; ++w)
                if (w * share < r.count) {
                    acc[0] += sums[w - 1][0][lane];
                    acc[1] += sums[w - 1][1][lane];
                }
            put_run<DO>(a, r, col, acc);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

// Tiles of 8 tokens while 8192 waves take them, a multiple of what the card holds:
// short ones hide the loads' latency, long ones leave fewer partial sums.
int tile_length(int64_t n, int64_t chunks) {
    int t = 8;
    while (t < 512 && n / t * chunks > 8192) t *= 2;
    return t;
}

struct Plan {
    int64_t tiles, part;        // part: elements of a sorting block
    int32_t tile, chunks, blocks, passes, digits;
    int64_t off_key[2], off_order[2], off_count, off_part, bytes;
};
Plan plan_for(int64_t n, int64_t rows, int64_t cols) {
    Plan p = {};
    p.chunks = int32_t((cols + kChunk - 1) / kChunk);
    p.tile = tile_length(n, p.chunks);
    p.tiles = (n + p.tile - 1) / p.tile;
    int bits = 1;   // rows is a key too
    while ((int64_t(1) << bits) <= rows) ++bits;
    p.passes = n <= kRankMost ? 0 : (bits + kDigitBits - 1) / kDigitBits;
    p.digits = p.passes ? 1 << ((bits + p.passes - 1) / p.passes) : 0;
    p.part = (n + kMaxSortBlocks - 1) / kMaxSortBlocks;
    p.part = p.part > 1024 ? (p.part + 1023) / 1024 * 1024 : 1024;
    p.blocks = int32_t((n + p.part - 1) / p.part);
    const auto take = [&](int64_t bytes) {
        const int64_t at = p.bytes;
        p.bytes += (bytes + 255) / 256 * 256;
        return at;
    };
    for (int i = 0; i < (p.passes > 1 ? 2 : 1); ++i) {
        p.off_key[i] = take(4 * n);
        p.off_order[i] = take(4 * n);
    }
    if (p.passes) p.off_count = take(4 * int64_t(p.blocks) * p.digits);
    p.off_part = take(p.tiles > 1 ? p.tiles * 2 * p.chunks * kChunk * 4 : 0);
    return p;
}

template <int DI, int DO>
void run_sum(const SumArgs& a, hipStream_t s, const KernelEvents& ev) {
    const bool join = a.tiles > 1;
    KernelEvents one = {ev.start, join ? nullptr : ev.stop};
    launch(tile_sum_kernel<DI, DO>, dim3(uint32_t((a.tiles * a.chunks + 3) / 4)), kThreads, s, one, a);
    if (!join) return;
    one = {nullptr, ev.stop};
    launch(join_kernel<DO>, dim3(uint32_t((a.tiles - 1 + kJoinWaves - 1) / kJoinWaves * a.chunks)), kThreads, s, one, a);
}

template <int DI, int DO>
void run_lookup(const LookupArgs& a, hipStream_t s, const KernelEvents& ev) {
    constexpr int64_t per = kThreads * kRowOctets;
    const dim3 grid(uint32_t((a.octets + per - 1) / per));
    if (a.e.token_bytes == 8) launch(lookup_kernel<DI, DO, int64_t>, grid, kThreads, s, ev, a);
    else launch(lookup_kernel<DI, DO, int32_t>, grid, kThreads, s, ev, a);
}

// f<in type, out type>() for the dtype numbers.
template <typename F>
void for_types(int32_t in, int32_t out, const F& f) {
    const auto with_in = [&](auto di) {
        if (out == ZERO_DTYPE_FP16) f(di, std::integral_constant<int, ZERO_DTYPE_FP16>{});
        else if (out == ZERO_DTYPE_BF16) f(di, std::integral_constant<int, ZERO_DTYPE_BF16>{});
        else f(di, std::integral_constant<int, ZERO_DTYPE_FP32>{});
    };
    if (in == ZERO_DTYPE_FP16) with_in(std::integral_constant<int, ZERO_DTYPE_FP16>{});
    else if (in == ZERO_DTYPE_BF16) with_in(std::integral_constant<int, ZERO_DTYPE_BF16>{});
    else with_in(std::integral_constant<int, ZERO_DTYPE_FP32>{});
}

}  // namespace

// Octets of a row: two at least, the second one of nothing where there is one.
static Divisor octets_of(int64_t cols) {
    const int64_t g = (cols + kOctet - 1) / kOctet;
    return divisor(uint32_t(g < 2 ? 2 : g));
}

hipError_t launch_lookup(const EmbedLaunch& e, hipStream_t s, const KernelEvents& ev) {
    LookupArgs a;
    a.e = e;
    a.per_row = octets_of(e.cols);
    a.octets = e.n * a.per_row.g;
    for_types(e.type, e.out_type, [&](auto di, auto d_o) { run_lookup<decltype(di)::value, decltype(d_o)::value>(a, s, ev); });
    return hipGetLastError();
}

int64_t embedding_work(int64_t n, int64_t rows, int64_t cols) { return plan_for(n, rows, cols).bytes; }

bool embedding_fits(int64_t n, int64_t rows, int64_t cols) {
    const Plan p = plan_for(n, rows, cols);
    constexpr int64_t most = int64_t(1) << 24;   // blocks of a launch
    // the first launch sorts and fills, by 512 threads a block
    const int64_t sorting = p.passes ? p.blocks : (n + kRankTokens - 1) / kRankTokens;
    return sorting + (rows + kFillRows - 1) / kFillRows < most / 2 && p.tiles * p.chunks < most;
}

hipError_t launch_embedding_grad(const EmbedLaunch& e, hipStream_t s, const KernelEvents& ev) {
    const Plan p = plan_for(e.n, e.rows, e.cols);
    char* work = static_cast<char*>(e.work);
    const auto list = [&](int64_t off) { return reinterpret_cast<uint32_t*>(work + off); };
    SumArgs a = {};
    a.e = e;
    a.tile = p.tile;
    a.tiles = p.tiles;
    a.chunks = p.chunks;
    a.part = reinterpret_cast<float*>(work + p.off_part);
    const int last = p.passes ? (p.passes - 1) & 1 : 0;   // the lists that the last pass writes
    a.key = list(p.off_key[last]);
    a.order = list(p.off_order[last]);

    SortArgs so = {e.tokens, e.n, e.first, e.rows, list(p.off_key[0]), list(p.off_order[0]), {}};
    const int64_t units = e.out_type == ZERO_DTYPE_FP32 ? 2 : 1;   // of 16 bits
    so.fill = {static_cast<char*>(e.out), 2 * units * e.s_out, e.accumulate ? 0 : e.rows, units * e.cols, octets_of(units * e.cols),
               p.passes ? p.blocks : int32_t((e.n + kRankTokens - 1) / kRankTokens)};
    const dim3 first(uint32_t(so.fill.before + so.fill.blocks()));
    KernelEvents one = {ev.start, nullptr};
    const bool wide = e.token_bytes == 8;
    if (p.passes == 0) {
        if (e.n == 0) one.stop = ev.stop;   // nothing comes after
        launch(wide ? rank_kernel<int64_t> : rank_kernel<int32_t>, first, kRankThreads, s, one, so);
        if (e.n == 0) return hipGetLastError();
        one.start = nullptr;
    }
    for (int k = 0; k < p.passes; ++k) {
        DigitArgs d = {};
        d.s = so;
        d.s.key = list(p.off_key[k & 1]);
        d.s.order = list(p.off_order[k & 1]);
        d.in_key = k ? list(p.off_key[(k - 1) & 1]) : nullptr;
        d.in_order = k ? list(p.off_order[(k - 1) & 1]) : nullptr;
        d.count = list(p.off_count);
        d.part = p.part;
        d.blocks = p.blocks;
        d.digits = p.digits;
        d.shift = k * __builtin_ctz(uint32_t(p.digits));
        const KernelEvents none;
        const auto count = k > 0 ? digit_count_kernel<int32_t, false> : wide ? digit_count_kernel<int64_t, true> : digit_count_kernel<int32_t, true>;
        launch(count, k > 0 ? dim3(p.blocks) : first, kThreads, s, one, d);
        one.start = nullptr;
        const auto move = k > 0 ? digit_move_kernel<int32_t, false> : wide ? digit_move_kernel<int64_t, true> : digit_move_kernel<int32_t, true>;
        launch(move, dim3(p.blocks), kThreads, s, none, d);
    }
    for_types(e.type, e.out_type, [&](auto di, auto d_o) { run_sum<decltype(di)::value, decltype(d_o)::value>(a, s, {one.start, ev.stop}); });
    return hipGetLastError();
}

}  // namespace zp
