// weight_grad.hip -- weight and bias gradient of a linear layer from the 8-bit
// checkpoint of its input (gfx950):
//   dw[n, k] = sum_t dy[t, n] x[t, k]        bias[n] = sum_t dy[t, n]
//
// A matrix product whose sum runs over the rows of both operands, one of them in
// 8 bits with a scale for each 32 values: nothing but a product of its own reads it
// without writing a 16-bit copy first.  Both operands go through LDS as they lie in memory,
// and LDS reads that transpose (ds_read_b64_tr_b16) make the matrix unit's fragments of
// them.  Bound by the matrix unit's feeding; measured, with 2 T n k operations:
//   8192 x 8192 x 8192           bf16 740 to 790 us (1390 to 1490 TFLOP/s), fp16 812 to 870 (1260 to 1354)
//   8192 x 20480 x 5120, bias    bf16 1283 to 1423 us (1208 to 1340)
//   8192 x 4096 x 4096           fp32 604 to 653 us (421 to 455: three products for one)
// for rows of dy that start on 16 bytes, and an even n.  Others go through registers:
//   8192 x 13653 x 5120, bias    bf16 1393 us (822), fp16 1445 to 1468 (780 to 793); n = 13656: 952, 986 to 1021
//   8192 x 50257 x 5120, bias    bf16 4940 us (853), fp16 4903 (860); n = 50264: 3250 to 3352, 3543 to 3623
// where the library's product of two 16-bit matrices takes 733 us for 8192^3 (1501) and
// 1075 to 1597 us for the second.
#include <type_traits>
#include <utility>

#include "octets.hpp"
#include "timed_launch.hpp"

#pragma clang fp contract(off)

namespace zp {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

template <typename T>
using Shared = __attribute__((address_space(3))) T;

// Bytes of LDS per row of a tile, and where pair q (16 columns) of row t is: the
// 16 lanes of a transposing read take 32 bytes of each of 4 rows, and the wave
// those of 16 rows.  Exchanging the pairs by the row's lowest bits spreads them
// over all banks.
template <int W>
__device__ __forceinline__ uint32_t pair_at(int t, int q) {
    return uint32_t(t * (W * 2) + ((q ^ (t & 7 & (W / 16 - 1))) << 5));
}

// The products are of 16-bit numbers, exact in fp32, and what they are made from is
// there whole:
//   bf16   dy as it is, x in bf16: an e4m3 number has 4 bits, and every scale is in range
//   fp32   dy as three bf16 numbers (24 bits) whose sum it is, x in bf16
//   fp16   dy as it is, x in fp16, which needs a common scale to be in range: each 32
//          columns' largest, over the tokens of the block, is brought to 57344 at most, and
//          the sums are brought back.  Blocks down to 2^-22 of the largest keep all
//          bits, and so does any x that was stored from fp16 (multiples of 2^-24) up to
//          57344.  Of smaller ones the low bits are rounded, at 2^-41 of the largest.
//          (As two bf16 numbers dy took twice the products: 242 us for 16384 tokens,
//          1600 x 1600 in the kernel below, and 32 KB more LDS.)
constexpr int parts_of(int d) { return d == ZERO_DTYPE_FP32 ? 3 : 1; }
constexpr int kTop = 134;   // the largest scale's byte in fp16 products: 448 2^7 = 57344

template <int D>
struct Op {   // fp16
    static constexpr bool kScaled = true;
    static constexpr short one = 0x3C00;
    static __device__ __forceinline__ uint32_t pair(uint32_t code, float f, bool high) {
        return high ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(code, f, true))
                    : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(code, f, false));
    }
    static __device__ __forceinline__ f32x4 multiply(s16x8 a, s16x8 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    }
    // c += a b in place: the compiler's own would move sums about.  A sum may be read 16
    // wait states later.
    static __device__ __forceinline__ void multiply_a(f32x4& c, s16x8 a, s16x8 b) {
        asm("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
    }
    static __device__ __forceinline__ void multiply_v(f32x4& c, s16x8 a, s16x8 b) {
        asm("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+v"(c) : "v"(a), "v"(b));
    }
};
struct OpBf16 {
    static constexpr bool kScaled = false;
    static constexpr short one = 0x3F80;
    static __device__ __forceinline__ uint32_t pair(uint32_t code, float f, bool high) {
        return high ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(code, f, true))
                    : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(code, f, false));
    }
    static __device__ __forceinline__ f32x4 multiply(s16x8 a, s16x8 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ void multiply_a(f32x4& c, s16x8 a, s16x8 b) {
        asm("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
    }
    static __device__ __forceinline__ void multiply_v(f32x4& c, s16x8 a, s16x8 b) {
        asm("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+v"(c) : "v"(a), "v"(b));
    }
};
template <>
struct Op<ZERO_DTYPE_BF16> : OpBf16 {};
template <>
struct Op<ZERO_DTYPE_FP32> : OpBf16 {};

// Two pairs of codes with scale byte `s`, `top` being the columns' largest.
template <int D>
__device__ __forceinline__ u32x4 decode(u32x2 code, uint32_t s, uint32_t top) {
    // beyond either end: what has no bits left is zero, and 255's codes are NaN
    if (Op<D>::kScaled) s = uint32_t(max(min(int(s) - int(top) + kTop, 255), 0));
    const float f = number(s << 23);
    return u32x4{Op<D>::pair(code.x, f, false), Op<D>::pair(code.x, f, true), Op<D>::pair(code.y, f, false), Op<D>::pair(code.y, f, true)};
}

// Tiles of W x W outputs, steps of STEP tokens.
constexpr int kTile = 256, kSmall = 64;
template <int D_, int STEP_, int W_>
struct Config {
    static constexpr int D = D_, W = W_, BM = W, BN = W, WM = 2, WN = W == kTile ? 4 : 2, STEP = STEP_;
    static constexpr int P = parts_of(D);
    static constexpr int threads = 64 * WM * WN;
    static constexpr int MI = BM / WM / 16, NI = BN / WN / 16;
    static constexpr int a_chunks = STEP * BM / 16 / threads;   // of 16 values, a thread's
    static constexpr int b_chunks = STEP * BN / 16 / threads;
    static constexpr int a_bytes = STEP * BM * 2, b_bytes = STEP * BN * 2;
    static constexpr int stage = a_bytes + P * b_bytes, lds_bytes = 2 * stage;
    static constexpr int G = W == kTile ? 1 : 2;   // fragments of n that leave at a time
    static_assert(a_chunks * threads * 16 == STEP * BM && b_chunks * threads * 16 == STEP * BN, "loads");
    static_assert(2 * stage <= 160 * 1024, "LDS");
};

struct GemmArgs {
    WeightGradLaunch w;
    int64_t pitch;       // of the codes
    int64_t blocks;      // scale bytes of a row
    int32_t tiles_k, tiles_n;
    int32_t whole;       // tiles that one block has for all tokens, the first ones; each of the others has
    int32_t splits;      // `splits` blocks (1: all are whole)
    int64_t per_split;   // tokens of a split, a multiple of kUnit
    float* part;         // sums of tile whole + i and split j: W x W at (i splits + j) part_size(W), as dw has
                         // them, then W of dy's columns
    int32_t shares;      // whose the bias is: 0: the first k-tile's, else k-tile i / 2's for fragments i shares on of each 8
};
constexpr int64_t part_size(int w) { return w * w + w; }
constexpr int64_t kUnit = 64;

// What is left of x without its first part, of bits u: nothing of an infinity, where the
// difference would be NaN.
__device__ __forceinline__ float less(float x, uint32_t u) { return fabsf(x) == INFINITY ? 0.0f : x - number(u); }

// 16 values of dy.
template <int D>
struct Chunk {
    Octet<D> o[2];
    __device__ __forceinline__ void load(const char* p, int64_t left) {
        o[0] = load_octet<D>(p, left);
        o[1] = load_octet<D>(p + sizeof(typename Type<D>::elem) * 8, left - 8);
    }
    // part j of the values, as pairs
    __device__ __forceinline__ void split(u32x4 to[parts_of(D)][2]) const {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (D != ZERO_DTYPE_FP32) {
                    to[0][h][i] = uint32_t(o[h].v[2 * i]) | uint32_t(o[h].v[2 * i + 1]) << 16;
                } else {
                    float a = o[h].get(2 * i), b = o[h].get(2 * i + 1);
#pragma unroll
                    for (int j = 0; j < parts_of(D); ++j) {
                        const uint32_t ua = bits(a) & 0xFFFF0000u, ub = bits(b) & 0xFFFF0000u;
                        to[j][h][i] = ua >> 16 | ub;
                        a = j ? a - number(ua) : less(a, ua);
                        b = j ? b - number(ub) : less(b, ub);
                    }
                }
            }
    }
};

// 16 codes and their scale.
struct Codes {
    u32x4 code;
    uint32_t scale;
};

// A fragment of 16 columns by 32 rows: the lane has column lane & 15 of rows
// 4 (lane / 16) + 0 .. 3 and 16 more.  (Which of the 32 rows come where does not
// matter as long as both operands have the same.)
__device__ __forceinline__ s16x8 fragment(uint32_t at, int row_bytes) {
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Shared<s16x4>*)uintptr_t(at));
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Shared<s16x4>*)uintptr_t(at + 16 * row_bytes));
    return s16x8{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}

// Where a block's results go: dw, or the fp32 sums of a split.
struct Target {
    char* p;
    int64_t rows, cols, ld;   // elements
    bool accumulate;
};

// Four neighbouring values of a row.
template <int DO>
struct Four {
    typedef typename Type<DO>::elem E;
    typedef E vec __attribute__((ext_vector_type(4)));
    typedef vec at __attribute__((aligned(sizeof(E))));
    static __device__ __forceinline__ float wide(E e) {
        if constexpr (DO == ZERO_DTYPE_FP32) return e;
        else return Type<DO>::wide(e);
    }
    static __device__ __forceinline__ E narrow(float x) {
        if constexpr (DO == ZERO_DTYPE_FP32) return x;
        else return Type<DO>::narrow(x);
    }
};

// Writes the R x N values that a wave has in LDS, rows of `pitch` floats, to the rows and
// columns from (row, col) on.
template <int DO, int R, int N, int kPitch>
__device__ __forceinline__ void store_rows(const Target& t, const float* stage, int64_t row, int64_t col) {
    typedef Four<DO> F;
    typedef typename F::E E;
    constexpr int fours = N / 4, per = 64 / fours, count = R / per, batch = count < 8 ? count : 8;   // rows a load, loads
    static_assert(64 % fours == 0 && R % per == 0 && count % batch == 0, "whole rows");
    const int lane = int(threadIdx.x) & 63, r0 = lane / fours, c = lane % fours * 4;
    const float* from = stage + r0 * kPitch + c;
    Global<E>* p = (Global<E>*)t.p + (row + r0) * t.ld + col + c;
    const int64_t step = per * t.ld;
    if (row + R <= t.rows && col + N <= t.cols) {   // all there
#pragma unroll 1
        for (int x = 0; x < count; x += batch) {
            f32x4 v[batch];
            typename F::vec y[batch];
#pragma unroll
            for (int i = 0; i < batch; ++i) v[i] = *reinterpret_cast<const f32x4*>(from + (x + i) * per * kPitch);
            if (t.accumulate)
#pragma unroll
                for (int i = 0; i < batch; ++i) y[i] = *(Global<typename F::at>*)(p + i * step);
#pragma unroll
            for (int i = 0; i < batch; ++i) {
#pragma unroll
                for (int k = 0; k < 4; ++k) y[i][k] = F::narrow(t.accumulate ? F::wide(y[i][k]) + v[i][k] : v[i][k]);
                *(Global<typename F::at>*)(p + i * step) = y[i];
            }
            p += batch * step;
        }
        return;
    }
    if (col >= t.cols) return;
    const int64_t left = t.cols - col - c;   // may be negative
#pragma unroll 1
    for (int64_t x = 0; x < R && row + x < t.rows; x += per) {
        const f32x4 v = *reinterpret_cast<const f32x4*>(from);
        from += per * kPitch;
        if (row + r0 + x < t.rows) {
            if (left >= 4) {
                typename F::vec y = {};
                if (t.accumulate) y = *(Global<typename F::at>*)p;
#pragma unroll
                for (int k = 0; k < 4; ++k) y[k] = F::narrow(t.accumulate ? F::wide(y[k]) + v[k] : v[k]);
                *(Global<typename F::at>*)p = y;
            } else {
#pragma unroll
                for (int k = 0; k < 3; ++k)
                    if (k < left) p[k] = F::narrow(t.accumulate ? F::wide(p[k]) + v[k] : v[k]);
            }
        }
        p += step;
    }
}

template <int DO>
__device__ __forceinline__ void put_bias(const GemmArgs& a, int64_t n, float v) {
    typedef typename Type<DO>::elem E;
    Global<E>* p = (Global<E>*)a.w.bias + n;
    if constexpr (DO == ZERO_DTYPE_FP32) *p = a.w.accumulate ? *p + v : v;
    else *p = Type<DO>::narrow(a.w.accumulate ? Type<DO>::wide(*p) + v : v);
}

// Which outputs and tokens a block has.  Blocks go round the 8 XCDs, so those of
// one XCD take neighbouring tiles, 4 n-tiles wide: the 32 that run there at a time
// are 8 by 4 and read 12 slabs from its L2 instead of up to 33.
constexpr int kGroup = 4;
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return uint32_t(__builtin_amdgcn_readfirstlane(int(x))); }
struct Part {
    int64_t k0, n0, t_begin, t_end;
    int64_t slot;   // of its sums in `part`; -1: it has all tokens
};
__device__ __forceinline__ uint32_t in_order(uint32_t id, uint32_t total) {
    const uint32_t xcd = id & 7, q8 = total >> 3, r8 = total & 7;
    return xcd * q8 + (xcd < r8 ? xcd : r8) + (id >> 3);
}
template <int W>
__device__ __forceinline__ Part part_of(const GemmArgs& a) {
    const uint32_t id = blockIdx.x, whole = uint32_t(a.whole);
    Part p;
    uint32_t tile;
    if (id < whole) {
        tile = in_order(id, whole);
        p.slot = -1;
        p.t_begin = 0;
        p.t_end = a.w.T;
    } else {
        const uint32_t tiles = uint32_t(a.tiles_k) * uint32_t(a.tiles_n) - whole;
        const uint32_t i = in_order(id - whole, gridDim.x - whole), split = uniform(i / tiles);
        tile = whole + i - split * tiles;
        p.slot = int64_t(tile - whole) * a.splits + split;
        p.t_begin = int64_t(split) * a.per_split;
        p.t_end = p.t_begin + a.per_split < a.w.T ? p.t_begin + a.per_split : a.w.T;
    }
    const uint32_t group = uniform(tile / (kGroup * a.tiles_k)), rest = tile - group * (kGroup * a.tiles_k);
    const uint32_t wide = a.tiles_n - group * kGroup < kGroup ? a.tiles_n - group * kGroup : kGroup;
    const uint32_t tile_k = uniform(rest / wide);
    p.k0 = int64_t(tile_k) * W;
    p.n0 = int64_t(group * kGroup + rest - tile_k * wide) * W;
    return p;
}

// The largest scale of each 32 of a tile's columns over its tokens (255, which is NaN, aside),
// 1 at least, into top[0 .. kBlocks - 1].
template <int kThreads, int kBlocks>
__device__ __forceinline__ void largest_scales(const GemmArgs& a, const Part& part, uint32_t* top) {
    const int64_t left = a.blocks - (part.k0 >> 5);
    const int there = left < kBlocks ? int(left) : kBlocks;
    if (threadIdx.x < 8) top[threadIdx.x] = 1;
    __syncthreads();
    constexpr int batch = 8;
    uint32_t most[8] = {};
    // eight bytes at once, the last ones from where eight end, whatever follows a row cut off
    const Global<const uint8_t>* all = (Global<const uint8_t>*)a.w.scale;
    const int64_t end = a.w.T * a.blocks - 8, first = part.k0 >> 5;
    const uint64_t mine = there > 0 ? ~uint64_t(0) >> (8 * (8 - there)) : 0;
    for (int64_t t = part.t_begin + threadIdx.x; t < part.t_end; t += batch * kThreads) {
        uint64_t x[batch];
        if (end >= 0) {
            typedef uint64_t at __attribute__((aligned(1)));
            int past[batch];
#pragma unroll
            for (int i = 0; i < batch; ++i) {
                const int64_t u = t + i * kThreads < part.t_end ? t + i * kThreads : t, from = u * a.blocks + first;
                past[i] = from > end ? int(from - end) : 0;
                x[i] = *(Global<const at>*)(all + from - past[i]);
            }
#pragma unroll
            for (int i = 0; i < batch; ++i) x[i] = x[i] >> (8 * past[i]) & mine;
        } else {   // 7 bytes at most in all
#pragma unroll
            for (int i = 0; i < batch; ++i) x[i] = 0;
            for (int b = 0; b < there; ++b) x[0] |= uint64_t(all[t * a.blocks + first + b]) << (8 * b);
        }
#pragma unroll
        for (int i = 0; i < batch; ++i)
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                const uint32_t s = uint32_t(x[i] >> (8 * b)) & 255;
                most[b] = max(most[b], s == 255 ? 0 : s);
            }
    }
    // the largest of each row of 16 lanes, so that LDS has few to put in order
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
        most[b] = max(most[b], across<0xB1>(most[b]));    // lanes 1, 0, 3, 2 of each four
        most[b] = max(most[b], across<0x4E>(most[b]));    // lanes 2, 3, 0, 1
        most[b] = max(most[b], across<0x141>(most[b]));   // eight lanes mirrored
        most[b] = max(most[b], across<0x140>(most[b]));   // sixteen
    }
    if ((threadIdx.x & 15) == 0)
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) atomicMax(&top[b], most[b]);
    __syncthreads();
}

// Writes a block's products: the result, or its part of one that the tokens are
// split for.  They go through LDS, `G` fragments of n at a time, so that a row's
// neighbours leave together whichever way round dw is, and the code for its types
// is there once.
template <typename C, bool kScaled>
__device__ __forceinline__ void finish(const GemmArgs& a, const Part& part, char* lds, const f32x4 (&acc)[C::MI][C::NI],
                                       const int (&power)[C::MI / 2]) {
    constexpr int G = C::G, K = C::MI * 16, N = 16 * G;
    constexpr int pitch_k = K + 4, pitch_n = N + 4;   // floats; 4 more spread the rows over the banks
    constexpr int bytes = 4 * (N * pitch_k > K * pitch_n ? N * pitch_k : K * pitch_n);
    static_assert(bytes * C::WM * C::WN <= C::lds_bytes, "LDS");
    const int lane = int(threadIdx.x) & 63, wave = int(threadIdx.x) >> 6;
    const int wm = wave / C::WN, wn = wave % C::WN;
    float* stage = reinterpret_cast<float*>(lds + wave * bytes);
    const bool parts = part.slot >= 0;
    const int64_t k_wave = (parts ? 0 : part.k0) + wm * K, n_wave = (parts ? 0 : part.n0) + wn * (C::NI * 16);
    const int k_lane = 4 * (lane >> 4), n_lane = lane & 15;
    const Target to = parts ? Target{reinterpret_cast<char*>(a.part + part.slot * part_size(C::W)), C::W, C::W, C::W, false}
                            : Target{static_cast<char*>(a.w.dw), a.w.transposed ? a.w.k : a.w.n, a.w.transposed ? a.w.n : a.w.k, a.w.s_dw,
                                     a.w.accumulate};
    // 2^power of fragments m and m + 1, 32 columns
    const auto value = [&](int m, int i) {
        f32x4 v = acc[m][i];
        if (kScaled)
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = ldexpf(v[j], power[m / 2]);
        return v;
    };
    const int type = parts ? int(ZERO_DTYPE_FP32) : a.w.out_type;
    __syncthreads();   // every wave has read its last fragments
#pragma unroll
    for (int g = 0; g < C::NI; g += G) {
        const auto store = [&](auto d) {
            constexpr int DO = decltype(d)::value;
            if (a.w.transposed) store_rows<DO, K, N, pitch_n>(to, stage, k_wave, n_wave + 16 * g);
            else store_rows<DO, N, K, pitch_k>(to, stage, n_wave + 16 * g, k_wave);
        };
        if (!a.w.transposed) {
#pragma unroll
            for (int i = 0; i < G; ++i)
#pragma unroll
                for (int m = 0; m < C::MI; ++m)
                    *reinterpret_cast<f32x4*>(stage + (16 * i + n_lane) * pitch_k + 16 * m + k_lane) = value(m, g + i);
        } else {
#pragma unroll
            for (int i = 0; i < G; ++i)
#pragma unroll
                for (int m = 0; m < C::MI; ++m) {
                    const f32x4 v = value(m, g + i);
#pragma unroll
                    for (int j = 0; j < 4; ++j) stage[(16 * m + k_lane + j) * pitch_n + 16 * i + n_lane] = v[j];
                }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (type == ZERO_DTYPE_FP16) store(std::integral_constant<int, ZERO_DTYPE_FP16>{});
        else if (type == ZERO_DTYPE_BF16) store(std::integral_constant<int, ZERO_DTYPE_BF16>{});
        else store(std::integral_constant<int, ZERO_DTYPE_FP32>{});
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
}

// The sum over dy of 16 columns of the tile, from n on.
template <int W>
__device__ __forceinline__ void finish_bias(const GemmArgs& a, const Part& part, int n, float sum) {
    const int lane = int(threadIdx.x) & 63;
    n += lane;
    if (lane >= 16 || part.n0 + n >= a.w.n) return;
    if (part.slot >= 0) ((Global<float>*)a.part)[part.slot * part_size(W) + W * W + n] = sum;
    else if (a.w.out_type == ZERO_DTYPE_FP16) put_bias<ZERO_DTYPE_FP16>(a, part.n0 + n, sum);
    else if (a.w.out_type == ZERO_DTYPE_BF16) put_bias<ZERO_DTYPE_BF16>(a, part.n0 + n, sum);
    else put_bias<ZERO_DTYPE_FP32>(a, part.n0 + n, sum);
}

// Any dy: eight waves, loads through registers, all 256 of which the large tiles take (16-bit
// types spill some).
template <typename C>
__global__ __launch_bounds__(C::threads) void weight_grad_kernel(const GemmArgs a) {
    constexpr int D = C::D, P = C::P;
    __shared__ __attribute__((aligned(1024))) char lds[2 * C::stage];
    const int tid = int(threadIdx.x), lane = tid & 63, wave = tid >> 6;
    const int wm = wave / C::WN, wn = wave % C::WN;

    const Part part = part_of<C::W>(a);
    const int64_t k0 = part.k0, n0 = part.n0, t_begin = part.t_begin, t_end = part.t_end;
    __shared__ uint32_t top[8];
    if (Op<D>::kScaled) largest_scales<C::threads, C::W / 32>(a, part, top);

    Codes ra[C::a_chunks];
    Chunk<D> rb[C::b_chunks];
    const auto load = [&](int64_t t0) {
#pragma unroll
        for (int j = 0; j < C::a_chunks; ++j) {
            const int c = tid + j * C::threads;
            const int64_t t = t0 + c / (C::BM / 16), k = k0 + c % (C::BM / 16) * 16;
            ra[j].code = u32x4{};
            ra[j].scale = 1;
            if (t < t_end && k < a.pitch) {
                ra[j].code = *(Global<const u32x4>*)(a.w.code + t * a.pitch + k);
                ra[j].scale = ((Global<const uint8_t>*)a.w.scale)[t * a.blocks + (k >> 5)];
            }
        }
#pragma unroll
        for (int j = 0; j < C::b_chunks; ++j) {
            const int c = tid + j * C::threads;
            const int64_t t = t0 + c / (C::BN / 16), n = n0 + c % (C::BN / 16) * 16;
            rb[j].load(place<D>(a.w.dy, t, a.w.s_dy, n), t < t_end ? a.w.n - n : 0);
        }
    };
    const auto stash = [&](int buf) {
        char* base = lds + buf * C::stage;
#pragma unroll
        for (int j = 0; j < C::a_chunks; ++j) {
            const int c = tid + j * C::threads;
            u32x4* to = reinterpret_cast<u32x4*>(base + pair_at<C::BM>(c / (C::BM / 16), c % (C::BM / 16)));
            const uint32_t most = Op<D>::kScaled ? top[c % (C::BM / 16) / 2] : 0;
            to[0] = decode<D>(u32x2{ra[j].code.x, ra[j].code.y}, ra[j].scale, most);
            to[1] = decode<D>(u32x2{ra[j].code.z, ra[j].code.w}, ra[j].scale, most);
        }
#pragma unroll
        for (int j = 0; j < C::b_chunks; ++j) {
            const int c = tid + j * C::threads;
            u32x4 v[P][2];
            rb[j].split(v);
#pragma unroll
            for (int p = 0; p < P; ++p) {
                u32x4* to = reinterpret_cast<u32x4*>(base + C::a_bytes + p * C::b_bytes +
                                                     pair_at<C::BN>(c / (C::BN / 16), c % (C::BN / 16)));
                to[0] = v[p][0];
                to[1] = v[p][1];
            }
        }
    };

    f32x4 acc[C::MI][C::NI];
    f32x4 sum[C::NI];   // of dy's columns: a product with ones
#pragma unroll
    for (int i = 0; i < C::NI; ++i) {
        sum[i] = f32x4{};
#pragma unroll
        for (int m = 0; m < C::MI; ++m) acc[m][i] = f32x4{};
    }
    const bool bias = a.w.bias && k0 == 0 && wm == 0;
    s16x8 ones;
#pragma unroll
    for (int i = 0; i < 8; ++i) ones[i] = Op<D>::one;

    // where the lane's fragments are
    const int row = 4 * (lane >> 4) + ((lane & 15) >> 2);
    const uint32_t base = uint32_t(reinterpret_cast<uintptr_t>((Shared<char>*)lds)) + (lane & 3) * 8;
    uint32_t at_a[C::MI], at_b[C::NI];
#pragma unroll
    for (int m = 0; m < C::MI; ++m) at_a[m] = base + pair_at<C::BM>(row, wm * C::MI + m);
#pragma unroll
    for (int i = 0; i < C::NI; ++i) at_b[i] = base + C::a_bytes + pair_at<C::BN>(row, wn * C::NI + i);

    const int64_t steps = t_end > t_begin ? (t_end - t_begin + C::STEP - 1) / C::STEP : 0;
    if (steps > 0) {
        load(t_begin);
        stash(0);
    }
    __syncthreads();
    for (int64_t s = 0; s < steps; ++s) {
        if (s + 1 < steps) load(t_begin + (s + 1) * C::STEP);
        const uint32_t buf = uint32_t(s & 1) * C::stage;
#pragma unroll
        for (int h = 0; h < C::STEP / 32; ++h) {
            s16x8 fa[C::MI], fb[C::NI];
#pragma unroll
            for (int m = 0; m < C::MI; ++m) fa[m] = fragment(at_a[m] + buf + h * 32 * C::BM * 2, C::BM * 2);
#pragma unroll
            for (int p = 0; p < P; ++p) {
#pragma unroll
                for (int i = 0; i < C::NI; ++i)
                    fb[i] = fragment(at_b[i] + buf + p * C::b_bytes + h * 32 * C::BN * 2, C::BN * 2);
#pragma unroll
                for (int i = 0; i < C::NI; ++i)
#pragma unroll
                    for (int m = 0; m < C::MI; ++m)
                        acc[m][i] = Op<D>::multiply(fa[m], fb[i], acc[m][i]);
                if (bias)
#pragma unroll
                    for (int i = 0; i < C::NI; ++i)
                        sum[i] = Op<D>::multiply(ones, fb[i], sum[i]);
            }
        }
        if (s + 1 < steps) stash((s + 1) & 1);
        __syncthreads();
    }

    int power[C::MI / 2];
#pragma unroll
    for (int m = 0; m < C::MI / 2; ++m) power[m] = Op<D>::kScaled ? int(top[wm * (C::MI / 2) + m]) - kTop : 0;
    finish<C, Op<D>::kScaled>(a, part, lds, acc, power);
    if (bias)
#pragma unroll
        for (int i = 0; i < C::NI; ++i) finish_bias<C::W>(a, part, (wn * C::NI + i) * 16, sum[i][0]);
}

// The same for a dy of 16 bits that is aligned to 16 bytes: four waves of 128 x 128
// outputs, one to a SIMD.
//
// A phase is 32 tokens: 64 products of a wave, 16 cycles each on its matrix unit,
// in which the wave can issue up to three other instructions each.  Loads bring dy,
// codes and scales straight into LDS, where they are rings; what a phase does besides
// its own products is
//   - the codes of the phase after the next are decoded, from and to LDS,
//   - the fragments of the next phase are read,
//   - dy four phases ahead and codes five ahead are sent for.
// With loads through registers the compiler would wait for the newest of them at each use;
// so it knows of none, and one wait a phase leaves those of the last two phases under way.
// The loop holds ten phases, so that all places in the rings are constants.
template <int... I, typename F>
__device__ __forceinline__ void each(std::integer_sequence<int, I...>, const F& f) {
    (f(std::integral_constant<int, I>{}), ...);
}

struct Fast {
    static constexpr int W = kTile, BM = W, BN = W, WM = 2, WN = 2, MI = 8, NI = 8, threads = 256, G = 4;
    static constexpr int rows = 32;                               // of a phase
    static constexpr int a_bytes = rows * BM * 2, b_bytes = rows * BN * 2, code_bytes = rows * BM, scale_bytes = rows * 8 * 4;
    static constexpr int a_ring = 2, b_ring = 5, code_ring = 5, turn = 10;
    static constexpr int b_at = a_ring * a_bytes, code_at = b_at + b_ring * b_bytes, scale_at = code_at + code_ring * code_bytes;
    static constexpr int lds_bytes = scale_at + code_ring * scale_bytes;
    static constexpr int b_loads = b_bytes / 4096, code_loads = code_bytes / 4096, loads = b_loads + code_loads + 1;   // a wave's
    static_assert(lds_bytes <= 160 * 1024 && loads == 7, "LDS, and the waits below");
};

// Loads into LDS, the lanes' 16 bytes, or bytes as words, one after the other from
// `to` + kOffset on (m0).
template <int kOffset>
__device__ __forceinline__ void load16(uint32_t to, uint32_t from, u32x4 buffer) {
    asm volatile("s_add_u32 m0, %0, %1\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %3, 0 offen lds" ::"s"(to), "i"(kOffset), "v"(from), "s"(buffer) : "scc", "m0");
}
template <int kOffset>
__device__ __forceinline__ void load1(uint32_t to, uint32_t from, u32x4 buffer) {
    asm volatile("s_add_u32 m0, %0, %1\n\ts_nop 0\n\tbuffer_load_ubyte %2, %3, 0 offen lds" ::"s"(to), "i"(kOffset), "v"(from), "s"(buffer) : "scc", "m0");
}

template <int D, int kSums>
__global__ __launch_bounds__(256, 1) void weight_grad_fast_kernel(const GemmArgs a) {
    typedef Fast C;
    __shared__ __attribute__((aligned(1024))) char lds[C::lds_bytes];
    const int tid = int(threadIdx.x), lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / C::WN, wn = wave % C::WN;
    const Part part = part_of<C::W>(a);
    const int64_t k0 = part.k0, n0 = part.n0, t_begin = part.t_begin;
    uint32_t* const tops = reinterpret_cast<uint32_t*>(lds);   // until the loads come
    uint32_t top = 0;
    int power[C::MI / 2] = {};
    if (Op<D>::kScaled) {
        largest_scales<C::threads, C::W / 32>(a, part, tops);
        top = tops[(tid & 15) >> 1];   // of the columns that the thread decodes
#pragma unroll
        for (int m = 0; m < C::MI / 2; ++m) power[m] = __builtin_amdgcn_readfirstlane(int(tops[wm * (C::MI / 2) + m]) - kTop);
        __syncthreads();
    }
    const int tokens = int(part.t_end - part.t_begin), phases = (tokens + C::rows - 1) / C::rows;
    const uint32_t lds0 = uint32_t(reinterpret_cast<uintptr_t>((Shared<char>*)lds));

    // Loads.  Beyond a buffer's size they give zeros: rows behind the last token, codes
    // behind a row's end.  Load j of dy fills two rows of a tile, a lane's 16 bytes
    // coming from where the exchanged pairs put them; load j of the codes four.
    uint32_t from_b[C::b_loads], from_code[C::code_loads], from_scale;
#pragma unroll
    for (int j = 0; j < C::b_loads; ++j) {
        const int r = 2 * (wave * C::b_loads + j) + (lane >> 5), c = lane & 31;
        from_b[j] = uint32_t(r) * uint32_t(a.w.s_dy) * 2 + ((((c >> 1) ^ (r & 7)) * 2 + (c & 1)) << 4);
    }
#pragma unroll
    for (int j = 0; j < C::code_loads; ++j) {
        const int r = 4 * (wave * C::code_loads + j) + (lane >> 4), c = lane & 15;
        from_code[j] = uint32_t(r * a.pitch + 16 * c) | (k0 + 16 * c < a.pitch ? 0 : 0x80000000u);
    }
    from_scale = uint32_t((8 * wave + (lane >> 3)) * a.blocks + (lane & 7));
    // What is left of a matrix from the next phase on that is loaded: its address and bytes.
    struct Source {
        uint64_t p;
        uint32_t bytes;
        __device__ __forceinline__ u32x4 buffer() const { return {uint32_t(p), uint32_t(p >> 32), bytes, 0x00020000u}; }
        __device__ __forceinline__ void advance(uint32_t step) {
            p += step;
            // what is left, or 0 (the compiler would take a vector instruction for it)
            asm("s_sub_u32 %0, %0, %1\n\ts_cselect_b32 %0, 0, %0" : "+s"(bytes) : "s"(step) : "scc");
        }
    };
    const auto source = [](const void* base, int64_t offset, int64_t bytes) {
        return Source{(reinterpret_cast<uint64_t>(base) + uint64_t(offset)) & 0xFFFFFFFFFFFFull, uint32_t(bytes)};
    };
    // (dy's stride is n at least, a row of codes no shorter than its part from k0 on)
    Source dy = source(a.w.dy, (t_begin * a.w.s_dy + n0) * 2, ((tokens - 1) * a.w.s_dy + a.w.n - n0) * 2);
    Source codes = source(a.w.code, t_begin * a.pitch + k0, tokens * a.pitch - k0);
    Source scales = source(a.w.scale, t_begin * a.blocks + (k0 >> 5), tokens * a.blocks - (k0 >> 5));
    const uint32_t step_b = uint32_t(C::rows * a.w.s_dy * 2), step_code = uint32_t(C::rows * a.pitch), step_scale = uint32_t(C::rows * a.blocks);
    // Where a wave's loads go in slot 0 of each ring.
    const uint32_t to_b = lds0 + C::b_at + wave * C::b_loads * 1024, to_code = lds0 + C::code_at + wave * C::code_loads * 1024,
                   to_scale = lds0 + C::scale_at + wave * 256;

    // Codes: a thread decodes pair q of rows t and t + 16.  Lanes whose place has bit 2
    // set take their second half first, so that eight lanes' stores meet all banks.
    const int ta = tid >> 4, qa = tid & 15;
    const uint32_t swap = ((qa ^ ta) >> 2) & 1;
    const uint32_t code_from = lds0 + C::code_at + tid * 16 + 8 * swap, scale_from = lds0 + C::scale_at + (ta * 8 + (qa >> 1)) * 4;
    const uint32_t code_to = lds0 + pair_at<C::BM>(ta, qa) + 16 * swap;
    const auto raw = [&](int j, int h, int slot) {
        return *(Shared<const u32x2>*)uintptr_t((code_from ^ (8 * h)) + slot * C::code_bytes + j * 4096);
    };
    const auto raw_scale = [&](int j, int slot) {
        return *(Shared<const uint32_t>*)uintptr_t(scale_from + slot * C::scale_bytes + j * 512);
    };
    const auto place_codes = [&](u32x4 v, int j, int h, int buf) {
        *(Shared<u32x4>*)uintptr_t((code_to ^ (16 * h)) + buf * C::a_bytes + j * 16 * 512) = v;
    };

    const int row = 4 * (lane >> 4) + ((lane & 15) >> 2);
    uint32_t at_a[8], at_b[8];
#pragma unroll
    for (int m = 0; m < 8; ++m) {
        const uint32_t at = lds0 + pair_at<256>(row, m) + (lane & 3) * 8;
        at_a[m] = at + wm * 256;
        at_b[m] = at + C::b_at + wn * 256;
    }
    struct Frags { s16x8 a[C::MI], b[C::NI]; };
    const auto read = [&](Frags& f, int i, int buf, int slot) {   // its 16 fragments, in the order of their use
        if (i < 8) f.a[i] = fragment(at_a[i] + buf * C::a_bytes, 512);
        else f.b[i - 8] = fragment(at_b[i - 8] + slot * C::b_bytes, 512);
    };

    f32x4 acc[C::MI][C::NI];
#pragma unroll
    for (int i = 0; i < C::NI; ++i)
#pragma unroll
        for (int m = 0; m < C::MI; ++m) acc[m][i] = f32x4{};
    const auto multiply = [&](const Frags& f, int j) {
        Op<D>::multiply_a(acc[j & 7][j >> 3], f.a[j & 7], f.b[j >> 3]);
        __builtin_amdgcn_sched_barrier(0);
    };

    // The bias: the waves that have the same columns of dy (two in each k-tile) share
    // their 8 fragments, kSums for one, and multiply them with ones.  A wave behind
    // the last share takes the last one too and drops it.
    const int share = (int(k0 / C::BM) * 2 + wm) * kSums, first = min(share, C::NI - kSums);
    f32x4 sum[kSums + 1];
    s16x8 ones, fb[kSums + 1];
#pragma unroll
    for (int i = 0; i < 8; ++i) ones[i] = Op<D>::one;
    uint32_t at_sum[kSums + 1];
#pragma unroll
    for (int i = 0; i < kSums; ++i) {
        sum[i] = f32x4{};
        at_sum[i] = lds0 + C::b_at + pair_at<256>(row, wn * 8 + first + i) + (lane & 3) * 8;
    }
    Frags f0, f1;
    // The Q-th phase of a turn with its fragments in f; those of the next go to g.
    const auto phase = [&](auto turn, const Frags& f, Frags& g) __attribute__((always_inline)) {
        constexpr int Q = decltype(turn)::value;
        u32x2 raws[2][2];
        uint32_t rs[2];
        u32x4 d;
        each(std::make_integer_sequence<int, 64>{}, [&](auto at) __attribute__((always_inline)) {
            constexpr int j = decltype(at)::value;
            multiply(f, j);
            if constexpr (j < 2) {
                raws[j][0] = raw(j, 0, (Q + 2) % C::code_ring);
                raws[j][1] = raw(j, 1, (Q + 2) % C::code_ring);
                rs[j] = raw_scale(j, (Q + 2) % C::code_ring);
            }
            if constexpr (j >= 2 && j < 50 && j % 3 == 2) read(g, (j - 2) / 3, (Q + 1) % 2, (Q + 1) % C::b_ring);
            if constexpr (j >= 16 && j < 40 && j % 6 == 4) d = decode<D>(raws[(j - 16) / 12][(j - 16) / 6 % 2], rs[(j - 16) / 12], top);
            if constexpr (j >= 16 && j < 40 && j % 6 == 0) place_codes(d, (j - 16) / 12, (j - 16) / 6 % 2, Q % 2);
            if constexpr (j >= 40 && j < 52 && j % 3 == 1) load16<(Q + 4) % C::b_ring * C::b_bytes + (j - 40) / 3 * 1024>(to_b, from_b[(j - 40) / 3], dy.buffer());
            if constexpr (j == 52 || j == 55) load16<Q % C::code_ring * C::code_bytes + (j - 52) / 3 * 1024>(to_code, from_code[(j - 52) / 3], codes.buffer());
            if constexpr (j == 58) load1<Q % C::code_ring * C::scale_bytes>(to_scale, from_scale, scales.buffer());
            if constexpr (j == 54) dy.advance(step_b);
            if constexpr (j == 60) codes.advance(step_code);
            if constexpr (j == 61) scales.advance(step_scale);
            if constexpr (j >= 12 && j < 12 + 4 * kSums && j % 4 == 0)
                fb[(j - 12) / 4] = fragment(at_sum[(j - 12) / 4] + Q % C::b_ring * C::b_bytes, 512);
            if constexpr (j >= 44 && j < 44 + 4 * kSums && j % 4 == 0)
                Op<D>::multiply_v(sum[(j - 44) / 4], ones, fb[(j - 44) / 4]);
        });
        __builtin_amdgcn_s_waitcnt(0x0F70 | 14);   // all loads but the last two phases'
        __syncthreads();
        __builtin_amdgcn_sched_barrier(0);
    };

    // before the first phase: dy of phases 0 .. 3, codes of 0 .. 4, and those of 0 and 1 decoded
    each(std::make_integer_sequence<int, 5>{}, [&](auto at) {
        constexpr int p = decltype(at)::value;
        if constexpr (p < 4) {
            each(std::make_integer_sequence<int, C::b_loads>{}, [&](auto i) {
                constexpr int j = decltype(i)::value;
                load16<p * C::b_bytes + j * 1024>(to_b, from_b[j], dy.buffer());
            });
            dy.advance(step_b);
        }
        load16<p * C::code_bytes>(to_code, from_code[0], codes.buffer());
        load16<p * C::code_bytes + 1024>(to_code, from_code[1], codes.buffer());
        load1<p * C::scale_bytes>(to_scale, from_scale, scales.buffer());
        codes.advance(step_code);
        scales.advance(step_scale);
    });
    __builtin_amdgcn_s_waitcnt(0x0F70);
    __syncthreads();
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) place_codes(decode<D>(raw(j, h, p), raw_scale(j, p), top), j, h, p);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; ++i) read(f0, i, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
    for (int p = 0; p < phases; p += C::turn) {   // phases behind the last multiply zeros
        each(std::make_integer_sequence<int, C::turn>{}, [&](auto turn) __attribute__((always_inline)) {
            if constexpr (decltype(turn)::value % 2 == 0) phase(turn, f0, f1);
            else phase(turn, f1, f0);
        });
        if (p + C::turn >= phases) asm volatile("s_nop 15\n\ts_nop 15");   // the last products are written before anything reads them
        __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);   // no load comes into what follows
    finish<C, Op<D>::kScaled>(a, part, lds, acc, power);
#pragma unroll
    for (int i = 0; i < kSums; ++i)
        if (share < C::NI) finish_bias<C::W>(a, part, (wn * 8 + first + i) * 16, sum[i][0]);
}

// Adds up the splits' sums of a tile, in order: four neighbouring elements a thread.
constexpr int kJoinThreads = 256;
constexpr int join_blocks(int w) { return w * w / 4 / kJoinThreads; }   // of a tile
template <int DO, int W>
__global__ __launch_bounds__(kJoinThreads) void split_join_kernel(const GemmArgs a) {
    typedef Four<DO> F;
    typedef typename F::E E;
    constexpr int blocks = join_blocks(W);
    const uint32_t i = blockIdx.x / blocks, x = (blockIdx.x % blocks) * kJoinThreads + threadIdx.x;
    const uint32_t tile = uint32_t(a.whole) + i;
    const uint32_t group = tile / (kGroup * a.tiles_k), rest = tile - group * (kGroup * a.tiles_k);
    const uint32_t wide = a.tiles_n - group * kGroup < kGroup ? a.tiles_n - group * kGroup : kGroup, tile_k = rest / wide;
    const int64_t k0 = int64_t(tile_k) * W, n0 = int64_t(group * kGroup + rest - tile_k * wide) * W;
    const float* part = a.part + int64_t(i) * a.splits * part_size(W);
    const int64_t rows = a.w.transposed ? a.w.k : a.w.n, cols = a.w.transposed ? a.w.n : a.w.k;
    const int64_t r = (a.w.transposed ? k0 : n0) + x / (W / 4), c = (a.w.transposed ? n0 : k0) + x % (W / 4) * 4;
    if (r < rows && c < cols) {
        f32x4 v = *(Global<const f32x4>*)(part + 4 * x);
#pragma unroll 8
        for (int s = 1; s < a.splits; ++s) v += *(Global<const f32x4>*)(part + s * part_size(W) + 4 * x);
        Global<E>* p = (Global<E>*)a.w.dw + r * a.w.s_dw + c;
        if (c + 4 <= cols) {
            typename F::vec y = {};
            if (a.w.accumulate) y = *(Global<typename F::at>*)p;
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = F::narrow(a.w.accumulate ? F::wide(y[j]) + v[j] : v[j]);
            *(Global<typename F::at>*)p = y;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + j < cols) p[j] = F::narrow(a.w.accumulate ? F::wide(p[j]) + v[j] : v[j]);
        }
    }
    if (a.w.bias && blockIdx.x % blocks == 0 && threadIdx.x < W && n0 + threadIdx.x < a.w.n) {
        const uint32_t fragment = threadIdx.x / 16 % 8;
        if (tile_k != (a.shares ? fragment / uint32_t(2 * a.shares) : 0)) return;
        float v = ((Global<const float>*)part)[W * W + threadIdx.x];
        for (int s = 1; s < a.splits; ++s) v += ((Global<const float>*)part)[s * part_size(W) + W * W + threadIdx.x];
        put_bias<DO>(a, n0 + threadIdx.x, v);
    }
}

// How a product is cut: into tiles of 256 x 256 outputs, one of which runs on a CU at a
// time, or of 64 x 64, of which several do; and where tiles are few, or some of the large are
// left over after whole rounds of all CUs, these by tokens, another kernel adding the parts up.
// Sums are in an order that the sizes alone fix, so where dy starts plays no part: one that only
// the general kernel takes is cut as for the fast one, if not at its best.
// What is expected to take the least time is taken, by this model of one MI355X in us: a round
// of blocks takes `fixed` and `step` for kUnit tokens (small ones overlap, so their rounds
// need not be whole, and `first` is what the first costs more), the other kernel 5 and its
// bytes at 4.5 TB/s.
//   bf16, large / small tiles      77 x 200 x 136: 15.5 / under 10.6, 1024 x 1024 x 1024: 26.4 / 12.5,
//       1024 x 2048 x 2048: 33 / 21, 4096 x 1024 x 1024: 35 / 32, 16384 x 1024 x 1024: 52 / 85
//   13B matrix, 1600 large tiles   1443 in seven rounds, 1364 with the last 64 tiles split
constexpr int kCUs = 256;
struct Cut {
    int32_t tile, tiles_k, tiles_n, whole, splits;
    int64_t per_split;
    double cost;
    int64_t blocks() const { return whole + (int64_t(tiles_k) * tiles_n - whole) * splits; }
    int64_t bytes() const { return splits > 1 ? (int64_t(tiles_k) * tiles_n - whole) * splits * part_size(tile) * 4 : 0; }
};
struct Times {
    int32_t tile, at_once;   // blocks that run on a CU at a time
    double first, fixed, step;
};
Cut cut_into(const Times& x, int64_t T, int64_t n, int64_t k) {
    const double part = part_size(x.tile) * 4 / 4.5e6;
    const int64_t slots = int64_t(kCUs) * x.at_once;
    const auto rounds = [&](int64_t blocks) {
        if (x.at_once == 1) return double((blocks + slots - 1) / slots);
        return blocks > slots ? double(blocks) / double(slots) : 1.0;
    };
    Cut c;
    c.tile = x.tile;
    c.tiles_k = k > 0 ? int32_t((k + x.tile - 1) / x.tile) : 1;   // the bias needs a tile
    c.tiles_n = int32_t((n + x.tile - 1) / x.tile);
    const int64_t tiles = int64_t(c.tiles_k) * c.tiles_n, units = (T + kUnit - 1) / kUnit;
    c.whole = int32_t(tiles);
    c.splits = 1;
    c.per_split = units * kUnit;
    c.cost = x.first + rounds(tiles) * (x.fixed + x.step * double(units));
    const int64_t rest = x.at_once == 1 ? tiles % slots : tiles;
    if (rest == 0) return c;
    const double before = x.first + double((tiles - rest) / slots) * (x.fixed + x.step * double(units));
    // at most 2 rounds of blocks, of 4 units at least
    for (int64_t s = 2; s <= 64 && rest * s <= 2 * slots && 4 * s <= units; ++s) {
        int64_t per = (units + s - 1) / s;
        per = (per + 4) / 5 * 5;   // the fast kernel goes by 5 of them
        const int64_t used = (units + per - 1) / per;
        if (used < 2) continue;
        const double cost = before + rounds(rest * used) * (x.fixed + x.step * double(per)) + 5 + double(rest * used) * part;
        if (cost < c.cost) {
            c.cost = cost;
            c.whole = int32_t(tiles - rest);
            c.splits = int32_t(used);
            c.per_split = per * kUnit;
        }
    }
    return c;
}
Cut cut_for(int64_t T, int64_t n, int64_t k, int32_t dy_type) {
    const bool few = T <= 3 * kUnit;   // not for the fast kernel
    Cut large, small;
    if (dy_type == ZERO_DTYPE_FP32) {
        large = cut_into({kTile, 1, 0, 10, 5}, T, n, k);
        small = cut_into({kSmall, 2, 4, 0.8, 1.8}, T, n, k);
    } else if (dy_type == ZERO_DTYPE_FP16) {
        large = cut_into(few ? Times{kTile, 1, 0, 13, 2.6} : Times{kTile, 1, 0, 16, 1.6}, T, n, k);
        small = cut_into({kSmall, 3, 4, 3.5, 0.87}, T, n, k);
    } else {
        large = cut_into(few ? Times{kTile, 1, 0, 7.5, 2.6} : Times{kTile, 1, 0, 10, 1.5}, T, n, k);
        small = cut_into({kSmall, 3, 4, 0.7, 0.85}, T, n, k);
    }
    const bool fits = small.blocks() < int64_t(1) << 23;   // threads of a launch, in 32 bits
    return fits && small.cost < large.cost ? small : large;
}

// Whether the loads of the fast kernel reach everything: 16 bytes of dy at a time,
// whole words up to the last value, dy's bytes of a block's `tokens` in 32 bits and
// the codes' in 31 (the highest one marks what is behind a row);
// and whether there are tokens enough for a turn of its loop.
bool fast(const WeightGradLaunch& w, int64_t tokens) {
    constexpr int64_t most = int64_t(1) << 31;
    return tokens > 3 * kUnit && tokens < most && reinterpret_cast<uintptr_t>(w.dy) % 16 == 0 && w.s_dy % 8 == 0 && w.s_dy >= w.n &&
           w.n % 2 == 0 && w.s_dy < most / 64 && tokens * w.s_dy < most && w.k < most / 64 && tokens * (w.k + 32) < most;
}

template <int D>
void run_fast(const GemmArgs& a, dim3 blocks, hipStream_t s, const KernelEvents& ev) {
    switch (a.shares) {
        case 0: launch(weight_grad_fast_kernel<D, 0>, blocks, Fast::threads, s, ev, a); break;
        case 1: launch(weight_grad_fast_kernel<D, 1>, blocks, Fast::threads, s, ev, a); break;
        case 2: launch(weight_grad_fast_kernel<D, 2>, blocks, Fast::threads, s, ev, a); break;
        default: launch(weight_grad_fast_kernel<D, 4>, blocks, Fast::threads, s, ev, a); break;
    }
}

template <int W>
void join(const GemmArgs& a, hipStream_t s, const KernelEvents& ev) {
    const dim3 grid(uint32_t((int64_t(a.tiles_k) * a.tiles_n - a.whole) * join_blocks(W)));
    if (a.w.out_type == ZERO_DTYPE_FP16) launch(split_join_kernel<ZERO_DTYPE_FP16, W>, grid, kJoinThreads, s, ev, a);
    else if (a.w.out_type == ZERO_DTYPE_BF16) launch(split_join_kernel<ZERO_DTYPE_BF16, W>, grid, kJoinThreads, s, ev, a);
    else launch(split_join_kernel<ZERO_DTYPE_FP32, W>, grid, kJoinThreads, s, ev, a);
}

template <int D>
hipError_t run(const WeightGradLaunch& w, hipStream_t s, const KernelEvents& ev) {
    const Cut c = cut_for(w.T, w.n, w.k, D);
    GemmArgs a = {};
    a.w = w;
    a.blocks = (w.k + 31) / 32;
    a.pitch = 32 * a.blocks;
    a.tiles_k = c.tiles_k;
    a.tiles_n = c.tiles_n;
    a.whole = c.whole;
    a.splits = c.splits;
    a.per_split = c.per_split;
    a.part = w.work;
    KernelEvents one = {ev.start, c.splits > 1 ? nullptr : ev.stop};
    const dim3 blocks{uint32_t(c.blocks())};
    typedef Config<D, D == ZERO_DTYPE_FP32 ? 32 : 64, kTile> Large;
    typedef Config<D, 64, kSmall> Small;
    if (c.tile == kSmall) {
        launch(weight_grad_kernel<Small>, blocks, Small::threads, s, one, a);
    } else if (D != ZERO_DTYPE_FP32 && fast(w, c.whole > 0 ? w.T : c.per_split)) {
        a.shares = !w.bias ? 0 : c.tiles_k >= 4 ? 1 : c.tiles_k >= 2 ? 2 : 4;
        if constexpr (D != ZERO_DTYPE_FP32) run_fast<D>(a, blocks, s, one);
    } else {
        launch(weight_grad_kernel<Large>, blocks, Large::threads, s, one, a);
    }
    if (c.splits > 1) {
        one = {nullptr, ev.stop};
        if (c.tile == kSmall) join<kSmall>(a, s, one);
        else join<kTile>(a, s, one);
    }
    return hipGetLastError();
}

}  // namespace

int64_t weight_grad_work(int64_t T, int64_t n, int64_t k, int32_t dy_type) { return cut_for(T, n, k, dy_type).bytes(); }

hipError_t launch_weight_grad(const WeightGradLaunch& w, hipStream_t s, const KernelEvents& ev) {
    if (w.dy_type == ZERO_DTYPE_BF16) return run<ZERO_DTYPE_BF16>(w, s, ev);
    if (w.dy_type == ZERO_DTYPE_FP16) return run<ZERO_DTYPE_FP16>(w, s, ev);
    return run<ZERO_DTYPE_FP32>(w, s, ev);
}

}  // namespace zp
