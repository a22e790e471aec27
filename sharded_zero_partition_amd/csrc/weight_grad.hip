// weight_grad.hip -- weight and bias gradient of a linear layer from the 8-bit
// checkpoint of its input (gfx950):
//   dw[n, k] = sum_t dy[t, n] x[t, k]        bias[n] = sum_t dy[t, n]
#include <type_traits>

#include "octets.hpp"
#include "timed_launch.hpp"

#pragma clang fp contract(off)

namespace zp {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <typename T>
using Shared = __attribute__((address_space(3))) T;

// Bytes of LDS per row of a tile, and where pair q (16 columns) of row t is: the
// 16 lanes of a transposing read take 32 bytes of each of 4 rows, and the wave
// those of 16 rows.  Exchanging the pairs by the row's lowest bits spreads them
// over all banks.
template <int W>
__device__ __forceinline__ uint32_t pair_at(int t, int q) {
    return uint32_t(t * (W * 2) + ((q ^ (t & 7)) << 5));
}

// A dy value as the sum of bf16 numbers, exactly: 1 for bf16, 2 for fp16 (11
// bits), 3 for fp32 (24 bits).
constexpr int parts_of(int d) { return d == ZERO_DTYPE_BF16 ? 1 : d == ZERO_DTYPE_FP16 ? 2 : 3; }

template <int D_, int BN_, int WM_, int WN_, int STEP_>
struct Config {
    static constexpr int D = D_, BM = 256, BN = BN_, WM = WM_, WN = WN_, STEP = STEP_;
    static constexpr int P = parts_of(D);
    static constexpr int threads = 64 * WM * WN;
    static constexpr int MI = BM / WM / 16, NI = BN / WN / 16;
    static constexpr int a_chunks = STEP * BM / 16 / threads;   // of 16 values, a thread's
    static constexpr int b_chunks = STEP * BN / 16 / threads;
    static constexpr int a_bytes = STEP * BM * 2, b_bytes = STEP * BN * 2;
    static constexpr int stage = a_bytes + P * b_bytes;
    static_assert(a_chunks * threads * 16 == STEP * BM && b_chunks * threads * 16 == STEP * BN, "loads");
    static_assert(2 * stage <= 160 * 1024, "LDS");
};

struct GemmArgs {
    WeightGradLaunch w;
    int64_t pitch;       // of the codes
    int64_t blocks;      // scale bytes of a row
    int32_t tiles_k, tiles_n, splits;
    int64_t per_split;   // steps
    float* part;         // splits > 1: [splits][n][k], or [splits][k][n] transposed, rows of ld_part
    float* part_bias;    // [splits][n]
    int64_t ld_part, part_size;
};

// 16 values of dy.
template <int D>
struct Chunk {
    Octet<D> o[2];
    __device__ __forceinline__ void load(const char* p, int64_t left) {
        o[0] = load_octet<D>(p, left);
        o[1] = load_octet<D>(p + sizeof(typename Type<D>::elem) * 8, left - 8);
    }
    // part j of the values, as bf16 pairs
    __device__ __forceinline__ void split(u32x4 to[parts_of(D)][2]) const {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (D == ZERO_DTYPE_BF16) {
                    to[0][h][i] = uint32_t(o[h].v[2 * i]) | uint32_t(o[h].v[2 * i + 1]) << 16;
                } else {
                    float a = o[h].get(2 * i), b = o[h].get(2 * i + 1);
#pragma unroll
                    for (int j = 0; j < parts_of(D); ++j) {
                        const uint32_t ua = bits(a) & 0xFFFF0000u, ub = bits(b) & 0xFFFF0000u;
                        to[j][h][i] = ua >> 16 | ub;
                        a -= number(ua);
                        b -= number(ub);
                    }
                }
            }
    }
};

// 16 codes and their scale.
struct Codes {
    u32x4 code;
    uint32_t scale;
    // as bf16 pairs, exactly: an e4m3 number has 4 bits
    __device__ __forceinline__ void decode(u32x4 to[2]) const {
        const float f = number(scale << 23);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            to[w >> 1][(2 * w) & 3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(code[w], f, false));
            to[w >> 1][(2 * w + 1) & 3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(code[w], f, true));
        }
    }
};

// A fragment of 16 columns by 32 rows: the lane has column lane & 15 of rows
// 4 (lane / 16) + 0 .. 3 and 16 more.  (Which of the 32 rows come where does not
// matter as long as both operands have the same.)
__device__ __forceinline__ bf16x8 fragment(uint32_t at, int row_bytes) {
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Shared<s16x4>*)uintptr_t(at));
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Shared<s16x4>*)uintptr_t(at + 16 * row_bytes));
    const s16x8 v = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    return __builtin_bit_cast(bf16x8, v);
}

template <int DO>
__device__ __forceinline__ void put(const GemmArgs& a, int64_t n, int64_t k, f32x4 v) {
    typedef typename Type<DO>::elem E;
    if (n >= a.w.n) return;
    E* p = static_cast<E*>(a.w.dw);
    const int64_t step = a.w.transposed ? a.w.s_dw : 1;
    p += a.w.transposed ? k * a.w.s_dw + n : n * a.w.s_dw + k;
    float old[4] = {};
    if (a.w.accumulate)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (k + i < a.w.k) {
                const E e = ((Global<const E>*)p)[i * step];
                if constexpr (DO == ZERO_DTYPE_FP32) old[i] = e;
                else old[i] = Type<DO>::wide(e);
            }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (k + i < a.w.k) {
            const float x = old[i] + v[i];
            if constexpr (DO == ZERO_DTYPE_FP32) ((Global<E>*)p)[i * step] = x;
            else ((Global<E>*)p)[i * step] = Type<DO>::narrow(x);
        }
}

template <int DO>
__device__ __forceinline__ void put_bias(const GemmArgs& a, int64_t n, float v) {
    typedef typename Type<DO>::elem E;
    Global<E>* p = (Global<E>*)a.w.bias + n;
    if constexpr (DO == ZERO_DTYPE_FP32) *p = a.w.accumulate ? *p + v : v;
    else *p = Type<DO>::narrow(a.w.accumulate ? Type<DO>::wide(*p) + v : v);
}

template <typename C>
__global__ __launch_bounds__(C::threads) void weight_grad_kernel(const GemmArgs a) {
    constexpr int D = C::D, P = C::P;
    __shared__ __attribute__((aligned(1024))) char lds[2 * C::stage];
    const int tid = int(threadIdx.x), lane = tid & 63, wave = tid >> 6;
    const int wm = wave / C::WN, wn = wave % C::WN;

    // neighbouring tiles on one XCD (blocks go round the 8 of them)
    const uint32_t total = gridDim.x, id = blockIdx.x, xcd = id & 7, q8 = total >> 3, r8 = total & 7;
    uint32_t tile = xcd * q8 + (xcd < r8 ? xcd : r8) + (id >> 3);
    const uint32_t tiles = uint32_t(a.tiles_k) * uint32_t(a.tiles_n);
    const uint32_t split = tile / tiles;
    tile -= split * tiles;
    const int64_t k0 = int64_t(tile % a.tiles_k) * C::BM, n0 = int64_t(tile / a.tiles_k) * C::BN;
    const int64_t t_begin = int64_t(split) * a.per_split * C::STEP;
    const int64_t t_end = t_begin + a.per_split * C::STEP < a.w.T ? t_begin + a.per_split * C::STEP : a.w.T;

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
            u32x4 v[2];
            ra[j].decode(v);
            to[0] = v[0];
            to[1] = v[1];
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
    bf16x8 ones;
#pragma unroll
    for (int i = 0; i < 8; ++i) ones[i] = __bf16(1.0f);

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
            bf16x8 fa[C::MI], fb[C::NI];
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
                        acc[m][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[m], fb[i], acc[m][i], 0, 0, 0);
                if (bias)
#pragma unroll
                    for (int i = 0; i < C::NI; ++i)
                        sum[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, fb[i], sum[i], 0, 0, 0);
            }
        }
        if (s + 1 < steps) stash((s + 1) & 1);
        __syncthreads();
    }

    const int64_t k_lane = k0 + wm * (C::MI * 16) + 4 * (lane >> 4), n_lane = n0 + wn * (C::NI * 16) + (lane & 15);
    if (a.splits > 1) {
        float* part = a.part + split * a.part_size;
#pragma unroll
        for (int i = 0; i < C::NI; ++i)
#pragma unroll
            for (int m = 0; m < C::MI; ++m) {
                const int64_t n = n_lane + 16 * i, k = k_lane + 16 * m;
                if (n >= a.w.n) continue;
                if (!a.w.transposed) {
                    if (k < a.w.k) *(Global<f32x4>*)(part + n * a.ld_part + k) = acc[m][i];   // rows padded to 4
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (k + j < a.w.k) ((Global<float>*)part)[(k + j) * a.ld_part + n] = acc[m][i][j];
                }
            }
        if (bias && lane < 16)
#pragma unroll
            for (int i = 0; i < C::NI; ++i)
                if (n_lane + 16 * i < a.w.n) ((Global<float>*)a.part_bias)[split * a.w.n + n_lane + 16 * i] = sum[i][0];
        return;
    }
    const auto write = [&](auto d) {
        constexpr int DO = decltype(d)::value;
#pragma unroll
        for (int i = 0; i < C::NI; ++i)
#pragma unroll
            for (int m = 0; m < C::MI; ++m) put<DO>(a, n_lane + 16 * i, k_lane + 16 * m, acc[m][i]);
        if (bias && lane < 16)
#pragma unroll
            for (int i = 0; i < C::NI; ++i)
                if (n_lane + 16 * i < a.w.n) put_bias<DO>(a, n_lane + 16 * i, sum[i][0]);
    };
    if (a.w.out_type == ZERO_DTYPE_FP16) write(std::integral_constant<int, ZERO_DTYPE_FP16>{});
    else if (a.w.out_type == ZERO_DTYPE_BF16) write(std::integral_constant<int, ZERO_DTYPE_BF16>{});
    else write(std::integral_constant<int, ZERO_DTYPE_FP32>{});
}

// Adds up the splits' sums, in order: four neighbouring elements a thread.
constexpr int kJoinThreads = 256;
template <int DO>
__global__ __launch_bounds__(kJoinThreads) void split_join_kernel(const GemmArgs a) {
    typedef typename Type<DO>::elem E;
    const int64_t cols = a.w.transposed ? a.w.n : a.w.k, rows = a.w.transposed ? a.w.k : a.w.n;
    const int64_t fours = a.ld_part / 4, i = int64_t(blockIdx.x) * kJoinThreads + threadIdx.x;
    if (i < rows * fours) {
        const int64_t r = i / fours, c = (i - r * fours) * 4;
        f32x4 v = *(Global<const f32x4>*)(a.part + r * a.ld_part + c);
        for (int s = 1; s < a.splits; ++s) v += *(Global<const f32x4>*)(a.part + s * a.part_size + r * a.ld_part + c);
        Global<E>* p = (Global<E>*)a.w.dw + r * a.w.s_dw + c;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (c + j < cols) {
                if constexpr (DO == ZERO_DTYPE_FP32) p[j] = a.w.accumulate ? p[j] + v[j] : v[j];
                else p[j] = Type<DO>::narrow(a.w.accumulate ? Type<DO>::wide(p[j]) + v[j] : v[j]);
            }
    }
    if (a.w.bias && i < a.w.n) {
        float v = ((Global<const float>*)a.part_bias)[i];
        for (int s = 1; s < a.splits; ++s) v += ((Global<const float>*)a.part_bias)[s * a.w.n + i];
        put_bias<DO>(a, i, v);
    }
}

// How a product is cut: tiles of 256 by `bn` outputs, and splits of the tokens
// where there are fewer tiles than CUs.
constexpr int kCUs = 256;
struct Cut {
    int32_t tiles_k, tiles_n, splits;
    int64_t per_split, ld_part, part_size, bytes;
};
Cut cut_for(int64_t T, int64_t n, int64_t k, int bn, int step) {
    Cut c;
    c.tiles_k = k > 0 ? int32_t((k + 255) / 256) : 1;   // the bias needs a tile
    c.tiles_n = int32_t((n + bn - 1) / bn);
    const int64_t tiles = int64_t(c.tiles_k) * c.tiles_n, steps = (T + step - 1) / step;
    int64_t best = 1, best_cost = -1;
    for (int64_t s = 1; s <= 64 && (s == 1 || (s <= steps / 4 && tiles * s <= 2 * kCUs)); ++s) {
        const int64_t per = (steps + s - 1) / s;
        const int64_t cost = ((tiles * s + kCUs - 1) / kCUs) * (per + 4) * 100 + (s > 1 ? 800 + 20 * s : 0);
        if (best_cost < 0 || cost < best_cost) {
            best = s;
            best_cost = cost;
        }
    }
    c.per_split = steps > 0 ? (steps + best - 1) / best : 0;
    c.splits = steps > 0 ? int32_t((steps + c.per_split - 1) / c.per_split) : 1;
    c.ld_part = 0;
    c.part_size = c.bytes = 0;
    if (c.splits > 1) {
        // either way round
        const int64_t a = n * ((k + 3) / 4 * 4), b = k * ((n + 3) / 4 * 4);
        c.part_size = a > b ? a : b;
        c.bytes = 4 * c.splits * (c.part_size + n);
    }
    return c;
}

template <typename C>
hipError_t run(const WeightGradLaunch& w, hipStream_t s, const KernelEvents& ev) {
    const Cut c = cut_for(w.T, w.n, w.k, C::BN, C::STEP);
    GemmArgs a = {};
    a.w = w;
    a.blocks = (w.k + 31) / 32;
    a.pitch = 32 * a.blocks;
    a.tiles_k = c.tiles_k;
    a.tiles_n = c.tiles_n;
    a.splits = c.splits;
    a.per_split = c.per_split;
    a.part_size = c.part_size;
    a.ld_part = ((w.transposed ? w.n : w.k) + 3) / 4 * 4;
    a.part = w.work;
    a.part_bias = c.splits > 1 ? w.work + c.splits * c.part_size : nullptr;
    KernelEvents one = {ev.start, c.splits > 1 ? nullptr : ev.stop};
    launch(weight_grad_kernel<C>, dim3(uint32_t(int64_t(c.tiles_k) * c.tiles_n * c.splits)), C::threads, s, one, a);
    if (c.splits > 1) {
        one = {nullptr, ev.stop};
        const int64_t rows = w.transposed ? w.k : w.n;
        int64_t items = rows * (a.ld_part / 4);
        if (w.bias && items < w.n) items = w.n;
        const dim3 grid(uint32_t((items + kJoinThreads - 1) / kJoinThreads));
        if (w.out_type == ZERO_DTYPE_FP16) launch(split_join_kernel<ZERO_DTYPE_FP16>, grid, kJoinThreads, s, one, a);
        else if (w.out_type == ZERO_DTYPE_BF16) launch(split_join_kernel<ZERO_DTYPE_BF16>, grid, kJoinThreads, s, one, a);
        else launch(split_join_kernel<ZERO_DTYPE_FP32>, grid, kJoinThreads, s, one, a);
    }
    return hipGetLastError();
}

typedef Config<ZERO_DTYPE_BF16, 256, 2, 4, 64> Bf16;
typedef Config<ZERO_DTYPE_FP16, 128, 4, 2, 64> Fp16;
typedef Config<ZERO_DTYPE_FP32, 256, 2, 4, 32> Fp32;

}  // namespace

int64_t weight_grad_work(int64_t T, int64_t n, int64_t k, int32_t dy_type) {
    if (dy_type == ZERO_DTYPE_BF16) return cut_for(T, n, k, Bf16::BN, Bf16::STEP).bytes;
    if (dy_type == ZERO_DTYPE_FP16) return cut_for(T, n, k, Fp16::BN, Fp16::STEP).bytes;
    return cut_for(T, n, k, Fp32::BN, Fp32::STEP).bytes;
}

hipError_t launch_weight_grad(const WeightGradLaunch& w, hipStream_t s, const KernelEvents& ev) {
    if (w.dy_type == ZERO_DTYPE_BF16) return run<Bf16>(w, s, ev);
    if (w.dy_type == ZERO_DTYPE_FP16) return run<Fp16>(w, s, ev);
    return run<Fp32>(w, s, ev);
}

}  // namespace zp
