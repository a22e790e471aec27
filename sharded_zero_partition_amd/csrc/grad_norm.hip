// grad_norm.hip -- sum of squares of every gradient value of a tensor set, in
// fp64 (gfx950).
//
// Every value is widened to fp64 before it is squared: an fp16 or bf16 square
// is exact there, no square of an fp32 overflows, and a sum over 10^10 values
// keeps 5 digits more than fp32 has.  A tensor's tiles start with it, an element
// goes to a lane by its number in the tensor, the tiles are dealt to blocks in a
// fixed way and the blocks' sums added in a fixed order: equal values in tensors
// of equal sizes give equal bits, wherever the tensors are.  There are no
// atomics.
//
// Bound by reading 2 or 4 bytes an element: 69 to 72 us for 200 M bf16 values
// (5.7 TB/s, a plain copy reaches 6.05), on 128-byte lines or off them.
// Non-temporal loads take 68, but the step
// that follows then finds nothing of the gradients in the last-level cache: norm
// and step together, 355 us with these loads and 385 with those (120 M elements,
// states in 8 bits).
#include "tensor_set.hpp"
#include "timed_launch.hpp"

namespace zp {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxBlocks = 1024;   // 4 blocks of 4 waves on each of 256 CUs (2048: 1 to 2% slower)
// Up to 64 tiles are summed by one block of 16 waves in one launch.  On the
// device the two ways meet there (replayed from a graph 2.6 us for 16 tiles,
// 4.4 for 64, 5.7 for 96; two launches 4.0 for any of them); called from a
// program, one launch takes 4.6 us where two take 8.6.
constexpr int kOneThreads = 1024;
constexpr int64_t kOneTiles = 64;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));

template <typename T>
using Global = __attribute__((address_space(1))) T;

template <int D>
struct Grad;
template <>
struct Grad<ZERO_DTYPE_FP16> {
    typedef uint16_t elem;
    typedef u16x8 at __attribute__((aligned(2)));
    static constexpr int kWide = 8, kLoads = int(kSetTile) / 512;
    static __device__ __forceinline__ double wide(uint16_t x) { return double(float(__builtin_bit_cast(_Float16, x))); }
};
template <>
struct Grad<ZERO_DTYPE_BF16> {
    typedef uint16_t elem;
    typedef u16x8 at __attribute__((aligned(2)));
    static constexpr int kWide = 8, kLoads = int(kSetTile) / 512;
    static __device__ __forceinline__ double wide(uint16_t x) { return double(__builtin_bit_cast(float, uint32_t(x) << 16)); }
};
template <>
struct Grad<ZERO_DTYPE_FP32> {
    typedef float elem;
    typedef f32x4 at __attribute__((aligned(4)));
    static constexpr int kWide = 4, kLoads = int(kSetTile) / 256;
    static __device__ __forceinline__ double wide(float x) { return double(x); }
};

// Sum over the block's threads, valid in thread 0.
template <int kBlock>
__device__ __forceinline__ double block_sum(double x) {
    constexpr int kWaves = kBlock / 64;
    __shared__ double part[kWaves];
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x += __shfl_down(x, d, 64);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
    __syncthreads();
    double s = 0.0;
    if (threadIdx.x == 0)
        for (int w = 0; w < kWaves; ++w) s += part[w];
    return s;
}

__device__ __forceinline__ void put(double* sumsq, double s, bool accumulate) { *sumsq = accumulate ? *sumsq + s : s; }

// A whole tile's vectors, element 8 (64 h + lane) on (4 for fp32) in x[h].
template <typename T>
__device__ __forceinline__ void load_tile(const Global<const typename T::elem>* g, int lane, typename T::at x[T::kLoads]) {
#pragma unroll
    for (int h = 0; h < T::kLoads; ++h) x[h] = *(Global<const typename T::at>*)(g + (h * 64 + lane) * T::kWide);
}

// The same for 16-bit values at an odd element, g[-1] being one of the tensor's:
// words from one value before on, so that loads are 4-byte aligned, and the
// eighth value from the next lane's.  (One tensor of 200 M bf16 values one
// element in: 77 us, and 88 by loads that are 2-byte aligned.)
template <typename T>
__device__ __forceinline__ void load_odd_tile(const Global<const typename T::elem>* g, int lane, typename T::at x[T::kLoads]) {
    typedef u32x4 at4 __attribute__((aligned(4)));
    u32x4 w[T::kLoads];
#pragma unroll
    for (int h = 0; h < T::kLoads; ++h) w[h] = *(Global<const at4>*)(g - 1 + (h * 64 + lane) * T::kWide);
    const uint32_t last = g[kSetTile - 1];
#pragma unroll
    for (int h = 0; h < T::kLoads; ++h) {
        const uint32_t after = h + 1 < T::kLoads ? uint32_t(__builtin_amdgcn_readfirstlane(int(w[h + 1].x))) : last;
        const uint32_t next = uint32_t(__shfl_down(int(w[h].x), 1, 64)), w4 = lane == 63 ? after : next;
        const u32x4 v = {__builtin_amdgcn_alignbit(w[h].y, w[h].x, 16), __builtin_amdgcn_alignbit(w[h].z, w[h].y, 16),
                         __builtin_amdgcn_alignbit(w[h].w, w[h].z, 16), __builtin_amdgcn_alignbit(w4, w[h].w, 16)};
        x[h] = __builtin_bit_cast(u16x8, v);
    }
}

template <int D, int kBlock>
__global__ __launch_bounds__(kBlock) void sumsq_kernel(const SetLaunch a, double* sumsq, bool accumulate, double* work) {
    typedef Grad<D> T;
    constexpr int kWaves = kBlock / 64;
    const int lane = threadIdx.x & 63;
    double s = 0.0;
    for (int64_t w = int64_t(blockIdx.x) * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); w < a.n_norm_tiles;
         w += int64_t(gridDim.x) * kWaves) {
        const TileRec tile = a.norm_tile[w];
        const TensorRec& r = a.rec[tile.tensor];
        const int64_t base = int64_t(tile.tile) * kSetTile;
        const auto* g = (Global<const typename T::elem>*)r.grad + base;
        const int64_t left = r.numel - base;   // > 0
        if (left >= kSetTile) {
            typename T::at x[T::kLoads];
            bool odd = false;
            if constexpr (sizeof(typename T::elem) == 2) {
                odd = (reinterpret_cast<uintptr_t>(r.grad) & 2u) != 0 && base > 0;
                if (odd) load_odd_tile<T>(g, lane, x);
            }
            if (!odd) load_tile<T>(g, lane, x);
#pragma unroll
            for (int h = 0; h < T::kLoads; ++h)
#pragma unroll
                for (int k = 0; k < T::kWide; ++k) {
                    const double y = T::wide(x[h][k]);
                    s += y * y;
                }
        } else {
            // groups of 64 vectors where the tensor has all of one, else of
            // single values, its last in the places of those it has not
            constexpr int kGroup = 64 * T::kWide;
            const int hi = int(left);
#pragma unroll
            for (int h = 0; h < T::kLoads; ++h) {
                const int first = h * kGroup;
                if (first >= hi) break;
                typename T::elem x[T::kWide] = {};
                bool has[T::kWide] = {};
                if (first + kGroup <= hi) {
                    const typename T::at v = *(Global<const typename T::at>*)(g + first + lane * T::kWide);
#pragma unroll
                    for (int k = 0; k < T::kWide; ++k) x[k] = v[k], has[k] = true;
                } else if (hi <= first + 64) {
                    const int e = first + lane;
                    has[0] = e < hi;
                    x[0] = g[e < hi ? e : hi - 1];
                } else {
#pragma unroll
                    for (int k = 0; k < T::kWide; ++k) {
                        const int e = first + k * 64 + lane;
                        has[k] = e < hi;
                        x[k] = g[e < hi ? e : hi - 1];
                    }
                }
#pragma unroll
                for (int k = 0; k < T::kWide; ++k) {
                    const double y = has[k] ? T::wide(x[k]) : 0.0;
                    s += y * y;
                }
            }
        }
    }
    s = block_sum<kBlock>(s);
    if (threadIdx.x != 0) return;
    if (gridDim.x == 1) put(sumsq, s, accumulate);
    else work[blockIdx.x] = s;
}

__global__ __launch_bounds__(kThreads) void sumsq_join_kernel(const double* work, int n, double* sumsq, bool accumulate) {
    double s = 0.0;
    for (int k = threadIdx.x; k < n; k += kThreads) s += work[k];
    s = block_sum<kThreads>(s);
    if (threadIdx.x == 0) put(sumsq, s, accumulate);
}

}  // namespace

int64_t sumsq_blocks(int64_t n_norm_tiles) {
    if (n_norm_tiles <= kOneTiles) return 1;
    const int64_t b = (n_norm_tiles + kThreads / 64 - 1) / (kThreads / 64);
    return b < kMaxBlocks ? b : kMaxBlocks;
}

namespace {

template <int D>
void run_sumsq(const SetLaunch& a, double* sumsq, bool accumulate, double* work, hipStream_t s, const KernelEvents& ev) {
    const int blocks = int(sumsq_blocks(a.n_norm_tiles));
    if (blocks == 1) {
        launch(sumsq_kernel<D, kOneThreads>, dim3(1), kOneThreads, s, ev, a, sumsq, accumulate, work);
        return;
    }
    KernelEvents first, last;
    first.start = ev.start;
    last.stop = ev.stop;
    launch(sumsq_kernel<D, kThreads>, dim3(blocks), kThreads, s, first, a, sumsq, accumulate, work);
    launch(sumsq_join_kernel, dim3(1), kThreads, s, last, (const double*)work, blocks, sumsq, accumulate);
}

}  // namespace

hipError_t launch_sumsq(const SetLaunch& a, double* sumsq, bool accumulate, double* work, hipStream_t stream,
                        const KernelEvents& ev) {
    switch (a.grad_type) {
        case ZERO_DTYPE_FP16: run_sumsq<ZERO_DTYPE_FP16>(a, sumsq, accumulate, work, stream, ev); break;
        case ZERO_DTYPE_BF16: run_sumsq<ZERO_DTYPE_BF16>(a, sumsq, accumulate, work, stream, ev); break;
        default: run_sumsq<ZERO_DTYPE_FP32>(a, sumsq, accumulate, work, stream, ev); break;
    }
    return hipGetLastError();
}

}  // namespace zp
