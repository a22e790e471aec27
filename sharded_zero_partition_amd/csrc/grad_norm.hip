// grad_norm.hip -- sum of squares of every gradient value of a tensor set, in
// fp64 (gfx950).
//
// Every value is widened to fp64 before it is squared: an fp16 or bf16 square
// is exact there, no square of an fp32 overflows, and a sum over 10^10 values
// keeps 5 digits more than fp32 has.  The tiles are dealt to blocks in a fixed
// way and the blocks' sums added in a fixed order, so equal inputs give equal
// bits; there are no atomics.
#include <hip/hip_ext.h>

#include "tensor_set.hpp"

namespace zp {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int64_t kMaxBlocks = 2048;   // 8 blocks of 4 waves on each of 256 CUs

typedef float f32x4 __attribute__((ext_vector_type(4)));
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
__device__ __forceinline__ double block_sum(double x) {
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

template <int D>
__global__ __launch_bounds__(kThreads) void sumsq_kernel(const SetLaunch a, double* sumsq, bool accumulate, double* work) {
    typedef Grad<D> T;
    const int lane = threadIdx.x & 63;
    double s = 0.0;
    for (int64_t w = int64_t(blockIdx.x) * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); w < a.n_tiles;
         w += int64_t(gridDim.x) * kWaves) {
        const TileRec tile = a.tile[w];
        const TensorRec& r = a.rec[tile.tensor];
        const int64_t base = int64_t(tile.tile) * kSetTile - tile_shift(r.grad, int(sizeof(typename T::elem)), r.spare);
        const auto* g = (Global<const typename T::elem>*)r.grad + base;
        const int64_t left = r.numel - base;
        if (base >= 0 && left >= kSetTile) {
            typename T::at x[T::kLoads];
#pragma unroll
            for (int h = 0; h < T::kLoads; ++h) x[h] = *(Global<const typename T::at>*)(g + (h * 64 + lane) * T::kWide);
#pragma unroll
            for (int h = 0; h < T::kLoads; ++h)
#pragma unroll
                for (int k = 0; k < T::kWide; ++k) {
                    const double y = T::wide(x[h][k]);
                    s += y * y;
                }
        } else {
            const int lo = base < 0 ? int(-base) : 0, hi = left < kSetTile ? int(left) : int(kSetTile);
#pragma unroll 4
            for (int e = lo + lane; e < hi; e += 64) {
                const double y = T::wide(g[e]);
                s += y * y;
            }
        }
    }
    s = block_sum(s);
    if (threadIdx.x != 0) return;
    if (gridDim.x == 1) put(sumsq, s, accumulate);
    else work[blockIdx.x] = s;
}

__global__ __launch_bounds__(kThreads) void sumsq_join_kernel(const double* work, int n, double* sumsq, bool accumulate) {
    double s = 0.0;
    for (int k = threadIdx.x; k < n; k += kThreads) s += work[k];
    s = block_sum(s);
    if (threadIdx.x == 0) put(sumsq, s, accumulate);
}

}  // namespace

int64_t sumsq_blocks(int64_t n_tiles) {
    const int64_t b = (n_tiles + kWaves - 1) / kWaves;
    return b < 1 ? 1 : b < kMaxBlocks ? b : kMaxBlocks;
}

hipError_t launch_sumsq(const SetLaunch& a, double* sumsq, bool accumulate, double* work, hipStream_t stream,
                        const KernelEvents& ev) {
    const int blocks = int(sumsq_blocks(a.n_tiles));
    const hipEvent_t stop = blocks == 1 ? ev.stop : nullptr;
    const auto pass = [&](auto kernel) {
        if (ev.start) hipExtLaunchKernelGGL(kernel, dim3(blocks), dim3(kThreads), 0, stream, ev.start, stop, 0, a, sumsq, accumulate, work);
        else hipLaunchKernelGGL(kernel, dim3(blocks), dim3(kThreads), 0, stream, a, sumsq, accumulate, work);
    };
    switch (a.grad_type) {
        case ZERO_DTYPE_FP16: pass(sumsq_kernel<ZERO_DTYPE_FP16>); break;
        case ZERO_DTYPE_BF16: pass(sumsq_kernel<ZERO_DTYPE_BF16>); break;
        default: pass(sumsq_kernel<ZERO_DTYPE_FP32>); break;
    }
    if (blocks > 1) {
        if (ev.stop) hipExtLaunchKernelGGL(sumsq_join_kernel, dim3(1), dim3(kThreads), 0, stream, nullptr, ev.stop, 0, work, blocks, sumsq, accumulate);
        else hipLaunchKernelGGL(sumsq_join_kernel, dim3(1), dim3(kThreads), 0, stream, work, blocks, sumsq, accumulate);
    }
    return hipGetLastError();
}

}  // namespace zp
