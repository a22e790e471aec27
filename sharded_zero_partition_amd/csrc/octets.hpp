// octets.hpp -- eight neighbouring values of a matrix's row, at any element's
// address (device translation units only).
#pragma once

#include "activations.hpp"
#include "mxfp8.hpp"

namespace zp {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <typename T>
using Global = __attribute__((address_space(1))) T;

// x / d.g for x < 2^31: m = magic is (2^(31 + l) + e) / g with 0 < e <= g <= 2^l,
// so x m / 2^(31 + l) is x / g and less than 1 / g more.
__device__ __forceinline__ uint32_t divide(uint32_t x, const Divisor& d) { return __umulhi(x, d.magic) >> d.shift; }

// x = q d.g + r for x < 2^52: the product is within 1 of the quotient.
__device__ __forceinline__ void divide(int64_t x, const Divisor& d, int64_t* q, uint32_t* r) {
    int64_t a = int64_t(double(x) * d.inv);
    int64_t b = x - a * int64_t(d.g);
    if (b < 0) { b += d.g; a -= 1; }
    if (b >= int64_t(d.g)) { b -= d.g; a += 1; }
    *q = a;
    *r = uint32_t(b);
}

// Eight values as they are in memory, at any element's address.  kPast: past the
// caches, which keep no such line for long.
template <int D>
struct Octet {   // 16-bit types
    typedef u16x8 at __attribute__((aligned(2)));
    u16x8 v;
    __device__ __forceinline__ void zero() { v = u16x8{}; }
    template <bool kPast>
    __device__ __forceinline__ void load(const void* p) {
        v = kPast ? __builtin_nontemporal_load((Global<const at>*)p) : *(Global<const at>*)p;
    }
    template <bool kPast>
    __device__ __forceinline__ void store(void* p) const {
        if (kPast) __builtin_nontemporal_store(v, (Global<at>*)p);
        else *(Global<at>*)p = v;
    }
    __device__ __forceinline__ float get(int i) const { return Type<D>::wide(v[i]); }
    __device__ __forceinline__ void set(int i, float x) { v[i] = Type<D>::narrow(x); }
};
template <>
struct Octet<ZERO_DTYPE_FP32> {
    typedef f32x4 at __attribute__((aligned(4)));
    f32x4 v[2];
    __device__ __forceinline__ void zero() { v[0] = v[1] = f32x4{}; }
    template <bool kPast>
    __device__ __forceinline__ void load(const void* p) {
#pragma unroll
        for (int h = 0; h < 2; ++h) v[h] = kPast ? __builtin_nontemporal_load((Global<const at>*)p + h) : ((Global<const at>*)p)[h];
    }
    template <bool kPast>
    __device__ __forceinline__ void store(void* p) const {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (kPast) __builtin_nontemporal_store(v[h], (Global<at>*)p + h);
            else ((Global<at>*)p)[h] = v[h];
    }
    __device__ __forceinline__ float get(int i) const { return v[i >> 2][i & 3]; }
    __device__ __forceinline__ void set(int i, float x) { v[i >> 2][i & 3] = x; }
};

// The octet at p of which `n` values exist (8 or more: all; 0 or less: none);
// the others are zero.
template <int D, bool kPast = false>
__device__ __forceinline__ Octet<D> load_octet(const void* p, int64_t n) {
    typedef typename Type<D>::elem E;
    Octet<D> x;
    if (n >= kOctet) {
        x.template load<kPast>(p);
        return x;
    }
    x.zero();
#pragma unroll
    for (int i = 0; i < kOctet; ++i)
        if (i < n) {
            const E e = ((Global<const E>*)p)[i];
            if constexpr (D == ZERO_DTYPE_FP32) x.set(i, e);
            else x.v[i] = e;
        }
    return x;
}
template <int D, bool kPast = false>
__device__ __forceinline__ void store_octet(void* p, int64_t n, const Octet<D>& x) {
    typedef typename Type<D>::elem E;
    if (n >= kOctet) {
        x.template store<kPast>(p);
        return;
    }
#pragma unroll
    for (int i = 0; i < kOctet; ++i)
        if (i < n) {
            if constexpr (D == ZERO_DTYPE_FP32) ((Global<E>*)p)[i] = x.get(i);
            else ((Global<E>*)p)[i] = x.v[i];
        }
}

// Another lane's value (DPP control).
template <int kCtrl>
__device__ __forceinline__ uint32_t across(uint32_t x) {
    return uint32_t(__builtin_amdgcn_update_dpp(0, int(x), kCtrl, 0xF, 0xF, true));
}

// Where the value at (row, col) of a matrix is.
template <int D>
__device__ __forceinline__ char* place(const void* p, int64_t row, int64_t stride, int64_t col) {
    return (char*)p + (row * stride + col) * int64_t(sizeof(typename Type<D>::elem));
}

}  // namespace zp
