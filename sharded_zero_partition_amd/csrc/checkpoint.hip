// checkpoint.hip -- activation checkpoints in 8 bits: store, load, activations
// that store the checkpoint of their input, and the gradients read from it
// (gfx950).
//
// A thread takes octets of 8 neighbouring values, so a block of 32 is four
// lanes: its largest magnitude takes two exchanges inside a quad.  Codes and
// scales of all rows lie back to back, so octet o of the matrix is codes
// 8 o .. 8 o + 7 and scale byte o / 4, whatever the rows' length; only the wide
// matrices need an octet's row and column.  All of it is bound by HBM: each
// value is read and written once, with the checkpoint's scales and codes
// computed from the registers that the activation is computed from.
//
// Wide values pass by the caches.  8192 x 20480 bf16 (845 MB), gelu_tanh and its gradient:
// 130 and 152 us, plain 144 and 162, where the same buffers come again (the last-level
// cache then keeps what does not pass by it); 141 and 149, plain 144 and 160, where all
// that is read comes from HBM.  Rows of 13653, which start anywhere, gated silu: 92 and 91,
// plain 106 and 107; from HBM 107 and 105, plain 105 and 104.  A plain store keeps its
// loads in the caches' way, where its input mostly comes from (8192 x 5120: 20.3 us, else
// 24), and so do all codes (24 us for loading them back, else 19).
// Results that pass by the caches are not there for the call that reads them.  Both calls
// in a row, results of 1 / 10 / 80 / 300 MB in bf16, us, and with plain stores:
//   lookup, checkpoint store           5.4 8.5 47 184       plain 5.4 9.1 47 197
//   silu, library product              14.4 26 142 434      plain 12.3 27 138 440
//   silu's gradient, weight gradient   13.6 40 124 400      plain 12.1 40 121 396
// Neither is better throughout, nor is there one size where it turns: one rule for all.
#include <type_traits>

#include "octets.hpp"
#include "timed_launch.hpp"

#pragma clang fp contract(off)

namespace zp {
namespace {

// ---------------------------------------------------------------------------
// blocks
// ---------------------------------------------------------------------------

// Codes and scale of a lane's octet, the quad's four lanes being its block.
struct Packed {
    u32x2 code;
    uint32_t scale;
};

__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }

// The bits, as an fp32's, of the largest magnitude of the octet.
template <int D>
__device__ __forceinline__ uint32_t largest(const Octet<D>& x) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kOctet; ++i) top = larger(top, bits(x.get(i)) & 0x7FFFFFFFu);
    return top;
}

// Of the octet's values `n` exist; the codes behind them are zero.
template <int D>
__device__ __forceinline__ Packed pack(const Octet<D>& x, int64_t n) {
    uint32_t top = largest(x);
    top = larger(top, across<0xB1>(top));   // lanes 1, 0, 3, 2 of each four
    top = larger(top, across<0x4E>(top));   // lanes 2, 3, 0, 1
    Packed r;
    if (top < 0x7F800000u) {
        const int s = scale_of(top);
        const float f = into_block(s);
        float y[kOctet];
#pragma unroll
        for (int i = 0; i < kOctet; ++i) y[i] = x.get(i) * f;
        if constexpr (D != ZERO_DTYPE_FP16) {   // nothing finite becomes 2^128: 240 is 1.875 2^127 there
            const float most = s < 247 ? 448.0f : 240.0f;
#pragma unroll
            for (int i = 0; i < kOctet; ++i) y[i] = __builtin_amdgcn_fmed3f(y[i], -most, most);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * h], y[4 * h + 1], 0, false);
            r.code[h] = uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(y[4 * h + 2], y[4 * h + 3], lo, true));
        }
        r.scale = uint32_t(s);
        return r;
    }
    r.scale = 255;
    const uint64_t code = n <= 0 ? 0 : 0x7F7F7F7F7F7F7F7Full >> (n >= kOctet ? 0 : 8 * (kOctet - n));
    r.code = u32x2{uint32_t(code), uint32_t(code >> 32)};
    return r;
}

// Octet o's codes, and the scales of the row of 16 lanes, whose first octet is a
// multiple of 16: four bytes that leave as one word.
__device__ __forceinline__ void keep(const Packed& r, int64_t o, int64_t octets, int64_t blocks, uint8_t* code,
                                     uint8_t* scale) {
    const int lane = int(threadIdx.x) & 15;
    uint32_t w = r.scale << (8 * (lane >> 2));
    w |= across<0x141>(w);   // eight lanes mirrored
    w |= across<0x140>(w);   // sixteen
    if (o >= octets) return;
    *(Global<u32x2>*)(code + 8 * o) = r.code;
    const int64_t b = o >> 2;
    if (lane == 0 && b + 4 <= blocks) {
        typedef uint32_t at __attribute__((aligned(1)));
        *(Global<at>*)(scale + b) = w;
    } else if ((lane & 3) == 0 && (b & ~int64_t(3)) + 4 > blocks) {   // the last blocks of all
        ((Global<uint8_t>*)scale)[b] = uint8_t(r.scale);
    }
}

// An octet of a checkpoint.
struct Kept {
    u32x2 code;
    uint32_t scale;
    __device__ __forceinline__ void load(const uint8_t* c, const uint8_t* s, int64_t o) {
        code = *(Global<const u32x2>*)(c + 8 * o);
        scale = ((Global<const uint8_t>*)s)[o >> 2];
    }
    __device__ __forceinline__ void values(float x[kOctet]) const {
        const float f = scale_value(int(scale));   // an infinity for 255, whose codes are NaN
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(int(code[h]), false);
            const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8(int(code[h]), true);
            x[4 * h] = a.x * f;
            x[4 * h + 1] = a.y * f;
            x[4 * h + 2] = b.x * f;
            x[4 * h + 3] = b.y * f;
        }
    }
};

// ---------------------------------------------------------------------------
// activations
// ---------------------------------------------------------------------------

// p = 1 / (1 + exp(-a)) and 1 - p = exp(-a) p, which a difference would round
// away near p = 1.  Where the exponential overflows both are 0.
__device__ __forceinline__ float sigmoid(float a, float* rest = nullptr) {
    const float e = __builtin_amdgcn_exp2f(a * -1.44269504f);
    const float p = __builtin_amdgcn_rcpf(1.0f + e);
    if (rest) *rest = fminf(e, 1e38f) * p;
    return p;
}

// The normal distribution's value at z, and exp(-z^2 / 2).  With x = |z| / sqrt 2 the
// lower tail is erfc(x) / 2 = exp(-x^2) t P(t), t = 1 / (1 + x / 2), where erfcx(x) / 2t is
// so smooth that a polynomial of degree 8, fitted to it for x up to 10 by weighted least
// squares, is within 5e-8, and within 2e-7 in fp32.  The exponential is the
// density's too.  (By the library's erfcf an activation took 258 us for 8192 x 20480 bf16
// values, bound by its instructions; by this 158.)
__device__ __forceinline__ float normal(float z, float* e) {
#pragma clang fp contract(fast)
    constexpr float c[9] = {0.141043208f,  0.141187664f,  0.121551807f, 0.101343742f,  -0.013313581f,
                            0.139034689f, -0.243600932f, 0.142287959f, -0.029534578f};
    const float t = __builtin_amdgcn_rcpf(1.0f + 0.35355339f * fabsf(z));
    *e = __builtin_amdgcn_exp2f(-0.72134752f * (z * z));
    float p = c[8];
#pragma unroll
    for (int i = 7; i >= 0; --i) p = p * t + c[i];
    const float tail = *e * (p * t);
    return z > 0.0f ? 1.0f - tail : tail;
}

// The value of an activation and its derivative.  With p = act(z) / z rising from 0
// to 1: p is a sigmoid of a(z) (silu: a = z, gelu_tanh: twice tanh's argument), or
// the normal distribution (gelu).  act' = p + z p', p' = p (1 - p) a' for a
// sigmoid.  For |z| beyond 20, p is 0 or 1 and p' 0 in fp32: z^2 stops there in
// a polynomial, which then neither overflows nor meets its own zero.
template <int K>
struct Act {
    static __device__ __forceinline__ float value(float z) {
        if constexpr (K == ZERO_ACT_RELU) return z <= 0.0f ? 0.0f : z;
        if constexpr (K == ZERO_ACT_SILU) return z * sigmoid(z);
        if constexpr (K == ZERO_ACT_GELU) {
            float e;
            return z * normal(z, &e);
        }
        if constexpr (K == ZERO_ACT_GELU_TANH) return z * sigmoid(angle(z, square(z)));
        return z;
    }
    static __device__ __forceinline__ void both(float z, float* a, float* da) {
#pragma clang fp contract(fast)
        if constexpr (K == ZERO_ACT_RELU) {
            *a = z <= 0.0f ? 0.0f : z;
            *da = z > 0.0f ? 1.0f : z <= 0.0f ? 0.0f : z;
        } else if constexpr (K == ZERO_ACT_GELU) {
            float e;
            const float p = normal(z, &e);
            *a = z * p;
            *da = p + z * (0.39894228f * e);
        } else if constexpr (K == ZERO_ACT_SILU) {
            float rest;
            const float p = sigmoid(z, &rest);
            *a = z * p;
            *da = p + *a * rest;
        } else {
            float rest;
            const float q = square(z), p = sigmoid(angle(z, q), &rest);
            *a = z * p;
            *da = p + *a * (rest * (float(k1) + float(3 * k3) * q));
        }
    }
    static constexpr double k1 = 1.5957691216057308, k3 = 0.044715 * k1;   // 2 sqrt(2 / pi)
    static __device__ __forceinline__ float square(float z) { return fminf(z * z, 400.0f); }
    static __device__ __forceinline__ float angle(float z, float q) {   // 2 sqrt(2 / pi) (z + 0.044715 z^3), q = z^2
#pragma clang fp contract(fast)
        return z * (float(k1) + float(k3) * q);
    }
};

// Where a thread's octets are: the wave's are neighbours.
struct At {
    int64_t o, row, col;
    int64_t left;   // the row's values from col on
};
__device__ __forceinline__ void find(const ActLaunch& a, At at[kRowOctets]) {
    const int64_t base = int64_t(blockIdx.x) * (kRowThreads * kRowOctets);
    int64_t row;
    uint32_t rest;
    divide(base, a.per_row, &row, &rest);
#pragma unroll
    for (int u = 0; u < kRowOctets; ++u) {
        const uint32_t i = threadIdx.x + u * kRowThreads;
        const uint32_t q = divide(rest + i, a.per_row);
        at[u].o = base + i;
        at[u].row = row + q;
        at[u].col = int64_t(rest + i - q * a.per_row.g) * kOctet;
        at[u].left = at[u].o < a.octets ? a.cols - at[u].col : 0;
    }
}

template <int D, int K, bool kGated>
__global__ __launch_bounds__(kRowThreads) void activation_kernel(const ActLaunch a) {
    At at[kRowOctets];
    find(a, at);
    Octet<D> x[kRowOctets], up[kRowOctets];
#pragma unroll
    for (int u = 0; u < kRowOctets; ++u) {
        x[u] = load_octet<D, (K >= 0)>(place<D>(a.x, at[u].row, a.sx, at[u].col), at[u].left);
        if (kGated) up[u] = load_octet<D, true>(place<D>(a.up, at[u].row, a.sup, at[u].col), at[u].left);
    }
#pragma unroll
    for (int u = 0; u < kRowOctets; ++u) {
        if (a.cx) keep(pack(x[u], at[u].left), at[u].o, a.octets, a.blocks, a.cx, a.cx_scale);
        if (kGated && a.cup) keep(pack(up[u], at[u].left), at[u].o, a.octets, a.blocks, a.cup, a.cup_scale);
        if constexpr (K >= 0) {
            Octet<D> h;
#pragma unroll
            for (int i = 0; i < kOctet; ++i) {
                const float v = Act<K>::value(x[u].get(i));
                h.set(i, kGated ? v * up[u].get(i) : v);
            }
            store_octet<D, true>(place<D>(a.out, at[u].row, a.sout, at[u].col), at[u].left, h);
            if (a.cout) keep(pack(h, at[u].left), at[u].o, a.octets, a.blocks, a.cout, a.cout_scale);
        }
    }
}

template <int D, int K, bool kGated>
__global__ __launch_bounds__(kRowThreads) void activation_grad_kernel(const ActLaunch a) {
    At at[kRowOctets];
    find(a, at);
    Octet<D> dy[kRowOctets];
    Kept x[kRowOctets], up[kRowOctets];
#pragma unroll
    for (int u = 0; u < kRowOctets; ++u) {
        if (at[u].left <= 0) continue;
        if constexpr (K >= 0) dy[u] = load_octet<D, true>(place<D>(a.x, at[u].row, a.sx, at[u].col), at[u].left);
        x[u].load(a.cx, a.cx_scale, at[u].o);
        if (kGated) up[u].load(a.cup, a.cup_scale, at[u].o);
    }
#pragma unroll
    for (int u = 0; u < kRowOctets; ++u) {
        if (at[u].left <= 0) continue;
        float z[kOctet], v[kOctet];
        x[u].values(z);
        if (kGated) up[u].values(v);
        Octet<D> dx, dup;
#pragma unroll
        for (int i = 0; i < kOctet; ++i) {
            if constexpr (K < 0) {
                dx.set(i, z[i]);
            } else {
                float h, dh;
                Act<K>::both(z[i], &h, &dh);
                const float g = dy[u].get(i);
                dx.set(i, kGated ? g * v[i] * dh : g * dh);
                if (kGated) dup.set(i, g * h);
            }
        }
        store_octet<D, true>(place<D>(a.out, at[u].row, a.sout, at[u].col), at[u].left, dx);
        if (kGated) store_octet<D, true>(place<D>(a.dup, at[u].row, a.sdup, at[u].col), at[u].left, dup);
    }
}

typedef void (*ActKernel)(const ActLaunch);

template <int D, bool kGrad>
ActKernel act_kernel(int kind, bool gated) {
#define ZP_ACT(K, G) (kGrad ? activation_grad_kernel<D, K, G> : activation_kernel<D, K, G>)
    switch (kind) {
        case ZERO_ACT_RELU: return gated ? ZP_ACT(ZERO_ACT_RELU, true) : ZP_ACT(ZERO_ACT_RELU, false);
        case ZERO_ACT_SILU: return gated ? ZP_ACT(ZERO_ACT_SILU, true) : ZP_ACT(ZERO_ACT_SILU, false);
        case ZERO_ACT_GELU: return gated ? ZP_ACT(ZERO_ACT_GELU, true) : ZP_ACT(ZERO_ACT_GELU, false);
        case ZERO_ACT_GELU_TANH: return gated ? ZP_ACT(ZERO_ACT_GELU_TANH, true) : ZP_ACT(ZERO_ACT_GELU_TANH, false);
        default: return ZP_ACT(-1, false);
    }
#undef ZP_ACT
}

template <bool kGrad>
hipError_t launch_act(const ActLaunch& a, hipStream_t s, const KernelEvents& ev) {
    const bool gated = kGrad ? a.dup != nullptr : a.up != nullptr;
    ActKernel k = a.type == ZERO_DTYPE_FP16   ? act_kernel<ZERO_DTYPE_FP16, kGrad>(a.kind, gated)
                  : a.type == ZERO_DTYPE_BF16 ? act_kernel<ZERO_DTYPE_BF16, kGrad>(a.kind, gated)
                                              : act_kernel<ZERO_DTYPE_FP32, kGrad>(a.kind, gated);
    constexpr int64_t per = kRowThreads * kRowOctets;
    launch(k, dim3(uint32_t((a.octets + per - 1) / per)), kRowThreads, s, ev, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_activation(const ActLaunch& a, hipStream_t s, const KernelEvents& ev) {
    return launch_act<false>(a, s, ev);
}
hipError_t launch_activation_grad(const ActLaunch& a, hipStream_t s, const KernelEvents& ev) {
    return launch_act<true>(a, s, ev);
}

}  // namespace zp
