// tensor_step.hip -- AdamW over a tensor set, the begin of its step, and the
// conversion of its states (gfx950).
//
// Per element (decoupled weight decay; the constants are the group's, from
// step_begin_kernel):
//   g = grad_mult * grad
//   m = beta1 m + (1 - beta1) g         v = beta2 v + (1 - beta2) g^2
//   p = p - (lr wd p + step (m / (sqrt(v) rbc2 + eps)))
// in fp32, one rounding per operation in that order, IEEE division and square
// root, so a scalar reference gives the same bits.
#include <hip/hip_ext.h>

#include "tensor_set.hpp"

#pragma clang fp contract(off)

namespace zp {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kGroups = int(kSetTile) / 256;   // 256-element groups of a tile, 4 elements a lane

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));

// Four consecutive elements of type T, at T's own alignment: tensors may start
// anywhere, and the hardware takes wide global accesses at any address.  The
// pointers come from a table, so they are cast to the global address space
// (generic ones would make flat accesses).
template <typename T>
struct Four;
template <>
struct Four<float> {
    typedef f32x4 vec;
    typedef f32x4 at __attribute__((aligned(4)));
};
template <>
struct Four<uint16_t> {
    typedef u16x4 vec;
    typedef u16x4 at __attribute__((aligned(2)));
};
template <>
struct Four<uint8_t> {   // as one word: the conversions take packed codes
    typedef uint32_t vec;
    typedef uint32_t at __attribute__((aligned(1)));
};

template <typename T>
using Global = __attribute__((address_space(1))) T;

// Elements p[0 .. n) (n = 1..4; zeros after them); non-temporal where whole:
// no line is used again.
template <typename T>
__device__ __forceinline__ typename Four<T>::vec load4(const T* p, int n) {
    typedef const typename Four<T>::at at;
    if (n == 4) return __builtin_nontemporal_load((Global<at>*)p);
    Global<const T>* q = (Global<const T>*)p;
    typename Four<T>::vec r = {};
    if constexpr (sizeof(T) == 1) {
#pragma unroll
        for (int k = 0; k < 3; ++k)
            if (k < n) r |= uint32_t(q[k]) << (8 * k);
    } else {
#pragma unroll
        for (int k = 0; k < 3; ++k)
            if (k < n) r[k] = q[k];
    }
    return r;
}

template <typename T>
__device__ __forceinline__ void store4(T* p, typename Four<T>::vec v, int n) {
    typedef typename Four<T>::at at;
    if (n == 4) {
        __builtin_nontemporal_store(v, (Global<at>*)p);
        return;
    }
    Global<T>* q = (Global<T>*)p;
#pragma unroll
    for (int k = 0; k < 3; ++k)
        if (k < n) {
            if constexpr (sizeof(T) == 1) q[k] = T(v >> (8 * k));
            else q[k] = v[k];
        }
}

// Types behind the ABI's dtype numbers.
template <int D>
struct Type;
template <>
struct Type<ZERO_DTYPE_FP16> {
    typedef uint16_t elem;
    static __device__ __forceinline__ float wide(uint16_t x) { return float(__builtin_bit_cast(_Float16, x)); }
    static __device__ __forceinline__ uint16_t narrow(float x) { return __builtin_bit_cast(uint16_t, _Float16(x)); }
};
template <>
struct Type<ZERO_DTYPE_BF16> {
    typedef uint16_t elem;
    static __device__ __forceinline__ float wide(uint16_t x) { return __builtin_bit_cast(float, uint32_t(x) << 16); }
    static __device__ __forceinline__ uint16_t narrow(float x) { return __builtin_bit_cast(uint16_t, __bf16(x)); }
};
template <>
struct Type<ZERO_DTYPE_FP32> {
    typedef float elem;
    static __device__ __forceinline__ float wide(float x) { return x; }
};
template <>
struct Type<ZERO_DTYPE_MXFP8> {
    typedef uint8_t elem;
};

// ---------------------------------------------------------------------------
// MXFP8 states: a block of 32 elements is 8 neighbouring lanes with 4 each
// ---------------------------------------------------------------------------

// Largest x (>= 0) of the 8 lanes of this lane's block: three exchanges inside
// a row, no LDS.
__device__ __forceinline__ float block_max(float x) {
    const auto other = [](float v, auto ctrl) {
        return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), decltype(ctrl)::value, 0xF, 0xF, false));
    };
    x = fmaxf(x, other(x, std::integral_constant<int, 0xB1>{}));    // lanes 1, 0, 3, 2 of each four
    x = fmaxf(x, other(x, std::integral_constant<int, 0x4E>{}));    // lanes 2, 3, 0, 1
    return fmaxf(x, other(x, std::integral_constant<int, 0x141>{}));   // eight lanes mirrored
}

// The scale byte of a block whose largest magnitude is `top`: the least s >= 1
// with top 2^(127 - s) <= 448 = 1.75 2^8.  The exponent of top less 8, and one
// more when its fraction is above 1.75.
__device__ __forceinline__ int scale_of(float top) {
    const int e = int((__builtin_bit_cast(uint32_t, top) + 0x1FFFFFu) >> 23) - 8;
    return e > 1 ? e : 1;
}
__device__ __forceinline__ float two_to(int biased) { return __builtin_bit_cast(float, biased << 23); }

// 2^(s - 127).  s = 0 is 2^-127, below the normal range.
__device__ __forceinline__ float scale_value(int s) { return s ? two_to(s) : __builtin_bit_cast(float, 0x00400000); }

__device__ __forceinline__ void decode4(uint32_t code, int s, float x[4]) {
    const float f = scale_value(s);
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(int(code), false);
    const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8(int(code), true);
    x[0] = a.x * f;
    x[1] = a.y * f;
    x[2] = b.x * f;
    x[3] = b.y * f;
}

// Codes of y (448 at most in magnitude), to nearest, ties to even.
__device__ __forceinline__ uint32_t encode4(const float y[4]) {
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
    return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], lo, true));
}

// The multiplier into a block's range, 2^(127 - s), exact for any value but
// those that fall below fp32's normal range.
__device__ __forceinline__ float into_block(int s) { return two_to(254 - s); }

__device__ __forceinline__ uint32_t encode_m(const float m[4], int* s) {
    *s = scale_of(block_max(fmaxf(fmaxf(fabsf(m[0]), fabsf(m[1])), fmaxf(fabsf(m[2]), fabsf(m[3])))));
    const float f = into_block(*s);
    const float y[4] = {m[0] * f, m[1] * f, m[2] * f, m[3] * f};
    return encode4(y);
}

// v (>= 0), to nearest, or to a neighbour at random where `chance` is given
// (16 random bits for each element); a value above zero gets at least code 1.
// At random: the lower 20 bits of an fp32 are what an e4m3 has no room for;
// adding random ones below them and cutting them off rounds up as often as they
// say.  Below 2^-6 an e4m3's steps stay 2^-9, the steps of [2^-6, 2^-5): such
// values are lifted into that range, rounded there and lowered again.
template <bool kRandom>
__device__ __forceinline__ uint32_t encode_v(const float v[4], const uint32_t* chance, int* s) {
    *s = scale_of(block_max(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]))));
    const float f = into_block(*s);
    float y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float x = v[k] * f;
        y[k] = x;
        if (kRandom) {
            const float lift = x < 0x1p-6f ? 0x1p-6f : 0.0f;
            const uint32_t up = (chance[k] << 4) | 8u;
            y[k] = __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, x + lift) + up) & 0xFFF00000u) - lift;
        }
        y[k] = fmaxf(y[k], v[k] > 0.0f ? 0x1p-9f : 0.0f);
    }
    return encode4(y);
}

// ---------------------------------------------------------------------------
// the step
// ---------------------------------------------------------------------------

struct Consts {   // zero_step_control.group
    float beta1, omb1, beta2, omb2;   // omb: 1 - beta
    float decay;                      // lr * weight_decay
    float step;                       // lr / (1 - beta1^t)
    float rbc2;                       // 1 / sqrt(1 - beta2^t)
    float eps;
};
static_assert(sizeof(Consts) == sizeof(zero_step_control::group) / ZERO_MAX_GROUPS, "group constants");

// One thread per group computes its constants in fp64; thread 0 decides and
// counts.
__global__ __launch_bounds__(64) void step_begin_kernel(const BeginLaunch a) {
    zero_step_control* c = a.ctl;
    const int64_t t = c->t + 1;
    const float scale = c->scale, lr_mult = c->lr_mult;
    bool ok = scale >= ZERO_MIN_LOSS_SCALE && scale <= 3.402823466e38f && fabsf(lr_mult) <= 3.402823466e38f;
    double norm = 0.0, clip = 1.0;
    if (a.check) {
        norm = sqrt(c->sumsq) / double(scale);
        if (a.max_norm > 0.0f && norm > double(a.max_norm)) clip = double(a.max_norm) / norm;
        // an infinite norm gives inf * 0: no comparison with NaN holds.  Below
        // 2^62 every square and its average stay inside fp32's range.
        ok = ok && norm * clip < 0x1p62;
    }
    __syncthreads();   // everything read
    const int k = int(threadIdx.x);
    if (k < a.n_groups && ok) {
        const zero_adam_hparams& h = a.group[k];
        const double lr = double(h.lr) * double(lr_mult);
        Consts g;
        g.beta1 = h.beta1;
        g.omb1 = 1.0f - h.beta1;
        g.beta2 = h.beta2;
        g.omb2 = 1.0f - h.beta2;
        g.decay = float(lr * double(h.weight_decay));
        g.step = float(lr / (1.0 - pow(double(h.beta1), double(t))));
        g.rbc2 = float(1.0 / sqrt(1.0 - pow(double(h.beta2), double(t))));
        g.eps = h.eps;
        *reinterpret_cast<Consts*>(c->group[k]) = g;
    }
    if (k != 0) return;
    c->norm = float(norm);
    c->grad_mult = ok ? float(clip / double(scale)) : 0.0f;
    c->skip = ok ? 0 : 1;
    if (ok) c->t = t;
    else c->skipped += 1;
    if (!a.scaler) return;
    if (!ok) {
        const float s = scale * a.backoff;
        c->scale = s < a.min_scale ? a.min_scale : s;
        c->good_steps = 0;
        return;
    }
    int32_t good = c->good_steps;
    if (good < INT32_MAX) good += 1;
    if (a.growth_interval > 0 && good >= a.growth_interval) {
        const float s = scale * a.growth;
        if (s <= 3.402823466e38f) c->scale = s;
        good = 0;
    }
    c->good_steps = good;
}

__device__ __forceinline__ void adamw_element(const Consts& c, float g, float& p, float& m, float& v) {
    m = c.beta1 * m + c.omb1 * g;
    v = c.beta2 * v + c.omb2 * (g * g);
    const float den = __builtin_sqrtf(v) * c.rbc2 + c.eps;
    p = p - (c.decay * p + c.step * (m / den));
}

template <int G, int S>
struct TileIn {
    typename Four<typename Type<G>::elem>::vec g[kGroups];
    f32x4 p[kGroups];
    typename Four<typename Type<S>::elem>::vec m[kGroups], v[kGroups];
    int ms[kGroups], vs[kGroups];
};

// Elements that a lane has from `e` on: 0..4.
__device__ __forceinline__ int count4(int64_t numel, int64_t e) {
    const int64_t left = numel - e;
    return left >= 4 ? 4 : left > 0 ? int(left) : 0;
}

template <int G, int S, bool kWhole>
__device__ __forceinline__ void load_tile(const TensorRec& r, int64_t base, int lane, TileIn<G, S>& t) {
    typedef typename Type<G>::elem GT;
    typedef typename Type<S>::elem ST;
#pragma unroll
    for (int h = 0; h < kGroups; ++h) {
        const int64_t e = base + h * 256 + 4 * lane;
        const int n = kWhole ? 4 : count4(r.numel, e);
        if (n == 0) {
            t.g[h] = {};
            t.p[h] = {};
            t.m[h] = {};
            t.v[h] = {};
            t.ms[h] = t.vs[h] = 1;
            continue;
        }
        t.g[h] = load4(static_cast<const GT*>(r.grad) + e, n);
        t.p[h] = load4(r.p + e, n);
        t.m[h] = load4(static_cast<const ST*>(r.m) + e, n);
        t.v[h] = load4(static_cast<const ST*>(r.v) + e, n);
        if constexpr (S == ZERO_DTYPE_MXFP8) {
            const int64_t b = e / ZERO_STATE_BLOCK;
            t.ms[h] = ((Global<const uint8_t>*)r.m_scale)[b];
            t.vs[h] = ((Global<const uint8_t>*)r.v_scale)[b];
        }
    }
}

template <int G, int O, int S, bool kWhole>
__device__ __forceinline__ void step_tile(const TensorRec& r, const Consts& c, float mult, uint32_t key, int64_t base,
                                          int lane) {
    typedef typename Type<S>::elem ST;
    TileIn<G, S> t;
    load_tile<G, S, kWhole>(r, base, lane, t);
#pragma unroll
    for (int h = 0; h < kGroups; ++h) {
        const int64_t e = base + h * 256 + 4 * lane;
        const int n = kWhole ? 4 : count4(r.numel, e);
        float p[4] = {t.p[h].x, t.p[h].y, t.p[h].z, t.p[h].w};
        float m[4], v[4];
        if constexpr (S == ZERO_DTYPE_MXFP8) {
            decode4(t.m[h], t.ms[h], m);
            decode4(t.v[h], t.vs[h], v);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) m[k] = t.m[h][k], v[k] = t.v[h][k];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) adamw_element(c, Type<G>::wide(t.g[h][k]) * mult, p[k], m[k], v[k]);
        if constexpr (S == ZERO_DTYPE_MXFP8) {
            // every lane takes part in its block's maxima; past the end all are zero
            const uint32_t pair = uint32_t(e >> 1);
            const uint32_t r0 = mix32(pair + key), r1 = mix32(pair + 1 + key);
            const uint32_t chance[4] = {r0 & 0xFFFFu, r0 >> 16, r1 & 0xFFFFu, r1 >> 16};
            int ms, vs;
            const uint32_t mc = encode_m(m, &ms), vc = encode_v<true>(v, chance, &vs);
            if (n > 0) {
                store4(static_cast<ST*>(r.m) + e, mc, n);
                store4(static_cast<ST*>(r.v) + e, vc, n);
                if ((lane & 7) == 0) {
                    const int64_t b = e / ZERO_STATE_BLOCK;
                    ((Global<uint8_t>*)r.m_scale)[b] = uint8_t(ms);
                    ((Global<uint8_t>*)r.v_scale)[b] = uint8_t(vs);
                }
            }
        } else if (n > 0) {
            store4(static_cast<ST*>(r.m) + e, f32x4{m[0], m[1], m[2], m[3]}, n);
            store4(static_cast<ST*>(r.v) + e, f32x4{v[0], v[1], v[2], v[3]}, n);
        }
        if (n > 0) {
            store4(r.p + e, f32x4{p[0], p[1], p[2], p[3]}, n);
            if constexpr (O != ZERO_DTYPE_NONE) {
                const u16x4 o = {Type<O>::narrow(p[0]), Type<O>::narrow(p[1]), Type<O>::narrow(p[2]), Type<O>::narrow(p[3])};
                store4(static_cast<uint16_t*>(r.out) + e, o, n);
            }
        }
    }
}

// The tile of this wave, the same in all its lanes; false past the last one.
__device__ __forceinline__ bool wave_tile(const SetLaunch& a, TileRec* tile) {
    const int64_t w = int64_t(blockIdx.x) * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (w >= a.n_tiles) return false;
    *tile = a.tile[w];
    return true;
}

template <int G, int O, int S>
__global__ __launch_bounds__(kThreads) void adamw_kernel(const SetLaunch a, const zero_step_control* __restrict__ ctl) {
    TileRec tile;
    if (!wave_tile(a, &tile) || ctl->skip) return;
    const TensorRec r = a.rec[tile.tensor];
    const Consts c = *reinterpret_cast<const Consts*>(ctl->group[r.group]);
    const float mult = ctl->grad_mult;
    const uint32_t key = mix32(r.key + uint32_t(ctl->t) * 0x9E3779B9u);
    const int64_t base = int64_t(tile.tile) * kSetTile;
    const int lane = threadIdx.x & 63;
    if (r.numel - base >= kSetTile) step_tile<G, O, S, true>(r, c, mult, key, base, lane);
    else step_tile<G, O, S, false>(r, c, mult, key, base, lane);
}

template <int G, int O>
void run_adamw(const SetLaunch& a, const zero_step_control* ctl, dim3 grid, hipStream_t s, const KernelEvents& ev);

// ---------------------------------------------------------------------------
// state conversion
// ---------------------------------------------------------------------------

template <bool kEncode>
__global__ __launch_bounds__(kThreads) void convert_kernel(const SetLaunch dst, const SetLaunch src) {
    TileRec tile;
    if (!wave_tile(src, &tile)) return;
    const TensorRec from = src.rec[tile.tensor], to = dst.rec[tile.tensor];
    const TensorRec& wide = kEncode ? from : to;
    const TensorRec& mx = kEncode ? to : from;
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int h = 0; h < kGroups; ++h) {
        const int64_t e = int64_t(tile.tile) * kSetTile + h * 256 + 4 * lane;
        const int n = count4(from.numel, e);
        const int64_t b = e / ZERO_STATE_BLOCK;
        float* wm = static_cast<float*>(wide.m) + e;
        float* wv = static_cast<float*>(wide.v) + e;
        uint8_t* cm = static_cast<uint8_t*>(mx.m) + e;
        uint8_t* cv = static_cast<uint8_t*>(mx.v) + e;
        if (kEncode) {
            f32x4 m4 = {}, v4 = {};
            if (n > 0) {
                m4 = load4(static_cast<const float*>(wm), n);
                v4 = load4(static_cast<const float*>(wv), n);
            }
            const float m[4] = {m4.x, m4.y, m4.z, m4.w}, v[4] = {v4.x, v4.y, v4.z, v4.w};
            int ms, vs;
            const uint32_t mc = encode_m(m, &ms), vc = encode_v<false>(v, nullptr, &vs);
            if (n > 0) {
                store4(cm, mc, n);
                store4(cv, vc, n);
                if ((lane & 7) == 0) {
                    ((Global<uint8_t>*)mx.m_scale)[b] = uint8_t(ms);
                    ((Global<uint8_t>*)mx.v_scale)[b] = uint8_t(vs);
                }
            }
        } else if (n > 0) {
            float m[4], v[4];
            decode4(load4(static_cast<const uint8_t*>(cm), n), ((Global<const uint8_t>*)mx.m_scale)[b], m);
            decode4(load4(static_cast<const uint8_t*>(cv), n), ((Global<const uint8_t>*)mx.v_scale)[b], v);
            store4(wm, f32x4{m[0], m[1], m[2], m[3]}, n);
            store4(wv, f32x4{v[0], v[1], v[2], v[3]}, n);
        }
    }
}

dim3 tile_grid(int64_t n_tiles) { return dim3(unsigned((n_tiles + kWaves - 1) / kWaves)); }

template <typename K, typename... Args>
void launch(K kernel, dim3 grid, hipStream_t s, const KernelEvents& ev, Args... args) {
    if (ev.start) hipExtLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, s, ev.start, ev.stop, 0, args...);
    else hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, s, args...);
}

template <int G, int O>
void run_adamw(const SetLaunch& a, const zero_step_control* ctl, dim3 grid, hipStream_t s, const KernelEvents& ev) {
    if (a.state_type == ZERO_DTYPE_MXFP8) launch(adamw_kernel<G, O, ZERO_DTYPE_MXFP8>, grid, s, ev, a, ctl);
    else launch(adamw_kernel<G, O, ZERO_DTYPE_FP32>, grid, s, ev, a, ctl);
}

template <int G>
void run_adamw_out(const SetLaunch& a, const zero_step_control* ctl, dim3 grid, hipStream_t s, const KernelEvents& ev) {
    switch (a.out_type) {
        case ZERO_DTYPE_FP16: run_adamw<G, ZERO_DTYPE_FP16>(a, ctl, grid, s, ev); break;
        case ZERO_DTYPE_BF16: run_adamw<G, ZERO_DTYPE_BF16>(a, ctl, grid, s, ev); break;
        default: run_adamw<G, ZERO_DTYPE_NONE>(a, ctl, grid, s, ev); break;
    }
}

}  // namespace

hipError_t launch_step_begin(const BeginLaunch& a, hipStream_t stream) {
    hipLaunchKernelGGL(step_begin_kernel, dim3(1), dim3(64), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_adamw(const SetLaunch& a, const zero_step_control* ctl, hipStream_t stream, const KernelEvents& ev) {
    const dim3 grid = tile_grid(a.n_tiles);
    switch (a.grad_type) {
        case ZERO_DTYPE_FP16: run_adamw_out<ZERO_DTYPE_FP16>(a, ctl, grid, stream, ev); break;
        case ZERO_DTYPE_BF16: run_adamw_out<ZERO_DTYPE_BF16>(a, ctl, grid, stream, ev); break;
        default: run_adamw_out<ZERO_DTYPE_FP32>(a, ctl, grid, stream, ev); break;
    }
    return hipGetLastError();
}

hipError_t launch_convert(const SetLaunch& dst, const SetLaunch& src, hipStream_t stream, const KernelEvents& ev) {
    const dim3 grid = tile_grid(src.n_tiles);
    if (src.state_type == ZERO_DTYPE_FP32) launch(convert_kernel<true>, grid, stream, ev, dst, src);
    else launch(convert_kernel<false>, grid, stream, ev, dst, src);
    return hipGetLastError();
}

}  // namespace zp
