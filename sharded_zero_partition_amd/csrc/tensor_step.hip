// tensor_step.hip -- AdamW over a tensor set, the begin of its step, and the
// conversion of its states (gfx950).
//
// Per element (decoupled weight decay; the constants are the group's, from
// step_begin_kernel):
//   g = grad_mult * grad
//   m = beta1 m + (1 - beta1) g         v = beta2 v + (1 - beta2) g^2
//   p = p - (lr wd p + step (m / (sqrt(v) rbc2 + eps)))
// in fp32, one rounding per operation in that order, so m, v and with fp32
// states p equal a scalar reference bit for bit.
#include <type_traits>

#include "mxfp8.hpp"
#include "tensor_set.hpp"
#include "timed_launch.hpp"

#pragma clang fp contract(off)

namespace zp {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kGroups = int(kSetTile) / 256;   // 256-element groups of a tile, 4 elements a lane

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

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

// Which of a lane's four elements exist: [a, b).
struct Part {
    int a, b;
    __device__ __forceinline__ bool none() const { return a >= b; }
    __device__ __forceinline__ bool all() const { return b - a == 4; }
    __device__ __forceinline__ bool has(int k) const { return k >= a && k < b; }
};

// Elements q .. q + 3 of a tile, p being where its element 0 is (the same in all
// lanes; outside the array for a tile that starts before it) and q a lane's
// first.  Non-temporal: no line is used again (plain loads and stores on whole
// lines: 1038 against 934 us for the step with fp32 states of 200 M elements,
// 607 against 546 us in 8 bits).
template <typename T>
__device__ __forceinline__ typename Four<T>::vec load4(const T* p, uint32_t q) {
    typedef const typename Four<T>::at at;
    return __builtin_nontemporal_load((Global<at>*)((Global<const char>*)p + q * uint32_t(sizeof(T))));
}

// The same in a group of lanes of which some have elements that do not exist:
// each lane loads four single elements, `at[k]` being element k or, where that
// is none, one that is there.  No branch and nothing to wait for until all
// arrays' loads are under way (20,000 tensors of 1000 elements, fp32 states:
// 86 us; with a branch for each element that exists, 101).
template <typename T>
struct Edge {   // each in a register of its own
    std::conditional_t<sizeof(T) == 4, T, uint32_t> e[4];
};
template <typename T>
__device__ __forceinline__ Edge<T> edge_load(const T* p, const int at[4]) {
    Edge<T> r;
#pragma unroll
    for (int k = 0; k < 4; ++k) r.e[k] = ((Global<const T>*)p)[at[k]];
    return r;
}
// ... and zeros in the places of those that are not.
template <typename T>
__device__ __forceinline__ typename Four<T>::vec edge_pack(const Edge<T>& x, Part n) {
    typename Four<T>::vec r = {};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const auto e = n.has(k) ? x.e[k] : 0;
        if constexpr (sizeof(T) == 1) r |= uint32_t(e) << (8 * k);
        else r[k] = T(e);
    }
    return r;
}

// Plain where not all four exist: single elements written non-temporally leave
// one by one (966 against 648 us for a misaligned step in 8 bits).
template <typename T>
__device__ __forceinline__ void store4(T* p, uint32_t q, typename Four<T>::vec v, Part n) {
    typedef typename Four<T>::at at;
    Global<T>* x = (Global<T>*)((Global<char>*)p + q * uint32_t(sizeof(T)));
    if (n.all()) {
        __builtin_nontemporal_store(v, (Global<at>*)x);
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (n.has(k)) {
            if constexpr (sizeof(T) == 1) x[k] = T(v >> (8 * k));
            else x[k] = v[k];
        }
}

// A tile: elements [lo, hi) of its kSetTile, its element 0 being `base` of the
// tensor.
struct Extent {
    int64_t base;
    int lo, hi;
    __device__ __forceinline__ bool whole() const { return hi - lo == int(kSetTile); }
    // whether the tile ends before its group h, and whether it has all of it
    // (the same in all lanes)
    template <bool kWhole>
    __device__ __forceinline__ bool without(int h) const {
        return !kWhole && h * 256 >= hi;
    }
    template <bool kWhole>
    __device__ __forceinline__ bool with(int h) const {
        return kWhole || (lo <= h * 256 && h * 256 + 256 <= hi);
    }
    // elements q .. q + 3, or the nearest of the tile's
    __device__ __forceinline__ void nearest(uint32_t q, int at[4]) const {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int e = int(q) + k;
            at[k] = e < lo ? lo : e < hi ? e : hi - 1;
        }
    }
    template <bool kWhole>
    __device__ __forceinline__ Part part(uint32_t q) const {
        if (kWhole) return {0, 4};
        const auto clamp = [](int x) { return x < 0 ? 0 : x > 4 ? 4 : x; };
        return {clamp(lo - int(q)), clamp(hi - int(q))};
    }
};
__device__ __forceinline__ Extent extent(const TensorRec& r, uint32_t tile, uint32_t shift) {
    const int64_t base = int64_t(tile) * kSetTile - shift, left = r.numel - base;
    return {base, base < 0 ? int(-base) : 0, left >= kSetTile ? int(kSetTile) : left < 0 ? 0 : int(left)};
}

// Where element 0 of a tile is in an array, as an integer-made pointer: it may
// lie before the array.
template <typename T>
__device__ __forceinline__ T* tile_at(const void* p, int64_t base) {
    return reinterpret_cast<T*>(reinterpret_cast<uintptr_t>(p) + uintptr_t(base * int64_t(sizeof(T))));
}

// ---------------------------------------------------------------------------
// MXFP8 states: a block of 32 elements is 8 neighbouring lanes with 4 each
// ---------------------------------------------------------------------------

// Largest of the 8 lanes' values, bits of fp32s that are not negative (these
// order like the numbers): three exchanges inside a row, no LDS.
__device__ __forceinline__ uint32_t block_max(uint32_t x) {
    const auto other = [](uint32_t v, auto ctrl) {
        return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), decltype(ctrl)::value, 0xF, 0xF, true));
    };
    const auto larger = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
    x = larger(x, other(x, std::integral_constant<int, 0xB1>{}));    // lanes 1, 0, 3, 2 of each four
    x = larger(x, other(x, std::integral_constant<int, 0x4E>{}));    // lanes 2, 3, 0, 1
    return larger(x, other(x, std::integral_constant<int, 0x141>{}));   // eight lanes mirrored
}
__device__ __forceinline__ uint32_t max4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    const uint32_t x = a > b ? a : b, y = c > d ? c : d;
    return x > y ? x : y;
}
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

// ... and to one of its two neighbours in magnitude at random: r0 holds 16 random
// bits for each of the first two elements, r1 for the others.  The conversion
// adds the upper 20 bits of its operand below the bits that an e4m3 has room for
// and cuts off there, so it rounds up as often as they say, below its least
// number too; the 16 are followed by 1000, the middle of what they leave open.
__device__ __forceinline__ uint32_t encode4_random(const float y[4], uint32_t r0, uint32_t r1) {
    int c = __builtin_amdgcn_cvt_sr_fp8_f32(y[0], (r0 << 16) | 0x8000u, 0, 0);
    c = __builtin_amdgcn_cvt_sr_fp8_f32(y[1], (r0 & 0xFFFF0000u) | 0x8000u, c, 1);
    c = __builtin_amdgcn_cvt_sr_fp8_f32(y[2], (r1 << 16) | 0x8000u, c, 2);
    return uint32_t(__builtin_amdgcn_cvt_sr_fp8_f32(y[3], (r1 & 0xFFFF0000u) | 0x8000u, c, 3));
}

// m, to nearest or at random (an m below the least number may become zero, so
// its mean is kept everywhere).
template <bool kRandom>
__device__ __forceinline__ uint32_t encode_m(const float m[4], uint32_t r0, uint32_t r1, int* s) {
    constexpr uint32_t kMag = 0x7FFFFFFFu;
    *s = scale_of(block_max(max4(bits(m[0]) & kMag, bits(m[1]) & kMag, bits(m[2]) & kMag, bits(m[3]) & kMag)));
    const float f = into_block(*s);
    const float y[4] = {m[0] * f, m[1] * f, m[2] * f, m[3] * f};
    return kRandom ? encode4_random(y, r0, r1) : encode4(y);
}

// v (>= 0, -0 among it), to nearest or at random; a value above zero gets at
// least code 1.  A step's v is the sum of +0 or more and never -0; a conversion's
// is the caller's, and -0 has the largest bits of all.
template <bool kRandom>
__device__ __forceinline__ uint32_t encode_v(const float v[4], uint32_t r0, uint32_t r1, int* s) {
    constexpr uint32_t kMag = kRandom ? 0xFFFFFFFFu : 0x7FFFFFFFu;
    *s = scale_of(block_max(max4(bits(v[0]) & kMag, bits(v[1]) & kMag, bits(v[2]) & kMag, bits(v[3]) & kMag)));
    const float f = into_block(*s);
    float y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float x = v[k] * f, least = v[k] > 0.0f ? 0x1p-9f : 0.0f;
        y[k] = x > least ? x : least;
    }
    return kRandom ? encode4_random(y, r0, r1) : encode4(y);
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
    const int64_t t = int64_t(uint64_t(c->t) + 1u);
    const float scale = c->scale, lr_mult = c->lr_mult;
    bool ok = t > 0 && scale >= ZERO_MIN_LOSS_SCALE && scale <= 3.402823466e38f && fabsf(lr_mult) <= 3.402823466e38f;
    double norm = 0.0, clip = 1.0;
    if (a.check) {
        norm = sqrt(c->sumsq) / double(scale);
        if (a.max_norm > 0.0f && norm > double(a.max_norm)) clip = double(a.max_norm) / norm;
        // an infinite norm gives inf * 0: no comparison with NaN holds.  Below
        // 2^62 every square and its average stay inside fp32's range.
        ok = ok && norm * clip < 0x1p62;
    }
    ok = ok && clip / double(scale) >= 0x1p-126;   // the factor is a normal fp32
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
        c->scale = s >= a.min_scale && s <= 3.402823466e38f ? s : a.min_scale;
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

// kFast (states in 8 bits): root and quotient by the hardware's approximations,
// within 1 ulp each, which puts the update within 14 half-ulps instead of 12 of
// the formula's; the states it came from are off by 2^-4.  With IEEE's sequences
// (21 instructions an element more) the kernel had 78 VALU instructions an
// element and the ALUs were busy for 400 of its 550 us at 200 M elements, which
// nothing could be added to.  The approximate root takes no subnormals: v counts
// as 2^-126 at least there.
template <bool kFast>
__device__ __forceinline__ void adamw_element(const Consts& c, float g, float& p, float& m, float& v) {
    m = c.beta1 * m + c.omb1 * g;
    v = c.beta2 * v + c.omb2 * (g * g);
    if (kFast) {
        const float den = __builtin_amdgcn_sqrtf(v > 0x1p-126f ? v : 0x1p-126f) * c.rbc2 + c.eps;
        p = p - (c.decay * p + c.step * (m * __builtin_amdgcn_rcpf(den)));
    } else {
        const float den = __builtin_sqrtf(v) * c.rbc2 + c.eps;
        p = p - (c.decay * p + c.step * (m / den));
    }
}

template <int G, int S>
struct TileIn {
    typename Four<typename Type<G>::elem>::vec g[kGroups];
    f32x4 p[kGroups];
    typename Four<typename Type<S>::elem>::vec m[kGroups], v[kGroups];
    int ms[kGroups], vs[kGroups];
};

template <int G, int S, bool kWhole>
__device__ __forceinline__ void load_tile(const TensorRec& r, const Extent& x, int lane, TileIn<G, S>& t) {
    typedef typename Type<G>::elem GT;
    typedef typename Type<S>::elem ST;
    const GT* g = tile_at<GT>(r.grad, x.base);
    const float* p = tile_at<float>(r.p, x.base);
    const ST *m = tile_at<ST>(r.m, x.base), *v = tile_at<ST>(r.v, x.base);
    Global<const uint8_t>* ms = (Global<const uint8_t>*)tile_at<uint8_t>(r.m_scale, x.base / ZERO_STATE_BLOCK);
    Global<const uint8_t>* vs = (Global<const uint8_t>*)tile_at<uint8_t>(r.v_scale, x.base / ZERO_STATE_BLOCK);
#pragma unroll
    for (int h = 0; h < kGroups; ++h) {
        const uint32_t q = h * 256 + 4 * lane;
        int b = int(q);   // an element of the lane's block (a tile starts with a block)
        t.g[h] = {};
        t.p[h] = {};
        t.m[h] = {};
        t.v[h] = {};
        t.ms[h] = t.vs[h] = 1;
        if (x.without<kWhole>(h)) break;
        if (x.with<kWhole>(h)) {
            t.g[h] = load4(g, q);
            t.p[h] = load4(p, q);
            t.m[h] = load4(m, q);
            t.v[h] = load4(v, q);
        } else {
            int at[4];
            x.nearest(q, at);
            b = at[0];
            const Part n = x.part<kWhole>(q);
            const Edge<GT> ge = edge_load(g, at);
            const Edge<float> pe = edge_load(p, at);
            const Edge<ST> me = edge_load(m, at), ve = edge_load(v, at);
            t.g[h] = edge_pack(ge, n);
            t.p[h] = edge_pack(pe, n);
            t.m[h] = edge_pack(me, n);
            t.v[h] = edge_pack(ve, n);
        }
        if constexpr (S == ZERO_DTYPE_MXFP8) {
            t.ms[h] = ms[b / ZERO_STATE_BLOCK];
            t.vs[h] = vs[b / ZERO_STATE_BLOCK];
        }
    }
}

template <int O>
__device__ __forceinline__ u16x4 narrow4(const float p[4]) {
    return u16x4{Type<O>::narrow(p[0]), Type<O>::narrow(p[1]), Type<O>::narrow(p[2]), Type<O>::narrow(p[3])};
}

// ---- results that leave through LDS ----------------------------------------

// A block's results of one array, wave w's tile from w kSetTile elements on, and
// 16 bytes past the end for the reads of whole vectors.
template <int BYTES>
struct Staged {
    u32x4 v[kWaves * kSetTile * BYTES / 16 + 1];
};

// How a wave's tile hangs together with its block's others: whether the wave
// before (after) it has the tile before (after) it of the same tensor, and how
// many elements that one after it has.
struct Chain {
    bool before, after;
    int next;
};
__device__ __forceinline__ Chain chain(const SetLaunch& a, const TileRec& tile, const TensorRec& r, const Extent& x) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t w = int64_t(blockIdx.x) * kWaves + wave;
    Chain c;
    c.before = wave > 0 && a.tile[w - 1].tensor == tile.tensor;
    c.after = wave < kWaves - 1 && w + 1 < a.n_tiles && a.tile[w + 1].tensor == tile.tensor;
    const int64_t left = r.numel - x.base - kSetTile;
    c.next = left >= kSetTile ? int(kSetTile) : left > 0 ? int(left) : 0;
    return c;
}

// The step of 200 M elements in 8 bits reads 3 and writes 0.2% more than it must
// this way and takes 556 to 588 us against 546 on lines; six blocks of 24 KB of
// LDS fit a CU, as many waves as the registers allow.
//
// A wave's tile, from the block's staged results to memory; `at` is where its
// element 0 belongs (maybe outside the tensor).  Lane l takes the aligned 16
// bytes l of each KiB, so a line is written whole by one instruction; where
// the tile's neighbours are in the block too, the wave takes the lines that
// begin in its tile, and only the ends of the block's run are left unfinished.
// (Each wave to its own ends: 648 us for 200 M elements one element off the
// lines, and 582 us sixteen off.)  A vector is cut out of two staged ones;
// the cut is the same for all lanes.
//
// `vec(c)` is the vector of the tile's bytes c .. c + 15, `one(k)` its
// element k.
template <typename T, typename Vec, typename One>
__device__ __forceinline__ void store_run(uintptr_t at, const Extent& x, const Chain& link, Vec vec, One one) {
    constexpr int kSize = int(sizeof(T)), kBytes = int(kSetTile) * kSize;
    const int mis = int(at & uintptr_t(kLine - 1)), begins = (kLine - mis) & (kLine - 1);   // the first line that begins in the tile
    const int lo = link.before ? begins : x.lo * kSize;
    const int to_next = begins < link.next * kSize ? begins : link.next * kSize;
    const int hi = link.after && x.hi == int(kSetTile) ? kBytes + to_next : x.hi * kSize;
    for (int c = (link.before ? begins : -mis) + int(threadIdx.x & 63) * 16; c < hi; c += 1024) {
        if (c >= lo && c + 16 <= hi) {
            __builtin_nontemporal_store(vec(c), (Global<u32x4>*)(at + uintptr_t(int64_t(c))));
        } else if (c + 16 > lo) {
            Global<T>* to = (Global<T>*)(at + uintptr_t(int64_t(c)));
#pragma unroll
            for (int k = 0; k < 16 / kSize; ++k)
                if (c + k * kSize >= lo && c + k * kSize < hi) to[k] = one(c / kSize + k);
        }
    }
}

// This wave's tile in staged results.
template <int BYTES>
__device__ __forceinline__ const u32x4* staged_tile(const Staged<BYTES>& s) {
    return s.v + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * int(kSetTile * BYTES / 16);
}

__device__ __forceinline__ void store_codes(const Staged<1>& staged, const void* codes, const Extent& x, const Chain& link) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(codes) + uintptr_t(x.base);
    const u32x4* s = staged_tile(staged);
    const int cut = int(-at & 15u);
    store_run<uint8_t>(at, x, link, [&](int c) {
        const u32x4 a = s[(c - cut) / 16], b = s[(c - cut) / 16 + 1];
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        const auto take = [&](int d) {
            return u32x4{__builtin_amdgcn_alignbyte(w[d + 1], w[d], cut & 3), __builtin_amdgcn_alignbyte(w[d + 2], w[d + 1], cut & 3),
                         __builtin_amdgcn_alignbyte(w[d + 3], w[d + 2], cut & 3), __builtin_amdgcn_alignbyte(w[d + 4], w[d + 3], cut & 3)};
        };
        switch (cut >> 2) {
            case 0: return take(0);
            case 1: return take(1);
            case 2: return take(2);
            default: return take(3);
        }
    }, [&](int k) { return reinterpret_cast<const uint8_t*>(s)[k]; });
}

__device__ __forceinline__ u32x4 four_of(const u32x4& a, const u32x4& b, int cut) {   // words cut .. cut + 3 of the eight
    switch (cut) {
        case 0: return a;
        case 1: return u32x4{a.y, a.z, a.w, b.x};
        case 2: return u32x4{a.z, a.w, b.x, b.y};
        default: return u32x4{a.w, b.x, b.y, b.z};
    }
}

__device__ __forceinline__ void store_p(const Staged<4>& staged, const void* p, const Extent& x, const Chain& link) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p) + uintptr_t(x.base * 4);
    const u32x4* s = staged_tile(staged);
    const int cut = int(-at & 15u);
    store_run<uint32_t>(at, x, link, [&](int c) { return four_of(s[(c - cut) / 16], s[(c - cut) / 16 + 1], cut / 4); },
                        [&](int k) { return reinterpret_cast<const uint32_t*>(s)[k]; });
}

// The 16-bit copies, from the staged p: they need no stage of their own, which
// leaves room for six blocks on a CU instead of four.
template <int O>
__device__ __forceinline__ void store_out(const Staged<4>& staged, const void* out, const Extent& x, const Chain& link) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(out) + uintptr_t(x.base * 2);
    const u32x4* s = staged_tile(staged);
    const int cut = int(-at & 7u) / 2;   // element c / 2 less its place in an aligned four
    store_run<uint16_t>(at, x, link, [&](int c) {
        const int q = (c / 2 - cut) / 4;
        const u32x4 mid = s[q + 1];
        const f32x4 a = __builtin_bit_cast(f32x4, four_of(s[q], mid, cut)), b = __builtin_bit_cast(f32x4, four_of(mid, s[q + 2], cut));
        const float lo[4] = {a.x, a.y, a.z, a.w}, hi[4] = {b.x, b.y, b.z, b.w};
        const u32x2 l = __builtin_bit_cast(u32x2, narrow4<O>(lo)), h = __builtin_bit_cast(u32x2, narrow4<O>(hi));
        return u32x4{l.x, l.y, h.x, h.y};
    }, [&](int k) { return Type<O>::narrow(reinterpret_cast<const float*>(s)[k]); });
}

struct StepStage {
    Staged<4> p;
    Staged<1> m, v;
};
struct NoStage {};

template <int G, int O, int S, bool kWhole, bool kStaged, bool kRandomM, typename Stage>
__device__ __forceinline__ void step_tile(const TensorRec& r, const Consts& c, float mult, uint32_t key, const Extent& x,
                                          int lane, Stage* stage) {
    const uint32_t own = kStaged ? (threadIdx.x >> 6) * uint32_t(kSetTile) : 0u;   // the wave's place in the stage
    typedef typename Type<S>::elem ST;
    TileIn<G, S> t;
    load_tile<G, S, kWhole>(r, x, lane, t);
    float* po = tile_at<float>(r.p, x.base);
    ST *mo = tile_at<ST>(r.m, x.base), *vo = tile_at<ST>(r.v, x.base);
    uint16_t* oo = tile_at<uint16_t>(r.out, x.base);
    Global<uint8_t>* ms_out = (Global<uint8_t>*)tile_at<uint8_t>(r.m_scale, x.base / ZERO_STATE_BLOCK);
    Global<uint8_t>* vs_out = (Global<uint8_t>*)tile_at<uint8_t>(r.v_scale, x.base / ZERO_STATE_BLOCK);
    // random bits of two elements: of v, and of m by a key of its own
    const uint32_t pair0 = uint32_t(x.base >> 1) + key, m_pair0 = uint32_t(x.base >> 1) + mix32(~key);
#pragma unroll
    for (int h = 0; h < kGroups; ++h) {
        if (x.without<kWhole>(h)) break;
        const uint32_t q = h * 256 + 4 * lane;
        const Part n = x.part<kWhole>(q);
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
        for (int k = 0; k < 4; ++k)
            adamw_element<S == ZERO_DTYPE_MXFP8>(c, Type<G>::wide(t.g[h][k]) * mult, p[k], m[k], v[k]);
        if constexpr (S == ZERO_DTYPE_MXFP8) {
            // every lane takes part in its block's maxima, with zeros for
            // elements that are not there
            if (!kWhole)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (!n.has(k)) m[k] = v[k] = 0.0f;
            const uint32_t r0 = mix32(pair0 + (q >> 1)), r1 = mix32(pair0 + (q >> 1) + 1);
            const uint32_t m0 = kRandomM ? mix32(m_pair0 + (q >> 1)) : 0u, m1 = kRandomM ? mix32(m_pair0 + (q >> 1) + 1) : 0u;
            int ms, vs;
            const uint32_t mc = encode_m<kRandomM>(m, m0, m1, &ms), vc = encode_v<true>(v, r0, r1, &vs);
            if (!n.none() && (lane & 7) == 0) {
                ms_out[q / ZERO_STATE_BLOCK] = uint8_t(ms);
                vs_out[q / ZERO_STATE_BLOCK] = uint8_t(vs);
            }
            if constexpr (kStaged) {
                reinterpret_cast<uint32_t*>(stage->m.v)[(own + q) / 4] = mc;
                reinterpret_cast<uint32_t*>(stage->v.v)[(own + q) / 4] = vc;
                stage->p.v[(own + q) / 4] = __builtin_bit_cast(u32x4, f32x4{p[0], p[1], p[2], p[3]});
                continue;
            }
            if (n.none()) continue;
            store4(mo, q, mc, n);
            store4(vo, q, vc, n);
        } else {
            if (n.none()) continue;
            store4(mo, q, f32x4{m[0], m[1], m[2], m[3]}, n);
            store4(vo, q, f32x4{v[0], v[1], v[2], v[3]}, n);
        }
        store4(po, q, f32x4{p[0], p[1], p[2], p[3]}, n);
        if constexpr (O != ZERO_DTYPE_NONE) store4(oo, q, narrow4<O>(p), n);
    }
}

// The tile of this wave, the same in all its lanes; false past the last one.
__device__ __forceinline__ bool wave_tile(const SetLaunch& a, TileRec* tile) {
    const int64_t w = int64_t(blockIdx.x) * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (w >= a.n_tiles) return false;
    *tile = a.tile[w];
    return true;
}

// m in 8 bits is rounded to nearest where that lets it decay: the codes' worst
// case is 1.125, which times beta1 has to come below 1.0625 to leave it.  Above,
// at random (or everywhere, when the set says so), which costs no time: 13B
// share, 200 M elements, 557 us either way.
template <int G, int O, int S, bool kStaged, typename Stage>
__device__ __forceinline__ void step_wave(const zero_step_control* __restrict__ ctl, const TensorRec& r, const Extent& x,
                                          bool random_m, Stage* stage) {
    const Consts c = *reinterpret_cast<const Consts*>(ctl->group[r.group]);
    const float mult = ctl->grad_mult;
    const uint32_t key = mix32(r.key + uint32_t(ctl->t) * 0x9E3779B9u);
    const int lane = threadIdx.x & 63;
    if constexpr (S == ZERO_DTYPE_MXFP8)
        if (random_m || c.beta1 > ZERO_NEAREST_BETA1) {
            if (x.whole()) step_tile<G, O, S, true, kStaged, true>(r, c, mult, key, x, lane, stage);
            else step_tile<G, O, S, false, kStaged, true>(r, c, mult, key, x, lane, stage);
            return;
        }
    if (x.whole()) step_tile<G, O, S, true, kStaged, false>(r, c, mult, key, x, lane, stage);
    else step_tile<G, O, S, false, kStaged, false>(r, c, mult, key, x, lane, stage);
}

template <int G, int O, int S>
__global__ __launch_bounds__(kThreads) void adamw_kernel(const SetLaunch a, const zero_step_control* __restrict__ ctl) {
    TileRec tile;
    if (!wave_tile(a, &tile) || ctl->skip) return;
    const TensorRec r = a.rec[tile.tensor];
    const Extent x = extent(r, tile.tile, S == ZERO_DTYPE_MXFP8 ? block_shift(r) : tile_shift(r.p, 4, r.spare));
    if (x.hi == 0) return;   // a tile counted for another array's shift
    NoStage* none = nullptr;
    step_wave<G, O, S, false>(ctl, r, x, a.random_m, none);
}

// For sets with MXFP8 states of which some tensors' tiles are not stored
// straight.
template <int G, int O>
__global__ __launch_bounds__(kThreads) void adamw_staged_kernel(const SetLaunch a, const zero_step_control* __restrict__ ctl) {
    __shared__ StepStage stage;
    const int skip = ctl->skip;
    TileRec tile = {};
    TensorRec r = {};
    Extent x = {0, 0, 0};
    Chain link = {};
    bool staged = false;
    const bool any = wave_tile(a, &tile);
    if (skip) return;   // the same for every wave
    if (any) {
        r = a.rec[tile.tensor];
        x = extent(r, tile.tile, block_shift(r));
        link = chain(a, tile, r, x);
        staged = x.hi > 0 && !step_direct(r);
        if (staged) step_wave<G, O, ZERO_DTYPE_MXFP8, true>(ctl, r, x, a.random_m, &stage);
        else if (x.hi > 0) step_wave<G, O, ZERO_DTYPE_MXFP8, false>(ctl, r, x, a.random_m, &stage);
    }
    __syncthreads();
    if (!staged) return;
    store_p(stage.p, r.p, x, link);
    if constexpr (O != ZERO_DTYPE_NONE) store_out<O>(stage.p, r.out, x, link);
    store_codes(stage.m, r.m, x, link);
    store_codes(stage.v, r.v, x, link);
}

// ---------------------------------------------------------------------------
// state conversion
// ---------------------------------------------------------------------------

struct CodeStage {
    Staged<1> m, v;
};

// A tile of both states.
template <typename T, bool kWhole>
__device__ __forceinline__ void load_states(const TensorRec& from, const Extent& x, int lane, typename Four<T>::vec m[kGroups],
                                            typename Four<T>::vec v[kGroups]) {
    const T *pm = tile_at<T>(from.m, x.base), *pv = tile_at<T>(from.v, x.base);
#pragma unroll
    for (int h = 0; h < kGroups; ++h) {
        const uint32_t q = h * 256 + 4 * lane;
        m[h] = v[h] = {};
        if (x.without<kWhole>(h)) break;
        if (x.with<kWhole>(h)) {
            m[h] = load4(pm, q);
            v[h] = load4(pv, q);
        } else {
            int at[4];
            x.nearest(q, at);
            const Edge<T> me = edge_load(pm, at), ve = edge_load(pv, at);
            m[h] = edge_pack(me, x.part<kWhole>(q));
            v[h] = edge_pack(ve, x.part<kWhole>(q));
        }
    }
}

template <bool kWhole>
__device__ __forceinline__ void encode_tile(const TensorRec& to, const TensorRec& from, const Extent& x, int lane,
                                            CodeStage* stage) {
    uint8_t *cm = tile_at<uint8_t>(to.m, x.base), *cv = tile_at<uint8_t>(to.v, x.base);
    Global<uint8_t>* ms_out = (Global<uint8_t>*)tile_at<uint8_t>(to.m_scale, x.base / ZERO_STATE_BLOCK);
    Global<uint8_t>* vs_out = (Global<uint8_t>*)tile_at<uint8_t>(to.v_scale, x.base / ZERO_STATE_BLOCK);
    f32x4 m4[kGroups], v4[kGroups];
    load_states<float, kWhole>(from, x, lane, m4, v4);
#pragma unroll
    for (int h = 0; h < kGroups; ++h) {
        if (x.without<kWhole>(h)) break;
        const uint32_t q = h * 256 + 4 * lane;
        const Part n = x.part<kWhole>(q);
        const float m[4] = {m4[h].x, m4[h].y, m4[h].z, m4[h].w}, v[4] = {v4[h].x, v4[h].y, v4[h].z, v4[h].w};
        int ms, vs;
        const uint32_t mc = encode_m<false>(m, 0, 0, &ms), vc = encode_v<false>(v, 0, 0, &vs);
        if (!n.none() && (lane & 7) == 0) {
            ms_out[q / ZERO_STATE_BLOCK] = uint8_t(ms);
            vs_out[q / ZERO_STATE_BLOCK] = uint8_t(vs);
        }
        if (stage) {
            const uint32_t own = (threadIdx.x >> 6) * uint32_t(kSetTile);
            reinterpret_cast<uint32_t*>(stage->m.v)[(own + q) / 4] = mc;
            reinterpret_cast<uint32_t*>(stage->v.v)[(own + q) / 4] = vc;
        } else if (!n.none()) {
            store4(cm, q, mc, n);
            store4(cv, q, vc, n);
        }
    }
}

__device__ __forceinline__ void encode_wave(const TensorRec& to, const TensorRec& from, const Extent& x, CodeStage* stage) {
    const int lane = threadIdx.x & 63;
    if (x.whole()) encode_tile<true>(to, from, x, lane, stage);
    else encode_tile<false>(to, from, x, lane, stage);
}

template <bool kStaged>
__global__ __launch_bounds__(kThreads) void encode_kernel(const SetLaunch dst, const TensorRec* __restrict__ src) {
    TileRec tile = {};
    TensorRec to = {};
    Extent x = {0, 0, 0};
    if (wave_tile(dst, &tile)) {
        to = dst.rec[tile.tensor];
        x = extent(to, tile.tile, block_shift(to));
    }
    if constexpr (kStaged) {
        __shared__ CodeStage stage;
        const bool staged = x.hi > 0 && !codes_direct(to);
        if (x.hi > 0) encode_wave(to, src[tile.tensor], x, staged ? &stage : nullptr);
        __syncthreads();
        if (!staged) return;
        const Chain link = chain(dst, tile, to, x);
        store_codes(stage.m, to.m, x, link);
        store_codes(stage.v, to.v, x, link);
    } else if (x.hi > 0) {
        encode_wave(to, src[tile.tensor], x, nullptr);
    }
}

// Decoding follows the fp32 arrays' lines, so a lane's four elements (the first
// of them element e of the tensor) may belong to two blocks.
__device__ __forceinline__ f32x4 decode_across(uint32_t code, const uint8_t* scale, int64_t e, Part n) {
    const int64_t b0 = (e + n.a) / ZERO_STATE_BLOCK, b1 = (e + n.b - 1) / ZERO_STATE_BLOCK;
    const float f0 = scale_value(((Global<const uint8_t>*)scale)[b0]), f1 = scale_value(((Global<const uint8_t>*)scale)[b1]);
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(int(code), false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(int(code), true);
    f32x4 x = {lo.x, lo.y, hi.x, hi.y};
    const int first = int((b0 + 1) * ZERO_STATE_BLOCK - e);   // the second block's first element, if it is one of the four
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = x[k] * (k < first ? f0 : f1);
    return x;
}

template <bool kWhole>
__device__ __forceinline__ void decode_tile(const TensorRec& to, const TensorRec& from, const Extent& x, int lane) {
    float *wm = tile_at<float>(to.m, x.base), *wv = tile_at<float>(to.v, x.base);
    uint32_t mc[kGroups], vc[kGroups];
    load_states<uint8_t, kWhole>(from, x, lane, mc, vc);
#pragma unroll
    for (int h = 0; h < kGroups; ++h) {
        const uint32_t q = h * 256 + 4 * lane;
        const Part n = x.part<kWhole>(q);
        if (x.without<kWhole>(h) || n.none()) continue;
        store4(wm, q, decode_across(mc[h], from.m_scale, x.base + q, n), n);
        store4(wv, q, decode_across(vc[h], from.v_scale, x.base + q, n), n);
    }
}

__global__ __launch_bounds__(kThreads) void decode_kernel(const SetLaunch dst, const TensorRec* __restrict__ src) {
    TileRec tile;
    if (!wave_tile(dst, &tile)) return;
    const TensorRec to = dst.rec[tile.tensor], from = src[tile.tensor];
    const Extent x = extent(to, tile.tile, tile_shift(to.m, 4, to.spare));
    if (x.hi == 0) return;
    const int lane = threadIdx.x & 63;
    if (x.whole()) decode_tile<true>(to, from, x, lane);
    else decode_tile<false>(to, from, x, lane);
}

dim3 tile_grid(int64_t n_tiles) { return dim3(unsigned((n_tiles + kWaves - 1) / kWaves)); }

template <int G, int O>
void run_adamw(const SetLaunch& a, const zero_step_control* ctl, dim3 grid, hipStream_t s, const KernelEvents& ev) {
    if (a.state_type == ZERO_DTYPE_FP32) launch(adamw_kernel<G, O, ZERO_DTYPE_FP32>, grid, kThreads, s, ev, a, ctl);
    else if (a.staged_step) launch(adamw_staged_kernel<G, O>, grid, kThreads, s, ev, a, ctl);
    else launch(adamw_kernel<G, O, ZERO_DTYPE_MXFP8>, grid, kThreads, s, ev, a, ctl);
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
    const dim3 grid = tile_grid(dst.n_tiles);
    if (dst.state_type == ZERO_DTYPE_FP32) launch(decode_kernel, grid, kThreads, stream, ev, dst, src.rec);
    else if (dst.staged_codes) launch(encode_kernel<true>, grid, kThreads, stream, ev, dst, src.rec);
    else launch(encode_kernel<false>, grid, kThreads, stream, ev, dst, src.rec);
    return hipGetLastError();
}

}  // namespace zp
