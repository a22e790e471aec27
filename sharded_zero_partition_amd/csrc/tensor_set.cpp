// tensor_set.cpp -- tensor sets: argument checks, device tables and the C ABI
// of the gradient norm, the AdamW step and the state conversion (host only).
//
// A ZeRO rank updates only its own partition of the parameters (Stage 1
// paragraph of the ZeRO explainer page, "ZeRO: Memory Optimizations Toward
// Training Trillion Parameter Models", azimuth.plus); a set names that
// partition as tensors, or pieces of tensors, rather than as one flat shard, so
// parameter groups and states in 8 bits follow tensor boundaries.  AdamW's
// decoupled decay, clipping and 8-bit states are not on the page.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <memory>
#include <new>
#include <utility>

#include "tensor_set.hpp"

struct zero_tensor_set {
    int device = -1;
    int32_t grad_type = ZERO_DTYPE_NONE;
    int32_t state_type = ZERO_DTYPE_NONE;
    int32_t out_type = ZERO_DTYPE_NONE;
    bool has_p = false;
    bool has_grads = false;
    bool staged_step = false;
    bool staged_codes = false;
    bool random_m = false;
    int32_t max_group = 0;
    int64_t n_tiles = 0;
    int64_t n_norm_tiles = 0;
    std::vector<int64_t> numel;              // as given, empty tensors too
    std::vector<zp::TensorRec> rec;          // host copy of the device records (non-empty tensors)
    zp::TensorRec* d_rec = nullptr;          // one allocation: the records, the tiles, the norm's tiles
    zp::TileRec* d_tile = nullptr;
    zp::TileRec* d_norm_tile = nullptr;      // d_tile where no tensor has one more there
    // byte ranges of the arrays that a step or a conversion writes, sorted;
    // they are disjoint
    std::vector<std::pair<uintptr_t, uintptr_t>> written;
    std::vector<std::pair<uintptr_t, uintptr_t>> states;   // those of the states among them, sorted
};

namespace zp {

// Events for a timed call; none while its stream is being captured (a graph's
// nodes carry no events of one call).
hipError_t set_events(hipStream_t s, KernelEvents* ev, bool* timed) {
    *timed = false;
    hipError_t e = timing_events(ev);
    if (e != hipSuccess || !ev->start) return e;
    hipStreamCaptureStatus status = hipStreamCaptureStatusNone;
    e = hipStreamIsCapturing(s, &status);
    if (e != hipSuccess) return e;
    if (status != hipStreamCaptureStatusNone) {
        *ev = KernelEvents();   // the pair stays open: the next timed call takes it
        return hipSuccess;
    }
    *timed = true;
    return hipSuccess;
}

namespace {

int dtype_bytes(int32_t t) {
    switch (t) {
        case ZERO_DTYPE_FP16: return 2;
        case ZERO_DTYPE_BF16: return 2;
        case ZERO_DTYPE_FP32: return 4;
        case ZERO_DTYPE_MXFP8: return 1;
        default: return 0;
    }
}

bool is_aligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % uintptr_t(bytes) == 0; }

int64_t scale_bytes(int64_t numel) { return (numel - 1) / ZERO_STATE_BLOCK + 1; }   // numel > 0

typedef std::vector<std::pair<uintptr_t, uintptr_t>> Ranges;

// Appends [p, p + n * width); false when it leaves the address space.
bool add_range(Ranges* r, const void* p, int64_t n, int width) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    if (uint64_t(n) > (UINTPTR_MAX - lo) / uint64_t(width)) return false;
    r->push_back({lo, lo + uintptr_t(n) * uintptr_t(width)});
    return true;
}

// Whether [lo, hi) meets one of the sorted, disjoint ranges.
bool meets(const Ranges& sorted, uintptr_t lo, uintptr_t hi) {
    const auto it = std::lower_bound(sorted.begin(), sorted.end(), std::make_pair(hi, uintptr_t(0)));
    return it != sorted.begin() && std::prev(it)->second > lo;   // the last range that starts below hi
}

// Whether two lists of sorted, disjoint ranges meet.
bool lists_meet(const Ranges& a, const Ranges& b) {
    for (size_t i = 0, j = 0; i < a.size() && j < b.size();) {
        if (a[i].second <= b[j].first) ++i;
        else if (b[j].second <= a[i].first) ++j;
        else return true;
    }
    return false;
}

// Checks of one gradient address against the set's written arrays.
int check_grad(const void* g, int64_t numel, int32_t grad_type, const Ranges& written) {
    const int w = dtype_bytes(grad_type);
    if (!is_aligned(g, w)) return fail(ZERO_ERR_ALIGNMENT, "a gradient lacks its element's alignment");
    const uintptr_t lo = reinterpret_cast<uintptr_t>(g);
    if (uint64_t(numel) > (UINTPTR_MAX - lo) / uint64_t(w))
        return fail(ZERO_ERR_INDEX_OVERFLOW, "a gradient's end is outside the address space");
    if (meets(written, lo, lo + uintptr_t(numel) * uintptr_t(w)))
        return fail(ZERO_ERR_INVALID_ARG, "a gradient overlaps an array that a step writes");
    return ZERO_OK;
}

// Device of a call on `set`: the current one, which must be the set's and the
// stream's.
int check_set_device(const zero_tensor_set* set, void* stream, const char* who) {
    int dev = 0;
    const hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return fail_hip(e, "hipGetDevice");
    if (dev != set->device) return fail(ZERO_ERR_STATE, std::string(who) + ": the set was made on another device");
    return check_stream_device(stream, dev, who);
}

// Uploads wait for their stream, which one that is being captured cannot.
int check_not_capturing(void* stream, const char* who) {
    hipStreamCaptureStatus status = hipStreamCaptureStatusNone;
    const hipError_t e = hipStreamIsCapturing(static_cast<hipStream_t>(stream), &status);
    if (e != hipSuccess) return fail_hip(e, "hipStreamIsCapturing");
    if (status != hipStreamCaptureStatusNone)
        return fail(ZERO_ERR_STATE, std::string(who) + ": not possible while the stream is being captured");
    return ZERO_OK;
}

// Takes the calling thread out of the capture mode in which calls that allocate,
// free or wait are refused while any stream of the process is being captured:
// these concern the sets' own tables alone, which no other capture holds.
class OutsideCaptures {
public:
    OutsideCaptures() { (void)hipThreadExchangeStreamCaptureMode(&mode_); }
    ~OutsideCaptures() { (void)hipThreadExchangeStreamCaptureMode(&mode_); }
    OutsideCaptures(const OutsideCaptures&) = delete;
    OutsideCaptures& operator=(const OutsideCaptures&) = delete;

private:
    hipStreamCaptureMode mode_ = hipStreamCaptureModeRelaxed;
};

SetLaunch set_launch(const zero_tensor_set* s) {
    return SetLaunch{s->d_rec, s->d_tile, s->n_tiles, s->d_norm_tile, s->n_norm_tiles, s->grad_type, s->state_type, s->out_type,
                     s->staged_step, s->staged_codes, s->random_m};
}

int create(const zero_tensor* tensors, int64_t n, int32_t grad_type, int32_t state_type, int32_t out_type,
           uint32_t seed, void* stream, zero_tensor_set** out) {
    if (!out) return fail(ZERO_ERR_INVALID_ARG, "zero_tensor_set_create: out is NULL");
    if (n < 0 || (n > 0 && !tensors)) return fail(ZERO_ERR_INVALID_ARG, "zero_tensor_set_create: no tensors");
    if (grad_type < ZERO_DTYPE_NONE || grad_type > ZERO_DTYPE_FP32)
        return fail(ZERO_ERR_INVALID_ARG, "grad_type must be FP16, BF16, FP32 or NONE");
    if (state_type != ZERO_DTYPE_NONE && state_type != ZERO_DTYPE_FP32 && state_type != ZERO_DTYPE_MXFP8)
        return fail(ZERO_ERR_INVALID_ARG, "state_type must be FP32, MXFP8 or NONE");
    if (out_type != ZERO_DTYPE_NONE && out_type != ZERO_DTYPE_FP16 && out_type != ZERO_DTYPE_BF16)
        return fail(ZERO_ERR_INVALID_ARG, "out_type must be FP16, BF16 or NONE");

    std::unique_ptr<zero_tensor_set> set(new zero_tensor_set());
    set->grad_type = grad_type;
    set->state_type = state_type;
    set->out_type = out_type;
    set->numel.reserve(size_t(n));
    int64_t first = -1;
    for (int64_t i = 0; i < n; ++i) {
        const zero_tensor& t = tensors[i];
        if (t.numel < 0) return fail(ZERO_ERR_INVALID_ARG, "a tensor's size is negative");
        if (t.group < 0 || t.group >= ZERO_MAX_GROUPS) return fail(ZERO_ERR_INVALID_ARG, "a tensor's group is outside 0..15");
        set->numel.push_back(t.numel);
        if (t.numel == 0) continue;
        if (first < 0) {
            first = i;
            set->has_p = t.p != nullptr;
            set->has_grads = t.grad != nullptr;
        }
        if ((t.p != nullptr) != set->has_p) return fail(ZERO_ERR_INVALID_ARG, "all tensors or none have p");
        if ((t.grad != nullptr) != set->has_grads) return fail(ZERO_ERR_INVALID_ARG, "all tensors or none have a gradient");
        if (t.grad && grad_type == ZERO_DTYPE_NONE) return fail(ZERO_ERR_INVALID_ARG, "a gradient without grad_type");
        const bool st = state_type != ZERO_DTYPE_NONE, mx = state_type == ZERO_DTYPE_MXFP8;
        if ((t.m != nullptr) != st || (t.v != nullptr) != st)
            return fail(ZERO_ERR_INVALID_ARG, "m and v are set exactly when state_type is");
        if ((t.m_scale != nullptr) != mx || (t.v_scale != nullptr) != mx)
            return fail(ZERO_ERR_INVALID_ARG, "m_scale and v_scale are set exactly when state_type is MXFP8");
        if ((t.out != nullptr) != (out_type != ZERO_DTYPE_NONE))
            return fail(ZERO_ERR_INVALID_ARG, "out is set exactly when out_type is");
        if (t.out && !t.p) return fail(ZERO_ERR_INVALID_ARG, "out without p");
        const int sw = dtype_bytes(state_type);
        if (t.p && !is_aligned(t.p, 4)) return fail(ZERO_ERR_ALIGNMENT, "p is not 4-byte aligned");
        if (st && (!is_aligned(t.m, sw) || !is_aligned(t.v, sw)))
            return fail(ZERO_ERR_ALIGNMENT, "a state lacks its element's alignment");
        if (t.out && !is_aligned(t.out, 2)) return fail(ZERO_ERR_ALIGNMENT, "out is not 2-byte aligned");
        if (t.numel > kMaxSetTiles * kSetTile) return fail(ZERO_ERR_OUT_OF_MEMORY, "more than 2^25 tiles of 1024 elements");
        // the arrays that a step or a conversion writes come first; the tiles
        // reach the end with any of their shifts
        int64_t shift = 0;
        const uint32_t any = uint32_t(kSetTile);
        if (t.p) shift = tile_shift(t.p, 4, any);
        if (state_type == ZERO_DTYPE_FP32) shift = std::max<int64_t>(shift, tile_shift(t.m, 4, any));
        if (mx) shift = ((reinterpret_cast<uintptr_t>(t.p) / 4) | reinterpret_cast<uintptr_t>(t.m)) & 32;
        const int64_t tiles = (t.numel + shift - 1) / kSetTile + 1;
        if (tiles > kMaxSetTiles - set->n_tiles) return fail(ZERO_ERR_OUT_OF_MEMORY, "more than 2^25 tiles of 1024 elements");
        set->n_tiles += tiles;
        set->n_norm_tiles += (t.numel - 1) / kSetTile + 1;
        set->max_group = std::max(set->max_group, t.group);
        bool ok = true;
        if (t.p) ok = ok && add_range(&set->written, t.p, t.numel, 4);
        if (st) ok = ok && add_range(&set->states, t.m, t.numel, sw) && add_range(&set->states, t.v, t.numel, sw);
        if (mx)
            ok = ok && add_range(&set->states, t.m_scale, scale_bytes(t.numel), 1) &&
                 add_range(&set->states, t.v_scale, scale_bytes(t.numel), 1);
        if (t.out) ok = ok && add_range(&set->written, t.out, t.numel, 2);
        if (!ok) return fail(ZERO_ERR_INDEX_OVERFLOW, "an array's end is outside the address space");
        TensorRec r;
        std::memset(&r, 0, sizeof(r));
        r.p = t.p;
        r.grad = t.grad;
        r.m = t.m;
        r.v = t.v;
        r.m_scale = t.m_scale;
        r.v_scale = t.v_scale;
        r.out = t.out;
        r.numel = t.numel;
        r.key = mix32(mix32(seed) + uint32_t(i));
        r.group = t.group;
        r.spare = uint32_t(tiles * kSetTile - t.numel);
        if (mx) {
            set->staged_step |= !step_direct(r);
            set->staged_codes |= !codes_direct(r);
        }
        set->rec.push_back(r);
    }
    std::sort(set->states.begin(), set->states.end());
    set->written.insert(set->written.end(), set->states.begin(), set->states.end());
    std::sort(set->written.begin(), set->written.end());
    for (size_t k = 1; k < set->written.size(); ++k)
        if (set->written[k].first < set->written[k - 1].second)
            return fail(ZERO_ERR_INVALID_ARG, "two arrays that a step writes overlap");
    if (set->has_grads)
        for (const TensorRec& r : set->rec) {
            const int rc = check_grad(r.grad, r.numel, grad_type, set->written);
            if (rc != ZERO_OK) return rc;
        }
    std::vector<TileRec> tiles;
    const bool own_norm_tiles = grad_type != ZERO_DTYPE_NONE && set->n_norm_tiles != set->n_tiles;
    tiles.reserve(size_t(set->n_tiles + (own_norm_tiles ? set->n_norm_tiles : 0)));
    for (size_t k = 0; k < set->rec.size(); ++k)
        for (int64_t j = 0; j * kSetTile < set->rec[k].numel + set->rec[k].spare; ++j) tiles.push_back({uint32_t(k), uint32_t(j)});
    if (own_norm_tiles)
        for (size_t k = 0; k < set->rec.size(); ++k)
            for (int64_t j = 0; j * kSetTile < set->rec[k].numel; ++j) tiles.push_back({uint32_t(k), uint32_t(j)});

    hipError_t e = hipGetDevice(&set->device);
    if (e != hipSuccess) return fail_hip(e, "hipGetDevice");
    int rc = check_stream_device(stream, set->device, "zero_tensor_set_create");
    if (rc == ZERO_OK) rc = check_not_capturing(stream, "zero_tensor_set_create");
    if (rc != ZERO_OK) return rc;
    const size_t rec_bytes = set->rec.size() * sizeof(TensorRec), tile_bytes = tiles.size() * sizeof(TileRec);
    if (rec_bytes) {
        const OutsideCaptures guard;
        void* d = nullptr;
        e = hipMalloc(&d, rec_bytes + tile_bytes);
        if (e != hipSuccess) return fail_hip(e, "hipMalloc (tensor set)");
        set->d_rec = static_cast<TensorRec*>(d);
        set->d_tile = reinterpret_cast<TileRec*>(static_cast<uint8_t*>(d) + rec_bytes);
        set->d_norm_tile = set->d_tile + (own_norm_tiles ? set->n_tiles : 0);
        hipStream_t s = static_cast<hipStream_t>(stream);
        e = hipMemcpyAsync(set->d_rec, set->rec.data(), rec_bytes, hipMemcpyHostToDevice, s);
        if (e == hipSuccess) e = hipMemcpyAsync(set->d_tile, tiles.data(), tile_bytes, hipMemcpyHostToDevice, s);
        if (e == hipSuccess) e = hipStreamSynchronize(s);
        if (e != hipSuccess) {
            (void)hipFree(d);
            return fail_hip(e, "uploading the tensor set");
        }
    }
    *out = set.release();
    return ZERO_OK;
}

int bind_grads(zero_tensor_set* set, const void* const* grads, void* stream) {
    if (!set) return fail(ZERO_ERR_INVALID_ARG, "zero_tensor_set_bind_grads: set is NULL");
    if (set->grad_type == ZERO_DTYPE_NONE) return fail(ZERO_ERR_STATE, "the set has no grad_type");
    if (!set->rec.empty() && !grads) return fail(ZERO_ERR_INVALID_ARG, "grads is NULL");
    std::vector<TensorRec> rec = set->rec;
    size_t k = 0;
    for (size_t i = 0; i < set->numel.size(); ++i) {
        if (set->numel[i] == 0) continue;
        if (!grads[i]) return fail(ZERO_ERR_INVALID_ARG, "NULL gradient for a non-empty tensor");
        const int rc = check_grad(grads[i], set->numel[i], set->grad_type, set->written);
        if (rc != ZERO_OK) return rc;
        rec[k++].grad = grads[i];
    }
    int rc = check_set_device(set, stream, "zero_tensor_set_bind_grads");
    if (rc == ZERO_OK) rc = check_not_capturing(stream, "zero_tensor_set_bind_grads");
    if (rc != ZERO_OK) return rc;
    if (!rec.empty()) {
        const OutsideCaptures guard;
        hipStream_t s = static_cast<hipStream_t>(stream);
        hipError_t e = hipMemcpyAsync(set->d_rec, rec.data(), rec.size() * sizeof(TensorRec), hipMemcpyHostToDevice, s);
        if (e == hipSuccess) e = hipStreamSynchronize(s);
        if (e != hipSuccess) return fail_hip(e, "uploading the gradients' addresses");
    }
    set->rec.swap(rec);
    set->has_grads = !set->rec.empty();
    return ZERO_OK;
}

// What the set lacks of what a call needs, or NULL.
const char* lacks(const zero_tensor_set* s, bool p, bool grads, bool states) {
    if (s->rec.empty()) return nullptr;   // nothing to do
    if (p && !s->has_p) return "the set has no p";
    if (grads && !s->has_grads) return "the set's gradients are not bound";
    if (states && s->state_type == ZERO_DTYPE_NONE) return "the set has no states";
    return nullptr;
}

}  // namespace
}  // namespace zp

using zp::fail;

extern "C" int zero_tensor_set_create(const zero_tensor* tensors, int64_t n, int32_t grad_type, int32_t state_type,
                                      int32_t out_type, uint32_t seed, void* stream, zero_tensor_set** out) {
    zp::clear_error();
    try {
        return zp::create(tensors, n, grad_type, state_type, out_type, seed, stream, out);
    } catch (...) {
        return fail(ZERO_ERR_OUT_OF_MEMORY, "host table allocation failed");
    }
}

extern "C" int zero_tensor_set_destroy(zero_tensor_set* set) {
    zp::clear_error();
    if (set && set->d_rec) {
        const zp::OutsideCaptures guard;
        const hipError_t e = hipFree(set->d_rec);
        if (e != hipSuccess) return zp::fail_hip(e, "hipFree (tensor set)");
    }
    delete set;
    return ZERO_OK;
}

extern "C" int zero_tensor_set_m_rounding(zero_tensor_set* set, int32_t mode) {
    zp::clear_error();
    if (!set) return fail(ZERO_ERR_INVALID_ARG, "zero_tensor_set_m_rounding: set is NULL");
    if (mode != ZERO_M_ROUNDING_AUTO && mode != ZERO_M_ROUNDING_RANDOM)
        return fail(ZERO_ERR_INVALID_ARG, "the rounding of m must be AUTO or RANDOM");
    if (set->state_type != ZERO_DTYPE_MXFP8) return fail(ZERO_ERR_STATE, "the set's states are not MXFP8");
    set->random_m = mode == ZERO_M_ROUNDING_RANDOM;
    return ZERO_OK;
}

extern "C" int zero_tensor_set_bind_grads(zero_tensor_set* set, const void* const* grads, void* stream) {
    zp::clear_error();
    try {
        return zp::bind_grads(set, grads, stream);
    } catch (...) {
        return fail(ZERO_ERR_OUT_OF_MEMORY, "host table allocation failed");
    }
}

extern "C" int64_t zero_grad_sumsq_work_bytes(const zero_tensor_set* set) {
    if (!set) return 0;
    const int64_t blocks = zp::sumsq_blocks(set->n_norm_tiles);
    return blocks > 1 ? blocks * int64_t(sizeof(double)) : 0;
}

extern "C" int zero_grad_sumsq(const zero_tensor_set* set, double* sumsq, int32_t accumulate, void* work, void* stream) {
    zp::clear_error();
    if (!set || !sumsq) return fail(ZERO_ERR_INVALID_ARG, "zero_grad_sumsq: NULL set or sumsq");
    if (accumulate != 0 && accumulate != 1) return fail(ZERO_ERR_INVALID_ARG, "accumulate must be 0 or 1");
    if (!zp::is_aligned(sumsq, 8) || !zp::is_aligned(work, 8))
        return fail(ZERO_ERR_ALIGNMENT, "sumsq or work is not 8-byte aligned");
    const uintptr_t work_bytes = uintptr_t(zero_grad_sumsq_work_bytes(set));
    if (!work && work_bytes > 0) return fail(ZERO_ERR_INVALID_ARG, "work is NULL");
    const uintptr_t lo = reinterpret_cast<uintptr_t>(sumsq), wlo = reinterpret_cast<uintptr_t>(work);
    if (zp::meets(set->written, lo, lo + sizeof(*sumsq)) || (work_bytes > 0 && zp::meets(set->written, wlo, wlo + work_bytes)))
        return fail(ZERO_ERR_INVALID_ARG, "sumsq or work overlaps an array of the set");
    if (lo < wlo + work_bytes && wlo < lo + sizeof(*sumsq) && work_bytes > 0)
        return fail(ZERO_ERR_INVALID_ARG, "sumsq is inside work");
    if (const char* what = zp::lacks(set, false, true, false)) return fail(ZERO_ERR_STATE, what);
    const int rc = zp::check_set_device(set, stream, "zero_grad_sumsq");
    if (rc != ZERO_OK) return rc;
    hipStream_t s = static_cast<hipStream_t>(stream);
    zp::KernelEvents ev;
    bool timed = false;
    hipError_t e = zp::set_events(s, &ev, &timed);
    if (e != hipSuccess) return zp::fail_hip(e, "timing event");
    e = zp::launch_sumsq(zp::set_launch(set), sumsq, accumulate != 0, static_cast<double*>(work), s, ev);
    if (e != hipSuccess) return zp::fail_hip(e, "sum of squares kernel launch");
    if (timed) zp::timing_done();
    return ZERO_OK;
}

extern "C" int zero_step_begin(zero_step_control* ctl, const zero_adam_hparams* groups, int32_t n_groups, float max_norm,
                               int32_t check, const zero_loss_scaler* scaler, void* stream) {
    zp::clear_error();
    if (!ctl || !groups) return fail(ZERO_ERR_INVALID_ARG, "zero_step_begin: NULL control or groups");
    if (!zp::is_aligned(ctl, 8)) return fail(ZERO_ERR_ALIGNMENT, "the control block is not 8-byte aligned");
    if (n_groups < 1 || n_groups > ZERO_MAX_GROUPS) return fail(ZERO_ERR_INVALID_ARG, "n_groups must be in 1..16");
    if (check != 0 && check != 1) return fail(ZERO_ERR_INVALID_ARG, "check must be 0 or 1");
    if (!(max_norm >= 0.0f) || !std::isfinite(max_norm))
        return fail(ZERO_ERR_INVALID_ARG, "max_norm must be finite and not negative");
    if (!check && max_norm > 0.0f) return fail(ZERO_ERR_INVALID_ARG, "clipping needs check = 1");
    zp::BeginLaunch a;
    std::memset(&a, 0, sizeof(a));
    for (int32_t k = 0; k < n_groups; ++k) {
        const zero_adam_hparams& h = groups[k];
        if (!std::isfinite(h.lr) || !std::isfinite(h.eps) || !(h.eps > 0.0f) || !std::isfinite(h.weight_decay) ||
            !(h.beta1 >= 0.0f && h.beta1 < 1.0f) || !(h.beta2 >= 0.0f && h.beta2 < 1.0f))
            return fail(ZERO_ERR_INVALID_ARG, "invalid Adam hyper-parameters (finite; eps > 0; betas in [0, 1))");
        a.group[k] = h;
    }
    if (scaler) {
        if (!std::isfinite(scaler->min_scale) || !(scaler->min_scale >= ZERO_MIN_LOSS_SCALE))
            return fail(ZERO_ERR_INVALID_ARG, "min_scale must be finite and >= 2^-24");
        if (!std::isfinite(scaler->backoff) || !(scaler->backoff > 0.0f) || !std::isfinite(scaler->growth) ||
            !(scaler->growth > 0.0f) || scaler->growth_interval < 0)
            return fail(ZERO_ERR_INVALID_ARG, "invalid loss-scaler settings");
        a.scaler = 1;
        a.backoff = scaler->backoff;
        a.growth = scaler->growth;
        a.min_scale = scaler->min_scale;
        a.growth_interval = scaler->growth_interval;
    }
    a.ctl = ctl;
    a.n_groups = n_groups;
    a.check = check;
    a.max_norm = max_norm;
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return zp::fail_hip(e, "hipGetDevice");
    const int rc = zp::check_stream_device(stream, dev, "zero_step_begin");
    if (rc != ZERO_OK) return rc;
    e = zp::launch_step_begin(a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return zp::fail_hip(e, "step begin kernel launch");
    return ZERO_OK;
}

extern "C" int zero_adamw_step(const zero_tensor_set* set, const zero_step_control* ctl, int32_t n_groups, void* stream) {
    zp::clear_error();
    if (!set || !ctl) return fail(ZERO_ERR_INVALID_ARG, "zero_adamw_step: NULL set or control");
    if (!zp::is_aligned(ctl, 8)) return fail(ZERO_ERR_ALIGNMENT, "the control block is not 8-byte aligned");
    if (n_groups < 1 || n_groups > ZERO_MAX_GROUPS) return fail(ZERO_ERR_INVALID_ARG, "n_groups must be in 1..16");
    if (set->max_group >= n_groups) return fail(ZERO_ERR_INVALID_ARG, "a tensor's group is not below n_groups");
    if (const char* what = zp::lacks(set, true, true, true)) return fail(ZERO_ERR_STATE, what);
    const uintptr_t lo = reinterpret_cast<uintptr_t>(ctl);
    if (zp::meets(set->written, lo, lo + sizeof(*ctl)))
        return fail(ZERO_ERR_INVALID_ARG, "the control block overlaps an array of the set");
    const int rc = zp::check_set_device(set, stream, "zero_adamw_step");
    if (rc != ZERO_OK) return rc;
    if (set->n_tiles == 0) return ZERO_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    zp::KernelEvents ev;
    bool timed = false;
    hipError_t e = zp::set_events(s, &ev, &timed);
    if (e != hipSuccess) return zp::fail_hip(e, "timing event");
    e = zp::launch_adamw(zp::set_launch(set), ctl, s, ev);
    if (e != hipSuccess) return zp::fail_hip(e, "AdamW kernel launch");
    if (timed) zp::timing_done();
    return ZERO_OK;
}

extern "C" int zero_states_convert(const zero_tensor_set* dst, const zero_tensor_set* src, void* stream) {
    zp::clear_error();
    if (!dst || !src) return fail(ZERO_ERR_INVALID_ARG, "zero_states_convert: NULL set");
    if (dst->numel != src->numel) return fail(ZERO_ERR_INVALID_ARG, "the sets' tensors have different sizes");
    for (const zero_tensor_set* s : {dst, src})
        if (const char* what = zp::lacks(s, false, false, true)) return fail(ZERO_ERR_STATE, what);
    if (!dst->rec.empty() && dst->state_type == src->state_type)
        return fail(ZERO_ERR_INVALID_ARG, "the sets' states have the same type");
    if (zp::lists_meet(dst->states, src->states)) return fail(ZERO_ERR_INVALID_ARG, "the sets' states overlap");
    int rc = zp::check_set_device(dst, stream, "zero_states_convert");
    if (rc == ZERO_OK) rc = zp::check_set_device(src, stream, "zero_states_convert");
    if (rc != ZERO_OK) return rc;
    if (dst->n_tiles == 0) return ZERO_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    zp::KernelEvents ev;
    bool timed = false;
    hipError_t e = zp::set_events(s, &ev, &timed);
    if (e != hipSuccess) return zp::fail_hip(e, "timing event");
    e = zp::launch_convert(zp::set_launch(dst), zp::set_launch(src), s, ev);
    if (e != hipSuccess) return zp::fail_hip(e, "state conversion kernel launch");
    if (timed) zp::timing_done();
    return ZERO_OK;
}
