// Host code of the tensor sets under the sanitizers: random sets of made-up
// addresses through zero_tensor_set_create and zero_tensor_set_bind_grads, whose
// verdicts are compared with a pairwise check written here.  No device is
// needed: an accepted set ends at the first HIP call (or is made and freed where
// there is a device; its addresses are never read).
#include <cstdio>
#include <cstdlib>
#include <random>
#include <string>
#include <vector>

#include "tensor_set.hpp"

namespace zp {
// what capi.cpp and the kernels provide
static std::string g_message;
int fail(int status, const std::string& msg) {
    g_message = msg;
    return status;
}
int fail_hip(hipError_t, const char* what) { return fail(ZERO_ERR_HIP, what); }
void clear_error() { g_message.clear(); }
int check_stream_device(void*, int, const char*) { return ZERO_OK; }
hipError_t timing_events(KernelEvents* ev) {
    *ev = KernelEvents();
    return hipSuccess;
}
void timing_done() {}
int64_t sumsq_blocks(int64_t n) { return n > 64 ? 1024 : 1; }
hipError_t launch_sumsq(const SetLaunch&, double*, bool, double*, hipStream_t, const KernelEvents&) { std::abort(); }
hipError_t launch_step_begin(const BeginLaunch&, hipStream_t) { std::abort(); }
hipError_t launch_adamw(const SetLaunch&, const zero_step_control*, hipStream_t, const KernelEvents&) { std::abort(); }
hipError_t launch_convert(const SetLaunch&, const SetLaunch&, hipStream_t, const KernelEvents&) { std::abort(); }
}  // namespace zp

namespace {

struct Span {
    uintptr_t lo, hi;
    bool written;
};

int check(bool ok, const char* what) {
    if (!ok) std::printf("FAILED: %s\n", what);
    return ok ? 0 : 1;
}

}  // namespace

int main() {
    std::mt19937_64 rng(7);
    const auto pick = [&](uint64_t n) { return int64_t(rng() % n); };
    int bad = 0, accepted = 0, overlapping = 0, misaligned = 0;
    for (int trial = 0; trial < 30000 && !bad; ++trial) {
        const int32_t grad = int32_t(1 + pick(3)), state = pick(2) ? ZERO_DTYPE_FP32 : ZERO_DTYPE_MXFP8, out = int32_t(pick(3));
        const int gw = grad == ZERO_DTYPE_FP32 ? 4 : 2, sw = state == ZERO_DTYPE_FP32 ? 4 : 1;
        const int64_t n = 1 + pick(6);
        // sparse or dense address space, so both verdicts come up
        const uint64_t room = pick(2) ? 1u << 20 : 1u << 14;
        std::vector<zero_tensor> t;
        std::vector<Span> spans;
        bool aligned = true;
        const auto place = [&](int64_t count, int width, bool written) -> uintptr_t {
            uintptr_t at = (uintptr_t(1) << 40) + uintptr_t(pick(room));
            if (pick(200)) at -= at % uintptr_t(width);
            if (count) {
                aligned = aligned && at % uintptr_t(width) == 0;
                spans.push_back({at, at + uintptr_t(count * width), written});
            }
            return at;
        };
        for (int64_t i = 0; i < n; ++i) {
            zero_tensor x = {};
            x.numel = pick(8) ? pick(300) : 0;
            const int64_t blocks = (x.numel + 31) / 32;
            x.p = reinterpret_cast<float*>(place(x.numel, 4, true));
            x.m = reinterpret_cast<void*>(place(x.numel, sw, true));
            x.v = reinterpret_cast<void*>(place(x.numel, sw, true));
            if (state == ZERO_DTYPE_MXFP8) {
                x.m_scale = reinterpret_cast<uint8_t*>(place(blocks, 1, true));
                x.v_scale = reinterpret_cast<uint8_t*>(place(blocks, 1, true));
            }
            if (out) x.out = reinterpret_cast<void*>(place(x.numel, 2, true));
            x.grad = reinterpret_cast<const void*>(place(x.numel, gw, false));
            x.group = int32_t(pick(16));
            t.push_back(x);
        }
        bool meet = false;
        for (size_t a = 0; a < spans.size(); ++a)
            for (size_t b = a + 1; b < spans.size(); ++b)
                meet = meet || ((spans[a].written || spans[b].written) && spans[a].lo < spans[b].hi && spans[b].lo < spans[a].hi);
        zero_tensor_set* set = nullptr;
        const int rc = zero_tensor_set_create(t.data(), n, grad, state, out, uint32_t(trial), nullptr, &set);
        if (!aligned) {
            ++misaligned;
            bad += check(rc == ZERO_ERR_ALIGNMENT || rc == ZERO_ERR_INVALID_ARG, "a misaligned address is refused");
        } else if (meet) {
            ++overlapping;
            bad += check(rc == ZERO_ERR_INVALID_ARG, "an overlap is refused");
        } else {
            ++accepted;
            bad += check(rc == ZERO_OK || rc == ZERO_ERR_HIP, "a sound set passes the checks");
        }
        bad += check((rc == ZERO_OK) == (set != nullptr), "a handle comes with success alone");
        zero_tensor_set_destroy(set);
    }
    // every tile shift of every small size: the tiles reach the end, and none is wanted past them
    for (int64_t numel = 1; numel < 5000; ++numel)
        for (uint32_t shift = 0; shift < uint32_t(zp::kAlign); ++shift) {
            const int64_t tiles = (numel + shift - 1) / zp::kSetTile + 1;
            const uint32_t spare = uint32_t(tiles * zp::kSetTile - numel);
            const void* p = reinterpret_cast<const void*>((uintptr_t(1) << 30) + 4 * uintptr_t(shift));
            const uint32_t got = zp::tile_shift(p, 4, spare);
            if (got != shift || tiles * zp::kSetTile - shift < numel || (tiles - 1) * zp::kSetTile - int64_t(shift) >= numel) {
                bad += check(false, "tiles of a shifted tensor");
                break;
            }
        }
    std::printf("%d accepted, %d overlapping, %d misaligned\n", accepted, overlapping, misaligned);
    bad += check(accepted > 2000 && overlapping > 2000 && misaligned > 200, "every verdict came up");
    std::printf(bad ? "FAILED\n" : "OK\n");
    return bad ? 1 : 0;
}
