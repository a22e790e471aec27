// Host code of the calls on activation checkpoints and embeddings under the
// sanitizers: random matrices, checkpoints, tokens and workspaces at made-up
// addresses, sizes up to the ends of their types.  Verdicts on overlaps are
// compared with a row-by-row check written here.  No device is needed: a call
// that passes the checks ends at the first HIP call (or at a launcher that does
// nothing where there is a device).
#include <cstdio>
#include <random>
#include <string>
#include <vector>

#include "activations.hpp"

namespace zp {
// what capi.cpp, tensor_set.cpp and the kernels provide
static std::string g_message;
int fail(int status, const std::string& msg) {
    g_message = msg;
    return status;
}
int fail_hip(hipError_t, const char* what) { return fail(ZERO_ERR_HIP, what); }
void clear_error() { g_message.clear(); }
int check_stream_device(void*, int, const char*) { return ZERO_OK; }
hipError_t set_events(hipStream_t, KernelEvents*, bool* timed) {
    *timed = false;
    return hipSuccess;
}
void timing_done() {}
static int g_bad = 0;
static void check(bool ok, const char* what) {
    if (!ok) std::printf("FAILED: %s\n", what);
    g_bad += ok ? 0 : 1;
}
hipError_t launch_activation(const ActLaunch& a, hipStream_t, const KernelEvents&) {
    check(a.octets > 0 && a.octets <= kMaxOctets, "octets of a launch");
    return hipSuccess;
}
hipError_t launch_activation_grad(const ActLaunch& a, hipStream_t s, const KernelEvents& ev) { return launch_activation(a, s, ev); }
int64_t weight_grad_work(int64_t T, int64_t n, int64_t, int32_t) { return T > 256 ? 4 * n : 0; }
hipError_t launch_weight_grad(const WeightGradLaunch& a, hipStream_t, const KernelEvents&) {
    check(a.work != nullptr || a.T <= 256, "a workspace");
    return hipSuccess;
}
hipError_t launch_lookup(const EmbedLaunch&, hipStream_t, const KernelEvents&) { return hipSuccess; }
int64_t embedding_work(int64_t n, int64_t, int64_t) { return 8 * n; }
bool embedding_fits(int64_t, int64_t rows, int64_t) { return rows < (int64_t(1) << 27); }
hipError_t launch_embedding_grad(const EmbedLaunch&, hipStream_t, const KernelEvents&) { return hipSuccess; }
}  // namespace zp

namespace {

using zp::check;

std::mt19937_64 rng(11);
int64_t pick(uint64_t n) { return int64_t(rng() % n); }

struct Row {
    uintptr_t lo, hi;
};
typedef std::vector<Row> Rows;

// An argument: what it occupies, and a name for those that may be in one place.
struct Arg {
    Rows rows;
    bool written;
    int pair;   // arguments of one pair > 0 may be the same matrix
    const zero_matrix* m;
};
bool meet(const Rows& a, const Rows& b) {
    for (const Row& x : a)
        for (const Row& y : b)
            if (x.lo < y.hi && y.lo < x.hi) return true;
    return false;
}
bool same(const zero_matrix* a, const zero_matrix* b) {
    return a->data == b->data && a->type == b->type && (a->rows <= 1 || a->stride == b->stride);
}

uint64_t room;
uintptr_t spot(int align) {
    const uintptr_t at = (uintptr_t(1) << 40) + uintptr_t(pick(room));
    return at - at % uintptr_t(align);
}
int width(int32_t t) { return t == ZERO_DTYPE_FP32 ? 4 : 2; }
zero_matrix matrix(int64_t rows, int64_t cols, int32_t type, int64_t stride) {
    return {reinterpret_cast<void*>(spot(width(type))), rows, cols, stride, type, 0};
}
Rows rows_of(const zero_matrix& m) {
    Rows r;
    const uintptr_t w = uintptr_t(width(m.type)), at = reinterpret_cast<uintptr_t>(m.data);
    for (int64_t i = 0; m.cols && i < m.rows; ++i)
        r.push_back({at + uintptr_t(i * m.stride) * w, at + uintptr_t(i * m.stride + m.cols) * w});
    return r;
}
Rows piece(const void* p, int64_t bytes) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    return bytes > 0 ? Rows{{at, at + uintptr_t(bytes)}} : Rows{};
}
zero_checkpoint checkpoint(int64_t rows, int64_t cols) {
    return {reinterpret_cast<uint8_t*>(spot(16)), reinterpret_cast<uint8_t*>(spot(1)), rows, cols};
}
void add(std::vector<Arg>* args, const zero_checkpoint& c, bool written) {
    int64_t code = 0, scale = 0;
    check(zero_checkpoint_bytes(c.rows, c.cols, &code, &scale) == ZERO_OK, "a checkpoint's size");
    args->push_back({piece(c.code, code), written, 0, nullptr});
    args->push_back({piece(c.scale, scale), written, 0, nullptr});
}

int accepted = 0, overlapping = 0, cautious = 0;
void judge(int rc, const std::vector<Arg>& args, bool strided, const char* what) {
    bool bad = false;
    for (size_t a = 0; a < args.size(); ++a)
        for (size_t b = a + 1; b < args.size(); ++b) {
            const Arg &x = args[a], &y = args[b];
            if (!x.written && !y.written) continue;
            if (x.pair && x.pair == y.pair && !(x.written && y.written) && same(x.m, y.m)) continue;
            bad = bad || meet(x.rows, y.rows);
        }
    if (bad) {
        ++overlapping;
        check(rc == ZERO_ERR_INVALID_ARG, what);
    } else if (rc == ZERO_ERR_INVALID_ARG && strided) {
        ++cautious;   // rows of different distances that lie between each other's are refused
    } else {
        ++accepted;
        check(rc == ZERO_OK || rc == ZERO_ERR_HIP, what);
    }
}

void trial() {
    room = pick(2) ? 1u << 20 : 1u << 13;
    const int32_t type = int32_t(1 + pick(3)), out = int32_t(1 + pick(3));
    const int64_t rows = pick(9), cols = pick(8) ? 1 + pick(70) : 0, wide = pick(2) ? cols : 2 * cols + pick(9);
    const bool strided = wide != cols;
    const auto mat = [&](int64_t r, int64_t c, int32_t t) { return matrix(r, c, t, c == cols ? wide : c); };
    std::vector<Arg> args;
    const auto put = [&](const zero_matrix& m, bool written, int pair = 0) { args.push_back({rows_of(m), written, pair, &m}); };
    zero_matrix x = mat(rows, cols, type), up = mat(rows, cols, type), y = mat(rows, cols, type), z = mat(rows, cols, type);
    zero_checkpoint c[3] = {checkpoint(rows, cols), checkpoint(rows, cols), checkpoint(rows, cols)};
    // the halves of one buffer, and one place for two
    if (strided && pick(2)) up.data = static_cast<char*>(x.data) + cols * width(type);
    if (pick(4) == 0) y.data = pick(2) ? x.data : up.data;
    const bool gated = pick(2), kept = pick(2), kept_out = pick(2);
    const int32_t kind = int32_t(pick(4)), accumulate = int32_t(pick(2));
    const int64_t n = 1 + pick(40), k = pick(70), T = pick(600);
    switch (pick(7)) {
        case 0:
            put(x, false);
            add(&args, c[0], true);
            return judge(zero_checkpoint_store(&x, &c[0], nullptr), args, strided, "store");
        case 1:
            put(y, true);
            add(&args, c[0], false);
            return judge(zero_checkpoint_load(&c[0], &y, nullptr), args, strided, "load");
        case 2:
            put(x, false, 1);
            if (gated) put(up, false, 1);
            put(y, true, 1);
            for (int i = 0; i < 3; ++i)
                if (i == 0 ? kept : i == 1 ? kept && gated : kept_out) add(&args, c[i], true);
            return judge(zero_activation(kind, &x, gated ? &up : nullptr, &y, kept ? &c[0] : nullptr, kept && gated ? &c[1] : nullptr,
                                         kept_out ? &c[2] : nullptr, nullptr), args, strided, "activation");
        case 3:
            put(x, false, 1);
            put(y, true, 1);
            if (gated) put(z, true, 1);
            add(&args, c[0], false);
            if (gated) add(&args, c[1], false);
            return judge(zero_activation_grad(kind, &x, &c[0], gated ? &c[1] : nullptr, &y, gated ? &z : nullptr, nullptr), args,
                         strided, "activation's gradient");
        case 4: {
            const zero_matrix dy = matrix(T, n, type, pick(2) ? n + pick(9) : 0), dw = gated ? matrix(k, n, out, n + pick(5)) : matrix(n, k, out, k + pick(5));
            const zero_checkpoint cx = checkpoint(T, k);
            void* bias = kept ? reinterpret_cast<void*>(spot(width(out))) : nullptr;
            void* work = reinterpret_cast<void*>(spot(16));
            args.push_back({rows_of(dy), false, 0, nullptr});
            args.push_back({rows_of(dw), true, 0, nullptr});
            add(&args, cx, false);
            if (bias) args.push_back({piece(bias, n * width(out)), true, 0, nullptr});
            args.push_back({piece(work, zero_weight_grad_work_bytes(T, n, k, type)), true, 0, nullptr});
            return judge(zero_weight_grad(&dy, &cx, &dw, gated, bias, accumulate, work, nullptr), args, true, "weight gradient");
        }
        case 5: {
            const zero_matrix table = mat(1 + pick(20), cols, type);
            const int32_t size = pick(2) ? 4 : 8;
            const void* tokens = reinterpret_cast<const void*>(spot(size));
            put(table, false);
            put(y, true);
            args.push_back({piece(tokens, rows * size), false, 0, nullptr});
            return judge(zero_embedding_lookup(&table, tokens, size, pick(100) - 50, 0.5f, &y, nullptr), args, strided, "lookup");
        }
        default: {
            const zero_matrix dt = mat(1 + pick(20), cols, out);
            const int32_t size = pick(2) ? 4 : 8;
            const void* tokens = reinterpret_cast<const void*>(spot(size));
            void* work = reinterpret_cast<void*>(spot(16));
            put(x, false);
            put(dt, true);
            args.push_back({piece(tokens, rows * size), false, 0, nullptr});
            args.push_back({piece(work, zero_embedding_grad_work_bytes(rows, dt.rows, cols)), true, 0, nullptr});
            return judge(zero_embedding_grad(&x, tokens, size, 0, 1.0f, &dt, accumulate, work, nullptr), args, strided || type != out,
                         "embedding's gradient");
        }
    }
}

// Numbers of every size, valid or not: a verdict, and no arithmetic that overflows.
int64_t number() {
    static const int64_t ends[] = {0, 1, -1, 31, 33, INT64_MAX, INT64_MIN, INT64_MAX - 1};
    switch (pick(4)) {
        case 0: return ends[pick(8)];
        case 1: return (int64_t(1) << pick(63)) + pick(3) - 1;
        case 2: return int64_t(rng());
        default: return pick(100);
    }
}
void any_numbers() {
    const auto pointer = [] { return reinterpret_cast<void*>(pick(8) ? spot(16) : uintptr_t(rng())); };
    const auto any = [&] { return zero_matrix{pointer(), number(), number(), number(), int32_t(pick(5)), 0}; };
    const auto kept = [&] { return zero_checkpoint{static_cast<uint8_t*>(pointer()), static_cast<uint8_t*>(pointer()), number(), number()}; };
    zero_matrix m[3] = {any(), any(), any()};
    zero_checkpoint c[3] = {kept(), kept(), kept()};
    const int64_t rows = number(), cols = number();
    if (pick(2)) {   // shapes that fit
        for (zero_matrix& x : m) x.rows = rows, x.cols = cols, x.type = 1 + int32_t(pick(3));
        for (zero_checkpoint& x : c) x.rows = rows, x.cols = cols;
    }
    room = 1u << 30;
    int64_t a, b;
    zero_checkpoint_bytes(rows, cols, &a, &b);
    zero_checkpoint_store(&m[0], &c[0], nullptr);
    zero_checkpoint_load(&c[0], &m[0], nullptr);
    zero_activation(int32_t(pick(6)) - 1, &m[0], pick(2) ? &m[1] : nullptr, &m[2], &c[0], pick(2) ? &c[1] : nullptr, &c[2], nullptr);
    zero_activation_grad(int32_t(pick(6)) - 1, &m[0], &c[0], pick(2) ? &c[1] : nullptr, &m[1], pick(2) ? &m[2] : nullptr, nullptr);
    zero_weight_grad_work_bytes(rows, cols, number(), int32_t(pick(5)));
    zero_embedding_grad_work_bytes(rows, cols, number());
    zero_embedding_lookup(&m[0], pointer(), pick(2) ? 8 : 4, number(), 1.0f, &m[1], nullptr);
    zero_embedding_grad(&m[0], pointer(), pick(2) ? 8 : 4, number(), 1.0f, &m[1], int32_t(pick(2)), pointer(), nullptr);
    // dy [rows, n], x [rows, k], dw [n, k]
    const int64_t n = number(), k = number();
    zero_matrix dy = any(), dw = any();
    dy.rows = c[0].rows = rows;
    dy.cols = dw.rows = n;
    c[0].cols = dw.cols = k;
    zero_weight_grad(&dy, &c[0], &dw, 0, pick(2) ? pointer() : nullptr, 0, pointer(), nullptr);
}

}  // namespace

int main() {
    room = 1u << 20;
    for (int i = 0; i < 60000 && !zp::g_bad; ++i) trial();
    for (int i = 0; i < 200000 && !zp::g_bad; ++i) any_numbers();
    // divisors: products instead of divisions, over their whole range
    for (int i = 0; i < 200000 && !zp::g_bad; ++i) {
        const uint32_t g = uint32_t(2 + pick(uint64_t(1) << pick(31)));
        const zp::Divisor d = zp::divisor(g);
        const uint32_t x = uint32_t(pick(2) ? pick(uint64_t(1) << 31) : (uint64_t(1) << 31) / g * g - uint64_t(pick(2)));
        if (x >= (uint32_t(1) << 31)) continue;
        check(uint32_t((uint64_t(x) * d.magic) >> 32) >> d.shift == x / g, "a quotient");
    }
    std::printf("%d accepted, %d overlapping, %d refused for their strides\n", accepted, overlapping, cautious);
    check(accepted > 5000 && overlapping > 5000, "every verdict came up");
    if (!zp::g_bad) std::printf("OK\n");
    return zp::g_bad ? 1 : 0;
}
