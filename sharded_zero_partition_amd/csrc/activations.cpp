// activations.cpp -- argument checks and entry points of the calls on activation
// checkpoints and embeddings.
#include <cmath>
#include <cstring>
#include <initializer_list>
#include <string>

#include "activations.hpp"

namespace zp {
namespace {

constexpr int64_t kMaxCols = int64_t(1) << 31;    // exclusive
constexpr int64_t kMaxSpan = int64_t(1) << 56;    // elements from a matrix's first to its last
constexpr int64_t kMaxTokens = int64_t(1) << 40;  // also of matrices without columns, and of one row for all tokens

int type_bytes(int32_t t) {
    switch (t) {
        case ZERO_DTYPE_FP16: return 2;
        case ZERO_DTYPE_BF16: return 2;
        case ZERO_DTYPE_FP32: return 4;
        default: return 0;
    }
}

// Memory that a call reads or writes: `rows` pieces of `width` bytes, `pitch` apart.
struct Area {
    uintptr_t lo = 0, hi = 0;   // all of it; lo == hi: none
    uint64_t pitch = 0, width = 0;
    bool one = true;            // a single piece
};

bool apart(const Area& a, const Area& b) {
    if (a.lo == a.hi || b.lo == b.hi || a.hi <= b.lo || b.hi <= a.lo) return true;
    if (a.one && b.one) return false;
    // the columns of one buffer: rows equally far apart, pieces that do not meet
    const uint64_t pitch = a.one ? b.pitch : a.pitch;
    if ((!b.one && b.pitch != pitch) || a.width > pitch || b.width > pitch) return false;
    const uint64_t d = b.lo >= a.lo ? (b.lo - a.lo) % pitch : (pitch - (a.lo - b.lo) % pitch) % pitch;
    return d >= a.width && d + b.width <= pitch;
}

int piece(Area* out, const void* p, int64_t bytes, const char* what) {
    *out = Area();
    if (bytes <= 0) return ZERO_OK;
    out->lo = reinterpret_cast<uintptr_t>(p);
    if (uint64_t(bytes) > UINTPTR_MAX - out->lo)
        return fail(ZERO_ERR_INDEX_OVERFLOW, std::string(what) + ": its end is outside the address space");
    out->hi = out->lo + uintptr_t(bytes);
    out->width = uint64_t(bytes);
    return ZERO_OK;
}

int check_matrix(const zero_matrix* m, const char* what, bool written, Area* area) {
    *area = Area();
    if (!m) return fail(ZERO_ERR_INVALID_ARG, std::string(what) + " is NULL");
    const int w = type_bytes(m->type);
    if (w == 0) return fail(ZERO_ERR_INVALID_ARG, std::string(what) + ": its type must be FP16, BF16 or FP32");
    if (m->rows < 0 || m->cols < 0) return fail(ZERO_ERR_INVALID_ARG, std::string(what) + ": a size is negative");
    if (m->cols >= kMaxCols) return fail(ZERO_ERR_INDEX_OVERFLOW, std::string(what) + ": too many columns");
    if (m->rows == 0 || m->cols == 0) return ZERO_OK;
    if (!m->data) return fail(ZERO_ERR_INVALID_ARG, std::string(what) + ": its data is NULL");
    if (reinterpret_cast<uintptr_t>(m->data) % uintptr_t(w) != 0)
        return fail(ZERO_ERR_ALIGNMENT, std::string(what) + " lacks its element's alignment");
    area->one = m->rows == 1;
    int64_t span = m->cols;
    if (!area->one) {
        if (m->stride < 0 || (written && m->stride < m->cols))
            return fail(ZERO_ERR_INVALID_ARG, std::string(what) + ": its stride is too small");
        if (m->stride > 0 && m->rows - 1 > (kMaxSpan - m->cols) / m->stride)
            return fail(ZERO_ERR_INDEX_OVERFLOW, std::string(what) + " is too large");
        span += (m->rows - 1) * m->stride;
    }
    const bool one = area->one;
    const int rc = piece(area, m->data, span * w, what);
    area->one = one;
    area->width = uint64_t(m->cols) * uint64_t(w);
    area->pitch = one ? 0 : uint64_t(m->stride) * uint64_t(w);
    return rc;
}

int64_t blocks_of(int64_t cols) { return (cols + 31) / 32; }

int check_checkpoint(const zero_checkpoint* c, const char* what, Area* code, Area* scale) {
    *code = *scale = Area();
    if (!c) return fail(ZERO_ERR_INVALID_ARG, std::string(what) + " is NULL");
    int64_t nc = 0, ns = 0;
    int rc = zero_checkpoint_bytes(c->rows, c->cols, &nc, &ns);
    if (rc != ZERO_OK) return rc;
    if (nc == 0) return ZERO_OK;
    if (!c->code || !c->scale) return fail(ZERO_ERR_INVALID_ARG, std::string(what) + ": its codes or scales are NULL");
    if (reinterpret_cast<uintptr_t>(c->code) % 16 != 0)
        return fail(ZERO_ERR_ALIGNMENT, std::string(what) + ": its codes are not 16-byte aligned");
    rc = piece(code, c->code, nc, what);
    return rc != ZERO_OK ? rc : piece(scale, c->scale, ns, what);
}

int overlap(const char* who) {
    return fail(ZERO_ERR_INVALID_ARG, std::string(who) + ": something that is written overlaps another argument");
}

// Whether all that is written is apart from each other and from all that is read.
bool all_apart(std::initializer_list<Area> written, std::initializer_list<Area> read) {
    for (const Area* a = written.begin(); a != written.end(); ++a) {
        for (const Area* b = written.begin(); b != a; ++b)
            if (!apart(*a, *b)) return false;
        for (const Area& b : read)
            if (!apart(*a, b)) return false;
    }
    return true;
}

bool same_shape(const zero_matrix* a, int64_t rows, int64_t cols) { return a->rows == rows && a->cols == cols; }

// One place for both: element by element, so a call may read one and write the other.
bool same_place(const zero_matrix* a, const zero_matrix* b) {
    return a->data == b->data && a->type == b->type && (a->rows <= 1 || a->stride == b->stride);
}

int on_device(void* stream, const char* who) {
    int dev = 0;
    const hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return fail_hip(e, "hipGetDevice");
    return check_stream_device(stream, dev, who);
}

template <typename F>
int timed(void* stream, const char* who, const F& launch) {
    hipStream_t s = static_cast<hipStream_t>(stream);
    KernelEvents ev;
    bool open = false;
    hipError_t e = set_events(s, &ev, &open);
    if (e != hipSuccess) return fail_hip(e, "timing event");
    e = launch(s, ev);
    if (e != hipSuccess) return fail_hip(e, who);
    if (open) timing_done();
    return ZERO_OK;
}

// The sizes of a pass over octets; false when one launch cannot take them.
bool set_sizes(ActLaunch* a, int64_t rows, int64_t cols) {
    const int64_t blocks = blocks_of(cols);
    if (rows > kMaxOctets / (4 * blocks)) return false;
    a->blocks = rows * blocks;
    a->octets = 4 * a->blocks;
    a->cols = cols;
    a->per_row = divisor(uint32_t(4 * blocks));
    return true;
}

int too_large(const char* who) { return fail(ZERO_ERR_INDEX_OVERFLOW, std::string(who) + ": too large for one launch"); }

int check_tokens(const void* tokens, int32_t token_bytes, int64_t n, Area* area) {
    if (token_bytes != 4 && token_bytes != 8) return fail(ZERO_ERR_INVALID_ARG, "token_bytes must be 4 or 8");
    *area = Area();
    if (n == 0) return ZERO_OK;
    if (n > kMaxTokens) return fail(ZERO_ERR_INDEX_OVERFLOW, "too many tokens");
    if (!tokens) return fail(ZERO_ERR_INVALID_ARG, "tokens is NULL");
    if (reinterpret_cast<uintptr_t>(tokens) % uintptr_t(token_bytes) != 0)
        return fail(ZERO_ERR_ALIGNMENT, "tokens lack their alignment");
    return piece(area, tokens, n * token_bytes, "tokens");
}

int check_work(void* work, int64_t bytes, Area* area) {
    *area = Area();
    if (bytes == 0) return ZERO_OK;
    if (!work) return fail(ZERO_ERR_INVALID_ARG, "work is NULL");
    if (reinterpret_cast<uintptr_t>(work) % 16 != 0) return fail(ZERO_ERR_ALIGNMENT, "work is not 16-byte aligned");
    return piece(area, work, bytes, "work");
}

}  // namespace
}  // namespace zp

using zp::Area;
using zp::fail;

extern "C" int zero_checkpoint_bytes(int64_t rows, int64_t cols, int64_t* code_bytes, int64_t* scale_bytes) {
    zp::clear_error();
    if (rows < 0 || cols < 0) return fail(ZERO_ERR_INVALID_ARG, "a checkpoint's size is negative");
    const int64_t blocks = zp::blocks_of(cols < zp::kMaxCols ? cols : 0);
    if (cols >= zp::kMaxCols || (blocks > 0 && rows > (int64_t(1) << 48) / (32 * blocks)))
        return fail(ZERO_ERR_INDEX_OVERFLOW, "a checkpoint is too large");
    if (code_bytes) *code_bytes = rows * blocks * 32;
    if (scale_bytes) *scale_bytes = rows * blocks;
    return ZERO_OK;
}

extern "C" int zero_checkpoint_store(const zero_matrix* x, const zero_checkpoint* c, void* stream) {
    zp::clear_error();
    Area ax, ac, as;
    int rc = zp::check_matrix(x, "x", false, &ax);
    if (rc == ZERO_OK) rc = zp::check_checkpoint(c, "the checkpoint", &ac, &as);
    if (rc != ZERO_OK) return rc;
    if (!zp::same_shape(x, c->rows, c->cols)) return fail(ZERO_ERR_INVALID_ARG, "x and the checkpoint differ in shape");
    if (!zp::all_apart({ac, as}, {ax})) return zp::overlap("zero_checkpoint_store");
    zp::ActLaunch a = {};
    if (x->rows > 0 && x->cols > 0 && !zp::set_sizes(&a, x->rows, x->cols)) return zp::too_large("zero_checkpoint_store");
    rc = zp::on_device(stream, "zero_checkpoint_store");
    if (rc != ZERO_OK || a.octets == 0) return rc;
    a.type = x->type;
    a.kind = -1;
    a.x = x->data;
    a.sx = x->stride;
    a.cx = c->code;
    a.cx_scale = c->scale;
    return zp::timed(stream, "checkpoint kernel launch",
                     [&](hipStream_t s, const zp::KernelEvents& ev) { return zp::launch_activation(a, s, ev); });
}

extern "C" int zero_checkpoint_load(const zero_checkpoint* c, const zero_matrix* out, void* stream) {
    zp::clear_error();
    Area ao, ac, as;
    int rc = zp::check_checkpoint(c, "the checkpoint", &ac, &as);
    if (rc == ZERO_OK) rc = zp::check_matrix(out, "out", true, &ao);
    if (rc != ZERO_OK) return rc;
    if (!zp::same_shape(out, c->rows, c->cols)) return fail(ZERO_ERR_INVALID_ARG, "out and the checkpoint differ in shape");
    if (!zp::all_apart({ao}, {ac, as})) return zp::overlap("zero_checkpoint_load");
    zp::ActLaunch a = {};
    if (out->rows > 0 && out->cols > 0 && !zp::set_sizes(&a, out->rows, out->cols)) return zp::too_large("zero_checkpoint_load");
    rc = zp::on_device(stream, "zero_checkpoint_load");
    if (rc != ZERO_OK || a.octets == 0) return rc;
    a.type = out->type;
    a.kind = -1;
    a.out = out->data;
    a.sout = out->stride;
    a.cx = c->code;
    a.cx_scale = c->scale;
    return zp::timed(stream, "checkpoint kernel launch",
                     [&](hipStream_t s, const zp::KernelEvents& ev) { return zp::launch_activation_grad(a, s, ev); });
}

extern "C" int zero_activation(int32_t kind, const zero_matrix* x, const zero_matrix* up, const zero_matrix* out,
                               const zero_checkpoint* c_x, const zero_checkpoint* c_up, const zero_checkpoint* c_out,
                               void* stream) {
    zp::clear_error();
    if (kind < ZERO_ACT_RELU || kind > ZERO_ACT_GELU_TANH) return fail(ZERO_ERR_INVALID_ARG, "unknown activation");
    if (up ? (c_x == nullptr) != (c_up == nullptr) : c_up != nullptr)
        return fail(ZERO_ERR_INVALID_ARG, "c_up comes with up and c_x");
    Area ax, aup, ao, c[6];
    int rc = zp::check_matrix(x, "x", false, &ax);
    if (rc == ZERO_OK && up) rc = zp::check_matrix(up, "up", false, &aup);
    if (rc == ZERO_OK) rc = zp::check_matrix(out, "out", true, &ao);
    const zero_checkpoint* kept[3] = {c_x, c_up, c_out};
    for (int i = 0; i < 3; ++i)
        if (rc == ZERO_OK && kept[i]) rc = zp::check_checkpoint(kept[i], "a checkpoint", &c[2 * i], &c[2 * i + 1]);
    if (rc != ZERO_OK) return rc;
    bool fits = zp::same_shape(out, x->rows, x->cols) && out->type == x->type;
    if (up) fits = fits && zp::same_shape(up, x->rows, x->cols) && up->type == x->type;
    for (const zero_checkpoint* k : kept) fits = fits && (!k || zp::same_shape(x, k->rows, k->cols));
    if (!fits) return fail(ZERO_ERR_INVALID_ARG, "zero_activation: shapes or types differ");
    // out in the place of x or up
    const Area none;
    const Area rx = zp::same_place(x, out) ? none : ax, rup = up && zp::same_place(up, out) ? none : aup;
    if (!zp::all_apart({ao, c[0], c[1], c[2], c[3], c[4], c[5]}, {rx, rup}) ||
        !zp::all_apart({c[0], c[1], c[2], c[3], c[4], c[5]}, {ax, aup}))
        return zp::overlap("zero_activation");
    zp::ActLaunch a = {};
    if (x->rows > 0 && x->cols > 0 && !zp::set_sizes(&a, x->rows, x->cols)) return zp::too_large("zero_activation");
    rc = zp::on_device(stream, "zero_activation");
    if (rc != ZERO_OK || a.octets == 0) return rc;
    a.type = x->type;
    a.kind = kind;
    a.x = x->data;
    a.sx = x->stride;
    if (up) {
        a.up = up->data;
        a.sup = up->stride;
    }
    a.out = out->data;
    a.sout = out->stride;
    if (c_x) {
        a.cx = c_x->code;
        a.cx_scale = c_x->scale;
    }
    if (c_up) {
        a.cup = c_up->code;
        a.cup_scale = c_up->scale;
    }
    if (c_out) {
        a.cout = c_out->code;
        a.cout_scale = c_out->scale;
    }
    return zp::timed(stream, "activation kernel launch",
                     [&](hipStream_t s, const zp::KernelEvents& ev) { return zp::launch_activation(a, s, ev); });
}

extern "C" int zero_activation_grad(int32_t kind, const zero_matrix* dy, const zero_checkpoint* c_x,
                                    const zero_checkpoint* c_up, const zero_matrix* dx, const zero_matrix* dup,
                                    void* stream) {
    zp::clear_error();
    if (kind < ZERO_ACT_RELU || kind > ZERO_ACT_GELU_TANH) return fail(ZERO_ERR_INVALID_ARG, "unknown activation");
    if ((c_up == nullptr) != (dup == nullptr)) return fail(ZERO_ERR_INVALID_ARG, "c_up and dup come together");
    Area ay, ax, aup, c[4];
    int rc = zp::check_matrix(dy, "dy", false, &ay);
    if (rc == ZERO_OK) rc = zp::check_checkpoint(c_x, "c_x", &c[0], &c[1]);
    if (rc == ZERO_OK && c_up) rc = zp::check_checkpoint(c_up, "c_up", &c[2], &c[3]);
    if (rc == ZERO_OK) rc = zp::check_matrix(dx, "dx", true, &ax);
    if (rc == ZERO_OK && dup) rc = zp::check_matrix(dup, "dup", true, &aup);
    if (rc != ZERO_OK) return rc;
    bool fits = zp::same_shape(dx, dy->rows, dy->cols) && dx->type == dy->type && zp::same_shape(dy, c_x->rows, c_x->cols);
    if (dup) fits = fits && zp::same_shape(dup, dy->rows, dy->cols) && dup->type == dy->type && zp::same_shape(dy, c_up->rows, c_up->cols);
    if (!fits) return fail(ZERO_ERR_INVALID_ARG, "zero_activation_grad: shapes or types differ");
    const Area none;
    const bool in_place = zp::same_place(dx, dy), up_in_place = dup && zp::same_place(dup, dy);
    if (!zp::all_apart({ax, aup}, {c[0], c[1], c[2], c[3]}) || !zp::all_apart({ax}, {in_place ? none : ay}) ||
        !zp::all_apart({aup}, {up_in_place ? none : ay}))
        return zp::overlap("zero_activation_grad");
    zp::ActLaunch a = {};
    if (dy->rows > 0 && dy->cols > 0 && !zp::set_sizes(&a, dy->rows, dy->cols)) return zp::too_large("zero_activation_grad");
    rc = zp::on_device(stream, "zero_activation_grad");
    if (rc != ZERO_OK || a.octets == 0) return rc;
    a.type = dy->type;
    a.kind = kind;
    a.x = dy->data;
    a.sx = dy->stride;
    a.out = dx->data;
    a.sout = dx->stride;
    a.cx = c_x->code;
    a.cx_scale = c_x->scale;
    if (dup) {
        a.cup = c_up->code;
        a.cup_scale = c_up->scale;
        a.dup = dup->data;
        a.sdup = dup->stride;
    }
    return zp::timed(stream, "activation gradient kernel launch",
                     [&](hipStream_t s, const zp::KernelEvents& ev) { return zp::launch_activation_grad(a, s, ev); });
}

extern "C" int64_t zero_weight_grad_work_bytes(int64_t T, int64_t n, int64_t k, int32_t dy_type) {
    if (T <= 0 || n <= 0 || k < 0 || T > zp::kMaxTokens || n >= zp::kMaxCols || k >= zp::kMaxCols || zp::type_bytes(dy_type) == 0) return 0;
    return zp::weight_grad_work(T, n, k, dy_type);
}

extern "C" int zero_weight_grad(const zero_matrix* dy, const zero_checkpoint* x, const zero_matrix* dw, int32_t transposed,
                                void* bias, int32_t accumulate, void* work, void* stream) {
    zp::clear_error();
    if ((transposed != 0 && transposed != 1) || (accumulate != 0 && accumulate != 1))
        return fail(ZERO_ERR_INVALID_ARG, "transposed and accumulate must be 0 or 1");
    Area ay, ac, as, aw, ab, ak;
    int rc = zp::check_matrix(dy, "dy", false, &ay);
    if (rc == ZERO_OK) rc = zp::check_checkpoint(x, "the checkpoint", &ac, &as);
    if (rc == ZERO_OK) rc = zp::check_matrix(dw, "dw", true, &aw);
    if (rc != ZERO_OK) return rc;
    const int64_t T = dy->rows, n = dy->cols, k = x->cols;
    if (T > zp::kMaxTokens) return fail(ZERO_ERR_INDEX_OVERFLOW, "zero_weight_grad: too many tokens");
    if (x->rows != T) return fail(ZERO_ERR_INVALID_ARG, "dy and the checkpoint have different numbers of rows");
    if (!zp::same_shape(dw, transposed ? k : n, transposed ? n : k))
        return fail(ZERO_ERR_INVALID_ARG, "dw's shape is not that of the gradient");
    if (bias && n > 0) {
        const int w = zp::type_bytes(dw->type);
        if (reinterpret_cast<uintptr_t>(bias) % uintptr_t(w) != 0) return fail(ZERO_ERR_ALIGNMENT, "bias lacks its element's alignment");
        rc = zp::piece(&ab, bias, n * w, "bias");
        if (rc != ZERO_OK) return rc;
    }
    rc = zp::check_work(work, zero_weight_grad_work_bytes(T, n, k, dy->type), &ak);
    if (rc != ZERO_OK) return rc;
    if (!zp::all_apart({aw, ab, ak}, {ay, ac, as})) return zp::overlap("zero_weight_grad");
    if ((k + 255) / 256 * ((n + 127) / 128) > (int64_t(1) << 22)) return zp::too_large("zero_weight_grad");
    rc = zp::on_device(stream, "zero_weight_grad");
    if (rc != ZERO_OK || n == 0 || (k == 0 && !bias)) return rc;
    zp::WeightGradLaunch a = {};
    a.dy_type = dy->type;
    a.out_type = dw->type;
    a.T = T;
    a.n = n;
    a.k = k;
    a.dy = dy->data;
    a.s_dy = dy->stride;
    a.code = x->code;
    a.scale = x->scale;
    a.dw = dw->data;
    a.s_dw = dw->stride;
    a.transposed = transposed != 0;
    a.accumulate = accumulate != 0;
    a.bias = bias;
    a.work = static_cast<float*>(work);
    return zp::timed(stream, "weight gradient kernel launch",
                     [&](hipStream_t s, const zp::KernelEvents& ev) { return zp::launch_weight_grad(a, s, ev); });
}

extern "C" int zero_embedding_lookup(const zero_matrix* table, const void* tokens, int32_t token_bytes, int64_t first,
                                     float scale, const zero_matrix* out, void* stream) {
    zp::clear_error();
    Area at, ao, an;
    int rc = zp::check_matrix(table, "the table", false, &at);
    if (rc == ZERO_OK) rc = zp::check_matrix(out, "out", true, &ao);
    if (rc == ZERO_OK) rc = zp::check_tokens(tokens, token_bytes, out->rows, &an);
    if (rc != ZERO_OK) return rc;
    if (table->cols != out->cols) return fail(ZERO_ERR_INVALID_ARG, "the table and out have different numbers of columns");
    if (!std::isfinite(scale)) return fail(ZERO_ERR_INVALID_ARG, "scale must be finite");
    if (!zp::all_apart({ao}, {at, an})) return zp::overlap("zero_embedding_lookup");
    if (out->cols > 0 && out->rows > zp::kMaxOctets / ((out->cols + 7) / 8 + 1)) return zp::too_large("zero_embedding_lookup");
    rc = zp::on_device(stream, "zero_embedding_lookup");
    if (rc != ZERO_OK || out->rows == 0 || out->cols == 0) return rc;
    zp::EmbedLaunch a = {};
    a.type = table->type;
    a.out_type = out->type;
    a.token_bytes = token_bytes;
    a.n = out->rows;
    a.rows = table->rows;
    a.cols = out->cols;
    a.first = first;
    a.scale = scale;
    a.tokens = tokens;
    a.in = table->data;
    a.s_in = table->stride;
    a.out = out->data;
    a.s_out = out->stride;
    return zp::timed(stream, "embedding lookup kernel launch",
                     [&](hipStream_t s, const zp::KernelEvents& ev) { return zp::launch_lookup(a, s, ev); });
}

extern "C" int64_t zero_embedding_grad_work_bytes(int64_t tokens, int64_t rows, int64_t cols) {
    constexpr int64_t most = int64_t(1) << 30;
    if (tokens <= 0 || tokens > most || rows <= 0 || rows > most || cols <= 0 || cols >= zp::kMaxCols) return 0;
    return zp::embedding_work(tokens, rows, cols);
}

extern "C" int zero_embedding_grad(const zero_matrix* dy, const void* tokens, int32_t token_bytes, int64_t first, float scale,
                                   const zero_matrix* dtable, int32_t accumulate, void* work, void* stream) {
    zp::clear_error();
    if (accumulate != 0 && accumulate != 1) return fail(ZERO_ERR_INVALID_ARG, "accumulate must be 0 or 1");
    Area ay, at, an, ak;
    int rc = zp::check_matrix(dy, "dy", false, &ay);
    if (rc == ZERO_OK) rc = zp::check_matrix(dtable, "dtable", true, &at);
    if (rc == ZERO_OK) rc = zp::check_tokens(tokens, token_bytes, dy->rows, &an);
    if (rc != ZERO_OK) return rc;
    const int64_t n = dy->rows, rows = dtable->rows, cols = dtable->cols;
    if (dy->cols != cols) return fail(ZERO_ERR_INVALID_ARG, "dy and dtable have different numbers of columns");
    if (!std::isfinite(scale)) return fail(ZERO_ERR_INVALID_ARG, "scale must be finite");
    if (n > (int64_t(1) << 30) || rows > (int64_t(1) << 30)) return zp::too_large("zero_embedding_grad");
    const int64_t bytes = zero_embedding_grad_work_bytes(n, rows, cols);
    if (rows > 0 && cols > 0 && !zp::embedding_fits(n, rows, cols)) return zp::too_large("zero_embedding_grad");
    rc = zp::check_work(work, bytes, &ak);
    if (rc != ZERO_OK) return rc;
    if (!zp::all_apart({at, ak}, {ay, an})) return zp::overlap("zero_embedding_grad");
    rc = zp::on_device(stream, "zero_embedding_grad");
    if (rc != ZERO_OK || rows == 0 || cols == 0 || (n == 0 && accumulate)) return rc;
    zp::EmbedLaunch a = {};
    a.type = dy->type;
    a.out_type = dtable->type;
    a.token_bytes = token_bytes;
    a.n = n;
    a.rows = rows;
    a.cols = cols;
    a.first = first;
    a.scale = scale;
    a.tokens = tokens;
    a.in = dy->data;
    a.s_in = dy->stride;
    a.out = dtable->data;
    a.s_out = dtable->stride;
    a.accumulate = accumulate != 0;
    a.work = work;
    return zp::timed(stream, "embedding gradient kernel launch",
                     [&](hipStream_t s, const zp::KernelEvents& ev) { return zp::launch_embedding_grad(a, s, ev); });
}
