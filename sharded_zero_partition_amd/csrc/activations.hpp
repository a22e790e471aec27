// activations.hpp -- launchers of the calls on activation checkpoints and
// embeddings (not part of the public ABI).
#pragma once

#include "zp_internal.hpp"

namespace zp {

// A checked matrix.
struct Matrix {
    void* p;
    int64_t rows, cols;
    int64_t stride;   // elements
};

// Division of 32-bit numbers below 2^31 by g, and of 64-bit ones below 2^52.
struct Divisor {
    uint32_t g;
    uint32_t magic;   // floor(2^(31 + l) / g) + 1, l = ceil(log2 g)
    uint32_t shift;   // l - 1
    double inv;
};
inline Divisor divisor(uint32_t g) {   // g in 2 .. 2^31
    uint32_t l = 1;
    while ((uint64_t(1) << l) < g) ++l;
    return {g, uint32_t((uint64_t(1) << (31 + l)) / g + 1), l - 1, 1.0 / double(g)};
}

// Matrices are taken in octets of 8 neighbouring columns; a row of a checkpoint
// has 4 a block.
constexpr int kOctet = 8;
constexpr int kRowThreads = 256;
constexpr int kRowOctets = 2;   // a thread's
constexpr int64_t kMaxOctets = ((int64_t(1) << 24) - 1) * kRowThreads * kRowOctets;

struct ActLaunch {
    int32_t type;
    int32_t kind;      // of ZERO_ACT_*; -1: no activation (a plain store or load)
    int64_t octets;    // rows * 4 blocks
    int64_t blocks;    // rows * blocks
    int64_t cols;
    Divisor per_row;   // octets of a row
    const void* x;     // dy in the gradient
    const void* up;
    void* out;         // dx
    void* dup;
    int64_t sx, sup, sout, sdup;   // strides
    uint8_t *cx, *cx_scale, *cup, *cup_scale, *cout, *cout_scale;
};
hipError_t launch_activation(const ActLaunch& a, hipStream_t s, const KernelEvents& ev);
// kind -1: x's values into out
hipError_t launch_activation_grad(const ActLaunch& a, hipStream_t s, const KernelEvents& ev);

struct WeightGradLaunch {
    int32_t dy_type, out_type;
    int64_t T, n, k;
    const void* dy;
    int64_t s_dy;
    const uint8_t* code;
    const uint8_t* scale;
    void* dw;
    int64_t s_dw;
    bool transposed, accumulate;
    void* bias;
    float* work;
};
int64_t weight_grad_work(int64_t T, int64_t n, int64_t k, int32_t dy_type);   // bytes
hipError_t launch_weight_grad(const WeightGradLaunch& a, hipStream_t s, const KernelEvents& ev);

struct EmbedLaunch {
    int32_t type, out_type;   // of the table and out, or of dy and the table's gradient
    int32_t token_bytes;
    int64_t n;                // tokens
    int64_t rows, cols;       // of the table
    int64_t first;
    float scale;
    const void* tokens;
    const void* in;
    int64_t s_in;
    void* out;
    int64_t s_out;
    bool accumulate;
    void* work;
};
hipError_t launch_lookup(const EmbedLaunch& a, hipStream_t s, const KernelEvents& ev);
int64_t embedding_work(int64_t n, int64_t rows, int64_t cols);   // bytes
bool embedding_fits(int64_t n, int64_t rows, int64_t cols);      // one launch takes it
hipError_t launch_embedding_grad(const EmbedLaunch& a, hipStream_t s, const KernelEvents& ev);

}  // namespace zp
