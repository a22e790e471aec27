// tensor_set.hpp -- tables and launchers of the tensor sets (AdamW over many
// tensors, gradient norm, state conversion); not part of the public ABI.
#pragma once

#include "zp_internal.hpp"

namespace zp {

// One tensor as the kernels see it (80 bytes, read with scalar loads).
struct TensorRec {
    float* p;
    const void* grad;
    void* m;
    void* v;
    uint8_t* m_scale;
    uint8_t* v_scale;
    void* out;
    int64_t numel;
    uint32_t key;     // of the tensor's random bits: mix32(mix32(seed) + index)
    int32_t group;
    int64_t pad;
};
static_assert(sizeof(TensorRec) == 80, "TensorRec layout");

// A tile is kSetTile consecutive elements of one tensor, from a multiple of
// kSetTile on (the tensor's last tile may be shorter); one wave takes it.
constexpr int64_t kSetTile = 1024;
struct TileRec {
    uint32_t tensor;   // index of its TensorRec
    uint32_t tile;     // which tile of the tensor
};
constexpr int64_t kMaxSetTiles = int64_t(1) << 25;
static_assert(kMaxSetTiles <= kMaxGridWaves, "one wave per tile fits one launch");
static_assert(kSetTile % ZERO_STATE_BLOCK == 0, "blocks do not cross tiles");

// MurmurHash3's 32-bit finaliser (Austin Appleby, public domain): every bit of
// the result depends on every bit of x.
__host__ __device__ inline uint32_t mix32(uint32_t x) {
    x ^= x >> 16;
    x *= 0x85EBCA6Bu;
    x ^= x >> 13;
    x *= 0xC2B2AE35u;
    return x ^ (x >> 16);
}

struct SetLaunch {
    const TensorRec* rec;    // device, one per non-empty tensor
    const TileRec* tile;     // device
    int64_t n_tiles;
    int32_t grad_type;
    int32_t state_type;
    int32_t out_type;
};

// Blocks of the sum-of-squares pass, each of which leaves one double in `work`
// for a second launch to add up; 1: the one block writes the result itself.
int64_t sumsq_blocks(int64_t n_tiles);

hipError_t launch_sumsq(const SetLaunch& a, double* sumsq, bool accumulate, double* work, hipStream_t stream,
                        const KernelEvents& ev);

// The constants of zero_step_begin as its kernel takes them.
struct BeginLaunch {
    zero_step_control* ctl;
    zero_adam_hparams group[ZERO_MAX_GROUPS];
    int32_t n_groups;
    int32_t check;
    int32_t scaler;      // 1: backoff ... growth_interval hold
    float max_norm;
    float backoff;
    float growth;
    float min_scale;
    int32_t growth_interval;
};
hipError_t launch_step_begin(const BeginLaunch& a, hipStream_t stream);

hipError_t launch_adamw(const SetLaunch& a, const zero_step_control* ctl, hipStream_t stream, const KernelEvents& ev);

// src's states into dst's; the tiles are src's (both sets have the same).
hipError_t launch_convert(const SetLaunch& dst, const SetLaunch& src, hipStream_t stream, const KernelEvents& ev);

}  // namespace zp
