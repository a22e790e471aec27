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
    uint32_t spare;   // tiles * kSetTile - numel
    uint32_t reserved;
};
static_assert(sizeof(TensorRec) == 80, "TensorRec layout");

// A tile is kSetTile consecutive elements of one tensor; one wave takes it.  The
// norm's tiles start with the tensor, so the order of its sum depends on sizes
// alone.  In a step and a conversion tile k of a tensor starts at element
// k kSetTile - shift, so the first and the last one may be shorter.  The shift
// (0 .. kAlign - 1) puts an array's whole tiles on kAlign-element boundaries in
// memory, for 16- and 32-bit elements on lines of 128 bytes.  A store that leaves
// a line unfinished is dear (state conversion to fp32, 200 M elements, tiles that
// start with the tensor: 348 us on lines, 469 us one element off them); loads off
// their lines cost little (the norm: nothing).  Flat buffers of several kinds
// mostly start on lines, so one tensor's shift is the same in all of them; where
// it is not, only the array it was taken from gains.
constexpr int64_t kSetTile = 1024;
constexpr int64_t kAlign = 64;
struct TileRec {
    uint32_t tensor;   // index of its TensorRec
    uint32_t tile;     // which tile of the tensor
};

// The shift of the tiles for an array of `bytes`-byte elements at p; none where
// the tensor's tiles would not reach its end.
__host__ __device__ inline uint32_t tile_shift(const void* p, int bytes, uint32_t spare) {
    const uint32_t s = uint32_t(reinterpret_cast<uintptr_t>(p) / uintptr_t(bytes)) & uint32_t(kAlign - 1);
    return s <= spare ? s : 0u;
}
// In a set with MXFP8 states blocks do not cross tiles, so a shift is a multiple
// of the block: 32 where p stands there (codes alone: where they do), else 0.
__host__ __device__ inline uint32_t block_shift(const TensorRec& r) {
    const uint32_t s = r.p ? uint32_t(reinterpret_cast<uintptr_t>(r.p) / 4) : uint32_t(reinterpret_cast<uintptr_t>(r.m));
    return (s & 32u) <= r.spare ? s & 32u : 0u;
}
// Whether the whole tiles of an array of `bytes`-byte elements then fill whole
// lines.
constexpr int kLine = 128;
__host__ __device__ inline bool on_lines(const void* p, int bytes, uint32_t shift) {
    return ((reinterpret_cast<uintptr_t>(p) - uintptr_t(bytes) * shift) & uintptr_t(kLine - 1)) == 0;
}
// Whether a step's, and a conversion's, tiles of a tensor are stored straight
// from the registers: those on lines, and tensors of a single tile, whose lines
// are shared with others in any case (20,000 tensors of 500 elements, step in 8
// bits: 39 us straight, 46 through LDS).  A set
// with another tensor runs kernels that put such tiles' results in order through
// LDS first.
__host__ __device__ inline bool step_direct(const TensorRec& r) {
    const uint32_t s = block_shift(r);
    return r.numel <= kSetTile ||
           (on_lines(r.p, 4, s) && on_lines(r.m, 1, s) && on_lines(r.v, 1, s) && (!r.out || on_lines(r.out, 2, s)));
}
__host__ __device__ inline bool codes_direct(const TensorRec& r) {
    const uint32_t s = block_shift(r);
    return r.numel <= kSetTile || (on_lines(r.m, 1, s) && on_lines(r.v, 1, s));
}
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
    const TileRec* norm_tile;   // device: tiles of kSetTile from each tensor's first element on
    int64_t n_norm_tiles;
    int32_t grad_type;
    int32_t state_type;
    int32_t out_type;
    bool staged_step;      // MXFP8: a tensor is not step_direct, or not codes_direct
    bool staged_codes;
    bool random_m;         // MXFP8: m rounded at random whatever beta1
};

// Blocks of the sum-of-squares pass, each of which leaves one double in `work`
// for a second launch to add up; 1: the one block writes the result itself.
int64_t sumsq_blocks(int64_t n_norm_tiles);

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

// src's states into dst's, by dst's tiles.
hipError_t launch_convert(const SetLaunch& dst, const SetLaunch& src, hipStream_t stream, const KernelEvents& ev);

}  // namespace zp
