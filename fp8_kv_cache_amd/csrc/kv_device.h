// kv_device.h -- device helpers shared by the paged cache's kernels: vector
// types, the status word, and the search for a workgroup's sequence.
#pragma once

#include "device_common.h"
#include "kv_internal.h"
#include "splitzip.h"

namespace kvi {

using sz::gptr;
using sz::u32x2;
using sz::u32x4;
using sz::uniform;

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ inline void flag(int32_t* status) {
    if (status) *gptr(status) = SZ_ERR_INVALID_ARGUMENT;
}

__device__ inline f32x8 to_f32(u32x4 x) { return __builtin_convertvector(__builtin_bit_cast(bf16x8, x), f32x8); }

// last_not_above() by a wave, each lane trying one place.  Every lane takes part.
template <typename Low>
__device__ inline uint32_t wave_last_not_above(uint32_t n, int64_t target, Low low) {
    return uniform(last_not_above(n, [&](uint32_t from, uint32_t step, uint32_t left) -> uint64_t {
        const uint32_t i = sz::lane_id() * step;
        return __ballot(i < left && low(from + (i < left ? i : 0)) <= target);
    }));
}

// The sequence that has token row t, cu[s] <= t < cu[s + 1]; where none has,
// some sequence: callers compare t with its span.
__device__ inline uint32_t wave_seq_of_token(const Batch& b, uint32_t t) {
    return wave_last_not_above(b.num_seqs, t, [&](uint32_t s) -> int64_t { return gptr(b.cu)[s]; });
}

// The tile in `slot`, if any.
__device__ inline Tile wave_tile_of(const Batch& b, const Mask& mask, uint64_t slot, uint32_t group, uint32_t M) {
    const uint32_t s = wave_last_not_above(b.num_seqs, static_cast<int64_t>(slot), [&](uint32_t i) -> int64_t {
        return static_cast<int64_t>(tile_slot(b, i, group, M));
    });
    return tile_in(b, mask, s, slot, group, M);
}

// Granules of all sequences, by a wave.
__device__ inline uint32_t wave_granules(const Batch& b, const Mask& mask, uint32_t group, uint32_t granule) {
    uint32_t total = 0;
    for (uint32_t i = sz::lane_id(); i < b.num_seqs; i += 64) total += granules_of(tile_of_seq(b, mask, i, group), granule);
    for (uint32_t m = 32; m; m /= 2) total += __shfl_xor(total, m);
    return uniform(total);
}

// The sequence that has granule `at` (below the total), and the granules before it.
__device__ inline uint32_t wave_seq_of_granule(const Batch& b, const Mask& mask, uint32_t group, uint32_t granule,
                                               uint32_t at, uint32_t& before) {
    before = 0;
    for (uint32_t from = 0; from < b.num_seqs; from += 64) {
        const uint32_t i = from + sz::lane_id();
        const uint32_t g = i < b.num_seqs ? granules_of(tile_of_seq(b, mask, i, group), granule) : 0;
        const uint32_t upto = sz::wave_scan_incl(g);
        const uint64_t past = __ballot(before + upto > at);
        if (past) {
            const uint32_t k = __builtin_ctzll(past);
            before += __builtin_amdgcn_readlane(upto - g, k);
            return from + k;
        }
        before += __builtin_amdgcn_readlane(upto, 63);
    }
    return b.num_seqs;
}

}  // namespace kvi
