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

// The last s in [0, n) with low(s) <= target, low ascending; 0 where there is
// none, and some s in [0, n) whatever low gives.  The 64 lanes try 64 places
// at a time, so that up to 64 sequences cost one trip to memory and 4096 two,
// where a binary search makes 6 and 12, each waiting for the last.  Every
// lane of the wave takes part.
template <typename Low>
__device__ inline uint32_t last_not_above(uint32_t n, int64_t target, Low low) {
    uint32_t from = 0;
    while (n > 1) {
        const uint32_t step = (n + 63) / 64, i = sz::lane_id() * step;
        const uint64_t not_above = __ballot(i < n && low(from + (i < n ? i : 0)) <= target);
        const uint32_t k = not_above ? 63 - __builtin_clzll(not_above) : 0;
        from += k * step;
        n = n - k * step < step ? n - k * step : step;
    }
    return uniform(from);
}

// seq_of_token() by a wave: where no sequence has the row, some sequence;
// callers compare t with its span.
__device__ inline uint32_t wave_seq_of_token(const Batch& b, uint32_t t) {
    return last_not_above(b.num_seqs, t, [&](uint32_t s) -> int64_t { return gptr(b.cu)[s]; });
}

// tile_of() by a wave.
__device__ inline Tile wave_tile_of(const Batch& b, const Mask& mask, uint64_t slot, uint32_t group, uint32_t M) {
    const uint32_t s = last_not_above(b.num_seqs, static_cast<int64_t>(slot), [&](uint32_t i) -> int64_t {
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
