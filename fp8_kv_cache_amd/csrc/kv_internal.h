// kv_internal.h -- the index arithmetic of the paged KV cache (shared by its
// kernels and its host checks) and the launch interfaces; the calls are
// documented in include/paged_kv.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sz_internal.h"

namespace kvi {

#define KV_HD __host__ __device__ inline

struct Cache {
    uint8_t* k;
    uint8_t* v;
    uint64_t page_stride, token_stride, head_stride;   // bytes
    uint32_t num_pages, log2_page, kv_heads, head_dim;
};

struct Batch {
    const int32_t* pages;
    const int32_t* cu;
    const int32_t* kv_lens;
    uint64_t pages_stride;
    uint32_t pages_per_seq, num_seqs, total_tokens, max_tokens, max_kv_len;
};

// One sequence of the batch as the device data give it.
struct Span {
    int32_t begin, n, kv;
    bool ok;
    KV_HD int32_t first() const { return kv - n; }   // position of its first new token (may be negative)
};

KV_HD Span span_of(const Batch& b, uint32_t s) {
    Span p;
    const int32_t lo = b.cu[s], hi = b.cu[s + 1];
    p.begin = lo;
    p.kv = b.kv_lens[s];
    p.ok = lo >= 0 && hi >= lo && static_cast<uint32_t>(hi) <= b.total_tokens &&
           static_cast<uint32_t>(hi - lo) <= b.max_tokens && p.kv >= 0 &&
           static_cast<uint32_t>(p.kv) <= b.max_kv_len;
    p.n = p.ok ? hi - lo : 0;
    return p;
}

// The last s in [0, n) with low(s) <= target, low ascending; 0 where there is
// none, and some s in [0, n) whatever low gives.  Up to 64 places are tried at
// a time: vote(from, step, n) has bit i set where i * step < n and
// low(from + i * step) <= target, so that a wave finds one of 64 sequences in
// one trip to memory and one of 4096 in two, where a binary search makes 6
// and 12, each waiting for the last.
template <typename Vote>
KV_HD uint32_t last_not_above(uint32_t n, Vote vote) {
    uint32_t from = 0;
    while (n > 1) {
        const uint32_t step = (n + 63) / 64;
        const uint64_t not_above = vote(from, step, n);
        const uint32_t k = not_above ? 63 - __builtin_clzll(not_above) : 0;
        from += k * step;
        n = n - k * step < step ? n - k * step : step;
    }
    return from;
}

// Page of a sequence's position p >= 0, or -1: past the table, or not a
// page of the pool.
KV_HD int32_t page_of(const Cache& c, const Batch& b, uint32_t s, int32_t p) {
    const uint32_t i = static_cast<uint32_t>(p) >> c.log2_page;
    if (i >= b.pages_per_seq) return -1;
    const int32_t page = b.pages[s * b.pages_stride + i];
    return static_cast<uint32_t>(page) < c.num_pages ? page : -1;
}

// Byte offset in a pool of slot p % page_size of `page` (not negative), head 0.
KV_HD uint64_t slot_offset(const Cache& c, int32_t page, int32_t p) {
    return static_cast<uint64_t>(page) * c.page_stride +
           static_cast<uint64_t>(static_cast<uint32_t>(p) & ((1u << c.log2_page) - 1)) * c.token_stride;
}

// ---- Attention's work: the rows of a sequence under one KV head are its
// (token, query head of the group) pairs, token-major, n * group of them,
// cut into tiles of M.  Sequence s has the tile slots from
// floor(cu[s] * group / M) + s: floor((a + x) / M) - floor(a / M) + 1 >=
// ceil(x / M), so its tiles fit before the next sequence's, and a workgroup
// finds its tile by a search in cu, with no table to build first.
KV_HD uint64_t tile_slot(const Batch& b, uint32_t s, uint32_t group, uint32_t M) {
    const int32_t c = b.cu[s];
    return static_cast<uint64_t>(c < 0 ? 0 : c) * group / M + s;
}
KV_HD uint64_t tile_slots(const Batch& b, uint32_t group, uint32_t M) {
    return static_cast<uint64_t>(b.total_tokens) * group / M + b.num_seqs;
}

struct Tile {
    Span seq;
    uint32_t s;
    uint32_t row0, rows;      // first row of the tile in the sequence, and how many
    int32_t seen, lo, hi;     // positions that any of its rows sees: [seen, hi); lo is seen, down to a multiple of 64
    int32_t p0, p1;           // positions of its first and last token
    bool any;
};

struct Mask {
    uint32_t causal, window;
    // row at position p of a sequence of kv tokens sees [first(p), last(p))
    KV_HD int32_t first(int32_t p) const {
        return window && p >= 0 && static_cast<uint32_t>(p) >= window ? p + 1 - static_cast<int32_t>(window) : 0;
    }
    KV_HD int32_t last(int32_t p, int32_t kv) const { return causal ? (p < 0 ? 0 : p + 1) : (p < 0 ? 0 : kv); }
};

KV_HD void tile_range(Tile& t, const Mask& mask, uint32_t group) {
    t.p0 = t.seq.first() + static_cast<int32_t>(t.row0 / group);
    t.p1 = t.seq.first() + static_cast<int32_t>((t.row0 + t.rows - 1) / group);
    t.seen = mask.first(t.p0);
    t.lo = t.seen & ~63;
    t.hi = mask.last(t.p1, t.seq.kv);
}

// The tile in `slot` of sequence s, the last whose tile_slot is not above it;
// any = false where there is none.
KV_HD Tile tile_in(const Batch& b, const Mask& mask, uint32_t s, uint64_t slot, uint32_t group, uint32_t M) {
    Tile t{};
    t.s = s;
    t.seq = span_of(b, s);
    const uint64_t first = tile_slot(b, s, group, M);
    if (slot < first || !t.seq.ok) return t;
    const uint64_t row0 = (slot - first) * M, rows = static_cast<uint64_t>(t.seq.n) * group;
    if (row0 >= rows) return t;
    t.any = true;
    t.row0 = static_cast<uint32_t>(row0);
    t.rows = static_cast<uint32_t>(rows - row0 < M ? rows - row0 : M);
    tile_range(t, mask, group);
    return t;
}

// Splits of a tile's positions: split z has [lo + z * len, lo + (z + 1) * len) of [lo, hi).
KV_HD uint32_t splits_of(const Tile& t, uint32_t len) {
    return t.hi > t.lo ? (static_cast<uint32_t>(t.hi - t.lo) + len - 1) / len : 0;
}

// ---- The few-rows kernel: every sequence has one tile, and its positions
// are cut into granules.  Either a workgroup takes a whole sequence under one
// KV head, or the granules of all sequences, one after the other, are dealt
// to a fixed number of units in equal runs, so that the lengths, which only
// the device knows, do not matter: a unit takes the end of one sequence, some
// whole ones and the beginning of another.  Of the sequences in a unit at
// most two are not whole: the one that began before it and the one that goes
// on behind it, places 0 and 1 of its partial sums.
constexpr uint32_t kFewRows = 16;

KV_HD Tile tile_of_seq(const Batch& b, const Mask& mask, uint32_t s, uint32_t group) {
    Tile t{};
    t.s = s;
    t.seq = span_of(b, s);
    const uint64_t rows = static_cast<uint64_t>(t.seq.n) * group;
    if (rows == 0 || rows > kFewRows) return t;
    t.any = true;
    t.rows = static_cast<uint32_t>(rows);
    tile_range(t, mask, group);
    return t;
}

// One at least, so that a sequence without keys has its rows written.
KV_HD uint32_t granules_of(const Tile& t, uint32_t granule) {
    if (!t.any) return 0;
    return t.hi > t.lo ? (static_cast<uint32_t>(t.hi - t.lo) + granule - 1) / granule : 1;
}

// Granules a unit takes: `least` at least, all of `total` in `units` units.
KV_HD uint32_t granules_each(uint32_t total, uint32_t units, uint32_t least) {
    const uint32_t each = total / units + (total % units != 0);
    return each < least ? least : each;
}

// Workgroups of 4 waves that a CU holds at once, by their registers and LDS.
KV_HD constexpr uint32_t few_a_cu(uint32_t head_dim, bool e5m2) {
    return head_dim <= 64 || (head_dim == 80 && !e5m2) ? 3 : head_dim <= 128 ? 2 : 1;
}

// Workgroups: 8 units or sequences at a time, each with all KV heads.
KV_HD uint64_t few_groups(uint64_t units, uint64_t kv_heads) { return (units + 7) / 8 * 8 * kv_heads; }

// ---- launch interfaces

struct AppendArgs {
    Cache cache;
    Batch batch;
    const uint16_t *k, *v, *q;
    uint16_t* q_out;
    uint64_t k_stride, v_stride, q_stride, q_out_stride;   // elements
    const float* cos_sin;
    const uint16_t *q_norm, *k_norm;
    float eps;
    uint32_t q_heads, rotary_dim, max_positions, interleaved;
    int32_t* status;
    bool e5m2;
    uint32_t rows, passes;   // of a workgroup, set by the launch
};

struct CopyArgs {
    Cache cache;
    Batch batch;
    uint8_t *k, *v;                // the layer tensors
    uint64_t k_stride, v_stride;   // bytes
    uint32_t head_bytes;
    int32_t* status;
    uint32_t rows, lanes, pieces, head_magic;   // set by the launch
};

struct AttentionPlan {
    uint32_t tile;                   // rows of a tile; kFewRows: the few-rows kernel
    uint32_t splits, split_len;      // tiles: at most `splits` of split_len positions each
    uint32_t heads;                  // few rows: KV heads a workgroup
    uint32_t units, granule, least;  // few rows: units (0: a workgroup a sequence), positions of a granule, granules of a unit
    uint64_t parts;                  // partial sums of a row: tiles [row][split]; few rows [unit][KV head][2][row of the tile]
    uint64_t workspace_bytes;
};

struct AttentionArgs {
    Cache cache;
    Batch batch;
    const uint16_t* q;
    uint16_t* out;
    float* lse;
    uint64_t q_stride, out_stride;   // elements
    float scale;
    Mask mask;
    uint32_t group;                  // query heads of a KV head
    AttentionPlan plan;
    float* part;                     // workspace: plan.parts x head_dim sums, plan.parts x (max, sum), plan.units x Cut
    int32_t* status;
    bool e5m2;
};

AttentionPlan attention_plan(const Cache& c, const Batch& b, uint32_t group, uint32_t window, bool e5m2);

hipError_t launch_append(AppendArgs a, hipStream_t s);
hipError_t launch_gather(const CopyArgs& a, hipStream_t s);
hipError_t launch_scatter(const CopyArgs& a, hipStream_t s);
hipError_t launch_attention(const AttentionArgs& a, hipStream_t s);

}  // namespace kvi
