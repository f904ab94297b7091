// kv_kernels.hip -- the paged KV cache's append (per-head norm, position
// rotation, conversion and paged store in one pass) and the gather and
// scatter between pages and contiguous layer tensors.  The calls are
// documented in include/paged_kv.h.
//
// All three move each byte once and are bound by memory.  What can keep them
// from that is the chain of dependent loads in front of a token's data (its
// sequence, the sequence's lengths, the page): a workgroup takes several
// tokens, a lane looks up one token's place, all lanes at once, and the
// places are handed round by lane reads.
#include "kv_device.h"

namespace kvi {

namespace {

constexpr uint32_t kThreads = 256;

// Where a token row goes, one row a lane.
struct Place {
    uint64_t slot;    // byte offset in the pools
    int32_t p;        // position
    int32_t state;    // 0: no sequence has the row, 1: it has no place (or none that may be used), 2: it has
};

// Of row t0 + lane, for lanes below `rows`.  Every lane of the wave takes part.
__device__ inline Place place_of(const Cache& c, const Batch& b, uint32_t t0, uint32_t rows, int32_t* status) {
    const uint32_t s0 = wave_seq_of_token(b, t0), lane = sz::lane_id();
    Place at{0, -1, 0};
    if (lane >= rows) return at;
    const int32_t t = static_cast<int32_t>(t0 + lane);
    uint32_t lo = s0, hi = b.num_seqs;   // the last s with cu[s] <= t
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) / 2;
        if (gptr(b.cu)[mid] <= t) lo = mid;
        else hi = mid;
    }
    const Span seq = span_of(b, lo);
    if (t < seq.begin || t >= seq.begin + seq.n) return at;
    at.state = 1;
    at.p = seq.first() + (t - seq.begin);
    if (at.p < 0) return at;
    const int32_t page = page_of(c, b, lo, at.p);
    if (page < 0) {
        flag(status);
        return at;
    }
    at.state = 2;
    at.slot = slot_offset(c, page, at.p);
    return at;
}

// Each sequence is looked at by one thread of the launch.
__device__ inline void check_spans(const Batch& b, int32_t* status) {
    if (blockIdx.y) return;
    for (uint32_t s = blockIdx.x * kThreads + threadIdx.x; s < b.num_seqs; s += gridDim.x * kThreads)
        if (!span_of(b, s).ok) flag(status);
}

__device__ inline uint64_t lane_value(uint64_t x, uint32_t lane) {
    return static_cast<uint64_t>(__builtin_amdgcn_readlane(static_cast<uint32_t>(x >> 32), lane)) << 32 |
           static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<uint32_t>(x), lane));
}

// to E5M2, nearest even: byte i of the result is element i
__device__ inline u32x2 to_e5m2(f32x8 x) {
    uint32_t lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_pk_bf8_f32(x[0], x[1], lo, false);
    lo = __builtin_amdgcn_cvt_pk_bf8_f32(x[2], x[3], lo, true);
    hi = __builtin_amdgcn_cvt_pk_bf8_f32(x[4], x[5], hi, false);
    hi = __builtin_amdgcn_cvt_pk_bf8_f32(x[6], x[7], hi, true);
    return u32x2{lo, hi};
}

// Lanes a head has: its D / 8 units of 8 elements, up to a power of two, so
// that no head crosses a wave and the norm's sum is a butterfly over them.
constexpr uint32_t lanes_of(uint32_t dim) { return dim <= 64 ? 8 : dim <= 128 ? 16 : 32; }

// A workgroup takes `rows` tokens and `passes` times kThreads / kLanes heads
// of each (q heads, then k heads, then v heads).  A thread has the same unit
// of every head, so a token's angles are read once a thread, and kBatch heads
// are read before the first is used.
template <uint32_t D, bool kE5M2>
__global__ __launch_bounds__(kThreads) void k_append(AppendArgs a) {
    constexpr uint32_t kUnits = D / 8, kLanes = lanes_of(D), kHeads = kThreads / kLanes, kBatch = 3;
    check_spans(a.batch, a.status);
    const uint32_t t0 = blockIdx.x * a.rows;
    const uint32_t rows = a.batch.total_tokens - t0 < a.rows ? a.batch.total_tokens - t0 : a.rows;
    Place at = place_of(a.cache, a.batch, t0, rows, a.status);
    if (a.cos_sin && at.state == 2 && static_cast<uint32_t>(at.p) >= a.max_positions) {
        flag(a.status);
        at.state = 1;
    }
    const uint32_t unit = threadIdx.x % kLanes, k_heads = a.cache.kv_heads, heads = a.q_heads + 2 * k_heads;
    const uint32_t head0 = blockIdx.y * a.passes * kHeads + threadIdx.x / kLanes;
    const bool in_head = unit < kUnits;
    // the unit's part in the rotation: pair partners are `half` units apart, or in the unit itself
    const uint32_t half = a.rotary_dim / 16;
    const bool first = unit < half, turns = a.cos_sin && unit < 2 * half;
    const uint32_t other = first ? unit + half : unit - half;   // only meant where `turns`
    const uint32_t angle = a.interleaved ? unit * 4 : (first ? unit : other) * 8;

    for (uint32_t r = 0; r < rows; ++r) {
        if (__builtin_amdgcn_readlane(at.state, r) != 2) continue;
        const uint64_t t = t0 + r, slot = lane_value(at.slot, r);
        f32x4 c0{}, c1{}, s0{}, s1{};
        if (turns) {
            const int32_t p = __builtin_amdgcn_readlane(at.p, r);
            const SZ_GLOBAL float* row = gptr(a.cos_sin) + static_cast<uint64_t>(p) * a.rotary_dim + angle;
            c0 = *reinterpret_cast<const SZ_GLOBAL f32x4*>(row);
            s0 = *reinterpret_cast<const SZ_GLOBAL f32x4*>(row + a.rotary_dim / 2);
            if (!a.interleaved) {
                c1 = *reinterpret_cast<const SZ_GLOBAL f32x4*>(row + 4);
                s1 = *reinterpret_cast<const SZ_GLOBAL f32x4*>(row + a.rotary_dim / 2 + 4);
            }
        }
        for (uint32_t pass = 0; pass < a.passes; pass += kBatch) {
            u32x4 raws[kBatch];
#pragma unroll
            for (uint32_t i = 0; i < kBatch; ++i) {
                const uint32_t head = head0 + (pass + i) * kHeads;
                raws[i] = u32x4{0, 0, 0, 0};
                if (pass + i >= a.passes || head >= heads || !in_head) continue;
                const SZ_GLOBAL uint16_t* from = head < a.q_heads ? gptr(a.q) + t * a.q_stride + head * D
                                                 : head < a.q_heads + k_heads
                                                     ? gptr(a.k) + t * a.k_stride + (head - a.q_heads) * D
                                                     : gptr(a.v) + t * a.v_stride + (head - a.q_heads - k_heads) * D;
                raws[i] = __builtin_nontemporal_load(reinterpret_cast<const SZ_GLOBAL u32x4*>(from + unit * 8));
            }
#pragma unroll
            for (uint32_t i = 0; i < kBatch; ++i) {
                const uint32_t head = head0 + (pass + i) * kHeads;
                if (pass + i >= a.passes) break;   // the same for the workgroup: the lanes below trade values
                const bool live = head < heads && in_head, is_q = head < a.q_heads, is_v = head >= a.q_heads + k_heads;
                const u32x4 raw = raws[i];
                f32x8 x = to_f32(raw);
                const uint16_t* w = is_v ? nullptr : is_q ? a.q_norm : a.k_norm;
                if (a.q_norm || a.k_norm) {
                    float sum = 0.f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum += x[j] * x[j];
#pragma unroll
                    for (uint32_t m = kLanes / 2; m; m /= 2) sum += __shfl_xor(sum, m, kLanes);
                    if (w && live) {
                        const float scale = 1.f / sqrtf(sum / D + a.eps);
                        const f32x8 g = to_f32(*reinterpret_cast<const SZ_GLOBAL u32x4*>(gptr(w) + unit * 8));
#pragma unroll
                        for (int j = 0; j < 8; ++j) x[j] = x[j] * scale * g[j];
                    }
                }
                if (a.cos_sin) {
                    if (a.interleaved) {
                        if (turns && !is_v) {
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const float u = x[2 * j], v = x[2 * j + 1];
                                x[2 * j] = u * c0[j] - v * s0[j];
                                x[2 * j + 1] = v * c0[j] + u * s0[j];
                            }
                        }
                    } else {
                        f32x8 y;
#pragma unroll
                        for (int j = 0; j < 8; ++j) y[j] = __shfl(x[j], other, kLanes);
                        if (turns && !is_v) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const float c = j < 4 ? c0[j] : c1[j - 4];
                                const float s = j < 4 ? s0[j] : s1[j - 4];
                                x[j] = first ? x[j] * c - y[j] * s : x[j] * c + y[j] * s;
                            }
                        }
                    }
                }
                if (!live) continue;
                const bool copied = is_v || (!w && !a.cos_sin);   // keeps NaN payloads
                const u32x4 rounded = __builtin_bit_cast(u32x4, __builtin_convertvector(x, bf16x8));
                if (is_q) {
                    *reinterpret_cast<SZ_GLOBAL u32x4*>(gptr(a.q_out) + t * a.q_out_stride + head * D + unit * 8) =
                        copied ? raw : rounded;
                    continue;
                }
                const uint32_t h = head - a.q_heads - (is_v ? k_heads : 0);
                SZ_GLOBAL uint8_t* to =
                    gptr(is_v ? a.cache.v : a.cache.k) + slot + h * a.cache.head_stride + unit * (kE5M2 ? 8 : 16);
                if constexpr (kE5M2) *reinterpret_cast<SZ_GLOBAL u32x2*>(to) = to_e5m2(x);
                else *reinterpret_cast<SZ_GLOBAL u32x4*>(to) = copied ? raw : rounded;
            }
        }
    }
}

// Keys and values between pages and layer tensors, 16 bytes a thread and
// step.  a.lanes (a power of two) threads share a token, each with every
// a.lanes-th piece of its keys' and then its values' row; the kThreads /
// a.lanes tokens side by side step through the workgroup's rows, kBatch reads
// in flight.  All reads stream, and what goes to pages does too: 209 us for
// 131072 BF16 tokens, and 228 through the caches.  A gathered layer is stored
// through them, for the call that it was gathered for: 131072 E5M2 tokens take
// 83 us against 96 streamed with the caches warm, 102 against 109 cold.
template <bool kToPages>
__global__ __launch_bounds__(kThreads) void k_copy(CopyArgs a) {
    constexpr uint32_t kBatch = 4;
    check_spans(a.batch, a.status);
    const uint32_t t0 = blockIdx.x * a.rows;
    const uint32_t rows = a.batch.total_tokens - t0 < a.rows ? a.batch.total_tokens - t0 : a.rows;
    const Place at = place_of(a.cache, a.batch, t0, rows, a.status);
    const uint32_t mine = threadIdx.x % a.lanes, side = threadIdx.x / a.lanes, sides = kThreads / a.lanes;
    for (uint32_t i0 = 0; i0 < 2 * a.pieces; i0 += a.lanes) {   // the same steps for every lane: they trade places
        const uint32_t i = i0 + mine;
        const bool is_v = i >= a.pieces;
        const uint32_t u = is_v ? i - a.pieces : i, head = __umulhi(u, a.head_magic);   // u / (head_bytes / 16)
        SZ_GLOBAL uint8_t* paged = gptr(is_v ? a.cache.v : a.cache.k) + head * a.cache.head_stride +
                                   (u - head * (a.head_bytes / 16)) * 16;
        SZ_GLOBAL uint8_t* flat = gptr(is_v ? a.v : a.k) + u * 16;
        const uint64_t stride = is_v ? a.v_stride : a.k_stride;
        for (uint32_t r0 = 0; r0 < rows; r0 += kBatch * sides) {
            u32x4 x[kBatch];
            int32_t state[kBatch];
            uint64_t slot[kBatch];
#pragma unroll
            for (uint32_t k = 0; k < kBatch; ++k) {
                const uint32_t r = r0 + k * sides + side, lane = r < 64 ? r : 0;
                state[k] = __shfl(at.state, lane);
                slot[k] = static_cast<uint64_t>(__shfl(static_cast<uint32_t>(at.slot >> 32), lane)) << 32 |
                          __shfl(static_cast<uint32_t>(at.slot), lane);
                if (r >= rows || i >= 2 * a.pieces || (kToPages && state[k] != 2)) state[k] = 0;
                x[k] = u32x4{0, 0, 0, 0};
                const SZ_GLOBAL uint8_t* from = kToPages ? flat + (t0 + r) * stride : paged + slot[k];
                if (state[k] == 2) x[k] = __builtin_nontemporal_load(reinterpret_cast<const SZ_GLOBAL u32x4*>(from));
            }
#pragma unroll
            for (uint32_t k = 0; k < kBatch; ++k) {
                if (state[k] == 0) continue;
                SZ_GLOBAL uint8_t* to = kToPages ? paged + slot[k] : flat + (t0 + r0 + k * sides + side) * stride;
                if constexpr (kToPages) __builtin_nontemporal_store(x[k], reinterpret_cast<SZ_GLOBAL u32x4*>(to));
                else *reinterpret_cast<SZ_GLOBAL u32x4*>(to) = x[k];
            }
        }
    }
}

// Tokens a workgroup takes: as many as leave 2048 workgroups, 16 at most, a
// power of two.  A workgroup's first accesses wait for its tokens' pages, so
// several tokens share them; at 131072 BF16 tokens 16 of them scatter in
// 209 us and 64 in 219, and at 8192 a workgroup of one token instead of four
// gathers in 18 us instead of 15.
uint32_t rows_each(uint32_t tokens) {
    uint32_t rows = 1;
    while (rows < 16 && tokens / (2 * rows) >= 2048) rows *= 2;
    return rows;
}

uint32_t up_to(uint32_t n, uint32_t of) { return (n + of - 1) / of; }

template <uint32_t D>
hipError_t append_of(AppendArgs& a, hipStream_t s) {
    const uint32_t passes = up_to(a.q_heads + 2 * a.cache.kv_heads, kThreads / lanes_of(D));
    a.passes = a.batch.total_tokens < 1024 ? 1 : passes;
    a.rows = rows_each(a.batch.total_tokens);
    const dim3 grid(up_to(a.batch.total_tokens, a.rows), up_to(passes, a.passes));
    if (a.e5m2) k_append<D, true><<<grid, kThreads, 0, s>>>(a);
    else k_append<D, false><<<grid, kThreads, 0, s>>>(a);
    return hipGetLastError();
}

template <bool kToPages>
hipError_t copy(CopyArgs a, hipStream_t s) {
    const uint32_t per_head = a.head_bytes / 16;
    a.pieces = a.cache.kv_heads * per_head;
    a.head_magic = static_cast<uint32_t>((uint64_t(1) << 32) / per_head + ((uint64_t(1) << 32) % per_head != 0));
    a.lanes = 8;
    while (a.lanes < kThreads && a.lanes < 2 * a.pieces) a.lanes *= 2;
    a.rows = rows_each(a.batch.total_tokens);
    k_copy<kToPages><<<up_to(a.batch.total_tokens, a.rows), kThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_append(AppendArgs a, hipStream_t s) {
    switch (a.cache.head_dim) {
        case 64: return append_of<64>(a, s);
        case 80: return append_of<80>(a, s);
        case 96: return append_of<96>(a, s);
        case 128: return append_of<128>(a, s);
        default: return append_of<256>(a, s);
    }
}

hipError_t launch_gather(const CopyArgs& a, hipStream_t s) { return copy<false>(a, s); }
hipError_t launch_scatter(const CopyArgs& a, hipStream_t s) { return copy<true>(a, s); }

}  // namespace kvi
