// kv_kernels.hip -- the paged KV cache's append (per-head norm, position
// rotation, conversion and paged store in one pass) and the gather and
// scatter between pages and contiguous layer tensors.  The calls are
// documented in include/paged_kv.h.
#include "kv_device.h"

namespace kvi {

namespace {

constexpr uint32_t kThreads = 256;

// The place of token row t, the same for every thread of the workgroup:
// false where nothing is to be done for it.
struct Place {
    uint32_t s;
    int32_t p, page;
};
__device__ inline bool place_of(const Cache& c, const Batch& b, uint32_t t, int32_t* status, Place& at) {
    for (uint32_t s = t; s < b.num_seqs; s += b.total_tokens)   // each sequence is looked at by one workgroup
        if (!span_of(b, s).ok && threadIdx.x == 0) flag(status);
    at.s = wave_seq_of_token(b, t);
    const Span seq = span_of(b, at.s);
    if (static_cast<int32_t>(t) < seq.begin || static_cast<int32_t>(t) >= seq.begin + seq.n) return false;
    at.p = seq.first() + (static_cast<int32_t>(t) - seq.begin);
    if (at.p < 0) {
        at.page = -1;
        return true;
    }
    at.page = page_of(c, b, at.s, at.p);
    if (at.page < 0 && threadIdx.x == 0) flag(status);
    return true;
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

// One token's heads: q heads, then k heads, then v heads.  A head is D / 8
// units of 8 elements on kLanes neighbouring lanes (a power of two, so that
// no head crosses a wave and the norm's sum is a butterfly over them).
template <uint32_t D, bool kE5M2>
__global__ __launch_bounds__(kThreads) void k_append(AppendArgs a) {
    constexpr uint32_t kUnits = D / 8;
    constexpr uint32_t kLanes = kUnits <= 8 ? 8 : kUnits <= 16 ? 16 : 32;
    const uint32_t t = blockIdx.x;
    Place at;
    if (!place_of(a.cache, a.batch, t, a.status, at) || at.page < 0) return;
    if (a.cos_sin && static_cast<uint32_t>(at.p) >= a.max_positions) {
        if (threadIdx.x == 0) flag(a.status);
        return;
    }
    const uint32_t unit = threadIdx.x % kLanes;
    const uint32_t head = blockIdx.y * (kThreads / kLanes) + threadIdx.x / kLanes;
    const uint32_t heads = a.q_heads + 2 * a.cache.kv_heads;
    const bool live = head < heads && unit < kUnits;
    const bool is_q = head < a.q_heads, is_v = head >= a.q_heads + a.cache.kv_heads;
    const uint32_t h = is_q ? head : head - a.q_heads - (is_v ? a.cache.kv_heads : 0);
    const uint16_t* base = is_q ? a.q + t * a.q_stride : is_v ? a.v + t * a.v_stride : a.k + t * a.k_stride;
    u32x4 raw = u32x4{0, 0, 0, 0};
    if (live) raw = *reinterpret_cast<const SZ_GLOBAL u32x4*>(gptr(base) + h * D + unit * 8);
    f32x8 x = to_f32(raw);

    const uint16_t* w = is_v ? nullptr : is_q ? a.q_norm : a.k_norm;
    if (a.q_norm || a.k_norm) {
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += x[j] * x[j];
#pragma unroll
        for (uint32_t m = kLanes / 2; m; m /= 2) sum += __shfl_xor(sum, m, kLanes);
        if (w && live) {
            const float r = 1.f / sqrtf(sum / D + a.eps);
            const f32x8 g = to_f32(*reinterpret_cast<const SZ_GLOBAL u32x4*>(gptr(w) + unit * 8));
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = x[j] * r * g[j];
        }
    }
    if (a.cos_sin) {
        const float* row = a.cos_sin + static_cast<uint64_t>(at.p) * a.rotary_dim;
        const uint32_t half = a.rotary_dim / 16;   // units of half the rotated part
        const bool turns = !is_v && live && unit < 2 * half;
        if (a.interleaved) {
            if (turns) {
                const f32x4 c = *reinterpret_cast<const SZ_GLOBAL f32x4*>(gptr(row) + unit * 4);
                const f32x4 s = *reinterpret_cast<const SZ_GLOBAL f32x4*>(gptr(row) + a.rotary_dim / 2 + unit * 4);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float u = x[2 * j], v = x[2 * j + 1];
                    x[2 * j] = u * c[j] - v * s[j];
                    x[2 * j + 1] = v * c[j] + u * s[j];
                }
            }
        } else {
            const bool first = unit < half;
            const uint32_t other = first ? unit + half : unit - half;   // only meant where `turns`
            f32x8 y;
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = __shfl(x[j], other, kLanes);
            if (turns) {
                const uint32_t i = (first ? unit : other) * 8;
                const SZ_GLOBAL f32x4* cs = reinterpret_cast<const SZ_GLOBAL f32x4*>(gptr(row) + i);
                const SZ_GLOBAL f32x4* sn =
                    reinterpret_cast<const SZ_GLOBAL f32x4*>(gptr(row) + a.rotary_dim / 2 + i);
                const f32x4 c0 = cs[0], c1 = cs[1], s0 = sn[0], s1 = sn[1];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float c = j < 4 ? c0[j] : c1[j - 4];
                    const float s = j < 4 ? s0[j] : s1[j - 4];
                    x[j] = first ? x[j] * c - y[j] * s : x[j] * c + y[j] * s;
                }
            }
        }
    }
    if (!live) return;
    const bool raw_copy = is_v || (!w && !a.cos_sin);   // keeps NaN payloads, and skips the conversion
    const u32x4 rounded = __builtin_bit_cast(u32x4, __builtin_convertvector(x, bf16x8));
    if (is_q) {
        *reinterpret_cast<SZ_GLOBAL u32x4*>(gptr(a.q_out) + t * a.q_out_stride + h * D + unit * 8) =
            raw_copy ? raw : rounded;
        return;
    }
    SZ_GLOBAL uint8_t* to = gptr(is_v ? a.cache.v : a.cache.k) + slot_offset(a.cache, at.page, at.p) +
                            h * a.cache.head_stride + unit * (kE5M2 ? 8 : 16);
    if constexpr (kE5M2) *reinterpret_cast<SZ_GLOBAL u32x2*>(to) = to_e5m2(x);
    else *reinterpret_cast<SZ_GLOBAL u32x4*>(to) = raw_copy ? raw : rounded;
}

// One token's keys and values between its page and its row of the layer
// tensors, 16 bytes a thread at a time.
template <bool kToPages>
__global__ __launch_bounds__(kThreads) void k_copy(CopyArgs a) {
    const uint32_t t = blockIdx.x;
    Place at;
    if (!place_of(a.cache, a.batch, t, a.status, at) || (kToPages && at.page < 0)) return;
    const uint32_t per_head = a.head_bytes / 16, units = a.cache.kv_heads * per_head;
    const uint64_t slot = at.page < 0 ? 0 : slot_offset(a.cache, at.page, at.p);
    for (uint32_t i = threadIdx.x; i < 2 * units; i += kThreads) {
        const bool is_v = i >= units;
        const uint32_t u = is_v ? i - units : i;
        const uint32_t head = u / per_head;
        SZ_GLOBAL u32x4* paged = reinterpret_cast<SZ_GLOBAL u32x4*>(
            gptr(is_v ? a.cache.v : a.cache.k) + slot + head * a.cache.head_stride + (u - head * per_head) * 16);
        SZ_GLOBAL u32x4* flat = reinterpret_cast<SZ_GLOBAL u32x4*>(gptr(is_v ? a.v : a.k) +
                                                                   t * (is_v ? a.v_stride : a.k_stride) + u * 16);
        if constexpr (kToPages) *paged = *flat;
        else *flat = at.page < 0 ? u32x4{0, 0, 0, 0} : *paged;
    }
}

template <uint32_t D>
hipError_t append_of(const AppendArgs& a, hipStream_t s) {
    constexpr uint32_t kLanes = D / 8 <= 8 ? 8 : D / 8 <= 16 ? 16 : 32;
    const uint32_t heads = a.q_heads + 2 * a.cache.kv_heads, per = kThreads / kLanes;
    const dim3 grid(a.batch.total_tokens, (heads + per - 1) / per);
    if (a.e5m2) k_append<D, true><<<grid, kThreads, 0, s>>>(a);
    else k_append<D, false><<<grid, kThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_append(const AppendArgs& a, hipStream_t s) {
    switch (a.cache.head_dim) {
        case 64: return append_of<64>(a, s);
        case 80: return append_of<80>(a, s);
        case 96: return append_of<96>(a, s);
        case 128: return append_of<128>(a, s);
        default: return append_of<256>(a, s);
    }
}

hipError_t launch_gather(const CopyArgs& a, hipStream_t s) {
    k_copy<false><<<a.batch.total_tokens, kThreads, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_scatter(const CopyArgs& a, hipStream_t s) {
    k_copy<true><<<a.batch.total_tokens, kThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace kvi
