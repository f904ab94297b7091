// kv_attention.hip -- attention of new tokens over the paged KV cache
// (include/paged_kv.h, kv_attention).
//
// Mathematics.  For the rows of one sequence under one KV head, with
// c = scale * log2(e):  s_j = q . k_j,  m = max_j c s_j,
// p_j = 2^(c s_j - m),  o = sum_j p_j v_j / sum_j p_j, in one pass over the
// keys: when a block raises m, the sums so far are multiplied by
// 2^(m_old - m).  lse = (m + log2 sum) ln 2.
//
// Layout.  Both products run transposed on the matrix cores, S^T = K Q^T and
// O^T = V^T P^T, so that a lane holds one query row (column of S^T and O^T):
// the row's maximum and sum are kept in that lane, its rescaling multiplies
// that lane's registers, and S^T's result layout is P^T's operand layout once
// the keys of the second product are numbered to fit it (any numbering will
// do as long as V^T has the same).  V^T's operand has the keys along a
// lane's registers: V is staged row-major in LDS and read with the
// transposing 4 x 16 LDS read.
//
// E5M2 is the upper byte of FP16, so an E5M2 cache is expanded by byte
// permutes and multiplied in FP16.  The query row is scaled by a power of
// two that brings its largest element to [2^14, 2^15) before it becomes FP16
// (and c by its inverse): elements down to 2^-28 of the largest keep all of
// BF16's bits, smaller ones lose less than 2^-38 of the largest.
#include "kv_device.h"

namespace kvi {

namespace {

typedef short i16x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kInf = __builtin_inff();

// Pointers into LDS stay in its address space: a cast from a generic pointer
// costs a null check at every use.
#define KV_LDS __attribute__((address_space(3)))
typedef KV_LDS uint8_t* LdsBytes;
template <typename T>
__device__ inline KV_LDS T* lds_as(LdsBytes p) {
    return (KV_LDS T*)p;
}
// 4 x 16 transposing read: 16 lanes give the addresses of 4 rows of 32 bytes
// (4 lanes a row), lane i gets element i of each row
__device__ inline u32x2 read_tr16(LdsBytes p) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(lds_as<i16x4>(p)));
}

// 8 x 16 transposing read of bytes: 2 lanes a row
__device__ inline u32x2 read_tr8(LdsBytes p) {
    typedef int32_t i32x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32(lds_as<i32x2>(p)));
}

// 8 E5M2 bytes -> 8 FP16
__device__ inline u32x4 expand(u32x2 b) {
    return u32x4{sz::perm(0, b[0], 0x010C000Cu), sz::perm(0, b[0], 0x030C020Cu), sz::perm(0, b[1], 0x010C000Cu),
                 sz::perm(0, b[1], 0x030C020Cu)};
}

template <bool kE5M2>
__device__ inline f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
    if constexpr (kE5M2)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

template <bool kE5M2>
__device__ inline u32x4 pack(f32x8 x) {   // to the matrix cores' 16-bit type, nearest even
    if constexpr (kE5M2) return __builtin_bit_cast(u32x4, __builtin_convertvector(x, f16x8));
    else return __builtin_bit_cast(u32x4, __builtin_convertvector(x, bf16x8));
}

template <bool kE5M2>
__device__ inline f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
    if constexpr (kE5M2)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// max or sum over the lanes that hold the same query row (lane, lane ^ 16, lane ^ 32, lane ^ 48)
__device__ inline float swap16(float x, bool hi) {
    const u32x2 r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(hi ? r[1] : r[0]);
}
__device__ inline float swap32(float x, bool hi) {
    const u32x2 r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(hi ? r[1] : r[0]);
}
__device__ inline float row_max(float x) {
    x = fmaxf(swap16(x, false), swap16(x, true));
    return fmaxf(swap32(x, false), swap32(x, true));
}
__device__ inline float row_sum(float x) {
    x = swap16(x, false) + swap16(x, true);
    return swap32(x, false) + swap32(x, true);
}

// A 16-byte piece of a value row as the cache holds it: whether it has Inf or
// NaN, and the piece with 0 in their places.
template <bool kE5M2>
__device__ inline bool not_finite(u32x4 x) {
    bool any = false;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int h = 0; h < 32; h += kE5M2 ? 8 : 16) {
            const uint32_t kExp = (kE5M2 ? 0x7Cu : 0x7F80u) << h;
            any |= (x[i] & kExp) == kExp;
        }
    return any;
}
template <bool kE5M2>
__device__ inline u32x4 finite_part(u32x4 x) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int h = 0; h < 32; h += kE5M2 ? 8 : 16) {
            const uint32_t kExp = (kE5M2 ? 0x7Cu : 0x7F80u) << h;
            if ((x[i] & kExp) == kExp) x[i] &= ~((kE5M2 ? 0xFFu : 0xFFFFu) << h);
        }
    return x;
}

// Adds the Inf and NaN among the 4 values at `from` to 4 sums.
template <bool kE5M2>
__device__ inline void add_not_finite(const SZ_GLOBAL uint8_t* from, float* o) {
    u32x2 x;   // BF16, or the E5M2 bytes as FP16
    if constexpr (kE5M2) {
        const uint32_t b = *reinterpret_cast<const SZ_GLOBAL uint32_t*>(from);
        x = u32x2{sz::perm(0, b, 0x010C000Cu), sz::perm(0, b, 0x030C020Cu)};
    } else {
        x = *reinterpret_cast<const SZ_GLOBAL u32x2*>(from);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t v = x[i / 2] >> (i % 2 * 16) & 0xFFFFu;
        if constexpr (kE5M2) {
            if ((v & 0x7C00u) == 0x7C00u) o[i] += static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(v)));
        } else {
            if ((v & 0x7F80u) == 0x7F80u) o[i] += __uint_as_float(v << 16);
        }
    }
}

// How far (powers of two) a row's maximum may pass the one its sums are
// scaled by before they are rescaled.  FP16 weights lose nothing by it (2 x
// 1000 of 12345 E5M2 keys: 690 us, 725 without).  BF16 ones do: scaled by the
// maximum itself, the largest weight is 1 and is not rounded, and the error
// of peaked rows is a quarter smaller (0.0018 of the result's norm at 64 x 1
// to 8192 keys, 0.0023 with this at 8), which is worth what it takes of long
// chunks (2048 new of 8192: 296 us, 293; a prompt of 8192 tokens under 64
// query heads: 1240, 1167) and nothing elsewhere.
template <bool kE5M2>
constexpr float kSlack = kE5M2 ? 8.f : 0.f;

// FP16 weights are 2^kLift times themselves, the sum with them: at most
// 2^(kSlack + kLift) = 2^15, and those below 2^-14 of a long row's largest
// keep 7 more of the bits that FP16's small exponents would take (131072 of
// 2^-25 each, half a step, were all lost against a weight of 1, and with them
// 2^-8 of the row).
template <bool kE5M2>
constexpr float kLift = kE5M2 ? 7.f : 0.f;

// LDS order inside one wave: its LDS instructions execute in order; this
// keeps the compiler from moving one lane's reads over another's writes.
__device__ inline void wave_lds_order() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
}

// A tile, the same for every lane, with its fields in scalar registers.
__device__ inline Tile scalar(Tile t) {
    auto one = [](int32_t& x) { x = __builtin_amdgcn_readfirstlane(x); };
    one(t.seq.begin);
    one(t.seq.n);
    one(t.seq.kv);
    one(t.seen);
    one(t.lo);
    one(t.hi);
    one(t.p0);
    one(t.p1);
    t.s = uniform(t.s);
    t.row0 = uniform(t.row0);
    t.rows = uniform(t.rows);
    t.any = uniform(t.any);
    return t;
}

// The page ids of a block's keys, a key a lane.  `ask` only loads (an entry
// that exists, whatever the position), so that nothing waits for it before
// `answer` a block later: -1 where the position has no page, or is outside
// [seen, end) and so none is needed.
struct Pages {
    const SZ_GLOBAL int32_t* row;
    uint32_t log2_page, last, num_pages;
    int32_t seen, end;
    bool bad;
    __device__ Pages(const AttentionArgs& a, const Tile& t, int32_t k1)
        : row(gptr(a.batch.pages) + t.s * a.batch.pages_stride), log2_page(a.cache.log2_page),
          last(a.batch.pages_per_seq - 1), num_pages(a.cache.num_pages), seen(t.seen), end(k1), bad(false) {}
    __device__ int32_t ask(int32_t p) const {
        const uint32_t i = static_cast<uint32_t>(p) >> log2_page;
        return row[i < last ? i : last];
    }
    __device__ int32_t answer(int32_t p, int32_t id) {
        if (p < seen || p >= end) return -1;
        const bool ok = static_cast<uint32_t>(p) >> log2_page <= last && static_cast<uint32_t>(id) < num_pages;
        bad |= !ok;
        return ok ? id : -1;
    }
};

// Query row `row` of the tile's sequence: its token and head.
struct RowAt {
    uint32_t token;   // row of the per-token tensors
    uint32_t head;
    int32_t p;
};
__device__ inline RowAt row_at(const Tile& t, uint32_t row, uint32_t group, uint32_t kv_head) {
    const uint32_t i = row / group;
    return RowAt{static_cast<uint32_t>(t.seq.begin) + i, kv_head * group + (row - i * group),
                 t.seq.first() + static_cast<int32_t>(i)};
}

// Writes one row's share: the output where the tile has one split, else the
// sums for k_join.  `put(d, x4)` style stores are done by the callers.
__device__ inline void put_lse(const AttentionArgs& a, const RowAt& r, float m, float l) {
    if (a.lse)
        gptr(a.lse)[static_cast<uint64_t>(r.token) * (a.group * a.cache.kv_heads) + r.head] =
            l == 0.f ? -kInf : (m + __builtin_log2f(l)) * kLn2;
}

// What a unit of the few-rows kernel leaves for k_join_few: the sequence that
// begins in it and goes on in `more` units behind it (0: there is none):
// (more, first token row, rows, 0)
__device__ inline SZ_GLOBAL u32x4* cuts(const AttentionArgs& a) {
    return reinterpret_cast<SZ_GLOBAL u32x4*>(gptr(a.part) + a.plan.parts * (a.cache.head_dim + 2));
}

// The places of a unit's KV head in the partial sums.
__device__ inline uint64_t place_of(const AttentionArgs& a, uint32_t unit, uint32_t kv_head, uint32_t place) {
    return (static_cast<uint64_t>(unit) * a.cache.kv_heads + kv_head) * 2 + place;
}

__device__ inline float* part_stats(const AttentionArgs& a) {
    return a.part + a.plan.parts * a.cache.head_dim;
}

// A query row's operands from BF16 to FP16, scaled by the power of two that
// brings its largest element to [2^14, 2^15); returns c scaled back.
template <uint32_t kFrags, typename Max>
__device__ inline float to_fp16(u32x4* q, float c, Max over_row) {
    float most = 0.f;
#pragma unroll
    for (uint32_t f = 0; f < kFrags; ++f) {
        const f32x8 x = to_f32(q[f]);
#pragma unroll
        for (int j = 0; j < 8; ++j) most = fmaxf(most, fabsf(x[j]));
    }
    most = over_row(most);
    const int32_t up = most > 0.f && most < kInf ? 15 - __builtin_amdgcn_frexp_expf(most) : 0;
#pragma unroll
    for (uint32_t f = 0; f < kFrags; ++f) {
        f32x8 x = to_f32(q[f]);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = __builtin_amdgcn_ldexpf(x[j], up);
        q[f] = pack<true>(x);
    }
    return __builtin_amdgcn_ldexpf(c, -up);
}

// Asks the scheduler to keep kAhead operands' LDS reads (kReads each) in
// flight before each of the block's kCount matrix instructions: left alone it
// reads an operand right before its use and waits for LDS every time.
template <uint32_t kCount, uint32_t kReads, uint32_t kAhead>
__device__ inline void interleave() {
    __builtin_amdgcn_sched_group_barrier(0x100, kReads * kAhead, 0);
#pragma unroll
    for (uint32_t i = 0; i < kCount; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if (i + kAhead < kCount) __builtin_amdgcn_sched_group_barrier(0x100, kReads, 0);
    }
}

// ---- Few rows: a workgroup takes one or two KV heads of its unit's sequences
// (kv_internal.h).  Its W waves, or each W / H of them, take blocks of keys
// in turn, each wave with its own running maximum and sums, joined through LDS
// at the end.  A block goes through the wave's own part of LDS as the cache
// has it: rows are read from memory in one run each, the next block's while
// this one is multiplied.  Bound by memory: a wave has 16 KB (D = 128) of K
// and V on the way, 8 waves a CU.  At D = 128 in BF16, head-major pages, one
// token of two sequences of 131072 keys is read at 6.3 TB/s, of the 7.0 that
// a plain read without caching reaches.
template <uint32_t D>
constexpr uint32_t kKeyRow = 2 * D + 16;   // rows of 16-bit K in LDS: 16-byte reads of 16 rows meet all banks

template <uint32_t D, bool kE5M2, uint32_t W>
struct Few {
    static constexpr uint32_t kKeys = kE5M2 ? 64 : 32;   // a block: 16 KB of K and V either way at D = 128
    static constexpr uint32_t kSize = kE5M2 ? 1 : 2;
    // Rows of whole 128-byte lines are read once and kept in no cache (64 x 1
    // to 8192 keys: 209 us, against 235 with plain loads); neighbouring heads
    // share the lines of others (D = 80, 32 x 5 tokens: 106 us plain, 117).
    static constexpr bool kOwnLines = D * kSize % 128 == 0;
    // rows in LDS; BF16 V: 8 dwords modulo 16, 16 rows of 32 bytes meet all banks
    static constexpr uint32_t kK = D * kSize + 16, kV = kE5M2 ? D + 16 : 2 * D + (D % 32 ? 0 : 32);
    static constexpr uint32_t kStage = kKeys * (kK + kV);
    static constexpr uint32_t kJoin = 16 * (D + 4) * 4;
    static constexpr uint32_t kLds = W * ((kStage > kJoin ? kStage : kJoin) + 16 * 8);
};

// One sequence's rows under H neighbouring KV heads over the positions
// [k0, k1): `whole_row` if these are all that they see, else sums into `place`
// and, for the next head, 2 places on.
template <uint32_t D, bool kE5M2, uint32_t W, uint32_t H>
__device__ inline void attend_few(const AttentionArgs& a, const Tile& t, uint32_t head0, int32_t k0, int32_t k1,
                                  bool whole_row, uint64_t place, uint8_t* lds, uint32_t lane, uint32_t wave) {
    constexpr uint32_t kTeam = W / H;   // waves of a KV head
    const uint32_t kv_head = head0 + wave / kTeam;
    typedef Few<D, kE5M2, W> F;
    constexpr uint32_t kKeys = F::kKeys, kSub = kKeys / 16, kFrags = (D + 31) / 32, kTiles = D / 16;
    constexpr uint32_t kUnits = D * F::kSize / 16;   // 16-byte pieces of a row
    constexpr uint32_t kPer = kKeys * kUnits / 64;   // pieces of K, and of V, a lane has of a block
    const uint32_t g = lane / 16, c16 = lane % 16;

    // Q^T operands: the lane's row c16, elements 32 f + 8 g ..
    const bool live = c16 < t.rows;
    const RowAt at = row_at(t, t.row0 + (live ? c16 : 0), a.group, kv_head);
    const int32_t first = live ? a.mask.first(at.p) : 0, last = live ? a.mask.last(at.p, t.seq.kv) : 0;
    u32x4 q[kFrags];
    const SZ_GLOBAL uint16_t* from = gptr(a.q) + static_cast<uint64_t>(at.token) * a.q_stride + at.head * D;
#pragma unroll
    for (uint32_t f = 0; f < kFrags; ++f)
        q[f] = live && 32 * f + 8 * g < D ? *reinterpret_cast<const SZ_GLOBAL u32x4*>(from + 32 * f + 8 * g)
                                          : u32x4{0, 0, 0, 0};
    float c = a.scale * kLog2e;
    if constexpr (kE5M2) c = to_fp16<kFrags>(q, c, [](float x) { return row_max(x); });
    c = fminf(fmaxf(c, 1.17549435e-38f), 3.402823466e38f);   // masked scores times c are -Inf and zeros 0, not NaN

    f32x4 o[kTiles];
#pragma unroll
    for (uint32_t d = 0; d < kTiles; ++d) o[d] = f32x4{0.f, 0.f, 0.f, 0.f};
    float m = -kInf, l = 0.f;

    const LdsBytes keys = (LdsBytes)lds + wave * F::kStage;
    const LdsBytes values = keys + kKeys * F::kK;
    const SZ_GLOBAL uint8_t* pool_k = gptr(a.cache.k) + kv_head * a.cache.head_stride;
    const SZ_GLOBAL uint8_t* pool_v = gptr(a.cache.v) + kv_head * a.cache.head_stride;
    Pages table(a, t, k1);
    const int32_t mine_at = static_cast<int32_t>(lane % kKeys);   // the key whose page this lane looks up

    // Keys without a page are loaded from page 0: their scores are masked,
    // their values get weight 0.
    u32x4 kreg[kPer], vreg[kPer];
    auto load = [&](int32_t kb, int32_t pages) {
#pragma unroll
        for (uint32_t j = 0; j < kPer; ++j) {
            const uint32_t u = lane + 64 * j, key = u / kUnits, col = u % kUnits;
            const int32_t page = __shfl(pages, key);
            const uint64_t off = slot_offset(a.cache, page < 0 ? 0 : page, kb + static_cast<int32_t>(key)) + col * 16;
            const SZ_GLOBAL u32x4* k = reinterpret_cast<const SZ_GLOBAL u32x4*>(pool_k + off);
            const SZ_GLOBAL u32x4* v = reinterpret_cast<const SZ_GLOBAL u32x4*>(pool_v + off);
            kreg[j] = F::kOwnLines ? __builtin_nontemporal_load(k) : *k;
            vreg[j] = F::kOwnLines ? __builtin_nontemporal_load(v) : *v;
        }
    };

    const int32_t step = kTeam * kKeys;
    int32_t kb = k0 + static_cast<int32_t>(wave % kTeam * kKeys);
    int32_t pages = -1, asked = -1;
    if (kb < k1) {
        pages = table.answer(kb + mine_at, table.ask(kb + mine_at));
        asked = table.ask(kb + step + mine_at);
        load(kb, pages);
    }
    for (; kb < k1; kb += step) {
        const bool more = kb + step < k1;
        const int32_t here_pages = pages;
        const uint64_t here = __ballot(pages >= 0);   // bit key: it has a page
        // every row sees every key of the block?
        const bool whole = here == ~0ull && kb >= a.mask.first(t.p1) &&
                           kb + static_cast<int32_t>(kKeys) <= a.mask.last(t.p0, t.seq.kv);
        bool special = false;   // a weight of 0 does not keep Inf and NaN out of the product
        if (!whole)
#pragma unroll
            for (uint32_t j = 0; j < kPer; ++j) {
                special |= not_finite<kE5M2>(vreg[j]);
                vreg[j] = finite_part<kE5M2>(vreg[j]);
            }
        wave_lds_order();
#pragma unroll
        for (uint32_t j = 0; j < kPer; ++j) {
            const uint32_t u = lane + 64 * j, key = u / kUnits, col = u % kUnits;
            *lds_as<u32x4>(keys + key * F::kK + col * 16) = kreg[j];
            *lds_as<u32x4>(values + key * F::kV + col * 16) = vreg[j];
        }
        wave_lds_order();
        if (more) {
            pages = table.answer(kb + step + mine_at, asked);
            asked = table.ask(kb + 2 * step + mine_at);
            load(kb + step, pages);
        }
        f32x4 s[kSub];
#pragma unroll
        for (uint32_t kt = 0; kt < kSub; ++kt) {
            s[kt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (uint32_t f = 0; f < kFrags; ++f) {
                const LdsBytes p = keys + (16 * kt + c16) * F::kK + (32 * f + 8 * g) * F::kSize;
                u32x4 x;
                if constexpr (kE5M2) x = expand(*lds_as<u32x2>(p));
                else x = *lds_as<u32x4>(p);
                // past the row's end (D = 80) Q is 0, and K must be too: LDS holds anything there
                if (32 * f + 32 > D && 32 * f + 8 * g >= D) x = u32x4{0, 0, 0, 0};
                s[kt] = mfma16<kE5M2>(x, q[f], s[kt]);
            }
        }
        if (!whole) {
            const int32_t lo = first - kb - static_cast<int32_t>(4 * g), hi = last - kb - static_cast<int32_t>(4 * g);
            const uint64_t mine = here >> (4 * g);
#pragma unroll
            for (uint32_t kt = 0; kt < kSub; ++kt)
#pragma unroll
                for (uint32_t j = 0; j < 4; ++j) {
                    const int32_t i = static_cast<int32_t>(16 * kt + j);   // key i + 4 g
                    s[kt][j] = i >= lo && i < hi && (mine >> i & 1) ? s[kt][j] : -kInf;
                }
        }
        float top = s[0][0];
#pragma unroll
        for (uint32_t i = 1; i < 4 * kSub; ++i) top = fmaxf(top, s[i / 4][i % 4]);
        top = row_max(top) * c;
        if (__any(top > m + kSlack<kE5M2>)) {
            const float now = fmaxf(m, top), r = now == -kInf ? 1.f : __builtin_amdgcn_exp2f(m - now);
            m = now;
            l *= r;
#pragma unroll
            for (uint32_t d = 0; d < kTiles; ++d) o[d] *= r;
        }
        const float base = m == -kInf ? 0.f : m - kLift<kE5M2>;
        u32x4 p[kSub / 2];
#pragma unroll
        for (uint32_t kk = 0; kk < kSub / 2; ++kk) {
            f32x8 e;
#pragma unroll
            for (uint32_t i = 0; i < 8; ++i) {
                e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[2 * kk + i / 4][i % 4], c, -base));
                l += e[i];
            }
            p[kk] = pack<kE5M2>(e);
        }
#pragma unroll
        for (uint32_t kk = 0; kk < kSub / 2; ++kk)
#pragma unroll
            for (uint32_t d = 0; d < kTiles; ++d) {
                // V^T operand: element 16 d + c16 of the keys 32 kk + 4 g .. + 3 and 32 kk + 16 + 4 g .. + 3
                u32x4 v;
                if constexpr (kE5M2) {   // 2 lanes a row
                    const uint32_t r = c16 / 2, key = 32 * kk + 4 * g + r % 4 + r / 4 * 16;
                    v = expand(read_tr8(values + key * F::kV + 16 * d + c16 % 2 * 8));
                } else {                 // 4 lanes a row
                    const LdsBytes row = values + (32 * kk + 4 * g + c16 / 4) * F::kV + 32 * d + c16 % 4 * 8;
                    const u32x2 lo = read_tr16(row), hi = read_tr16(row + 16 * F::kV);
                    v = u32x4{lo[0], lo[1], hi[0], hi[1]};
                }
                o[d] = mfma16<kE5M2>(v, p[kk], o[d]);
            }
        if (__any(special)) {   // to the rows that see them
#pragma unroll 1
            for (uint32_t key = 0; key < kKeys; ++key) {
                const int32_t pos = kb + static_cast<int32_t>(key), page = __builtin_amdgcn_readlane(here_pages, key);
                if (page < 0 || pos < first || pos >= last) continue;
                const SZ_GLOBAL uint8_t* row = pool_v + slot_offset(a.cache, page, pos);
#pragma unroll
                for (uint32_t d = 0; d < kTiles; ++d) {
                    float x[4] = {o[d][0], o[d][1], o[d][2], o[d][3]};
                    add_not_finite<kE5M2>(row + (16 * d + 4 * g) * F::kSize, x);
                    o[d] = f32x4{x[0], x[1], x[2], x[3]};
                }
            }
        }
    }
    if (__any(table.bad) && lane == 0) flag(a.status);

    // ---- join the waves
    KV_LDS f32x2* stats = lds_as<f32x2>((LdsBytes)lds + (F::kLds - W * 16 * 8));   // [wave][row]
    KV_LDS float* sums = lds_as<float>((LdsBytes)lds);                                   // [wave][row][D + 4]
    l = row_sum(l);
    __syncthreads();   // the stages have been read
    if (g == 0) stats[wave * 16 + c16] = f32x2{m - kLift<kE5M2>, l};
#pragma unroll
    for (uint32_t d = 0; d < kTiles; ++d)
        *(KV_LDS f32x4*)(sums + (wave * 16 + c16) * (D + 4) + 16 * d + 4 * g) = o[d];
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < H * t.rows * (D / 4); i += 64 * W) {
        const uint32_t all = i / (D / 4), d4 = i % (D / 4) * 4, team = all / t.rows, row = all - team * t.rows;
        float top = -kInf;
        f32x2 st[kTeam];
#pragma unroll
        for (uint32_t w = 0; w < kTeam; ++w) {
            st[w] = stats[(team * kTeam + w) * 16 + row];
            top = fmaxf(top, st[w][0]);
        }
        const float base = top == -kInf ? 0.f : top;
        f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
        float sum = 0.f;
#pragma unroll
        for (uint32_t w = 0; w < kTeam; ++w) {
            const float r = __builtin_amdgcn_exp2f(st[w][0] - base);
            sum += r * st[w][1];
            acc += r * *(KV_LDS f32x4*)(sums + ((team * kTeam + w) * 16 + row) * (D + 4) + d4);
        }
        const RowAt to = row_at(t, t.row0 + row, a.group, head0 + team);
        if (whole_row) {
            const float inv = 1.f / sum;
            f32x4 y;
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = sum == 0.f ? 0.f : acc[j] * inv;
            *reinterpret_cast<SZ_GLOBAL u32x2*>(gptr(a.out) + static_cast<uint64_t>(to.token) * a.out_stride +
                                                to.head * D + d4) =
                __builtin_bit_cast(u32x2, __builtin_convertvector(y, bf16x4));
            if (d4 == 0) put_lse(a, to, base, sum);
        } else {
            const uint64_t r = (place + 2 * team) * kFewRows + row;
            *reinterpret_cast<SZ_GLOBAL f32x4*>(gptr(a.part) + r * D + d4) = acc;
            if (d4 == 0) *reinterpret_cast<SZ_GLOBAL f32x2*>(gptr(part_stats(a)) + 2 * r) = f32x2{base, sum};
        }
    }
    __syncthreads();   // the sums have been read: the next sequence's blocks may take their place
}

template <uint32_t D, bool kE5M2, uint32_t W, uint32_t H>
__global__ __launch_bounds__(64 * W, W == 8 ? 2 : few_a_cu(D, kE5M2)) void k_attend_few(AttentionArgs a) {
    __shared__ __align__(16) uint8_t lds[Few<D, kE5M2, W>::kLds];
    // Workgroups go to the 8 XCDs in turn.  The KV heads of a unit go to one
    // of them, one after the other: in a token-major page their rows are
    // neighbours, and lines that two rows share are read into one L2.
    const uint32_t turn = blockIdx.x / 8, teams = a.cache.kv_heads / H, kv_head = turn % teams * H;
    const uint32_t unit = turn / teams * 8 + blockIdx.x % 8;
    if (kv_head == 0 && threadIdx.x == 0)
        for (uint32_t s = unit; s < a.batch.num_seqs; s += a.plan.units ? a.plan.units : a.batch.num_seqs)
            if (!span_of(a.batch, s).ok) flag(a.status);
    const uint32_t lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64);

    // the unit's granules [start, end) of all, and the sequence s they begin in, with `before` granules before it
    uint32_t s = unit, before = 0, start = 0, end = ~0u;
    if (a.plan.units) {
        const uint32_t total = wave_granules(a.batch, a.mask, a.group, a.plan.granule);
        const uint32_t each = granules_each(total, a.plan.units, a.plan.least);
        if (static_cast<uint64_t>(unit) * each >= total) {
            if (unit < a.plan.units && kv_head == 0 && threadIdx.x == 0) cuts(a)[unit] = u32x4{0, 0, 0, 0};
            return;
        }
        start = unit * each;
        end = total - start < each ? total : start + each;
        s = wave_seq_of_granule(a.batch, a.mask, a.group, a.plan.granule, start, before);
    }
    u32x4 cut = u32x4{0, 0, 0, 0};
    for (; s < a.batch.num_seqs && before < end; ++s) {
        const Tile t = scalar(tile_of_seq(a.batch, a.mask, s, a.group));
        if (!t.any) {
            if (!a.plan.units) return;
            continue;
        }
        const uint32_t granules = granules_of(t, a.plan.granule);
        const uint32_t from = before < start ? start - before : 0, to = end - before < granules ? end - before : granules;
        const bool whole = from == 0 && to == granules;
        const uint64_t place = place_of(a, unit, kv_head, before < start ? 0 : 1);
        const int32_t k0 = t.lo + static_cast<int32_t>(from * a.plan.granule);
        const int32_t k1 = to == granules ? t.hi : t.lo + static_cast<int32_t>(to * a.plan.granule);
        attend_few<D, kE5M2, W, H>(a, t, kv_head, k0, k1, whole, place, lds, lane, wave);
        if (!a.plan.units) return;
        if (before >= start && !whole)
            cut = u32x4{(before + granules - 1) / (end - start) - unit, static_cast<uint32_t>(t.seq.begin), t.rows, 0};
        before += granules;
    }
    if (a.plan.units && kv_head == 0 && threadIdx.x == 0) cuts(a)[unit] = cut;
}

// ---- Many rows: tiles of 128 or 256 rows, 32 a wave; the 4 or 8 waves share
// tiles of N keys and values in LDS, two of each, so that one barrier a tile
// does: the next tile's 16-byte pieces are on their way into registers while
// this one is multiplied, and are put into the other buffer behind it.
// A lane's row needs 32 x D of K and of V from LDS for 4 x 32 x N x D
// operations; with fewer rows a wave, LDS would bound it.  What bounds it is
// the work between the products (a wave and tile of 64 keys: 1024 cycles of
// matrix instructions, about as many of vector ones), which overlaps with the
// other wave of the SIMD only in part: 2048 new of 8192 keys at D = 128, 32
// query heads, 275 us in tiles of 256 rows, 875 TFLOP/s of the 1330 that a
// large library product reaches here.  Taking turns by barriers (one half of
// the workgroup multiplies while the other computes weights) was no better
// than leaving them alone.
template <uint32_t D>
constexpr uint32_t kValueRow = ((2 * D + 63) / 64 | 1) * 64;      // V rows: 4 rows of 64 bytes meet all banks

template <uint32_t D, bool kE5M2, uint32_t N, uint32_t W>
__global__ __launch_bounds__(64 * W, D <= 128 ? 2 : 1) void k_attend_tile(AttentionArgs a) {
    constexpr uint32_t M = 32 * W, kTileThreads = 64 * W, kFrags = D / 16, kTiles = (D + 31) / 32, kSub = N / 32;
    constexpr uint32_t kSize = kE5M2 ? 1 : 2, kUnits = D * kSize / 16;   // 16-byte pieces of a row of the cache
    constexpr uint32_t kPieces = N * kUnits, kPer = (kPieces + kTileThreads - 1) / kTileThreads;
    constexpr uint32_t kBuffer = N * (kKeyRow<D> + kValueRow<D>);
    __shared__ __align__(16) uint8_t lds[2 * kBuffer];
    __shared__ int32_t marks[2];   // first key of the tile in each buffer, if Inf or NaN were left out of it
    const uint32_t kv_head = blockIdx.x % a.cache.kv_heads;
    // a sequence's last tiles, which see the most keys, first
    const uint64_t slot = (gridDim.x - 1 - blockIdx.x) / a.cache.kv_heads;
    if (kv_head == 0 && blockIdx.y == 0 && slot < a.batch.num_seqs && threadIdx.x == 0 &&
        !span_of(a.batch, static_cast<uint32_t>(slot)).ok)
        flag(a.status);
    const Tile t = scalar(wave_tile_of(a.batch, a.mask, slot, a.group, M));
    if (!t.any) return;
    const uint32_t splits = splits_of(t, a.plan.split_len);
    if (blockIdx.y && blockIdx.y >= splits) return;
    const int32_t k0 = t.lo + static_cast<int32_t>(blockIdx.y * a.plan.split_len);
    const int32_t k1 = t.hi - k0 < static_cast<int32_t>(a.plan.split_len) ? t.hi : k0 + static_cast<int32_t>(a.plan.split_len);

    const uint32_t lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64), half = lane / 32, c32 = lane % 32;

    // Q^T operands: the lane's row, elements 16 f + 8 half ..
    const uint32_t row = 32 * wave + c32;
    const bool live = row < t.rows;
    const RowAt at = row_at(t, t.row0 + (live ? row : 0), a.group, kv_head);
    const int32_t first = live ? a.mask.first(at.p) : 0, last = live ? a.mask.last(at.p, t.seq.kv) : 0;
    // positions of the wave's first and last row: what all of its rows see, and what any does
    const bool wave_live = 32 * wave < t.rows;
    const uint32_t wave_end = 32 * wave + 31 < t.rows ? 32 * wave + 31 : t.rows - 1;
    const int32_t wave_p0 = t.seq.first() + static_cast<int32_t>((t.row0 + (wave_live ? 32 * wave : 0)) / a.group);
    const int32_t wave_p1 = t.seq.first() + static_cast<int32_t>((t.row0 + wave_end) / a.group);
    const int32_t all_from = a.mask.first(wave_p1), all_to = a.mask.last(wave_p0, t.seq.kv);
    const int32_t any_from = a.mask.first(wave_p0), any_to = wave_live ? a.mask.last(wave_p1, t.seq.kv) : 0;

    u32x4 q[kFrags];
    const SZ_GLOBAL uint16_t* from = gptr(a.q) + static_cast<uint64_t>(at.token) * a.q_stride + at.head * D;
#pragma unroll
    for (uint32_t f = 0; f < kFrags; ++f)
        q[f] = live ? *reinterpret_cast<const SZ_GLOBAL u32x4*>(from + 16 * f + 8 * half) : u32x4{0, 0, 0, 0};
    float c = a.scale * kLog2e;
    if constexpr (kE5M2) c = to_fp16<kFrags>(q, c, [](float x) { return fmaxf(swap32(x, false), swap32(x, true)); });
    c = fminf(fmaxf(c, 1.17549435e-38f), 3.402823466e38f);   // masked scores times c are -Inf and zeros 0, not NaN

    f32x16 o[kTiles];
#pragma unroll
    for (uint32_t d = 0; d < kTiles; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
    float m = -kInf, l = 0.f;

    const SZ_GLOBAL uint8_t* pool_k = gptr(a.cache.k) + kv_head * a.cache.head_stride;
    const SZ_GLOBAL uint8_t* pool_v = gptr(a.cache.v) + kv_head * a.cache.head_stride;
    Pages table(a, t, k1);
    const int32_t mine_at = static_cast<int32_t>(lane % N);   // the key whose page this lane looks up
    u32x4 kreg[kPer], vreg[kPer];
    // Tiles begin at multiples of N, so a key's slot is its own part of it, the same in every tile, and in pages of
    // more than a tile the tile's first slot.
    const uint32_t page_mask = (1u << a.cache.log2_page) - 1;
    uint64_t own[kPer];
#pragma unroll
    for (uint32_t j = 0; j < kPer; ++j) {
        const uint32_t u = threadIdx.x + kTileThreads * j;
        own[j] = (u / kUnits % N & page_mask) * a.cache.token_stride + u % kUnits * 16;
    }
    // Keys without a page are loaded from page 0: their scores are masked, their values get weight 0.
    auto load = [&](int32_t kb, int32_t pages) {
        const uint64_t first_slot = (static_cast<uint32_t>(kb) & page_mask & ~(N - 1)) * a.cache.token_stride;
#pragma unroll
        for (uint32_t j = 0; j < kPer; ++j) {
            const int32_t page = __shfl(pages, (threadIdx.x + kTileThreads * j) / kUnits % N);
            const uint64_t off = static_cast<uint32_t>(page < 0 ? 0 : page) * a.cache.page_stride + (own[j] + first_slot);
            kreg[j] = *reinterpret_cast<const SZ_GLOBAL u32x4*>(pool_k + off);
            vreg[j] = *reinterpret_cast<const SZ_GLOBAL u32x4*>(pool_v + off);
        }
    };
    // Rows of the tile all see all of [all_from, all_to); a tile of keys that
    // is not inside, or has keys without a page, is an edge.
    const int32_t tile_from = a.mask.first(t.p1), tile_to = a.mask.last(t.p0, t.seq.kv);
    auto is_edge = [&](int32_t kb, uint64_t here) {
        return here != ~0ull || kb < tile_from || kb + static_cast<int32_t>(N) > tile_to;
    };
    // The pieces into LDS, as 16-bit values.  On an edge a weight of 0 would
    // not keep an Inf or NaN out of the product: they are left out, and the
    // buffer's mark says so.
    auto put = [&](uint32_t turn, int32_t kb, bool edge) {
        const LdsBytes buffer = (LdsBytes)lds + turn * kBuffer;
        if (edge) {
            bool special = false;
#pragma unroll
            for (uint32_t j = 0; j < kPer; ++j) {
                special |= not_finite<kE5M2>(vreg[j]);
                vreg[j] = finite_part<kE5M2>(vreg[j]);
            }
            if (special) marks[turn] = kb;
        }
#pragma unroll
        for (uint32_t j = 0; j < kPer; ++j) {
            const uint32_t u = threadIdx.x + kTileThreads * j, key = u / kUnits, col = u % kUnits;
            if (kPieces % kTileThreads && u >= kPieces) break;
            const LdsBytes k = buffer + key * kKeyRow<D>, v = buffer + N * kKeyRow<D> + key * kValueRow<D>;
            if constexpr (kE5M2) {
                *lds_as<u32x4>(k + col * 32) = expand(u32x2{kreg[j][0], kreg[j][1]});
                *lds_as<u32x4>(k + col * 32 + 16) = expand(u32x2{kreg[j][2], kreg[j][3]});
                *lds_as<u32x4>(v + col * 32) = expand(u32x2{vreg[j][0], vreg[j][1]});
                *lds_as<u32x4>(v + col * 32 + 16) = expand(u32x2{vreg[j][2], vreg[j][3]});
            } else {
                *lds_as<u32x4>(k + col * 16) = kreg[j];
                *lds_as<u32x4>(v + col * 16) = vreg[j];
            }
        }
    };

    constexpr int32_t kStep = static_cast<int32_t>(N);
    int32_t pages = -1, asked = -1;
    if (k0 < k1) {
        pages = table.answer(k0 + mine_at, table.ask(k0 + mine_at));
        asked = table.ask(k0 + kStep + mine_at);
        load(k0, pages);
        if (threadIdx.x < 2) marks[threadIdx.x] = -1;
        __syncthreads();
        put(0, k0, is_edge(k0, __ballot(pages >= 0)));
    }
    uint32_t turn = 0;
    for (int32_t kb = k0; kb < k1; kb += kStep, turn ^= 1) {
        const bool more = kb + kStep < k1;
        const int32_t here_pages = pages;
        const uint64_t here = __ballot(pages >= 0);   // bit key: it has a page
        const LdsBytes buffer = (LdsBytes)lds + turn * kBuffer;
        __syncthreads();   // this tile is in LDS; the other buffer has been read by every wave
        auto fetch = [&] {
            if (!more) return;
            pages = table.answer(kb + kStep + mine_at, asked);
            asked = table.ask(kb + 2 * kStep + mine_at);
            load(kb + kStep, pages);
        };
        if (kb < any_to && kb + kStep > any_from) {
            f32x16 s[kSub];
#pragma unroll
            for (uint32_t kt = 0; kt < kSub; ++kt)
#pragma unroll
                for (int i = 0; i < 16; ++i) s[kt][i] = 0.f;
#pragma unroll
            for (uint32_t f = 0; f < kFrags; ++f)
#pragma unroll
                for (uint32_t kt = 0; kt < kSub; ++kt) {
                    const u32x4 x = *lds_as<u32x4>(buffer + (32 * kt + c32) * kKeyRow<D> + 32 * f + 16 * half);
                    s[kt] = mfma32<kE5M2>(x, q[f], s[kt]);
                }
            interleave<kFrags * kSub, 1, 4>();
            fetch();   // behind the first product: its operands' registers are then free
            const bool whole = here == ~0ull && kb >= all_from && kb + kStep <= all_to;
            if (!whole) {
                const int32_t from = first - kb - static_cast<int32_t>(4 * half), to = last - kb - static_cast<int32_t>(4 * half);
#pragma unroll
                for (uint32_t kt = 0; kt < kSub; ++kt) {
                    const uint32_t mine = static_cast<uint32_t>(here >> (32 * kt)) >> (4 * half);
#pragma unroll
                    for (uint32_t i = 0; i < 16; ++i) {
                        const int32_t key = static_cast<int32_t>(8 * (i / 4) + i % 4);   // and 32 kt + 4 half
                        const bool sees = key + static_cast<int32_t>(32 * kt) >= from && key + static_cast<int32_t>(32 * kt) < to &&
                                          (mine >> key & 1);
                        s[kt][i] = sees ? s[kt][i] : -kInf;
                    }
                }
            }
            float top = s[0][0];
#pragma unroll
            for (uint32_t i = 1; i < 16 * kSub; ++i) top = fmaxf(top, s[i / 16][i % 16]);
            top = fmaxf(swap32(top, false), swap32(top, true)) * c;
            if (__any(top > m + kSlack<kE5M2>)) {
                const float now = fmaxf(m, top), r = now == -kInf ? 1.f : __builtin_amdgcn_exp2f(m - now);
                m = now;
                l *= r;
#pragma unroll
                for (uint32_t d = 0; d < kTiles; ++d)
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[d][i] *= r;
            }
            const float base = m == -kInf ? 0.f : m - kLift<kE5M2>;
            auto weights = [&](uint32_t kk) {   // P^T operand of keys 16 kk ..
                f32x8 e;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kk / 2][8 * (kk % 2) + i], c, -base));
                    l += e[i];
                }
                return pack<kE5M2>(e);
            };
            const LdsBytes values = buffer + N * kKeyRow<D>;
            const LdsBytes read = values + (4 * half + lane % 16 / 4) * kValueRow<D> + c32 / 16 * 32 + lane % 4 * 8;
            __builtin_amdgcn_s_setprio(1);   // ahead of a wave at its scores (2 x 1000 of 12345: 690 us, 727 without)
#pragma unroll
            for (uint32_t kk = 0; kk < 2 * kSub; ++kk) {
                const u32x4 p = weights(kk);
#pragma unroll
                for (uint32_t d = 0; d < kTiles; ++d) {
                    const u32x2 lo = read_tr16(read + 16 * kk * kValueRow<D> + 64 * d);
                    const u32x2 hi = read_tr16(read + (16 * kk + 8) * kValueRow<D> + 64 * d);
                    o[d] = mfma32<kE5M2>(u32x4{lo[0], lo[1], hi[0], hi[1]}, p, o[d]);
                }
            }
            interleave<2 * kSub * kTiles, 2, 4>();
            __builtin_amdgcn_s_setprio(0);
            if (is_edge(kb, here) && marks[turn] == kb) {   // Inf and NaN, to the rows that see them
#pragma unroll 1
                for (uint32_t key = 0; key < N; ++key) {
                    const int32_t p = kb + static_cast<int32_t>(key), page = __builtin_amdgcn_readlane(here_pages, key);
                    if (page < 0 || p < first || p >= last) continue;
                    const SZ_GLOBAL uint8_t* from_v = pool_v + slot_offset(a.cache, page, p);
#pragma unroll
                    for (uint32_t d = 0; d < kTiles; ++d)
#pragma unroll
                        for (uint32_t b = 0; b < 4; ++b) {
                            if (32 * d + 8 * b >= D) continue;
                            float x[4] = {o[d][4 * b], o[d][4 * b + 1], o[d][4 * b + 2], o[d][4 * b + 3]};
                            add_not_finite<kE5M2>(from_v + (32 * d + 8 * b + 4 * half) * kSize, x);
#pragma unroll
                            for (int i = 0; i < 4; ++i) o[d][4 * b + i] = x[i];
                        }
                }
            }
        } else {
            fetch();
        }
        if (more) put(turn ^ 1, kb + kStep, is_edge(kb + kStep, __ballot(pages >= 0)));
    }
    if (__any(table.bad) && lane == 0) flag(a.status);

    const float sum = swap32(l, false) + swap32(l, true);
    const float base = m == -kInf ? 0.f : m - kLift<kE5M2>;
    if (splits <= 1) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        SZ_GLOBAL uint16_t* to = gptr(a.out) + static_cast<uint64_t>(at.token) * a.out_stride + at.head * D;
#pragma unroll
        for (uint32_t d = 0; d < kTiles; ++d) {
            // a lane has 4 of each 8 elements, its other half the other 4: after
            // the exchange each has 8 in a row of every other 8
#pragma unroll
            for (uint32_t b = 0; b < 2; ++b) {
                f32x8 y;
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = sum == 0.f ? 0.f : o[d][8 * b + i] * inv;
                const u32x4 w = pack<false>(y);
                const u32x2 e = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
                const u32x2 f = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
                const uint32_t at8 = 32 * d + 16 * b + 8 * half;
                if (live && at8 < D) *reinterpret_cast<SZ_GLOBAL u32x4*>(to + at8) = u32x4{e[0], f[0], e[1], f[1]};
            }
        }
        if (live && half == 0) put_lse(a, at, base, sum);
    } else if (live) {
        const uint64_t r = (static_cast<uint64_t>(at.token) * (a.group * a.cache.kv_heads) + at.head) * a.plan.splits + blockIdx.y;
#pragma unroll
        for (uint32_t d = 0; d < kTiles; ++d)
#pragma unroll
            for (uint32_t b = 0; b < 4; ++b) {
                const uint32_t at4 = 32 * d + 8 * b + 4 * half;
                if (at4 < D)
                    *reinterpret_cast<SZ_GLOBAL f32x4*>(gptr(a.part) + r * D + at4) =
                        f32x4{o[d][4 * b], o[d][4 * b + 1], o[d][4 * b + 2], o[d][4 * b + 3]};
            }
        if (half == 0) *reinterpret_cast<SZ_GLOBAL f32x2*>(gptr(part_stats(a)) + 2 * r) = f32x2{base, sum};
    }
}

// A row's output from its parts, one wave a row: part z (below n) is
// part_of(z).  The parts' weights are computed by a lane each, 64 at a time.
template <uint32_t D, typename Part>
__device__ inline void join_row(const AttentionArgs& a, uint32_t token, uint32_t head, uint32_t n, Part part_of) {
    constexpr uint32_t kWide = D <= 64 ? 1 : D <= 128 ? 2 : 4;   // elements a lane
    typedef float Vec __attribute__((ext_vector_type(kWide)));
    typedef __bf16 Out __attribute__((ext_vector_type(kWide)));
    const uint32_t lane = sz::lane_id(), at = lane * kWide < D ? lane * kWide : 0;
    const SZ_GLOBAL f32x2* stats = reinterpret_cast<const SZ_GLOBAL f32x2*>(gptr(part_stats(a)));
    float base = -kInf, sum = 0.f;
    Vec acc = Vec(0.f);
    constexpr uint32_t kAhead = 8;   // parts in flight; past the last, the last again, not added
    for (uint32_t from = 0; from < n; from += 64) {
        const uint32_t count = n - from < 64 ? n - from : 64;
        const f32x2 st = lane < count ? stats[part_of(from + lane)] : f32x2{-kInf, 0.f};
        Vec x[kAhead];
        auto take = [&](uint32_t z) {
#pragma unroll
            for (uint32_t i = 0; i < kAhead; ++i) {
                const uint32_t part = from + (z + i < count ? z + i : count - 1);
                x[i] = *reinterpret_cast<const SZ_GLOBAL Vec*>(gptr(a.part) + part_of(part) * D + at);
            }
        };
        take(0);
        float top = st[1] != 0.f ? st[0] : -kInf;   // a part whose keys the row does not see has no maximum
        for (uint32_t m = 32; m; m /= 2) top = fmaxf(top, __shfl_xor(top, m));
        const float now = fmaxf(base, top), safe = now == -kInf ? 0.f : now;
        const float keep = __builtin_amdgcn_exp2f(base - safe);
        base = now;
        const float weight = st[1] != 0.f ? __builtin_amdgcn_exp2f(st[0] - safe) : 0.f;
        float add = st[1] != 0.f ? weight * st[1] : 0.f;
        for (uint32_t m = 32; m; m /= 2) add += __shfl_xor(add, m);
        sum = sum * keep + add;
        acc *= keep;
        for (uint32_t z = 0; z < count; z += kAhead) {
            if (z) take(z);
#pragma unroll
            for (uint32_t i = 0; i < kAhead; ++i) acc += z + i < count ? __shfl(weight, z + i) * x[i] : Vec(0.f);
        }
    }
    Vec y = acc / sum;
    if (sum == 0.f) y = Vec(0.f);
    if (lane * kWide < D)
        *reinterpret_cast<SZ_GLOBAL Out*>(gptr(a.out) + static_cast<uint64_t>(token) * a.out_stride + head * D + at) =
            __builtin_convertvector(y, Out);
    if (lane == 0) put_lse(a, RowAt{token, head, 0}, base == -kInf ? 0.f : base, sum);
}

constexpr uint32_t kJoinThreads = 256;

// The sequences that were cut: a workgroup has 4 rows of one unit and KV head.
template <uint32_t D>
__global__ __launch_bounds__(kJoinThreads) void k_join_few(AttentionArgs a) {
    const uint32_t kv_head = blockIdx.x % a.cache.kv_heads, unit = blockIdx.x / a.cache.kv_heads;
    const uint32_t row = blockIdx.y * 4 + uniform(threadIdx.x / 64);
    const u32x4 cut = cuts(a)[unit];
    const uint32_t more = uniform(cut[0]), begin = uniform(cut[1]), rows = uniform(cut[2]);
    if (more == 0 || row >= rows) return;
    const uint32_t i = row / a.group;
    join_row<D>(a, begin + i, kv_head * a.group + (row - i * a.group), more + 1, [&](uint32_t z) {
        return place_of(a, unit + z, kv_head, z == 0 ? 1 : 0) * kFewRows + row;
    });
}

// The splits of the tiles' rows, 4 rows a workgroup.
template <uint32_t D>
__global__ __launch_bounds__(kJoinThreads) void k_join_tiles(AttentionArgs a) {
    const uint32_t heads = a.group * a.cache.kv_heads;
    const uint64_t row = static_cast<uint64_t>(blockIdx.x) * 4 + uniform(threadIdx.x / 64);
    if (row >= static_cast<uint64_t>(a.batch.total_tokens) * heads) return;
    const uint32_t token = uniform(static_cast<uint32_t>(row / heads)), head = uniform(static_cast<uint32_t>(row % heads));
    Tile t{};
    t.seq = span_of(a.batch, wave_seq_of_token(a.batch, token));
    if (static_cast<int32_t>(token) < t.seq.begin || static_cast<int32_t>(token) >= t.seq.begin + t.seq.n) return;
    // the tile that had the row
    t.row0 = ((token - t.seq.begin) * a.group + head % a.group) / a.plan.tile * a.plan.tile;
    const uint32_t rows = static_cast<uint32_t>(t.seq.n) * a.group - t.row0;
    t.rows = rows < a.plan.tile ? rows : a.plan.tile;
    tile_range(t, a.mask, a.group);
    const uint32_t splits = uniform(splits_of(t, a.plan.split_len));
    if (splits <= 1) return;   // written by its workgroup
    join_row<D>(a, token, head, splits, [&](uint32_t z) { return row * a.plan.splits + z; });
}

template <uint32_t D, bool kE5M2>
hipError_t attend(const AttentionArgs& a, hipStream_t s) {
    if (a.plan.tile == kFewRows) {
        const uint32_t units = a.plan.units ? a.plan.units : a.batch.num_seqs;
        const uint32_t groups = static_cast<uint32_t>(few_groups(units, a.cache.kv_heads / a.plan.heads));
        // A sequence a workgroup: twice the waves where the GPU is not full and LDS has room for their blocks (one
        // token over 777 keys: 13.3 us in a graph, 15.5 with 4; 256 sequences of up to 1000: 121, 111).
        constexpr uint32_t kShort = D <= 128 ? 8 : 4;
        if (!a.plan.units && a.batch.num_seqs * a.cache.kv_heads <= 256)
            k_attend_few<D, kE5M2, kShort, 1><<<groups, 64 * kShort, 0, s>>>(a);
        else if (!a.plan.units) k_attend_few<D, kE5M2, 4, 1><<<groups, 256, 0, s>>>(a);
        else if (a.plan.heads == 2) k_attend_few<D, kE5M2, 4, 2><<<groups, 256, 0, s>>>(a);
        else k_attend_few<D, kE5M2, 4, 1><<<groups, 256, 0, s>>>(a);
        if (a.plan.units)
            k_join_few<D><<<dim3(a.plan.units * a.cache.kv_heads, (a.batch.max_tokens * a.group + 3) / 4), kJoinThreads, 0, s>>>(a);
    } else {
        const dim3 grid(static_cast<uint32_t>(tile_slots(a.batch, a.group, a.plan.tile)) * a.cache.kv_heads, a.plan.splits);
        if constexpr (D <= 128) {
            if (a.plan.tile == 256) k_attend_tile<D, kE5M2, 64, 8><<<grid, 512, 0, s>>>(a);
            else k_attend_tile<D, kE5M2, 64, 4><<<grid, 256, 0, s>>>(a);
        } else {
            k_attend_tile<D, kE5M2, 32, 4><<<grid, 256, 0, s>>>(a);
        }
        const uint64_t rows = static_cast<uint64_t>(a.batch.total_tokens) * a.group * a.cache.kv_heads;
        if (a.plan.splits > 1) k_join_tiles<D><<<static_cast<uint32_t>((rows + 3) / 4), kJoinThreads, 0, s>>>(a);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attention(const AttentionArgs& a, hipStream_t s) {
    switch (a.cache.head_dim) {
        case 64: return a.e5m2 ? attend<64, true>(a, s) : attend<64, false>(a, s);
        case 80: return a.e5m2 ? attend<80, true>(a, s) : attend<80, false>(a, s);
        case 96: return a.e5m2 ? attend<96, true>(a, s) : attend<96, false>(a, s);
        case 128: return a.e5m2 ? attend<128, true>(a, s) : attend<128, false>(a, s);
        default: return a.e5m2 ? attend<256, true>(a, s) : attend<256, false>(a, s);
    }
}

}  // namespace kvi
