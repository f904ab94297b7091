// kv_api.cpp -- C ABI entry points of the paged KV cache (declared and
// documented in include/paged_kv.h).  Host-side argument checks, then kernel
// launches on the caller's stream; nothing is allocated, freed or
// synchronised.
#include "paged_kv.h"

#include <cstring>

#include "kv_internal.h"

#define KV_EXPORT extern "C" __attribute__((visibility("default")))

namespace {

using namespace kvi;

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool usable(const void* p) { return p != nullptr && aligned(p, 16); }
sz_status from_hip(hipError_t e) { return e == hipSuccess ? SZ_OK : SZ_ERR_HIP; }

// an enum read from a caller's struct may hold any int: looked at through its bytes
int raw_value(const sz_dtype& e) {
    static_assert(sizeof(sz_dtype) == sizeof(int), "C enums are int-sized");
    int v;
    std::memcpy(&v, &e, sizeof v);
    return v;
}

// Largest stride taken (elements): a pool of 2^31 pages or 2^24 rows of it
// still has its last byte's offset inside 64 bits.
constexpr uint64_t kMaxStride = uint64_t(1) << 31;
// A launch has less than 2^32 threads in x: 2^23 workgroups of 512.
constexpr uint64_t kMaxGroups = uint64_t(1) << 23;

constexpr uint64_t kMaxTokens = uint64_t(1) << 24;

bool head_dim_ok(uint32_t d) { return d == 64 || d == 80 || d == 96 || d == 128 || d == 256; }

bool is_e5m2(const kv_cache& c) { return raw_value(c.dtype) == SZ_DTYPE_FP8_E5M2; }

// A stride over `count` entries that each hold `least` elements, in 16-byte steps of `size`-byte elements
bool stride_ok(uint64_t stride, uint64_t least, uint64_t count, uint32_t size) {
    return stride <= kMaxStride && stride * size % 16 == 0 && (count <= 1 || stride >= least);
}

bool take_cache(const kv_cache* c, Cache& to) {
    if (!c || !usable(c->d_k) || !usable(c->d_v) || c->reserved) return false;
    const int dt = raw_value(c->dtype);
    if (dt != SZ_DTYPE_BF16 && dt != SZ_DTYPE_FP8_E5M2) return false;
    const uint32_t size = dt == SZ_DTYPE_BF16 ? 2 : 1;
    if (c->num_pages == 0 || c->num_pages >= (1u << 31) || c->page_size == 0 || c->page_size > 65536 ||
        (c->page_size & (c->page_size - 1)) || c->kv_heads == 0 || c->kv_heads > 1024 || !head_dim_ok(c->head_dim))
        return false;
    if (!stride_ok(c->page_stride, c->head_dim, c->num_pages, size) ||
        !stride_ok(c->token_stride, c->head_dim, c->page_size, size) ||
        !stride_ok(c->head_stride, c->head_dim, c->kv_heads, size))
        return false;
    to.k = static_cast<uint8_t*>(c->d_k);
    to.v = static_cast<uint8_t*>(c->d_v);
    to.page_stride = c->page_stride * size;
    to.token_stride = c->token_stride * size;
    to.head_stride = c->head_stride * size;
    to.num_pages = c->num_pages;
    to.log2_page = 0;
    while ((1u << to.log2_page) < c->page_size) ++to.log2_page;
    to.kv_heads = c->kv_heads;
    to.head_dim = c->head_dim;
    return true;
}

bool take_batch(const kv_batch* b, Batch& to) {
    if (!b || b->reserved) return false;
    if (b->num_seqs >= (1u << 20) || b->total_tokens >= kMaxTokens || b->max_kv_len >= (1u << 31) - (1u << 17)) return false;
    to.num_seqs = b->num_seqs;
    to.total_tokens = b->total_tokens;
    if (b->num_seqs == 0 || b->total_tokens == 0) return true;   // nothing to do: no table is read
    if (!b->d_pages || !aligned(b->d_pages, 4) || !b->d_cu_tokens || !aligned(b->d_cu_tokens, 4) || !b->d_kv_lens ||
        !aligned(b->d_kv_lens, 4) || b->pages_per_seq == 0 || b->pages_stride < b->pages_per_seq ||
        b->pages_stride > kMaxStride || b->max_tokens == 0)
        return false;
    to.pages = b->d_pages;
    to.cu = b->d_cu_tokens;
    to.kv_lens = b->d_kv_lens;
    to.pages_stride = b->pages_stride;
    to.pages_per_seq = b->pages_per_seq;
    to.max_tokens = b->max_tokens;
    to.max_kv_len = b->max_kv_len;
    return true;
}

bool empty(const Batch& b) { return b.num_seqs == 0 || b.total_tokens == 0; }

// Workgroups of the attention's first launch in x.
uint64_t attention_groups(const AttentionArgs& a) {
    if (a.plan.tile == kFewRows)
        return few_groups(a.plan.units ? a.plan.units : a.batch.num_seqs, a.cache.kv_heads);
    return tile_slots(a.batch, a.group, a.plan.tile) * a.cache.kv_heads;
}

// Everything of kv_attention's arguments but the workspace.
bool take_attention(const kv_cache* cache, const kv_batch* batch, const kv_attention_args* x, AttentionArgs& a) {
    if (!x || !take_cache(cache, a.cache) || !take_batch(batch, a.batch)) return false;
    if (x->q_heads == 0 || x->q_heads % a.cache.kv_heads || x->q_heads / a.cache.kv_heads > 64 || x->causal > 1 ||
        (x->window && !x->causal) || x->window >= (1u << 31) || !(x->scale > 0.f) || !(x->scale <= 3.402823466e38f))
        return false;
    a.group = x->q_heads / a.cache.kv_heads;
    a.e5m2 = is_e5m2(*cache);
    a.mask = Mask{x->causal, x->window};
    if (empty(a.batch)) return true;
    const uint64_t row = static_cast<uint64_t>(x->q_heads) * a.cache.head_dim;
    if (!usable(x->d_q) || !usable(x->d_out) || (x->d_lse && !aligned(x->d_lse, 4)) ||
        !stride_ok(x->q_stride, row, a.batch.total_tokens, 2) || !stride_ok(x->out_stride, row, a.batch.total_tokens, 2) ||
        (x->d_q == x->d_out && x->q_stride != x->out_stride && a.batch.total_tokens > 1))
        return false;
    a.plan = attention_plan(a.cache, a.batch, a.group, x->window, a.e5m2);
    if (attention_groups(a) >= kMaxGroups) return false;
    a.q = static_cast<const uint16_t*>(x->d_q);
    a.out = static_cast<uint16_t*>(x->d_out);
    a.lse = x->d_lse;
    a.q_stride = x->q_stride;
    a.out_stride = x->out_stride;
    a.scale = x->scale;
    return true;
}

bool take_copy(const kv_cache* cache, const kv_batch* batch, void* k, uint64_t k_stride, void* v, uint64_t v_stride,
               int32_t* d_status, CopyArgs& a) {
    if (!take_cache(cache, a.cache) || !take_batch(batch, a.batch) || (d_status && !aligned(d_status, 4))) return false;
    if (empty(a.batch)) return true;
    const uint32_t size = is_e5m2(*cache) ? 1 : 2;
    const uint64_t row = static_cast<uint64_t>(a.cache.kv_heads) * a.cache.head_dim;
    if (!usable(k) || !usable(v) || !stride_ok(k_stride, row, a.batch.total_tokens, size) ||
        !stride_ok(v_stride, row, a.batch.total_tokens, size))
        return false;
    a.k = static_cast<uint8_t*>(k);
    a.v = static_cast<uint8_t*>(v);
    a.k_stride = k_stride * size;
    a.v_stride = v_stride * size;
    a.head_bytes = a.cache.head_dim * size;
    a.status = d_status;
    return true;
}

}  // namespace

KV_EXPORT uint32_t kv_abi_version(void) { return KV_ABI_VERSION; }

KV_EXPORT sz_status kv_append(const kv_cache* cache, const kv_batch* batch, const kv_append_args* x,
                              int32_t* d_status, hipStream_t stream) {
    AppendArgs a{};
    if (!x || x->reserved || !take_cache(cache, a.cache) || !take_batch(batch, a.batch) ||
        (d_status && !aligned(d_status, 4)))
        return SZ_ERR_INVALID_ARGUMENT;
    const uint32_t dim = a.cache.head_dim;
    if (x->d_cos_sin && (!usable(x->d_cos_sin) || x->rotary_dim == 0 || x->rotary_dim % 16 || x->rotary_dim > dim ||
                         x->max_positions == 0 || x->interleaved > 1))
        return SZ_ERR_INVALID_ARGUMENT;
    if ((x->d_q_norm && !usable(x->d_q_norm)) || (x->d_k_norm && !usable(x->d_k_norm))) return SZ_ERR_INVALID_ARGUMENT;
    if ((x->d_q_norm || x->d_k_norm) && (!(x->eps >= 0.f) || !(x->eps <= 3.402823466e38f))) return SZ_ERR_INVALID_ARGUMENT;
    if (x->d_q && (x->q_heads == 0 || x->q_heads > 65536)) return SZ_ERR_INVALID_ARGUMENT;
    if (empty(a.batch)) return SZ_OK;
    const uint64_t row = static_cast<uint64_t>(a.cache.kv_heads) * dim;
    if (!usable(x->d_k) || !usable(x->d_v) || !stride_ok(x->k_stride, row, a.batch.total_tokens, 2) ||
        !stride_ok(x->v_stride, row, a.batch.total_tokens, 2))
        return SZ_ERR_INVALID_ARGUMENT;
    if (x->d_q) {
        const uint64_t q_row = static_cast<uint64_t>(x->q_heads) * dim;
        if (!usable(x->d_q) || !usable(x->d_q_out) || !stride_ok(x->q_stride, q_row, a.batch.total_tokens, 2) ||
            !stride_ok(x->q_out_stride, q_row, a.batch.total_tokens, 2) ||
            (x->d_q == x->d_q_out && x->q_stride != x->q_out_stride && a.batch.total_tokens > 1))
            return SZ_ERR_INVALID_ARGUMENT;
        a.q = static_cast<const uint16_t*>(x->d_q);
        a.q_out = static_cast<uint16_t*>(x->d_q_out);
        a.q_stride = x->q_stride;
        a.q_out_stride = x->q_out_stride;
        a.q_heads = x->q_heads;
        a.q_norm = static_cast<const uint16_t*>(x->d_q_norm);
    }
    a.k = static_cast<const uint16_t*>(x->d_k);
    a.v = static_cast<const uint16_t*>(x->d_v);
    a.k_stride = x->k_stride;
    a.v_stride = x->v_stride;
    a.k_norm = static_cast<const uint16_t*>(x->d_k_norm);
    a.eps = x->eps;
    if (x->d_cos_sin) {
        a.cos_sin = x->d_cos_sin;
        a.rotary_dim = x->rotary_dim;
        a.max_positions = x->max_positions;
        a.interleaved = x->interleaved;
    }
    a.status = d_status;
    a.e5m2 = is_e5m2(*cache);
    return from_hip(launch_append(a, stream));
}

KV_EXPORT uint64_t kv_attention_workspace_bytes(const kv_cache* cache, const kv_batch* batch,
                                                const kv_attention_args* args) {
    AttentionArgs a{};
    if (!take_attention(cache, batch, args, a) || empty(a.batch)) return 0;
    return a.plan.workspace_bytes;
}

KV_EXPORT sz_status kv_attention(const kv_cache* cache, const kv_batch* batch, const kv_attention_args* args,
                                 void* d_workspace, uint64_t workspace_bytes, int32_t* d_status, hipStream_t stream) {
    AttentionArgs a{};
    if (!take_attention(cache, batch, args, a) || (d_status && !aligned(d_status, 4))) return SZ_ERR_INVALID_ARGUMENT;
    if (empty(a.batch)) return SZ_OK;
    const uint64_t need = a.plan.workspace_bytes;
    if (need) {
        if (!usable(d_workspace)) return SZ_ERR_INVALID_ARGUMENT;
        if (workspace_bytes < need) return SZ_ERR_BUFFER_TOO_SMALL;
        a.part = static_cast<float*>(d_workspace);
    }
    a.status = d_status;
    return from_hip(launch_attention(a, stream));
}

KV_EXPORT sz_status kv_gather(const kv_cache* cache, const kv_batch* batch, void* d_k, uint64_t k_stride, void* d_v,
                              uint64_t v_stride, int32_t* d_status, hipStream_t stream) {
    CopyArgs a{};
    if (!take_copy(cache, batch, d_k, k_stride, d_v, v_stride, d_status, a)) return SZ_ERR_INVALID_ARGUMENT;
    return empty(a.batch) ? SZ_OK : from_hip(launch_gather(a, stream));
}

KV_EXPORT sz_status kv_scatter(const kv_cache* cache, const kv_batch* batch, const void* d_k, uint64_t k_stride,
                               const void* d_v, uint64_t v_stride, int32_t* d_status, hipStream_t stream) {
    CopyArgs a{};
    if (!take_copy(cache, batch, const_cast<void*>(d_k), k_stride, const_cast<void*>(d_v), v_stride, d_status, a))
        return SZ_ERR_INVALID_ARGUMENT;
    return empty(a.batch) ? SZ_OK : from_hip(launch_scatter(a, stream));
}

// How a call's rows and keys are cut: a function of the shapes and limits
// that the host knows, so that the same shapes always run the same way.
kvi::AttentionPlan kvi::attention_plan(const Cache& c, const Batch& b, uint32_t group, uint32_t window, bool e5m2) {
    AttentionPlan p{};
    const uint64_t most_rows = static_cast<uint64_t>(b.max_tokens) * group;
    const uint64_t rows = static_cast<uint64_t>(b.total_tokens) * group;
    // 256 rows share a tile of keys where a sequence has many (a prompt of 8192: 1240 us, against 1304 with 128), 128
    // where it has few (100 new of 400, 400 rows: 19 us, 22) and where the registers of a wave fill a SIMD (D = 256).
    p.tile = most_rows <= kFewRows ? kFewRows : most_rows <= 512 || c.head_dim > 128 ? 128 : 256;
    // positions that a tile can see
    uint64_t range = b.max_kv_len;
    if (window && static_cast<uint64_t>(window) + p.tile + 64 < range) range = static_cast<uint64_t>(window) + p.tile + 64;
    if (range == 0) range = 1;
    // Rows are joined by a workgroup each; where there are too many for one launch (padding among them), none is cut.
    const bool joins = rows * c.kv_heads < kMaxGroups;
    if (p.tile == kFewRows) {
        p.heads = 1;
        p.granule = e5m2 ? 256 : 128;   // a block for each of a workgroup's waves
        p.least = 512 / p.granule;
        // As many units as run at once on 256 CUs, in one round, where a sequence is worth cutting and there are few
        // enough of them to need it: each unit looks through all sequences.
        const uint64_t at_once = 256 * few_a_cu(c.head_dim, e5m2);
        const uint64_t most = range / p.granule + 2;
        if (joins && range > 1024 && static_cast<uint64_t>(b.num_seqs) * c.kv_heads < 4096 && b.num_seqs * most < (uint64_t(1) << 32)) {
            // Two heads a workgroup where their rows are neighbours in a token-major page and there are positions
            // enough (64 x 1 to 8192 keys: 209 us, against 220; E5M2: 127, 138; but 8 x 1 to 8192: 41, 37).
            const bool neighbours = c.head_stride < c.token_stride && c.kv_heads % 2 == 0;
            p.heads = neighbours && b.num_seqs * range >= 3 << 16 ? 2 : 1;
            p.units = static_cast<uint32_t>(at_once * p.heads / c.kv_heads / 8 * 8);
            if (p.units == 0) p.units = 8;
            p.parts = static_cast<uint64_t>(p.units) * c.kv_heads * 2 * kFewRows;
        }
    } else {
        uint64_t tiles = rows / p.tile + b.num_seqs;
        const uint64_t each = (most_rows + p.tile - 1) / p.tile;
        if (b.num_seqs * each < tiles) tiles = b.num_seqs * each;
        tiles *= c.kv_heads;
        // Enough workgroups to fill the GPU, each with at least 256 positions.
        const uint64_t kGroups = p.tile == 256 ? 256 : 512, kLeast = 256;
        uint64_t splits = joins && tiles < kGroups ? (kGroups + tiles - 1) / tiles : 1;
        const uint64_t most = (range + kLeast - 1) / kLeast;
        if (splits > most) splits = most;
        uint64_t len = (range + splits - 1) / splits;
        len = (len + 127) / 128 * 128;
        p.split_len = static_cast<uint32_t>(len);
        p.splits = static_cast<uint32_t>((range + len - 1) / len);
        if (p.splits > 1) p.parts = rows * c.kv_heads * p.splits;
    }
    if (p.parts) p.workspace_bytes = sz::align256(p.parts * (c.head_dim + 2) * 4 + p.units * 16);
    return p;
}
