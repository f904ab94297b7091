// Host-side checks of the paged cache's C ABI (kv_api.cpp) under
// AddressSanitizer, UBSan and the unsigned-overflow check, built by
// tests/test_api_sanitized_paged.py with this file's stub launchers in the
// place of the kernels.  Descriptors take the edges of every field's domain,
// each alone and in random mixtures; nothing may wrap, overflow or read a
// value outside an enum as one, and what reaches a launcher has a grid
// inside the launch limits and a workspace that holds its partial sums.
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "kv_internal.h"
#include "paged_kv.h"

static int g_launches = 0, g_failures = 0;
static uint64_t g_workspace = 0;
#define EXPECT(x)                                              \
    do {                                                       \
        if (!(x)) {                                            \
            printf("failed at %d: %s\n", __LINE__, #x);        \
            ++g_failures;                                      \
        }                                                      \
    } while (0)

namespace kvi {
hipError_t launch_append(AppendArgs a, hipStream_t) {
    ++g_launches;
    EXPECT(a.batch.total_tokens > 0 && a.batch.total_tokens < (1u << 24));
    EXPECT((a.q_heads + 2 * a.cache.kv_heads + 7) / 8 <= 65535);
    return hipSuccess;
}
hipError_t launch_gather(const CopyArgs&, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_scatter(const CopyArgs&, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_attention(const AttentionArgs& a, hipStream_t) {
    ++g_launches;
    const uint64_t rows = uint64_t(a.batch.total_tokens) * a.group * a.cache.kv_heads;
    if (a.plan.tile == kFewRows) {
        EXPECT(few_groups(a.plan.units ? a.plan.units : a.batch.num_seqs, a.cache.kv_heads) < (1u << 24));
        EXPECT(uint64_t(a.batch.max_tokens) * a.group <= kFewRows && a.plan.granule && a.plan.least);
        EXPECT(a.plan.parts == uint64_t(a.plan.units) * a.cache.kv_heads * 2 * kFewRows);
        EXPECT(!a.plan.units || (uint64_t(a.batch.max_kv_len) / a.plan.granule + 1) * a.batch.num_seqs < (1ull << 32) || a.mask.window);
    } else {
        EXPECT(tile_slots(a.batch, a.group, a.plan.tile) * a.cache.kv_heads < (1u << 24));
        EXPECT(a.plan.splits >= 1 && a.plan.splits <= 65535 && a.plan.split_len % 32 == 0);
        EXPECT(uint64_t(a.plan.splits) * a.plan.split_len >= (a.mask.window ? 1 : a.batch.max_kv_len));
        EXPECT(a.plan.parts == (a.plan.splits > 1 ? rows * a.plan.splits : 0));
    }
    if (a.plan.parts) EXPECT(a.part && g_workspace >= a.plan.parts * (a.cache.head_dim + 2) * 4 && rows < (1u << 24));
    return hipSuccess;
}
}  // namespace kvi

int main() {
    uint64_t state = 0x9E3779B97F4A7C15u;
    auto rng = [&] {   // xorshift: no arithmetic that wraps
        state ^= state << 13;
        state ^= state >> 7;
        state ^= state << 17;
        return state;
    };
    uint8_t* fake = reinterpret_cast<uint8_t*>(uintptr_t(0x7F0000000000));
    const uint32_t edges[] = {0, 1, 2, 3, 8, 16, 31, 32, 64, 80, 128, 255, 1024, 4096, 65536, 1u << 20, (1u << 24) - 1,
                              1u << 24, (1u << 30), (1u << 31) - (1u << 17) - 1, (1u << 31) - 1, 1u << 31, 0xFFFFFFFFu};
    auto edge = [&] { return edges[rng() % (sizeof edges / sizeof *edges)]; };
    const uint32_t dims[] = {64, 80, 96, 128, 256};
    for (int i = 0; i < 400000; ++i) {
        kv_cache c{};
        c.d_k = c.d_v = fake;
        c.kv_heads = rng() % 3 ? 1 + rng() % 16 : edge();
        c.head_dim = rng() % 8 ? dims[rng() % 5] : edge();
        c.head_stride = c.head_dim;
        c.token_stride = uint64_t(c.head_dim) * c.kv_heads;
        c.page_size = rng() % 3 ? 1u << rng() % 10 : edge();
        c.page_stride = c.token_stride < (1u << 24) && c.page_size <= 65536 ? c.token_stride * c.page_size : 1u << 30;
        c.num_pages = rng() % 3 ? 100 : edge();
        int dtype = rng() % 8 ? 1 + int(rng() % 2) : int(edge());
        memcpy(&c.dtype, &dtype, sizeof dtype);
        kv_batch b{};
        b.d_pages = b.d_cu_tokens = b.d_kv_lens = reinterpret_cast<int32_t*>(fake);
        b.num_seqs = rng() % 3 ? 1 + rng() % 100 : edge();
        b.total_tokens = rng() % 3 ? 1 + rng() % 5000 : edge();
        b.max_tokens = rng() % 3 ? 1 + rng() % 5000 : edge();
        b.max_kv_len = rng() % 3 ? rng() % 200000 : edge();
        b.pages_per_seq = 1 + rng() % 100;
        b.pages_stride = rng() % 4 ? b.pages_per_seq : edge();
        kv_attention_args a{};
        a.d_q = a.d_out = fake;
        a.q_heads = rng() % 3 ? uint32_t(uint64_t(c.kv_heads) * (1 + rng() % 8) % (1u << 16)) : edge();
        a.q_stride = a.out_stride = uint64_t(a.q_heads) * c.head_dim;
        a.scale = 0.1f;
        a.causal = rng() % 4 ? 1 : 0;
        a.window = rng() % 3 ? 0 : edge();
        g_workspace = kv_attention_workspace_bytes(&c, &b, &a);
        int before = g_launches;
        sz_status st = kv_attention(&c, &b, &a, fake, g_workspace, nullptr, nullptr);
        EXPECT((st == SZ_OK && (g_launches == before + 1 || b.num_seqs == 0 || b.total_tokens == 0)) ||
               (st == SZ_ERR_INVALID_ARGUMENT && g_launches == before && g_workspace == 0));
        if (g_workspace) EXPECT(kv_attention(&c, &b, &a, fake, g_workspace - 1, nullptr, nullptr) == SZ_ERR_BUFFER_TOO_SMALL);
        kv_append_args p{};
        p.d_k = p.d_v = p.d_q = p.d_q_out = fake;
        p.k_stride = p.v_stride = c.token_stride;
        p.q_heads = a.q_heads;
        p.q_stride = p.q_out_stride = a.q_stride;
        p.d_cos_sin = rng() % 2 ? reinterpret_cast<float*>(fake) : nullptr;
        p.rotary_dim = rng() % 2 ? c.head_dim : edge();
        p.max_positions = edge();
        before = g_launches;
        st = kv_append(&c, &b, &p, nullptr, nullptr);
        EXPECT(st == SZ_OK || (st == SZ_ERR_INVALID_ARGUMENT && g_launches == before));
        before = g_launches;
        st = kv_gather(&c, &b, fake, c.token_stride, fake, rng() % 4 ? c.token_stride : edge(), nullptr, nullptr);
        EXPECT(st == SZ_OK || (st == SZ_ERR_INVALID_ARGUMENT && g_launches == before));
        before = g_launches;
        st = kv_scatter(&c, &b, fake, c.token_stride, fake, c.token_stride, nullptr, nullptr);
        EXPECT(st == SZ_OK || (st == SZ_ERR_INVALID_ARGUMENT && g_launches == before));
        if (g_failures > 20) break;
    }
    EXPECT(g_launches > 100000);
    printf("%s\n", g_failures ? "FAILED" : "ok");
    return g_failures != 0;
}
