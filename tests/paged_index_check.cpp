// Host check of the paged cache's index arithmetic (kv_internal.h, the
// functions its kernels call), over random and hostile batches:
// - every token of every well-formed sequence is found by its search, and
//   every (token, query head) row lies in exactly one tile, for each tile
//   size, at a slot below tile_slots();
// - a tile's rows, positions and key range are its sequence's, its splits
//   cover its keys once, and the range holds what every row's mask sees;
// - with token ranges and lengths that are anything at all, every read of
//   cu stays in its array (checked by guard values through a copy on the
//   heap of exactly that size, run under AddressSanitizer), and every tile
//   that claims rows claims rows inside [0, total_tokens);
// - the few-rows kernel's granules: dealt to units, each sequence's lie in one
//   run of units, whole or cut; a unit has at most one sequence that began
//   before it and one that begins in it and goes on, so that its two places
//   hold their sums, and the count of units behind the first is what the
//   units' own arithmetic gives;
// - page_of gives -1 for every id outside the pool and index past the table.
// Prints "ok <checks>".
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "kv_internal.h"

using namespace kvi;

static long checks = 0;
#define CHECK(x)                                                  \
    do {                                                          \
        ++checks;                                                 \
        if (!(x)) {                                               \
            std::printf("failed at %d: %s\n", __LINE__, #x);      \
            std::exit(1);                                         \
        }                                                         \
    } while (0)

struct Data {
    std::vector<int32_t> cu, kv, pages;
    Batch b{};
    void bind(uint32_t total, uint32_t most, uint32_t most_kv, uint32_t per_seq) {
        b.cu = cu.data();
        b.kv_lens = kv.data();
        b.pages = pages.data();
        b.num_seqs = static_cast<uint32_t>(kv.size());
        b.total_tokens = total;
        b.max_tokens = most;
        b.max_kv_len = most_kv;
        b.pages_per_seq = per_seq;
        b.pages_stride = per_seq;
    }
};

// The kernels' searches, the wave's 64 lanes one after the other.
template <typename Low>
static uint32_t search(uint32_t n, int64_t target, Low low) {
    const uint32_t s = last_not_above(n, [&](uint32_t from, uint32_t step, uint32_t left) {
        uint64_t bits = 0;
        for (uint64_t i = 0; i < 64; ++i)
            if (i * step < left) {
                CHECK(from + i * step < n);
                if (low(static_cast<uint32_t>(from + i * step)) <= target) bits |= uint64_t(1) << i;
            }
        return bits;
    });
    CHECK(s < n);
    return s;
}
static uint32_t seq_of_token(const Batch& b, uint32_t t) {
    return search(b.num_seqs, t, [&](uint32_t s) -> int64_t { return b.cu[s]; });
}
static Tile tile_of(const Batch& b, const Mask& mask, uint64_t slot, uint32_t group, uint32_t M) {
    const uint32_t s = search(b.num_seqs, static_cast<int64_t>(slot),
                              [&](uint32_t i) { return static_cast<int64_t>(tile_slot(b, i, group, M)); });
    return tile_in(b, mask, s, slot, group, M);
}

int main() {
    std::mt19937 rng(1);
    auto upto = [&](int n) { return static_cast<int>(rng() % static_cast<unsigned>(n + 1)); };
    for (int round = 0; round < 400; ++round) {
        Data d;
        const int seqs = 1 + upto(9);
        std::vector<int> n(seqs);
        int at = upto(1) * upto(3);
        d.cu.push_back(at);
        int most = 1, most_kv = 0;
        for (int s = 0; s < seqs; ++s) {
            n[s] = upto(2) ? upto(40) : upto(300);
            if (!upto(3)) n[s] = 0;
            at += n[s];
            d.cu.push_back(at);
            d.kv.push_back(upto(4) ? n[s] + upto(500) : upto(n[s]));
            most = n[s] > most ? n[s] : most;
            most_kv = d.kv[s] > most_kv ? d.kv[s] : most_kv;
        }
        d.bind(at + upto(5), most, most_kv, 1);
        for (uint32_t t = 0; t < d.b.total_tokens; ++t) {
            const uint32_t s = seq_of_token(d.b, t);
            const bool in = d.cu[s] <= static_cast<int>(t) && static_cast<int>(t) < d.cu[s + 1];
            CHECK(in == (static_cast<int>(t) >= d.cu[0] && static_cast<int>(t) < at));
        }
        for (uint32_t group : {1u, 3u, 4u, 8u, 64u})
            for (uint32_t M : {16u, 32u, 64u, 128u, 256u}) {
                const Mask mask{upto(3) ? 1u : 0u, 0};
                Mask m = mask;
                if (m.causal && upto(1)) m.window = 1 + upto(200);
                std::vector<std::vector<int>> had(seqs);
                for (int s = 0; s < seqs; ++s) had[s].assign(n[s] * group, 0);
                for (uint64_t slot = 0; slot < tile_slots(d.b, group, M); ++slot) {
                    const Tile t = tile_of(d.b, m, slot, group, M);
                    if (!t.any) continue;
                    CHECK(t.rows >= 1 && t.rows <= M && t.row0 % M == 0);
                    for (uint32_t r = 0; r < t.rows; ++r) {
                        ++had[t.s][t.row0 + r];
                        const int32_t p = t.seq.first() + static_cast<int32_t>((t.row0 + r) / group);
                        const int32_t lo = m.first(p), hi = m.last(p, t.seq.kv);
                        CHECK(p >= t.p0 && p <= t.p1);
                        if (hi > lo) CHECK(lo >= t.seen && hi <= t.hi);
                        CHECK(hi <= t.seq.kv);
                    }
                    CHECK(t.lo % 64 == 0 && t.lo <= t.seen && t.lo > t.seen - 64 && t.lo >= 0);
                    const uint32_t len = 128u << upto(3), splits = splits_of(t, len);
                    if (t.hi > t.lo)
                        CHECK(t.lo + static_cast<int64_t>(splits) * len >= t.hi && t.lo + static_cast<int64_t>(splits - 1) * len < t.hi);
                    else CHECK(splits == 0);
                }
                for (auto& rows : had)
                    for (int times : rows) CHECK(times == 1);
            }
    }
    // many sequences, and some of them empty
    for (uint32_t seqs : {1u, 2u, 63u, 64u, 65u, 128u, 129u, 4095u, 4096u, 4097u, 9999u}) {
        Data d;
        d.cu.push_back(0);
        for (uint32_t s = 0; s < seqs; ++s) d.cu.push_back(d.cu.back() + upto(2));
        d.kv.assign(seqs, 3);
        d.bind(d.cu.back() + 3, 2, 3, 1);
        for (uint32_t s = 0; s < seqs; ++s)
            for (int32_t t = d.cu[s]; t < d.cu[s + 1]; ++t) CHECK(seq_of_token(d.b, t) == s);
    }
    // granules and units
    for (int round = 0; round < 3000; ++round) {
        Data d;
        const int seqs = 1 + upto(40);
        d.cu.push_back(0);
        int most = 1, most_kv = 0;
        for (int s = 0; s < seqs; ++s) {
            const int n = upto(3);
            d.cu.push_back(d.cu.back() + n);
            d.kv.push_back(upto(5) ? upto(9000) : upto(2));
            most = n > most ? n : most;
            most_kv = d.kv[s] > most_kv ? d.kv[s] : most_kv;
        }
        d.bind(d.cu.back(), most, most_kv, 1);
        const uint32_t group = 1u << upto(2), granule = 128u << upto(1), least = 1 + upto(5), units = 8u * (1 + upto(8));
        const Mask mask{1, upto(2) ? 0u : 1u + upto(3000)};
        uint32_t total = 0;
        std::vector<uint32_t> before;
        for (int s = 0; s < seqs; ++s) {
            const Tile t = tile_of_seq(d.b, mask, s, group);
            CHECK(t.any == (t.seq.n > 0) && (!t.any || t.rows == t.seq.n * group));
            before.push_back(total);
            total += granules_of(t, granule);
        }
        const uint32_t each = granules_each(total, units, least);
        CHECK(static_cast<uint64_t>(each) * units >= total && each >= least);
        std::vector<int> had(total, 0);
        for (uint32_t unit = 0; unit < units; ++unit) {
            const uint64_t start = static_cast<uint64_t>(unit) * each;
            if (start >= total) continue;
            const uint32_t end = total - start < each ? total : static_cast<uint32_t>(start) + each;
            int places[2] = {0, 0};
            for (int s = 0; s < seqs; ++s) {
                const Tile t = tile_of_seq(d.b, mask, s, group);
                const uint32_t n = granules_of(t, granule);
                if (n == 0 || before[s] >= end || before[s] + n <= start) continue;
                const uint32_t from = before[s] < start ? static_cast<uint32_t>(start) - before[s] : 0;
                const uint32_t to = end - before[s] < n ? end - before[s] : n;
                for (uint32_t g = from; g < to; ++g) ++had[before[s] + g];
                CHECK(t.lo + static_cast<int64_t>(from) * granule <= t.hi);
                if (from == 0 && to == n) continue;
                ++places[before[s] < start ? 0 : 1];
                if (before[s] >= start) {
                    const uint32_t more = (before[s] + n - 1) / (end - static_cast<uint32_t>(start)) - unit;
                    CHECK(more >= 1 && unit + more < units);
                    CHECK(static_cast<uint64_t>(unit + more) * each < before[s] + n &&
                          static_cast<uint64_t>(unit + more + 1) * each >= before[s] + n);
                }
            }
            CHECK(places[0] <= 1 && places[1] <= 1);
        }
        for (int times : had) CHECK(times == 1);
    }
    // anything at all in cu and kv_lens
    for (int round = 0; round < 2000; ++round) {
        Data d;
        const int seqs = 1 + upto(6);
        auto wild = [&]() -> int32_t {
            switch (upto(4)) {
                case 0: return static_cast<int32_t>(rng());
                case 1: return 2147483647 - upto(2);
                case 2: return -upto(2000);
                default: return upto(60);
            }
        };
        for (int s = 0; s <= seqs; ++s) d.cu.push_back(wild());
        for (int s = 0; s < seqs; ++s) d.kv.push_back(wild());
        d.cu.shrink_to_fit();
        d.bind(1 + upto(60), 1 + upto(60), upto(100), 1);
        for (uint32_t t = 0; t < d.b.total_tokens; ++t) CHECK(seq_of_token(d.b, t) < d.b.num_seqs);
        for (uint32_t group : {1u, 8u})
            for (uint64_t slot = 0; slot < tile_slots(d.b, group, 16); ++slot) {
                const Tile t = tile_of(d.b, Mask{1, 0}, slot, group, 16);
                if (!t.any) continue;
                const int64_t last = t.seq.begin + static_cast<int64_t>(t.row0 + t.rows - 1) / group;
                CHECK(t.seq.begin >= 0 && last < static_cast<int64_t>(d.b.total_tokens));
                CHECK(t.hi <= static_cast<int32_t>(d.b.max_kv_len) && t.lo >= 0);
            }
    }
    // pages
    Cache c{};
    c.num_pages = 7;
    c.log2_page = 4;
    c.page_stride = uint64_t(1) << 33;
    c.token_stride = 512;
    Data d;
    d.cu = {0, 1, 2};
    d.kv = {1, 1};
    d.pages = {0, 6, 7, -1, 2147483647, -2147483647 - 1, 3, 5};
    d.bind(2, 1, 100, 4);
    const int32_t want[8] = {0, 6, -1, -1, -1, -1, 3, 5};
    for (uint32_t s = 0; s < 2; ++s)
        for (int32_t p = 0; p < 200; ++p) CHECK(page_of(c, d.b, s, p) == (p / 16 < 4 ? want[4 * s + p / 16] : -1));
    CHECK(page_of(c, d.b, 1, 2147483647) == -1);
    CHECK(slot_offset(c, 6, 16 * 5 + 3) == 6 * c.page_stride + 3 * 512);
    std::printf("ok %ld\n", checks);
    return 0;
}
