// Host check of the paged attention's work split (csrc/qdq_attend_plan.h): over random
// batches, every (row tile, key tile) that some token attends to is dealt exactly once,
// the CTAs' shares differ by at most one key tile, parts of an item name each other
// consistently, and no page index leaves the table. Prints "ok" or the first fault.
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <vector>

#include "qdq_attend_plan.h"

using namespace qdq;

#define CHECK(c)                                        \
    do {                                                \
        if (!(c)) {                                     \
            std::printf("line %d: %s\n", __LINE__, #c); \
            return 1;                                   \
        }                                               \
    } while (0)

static int one(std::mt19937 &rng) {
    auto pick = [&](int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); };
    AttendGeometry g;
    g.group = pick(1, 32);
    g.tokens = kTileM / g.group;
    g.kv_heads = pick(1, 8);
    g.window = pick(0, 2) ? 0 : pick(1, 700);
    const int page = 16 << pick(0, 4), max_pages = pick(0, 40);
    g.table_end = page * max_pages;
    const int n_seqs = pick(1, 20), ctas_most = pick(1, 152);
    std::vector<int> count(n_seqs), kv(n_seqs);
    for (int s = 0; s < n_seqs; ++s) {
        count[s] = pick(0, 3) ? pick(0, 3) : pick(0, 900);
        kv[s] = pick(0, 5) ? count[s] + pick(0, 1500) : pick(0, 400);
    }
    // the items in order
    struct Item {
        int s, b, h;
        AttendBlock k;
    };
    std::vector<Item> items;
    std::vector<int64_t> at;
    int64_t total = 0;
    for (int s = 0; s < n_seqs; ++s) {
        int covered = 0;
        for (int b = 0; b < seq_blocks(g, count[s]); ++b) {
            const AttendBlock k = block_of(g, count[s], kv[s], b);
            CHECK(k.i0 == covered && k.i1 > k.i0 && k.i1 <= count[s]);
            covered = k.i1;
            CHECK(k.t1 > k.t0 && k.hi <= g.table_end && k.lo >= 0);
            for (int i = k.i0; i < k.i1; ++i) {
                const int p = kv[s] - count[s] + i;
                int lo, hi;
                span(g, p, 1, lo, hi);
                for (int j = lo; j < hi; ++j) CHECK(j <= p && (!g.window || j > p - g.window) && j < g.table_end);
                if (hi <= lo) continue;
                CHECK(lo >= k.lo && hi <= k.hi && k.t0 * kTileN <= lo && k.t1 * kTileN >= hi);
                const int q = (i - k.i0) / g.tokens;
                CHECK(q < 2 && k.tile_t0[q] * kTileN <= lo && k.tile_t1[q] * kTileN >= hi);
                CHECK(k.tile_t0[q] >= k.t0 && k.tile_t1[q] <= k.t1);
            }
            // tiles that neither set uses lie outside both ranges only when nothing is attended to
            if (block_alternates(g, k)) CHECK(k.tile_t0[0] == k.t0 && k.tile_t1[0] == k.t1 && k.tile_t1[1] == 0);
            for (int h = 0; h < g.kv_heads; ++h) {
                items.push_back({s, b, h, k});
                at.push_back(total);
                total += item_units(k);
            }
        }
        CHECK(covered == count[s]);
    }
    if (total == 0) return 0;
    const int ctas = (int)std::min<int64_t>(ctas_most, total);
    std::map<std::pair<int, int>, int> slots;  // (cta, slot) -> item
    std::vector<std::vector<int>> owner(items.size());
    for (size_t i = 0; i < items.size(); ++i) owner[i].assign(items[i].k.t1 - items[i].k.t0, -1);
    for (int c = 0; c < ctas; ++c) {
        const int64_t a = range_start(total, ctas, c), b = range_start(total, ctas, c + 1);
        CHECK(b > a && b - a >= total / ctas && b - a <= total / ctas + 1);
        int cut = 0;
        for (size_t i = 0; i < items.size(); ++i) {
            if (at[i] >= b || at[i] + item_units(items[i].k) <= a) continue;
            int first, last;
            piece_of(items[i].k, at[i], std::max(a, at[i]), b, first, last);
            CHECK(first >= 0 && last >= first && last <= (int)owner[i].size());
            for (int t = first; t < last; ++t) {
                CHECK(owner[i][t] == -1);
                owner[i][t] = c;
                CHECK(range_owner(total, ctas, at[i] + kItemUnits + t) == c);
            }
            const int from = range_owner(total, ctas, at[i] + kItemUnits);
            const int to = range_owner(total, ctas, at[i] + item_units(items[i].k) - 1);
            if (last == first || from == to) continue;
            CHECK(from <= c && c <= to && ++cut <= 2);
            const auto key = std::make_pair(c, c == from ? 1 : 0);
            CHECK(!slots.count(key));
            slots[key] = (int)i;
        }
    }
    CHECK(range_start(total, ctas, 0) == 0 && range_start(total, ctas, ctas) == total);
    // every tile is dealt; every CTA from an item's first to its last holds a part of it, in
    // the slot that the others look in; a counter per first CTA serves one cut item
    std::map<int, int> counters;
    for (size_t i = 0; i < items.size(); ++i) {
        for (int t : owner[i]) CHECK(t >= 0);
        const int from = owner[i].front(), to = owner[i].back();
        if (from == to) continue;
        CHECK(!counters.count(from));
        counters[from] = (int)i;
        for (int c = from; c <= to; ++c) CHECK(slots.at({c, c == from ? 1 : 0}) == (int)i);
    }
    return 0;
}

int main() {
    std::mt19937 rng(7);
    for (int i = 0; i < 3000; ++i)
        if (one(rng)) return 1;
    std::printf("ok\n");
    return 0;
}
