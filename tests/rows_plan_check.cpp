// Host check of the work split (csrc/qdq_attend_plan.h) as the kernel of few rows uses it: blocks of a few
// whole tokens, or one token's list of pages. Over random batches every tile of every block is dealt
// exactly once, at any own cost of an item, no place lies past a list or a table, and parts name each
// other consistently. Prints "ok" or the first fault.
#include <cstdio>
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
    const int mode = g.group > 16 ? 2 : g.group > 8 ? pick(1, 2) : pick(0, 2);
    g.page_shift = pick(4, 8);
    g.list = pick(0, 1) ? pick(1, 60) : 0;
    g.tokens = g.block = g.list ? 1 : (8 << mode) / g.group;
    g.kv_heads = pick(1, 8);
    g.window = g.list || pick(0, 2) ? 0 : pick(1, 700);
    g.item = pick(1, 8);
    const int page = 1 << g.page_shift, max_pages = pick(0, 40), ctas_most = pick(1, 152), n_seqs = pick(1, 20);
    g.table_end = page * max_pages;
    struct Item {
        int tiles;
        std::vector<int> dealt, parts;
    };
    std::vector<Item> items;
    std::vector<int64_t> at;
    int64_t total = 0;
    for (int s = 0; s < n_seqs; ++s) {
        const int count = pick(0, 3) ? pick(0, 3) : pick(0, 300), kv = pick(0, 5) ? count + pick(0, 1500) : pick(0, 400);
        int covered = 0;
        for (int b = 0; b < seq_blocks(g, count); ++b) {
            const AttendBlock k = block_of(g, count, kv, b);
            CHECK(k.i0 == covered && k.i1 > k.i0 && k.i1 <= count && (k.i1 - k.i0) * g.group <= 8 << mode);
            covered = k.i1;
            CHECK(k.t1 > k.t0 && k.lo >= 0 && k.t0 * kTileN <= k.lo && k.t1 * kTileN >= k.hi);
            if (g.list) {
                const int p = kv - count + k.i0, held = plan_max(plan_min(p + 1, g.table_end), 0);
                CHECK(k.lo == 0 && k.hi <= g.list * page && k.hi % page == 0);
                CHECK(k.hi == plan_min(g.list, (held + page - 1) / page) * page);
            } else {
                CHECK(k.hi <= g.table_end);
            }
            for (int h = 0; h < g.kv_heads; ++h) {
                at.push_back(total);
                items.push_back({k.t1 - k.t0, std::vector<int>(k.t1 - k.t0, 0), {}});
                total += item_units(k, g.item);
            }
        }
        CHECK(covered == count);
    }
    if (!total) return 0;
    const int n = (int)(total < ctas_most ? total : ctas_most);
    size_t i = 0;
    for (int c = 0; c < n; ++c) {
        int64_t x = range_start(total, n, c);
        const int64_t end = range_start(total, n, c + 1);
        while (i + 1 < items.size() && at[i + 1] <= x) ++i;
        for (size_t j = i; j < items.size() && at[j] < end; ++j) {
            AttendBlock b = {};
            b.t1 = items[j].tiles;
            int first, last;
            piece_of(b, at[j], x > at[j] ? x : at[j], end, first, last, g.item);
            CHECK(first >= 0 && last <= items[j].tiles);
            for (int t = first; t < last; ++t) ++items[j].dealt[t];
            if (last > first) items[j].parts.push_back(c);
        }
    }
    for (size_t j = 0; j < items.size(); ++j) {
        for (int d : items[j].dealt) CHECK(d == 1);
        CHECK(!items[j].parts.empty());
        CHECK(items[j].parts.front() == range_owner(total, n, at[j] + g.item));
        CHECK(items[j].parts.back() == range_owner(total, n, at[j] + g.item + items[j].tiles - 1));
        CHECK((int)items[j].parts.size() == items[j].parts.back() - items[j].parts.front() + 1);
    }
    return 0;
}

int main() {
    std::mt19937 rng(1);
    for (int i = 0; i < 3000; ++i)
        if (one(rng)) return 1;
    std::puts("ok");
    return 0;
}
