// qdq_attend_plan.h -- how the paged attention's work is cut, in plain integer
// arithmetic that the kernel and a host test both compile (qdq_attend.cu).
//
// Rows. The g query heads that share a kv head are rows of the same matrix: a tile of
// kTileM rows holds kTileM / g whole tokens (row = token * g + head), a block two tiles.
// Items. (sequence, block, kv head), in that order; an item's length is the number of
// key tiles (kTileN positions) from the first one that any of its tokens attends to up
// to the last.
// Work. An item is kItemUnits units (its queries, its output), then one for each key
// tile. The items' units, laid end to end, are dealt to the CTAs in equal contiguous
// ranges, so whatever the lengths, every CTA has the same work; a key tile belongs to the
// CTA that holds its unit, and an item whose tiles belong to several is joined from its
// parts. A CTA's range can cut at most the item it starts in and the item it ends in.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define QDQ_PLAN_FN __host__ __device__ __forceinline__
#else
#define QDQ_PLAN_FN inline
#endif

namespace qdq {

constexpr int kTileM = 128, kTileN = 128;
// (8191 prompt tokens, 32 + 8 heads of 128: 486, 410, 402, 405, 435 us at 2, 3, 4, 5, 6 units;
// without it the CTA with the shortest items ran two and a half times as long as the rest.)
constexpr int kItemUnits = 4;

struct AttendGeometry {
    int group;        // query heads per kv head
    int tokens;       // whole tokens of a tile: kTileM / group
    int kv_heads;
    int window;       // 0: none
    int table_end;    // positions that the page table covers
};

// One block of a sequence: its tokens i0..i1-1, the positions lo..hi-1 that some token
// of it attends to, and the key tiles of the whole block and of each of its two tiles.
struct AttendBlock {
    int i0, i1, lo, hi, t0, t1;
    int tile_t0[2], tile_t1[2];
};

QDQ_PLAN_FN int plan_min(int a, int b) { return a < b ? a : b; }
QDQ_PLAN_FN int plan_max(int a, int b) { return a > b ? a : b; }
QDQ_PLAN_FN int seq_blocks(const AttendGeometry &g, int count) {
    const int b = 2 * g.tokens;
    return count <= b ? (count > 0 ? 1 : 0) : (count + b - 1) / b;
}

// Positions first..last-1 of tokens i0..i1-1, the first of which is at position p0.
QDQ_PLAN_FN void span(const AttendGeometry &g, int p0, int n, int &lo, int &hi) {
    lo = g.window ? plan_max(p0 - g.window + 1, 0) : 0;
    hi = plan_max(plan_min(p0 + n, g.table_end), 0);
}

// Block b of a sequence with `count` new tokens and kv positions in all.
QDQ_PLAN_FN AttendBlock block_of(const AttendGeometry &g, int count, int kv, int b) {
    const int tq = g.tokens, base = kv - count;
    AttendBlock r;
    r.i0 = b * 2 * tq;
    r.i1 = plan_min(r.i0 + 2 * tq, count);
    span(g, base + r.i0, r.i1 - r.i0, r.lo, r.hi);
    r.t0 = r.lo / kTileN;
    r.t1 = plan_max((r.hi + kTileN - 1) / kTileN, r.t0 + 1);  // a block with nothing to attend to is one empty tile
    for (int i = 0; i < 2; ++i) {
        const int a = r.i0 + i * tq, n = plan_min(tq, r.i1 - a);
        int lo, hi;
        r.tile_t0[i] = r.tile_t1[i] = 0;
        if (n <= 0) continue;
        span(g, base + a, n, lo, hi);
        if (hi <= lo) continue;
        r.tile_t0[i] = lo / kTileN;
        r.tile_t1[i] = (hi + kTileN - 1) / kTileN;
    }
    return r;
}

// Item of one tile of rows that attends to anything: its two softmax groups take alternate
// key tiles of the same rows (the first group has the only one of a single tile).
QDQ_PLAN_FN bool block_alternates(const AttendGeometry &g, const AttendBlock &b) {
    return b.i1 - b.i0 <= g.tokens && b.hi > b.lo;
}

// CTA c of n takes units range_start(c) .. range_start(c + 1) - 1 of `total`.
// (Small totals divide in 32 bits: a 64-bit division is some 500 clocks of a kernel's start.)
QDQ_PLAN_FN int64_t range_start(int64_t total, int n, int c) {
    return total < (1 << 22) && n < 512 ? (int64_t)((uint32_t)total * (uint32_t)c / (uint32_t)n) : total * c / n;
}
QDQ_PLAN_FN int range_owner(int64_t total, int n, int64_t x) {
    return total < (1 << 22) && n < 512 ? (int)((((uint32_t)x + 1) * (uint32_t)n - 1) / (uint32_t)total)
                                        : (int)(((x + 1) * n - 1) / total);
}
QDQ_PLAN_FN int item_units(const AttendBlock &b) { return kItemUnits + b.t1 - b.t0; }
// Of an item whose units begin at `item`, the key tiles [first, last) of the range [x, end).
QDQ_PLAN_FN void piece_of(const AttendBlock &b, int64_t item, int64_t x, int64_t end, int &first, int &last) {
    const int64_t tile0 = item + kItemUnits, n = b.t1 - b.t0;
    const int64_t f = x > tile0 ? x - tile0 : 0, l = end - tile0 < n ? end - tile0 : n;
    first = (int)f;
    last = l > f ? (int)l : (int)f;
}

}  // namespace qdq
