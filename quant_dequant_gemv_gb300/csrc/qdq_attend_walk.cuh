// qdq_attend_walk.cuh -- where a CTA's share of the attention's work begins, and the walk over
// its pieces (the work's division is qdq_attend_plan.h). A kernel's arguments `a` have the batch
// (n_seqs, n_tokens, max_pages, q_start, kv_len, page_table) and the geometry g.
#pragma once
#include "qdq_attend_plan.h"
#include "qdq_paged.cuh"

namespace qdq {

struct Start {
    long long total, item, pos, end;  // units: of all items, where the first one begins, the CTA's range
    int seq, block, head, ctas, live;
    int first, count, kv;  // of the sequence: its first row, its rows, its positions
};

// A walk over the pieces of a CTA's range, by the copying warp.
struct Walk {
    long long item, pos, end;  // units: where the item begins, the rest of the range
    int seq, block, head, off, n;  // the piece: n key tiles from the item's off-th on
    int first, count, kv, blocks;
    const int32_t *pages;  // the sequence's page table
    AttendBlock b;
    template <typename A>
    QDQ_DEV void load_seq(const A &a) {
        seq_tokens(a.q_start, seq, a.n_tokens, first, count);
        kv = max(a.kv_len[seq], 0);
        blocks = seq_blocks(a.g, count);
        pages = a.page_table + (int64_t)seq * a.max_pages;
    }
    template <typename A>
    QDQ_DEV Walk(const A &a, const Start &s)
        : item(s.item), pos(s.pos), end(s.end), seq(s.seq), block(s.block), head(s.head), first(s.first), count(s.count), kv(s.kv) {
        blocks = seq_blocks(a.g, count);
        pages = a.page_table + (int64_t)seq * a.max_pages;
        b = block_of(a.g, count, kv, block);
        int last;
        piece_of(b, item, pos, end, off, last, a.g.item);
        n = last - off;
        if (n == 0) next(a);  // (the range begins past the item's tiles or ends before them)
    }
    QDQ_DEV bool more() const { return n > 0; }
    QDQ_DEV int t_beg() const { return b.t0 + off; }
    QDQ_DEV bool whole() const { return n == b.t1 - b.t0; }
    template <typename A>
    QDQ_DEV void next(const A &a) {
        item += item_units(b, a.g.item);
        pos = item;
        n = 0;
        if (item >= end) return;
        if (++head == a.g.kv_heads) {
            head = 0;
            if (++block >= blocks) {
                block = 0;
                do {
                    if (++seq >= a.n_seqs) return;  // (only if the batch changed under the kernel)
                    load_seq(a);
                } while (count == 0);
            }
            b = block_of(a.g, count, kv, block);
        }
        int last;
        piece_of(b, item, pos, end, off, last, a.g.item);
        n = last - off;  // 0 at the end of the range, where only the item's first units are left
    }
};

// Where the CTA's range starts: sums of key tiles per sequence, a scan, and a search.
// `room`: 20 * kMaxSeqs bytes of shared memory; every one of the CTA's kThreads threads comes here.
template <int kThreads, typename A>
QDQ_DEV void find_start(const A &a, char *room, Start *start) {
    int *cnt = reinterpret_cast<int *>(room), *kvs = cnt + kMaxSeqs;
    long long *pre = reinterpret_cast<long long *>(room + 8 * kMaxSeqs);  // [n_seqs]
    int *rows = reinterpret_cast<int *>(room + 16 * kMaxSeqs);
    constexpr int kAlone = 8;  // blocks that one thread sums; longer sequences are summed by a warp
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    bool longer = false;
    for (int s = tid; s < a.n_seqs; s += kThreads) {
        int first, count;
        seq_tokens(a.q_start, s, a.n_tokens, first, count);
        const int kv = max(a.kv_len[s], 0), nb = seq_blocks(a.g, count);
        cnt[s] = count;
        rows[s] = first;
        kvs[s] = kv;
        int sum = 0;
        if (nb <= kAlone) {
            for (int b = 0; b < nb; ++b) sum += item_units(block_of(a.g, count, kv, b), a.g.item);
        } else {
            longer = true;
        }
        pre[s] = (long long)sum * a.g.kv_heads;
    }
    if (__syncthreads_or(longer)) {
        for (int s = warp; s < a.n_seqs; s += kThreads / 32) {
            const int nb = seq_blocks(a.g, cnt[s]);
            if (nb <= kAlone) continue;
            long long sum = 0;
            for (int b = lane; b < nb; b += 32) sum += item_units(block_of(a.g, cnt[s], kvs[s], b), a.g.item);
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
            if (lane == 0) pre[s] = sum * a.g.kv_heads;
        }
        __syncthreads();
    }
    if (warp == 0) {
        // a scan over lanes, each with a contiguous run of sequences
        const int per = (a.n_seqs + 31) / 32, s0 = min(lane * per, a.n_seqs), s1 = min(s0 + per, a.n_seqs);
        long long mine = 0;
        for (int s = s0; s < s1; ++s) mine += pre[s];
        long long incl = mine;
        for (int o = 1; o < 32; o <<= 1) {
            const long long e = __shfl_up_sync(0xFFFFFFFFu, incl, o);
            if (lane >= o) incl += e;
        }
        const long long total = __shfl_sync(0xFFFFFFFFu, incl, 31);
        const int ctas = (int)min((long long)gridDim.x, total);
        const bool live = (int)blockIdx.x < ctas;
        const long long x = live ? range_start(total, ctas, blockIdx.x) : 0;
        const long long excl = incl - mine;
        if (lane == 0) {
            start->live = live;
            start->ctas = ctas;
            start->total = total;
            start->pos = x;
            start->end = live ? range_start(total, ctas, blockIdx.x + 1) : 0;
        }
        // the lane whose run of sequences holds x walks it
        const unsigned owner = __ballot_sync(0xFFFFFFFFu, live && mine > 0 && excl <= x && x < incl);
        int s = 0;
        long long rem = 0;
        if (owner && lane == __ffs(owner) - 1) {
            rem = x - excl;
            s = s0;
            while (rem >= pre[s]) rem -= pre[s++];
        }
        if (owner) {
            const int src = __ffs(owner) - 1;
            s = __shfl_sync(0xFFFFFFFFu, s, src);
            rem = __shfl_sync(0xFFFFFFFFu, rem, src);
            // the block: 32 at a time
            const int nb = seq_blocks(a.g, cnt[s]);
            for (int b0 = 0; b0 < nb; b0 += 32) {
                int n = 0;
                if (b0 + lane < nb) n = item_units(block_of(a.g, cnt[s], kvs[s], b0 + lane), a.g.item);
                long long run = (long long)n * a.g.kv_heads;
                const long long own = run;
                for (int o = 1; o < 32; o <<= 1) {
                    const long long e = __shfl_up_sync(0xFFFFFFFFu, run, o);
                    if (lane >= o) run += e;
                }
                const unsigned m = __ballot_sync(0xFFFFFFFFu, rem < run);
                if (m) {
                    const int l = __ffs(m) - 1;
                    if (lane == l) {
                        const int r = (int)(rem - (run - own));
                        start->seq = s;
                        start->first = rows[s], start->count = cnt[s], start->kv = kvs[s];
                        start->block = b0 + l;
                        start->head = r / n;
                        start->item = x - r % n;
                    }
                    break;
                }
                rem -= __shfl_sync(0xFFFFFFFFu, run, 31);
            }
        }
    }
    __syncthreads();
}

}  // namespace qdq
