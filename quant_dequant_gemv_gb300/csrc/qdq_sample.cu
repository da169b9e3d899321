// qdq_sample.cu -- sampling: temperature, top-k, top-p and min-p from given random
// numbers.
//
// One pass over the logits: a cluster of up to eight CTAs holds a row in shared memory, a
// contiguous slice each, and everything after the load works on those.
//
// The filters are cuts of one order (logit descending, index ascending), so nothing is
// sorted. A cut is found by narrowing: 512 bins over an interval of the logits' order-
// preserving 32-bit keys, a scan, and the bin that reaches the wanted count or mass
// becomes the next interval until it is one key. The first bins are linear in the
// exponent (1/16 wide) instead of the key; the last of them is open, and its entries
// weigh less than half a unit each. The entries that share the cut's key are told apart
// by narrowing over their indices, and so is the draw itself (an inverse CDF in index
// order).
//
// Most cuts lie near the top. A bin that certainly holds top-k's is found from the largest
// entry of each thread alone (the k-th largest of those is not above the k-th of all), top-
// p's from the bins' masses. If the bins down to that one have at most kList entries, those
// are gathered in the first CTA, which finishes alone while the others leave (with up to
// kFew entries by comparing all pairs). Otherwise only the cut's own bin is gathered and
// narrowed there, and the whole cluster draws; a bin with more than kList entries (ties,
// as a rule) is narrowed by the whole cluster.
//
// Masses are integers (weights in units of 2^-44 of the largest), so neither the order of
// the additions nor the split over CTAs changes a sum. In the bins they are kept as three
// 15-bit pieces, each added with a native 32-bit shared-memory atomic (at most 2^15
// entries a CTA, so a piece cannot overflow).
//
// Bound by latency, not by the read: a row is some 15 dependent steps, of which a list takes
// five. Measured (GB300, 1 x 32000 / 64 x 32000 / 256 x 131071 logits, filters mixed):
// 10.0 / 26 / 171 us (158 to 179 between runs); a listed row of 32000 takes 15 000 clocks from its first load, one
// whose nucleus is a large part of the vocabulary 43 000, of which the pass that bins the
// masses (three shared-memory atomics an entry) and the draw's pass take 7000 and 6000.
//
// CTAs of a cluster send sums to each other before a cluster barrier and read each
// other's bins after one; two sets of buffers take turns, so a step needs one barrier.
// Another CTA's shared memory may be touched only once that CTA is known to run: every CTA
// arrives at a first barrier as it starts and waits there before it sends anything, with
// the load of its slice in between.
#include <cmath>
#include <mutex>

#include "qdq_internal.h"
#include "qdq_paged.cuh"

namespace qdq {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32, kBins = kThreads, kMaxCluster = 8;
constexpr int kSlice = 1 << 15;  // entries of a row that a CTA holds at most
constexpr int kList = 2048, kFew = kThreads / 4;
constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr uint32_t kLowest = 0x00800000u;  // the key of the lowest finite logit (-inf is one below)
typedef unsigned long long u64;

#ifdef QDQ_DEBUG
__device__ int g_sample_status;
#endif

struct SampleArgs {
    const void *logits;
    int64_t stride;
    int rows, vocab, slice;
    const float *temperature, *top_p, *min_p, *u;
    const int32_t *top_k;
    int64_t *tokens;
    float *logprobs;
};

QDQ_DEV uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x);
    return b ^ (b & 0x80000000u ? 0xFFFFFFFFu : 0x80000000u);
}
QDQ_DEV float value_of(uint32_t k) { return __uint_as_float(k ^ (k & 0x80000000u ? 0x80000000u : 0xFFFFFFFFu)); }

struct Shared {
    unsigned bins[2][3][kBins];   // three pieces of mass, or a count in the first
    u64 sums[2][kMaxCluster][2];  // what the cluster's CTAs sent
    u64 warp[kWarps + 1][2];
    u64 found[2];                 // the bin a cut lies in, and the measure above it
    uint32_t edge[2];
    u64 cut[3];                   // the first CTA's word on a cut: key, measure above it, measure at it
    u64 list[kList];              // key << 32 | ~index: in the order of the cuts
    __align__(16) float x[4];     // the slice (slice entries)
};

QDQ_DEV void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The two halves of a barrier that says only that every CTA of the cluster has started.
QDQ_DEV void cluster_started_arrive() { asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory"); }
QDQ_DEV void cluster_started_wait() { asm volatile("barrier.cluster.wait;" ::: "memory"); }
QDQ_DEV uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
QDQ_DEV uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
QDQ_DEV uint32_t remote(const void *p, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
QDQ_DEV void store_remote(uint32_t at, u64 v) { asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(v) : "memory"); }
template <typename V>
QDQ_DEV V warp_sum(V v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

// One CTA's part in the work on one row. ALONE: the first CTA on the gathered list;
// otherwise every CTA of the cluster on its slice, each with the same results.
struct Row {
    Shared &sh;
    const int tid, lane, warp;
    const uint32_t rank, ctas;
    int n = 0, i_first = 0;  // the slice
    int turn_s = 0, turn_b = 0;
    float top = 0.0f, inv = 1.0f;

    QDQ_DEV Row(Shared &s, uint32_t r, uint32_t c)
        : sh(s), tid(threadIdx.x), lane(threadIdx.x & 31), warp(threadIdx.x >> 5), rank(r), ctas(c) {}

    QDQ_DEV float weight(float x) const { return x == top ? 1.0f : expf((x - top) * inv); }  // (-inf weighs 0)
    // A weight in units of 2^-44, as three pieces of 15 bits (the highest may be 2^14): adding
    // 2^23 and rounding down leaves the whole part in the low mantissa bits.
    static QDQ_DEV unsigned whole(float &v) {
        const float t = __fadd_rz(v, 8388608.0f);
        v -= t - 8388608.0f;
        return __float_as_uint(t) & 0x7FFFFFu;
    }
    static QDQ_DEV void pieces(float w, unsigned (&p)[3]) {
        float v = w * 16384.0f;
        p[2] = whole(v);
        v *= 32768.0f;
        p[1] = whole(v);
        v = v * 32768.0f + 0.5f;
        p[0] = whole(v);  // (2^15 where the half carries)
    }
    static QDQ_DEV u64 fixed(float w) {
        unsigned p[3];
        pieces(w, p);
        return ((u64)p[2] << 30) + ((u64)p[1] << 15) + p[0];
    }
    // The first level's bin: 1/16 of the exponent wide, falling logits, the last one open.
    QDQ_DEV int bin_of(float x) const {
        const float v = (top - x) * inv * 16.0f;
        if (!(v < (float)(kBins - 1))) return x == top ? 0 : kBins - 1;  // (inf - inf, 0 x inf)
        return (int)(__float_as_uint(__fadd_rz(v, 8388608.0f)) & (kBins - 1));
    }

    template <bool ALONE>
    QDQ_DEV void sync() {
        if (ALONE) __syncthreads();
        else cluster_sync();
    }
    // f(logit, index) over this CTA's entries (and over the -inf that fill the slice up).
    template <bool ALONE, typename F>
    QDQ_DEV void each(F f) {
        if (ALONE) {
            for (int i = tid; i < n; i += kThreads) f(value_of((uint32_t)(sh.list[i] >> 32)), ~(uint32_t)sh.list[i]);
        } else {
            for (int i = 4 * tid; i < n; i += 4 * kThreads) {
                const float4 x = *reinterpret_cast<const float4 *>(sh.x + i);
                f(x.x, (uint32_t)(i_first + i));
                f(x.y, (uint32_t)(i_first + i + 1));
                f(x.z, (uint32_t)(i_first + i + 2));
                f(x.w, (uint32_t)(i_first + i + 3));
            }
        }
    }

    // The warps' values (maximum or sum of the first, sum of the second) to the CTAs below
    // `to`; part(r, i) is CTA r's after the barrier that the caller passes next.
    template <bool MAX>
    QDQ_DEV void send(u64 a, u64 b, uint32_t to) {
        if (lane == 0) sh.warp[warp][0] = a, sh.warp[warp][1] = b;
        __syncthreads();
        if (warp == 0) {
            u64 x = lane < kWarps ? sh.warp[lane][0] : 0, y = lane < kWarps ? sh.warp[lane][1] : 0;
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) {
                const u64 e = __shfl_xor_sync(kAll, x, o);
                x = MAX ? (e > x ? e : x) : x + e;
                y += __shfl_xor_sync(kAll, y, o);
            }
            if (lane < (int)to) {  // (lanes 0..15 hold the result)
                const uint32_t at = remote(&sh.sums[turn_s][rank][0], lane);
                store_remote(at, x);
                store_remote(at + 8, y);
            }
        }
        turn_s ^= 1;
    }
    QDQ_DEV u64 part(uint32_t r, int i) const { return sh.sums[turn_s ^ 1][r][i]; }

    QDQ_DEV void count(int piece, int b, unsigned v) {
        if (QDQ_CHECK(&g_sample_status, b >= 0 && b < kBins)) atomicAdd(&sh.bins[turn_b][piece][b], v);
    }
    QDQ_DEV void clear_bins(int pieces) {
        for (int i = 0; i < pieces; ++i) sh.bins[turn_b][i][tid] = 0;
        __syncthreads();
    }
    QDQ_DEV void add_mass(int b, float w) {
        unsigned p[3];
        pieces(w, p);
        for (int i = 0; i < 3; ++i) count(i, b, p[i]);
    }
    // Bin `tid` over the whole cluster (each CTA reads all the others'): PIECES of mass, or a
    // count with PIECES = 1. Ends the turn.
    template <bool ALONE, int PIECES>
    QDQ_DEV u64 gather_bins() {
        sync<ALONE>();
        u64 v = 0;
        if (ALONE) {
#pragma unroll
            for (int i = 0; i < PIECES; ++i) v += (u64)sh.bins[turn_b][i][tid] << (15 * i);
        } else {
#pragma unroll 4
            for (uint32_t r = 0; r < ctas; ++r) {
                unsigned x[PIECES];
#pragma unroll
                for (int i = 0; i < PIECES; ++i)
                    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x[i]) : "r"(remote(&sh.bins[turn_b][i][tid], r)));
#pragma unroll
                for (int i = 0; i < PIECES; ++i) v += (u64)x[i] << (15 * i);
            }
        }
        turn_b ^= 1;
        return v;
    }
    // Sum over the bins before this thread's; *all: over every bin.
    template <typename V>
    QDQ_DEV V before(V v, V *all) {
        V incl = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const V e = __shfl_up_sync(kAll, incl, o);
            if (lane >= o) incl += e;
        }
        V *w = reinterpret_cast<V *>(&sh.warp[0][0]);
        __syncthreads();
        if (lane == 31) w[warp] = incl;
        __syncthreads();
        V t = lane < kWarps ? w[lane] : 0, ti = t;
#pragma unroll
        for (int o = 1; o < kWarps; o <<= 1) {
            const V e = __shfl_up_sync(kAll, ti, o);
            if (lane >= o) ti += e;
        }
        *all = __shfl_sync(kAll, ti, kWarps - 1);
        return __shfl_sync(kAll, ti - t, warp) + incl - v;
    }
    // The first bin whose sum (v in this thread's, excl before it) reaches the target: one
    // thread's. found[] is set for every thread after the barrier.
    QDQ_DEV void find(u64 v, u64 excl, u64 target) {
        if (excl < target && excl + v >= target) sh.found[0] = tid, sh.found[1] = excl;
        __syncthreads();
    }

    // The keys whose first-level bin is b: [lo, hi]. Two warps look for the smallest key
    // whose bin is at most b, and at most b - 1: among the 32 keys around where it should
    // be, then, if rounding put it elsewhere, 32 probes at a time from the whole range.
    QDQ_DEV void keys_of(int b, uint32_t &lo, uint32_t &hi) {
        if (warp < 2) {
            const int want = b - warp;
            uint32_t first = kLowest, last = key_of(top);  // the answer is in [first, last] (the top's bin is 0)
            if (want >= kBins - 1) last = first;
            if (want >= 0 && first < last) {
                const uint32_t mid = key_of(top - (float)(want + 1) * 0.0625f / inv);
                const uint32_t at = min(max(mid, first + 16) - 16 + lane, last);
                const unsigned m = __ballot_sync(kAll, bin_of(value_of(at)) <= want);
                if (m && !(m & 1)) first = last = __shfl_sync(kAll, at, __ffs(m) - 1);
            }
            while (first < last && want >= 0) {
                const uint32_t step = (last - first) / 32 + 1;
                const u64 at = (u64)first + (u64)step * lane;
                const unsigned m = __ballot_sync(kAll, at >= last || bin_of(value_of((uint32_t)at)) <= want);
                const int l = __ffs(m) - 1;  // the answer is at most lane l's probe, above lane l - 1's
                if (m == 0) {
                    first = first + step * 31 + 1;
                } else {
                    const u64 e = (u64)first + (u64)step * l;
                    if (l > 0) first = first + step * (l - 1) + 1;
                    last = e < last ? (uint32_t)e : last;
                }
            }
            if (lane == 0) sh.edge[warp] = want < 0 ? key_of(top) + 1 : last;
        }
        __syncthreads();
        lo = sh.edge[0];
        hi = sh.edge[1] - 1;
    }

    // Counts over the index: 128 neighbours share a bin of 128 or more, so a warp adds its sum
    // once (their atomics would all meet at one address).
    template <typename GET>
    QDQ_DEV void bin_neighbours(int shift, GET get) {
        for (int i0 = warp * 128; i0 < n; i0 += 4 * kThreads) {
            const int i = i0 + 4 * lane;  // (the slice is filled up to a multiple of 128)
            const float4 v = *reinterpret_cast<const float4 *>(sh.x + i);
            const float x[4] = {v.x, v.y, v.z, v.w};
            unsigned sum = 0;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                uint32_t k;
                sum += get(x[y], (uint32_t)(i_first + i + y), k);
            }
            sum = __reduce_add_sync(kAll, sum);
            if (lane == 0 && sum) count(0, (i_first + i0) >> shift, sum);
        }
    }

    // The largest key in [lo, hi] at which the measure from hi down (from `ahead` on)
    // reaches the target; `ahead` becomes the measure above it; returns its own. get(key,
    // index, k): whether an entry counts, and under which key. With SHARE the target is the
    // draw's mark in the whole, which the first level finds.
    // INDEX: the keys are inverted indices, and [lo, hi] begins as all of them.
    template <bool ALONE, bool MASS, bool INDEX = false, bool SHARE = false, typename GET>
    QDQ_DEV u64 narrow(uint32_t lo, uint32_t hi, u64 &ahead, u64 target, uint32_t &key, GET get, u64 *whole = nullptr,
                       const SampleArgs *a = nullptr, int row = 0) {
        for (int level = 0; level < 4; ++level) {  // 9 bits a level: 32 bits take four
            // (a level over neighbours has bins of 128 at least)
            const bool neighbours = INDEX && !ALONE && !MASS && level == 0;
            const int shift = max(neighbours ? 7 : 0, 32 - 9 - __clz(hi - lo));
            clear_bins(MASS ? 3 : 1);
            if (neighbours) {
                bin_neighbours(shift, get);
            } else {
                const float x_lo = value_of(lo), x_hi = value_of(hi);
                each<ALONE>([&](float x, uint32_t index) {
                    if (!INDEX && !(x >= x_lo && x <= x_hi)) return;
                    uint32_t k;
                    if (!get(x, index, k) || k < lo || k > hi) return;
                    const int b = (int)((hi - k) >> shift);
                    if (MASS) add_mass(b, weight(x));
                    else count(0, b, 1u);
                });
            }
            const u64 v = gather_bins<ALONE, MASS ? 3 : 1>();
            u64 all;
            const u64 excl = ahead + before(v, &all);
            if (SHARE && level == 0) {
                *whole = all;
                target = mark(*a, row, all);
            }
            find(v, excl, target);
            const uint32_t b = (uint32_t)sh.found[0] & (kBins - 1);
            ahead = sh.found[1];
            const uint32_t last = hi - (b << shift);
            if (shift == 0) {
                if (tid == (int)b) sh.warp[kWarps][0] = v;
                __syncthreads();
                key = last;
                return sh.warp[kWarps][0];
            }
            const uint32_t wide = (1u << shift) - 1;
            lo = last - lo > wide ? last - wide : lo;
            hi = last;
        }
        key = hi;  // not reached
        return 1;
    }

    // Counts of the first level (without the open bin, which gets what the others leave of
    // `total`), and the bin of the top_k-th entry with the count above it.
    template <bool ALONE>
    QDQ_DEV void first_counts(u64 top_k, u64 total, int &bin, u64 &ahead) {
        clear_bins(1);
        each<ALONE>([&](float x, uint32_t) {
            const int k = bin_of(x);
            if (k < kBins - 1) count(0, k, 1u);
        });
        const u64 counted = gather_bins<ALONE, 1>();
        u64 all;
        const u64 excl = before(counted, &all);
        find(tid == kBins - 1 ? total - excl : counted, excl, top_k);
        bin = (int)sh.found[0] & (kBins - 1);
        ahead = sh.found[1];
    }

    // The key of a cut in first-level bin b (narrow(), which see, from `ahead` above the bin, not
    // below `least`): alone, or by the first CTA for all, or by the cluster.
    template <bool ALONE, bool MASS>
    QDQ_DEV u64 resolve(int b, uint32_t least, u64 &ahead, u64 target, uint32_t &key) {
        const auto by_key = [](float x, uint32_t, uint32_t &k) { return k = key_of(x), true; };
        uint32_t lo, hi;
        if (ALONE) {
            keys_of(b, lo, hi);
            return narrow<true, MASS>(max(lo, least), hi, ahead, target, key, by_key);
        }
        u64 own = 0;
        each_bit([&](float x, u64 bit) { own |= bin_of(x) == b && x != -INFINITY ? bit : 0; });
        send<false>(__reduce_add_sync(kAll, __popcll(own)), 0, ctas);
        cluster_sync();
        return resolve_listed<MASS>(b, own, 0, least, ahead, target, key);
    }
    // The same for the cluster, from the threads' entries in the bin and, sent as value i, how
    // many a CTA has.
    template <bool MASS>
    QDQ_DEV u64 resolve_listed(int b, u64 own, int i, uint32_t least, u64 &ahead, u64 target, uint32_t &key) {
        const auto by_key = [](float x, uint32_t, uint32_t &k) { return k = key_of(x), true; };
        uint32_t lo, hi;
        u64 listed;
        if (!gather_list(own, i, listed)) {
            keys_of(b, lo, hi);
            return narrow<false, MASS>(max(lo, least), hi, ahead, target, key, by_key);
        }
        if (rank == 0) {
            const int slice = n, turn = turn_b;  // (the bins' turns are the cluster's)
            n = (int)listed;
            keys_of(b, lo, hi);
            const u64 here = narrow<true, MASS>(max(lo, least), hi, ahead, target, key, by_key);
            n = slice;
            turn_b = turn;
            if (tid < (int)ctas) {
                const uint32_t to = remote(&sh.cut[0], tid);
                store_remote(to, key);
                store_remote(to + 8, ahead);
                store_remote(to + 16, here);
            }
        }
        cluster_sync();
        key = (uint32_t)sh.cut[0];
        ahead = sh.cut[1];
        return sh.cut[2];
    }

    // f(logit, bit) over the slice, for sets of a thread's entries (64 at most).
    template <typename F>
    QDQ_DEV void each_bit(F f) {
        u64 bit = 1;
        for (int i = 4 * tid; i < n; i += 4 * kThreads, bit <<= 4) {
            const float4 x = *reinterpret_cast<const float4 *>(sh.x + i);
            f(x.x, bit);
            f(x.y, bit << 1);
            f(x.z, bit << 2);
            f(x.w, bit << 3);
        }
    }
    // The threads' sets of entries into the first CTA's list; false, and nothing is moved, if
    // they are more than it holds. The CTAs' counts were sent, as value i.
    QDQ_DEV bool gather_list(u64 own, int i, u64 &listed) {
        u64 at = 0;
        listed = 0;
        for (uint32_t c = 0; c < ctas; ++c) {
            if (c == rank) at = listed;
            listed += part(c, i);
        }
        if (listed > kList) return false;
        unsigned all;
        uint32_t to = remote(&sh.list[0], 0) + 8 * ((uint32_t)at + before((unsigned)__popcll(own), &all));
        for (; own; own &= own - 1, to += 8) {
            const int k = __ffsll(own) - 1, e = 4 * tid + (k >> 2) * 4 * kThreads + (k & 3);
            if (QDQ_CHECK(&g_sample_status, to - remote(&sh.list[0], 0) < 8u * kList && e < n))
                store_remote(to, ((u64)key_of(sh.x[e]) << 32) | (uint32_t)~(uint32_t)(i_first + e));
        }
        cluster_sync();
        return true;
    }

    // The cluster's draw: the kept mass of each warp's segment of the slice, of each CTA, and
    // then the warp whose segment holds the mark looks for it. keep(x, index) names the kept.
    template <typename KEEP>
    QDQ_DEV void draw(const SampleArgs &a, int b, float floor_w, KEEP keep) {
        const int seg = (((n + kWarps - 1) / kWarps) + 127) / 128 * 128;
        const int s0 = warp * seg, s1 = min(s0 + seg, n);
        unsigned sum[3] = {};  // (at most 64 entries a thread)
        const auto mass4 = [&](int i, unsigned (&p)[4][3], float (&w)[4]) {
            const float4 v = *reinterpret_cast<const float4 *>(sh.x + i);
            const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                w[y] = keep(x[y], (uint32_t)(i_first + i + y)) ? weight(x[y]) : 0.0f;
                if (!(w[y] >= floor_w)) w[y] = 0.0f;
                pieces(w[y], p[y]);
            }
        };
        for (int i = s0 + 4 * lane; i < s1; i += 128) {
            unsigned p[4][3];
            float w[4];
            mass4(i, p, w);
#pragma unroll
            for (int y = 0; y < 4; ++y)
                for (int z = 0; z < 3; ++z) sum[z] += p[y][z];
        }
        u64 mass = 0;
        for (int z = 0; z < 3; ++z) mass += (u64)__reduce_add_sync(kAll, sum[z]) << (15 * z);
        send<false>(mass, 0, ctas);
        cluster_sync();
        u64 whole = 0, ahead = 0;
        for (uint32_t c = 0; c < ctas; ++c) {
            if (c == rank) ahead = whole;
            whole += part(c, 0);
        }
        const u64 target = mark(a, b, whole);
        for (int w = 0; w < warp; ++w) ahead += sh.warp[w][0];
        if (!(ahead < target && target <= ahead + mass)) return;
        for (int i0 = s0; i0 < s1; i0 += 128) {
            unsigned p[4][3];
            float w[4];
            mass4(i0 + 4 * lane, p, w);
            u64 f[4], own = 0;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                f[y] = ((u64)p[y][2] << 30) + ((u64)p[y][1] << 15) + p[y][0];
                own += f[y];
            }
            u64 incl = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 e = __shfl_up_sync(kAll, incl, o);
                if (lane >= o) incl += e;
            }
            const u64 all = __shfl_sync(kAll, incl, 31);
            if (ahead + all < target) {
                ahead += all;
                continue;
            }
            u64 excl = ahead + incl - own;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                if (excl < target && target <= excl + f[y] &&
                    QDQ_CHECK(&g_sample_status, i_first + i0 + 4 * lane + y < a.vocab && b < a.rows)) {
                    a.tokens[b] = (int64_t)(i_first + i0 + 4 * lane + y);
                    if (a.logprobs) a.logprobs[b] = share_log(w[y], whole);
                }
                excl += f[y];
            }
            return;
        }
    }
    // The mass at which the draw stops: the first unit above u of the whole (at u = 1, the last).
    static QDQ_DEV u64 mark(const SampleArgs &a, int b, u64 whole_mass) {
        return min((u64)(fmin(fmax((double)a.u[b], 0.0), 1.0) * (double)whole_mass) + 1, whole_mass);
    }
    static QDQ_DEV float share_log(float w, u64 whole_mass) {
        return (float)log((double)w / ((double)whole_mass * 0x1p-44));
    }

    // Everything after the first level: the cuts, the ties, the draw. top_k: 0, or with the
    // first-level bin of its cut and the count above that; top_p: below 1 if it is used, and
    // without top-k with its cut's bin, the mass above that and the mass to reach.
    struct First {
        u64 top_k, ahead, target;
        int bin;
    };
    // `own`: with top-p alone, in a cluster, the thread's entries in that bin (sent as value 1).
    template <bool ALONE>
    QDQ_DEV void finish(const SampleArgs &a, int b, First first, float top_p, float floor_w, u64 own = 0) {
        uint32_t cut = kLowest;
        u64 ties = ~0ull, here = 0;  // entries above `cut` are kept, and the first `ties` at it
        if (first.top_k) {
            if (ALONE) first_counts<true>(first.top_k, n, first.bin, first.ahead);
            here = resolve<ALONE, false>(first.bin, kLowest, first.ahead, first.top_k, cut);
            ties = first.top_k - first.ahead;
        }
        if (top_p < 1.0f) {
            if (first.top_k) {
                // exact masses of what top-k left, in the first level's bins. The cut's own bin may
                // hold more ties than top-k kept: the lowest entries, none that the target needs.
                clear_bins(3);
                const float x_cut = value_of(cut);
                each<ALONE>([&](float x, uint32_t) {
                    if (!(x >= x_cut)) return;
                    const int k = bin_of(x);
                    if (k < kBins - 1) add_mass(k, weight(x));
                });
                const u64 v = gather_bins<ALONE, 3>();
                u64 all;
                const u64 excl = before(v, &all);
                const u64 dropped = bin_of(x_cut) < kBins - 1 ? (here - ties) * fixed(weight(x_cut)) : 0;
                first.target = reach(top_p, all - dropped);
                find(v, excl, first.target);
                first.bin = (int)sh.found[0] & (kBins - 1);
                first.ahead = sh.found[1];
            }
            uint32_t key;
            const u64 mass = ALONE || first.top_k
                                 ? resolve<ALONE, true>(first.bin, cut, first.ahead, first.target, key)
                                 : resolve_listed<true>(first.bin, own, 1, cut, first.ahead, first.target, key);
            // the fewest of the entries at the key that reach the target (one alone, mostly)
            const u64 f = fixed(weight(value_of(key)));
            u64 need = 1;
            const u64 most = first.top_k && key == cut ? ties : ~0ull;
            here = 1;
            if (mass != f) {
                need = (first.target - first.ahead + f - 1) / f;
                here = mass / f;
            }
            ties = min(need, most);
            cut = key;
        }
        const float x_cut = value_of(cut);
        // ties: the index of the last one kept (narrowing runs over inverted indices, so that
        // the lowest come first)
        uint32_t tie_last = 0xFFFFFFFFu;
        if (ties < here) {
            u64 none = 0;
            uint32_t inverted;
            narrow<ALONE, false, true>(0xFFFFFFFFu - (uint32_t)(a.vocab - 1), 0xFFFFFFFFu, none, ties, inverted,
                                       [&](float x, uint32_t i, uint32_t &k) { return k = ~i, x == x_cut; });
            tie_last = ~inverted;
        }
        // the draw: the first index at which the running mass of the kept entries exceeds u of
        // the whole
        const auto keep = [&](float x, uint32_t i) { return x > x_cut || (x == x_cut && i <= tie_last); };
        if (!ALONE) {
            draw(a, b, floor_w, keep);
            return;
        }
        uint32_t inverted;
        u64 mass_ahead = 0, whole_mass = 0;
        narrow<ALONE, true, true, true>(0xFFFFFFFFu - (uint32_t)(a.vocab - 1), 0xFFFFFFFFu, mass_ahead, first.target, inverted,
                                        [&](float x, uint32_t i, uint32_t &k) { return k = ~i, keep(x, i) && weight(x) >= floor_w; },
                                        &whole_mass, &a, b);
        const uint32_t token = ~inverted;
        each<ALONE>([&](float x, uint32_t index) {
            if (index != token || !QDQ_CHECK(&g_sample_status, token < (uint32_t)a.vocab && b < a.rows)) return;
            a.tokens[b] = (int64_t)token;
            if (a.logprobs) a.logprobs[b] = share_log(weight(x), whole_mass);
        });
    }
    // The same for a list of at most kFew entries: four threads to an entry. Its rank in the
    // list, the cuts as positions in that order (one warp), then the kept mass up to its
    // index, which is the draw.
    QDQ_DEV void finish_few(const SampleArgs &a, int b, const First &first, float top_p, float floor_w) {
        const int e = tid >> 2, q = tid & 3;
        u64 *sorted = sh.list + kFew, *mass = sh.list + 2 * kFew;
        const u64 mine = e < n ? sh.list[e] : 0;
        int rank_e = 0;
        for (int j = q; j < n; j += 4) rank_e += sh.list[j] > mine;
        rank_e += __shfl_xor_sync(kAll, rank_e, 1);
        rank_e += __shfl_xor_sync(kAll, rank_e, 2);
        if (e < n && q == 0) {
            sorted[rank_e] = mine;
            mass[rank_e] = fixed(weight(value_of((uint32_t)(mine >> 32))));
        }
        __syncthreads();
        if (warp == 0) {
            u64 f[4], incl = 0, excl;
            const int keep = first.top_k ? min((int)first.top_k, n) : n;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                f[y] = 4 * lane + y < keep ? mass[4 * lane + y] : 0;
                incl += f[y];
            }
            u64 sum = incl;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 t = __shfl_up_sync(kAll, sum, o);
                if (lane >= o) sum += t;
            }
            excl = sum - incl;
            // an entry is kept while the mass before it is below top-p's share
            const u64 target = top_p >= 1.0f ? ~0ull : first.top_k ? reach(top_p, __shfl_sync(kAll, sum, 31)) : first.target;
            u64 whole = 0;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int at = 4 * lane + y;
                const bool in = at < keep && excl < target && weight(value_of((uint32_t)(sorted[at] >> 32))) >= floor_w;
                excl += f[y];
                if (!in) f[y] = 0;
                if (at < n) mass[at] = f[y];
                whole += f[y];
            }
            whole = warp_sum(whole);
            if (lane == 0) sh.found[0] = whole;
        }
        __syncthreads();
        const u64 whole = sh.found[0];
        const u64 target = mark(a, b, whole);
        const u64 at = e < n ? sorted[e] : 0, f = e < n ? mass[e] : 0;
        u64 sum = 0;
        for (int j = q; j < n; j += 4)
            if ((uint32_t)sorted[j] >= (uint32_t)at) sum += mass[j];  // (inverted: an index not above this one)
        sum += __shfl_xor_sync(kAll, sum, 1);
        sum += __shfl_xor_sync(kAll, sum, 2);
        if (q == 0 && f && sum >= target && sum - f < target &&
            QDQ_CHECK(&g_sample_status, (uint32_t)~(uint32_t)at < (uint32_t)a.vocab && b < a.rows)) {
            a.tokens[b] = (int64_t)(uint32_t)~(uint32_t)at;
            if (a.logprobs) a.logprobs[b] = share_log(weight(value_of((uint32_t)(at >> 32))), whole);
        }
    }
    // top-p's mass to reach: at least one unit, so that the first entry is kept whatever it is.
    static QDQ_DEV u64 reach(float top_p, u64 whole_mass) {
        const double share = (double)top_p * (double)whole_mass;
        return share < 1.0 ? 1 : (u64)ceil(share);
    }
};

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleArgs a) {
    extern __shared__ __align__(16) char smem[];
    cluster_started_arrive();
    follow_last_kernel();
    Shared &sh = *reinterpret_cast<Shared *>(smem);
    Row r(sh, cluster_rank(), cluster_size());
    const uint32_t ctas = r.ctas, rank = r.rank;
    const int b = blockIdx.x / ctas, tid = r.tid;
    r.i_first = min((int)rank * a.slice, a.vocab);
    r.n = min(a.slice, a.vocab - r.i_first);
    const T *src = (const T *)a.logits + (int64_t)b * a.stride + r.i_first;
    const float temp = a.temperature ? a.temperature[b] : 1.0f;
    const int top_k = a.top_k ? a.top_k[b] : 0;
    const float top_p = a.top_p ? a.top_p[b] : 1.0f;
    const float floor_w = a.min_p ? fminf(a.min_p[b], 1.0f) : 0.0f;
    const bool greedy = !(temp > 0.0f);
    r.inv = greedy ? 1.0f : fmaxf(1.0f / temp, 1e-38f);  // (not 0: -inf x 0 is no number)

    // The slice, with the row's largest key and the lowest index that has it. NaN becomes
    // -inf and -0 becomes +0: equal logits have equal keys.
    float top_x = -INFINITY;
    int top_i = -1;
    unsigned live = 0;
    const auto put = [&](float x, int i) {
        x = x == x ? x + 0.0f : -INFINITY;
        live += x != -INFINITY;
        if (x > top_x) top_x = x, top_i = i;  // (a thread's indices rise)
        return x;
    };
    int done = 0;
    if (((uintptr_t)src & (4 * sizeof(T) - 1)) == 0) {  // four at a time where the row allows it
        done = r.n & ~3;
#pragma unroll 4
        for (int i = 4 * tid; i < done; i += 4 * kThreads) {
            if (!QDQ_CHECK(&g_sample_status, i + 4 <= a.slice && r.i_first + i + 4 <= a.vocab && b < a.rows)) break;
            float x[4];
            load4(src + i, x);
            *reinterpret_cast<float4 *>(sh.x + i) = make_float4(put(x[0], i), put(x[1], i + 1), put(x[2], i + 2), put(x[3], i + 3));
        }
    }
#pragma unroll 8
    for (int i = done + tid; i < r.n; i += kThreads)
        if (QDQ_CHECK(&g_sample_status, i < a.slice && r.i_first + i < a.vocab && b < a.rows)) sh.x[i] = put((float)src[i], i);
    u64 best = top_i < 0 ? 0 : ((u64)key_of(top_x) << 32) | (0xFFFFFFFFu - (unsigned)(r.i_first + top_i));
    for (int i = r.n + tid; i < (r.n + 127) / 128 * 128; i += kThreads)
        if (QDQ_CHECK(&g_sample_status, i < a.slice)) sh.x[i] = -INFINITY;
    for (int i = 0; i < 3; ++i) sh.bins[0][i][tid] = 0;
    const uint32_t mine = (uint32_t)(best >> 32);  // (0, which is no logit's, for a thread without any)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const u64 e = __shfl_xor_sync(kAll, best, o);
        best = e > best ? e : best;
    }
    cluster_started_wait();
    r.send<true>(best, __reduce_add_sync(kAll, live), ctas);
    cluster_sync();
    best = 0;
    u64 alive = 0;
    for (uint32_t c = 0; c < ctas; ++c) {
        best = r.part(c, 0) > best ? r.part(c, 0) : best;
        alive += r.part(c, 1);
    }
    r.top = value_of((uint32_t)(best >> 32));
    if (alive == 0 || greedy) {
        if (rank == 0 && tid == 0) {
            a.tokens[b] = alive ? (int64_t)(0xFFFFFFFFu - (unsigned)best) : -1;
            if (a.logprobs) a.logprobs[b] = alive ? 0.0f : -INFINITY;
        }
        return;
    }

    const bool by_k = top_k > 0 && (u64)top_k < alive, by_p = top_p < 1.0f;
    Row::First first = {by_k ? (u64)top_k : 0, 0, 0, 0};
    const float share = by_p ? top_p : 1.0f;
    if (!by_k && !by_p) {
        r.finish<false>(a, b, first, share, floor_w);
        return;
    }
    // the first level: the bin down to which entries are gathered
    const bool maxima = by_k && 4 * (int64_t)top_k <= min(a.vocab, kThreads * (int)ctas);
    if (tid == 0) sh.found[0] = kBins - 1;
    u64 all;
    if (maxima) {
        const int k = mine >= kLowest ? r.bin_of(value_of(mine)) : kBins - 1;
        __syncthreads();
        if (k < kBins - 1) r.count(0, k, 1u);
        const u64 count = r.gather_bins<false, 1>();
        const u64 ahead = r.before(count, &all);
        r.find(count, ahead, (u64)top_k);  // (the open bin if there are not as many)
        first.bin = (int)sh.found[0] & (kBins - 1);
    } else if (by_k) {
        r.first_counts<false>((u64)top_k, alive, first.bin, first.ahead);
    } else {
        r.each<false>([&](float x, uint32_t) {
            const int k = r.bin_of(x);
            if (k < kBins - 1) r.add_mass(k, r.weight(x));
        });
        const u64 mass = r.gather_bins<false, 3>();
        const u64 ahead = r.before(mass, &all);
        first.target = Row::reach(top_p, all);
        r.find(mass, ahead, first.target);
        first.bin = (int)sh.found[0] & (kBins - 1);
        first.ahead = sh.found[1];
    }
    u64 in_bin = 0;
    if (first.bin < kBins - 1) {
        // the entries down to that bin, and those in it
        u64 own = 0, listed;
        r.each_bit([&](float x, u64 bit) {
            const int k = r.bin_of(x);
            own |= k <= first.bin ? bit : 0;
            in_bin |= k == first.bin ? bit : 0;
        });
        r.send<false>(__reduce_add_sync(kAll, __popcll(own)), __reduce_add_sync(kAll, __popcll(in_bin)), ctas);
        cluster_sync();
        if (r.gather_list(own, 0, listed)) {
            if (rank || !QDQ_CHECK(&g_sample_status, listed <= kList)) return;
            r.n = (int)listed;
            if (listed <= kFew) r.finish_few(a, b, first, share, floor_w);
            else r.finish<true>(a, b, first, share, floor_w);
            return;
        }
    }
    if (maxima) r.first_counts<false>((u64)top_k, alive, first.bin, first.ahead);
    r.finish<false>(a, b, first, share, floor_w, in_bin);
}

// CTAs per row: enough to hold it (16384 entries each, which leaves room for two CTAs an
// SM, 32768 above 2^17), and more while all of them still run at once, down to slices of
// 2048 entries.
int cluster_for(int rows, int vocab, int sm_count) {
    int c = 1;
    while (c < kMaxCluster && vocab > c * (kSlice / 2)) c *= 2;
    while (c < kMaxCluster && 2 * c * rows <= 2 * sm_count && vocab > c * 2048) c *= 2;
    return c;
}

template <typename T>
int launch_sample(SampleArgs a, int sm_count, cudaStream_t stream) {
    const int c = cluster_for(a.rows, a.vocab, sm_count);
    a.slice = ((a.vocab + c - 1) / c + 127) / 128 * 128;  // (a warp's 128 neighbours share an index bin)
    const size_t smem = sizeof(Shared) + sizeof(float) * a.slice;
    static std::mutex mu;
    static bool attr_set[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return QDQ_ERR_CUDA;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!attr_set[dev]) {
            const RelaxedCaptureScope relaxed;
            if (cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)(sizeof(Shared) + sizeof(float) * kSlice)) != cudaSuccess) {
                cudaGetLastError();
                return QDQ_ERR_CUDA;
            }
            attr_set[dev] = true;
        }
    }
    return launch_following(sample_kernel<T>, (unsigned)a.rows * c, kThreads, smem, c, stream, a);
}

}  // namespace

int take_status_sample() {
    int v = 0;
#ifdef QDQ_DEBUG
    const int zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_sample_status, sizeof(int)) != cudaSuccess ||
        (v && cudaMemcpyToSymbol(g_sample_status, &zero, sizeof(int)) != cudaSuccess)) {
        cudaGetLastError();
        return QDQ_ERR_CUDA;
    }
#endif
    return v;
}

}  // namespace qdq

using namespace qdq;

extern "C" int qdq_sample(int type, const void *logits, int64_t stride, int rows, int vocab, const float *temperature,
                          const int32_t *top_k, const float *top_p, const float *min_p, const float *u,
                          int64_t *tokens, float *logprobs, qdq_stream_t stream) {
    if (type != QDQ_F32 && type != QDQ_F16 && type != QDQ_BF16) return QDQ_ERR_TYPE;
    if (rows < 0 || vocab < 1 || (rows > 1 && stride < vocab)) return QDQ_ERR_SHAPE;
    if (vocab > (1 << 18)) return QDQ_ERR_LIMIT;
    if (rows == 0) return QDQ_OK;
    int rc;
    const DeviceInfo &dev = current_device(&rc);
    if (rc) return rc;
    if ((rc = check_dev_ptr(logits, dev.device, type == QDQ_F32 ? 4 : 2)) || (rc = check_dev_ptr(u, dev.device, 4)) ||
        (rc = check_dev_ptr(tokens, dev.device, 8)) || (logprobs && (rc = check_dev_ptr(logprobs, dev.device, 4))) ||
        (temperature && (rc = check_dev_ptr(temperature, dev.device, 4))) ||
        (top_k && (rc = check_dev_ptr(top_k, dev.device, 4))) || (top_p && (rc = check_dev_ptr(top_p, dev.device, 4))) ||
        (min_p && (rc = check_dev_ptr(min_p, dev.device, 4))))
        return rc;
    if (rows > 0x7FFFFFFF / kMaxCluster) return QDQ_ERR_LIMIT;
    const SampleArgs a = {logits, stride, rows, vocab, 0, temperature, top_p, min_p, u, top_k, tokens, logprobs};
    cudaStream_t s = (cudaStream_t)stream;
    return type == QDQ_F32   ? launch_sample<float>(a, dev.sm_count, s)
           : type == QDQ_F16 ? launch_sample<__half>(a, dev.sm_count, s)
                             : launch_sample<__nv_bfloat16>(a, dev.sm_count, s);
}
