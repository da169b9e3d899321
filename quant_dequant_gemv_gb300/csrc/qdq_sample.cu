// qdq_sample.cu -- sampling: temperature, top-k, top-p and min-p from given random
// numbers.
//
// One pass over the logits: a cluster of up to eight CTAs holds a row's order-preserving
// 32-bit keys in shared memory, a contiguous slice each, and everything after the load
// works on those.
//
// The filters are cuts of one order (logit descending, index ascending), so nothing is
// sorted. A cut is found by narrowing: 512 bins over an interval of keys, a scan, and the
// bin that reaches the wanted count or mass becomes the next interval until it is one
// key. The first bins are linear in the exponent (1/16 wide, the last one open) instead
// of the key; the entries that share the cut's key are told apart by narrowing over their
// indices, and so is the draw itself (an inverse CDF in index order).
//
// The first counts bound the kept set from above: all entries of a bin have weights
// within a factor e^(1/16), so a prefix of bins whose estimated mass exceeds top-p's share
// of the estimated whole by 1/15 is certain to hold the cut. If that prefix (or top-k's
// bin) has at most kList entries, they are gathered in the first CTA, which finishes
// alone while the others leave; otherwise the cluster narrows together.
//
// Masses are integers (weights in units of 2^-44 of the largest), so neither the order of
// the additions nor the split over CTAs changes a sum. In the bins they are kept as three
// 15-bit pieces, each added with a native 32-bit shared-memory atomic (at most 2^15
// entries a CTA, so a piece cannot overflow).
//
// CTAs of a cluster send sums to each other before a cluster barrier and read each
// other's bins after one; two sets of buffers take turns, so a step needs one barrier.
#include <cmath>
#include <mutex>

#include "qdq_internal.h"
#include "qdq_paged.cuh"

namespace qdq {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32, kBins = kThreads, kMaxCluster = 8;
constexpr int kSlice = 1 << 15;  // entries of a row that a CTA holds at most
constexpr int kList = 2048;
constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr uint32_t kLowest = 0x00800000u;  // the key of the lowest finite logit (-inf is one below)
typedef unsigned long long u64;

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
    unsigned bins[2][3][kBins];
    u64 sums[2][kMaxCluster][2];  // what the cluster's CTAs sent
    u64 warp[kWarps + 1][2];
    u64 found[2];                 // the bin a cut lies in, and the measure above it
    uint32_t edge[2];
    u64 list[kList];              // key << 32 | index
    uint32_t key[1];              // the slice (slice entries)
};

QDQ_DEV void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
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

    QDQ_DEV float weight(uint32_t key) const {  // (-inf weighs 0)
        const float x = value_of(key);
        return x == top ? 1.0f : expf((x - top) * inv);
    }
    static QDQ_DEV u64 fixed(float w) { return __float2ull_rn(w * 0x1p44f); }
    // The first level's bin: 1/16 of the exponent wide, falling logits, the last one open.
    QDQ_DEV int bin_of(uint32_t key) const { return min((int)((top - value_of(key)) * inv * 16.0f), kBins - 1); }

    template <bool ALONE>
    QDQ_DEV void sync() {
        if (ALONE) __syncthreads();
        else cluster_sync();
    }
    template <bool ALONE, typename F>
    QDQ_DEV void each(F f) {  // f(key, index) over this CTA's entries
        if (ALONE) {
            for (int i = tid; i < n; i += kThreads) f((uint32_t)(sh.list[i] >> 32), (uint32_t)sh.list[i]);
        } else {
            for (int i = tid; i < n; i += kThreads) f(sh.key[i], (uint32_t)(i_first + i));
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

    QDQ_DEV void clear_bins(int pieces) {
        for (int i = 0; i < pieces; ++i) sh.bins[turn_b][i][tid] = 0;
        __syncthreads();
    }
    QDQ_DEV void add_mass(int b, u64 f) {
        atomicAdd(&sh.bins[turn_b][0][b], (unsigned)f & 0x7FFFu);
        atomicAdd(&sh.bins[turn_b][1][b], (unsigned)(f >> 15) & 0x7FFFu);
        atomicAdd(&sh.bins[turn_b][2][b], (unsigned)(f >> 30));
    }
    // Bin `tid` over the whole cluster (each CTA reads all the others'), and over the CTAs
    // below this one; ends the turn.
    template <bool ALONE, int PIECES>
    QDQ_DEV u64 gather_bins(u64 *below = nullptr) {
        sync<ALONE>();
        u64 v = 0, low = 0;
        if (ALONE) {
#pragma unroll
            for (int i = 0; i < PIECES; ++i) v += (u64)sh.bins[turn_b][i][tid] << (15 * i);
        } else {
            unsigned x[PIECES];
#pragma unroll 4
            for (uint32_t r = 0; r < ctas; ++r) {
                if (r == rank) low = v;
#pragma unroll
                for (int i = 0; i < PIECES; ++i)
                    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x[i]) : "r"(remote(&sh.bins[turn_b][i][tid], r)));
#pragma unroll
                for (int i = 0; i < PIECES; ++i) v += (u64)x[i] << (15 * i);
            }
        }
        if (below) *below = low;
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
                const unsigned m = __ballot_sync(kAll, bin_of(at) <= want);
                if (m && !(m & 1)) first = last = __shfl_sync(kAll, at, __ffs(m) - 1);
            }
            while (first < last && want >= 0) {
                const uint32_t step = (last - first) / 32 + 1;
                const u64 at = (u64)first + (u64)step * lane;
                const unsigned m = __ballot_sync(kAll, at >= last || bin_of((uint32_t)at) <= want);
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

    // The largest key in [lo, hi] at which the measure from hi down (from `ahead` on)
    // reaches the target; `ahead` becomes the measure above it; returns its own. get(key,
    // index, k, f): whether an entry counts, under which key, with which mass. With SHARE
    // the target is the share of the whole that `share` asks for, set at the first level.
    template <bool ALONE, bool MASS, bool SHARE = false, typename GET>
    QDQ_DEV u64 narrow(uint32_t lo, uint32_t hi, u64 &ahead, u64 &target, uint32_t &key, GET get, double share = 0.0,
                       u64 *whole = nullptr) {
        for (int level = 0; level < 4; ++level) {  // 9 bits a level: 32 bits take four
            const int shift = max(0, 32 - 9 - __clz(hi - lo));
            clear_bins(MASS ? 3 : 1);
            each<ALONE>([&](uint32_t entry, uint32_t index) {
                uint32_t k;
                if (!get(entry, index, k) || k < lo || k > hi) return;
                const int b = (int)((hi - k) >> shift);
                if (MASS) add_mass(b, fixed(weight(entry)));
                else atomicAdd(&sh.bins[turn_b][0][b], 1u);
            });
            const u64 v = gather_bins<ALONE, MASS ? 3 : 1>();
            u64 all;
            const u64 excl = ahead + before(v, &all);
            if (SHARE && level == 0) {
                *whole = all;
                target = min((u64)(share * (double)all) + 1, all);
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

    // Everything after the first counts: the cuts, the ties, the draw. bin, ahead: top-k's
    // first-level bin and the count above it.
    template <bool ALONE>
    QDQ_DEV void finish(const SampleArgs &a, int b, u64 top_k, int bin, u64 ahead, bool by_p, float top_p, float floor_w,
                        u64 total) {
        uint32_t cut = kLowest, lo, hi;
        u64 ties = ~0ull, here = 0, target;  // entries above `cut` are kept, and the first `ties` at it
        if (top_k) {
            keys_of(bin, lo, hi);
            target = top_k;
            here = narrow<ALONE, false>(lo, hi, ahead, target, cut, [](uint32_t e, uint32_t, uint32_t &k) { return k = e, true; });
            ties = top_k - ahead;
        }
        if (by_p) {
            // exact masses of the first-level bins of what top-k left; their sum is the whole,
            // but for a list, which holds part of it unless top-k chose it. The cut's own bin
            // may hold more ties than top-k kept: none that the target reaches.
            clear_bins(3);
            u64 low = 0;  // mass of the ties that top-k dropped
            each<ALONE>([&](uint32_t key, uint32_t) {
                if (key >= cut) add_mass(bin_of(key), fixed(weight(key)));
            });
            if (top_k) low = (here - ties) * fixed(weight(cut));
            const u64 v = gather_bins<ALONE, 3>();
            u64 all;
            const u64 excl = before(v, &all);
            if (!ALONE || top_k) total = all - low;
            // (at least one unit, so that the first entry is kept whatever top_p is)
            const double share = (double)top_p * (double)total;
            target = share < 1.0 ? 1 : (u64)ceil(share);
            find(v, excl, target);
            const int p_bin = (int)sh.found[0] & (kBins - 1);
            u64 above = sh.found[1];
            keys_of(p_bin, lo, hi);
            uint32_t key;
            const u64 mass = narrow<ALONE, true>(max(lo, cut), hi, above, target, key,
                                                 [](uint32_t e, uint32_t, uint32_t &k) { return k = e, true; });
            // the fewest of the entries at the key that reach the target
            const u64 f = fixed(weight(key)), need = (target - above + f - 1) / f;
            const u64 most = top_k && key == cut ? ties : mass / f;
            here = mass / f;
            cut = key;
            ties = min(need, most);
        }
        // ties: the index of the last one kept (narrowing runs over inverted indices, so that
        // the lowest come first)
        uint32_t tie_last = 0xFFFFFFFFu;
        if (ties < here) {
            u64 none = 0;
            uint32_t inverted;
            narrow<ALONE, false>(0xFFFFFFFFu - (uint32_t)(a.vocab - 1), 0xFFFFFFFFu, none, ties, inverted,
                                 [&](uint32_t e, uint32_t i, uint32_t &k) { return k = ~i, e == cut; });
            tie_last = ~inverted;
        }
        // the draw: the first index at which the running mass of the kept entries exceeds u of
        // the whole (at u = 1, reaches the whole)
        uint32_t inverted;
        u64 mass_ahead = 0, whole;
        narrow<ALONE, true, true>(0xFFFFFFFFu - (uint32_t)(a.vocab - 1), 0xFFFFFFFFu, mass_ahead, target, inverted,
                                  [&](uint32_t e, uint32_t i, uint32_t &k) {
                                      k = ~i;
                                      return (e > cut || (e == cut && i <= tie_last)) && weight(e) >= floor_w;
                                  },
                                  fmin(fmax((double)a.u[b], 0.0), 1.0), &whole);
        const uint32_t token = ~inverted;
        each<ALONE>([&](uint32_t key, uint32_t index) {
            if (index != token) return;
            a.tokens[b] = (int64_t)token;
            if (a.logprobs) a.logprobs[b] = (float)log((double)weight(key) / ((double)whole * 0x1p-44));
        });
    }
};

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleArgs a) {
    extern __shared__ __align__(16) char smem[];
    Shared &sh = *reinterpret_cast<Shared *>(smem);
    Row r(sh, cluster_rank(), cluster_size());
    const uint32_t ctas = r.ctas, rank = r.rank;
    const int b = blockIdx.x / ctas, tid = r.tid, lane = r.lane;
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
    u64 best = 0;
    unsigned live = 0;
#pragma unroll 8
    for (int i = tid; i < r.n; i += kThreads) {
        float x = (float)src[i];
        x = x == x ? x + 0.0f : -INFINITY;
        const uint32_t k = key_of(x);
        sh.key[i] = k;
        live += k >= kLowest;
        const u64 e = ((u64)k << 32) | (0xFFFFFFFFu - (unsigned)(r.i_first + i));
        best = e > best ? e : best;
    }
    sh.bins[0][0][tid] = 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const u64 e = __shfl_xor_sync(kAll, best, o);
        best = e > best ? e : best;
    }
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
    if (!by_k && !by_p) {
        r.finish<false>(a, b, 0, 0, 0, false, top_p, floor_w, 0);
        cluster_sync();  // (no CTA leaves while another reads its bins)
        return;
    }
    // first level: counts (the open bin's is what the others leave)
    for (int i = tid; i < r.n; i += kThreads) {
        const int k = r.bin_of(sh.key[i]);
        if (k < kBins - 1) atomicAdd(&sh.bins[0][0][k], 1u);
    }
    u64 below, all;
    u64 count = r.gather_bins<false, 1>(&below);
    const u64 count_before = r.before(count, &all);
    if (tid == kBins - 1) count = alive - count_before;
    int bin = 0;
    u64 ahead = 0;
    if (by_k) {
        r.find(count, count_before, (u64)top_k);
    } else {
        // a prefix of bins that is certain to hold top-p's cut (the open bin weighs nothing
        // next to the slack: 2^18 e^-32)
        const float mid = expf(-((float)tid + 0.5f) * 0.0625f);
        float sum;
        const float est = tid == kBins - 1 ? 0.0f : (float)count * mid, est_before = r.before(est, &sum);
        const float want = top_p * sum * 1.0667f + 1e-6f;
        if (tid == 0) sh.found[0] = kBins - 1;
        __syncthreads();
        if (est > 0.0f && est_before + est >= want) atomicMin(&sh.found[0], (u64)tid);
        __syncthreads();
    }
    bin = (int)sh.found[0];
    ahead = sh.found[1];
    // entries in the bins up to that one: in the cluster, and in the CTAs below this one
    u64 listed, at;
    {
        const u64 both = ((tid <= bin ? count : 0) << 32) + (tid <= bin ? below : 0);
        u64 sum;
        r.before(both, &sum);
        listed = sum >> 32;
        at = sum & 0xFFFFFFFFu;
    }
    if (listed <= kList && bin < kBins - 1) {
        // into the first CTA's list, this CTA's entries from `at` on; their order is of no
        // consequence. With top-p alone the whole mass is needed too.
        if (tid == 0) sh.edge[0] = 0;
        __syncthreads();
        const uint32_t to = remote(&sh.list[0], 0);
        u64 mass = 0;
        for (int i0 = 0; i0 < r.n; i0 += kThreads) {
            const int i = i0 + tid;
            const uint32_t k = i < r.n ? sh.key[i] : 0;
            const bool take = i < r.n && r.bin_of(k) <= bin;
            const unsigned m = __ballot_sync(kAll, take);
            if (m) {
                unsigned base = 0;
                if (lane == 0) base = atomicAdd(&sh.edge[0], (unsigned)__popc(m));
                base = __shfl_sync(kAll, base, 0) + __popc(m & ((1u << lane) - 1));
                if (take && at + base < kList) store_remote(to + 8 * ((uint32_t)at + base), ((u64)k << 32) | (uint32_t)(r.i_first + i));
            }
            if (!by_k && i < r.n) mass += Row::fixed(r.weight(k));
        }
        r.send<false>(warp_sum(mass), 0, 1);
        cluster_sync();
        if (rank) return;
        u64 total = 0;
        for (uint32_t c = 0; c < ctas; ++c) total += r.part(c, 0);
        r.n = (int)listed;
        r.finish<true>(a, b, by_k ? (u64)top_k : 0, bin, ahead, by_p, top_p, floor_w, total);
        return;
    }
    r.finish<false>(a, b, by_k ? (u64)top_k : 0, bin, ahead, by_p, top_p, floor_w, 0);
    cluster_sync();
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
    a.slice = ((a.vocab + c - 1) / c + 7) / 8 * 8;
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
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.rows * c, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)c;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, sample_kernel<T>, a) != cudaSuccess) {
        cudaGetLastError();
        return QDQ_ERR_CUDA;
    }
    return QDQ_OK;
}

}  // namespace
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
