// qdq_sample.cu -- sampling: temperature, top-k, top-p and min-p from given random
// numbers.
//
// One pass over the logits: a cluster of up to eight CTAs holds a row in shared memory,
// a contiguous slice each, and everything after the load works on that copy.
//
// The filters are cuts of one order (logit descending, index ascending), so nothing is
// sorted. A cut is found by narrowing an interval of the logits' order-preserving 32-bit
// keys: first 512 bins that are linear in the exponent (1/16 wide, the last one open;
// counts only), then 512 equal parts of the interval at a time until it is one key; the
// entries with exactly that key are then kept by index. Top-k narrows by count. Top-p
// needs masses: the first level's bin is guessed from the counts (a bin's mass is close
// to count x e^-middle) and checked with the exact mass above it, moving to the next bin
// where the guess was off; below it the bins hold exact masses.
//
// Masses are integers (weights in units of 2^-44 of the largest), so neither the order of
// the additions nor the split over CTAs changes a sum. In the bins they are kept as three
// 15-bit pieces, each added with a native 32-bit shared-memory atomic (at most 2^15
// entries a slice, so a piece cannot overflow).
//
// The draw is an inverse CDF in index order: kept mass per CTA, per warp, per entry.
// CTAs of a cluster exchange sums by writing them to each other before a cluster barrier,
// and read each other's bins after one; two sets of buffers take turns, so one barrier
// per step is enough.
#include <cmath>
#include <mutex>

#include "qdq_internal.h"
#include "qdq_paged.cuh"

namespace qdq {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32, kBins = 512, kMaxCluster = 8;
constexpr int kSlice = 1 << 15;  // entries of a row that a CTA holds at most
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
    u64 sums[2][kMaxCluster][3];  // what the cluster's CTAs sent
    u64 warp[kWarps][3];
    u64 found[2];                 // the bin a cut lies in, and the measure above it
    uint32_t edge[2];
    float x[1];                   // the slice (slice entries)
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
QDQ_DEV u64 warp_sum(u64 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

// One CTA's part in the work on one row.
struct Row {
    Shared &sh;
    const int n;  // entries of the slice
    const int tid, lane, warp;
    const uint32_t rank, ctas;
    int turn_s = 0, turn_b = 0;
    float top = 0.0f, inv = 1.0f;

    QDQ_DEV Row(Shared &s, int n_, uint32_t r, uint32_t c)
        : sh(s), n(n_), tid(threadIdx.x), lane(threadIdx.x & 31), warp(threadIdx.x >> 5), rank(r), ctas(c) {}

    QDQ_DEV float weight(float x) const { return x == top ? 1.0f : expf((x - top) * inv); }  // (-inf weighs 0)
    static QDQ_DEV u64 fixed(float w) { return __float2ull_rn(w * 0x1p44f); }
    // The first level's bin: 1/16 of the exponent wide, falling logits, the last one open.
    QDQ_DEV int bin_of(float x) const { return min((int)((top - x) * inv * 16.0f), kBins - 1); }

    // Every warp's sums (lane 0's arguments) to every CTA; after it, part(r, i) is CTA r's.
    template <bool MAX>
    QDQ_DEV void send(u64 a, u64 b) {
        if (lane == 0) sh.warp[warp][0] = a, sh.warp[warp][1] = b;
        __syncthreads();
        if (tid < (int)ctas) {
            u64 x = 0, y = 0;
            for (int w = 0; w < kWarps; ++w) {
                x = MAX ? (sh.warp[w][0] > x ? sh.warp[w][0] : x) : x + sh.warp[w][0];
                y += sh.warp[w][1];
            }
            const uint32_t to = remote(&sh.sums[turn_s][rank][0], tid);
            asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to), "l"(x) : "memory");
            asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to + 8), "l"(y) : "memory");
        }
        cluster_sync();
        turn_s ^= 1;
    }
    QDQ_DEV u64 part(uint32_t r, int i) const { return sh.sums[turn_s ^ 1][r][i]; }
    QDQ_DEV u64 all(int i) const {
        u64 v = 0;
        for (uint32_t r = 0; r < ctas; ++r) v += part(r, i);
        return v;
    }

    QDQ_DEV void clear_bins(int pieces) {
        for (int i = tid; i < pieces * kBins; i += kThreads) (&sh.bins[turn_b][0][0])[i] = 0;
        __syncthreads();
    }
    QDQ_DEV void add_mass(int b, u64 f) {
        atomicAdd(&sh.bins[turn_b][0][b], (unsigned)f & 0x7FFFu);
        atomicAdd(&sh.bins[turn_b][1][b], (unsigned)(f >> 15) & 0x7FFFu);
        atomicAdd(&sh.bins[turn_b][2][b], (unsigned)(f >> 30));
    }
    // The cluster's sum of bin `tid` (each CTA reads all the others'); ends the turn.
    template <int PIECES>
    QDQ_DEV u64 gather_bins() {
        cluster_sync();
        u64 v = 0;
        for (uint32_t r = 0; r < ctas; ++r)
#pragma unroll
            for (int i = 0; i < PIECES; ++i) {
                unsigned x;
                asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(remote(&sh.bins[turn_b][i][tid], r)) : "memory");
                v += (u64)x << (15 * i);
            }
        turn_b ^= 1;
        return v;
    }
    // Sum over the bins before this thread's.
    template <typename V>
    QDQ_DEV V before(V v) {
        V incl = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const V e = __shfl_up_sync(kAll, incl, o);
            if (lane >= o) incl += e;
        }
        V *w = reinterpret_cast<V *>(&sh.warp[0][0]);
        if (lane == 31) w[warp] = incl;
        __syncthreads();
        V sum = 0;
        for (int i = 0; i < warp; ++i) sum += w[i];
        __syncthreads();
        return sum + incl - v;
    }

    // The bin where above + its prefix first reaches the target (count or mass), and the
    // prefix before it.
    template <typename REACHED>
    QDQ_DEV void find(u64 v, u64 above, REACHED reached, int &bin, u64 &ahead) {
        const u64 excl = above + before(v);
        if (v && !reached(excl) && reached(excl + v)) sh.found[0] = tid, sh.found[1] = excl;
        __syncthreads();
        bin = (int)sh.found[0];
        ahead = sh.found[1];
        __syncthreads();
    }

    // The keys whose first-level bin is b: [lo, hi]. Two warps search 32 probes at a time
    // for the smallest key whose bin is at most b, and at most b - 1.
    QDQ_DEV void keys_of(int b, uint32_t &lo, uint32_t &hi) {
        if (warp < 2) {
            const int want = b - warp;
            uint32_t first = kLowest, last = key_of(top);  // the answer lies in [first, last] (the top's bin is 0)
            if (want >= kBins - 1) last = first;
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
        __syncthreads();
    }

    // Narrows [lo, hi], which holds the cut, to the cut's key. `ahead`: the measure above hi,
    // and at the end above the key; returns the measure of the entries with that key.
    template <bool MASS, typename REACHED>
    QDQ_DEV u64 narrow(uint32_t lo, uint32_t hi, u64 &ahead, REACHED reached, uint32_t &key) {
        for (int level = 0; level < 4; ++level) {  // 9 bits a level: 32 bits take four
            int shift = 0;
            while (((hi - lo) >> shift) >= kBins) ++shift;
            clear_bins(MASS ? 3 : 1);
            for (int i = tid; i < n; i += kThreads) {
                const float x = sh.x[i];
                const uint32_t k = key_of(x);
                if (k < lo || k > hi) continue;
                const int b = (int)((hi - k) >> shift);
                if (MASS) add_mass(b, fixed(weight(x)));
                else atomicAdd(&sh.bins[turn_b][0][b], 1u);
            }
            const u64 v = gather_bins<MASS ? 3 : 1>();
            int b;
            find(v, ahead, reached, b, ahead);
            const uint32_t top_key = hi - ((uint32_t)b << shift);
            if (shift == 0) {
                key = top_key;
                if (tid == b) sh.found[0] = v;
                __syncthreads();
                const u64 here = sh.found[0];
                __syncthreads();
                return here;
            }
            const uint32_t wide = (1u << shift) - 1;
            lo = top_key - lo > wide ? top_key - wide : lo;
            hi = top_key;
        }
        key = hi;  // not reached
        return 1;
    }
};

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleArgs a) {
    extern __shared__ __align__(16) char smem[];
    Shared &sh = *reinterpret_cast<Shared *>(smem);
    const uint32_t ctas = cluster_size(), rank = cluster_rank();
    const int b = blockIdx.x / ctas, i_first = min((int)rank * a.slice, a.vocab);
    Row r(sh, min(a.slice, a.vocab - i_first), rank, ctas);
    const int tid = r.tid, lane = r.lane, warp = r.warp, n = r.n;
    const T *src = (const T *)a.logits + (int64_t)b * a.stride + i_first;
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
    for (int i = tid; i < n; i += kThreads) {
        float x = (float)src[i];
        x = x == x ? x + 0.0f : -INFINITY;
        sh.x[i] = x;
        live += x != -INFINITY;
        const u64 e = ((u64)key_of(x) << 32) | (0xFFFFFFFFu - (unsigned)(i_first + i));
        best = e > best ? e : best;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const u64 e = __shfl_xor_sync(kAll, best, o);
        best = e > best ? e : best;
    }
    r.send<true>(best, __reduce_add_sync(kAll, live));
    best = 0;
    for (uint32_t c = 0; c < ctas; ++c) best = r.part(c, 0) > best ? r.part(c, 0) : best;
    const u64 alive = r.all(1);
    r.top = value_of((uint32_t)(best >> 32));
    if (alive == 0 || greedy) {
        if (rank == 0 && tid == 0) {
            a.tokens[b] = alive ? (int64_t)(0xFFFFFFFFu - (unsigned)best) : -1;
            if (a.logprobs) a.logprobs[b] = alive ? 0.0f : -INFINITY;
        }
        return;
    }

    // The cut: entries with a key above `cut` are kept, and the first `ties` with that key.
    const bool by_k = top_k > 0 && (u64)top_k < alive, by_p = top_p < 1.0f;
    uint32_t cut = kLowest;
    u64 ties = ~0ull;
    if (by_k || by_p) {
        // first level: counts (the open bin's is what the others leave)
        r.clear_bins(1);
        for (int i = tid; i < n; i += kThreads) {
            const int k = r.bin_of(sh.x[i]);
            if (k < kBins - 1) atomicAdd(&sh.bins[r.turn_b][0][k], 1u);
        }
        u64 count = r.gather_bins<1>();
        const u64 count_before = r.before(count);
        if (tid == kBins - 1) count = alive - count_before;
        u64 total = 0;
        if (by_k) {
            const auto reached = [&](u64 v) { return v >= (u64)top_k; };
            int bin;
            u64 ahead;
            r.find(count, 0, reached, bin, ahead);
            uint32_t lo, hi;
            r.keys_of(bin, lo, hi);
            r.narrow<false>(lo, hi, ahead, reached, cut);
            ties = (u64)top_k - ahead;
            if (tid > bin) count = 0;
            if (tid == bin) count = (u64)top_k - count_before;
        }
        if (by_p) {
            // the mass that top-k left
            u64 m = 0;
            for (int i = tid; i < n; i += kThreads) {
                const float x = sh.x[i];
                if (by_k ? key_of(x) > cut : true) m += Row::fixed(r.weight(x));
            }
            r.send<false>(warp_sum(m), 0);
            total = r.all(0) + (by_k ? ties * Row::fixed(r.weight(value_of(cut))) : 0);
            // (at least one unit, so that the first entry is kept whatever top_p is)
            const double target = fmax((double)top_p * (double)total, 1.0);
            const auto reached = [&](u64 v) { return (double)v >= target; };
            // a guess of the bin: mass close to count x e^-middle, in double
            const double guess = (double)count * (double)expf(-((float)tid + 0.5f) * 0.0625f);
            const double g0 = r.before(guess), share = target * 0x1p-44;
            if (tid == 0) sh.found[0] = kBins;
            __syncthreads();
            if (count && g0 + guess >= share) atomicMin(&sh.found[0], (u64)tid);
            __syncthreads();
            int bin = (int)sh.found[0];
            __syncthreads();
            bin = min(bin, kBins - 1);
            for (;;) {
                // the exact mass above the bin and in it
                u64 above = 0, in = 0;
                for (int i = tid; i < n; i += kThreads) {
                    const float x = sh.x[i];
                    const int k = r.bin_of(x);
                    if (k <= bin) {
                        const u64 f = Row::fixed(r.weight(x));
                        if (k < bin) above += f;
                        else in += f;
                    }
                }
                r.send<false>(warp_sum(above), warp_sum(in));
                above = r.all(0);
                in = r.all(1);
                if (reached(above)) {
                    --bin;
                } else if (!reached(above + in) && bin < kBins - 1) {
                    ++bin;
                } else {
                    uint32_t lo, hi, key;
                    r.keys_of(bin, lo, hi);
                    u64 ahead = above;
                    const u64 here = r.narrow<true>(lo, hi, ahead, reached, key);
                    const u64 f = Row::fixed(r.weight(value_of(key)));
                    // the fewest ties that reach the target, out of those that top-k kept
                    u64 most = here / f, need = 1;
                    if (by_k && key == cut) most = min(most, ties);
                    const double left = target - (double)ahead;
                    if (left > (double)f) need = (u64)ceil(left / (double)f);
                    while (need > 1 && reached(ahead + (need - 1) * f)) --need;
                    while (need < most && !reached(ahead + need * f)) ++need;
                    cut = key;
                    ties = min(need, most);
                    break;
                }
            }
        }
    }

    // Kept mass, in index order: per warp's segment of the slice, per CTA. Ties are counted
    // apart: they weigh the same, and how many of a segment's are kept follows from the
    // ties ahead of it.
    const bool all_ties = ties == ~0ull;  // nothing was cut: `cut` is the lowest key, and kept
    const u64 tie_f = [&] {
        const float w = r.weight(value_of(cut));
        return w >= floor_w ? Row::fixed(w) : 0ull;
    }();
    const int per = (n + kWarps - 1) / kWarps, s0 = min(warp * per, n), s1 = min(s0 + per, n);
    u64 mass = 0;
    unsigned tied = 0;
    for (int i = s0 + lane; i < s1; i += 32) {
        const float x = sh.x[i];
        const uint32_t k = key_of(x);
        if (k > cut || (all_ties && k == cut)) {
            const float w = r.weight(x);
            mass += w >= floor_w ? Row::fixed(w) : 0ull;
        }
        tied += !all_ties && k == cut;
    }
    mass = warp_sum(mass);
    tied = __reduce_add_sync(kAll, tied);
    r.send<false>(mass, tied);
    const auto clip = [&](u64 t0, u64 t) {  // of t ties after t0 others, how many are kept
        return t0 >= ties ? 0ull : min(t, ties - t0);
    };
    u64 whole = 0, ahead = 0, t_ahead = 0, t_all = 0;
    for (uint32_t c = 0; c < ctas; ++c) {
        const u64 m = r.part(c, 0) + clip(t_all, r.part(c, 1)) * tie_f;
        if (c == rank) ahead = whole, t_ahead = t_all;
        whole += m;
        t_all += r.part(c, 1);
    }
    // sums of the warps' segments ahead of this one (send() left them in place)
    for (int w = 0; w < warp; ++w) {
        ahead += sh.warp[w][0] + clip(t_ahead, sh.warp[w][1]) * tie_f;
        t_ahead += sh.warp[w][1];
    }
    const u64 mine = mass + clip(t_ahead, tied) * tie_f;
    const double target = fmax((double)a.u[b], 0.0) * (double)whole;
    // u = 1 asks for the last kept entry: the segment that ends at the whole
    const bool at_end = !((double)whole > target);
    if (mine == 0 || !(at_end ? ahead + mine == whole : (double)ahead <= target && (double)(ahead + mine) > target)) return;
    u64 sum = ahead, seen = t_ahead;
    for (int i = s0; i < s1; i += 32) {
        const float x = i + lane < s1 ? sh.x[i + lane] : -INFINITY;
        const uint32_t k = key_of(x);
        const bool tie = !all_ties && k == cut;
        const unsigned m = __ballot_sync(kAll, tie);
        const bool keep = k > cut || (all_ties && k == cut) || (tie && seen + __popc(m & ((1u << lane) - 1)) < ties);
        const float w = keep ? r.weight(x) : 0.0f;
        const u64 f = keep && w >= floor_w ? Row::fixed(w) : 0ull;
        u64 incl = f;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 e = __shfl_up_sync(kAll, incl, o);
            if (lane >= o) incl += e;
        }
        const unsigned hit = __ballot_sync(kAll, f && (at_end ? sum + incl == whole : (double)(sum + incl) > target));
        if (hit) {
            const int l = __ffs(hit) - 1;
            if (lane == l) {
                a.tokens[b] = i_first + i + l;
                if (a.logprobs) a.logprobs[b] = (float)log((double)w / ((double)whole * 0x1p-44));
            }
            return;
        }
        sum += __shfl_sync(kAll, incl, 31);
        seen += __popc(m);
    }
}

// CTAs per row: enough to hold it (32768 entries each, half of that where it leaves two
// CTAs an SM), and, with few rows, to give every SM two, down to slices of 2048 entries.
int cluster_for(int rows, int vocab, int sm_count) {
    int c = 1;
    while (c < kMaxCluster && vocab > c * (kSlice / 2)) c *= 2;
    while (c < kMaxCluster && rows * c < 2 * sm_count && vocab > c * 2048) c *= 2;
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
