// qdq_pages.cu -- for attention over a few of a sequence's pages: bounds of each page's keys, and the
// pages that a cheap score over those bounds selects.
//
// Bounds. For each page and kv head, per dim the largest and the smallest key in units of 2^E,
//   mx = ceil(max k * 2^-E), mn = floor(min k * 2^-E),  E the least with max |k| <= 127 * 2^E,
// as signed bytes: all of max k * 2^-E is exact, so the bounds are the same whatever the order.
// Score. A query head is rounded to bytes qi in units of 2^Eq in the same way; a page's score is
//   max over the group's heads of 2^(Eq + E) * sum_d (qi_d < 0 ? qi_d * mn_d : qi_d * mx_d),
// no less than 2^E * 2^Eq * qi . k 2^-E for any key of the page. The sum is an integer below 2^21 and
// the scale a power of two, so a score is exact and the selection does not depend on any order.
// Both are bound by their steps' latency: bounds of 61 tokens' pages (8 heads of 128, e4m3, 64 positions)
// 5.1 us, of 7436 tokens' (bf16) 8.2; a selection for 64 tokens over 15 to 626 pages 15.5 us, for one
// over 8188 pages 16.7, where HBM would need 5.3 and 2.5.
#include <algorithm>

#include "qdq_internal.h"
#include "qdq_paged.cuh"

namespace qdq {
namespace {

#ifdef QDQ_DEBUG
__device__ int g_pages_status;
#endif

constexpr int kLeastBound = -100, kMostBound = 121;  // of E and Eq
constexpr int kMostWindow = 16;

// The least E with amax <= 127 * 2^E (= 1.984375 * 2^(6 + E)), inside its range.
QDQ_DEV int bound_exponent(float amax) {
    const int bits = __float_as_int(amax);
    return min(max((bits >> 23) - 127 - 6 + ((bits & 0x7FFFFF) > 0x7E0000), kLeastBound), kMostBound);
}

template <int TYPE>
struct Pair;  // two values in 32 bits
template <>
struct Pair<QDQ_F16> {
    using T = __half2;
    static QDQ_DEV uint32_t infinity() { return 0x7C007C00u; }
    static QDQ_DEV float2 unpack(uint32_t v) { return Float16<__half>::unpack(v); }
};
template <>
struct Pair<QDQ_BF16> {
    using T = __nv_bfloat162;
    static QDQ_DEV uint32_t infinity() { return 0x7F807F80u; }
    static QDQ_DEV float2 unpack(uint32_t v) { return Float16<__nv_bfloat16>::unpack(v); }
};
template <>
struct Pair<QDQ_E4M3> : Pair<QDQ_F16> {};

template <typename T>
QDQ_DEV uint32_t least(uint32_t a, uint32_t b) {
    T r = __hmin2(*reinterpret_cast<T *>(&a), *reinterpret_cast<T *>(&b));
    return *reinterpret_cast<uint32_t *>(&r);
}
template <typename T>
QDQ_DEV uint32_t most(uint32_t a, uint32_t b) {
    T r = __hmax2(*reinterpret_cast<T *>(&a), *reinterpret_cast<T *>(&b));
    return *reinterpret_cast<uint32_t *>(&r);
}

// A CTA takes one kv head of the pages that a window of tokens is the first new one of; its four
// warps take the page's blocks of 16 positions in turn, 16 bytes of a row a lane, and join at the end.
template <int TYPE, int D>
__global__ void __launch_bounds__(128) bounds_kernel(const PagesArgs a) {
    using P = Pair<TYPE>;
    using T = typename P::T;
    constexpr int kSize = TYPE == QDQ_E4M3 ? 1 : 2, kValues = 16 / kSize;  // of a lane's 16 bytes
    constexpr int kLanes = D * kSize / 16, kRows = 32 / kLanes, kSteps = 16 / kRows;  // a row's lanes, rows a step
    __shared__ float s_most[4][D], s_least[4][D];
    __shared__ float s_top[4];
    follow_last_kernel();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, at = lane % kLanes, sub = lane / kLanes;
    const int head = blockIdx.x % a.n_kv_heads, t0 = (int)(blockIdx.x / a.n_kv_heads) * a.window;
    const int page_size = 1 << a.page_shift;
    int s = find_seq(a.q_start, a.n_seqs, t0);
    if (s < 0) return;
    for (int t = t0; t < min(t0 + a.window, a.n_tokens);) {
        while (s + 1 < a.n_seqs && a.q_start[s + 1] <= t) ++s;
        int first, count;
        seq_tokens(a.q_start, s, a.n_tokens, first, count);
        if (t < first || t >= first + count) return;  // rows of no sequence: the batch's last
        const int kv = max(a.kv_len[s], 0), p = kv - count + (t - first);
        const int in_page = p & (page_size - 1);
        const int next = p < 0 ? -p : page_size - in_page;  // tokens to the next page's first
        const bool lead = p >= 0 && (t == first || in_page == 0);
        t = min(t + next, first + count);
        if (!lead) continue;
        const int logical = p >> a.page_shift;
        const int page = logical < a.max_pages ? a.page_table[(int64_t)s * a.max_pages + logical] : -1;
        if (page < 0 || page >= a.n_pages) continue;
        const int held = min(page_size, kv - (logical << a.page_shift));

        float hi[kValues], lo[kValues];
#pragma unroll
        for (int i = 0; i < kValues; ++i) hi[i] = -INFINITY, lo[i] = INFINITY;
        for (int b = warp; 16 * b < held; b += 4) {
            uint4 x[kSteps];
            float scale = 1.0f;
            if (TYPE == QDQ_E4M3)
                scale = power_of_two(exponent_of(a.k_scales[(((int64_t)page * a.n_kv_heads + head) << (a.page_shift - 4)) + b]));
#pragma unroll
            for (int y = 0; y < kSteps; ++y) {
                const int row = 16 * b + y * kRows + sub;
                x[y] = make_uint4(0, 0, 0, 0);
                // (e4m3 pools hold a page's heads one after the other, the others its positions)
                const int64_t r = TYPE == QDQ_E4M3 ? (((int64_t)page * a.n_kv_heads + head) << a.page_shift) + row
                                                   : (((int64_t)page << a.page_shift) + row) * a.n_kv_heads + head;
                if (row < held && QDQ_CHECK(&g_pages_status, page < a.n_pages && row < page_size))
                    x[y] = __ldg(reinterpret_cast<const uint4 *>((const char *)a.k_pages + r * D * kSize) + at);
            }
            uint32_t u_hi[kValues / 2], u_lo[kValues / 2];
#pragma unroll
            for (int i = 0; i < kValues / 2; ++i) u_lo[i] = P::infinity(), u_hi[i] = P::infinity() | 0x80008000u;
#pragma unroll
            for (int y = 0; y < kSteps; ++y) {
                if (16 * b + y * kRows + sub >= held) continue;
                const uint32_t v[4] = {x[y].x, x[y].y, x[y].z, x[y].w};
#pragma unroll
                for (int i = 0; i < kValues / 2; ++i) {
                    uint32_t w[2];
                    if constexpr (TYPE == QDQ_E4M3) e4m3x4_to_f16(v[i / 2], w[0], w[1]);
                    else w[0] = w[1] = v[i];
                    u_hi[i] = most<T>(u_hi[i], w[i & 1]);
                    u_lo[i] = least<T>(u_lo[i], w[i & 1]);
                }
            }
#pragma unroll
            for (int i = 0; i < kValues / 2; ++i) {
                const float2 h = P::unpack(u_hi[i]), l = P::unpack(u_lo[i]);
                hi[2 * i] = fmaxf(hi[2 * i], h.x * scale), hi[2 * i + 1] = fmaxf(hi[2 * i + 1], h.y * scale);
                lo[2 * i] = fminf(lo[2 * i], l.x * scale), lo[2 * i + 1] = fminf(lo[2 * i + 1], l.y * scale);
            }
        }
#pragma unroll
        for (int o = kLanes; o < 32; o <<= 1)
#pragma unroll
            for (int i = 0; i < kValues; ++i) {
                hi[i] = fmaxf(hi[i], __shfl_xor_sync(0xFFFFFFFFu, hi[i], o));
                lo[i] = fminf(lo[i], __shfl_xor_sync(0xFFFFFFFFu, lo[i], o));
            }
        if (sub == 0) {
#pragma unroll
            for (int i = 0; i < kValues; ++i) s_most[warp][at * kValues + i] = hi[i], s_least[warp][at * kValues + i] = lo[i];
        }
        __syncthreads();
        const int d = threadIdx.x;
        float mx = 0.0f, mn = 0.0f, top = 0.0f;
        if (d < D) {
            mx = fmaxf(fmaxf(s_most[0][d], s_most[1][d]), fmaxf(s_most[2][d], s_most[3][d]));
            mn = fminf(fminf(s_least[0][d], s_least[1][d]), fminf(s_least[2][d], s_least[3][d]));
            if (mx < mn) mx = mn = 0.0f;  // (no key here is a number)
            top = fmaxf(fabsf(mx), fabsf(mn));
        }
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        if (lane == 0) s_top[warp] = top;
        __syncthreads();
        const int e = bound_exponent(fmaxf(fmaxf(s_top[0], s_top[1]), fmaxf(s_top[2], s_top[3])));
        const int64_t unit = (int64_t)page * a.n_kv_heads + head;
        if (d < D) {
            // (2^-e in two steps: it may lie below fp32's normal range)
            const float f0 = power_of_two(-e / 2), f1 = power_of_two(-e - -e / 2);
            a.bounds[unit * 2 * D + d] = (int8_t)fminf(fmaxf(ceilf(mx * f0 * f1), -127.0f), 127.0f);
            a.bounds[unit * 2 * D + D + d] = (int8_t)fminf(fmaxf(floorf(mn * f0 * f1), -127.0f), 127.0f);
        }
        if (d == 0) a.bound_scales[unit] = (uint8_t)(e + 127);
        __syncthreads();
    }
}

// ---- selection --------------------------------------------------------------------------------
constexpr int kMostGroup = 32;
constexpr int kMostPages = 32768;
constexpr uint32_t kForced = 0xFFFFFFFFu;  // above the key of any score

QDQ_DEV uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
QDQ_DEV uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
QDQ_DEV void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
QDQ_DEV void store_to_rank0(uint32_t addr, uint32_t v) {
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(remote) : "r"(addr));
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(remote), "r"(v) : "memory");
}
// c (16 x 8) += a (16 x 32 signed bytes) x b (32 x 8).
QDQ_DEV void mma_s8(int *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Sums `v` over the CTA's threads before this one; total in every thread. `room`: a word a warp.
template <int kSelectWarps>
QDQ_DEV uint32_t scan(uint32_t v, uint32_t *room, uint32_t &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t e = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += e;
    }
    __syncthreads();
    if (lane == 31) room[warp] = incl;
    __syncthreads();
    uint32_t before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kSelectWarps; ++w) {
        if (w < warp) before += room[w];
        total += room[w];
    }
    return before + incl - v;
}

// A cluster takes a token and kv head. Its CTAs score a share of the pages each, 16 a warp and step, by
// the integer matrix instruction (16 pages x 8 heads x 32 dims; a lane's operands are 16 consecutive bytes
// of a page's bounds, and the query's in the same order: a sum may take its terms in any), and send the
// scores, as integers in their order, to the first CTA's shared memory. That one selects: it narrows the
// range of the k-th largest by a bin a thread at a time, and then writes what lies above it and the first of
// its equals, in order. (The instruction takes 64 clocks, 512 for 16 pages of 128 dims; in fp16, which holds
// the bytes and their sums exactly too, it would be 128, but the widening takes more registers than the
// CTAs that share an SM have: 64 tokens 26 us and not 16.)
// Few items: 512 threads, and the next step's bounds on their way while one is scored. Many: 256 threads
// with no more registers than let three CTAs share an SM.
template <int TYPE, int D, bool FEW>
__global__ void __launch_bounds__(FEW ? 512 : 256, FEW ? 1 : 3) select_kernel(const PagesArgs a) {
    constexpr int kSelectThreads = FEW ? 512 : 256, kSelectWarps = kSelectThreads / 32;
    constexpr int kAtOnce = 16;  // pages of a warp step
    extern __shared__ __align__(16) char smem[];
    uint32_t *keys = reinterpret_cast<uint32_t *>(smem);  // [max_pages], the first CTA's
    __shared__ __align__(16) uint32_t s_q[2][kMostGroup][D == 128 ? 48 : 16];  // max(q, 0) and min(q, 0)
    __shared__ int s_eq[kMostGroup];
    __shared__ uint32_t s_bins[kSelectThreads], s_room[kSelectWarps], s_pick[3];
    __shared__ uint32_t s_range[3][kSelectWarps];
    follow_last_kernel();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = cluster_rank(), size = cluster_size(), item = blockIdx.x / size;
    const int t = item / a.n_kv_heads, head = item - t * a.n_kv_heads, group = a.n_heads / a.n_kv_heads;

    // (loads that do not wait for each other come first)
    constexpr int kEach = D / 32;  // dims of a lane
    float v[kEach];
    auto query = [&](int h) {
        const uint16_t *q = (const uint16_t *)a.q + (int64_t)t * a.q_stride + (int64_t)(head * group + h) * D + lane * kEach;
#pragma unroll
        for (int i = 0; i < kEach; i += 2) {
            const float2 x = Pair<TYPE>::unpack(__ldg(reinterpret_cast<const uint32_t *>(q + i)));
            v[i] = x.x, v[i + 1] = x.y;
        }
    };
    query(min(warp, group - 1));
    const int s = find_seq(a.q_start, a.n_seqs, t);
    int first, count;
    seq_tokens(a.q_start, max(s, 0), a.n_tokens, first, count);
    const int kv = max(a.kv_len[max(s, 0)], 0);
    const bool live = s >= 0 && t >= first && t < first + count;
    const int p = live ? kv - count + (t - first) : -1;
    const int newest = p >= 0 ? p >> a.page_shift : -1, pages = min(newest + 1, a.max_pages);
    const int32_t *table = a.page_table + (int64_t)max(s, 0) * a.max_pages;

    // The first step's bounds are on their way before the queries are looked at.
    constexpr int kLoads = D / 64;  // 16-byte pieces of each bound that a lane reads
    const int g = lane >> 2, c = lane & 3;
    const int stride = size * kSelectWarps * kAtOnce;
    struct Bounds {  // of the lane's rows g and g + 8 of a step
        uint4 b[2][2][kLoads];  // [row][largest, smallest][piece]
        int page[2], e[2];
    } ahead;
    int next[2], j0 = (rank * kSelectWarps + warp) * kAtOnce;
    auto pages_at = [&](int j0) {
#pragma unroll
        for (int y = 0; y < 2; ++y) next[y] = j0 + 8 * y + g < pages ? table[j0 + 8 * y + g] : -1;
    };
    // the step at j0 (its pages are in `next`)
    auto fetch = [&](int j0, Bounds &to) {
        if (j0 < pages) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                to.page[y] = (unsigned)next[y] < (unsigned)a.n_pages ? next[y] : -1;
                const int64_t unit = (int64_t)max(to.page[y], 0) * a.n_kv_heads + head;
                const int8_t *from = a.bounds + unit * 2 * D + 16 * c;
#pragma unroll
                for (int z = 0; z < 2; ++z)
#pragma unroll
                    for (int i = 0; i < kLoads; ++i) to.b[y][z][i] = __ldg(reinterpret_cast<const uint4 *>(from + z * D + 64 * i));
                to.e[y] = a.bound_scales[unit] - 127;
            }
            pages_at(j0 + stride);
        }
    };
    pages_at(j0);
    fetch(j0, ahead);

    // the group's query heads as bytes
    for (int h = warp; h < group; h += kSelectWarps) {
        if (h != warp) query(h);
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < kEach; ++i) top = fmaxf(top, fabsf(v[i]));
        top = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top)));  // (not negative: its bits are in its order)
        const int e = bound_exponent(top);
        const float f0 = power_of_two(-e / 2), f1 = power_of_two(-e - -e / 2);
        uint32_t over = 0, under = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int x = (int)fminf(fmaxf(rintf(v[i] * f0 * f1), -127.0f), 127.0f);
            over |= (uint32_t)(max(x, 0) & 0xFF) << (8 * i);
            under |= (uint32_t)(min(x, 0) & 0xFF) << (8 * i);
        }
        if (kEach == 4) {
            s_q[0][h][lane] = over, s_q[1][h][lane] = under;
        } else {  // two dims a lane
            reinterpret_cast<uint16_t *>(s_q[0][h])[lane] = (uint16_t)over, reinterpret_cast<uint16_t *>(s_q[1][h])[lane] = (uint16_t)under;
        }
        if (lane == 0) s_eq[h] = e;
    }
    cluster_sync();  // (and the first CTA is known to run before anything is sent to it)

    // scores of this CTA's pages
    {
        for (; j0 < pages; j0 += stride) {
            Bounds now = ahead;
            if (FEW) fetch(j0 + stride, ahead);
            const auto &b = now.b;
            const auto &page = now.page;
            const auto &e = now.e;
            float best[2] = {-INFINITY, -INFINITY};
            for (int h0 = 0; h0 < group; h0 += 8) {
                int sum[4] = {};
                const int h = min(h0 + g, group - 1);  // (column g of the product)
#pragma unroll
                for (int z = 0; z < 2; ++z)
#pragma unroll
                    for (int i = 0; i < kLoads; ++i) {
                        const uint4 q = *reinterpret_cast<const uint4 *>(&s_q[z][h][16 * i + 4 * c]);
                        mma_s8(sum, b[0][z][i].x, b[1][z][i].x, b[0][z][i].y, b[1][z][i].y, q.x, q.y);
                        mma_s8(sum, b[0][z][i].z, b[1][z][i].z, b[0][z][i].w, b[1][z][i].w, q.z, q.w);
                    }
#pragma unroll
                for (int x = 0; x < 2; ++x) {  // heads h0 + 2 c and the next
                    const int eq = s_eq[min(h0 + 2 * c + x, group - 1)];
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float v = (float)sum[2 * y + x] * power_of_two(min(max(eq + e[y], -100), 100));
                        best[y] = fmaxf(best[y], v);  // (the last head once more, past the group's end)
                    }
                }
            }
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                best[y] = fmaxf(best[y], __shfl_xor_sync(0xFFFFFFFFu, best[y], 1));
                best[y] = fmaxf(best[y], __shfl_xor_sync(0xFFFFFFFFu, best[y], 2));
                const int j = j0 + 8 * y + g;
                if (c == 0 && j < pages) {
                    const uint32_t bits = __float_as_uint(best[y]);
                    uint32_t key = bits & 0x80000000u ? ~bits : bits | 0x80000000u;  // (finite: neither 0 nor the largest)
                    if (j < a.first || j > newest - a.last) key = kForced;           // always taken
                    if (page[y] < 0) key = 0;                                        // never
                    if (QDQ_CHECK(&g_pages_status, j >= 0 && j < a.max_pages)) store_to_rank0(smem_u32(keys + j), key);
                }
            }
            if (!FEW) fetch(j0 + stride, ahead);
        }
    }
    cluster_sync();
    if (rank != 0 || !live) return;

    // ---- the first CTA selects -------------------------------------------------------------------
    // a thread has a run of consecutive pages (an odd number, which are in other banks than its neighbours')
    const int tid = threadIdx.x, per = ((pages + kSelectThreads - 1) / kSelectThreads) | 1;
    const int i0 = min(tid * per, pages), i1 = min(i0 + per, pages);
    uint32_t valid = 0, forced = 0, own = 0, small = 0xFFFFFFFFu;  // this thread's largest and smallest score
    for (int j = tid; j < pages; j += kSelectThreads) {
        const uint32_t k = keys[j];
        if (k == 0) continue;
        ++valid;
        if (k == kForced) ++forced;
        else own = max(own, k), small = min(small, k);
    }
    uint32_t all;
    scan<kSelectWarps>(valid | forced << 16, s_room, all);
    forced = all >> 16, all &= 0xFFFFu;
    uint32_t threshold = 1, equals = 0xFFFFFFFFu;  // taken: above the threshold, and of its equals the first so many
    if (all > (uint32_t)a.select) {
        // (of the threads' largest scores the smallest, and of all scores)
        const uint32_t low = __reduce_min_sync(0xFFFFFFFFu, own ? own : 0xFFFFFFFFu), top = __reduce_max_sync(0xFFFFFFFFu, own);
        small = __reduce_min_sync(0xFFFFFFFFu, small);
        if (lane == 0) s_range[0][warp] = low, s_range[1][warp] = top, s_range[2][warp] = small;
        const uint32_t some = __syncthreads_count(own != 0);
        uint32_t low_own = 0xFFFFFFFFu, most_key = 0, from = 0xFFFFFFFFu;
#pragma unroll
        for (int w = 0; w < kSelectWarps; ++w)
            low_own = min(low_own, s_range[0][w]), most_key = max(most_key, s_range[1][w]), from = min(from, s_range[2][w]);
        // The want-th largest of the scores lies in from .. from + width. It is no less than the want-th largest
        // of the threads' largest, where there are so many, and with many scores that is looked for first, so
        // that few are left to be counted (8188 scores: 5100 clocks and not 7200).
        uint32_t want = a.select - forced;
        if (want == 0) threshold = kForced;
        bool firsts = some >= want && pages > 4 * kSelectThreads;
        if (firsts) from = low_own;
        uint32_t width = most_key - from;
        while (want) {
            constexpr int kBits = FEW ? 9 : 8;  // of kSelectThreads
            const int bits = 32 - __clz(width), shift = max(bits - kBits, 0);
            s_bins[tid] = 0;
            __syncthreads();
            if (firsts) {
                if (own) atomicAdd(&s_bins[(own - from) >> shift], 1u);
            } else {
                for (int j = tid; j < pages; j += kSelectThreads) {
                    const uint32_t k = keys[j];
                    if (k >= from && k - from <= width) atomicAdd(&s_bins[(k - from) >> shift], 1u);
                }
            }
            __syncthreads();
            // from the top: thread i has bin kSelectThreads - 1 - i
            uint32_t total;
            const uint32_t mine = s_bins[kSelectThreads - 1 - tid], above = scan<kSelectWarps>(mine, s_room, total);
            if (above < want && want <= above + mine) s_pick[0] = kSelectThreads - 1 - tid, s_pick[1] = want - above, s_pick[2] = mine;
            __syncthreads();
            const uint32_t bin = s_pick[0], here = s_pick[2], next_want = s_pick[1];
            __syncthreads();
            if (firsts) {  // (all of what lies above the bin's lower end)
                firsts = false;
                from += bin << shift;
                width = most_key - from;
                continue;
            }
            want = next_want;
            from += bin << shift;
            // (the last bin may reach past the range)
            width = min((1u << shift) - 1, width - (bin << shift));
            if (shift == 0 || here == want) {  // one value, or the whole bin
                threshold = from;
                if (shift == 0) equals = want;
                break;
            }
        }
    }
    const bool exact = equals != 0xFFFFFFFFu;
    uint32_t over = 0, same = 0;
    for (int j = i0; j < i1; ++j) {
        const uint32_t k = keys[j];
        if (exact ? k > threshold : k >= threshold) ++over;
        else if (exact && k == threshold) ++same;
    }
    uint32_t total;
    uint32_t rank_same = scan<kSelectWarps>(same, s_room, total);
    // entries before this thread's: those over, and of the equals the first `equals`
    const uint32_t taken_same = exact ? (rank_same >= equals ? 0 : min(same, equals - rank_same)) : 0;
    uint32_t to = scan<kSelectWarps>(over + taken_same, s_room, total);
    int32_t *out = a.lists + ((int64_t)t * a.n_kv_heads + head) * a.select;
    for (int j = i0; j < i1; ++j) {
        const uint32_t k = keys[j];
        const bool is_same = exact && k == threshold;
        const bool take = is_same ? rank_same < equals : k >= threshold && k != 0;
        rank_same += is_same;
        if (take && to < (uint32_t)a.select) out[to++] = j;
    }
    for (int j = (int)total + tid; j < a.select; j += kSelectThreads) out[j] = -1;
}

using Kernel = void (*)(PagesArgs);
#define QDQ_BY_TYPE(NAME, D) (type == QDQ_E4M3 ? NAME<QDQ_E4M3, D> : type == QDQ_BF16 ? NAME<QDQ_BF16, D> : NAME<QDQ_F16, D>)
template <int D, bool FEW>
Kernel select_of(int type) {
    return type == QDQ_E4M3 ? select_kernel<QDQ_E4M3, D, FEW> : type == QDQ_BF16 ? select_kernel<QDQ_BF16, D, FEW> : select_kernel<QDQ_F16, D, FEW>;
}
Kernel select_of(int type, int head_dim, bool few) {
    if (head_dim == 64) return few ? select_of<64, true>(type) : select_of<64, false>(type);
    return few ? select_of<128, true>(type) : select_of<128, false>(type);
}

}  // namespace

int launch_bounds(PagesArgs a, int type, int head_dim, cudaStream_t stream, int sm_count) {
    // Many tokens are mostly ones that begin no page: a window of them is one CTA's.
    a.window = (int64_t)a.n_tokens * a.n_kv_heads >= (int64_t)sm_count * 64 ? kMostWindow : 1;
    const int64_t grid = ((int64_t)a.n_tokens + a.window - 1) / a.window * a.n_kv_heads;
    if (grid > 0x7FFFFFFF) return QDQ_ERR_LIMIT;
    const Kernel k = head_dim == 64 ? QDQ_BY_TYPE(bounds_kernel, 64) : QDQ_BY_TYPE(bounds_kernel, 128);
    return launch_following(k, (unsigned)grid, 128, 0, 1, stream, a);
}

int launch_select(const PagesArgs &a, int type, int head_dim, cudaStream_t stream, int sm_count) {
    // CTAs of a cluster: as many as the SMs have room for beside the other items, up to 8, with 256 pages
    // each at least.
    const int64_t items = (int64_t)a.n_tokens * a.n_kv_heads;
    unsigned size = 1;
    while (size < 8 && items * size * 2 <= sm_count && a.max_pages >= 256 * (int)size) size *= 2;
    if (items * size > 0x7FFFFFFF) return QDQ_ERR_LIMIT;
    const bool few = items * size <= sm_count;
    return launch_following(select_of(type, head_dim, few), (unsigned)(items * size), few ? 512 : 256, (size_t)a.max_pages * 4, size,
                            stream, a);
}

// The selection's shared memory, for every handle: called where one is created.
int pages_setup() {
    for (int type : {QDQ_F16, QDQ_BF16, QDQ_E4M3})
        for (int dim : {64, 128})
            for (bool few : {false, true})
                if (cudaFuncSetAttribute(select_of(type, dim, few), cudaFuncAttributeMaxDynamicSharedMemorySize, kMostPages * 4) != cudaSuccess) {
                    cudaGetLastError();
                    return QDQ_ERR_CUDA;
                }
    return QDQ_OK;
}

int take_status_pages() {
    int v = 0;
#ifdef QDQ_DEBUG
    const int zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_pages_status, sizeof(int)) != cudaSuccess ||
        (v && cudaMemcpyToSymbol(g_pages_status, &zero, sizeof(int)) != cudaSuccess)) {
        cudaGetLastError();
        return QDQ_ERR_CUDA;
    }
#endif
    return v;
}

}  // namespace qdq
