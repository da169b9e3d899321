// qdq_append8.cu -- the append of a step's new tokens to a cache of e4m3 values: head norms,
// rotation, a scale for each 16 positions and head, and the cache write in one pass.
//
//   e = the least exponent with max |x| <= 448 * 2^e over the block's new rows (and not below the
//   block's own where it holds earlier rows, which are then rescaled), stored = e4m3(x * 2^-e).
// Scales are powers of two, so a value is scaled exactly and rounded once, and a rescaled one is
// rounded again only where it leaves e4m3's normal range.
// Bound by HBM and by its instructions: 259 MB (7436 tokens of 32 + 2 x 8 heads of 128, norms, fp32 in) in
// 51.8 us = 5.0 TB/s, 74 % of the copy rate, half the issue slots used; a token takes 3.8 us.
#include <algorithm>

#include "qdq_internal.h"
#include "qdq_paged.cuh"

namespace qdq {
namespace {

#ifdef QDQ_DEBUG
__device__ int g_append8_status;
#endif

constexpr int kThreads = 256, kMostWindow = 17;
static_assert(kMostWindow + kScaleBlock - 1 <= 32, "a lane a token");
constexpr int kSpan = kMostWindow + kScaleBlock - 1;  // tokens that a window's blocks reach

// Two values as fp16; beyond its range they become its largest, what is no number stays none.
QDQ_DEV uint32_t pack_finite(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// A CTA takes a window of tokens: their q rows, and the keys and values of the blocks that begin
// (or are first written to) there, which may reach past it. A block of one head, keys or values, is
// a pair of warps', eight rows each: D/8 lanes take a row, eight values a lane, as in the 16-bit append
// (qdq_paged.cu), all in registers, so that the scale is known before anything is stored. The angles of the
// window's positions are formed once for all heads, in shared memory.
template <typename TI, int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, 3) append8_kernel(const Append8Args a) {
    constexpr int G = D / 8, RW = 32 / G;            // lanes per row, rows per warp step
    constexpr int kSteps = 8 / RW;                   // of half a block
    constexpr int kBatch = 4;                        // steps of a q task
    __shared__ float2 turn[kSpan * (D / 2)];         // cosine and sine of each token's pairs
    __shared__ int s_pos[kSpan], s_rows[kSpan], s_lead[kMostWindow], s_count;
    __shared__ bool s_live[kSpan], s_turn[kSpan];
    __shared__ float s_top[2][kThreads / 32];
    __shared__ int64_t s_block[kMostWindow];         // (page * heads) and the block's number in it, or -1
    follow_last_kernel();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, u = lane % G, sub = lane / G;
    const int t0 = (int)(blockIdx.x / a.parts) * a.window, part = blockIdx.x % a.parts;
    const int in_window = min(a.window, a.n_tokens - t0), reach = min(a.window + kScaleBlock - 1, a.n_tokens - t0);
    const int page_mask = (1 << a.page_shift) - 1;

    if (warp == 0) {
        int s = find_seq(a.q_start, a.n_seqs, t0);
        const int t = t0 + lane;
        bool live = false, lead = false, turns = false;
        int p = 0, rows = 0;
        int64_t block = -1;
        if (s >= 0 && lane < reach) {
            while (s + 1 < a.n_seqs && a.q_start[s + 1] <= t) ++s;
            int first, count;
            seq_tokens(a.q_start, s, a.n_tokens, first, count);
            live = t >= first && t < first + count;
            if (live) {
                p = max(a.kv_len[s], 0) - count + (t - first);
                const int in_block = p & (kScaleBlock - 1), head = max(t - in_block, first);  // the block's first new token
                lead = lane < a.window && p >= 0 && head == t;
                // (its angles: for its q row, or for its key where its block begins in the window)
                turns = p >= 0 && (lane < a.window || (p >= 0 && head < t0 + a.window));
                if (lead) {
                    rows = min(kScaleBlock - in_block, first + count - t);
                    if ((p >> a.page_shift) < a.max_pages) {
                        const int page = a.page_table[(int64_t)s * a.max_pages + (p >> a.page_shift)];
                        if (page >= 0 && page < a.n_pages) block = ((int64_t)page << 32) | (p & page_mask);
                    }
                }
            }
        }
        if (lane < kSpan) s_live[lane] = live, s_turn[lane] = turns, s_pos[lane] = p, s_rows[lane] = rows;
        const unsigned leads = __ballot_sync(0xFFFFFFFFu, lead && block >= 0);
        if (lead && block >= 0) {
            const int at = __popc(leads & ((1u << lane) - 1));
            s_lead[at] = lane;
            s_block[at] = block;
        }
        if (lane == 0) s_count = __popc(leads);
    }
    __syncthreads();
    const int pairs = a.rope_dim / 2;
    for (int x = threadIdx.x; x < reach * pairs; x += kThreads) {
        const int i = x / pairs, pair = x - i * pairs;
        if (!s_turn[i]) continue;
        // (the fraction of a turn: qdq_paged.cu)
        const int32_t frac = (int32_t)(uint32_t)((a.freq[pair] * (uint64_t)(uint32_t)s_pos[i]) >> 32);
        float2 cs;
        sincospif((float)frac * 0x1p-31f, &cs.y, &cs.x);
        turn[i * (D / 2) + pair] = cs;
    }
    __syncthreads();

    const bool turns = 8 * u < a.rope_dim;
    const int c0 = !INTERLEAVED && turns ? 4 * u : 8 * u;
    const int c1 = !INTERLEAVED && turns ? a.rope_dim / 2 + 4 * u : 8 * u + 4;
    auto norm = [&](float *v, const float *w) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
#pragma unroll
        for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        const float inv = rsqrtf(ss * (1.0f / D) + a.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] * inv * w[i];
    };
    auto rotate = [&](float *v, int token) {
        if (!turns) return;
        const float4 *at = reinterpret_cast<const float4 *>(turn + token * (D / 2) + 4 * u);
        const float4 x = at[0], y = at[1];
        const float cs[4] = {x.x, x.z, y.x, y.z}, sn[4] = {x.y, x.w, y.y, y.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = INTERLEAVED ? 2 * i : i, o = INTERLEAVED ? 2 * i + 1 : i + 4;
            const float xe = v[e], xo = v[o];
            v[e] = xe * cs[i] - xo * sn[i];
            v[o] = xe * sn[i] + xo * cs[i];
        }
    };
    auto weights = [&](const float *w, float *to) {
#pragma unroll
        for (int i = 0; i < 8; ++i) to[i] = w ? w[i < 4 ? c0 + i : c1 + i - 4] : 1.0f;
    };

    const int kv_tasks = s_count * 2 * a.n_kv_heads, per_token = (a.n_heads + kBatch * RW - 1) / (kBatch * RW);
    const int tasks = kv_tasks + in_window * per_token;
    const int pair = warp >> 1, half = warp & 1;
    int turn_no = 0;
    for (int task = pair * a.parts + part; task < kv_tasks; task += (kThreads / 64) * a.parts) {
        // ---- a block of keys or values of one head ----------------------------------------------
        const int at = task / (2 * a.n_kv_heads), which = task - at * 2 * a.n_kv_heads;
        const bool is_k = which < a.n_kv_heads;
        const int head = is_k ? which : which - a.n_kv_heads, token = s_lead[at], rows = s_rows[token];
        if (rows <= 8 && half) continue;  // (the first warp's alone)
        const int64_t block = s_block[at];
        const int page = (int)(block >> 32), in_page = (int)block, row0 = in_page & (kScaleBlock - 1);
        const int64_t unit = (int64_t)page * a.n_kv_heads + head;  // a page's rows of the head
        uint8_t *scale = (is_k ? a.k_scales : a.v_scales) + (unit << (a.page_shift - 4)) + (in_page >> 4);
        uint8_t *code = (is_k ? a.k_pages : a.v_pages) + ((unit << a.page_shift) + in_page) * D;
        const TI *src = (is_k ? (const TI *)a.k + (int64_t)(t0 + token) * a.k_stride : (const TI *)a.v + (int64_t)(t0 + token) * a.v_stride) + head * D;
        const int64_t stride = is_k ? a.k_stride : a.v_stride;
        float x[kSteps][8];
#pragma unroll
        for (int y = 0; y < kSteps; ++y) {
            const int i = 8 * half + y * RW + sub;
#pragma unroll
            for (int z = 0; z < 8; ++z) x[y][z] = 0.0f;
            if (i < rows && QDQ_CHECK(&g_append8_status, t0 + token + i < a.n_tokens && page < a.n_pages && row0 + i < kScaleBlock)) {
                load4(src + i * stride + c0, x[y]);
                load4(src + i * stride + c1, x[y] + 4);
            }
        }
        const int before = row0 ? exponent_of(*scale) : -kMostExponent;
        float w[8], top = 0.0f;
        if (is_k && a.k_norm) weights(a.k_norm, w);
#pragma unroll
        for (int y = 0; y < kSteps; ++y) {
            if (8 * half + y * RW >= rows) break;
            if (is_k) {
                if (a.k_norm) norm(x[y], w);
                rotate(x[y], token + min(8 * half + y * RW + sub, rows - 1));
            }
            if (8 * half + y * RW + sub < rows) {
#pragma unroll
                for (int z = 0; z < 8; ++z) top = fmaxf(top, fabsf(x[y][z]));
            }
        }
        if (__any_sync(0xFFFFFFFFu, top == INFINITY)) {  // (seldom: the largest of the finite ones)
            top = 0.0f;
#pragma unroll
            for (int y = 0; y < kSteps; ++y)
#pragma unroll
                for (int z = 0; z < 8; ++z) top = fmaxf(top, 8 * half + y * RW + sub < rows && isfinite(x[y][z]) ? fabsf(x[y][z]) : 0.0f);
        }
        top = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top)));  // (not negative: its bits are in its order)
        if (rows > 8) {
            if (lane == 0) s_top[turn_no][warp] = top;
            named_bar_sync(1 + pair, 64);
            top = fmaxf(top, s_top[turn_no][warp ^ 1]);
            turn_no ^= 1;  // (the other warp may still read this place)
        }
        const int e = max(least_exponent(top), before);
        const float f = power_of_two(-e);
#pragma unroll
        for (int y = 0; y < kSteps; ++y) {
            const int i = 8 * half + y * RW + sub;
            if (i >= rows) continue;
            const float *v = x[y];
            const uint32_t lo = f32_to_e4m3x4(v[0] * f, v[1] * f, v[2] * f, v[3] * f);
            const uint32_t hi = f32_to_e4m3x4(v[4] * f, v[5] * f, v[6] * f, v[7] * f);
            uint8_t *to = code + i * D;
            if (INTERLEAVED) {
                *reinterpret_cast<uint2 *>(to + c0) = make_uint2(lo, hi);
            } else {
                *reinterpret_cast<uint32_t *>(to + c0) = lo;
                *reinterpret_cast<uint32_t *>(to + c1) = hi;
            }
        }
        if (row0 && e > before && half == 0) {  // the block's earlier rows come to the new scale
            const float g = power_of_two(before - e);
            for (int i = sub; i < row0; i += RW) {
                uint2 *at8 = reinterpret_cast<uint2 *>(code + (i - row0) * D + 8 * u);
                const uint2 old = *at8;
                auto rescaled = [&](uint32_t v) {
                    uint32_t lo, hi;
                    e4m3x4_to_f16(v, lo, hi);
                    const float2 p = Float16<__half>::unpack(lo), q = Float16<__half>::unpack(hi);
                    return f32_to_e4m3x4(p.x * g, p.y * g, q.x * g, q.y * g);
                };
                *at8 = make_uint2(rescaled(old.x), rescaled(old.y));
            }
        }
        // (both warps have read the old scale)
        if (lane == 0 && half == 0) *scale = (uint8_t)(e + 127);
    }
    for (int task = kv_tasks + warp * a.parts + part; task < tasks; task += (kThreads / 32) * a.parts) {
        // ---- kBatch steps of a token's q rows ---------------------------------------------------
        const int at = task - kv_tasks, token = at / per_token, r0 = (at - token * per_token) * kBatch * RW;
        if (!s_live[token]) continue;
        const TI *src = (const TI *)a.q + (int64_t)(t0 + token) * a.q_stride;
        __half *to = (__half *)a.q_out + (int64_t)(t0 + token) * a.n_heads * D;
        float x[kBatch][8], w[8];
#pragma unroll
        for (int y = 0; y < kBatch; ++y) {
            const int r = min(r0 + y * RW + sub, a.n_heads - 1);
            load4(src + r * D + c0, x[y]);
            load4(src + r * D + c1, x[y] + 4);
        }
        if (a.q_norm) weights(a.q_norm, w);
        const bool none = s_pos[token] < 0;
#pragma unroll
        for (int y = 0; y < kBatch; ++y) {
            const int r = r0 + y * RW + sub;
            float *v = x[y];
            if (a.q_norm) norm(v, w);
            if (!none) rotate(v, token);
#pragma unroll
            for (int z = 0; z < 8; ++z) v[z] = none ? 0.0f : v[z];
            if (r >= a.n_heads) continue;
            const uint2 lo = make_uint2(pack_finite(v[0], v[1]), pack_finite(v[2], v[3]));
            const uint2 hi = make_uint2(pack_finite(v[4], v[5]), pack_finite(v[6], v[7]));
            if (INTERLEAVED) {
                *reinterpret_cast<uint4 *>(to + r * D + c0) = make_uint4(lo.x, lo.y, hi.x, hi.y);
            } else {
                *reinterpret_cast<uint2 *>(to + r * D + c0) = lo;
                *reinterpret_cast<uint2 *>(to + r * D + c1) = hi;
            }
        }
    }
}

template <typename TI, int D>
int launch_typed(const Append8Args &a, bool interleaved, unsigned grid, cudaStream_t stream) {
    return launch_following(interleaved ? append8_kernel<TI, D, true> : append8_kernel<TI, D, false>, grid, kThreads, 0, 1,
                            stream, a);
}

}  // namespace

int launch_append8(Append8Args a, int in_type, bool interleaved, int head_dim, cudaStream_t stream, int sm_count) {
    // Many tokens: the window that ends soonest, at three CTAs an SM in turn and three tokens' time for each CTA's
    // start (7436 tokens: 17 of them, one wave; at 16 a second one of nine CTAs, 64.7 and not 51.8 us).
    const int warps = kThreads / 32, slots = 3 * sm_count;
    a.window = 1;
    if (a.n_tokens >= 2048) {
        int64_t least = INT64_MAX;
        for (int w = 8; w <= kMostWindow; ++w) {
            const int64_t time = (((int64_t)a.n_tokens + w - 1) / w + slots - 1) / slots * (w + 3);
            if (time <= least) least = time, a.window = w;
        }
    }
    const int64_t windows = ((int64_t)a.n_tokens + a.window - 1) / a.window;
    const int rw = 256 / head_dim;
    // with few tokens their rows are shared by CTAs, until about 16 warps per SM have work
    const int tasks = a.window == 1 ? 2 * a.n_kv_heads + (a.n_heads + 4 * rw - 1) / (4 * rw) : 16 * warps;
    const int64_t want = std::max<int64_t>(1, ((int64_t)sm_count * 2 + windows - 1) / windows);
    a.parts = a.window > 1 ? 1 : (int)std::min<int64_t>(want, (tasks + warps - 1) / warps);
    const int64_t grid = windows * a.parts;
    if (grid > 0x7FFFFFFF) return QDQ_ERR_LIMIT;
    const unsigned g = (unsigned)grid;
#define QDQ_APPEND8(TI) (head_dim == 64 ? launch_typed<TI, 64>(a, interleaved, g, stream) : launch_typed<TI, 128>(a, interleaved, g, stream))
    if (in_type == QDQ_F32) return QDQ_APPEND8(float);
    return in_type == QDQ_BF16 ? QDQ_APPEND8(__nv_bfloat16) : QDQ_APPEND8(__half);
#undef QDQ_APPEND8
}

int take_status_append8() {
    int v = 0;
#ifdef QDQ_DEBUG
    const int zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_append8_status, sizeof(int)) != cudaSuccess ||
        (v && cudaMemcpyToSymbol(g_append8_status, &zero, sizeof(int)) != cudaSuccess)) {
        cudaGetLastError();
        return QDQ_ERR_CUDA;
    }
#endif
    return v;
}

}  // namespace qdq
