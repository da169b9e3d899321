// qdq_sample.cu -- sampling: temperature, top-k, top-p and min-p from given random
// numbers.
//
// The filters are cuts of one order (logit descending, index ascending), so no sort
// is needed: a radix select over the logits' order-preserving 32-bit keys, eight bits
// a round, finds the key at which top-k's count or top-p's mass is reached, and how
// many of the entries with exactly that key are kept. Masses are 64-bit integers
// (weights in units of 2^-44 of the largest), so the histograms' atomic additions
// give the same sums in any order. The draw is then an inverse CDF in index order:
// kept mass per segment of the row, the segment that crosses u times the whole, and
// the entry inside it.
#include <cmath>

#include "qdq_internal.h"
#include "qdq_paged.cuh"

namespace qdq {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr unsigned kAll = 0xFFFFFFFFu;

struct SampleArgs {
    const void *logits;
    int64_t stride;
    int rows, vocab;
    const float *temperature, *top_p, *min_p, *u;
    const int32_t *top_k;
    int64_t *tokens;
    float *logprobs;
};

// NaN -> -inf, -0 -> +0 (equal logits must have equal keys).
template <typename T>
QDQ_DEV float logit(const T *row, int i) {
    const float x = (float)row[i];
    return x == x ? x + 0.0f : -INFINITY;
}
QDQ_DEV uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x);
    return b ^ (b & 0x80000000u ? 0xFFFFFFFFu : 0x80000000u);
}
QDQ_DEV float value_of(uint32_t k) { return __uint_as_float(k ^ (k & 0x80000000u ? 0x80000000u : 0xFFFFFFFFu)); }
QDQ_DEV float weight(float x, float top, float inv) {
    return x == top ? 1.0f : x == -INFINITY ? 0.0f : expf((x - top) * inv);
}
QDQ_DEV uint64_t fixed(float w) { return __float2ull_rn(w * 0x1p44f); }

struct Shared {
    unsigned count[256];
    unsigned long long mass[256];
    unsigned long long warp_mass[kWarps];
    unsigned warp_count[kWarps];
    uint32_t key;
    unsigned above_count;
    unsigned long long above_mass;
    int found;
};

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleArgs a) {
    __shared__ Shared sh;
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, V = a.vocab;
    const T *row = (const T *)a.logits + (int64_t)b * a.stride;
    const float temp = a.temperature ? a.temperature[b] : 1.0f;
    const bool greedy = !(temp > 0.0f);
    const float inv = greedy ? 1.0f : 1.0f / temp;

    // the largest key, and the lowest index that has it
    unsigned long long best = 0;
    for (int i = tid; i < V; i += kThreads) {
        const unsigned long long e = ((unsigned long long)key_of(logit(row, i)) << 32) | (0xFFFFFFFFu - (unsigned)i);
        best = e > best ? e : best;
    }
    for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long e = __shfl_xor_sync(kAll, best, o);
        best = e > best ? e : best;
    }
    if (lane == 0) sh.warp_mass[warp] = best;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) best = sh.warp_mass[w] > best ? sh.warp_mass[w] : best;
    __syncthreads();
    const float top = value_of((uint32_t)(best >> 32));
    if (V == 0 || top == -INFINITY || greedy) {
        if (tid == 0) {
            const bool none = V == 0 || top == -INFINITY;
            a.tokens[b] = none ? -1 : (int64_t)(0xFFFFFFFFu - (unsigned)best);
            if (a.logprobs) a.logprobs[b] = none ? -INFINITY : 0.0f;
        }
        return;
    }

    // the cut: entries with key > cut are kept, and the first `ties` with key == cut
    uint32_t cut = key_of(-INFINITY);
    unsigned ties = 0;
    unsigned long long total = 0;  // mass of top-k's entries
    // One select: by count (k > 0) or by mass (reach `target`).
    auto select = [&](bool by_mass, unsigned k, double target) {
        uint32_t prefix = 0, mask = 0;
        unsigned above_c = 0;
        unsigned long long above_m = 0;
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256; i += kThreads) sh.count[i] = 0, sh.mass[i] = 0;
            __syncthreads();
            for (int i = tid; i < V; i += kThreads) {
                const float x = logit(row, i);
                const uint32_t key = key_of(x);
                if (x == -INFINITY || (key & mask) != prefix) continue;
                atomicAdd(&sh.count[(key >> shift) & 255], 1u);
                atomicAdd(&sh.mass[(key >> shift) & 255], (unsigned long long)fixed(weight(x, top, inv)));
            }
            __syncthreads();
            if (tid == 0) {
                int d = 255;
                for (; d > 0; --d) {
                    const unsigned c = above_c + sh.count[d];
                    const unsigned long long m = above_m + sh.mass[d];
                    if (by_mass ? (double)m >= target : c >= k) break;
                    above_c = c, above_m = m;
                }
                sh.key = prefix | ((uint32_t)d << shift);
                sh.above_count = above_c;
                sh.above_mass = above_m;
            }
            __syncthreads();
            prefix = sh.key;
            above_c = sh.above_count;
            above_m = sh.above_mass;
            mask |= 255u << shift;
        }
        const unsigned here = sh.count[prefix & 255];
        const uint64_t f = fixed(weight(value_of(prefix), top, inv));
        unsigned n;
        if (by_mass) {
            n = 1;
            while (n < here && (double)(above_m + n * f) < target) ++n;
            if (prefix == cut && ties) n = min(n, ties);
        } else {
            n = min(k - above_c, here);
        }
        cut = prefix;
        ties = n;
        total = above_m + n * f;
        __syncthreads();
    };

    auto sum_all = [&](unsigned long long v) {
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
        if (lane == 0) sh.warp_mass[warp] = v;
        __syncthreads();
        v = 0;
        for (int w = 0; w < kWarps; ++w) v += sh.warp_mass[w];
        __syncthreads();
        return v;
    };

    const int k = a.top_k ? a.top_k[b] : 0;
    const float p = a.top_p ? a.top_p[b] : 1.0f;
    const float floor_w = a.min_p ? fminf(a.min_p[b], 1.0f) : 0.0f;
    if (k > 0 && k < V) {
        unsigned long long live = 0;
        for (int i = tid; i < V; i += kThreads) live += logit(row, i) != -INFINITY;
        if ((unsigned long long)k < sum_all(live)) select(false, (unsigned)k, 0.0);
    }
    if (p < 1.0f) {
        if (ties == 0) {
            unsigned long long m = 0;
            for (int i = tid; i < V; i += kThreads) m += fixed(weight(logit(row, i), top, inv));
            total = sum_all(m);
        }
        // (at least one unit, so that the first entry is kept whatever top_p is)
        select(true, 0, fmax((double)p * (double)total, 1.0));
    }

    // kept mass of each warp's segment of the row, in index order
    const int per = (V + kWarps - 1) / kWarps, i0 = min(warp * per, V), i1 = min(i0 + per, V);
    unsigned before = 0;  // ties ahead of this warp's segment
    if (ties) {
        unsigned n = 0;
        for (int i = i0 + lane; i < i1; i += 32) n += key_of(logit(row, i)) == cut;
        n = __reduce_add_sync(kAll, n);
        if (lane == 0) sh.warp_count[warp] = n;
        __syncthreads();
        for (int w = 0; w < warp; ++w) before += sh.warp_count[w];
    }
    // the kept weight of entry i (the whole warp takes 32 entries at once)
    auto kept = [&](int i, unsigned &seen, float &w) {
        const float x = i < i1 ? logit(row, i) : -INFINITY;
        const uint32_t key = key_of(x);
        bool keep = x != -INFINITY && key > cut;
        if (ties) {
            const unsigned m = __ballot_sync(kAll, i < i1 && key == cut);
            keep = keep || (i < i1 && key == cut && seen + __popc(m & ((1u << lane) - 1)) < ties);
            seen += __popc(m);
        }
        w = weight(x, top, inv);
        return keep && w >= floor_w ? fixed(w) : 0ull;
    };
    unsigned seen = before;
    unsigned long long m = 0;
    float w;
    for (int i = i0; i < i1; i += 32) m += kept(i + lane, seen, w);
    for (int o = 16; o > 0; o >>= 1) m += __shfl_xor_sync(kAll, m, o);
    if (lane == 0) sh.warp_mass[warp] = m;
    if (tid == 0) sh.found = 0;
    __syncthreads();
    unsigned long long ahead = 0, whole = 0;
    int last = 0;
    for (int v = 0; v < kWarps; ++v) {
        if (v < warp) ahead += sh.warp_mass[v];
        whole += sh.warp_mass[v];
        if (sh.warp_mass[v]) last = v;
    }
    const double target = (double)a.u[b] * (double)whole;
    const bool mine = (double)ahead <= target && (double)(ahead + m) > target;
    if (mine || ((double)whole <= target && warp == last)) {
        seen = before;
        unsigned long long sum = ahead;
        int token = -1;
        float tw = 0.0f;
        for (int i = i0; i < i1; i += 32) {
            unsigned long long f = kept(i + lane, seen, w), incl = f;
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned long long e = __shfl_up_sync(kAll, incl, o);
                if (lane >= o) incl += e;
            }
            const unsigned hit = __ballot_sync(kAll, f && (!mine || (double)(sum + incl) > target));
            if (hit) {
                const int l = mine ? __ffs(hit) - 1 : 31 - __clz(hit);
                token = i + l;
                tw = __shfl_sync(kAll, w, l);
                if (mine) break;
            }
            sum += __shfl_sync(kAll, incl, 31);
        }
        if (lane == 0) {
            a.tokens[b] = token;
            if (a.logprobs) a.logprobs[b] = (float)log((double)tw / ((double)whole * 0x1p-44));
        }
    }
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
    const SampleArgs a = {logits, stride, rows, vocab, temperature, top_p, min_p, u, top_k, tokens, logprobs};
    cudaStream_t s = (cudaStream_t)stream;
    if (type == QDQ_F32) sample_kernel<float><<<rows, kThreads, 0, s>>>(a);
    else if (type == QDQ_F16) sample_kernel<__half><<<rows, kThreads, 0, s>>>(a);
    else sample_kernel<__nv_bfloat16><<<rows, kThreads, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? QDQ_OK : QDQ_ERR_CUDA;
}
