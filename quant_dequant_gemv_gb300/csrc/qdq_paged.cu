// qdq_paged.cu -- the paged key/value cache: the handle, its argument checks, and
// the append of a step's new tokens (head norms, rotation and the cache write in
// one pass). The attention over the cache is in qdq_attend.cu.
#include <cmath>
#include <cstring>
#include <new>

#include "qdq_internal.h"
#include "qdq_paged.cuh"

namespace qdq {
namespace {

#ifdef QDQ_DEBUG
__device__ int g_append_status;
#endif

struct AppendArgs {
    int n_seqs, n_tokens, max_pages;
    const int32_t *q_start, *kv_len, *page_table;
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;  // elements
    const float *q_norm, *k_norm;
    const uint64_t *freq;  // turns per position of pair i, in units of 2^-64
    void *q_out, *k_pages, *v_pages;
    float eps;
    int n_heads, n_kv_heads, rope_dim, n_pages, page_shift, rows_per_warp, splits;
};

// A group of D/8 lanes takes one head row, eight values a lane. A lane's values are
// whole rotation pairs: in the interleaved layout eight consecutive values, in the
// split layout four from each half of the turning dims (lanes past the turning dims
// hold eight consecutive values either way), so the rotation needs no exchange
// between lanes, the norm's sum is log2(D/8) shuffles, and every load and store is a
// vector. A warp takes `rows_per_warp` of one token's n_heads + 2 n_kv_heads rows: a
// lane sits at the same place of every row, so the angles are formed once per warp.
// Angles: position * frequency in turns, modulo one turn, is a 64-bit integer product
// that wraps (the frequency is kept in units of 2^-64 turn), so the reduction is exact; the
// frequency itself comes from doubles and is off by at most 2^-54 turn (2^-55.1 found over
// bases 2 to 8e6), which up to position 2^28 is less than the fraction's own rounding to
// fp32. The fraction then goes through sincospi.
// Bound by HBM: 274 MB (7436 tokens of 32 + 2 x 8 heads of 128, fp32 in, bf16 out) in
// 51 us = 5.38 TB/s, 79 % of the copy rate with issue slots half used; a few tokens take 2.7 us,
// which is the launch and three dependent loads.
template <typename TI, typename TC, int D, bool INTERLEAVED>
__global__ void __launch_bounds__(128) append_kernel(const AppendArgs a) {
    constexpr int G = D / 8, RW = 32 / G;  // lanes per row, rows per warp step
    follow_last_kernel();
    const int lane = threadIdx.x & 31, u = lane % G, sub = lane / G;
    const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int t = (int)(unit / a.splits);
    if (t >= a.n_tokens) return;
    const int rows = a.n_heads + 2 * a.n_kv_heads;
    const int r0 = (int)(unit % a.splits) * a.rows_per_warp, r1 = min(r0 + a.rows_per_warp, rows);

    const bool turns = 8 * u < a.rope_dim;
    // the lane's first four and last four values
    const int c0 = !INTERLEAVED && turns ? 4 * u : 8 * u;
    const int c1 = !INTERLEAVED && turns ? a.rope_dim / 2 + 4 * u : 8 * u + 4;
    // Four steps' rows are loaded before the first is worked on, the first four before the
    // token's place is looked up (three loads that wait for each other).
    constexpr int kBatch = 4;
    float x[kBatch][8];
    auto load = [&](int rb) {
#pragma unroll
        for (int y = 0; y < kBatch; ++y) {
            const int r = min(rb + y * RW + sub, rows - 1);
            const bool is_q = r < a.n_heads, is_k = !is_q && r < a.n_heads + a.n_kv_heads;
            const TI *src = is_q   ? (const TI *)a.q + (int64_t)t * a.q_stride + r * D
                            : is_k ? (const TI *)a.k + (int64_t)t * a.k_stride + (r - a.n_heads) * D
                                   : (const TI *)a.v + (int64_t)t * a.v_stride + (r - a.n_heads - a.n_kv_heads) * D;
            if (rb + y * RW < r1 && QDQ_CHECK(&g_append_status, t < a.n_tokens && r >= 0 && r < rows && c0 + 4 <= D && c1 + 4 <= D &&
                                                                    ((uintptr_t)(src + c0) | (uintptr_t)(src + c1)) % (4 * sizeof(TI)) == 0)) {  // (the whole warp)
                load4(src + c0, x[y]);
                load4(src + c1, x[y] + 4);
            }
        }
    };
    load(r0);

    const int s = find_seq(a.q_start, a.n_seqs, t);
    if (s < 0) return;
    int first, count;
    seq_tokens(a.q_start, s, a.n_tokens, first, count);
    if (t < first || t >= first + count) return;  // a row of no sequence
    const int p = max(a.kv_len[s], 0) - count + (t - first);
    int64_t slot = -1;
    if (p >= 0 && (p >> a.page_shift) < a.max_pages) {
        const int page = a.page_table[(int64_t)s * a.max_pages + (p >> a.page_shift)];
        if (page >= 0 && page < a.n_pages) slot = ((int64_t)page << a.page_shift) + (p & ((1 << a.page_shift) - 1));
    }

    float cs[4], sn[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        cs[i] = 1.0f, sn[i] = 0.0f;
        if (turns) {
            const int32_t frac = (int32_t)(uint32_t)((a.freq[4 * u + i] * (uint64_t)(uint32_t)p) >> 32);
            sincospif((float)frac * 0x1p-31f, &sn[i], &cs[i]);
        }
    }
    float wq[8], wk[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int c = i < 4 ? c0 + i : c1 + i - 4;
        wq[i] = a.q_norm ? a.q_norm[c] : 1.0f;
        wk[i] = a.k_norm ? a.k_norm[c] : 1.0f;
    }

    for (int rb = r0; rb < r1; rb += kBatch * RW) {
        if (rb > r0) load(rb);
#pragma unroll
        for (int y = 0; y < kBatch; ++y) {
            if (rb + y * RW >= r1) break;
            const int r = rb + y * RW + sub;
            const bool is_q = r < a.n_heads, is_k = !is_q && r < a.n_heads + a.n_kv_heads;
            float *v = x[y];
            if (a.q_norm || a.k_norm) {
                float ss = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
#pragma unroll
                for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
                const float inv = rsqrtf(ss * (1.0f / D) + a.eps);
                const bool normed = (is_q && a.q_norm) || (is_k && a.k_norm);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = normed ? v[i] * inv * (is_q ? wq[i] : wk[i]) : v[i];
            }
            if (is_q || is_k) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int e = INTERLEAVED ? 2 * i : i, o = INTERLEAVED ? 2 * i + 1 : i + 4;
                    const float xe = v[e], xo = v[o];
                    v[e] = xe * cs[i] - xo * sn[i];
                    v[o] = xe * sn[i] + xo * cs[i];
                }
                if (p < 0) {  // only q rows are written then
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
                }
            }
            if (r >= r1 || (!is_q && slot < 0)) continue;
            TC *dst = is_q   ? (TC *)a.q_out + ((int64_t)t * a.n_heads + r) * D
                      : is_k ? (TC *)a.k_pages + (slot * a.n_kv_heads + r - a.n_heads) * D
                             : (TC *)a.v_pages + (slot * a.n_kv_heads + r - a.n_heads - a.n_kv_heads) * D;
            if (!QDQ_CHECK(&g_append_status, (is_q || (slot >> a.page_shift) < a.n_pages) && r < rows &&
                                                 (uintptr_t)(dst + c0) % (INTERLEAVED ? 16 : 8) == 0 && (uintptr_t)(dst + c1) % 8 == 0))
                continue;
            // (v's values were loaded from the same two places and are only rounded)
            const uint2 lo2 = make_uint2(Float16<TC>::pack(v[0], v[1]), Float16<TC>::pack(v[2], v[3]));
            const uint2 hi2 = make_uint2(Float16<TC>::pack(v[4], v[5]), Float16<TC>::pack(v[6], v[7]));
            if (INTERLEAVED) {
                *reinterpret_cast<uint4 *>(dst + c0) = make_uint4(lo2.x, lo2.y, hi2.x, hi2.y);
            } else {
                *reinterpret_cast<uint2 *>(dst + c0) = lo2;
                *reinterpret_cast<uint2 *>(dst + c1) = hi2;
            }
        }
    }
}

template <typename TI, typename TC, int D>
int launch_append_typed(const AppendArgs &a, bool interleaved, unsigned grid, cudaStream_t stream) {
    return launch_following(interleaved ? append_kernel<TI, TC, D, true> : append_kernel<TI, TC, D, false>, grid, 128, 0,
                            1, stream, a);
}

int launch_append(AppendArgs a, bool in_f32, bool bf16, bool interleaved, int head_dim, cudaStream_t stream,
                  int sm_count) {
    // A warp takes up to 12 steps of a token's rows (7436 tokens of 32 + 2 x 8 heads of 128, launches
    // that wait for each other: 53.2 us, against 55.1 at 8, 60.6 at 4 and 55.3 with whole tokens,
    // whose last wave of warps is ragged; 51 us with launches that follow one another); with few
    // tokens fewer, down to one, until about 16 warps per SM have work.
    const int rows = a.n_heads + 2 * a.n_kv_heads, rw = 256 / head_dim;
    const int steps = (rows + rw - 1) / rw;
    const int64_t want = ((int64_t)sm_count * 16 + a.n_tokens - 1) / a.n_tokens;
    const int least = (steps + 11) / 12;
    const int splits = want < least ? least : want > steps ? steps : (int)want;
    a.rows_per_warp = (steps + splits - 1) / splits * rw;
    a.splits = (rows + a.rows_per_warp - 1) / a.rows_per_warp;
    const int64_t grid = ((int64_t)a.n_tokens * a.splits + 3) / 4;
    if (grid > 0x7FFFFFFF) return QDQ_ERR_LIMIT;
    const unsigned g = (unsigned)grid;
#define QDQ_APPEND(TI, TC)                                                          \
    (head_dim == 64 ? launch_append_typed<TI, TC, 64>(a, interleaved, g, stream)    \
                    : launch_append_typed<TI, TC, 128>(a, interleaved, g, stream))
    if (in_f32) return bf16 ? QDQ_APPEND(float, __nv_bfloat16) : QDQ_APPEND(float, __half);
    return bf16 ? QDQ_APPEND(__nv_bfloat16, __nv_bfloat16) : QDQ_APPEND(__half, __half);
#undef QDQ_APPEND
}

}  // namespace

int take_status_append() {
    int v = 0;
#ifdef QDQ_DEBUG
    const int zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_append_status, sizeof(int)) != cudaSuccess ||
        (v && cudaMemcpyToSymbol(g_append_status, &zero, sizeof(int)) != cudaSuccess)) {
        cudaGetLastError();
        return QDQ_ERR_CUDA;
    }
#endif
    return v;
}

}  // namespace qdq

using namespace qdq;

struct qdq_paged {
    qdq_paged_config cfg{};
    int device = -1, sm_count = 0;
    char *k_pages = nullptr, *v_pages = nullptr;
    int64_t layer_bytes = 0;
    uint64_t *freq = nullptr;  // [rope_dim / 2]
    AttendPools pools{};
    AttendState *attend = nullptr;
};

namespace {

int check_paged_config(const qdq_paged_config *c) {
    if (c->type != QDQ_F16 && c->type != QDQ_BF16) return QDQ_ERR_TYPE;
    if (c->n_layers < 1 || c->n_pages < 1 || c->n_heads < 1 || c->n_kv_heads < 1) return QDQ_ERR_SHAPE;
    if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1))) return QDQ_ERR_SHAPE;
    if (c->head_dim != 64 && c->head_dim != 128) return QDQ_ERR_SHAPE;
    if (c->n_heads % c->n_kv_heads || c->n_heads / c->n_kv_heads > 32) return QDQ_ERR_SHAPE;
    if (c->rope_dim < 0 || c->rope_dim > c->head_dim || c->rope_dim % 8) return QDQ_ERR_SHAPE;
    if (c->rope_interleaved != 0 && c->rope_interleaved != 1) return QDQ_ERR_SHAPE;
    if (c->rope_dim && !(c->rope_base > 1.0f && std::isfinite(c->rope_base))) return QDQ_ERR_SHAPE;
    // (rows of the whole pool are numbered in groups of 8 by 32-bit coordinates)
    if (c->n_kv_heads > 1024 || (int64_t)c->n_pages * c->page_size > ((int64_t)1 << 30) ||
        (int64_t)c->n_pages * c->page_size > ((int64_t)1 << 33) / c->n_layers)
        return QDQ_ERR_LIMIT;
    return QDQ_OK;
}

// The checks that append and attention share; *work is false when nothing is to do.
int check_paged_call(const qdq_paged *c, int layer, const qdq_paged_batch *b, bool *work) {
    *work = false;
    if (c == nullptr || b == nullptr) return QDQ_ERR_PTR;
    if (layer < 0 || layer >= c->cfg.n_layers || b->n_seqs < 0 || b->n_tokens < 0 || b->max_pages < 0)
        return QDQ_ERR_SHAPE;
    if (b->n_seqs > kMaxSeqs || (int64_t)b->max_pages * c->cfg.page_size > ((int64_t)1 << 30)) return QDQ_ERR_LIMIT;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev != c->device) return QDQ_ERR_DEVICE;
    if (b->n_seqs == 0 || b->n_tokens == 0) return QDQ_OK;
    int rc = check_dev_ptr(b->q_start, dev, 4);
    if (!rc) rc = check_dev_ptr(b->kv_len, dev, 4);
    if (!rc && b->max_pages) rc = check_dev_ptr(b->page_table, dev, 4);
    *work = rc == QDQ_OK;
    return rc;
}

// A [n_tokens][heads * head_dim] operand: its pointer, and rows that are 16-byte
// aligned and do not overlap.
int check_rows(const void *p, int64_t stride, int64_t width, int size, int n_tokens, int device) {
    const int rc = check_dev_ptr(p, device);
    if (rc) return rc;
    if (n_tokens > 1 && stride < width) return QDQ_ERR_SHAPE;
    return n_tokens > 1 && (stride * size) % 16 ? QDQ_ERR_ALIGN : QDQ_OK;
}

}  // namespace

extern "C" {

int qdq_paged_create(const qdq_paged_config *cfg, void *k_pages, void *v_pages, qdq_paged **out) {
    if (out == nullptr || cfg == nullptr) return QDQ_ERR_PTR;
    *out = nullptr;
    int rc = check_paged_config(cfg);
    if (rc) return rc;
    const DeviceInfo &dev = current_device(&rc);
    if (rc) return rc;
    if ((rc = check_dev_ptr(k_pages, dev.device)) || (rc = check_dev_ptr(v_pages, dev.device))) return rc;
    qdq_paged *c = new (std::nothrow) qdq_paged();
    if (!c) return QDQ_ERR_CUDA;
    c->cfg = *cfg;
    c->device = dev.device;
    c->sm_count = dev.sm_count;
    c->k_pages = (char *)k_pages;
    c->v_pages = (char *)v_pages;
    c->layer_bytes = (int64_t)cfg->n_pages * cfg->page_size * cfg->n_kv_heads * cfg->head_dim * 2;
    // pair i turns by base^(-2i/R) radians a position: that over 2 pi turns, in units of
    // 2^-64 turn (below one sixth of a turn, so it fits; a double's 53 bits of it are kept)
    uint64_t freq[64] = {};
    for (int i = 0; i < cfg->rope_dim / 2; ++i)
        freq[i] = (uint64_t)std::ldexp(std::pow((double)cfg->rope_base, -2.0 * i / cfg->rope_dim) / 6.283185307179586476925, 64);
    if (cudaMalloc((void **)&c->freq, sizeof(freq)) != cudaSuccess ||
        cudaMemcpy(c->freq, freq, sizeof(freq), cudaMemcpyHostToDevice) != cudaSuccess) {
        cudaGetLastError();
        qdq_paged_destroy(c);
        return QDQ_ERR_CUDA;
    }
    c->pools = {k_pages, v_pages, cfg->n_layers, cfg->n_pages, cfg->page_size, cfg->n_heads, cfg->n_kv_heads,
                cfg->head_dim, cfg->type == QDQ_BF16};
    rc = attend_create(c->pools, c->sm_count, &c->attend);
    // The table's copy and the counters' clearing are asynchronous and in the default stream,
    // which non-blocking streams do not follow: both are done before the handle is used.
    if (!rc && cudaStreamSynchronize(nullptr) != cudaSuccess) {
        cudaGetLastError();
        rc = QDQ_ERR_CUDA;
    }
    if (rc) {
        qdq_paged_destroy(c);
        return rc;
    }
    *out = c;
    return QDQ_OK;
}

void qdq_paged_destroy(qdq_paged *c) {
    if (c == nullptr) return;
    if (c->freq) cudaFree(c->freq);
    attend_destroy(c->attend);
    delete c;
}

int qdq_paged_append(qdq_paged *c, int layer, const qdq_paged_batch *b, int in_type, const void *q, int64_t q_stride,
                     const void *k, int64_t k_stride, const void *v, int64_t v_stride, const float *q_norm,
                     const float *k_norm, float eps, void *q_out, qdq_stream_t stream) {
    bool work;
    int rc = check_paged_call(c, layer, b, &work);
    if (rc) return rc;
    const qdq_paged_config &g = c->cfg;
    if (in_type != QDQ_F32 && in_type != g.type) return QDQ_ERR_TYPE;
    if (!(eps >= 0.0f) || eps > 1.0f) return QDQ_ERR_SHAPE;
    if (!work) return QDQ_OK;
    const int size = in_type == QDQ_F32 ? 4 : 2, n = b->n_tokens, kv = g.n_kv_heads * g.head_dim;
    if ((rc = check_rows(q, q_stride, (int64_t)g.n_heads * g.head_dim, size, n, c->device)) ||
        (rc = check_rows(k, k_stride, kv, size, n, c->device)) ||
        (rc = check_rows(v, v_stride, kv, size, n, c->device)) || (rc = check_dev_ptr(q_out, c->device)) ||
        (q_norm && (rc = check_dev_ptr(q_norm, c->device, 4))) || (k_norm && (rc = check_dev_ptr(k_norm, c->device, 4))))
        return rc;
    AppendArgs a = {};
    a.n_seqs = b->n_seqs, a.n_tokens = n, a.max_pages = b->max_pages;
    a.q_start = b->q_start, a.kv_len = b->kv_len, a.page_table = b->page_table;
    a.q = q, a.k = k, a.v = v;
    a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride;
    a.q_norm = q_norm, a.k_norm = k_norm, a.eps = eps;
    a.freq = c->freq;
    a.q_out = q_out;
    a.k_pages = c->k_pages + layer * c->layer_bytes;
    a.v_pages = c->v_pages + layer * c->layer_bytes;
    a.n_heads = g.n_heads, a.n_kv_heads = g.n_kv_heads, a.rope_dim = g.rope_dim, a.n_pages = g.n_pages;
    a.page_shift = 0;
    while ((1 << a.page_shift) < g.page_size) ++a.page_shift;
    return launch_append(a, in_type == QDQ_F32, g.type == QDQ_BF16, g.rope_interleaved != 0, g.head_dim,
                         (cudaStream_t)stream, c->sm_count);
}

int qdq_paged_attention(qdq_paged *c, int layer, const qdq_paged_batch *b, const void *q, int64_t q_stride,
                        int out_type, void *out, int64_t out_stride, float scale, int window, float *lse,
                        qdq_stream_t stream) {
    bool work;
    int rc = check_paged_call(c, layer, b, &work);
    if (rc) return rc;
    const qdq_paged_config &g = c->cfg;
    if (out_type != QDQ_F32 && out_type != g.type) return QDQ_ERR_TYPE;
    // (the kernel takes scale * log2(e) as fp32)
    if (!std::isfinite((float)(scale * 1.4426950408889634)) || window < 0) return QDQ_ERR_SHAPE;
    if (!work) return QDQ_OK;
    const int n = b->n_tokens;
    const int64_t width = (int64_t)g.n_heads * g.head_dim;
    if ((rc = check_rows(q, q_stride, width, 2, n, c->device)) ||
        (rc = check_rows(out, out_stride, width, out_type == QDQ_F32 ? 4 : 2, n, c->device)) ||
        (lse && (rc = check_dev_ptr(lse, c->device, 4))))
        return rc;
    AttendArgs a = {};
    a.pools = &c->pools;
    a.layer = layer;
    a.n_seqs = b->n_seqs, a.n_tokens = n, a.max_pages = b->max_pages;
    a.q_start = b->q_start, a.kv_len = b->kv_len, a.page_table = b->page_table;
    a.q = q, a.out = out, a.lse = lse;
    a.q_stride = q_stride, a.out_stride = out_stride;
    a.scale = scale, a.window = window, a.out_f32 = out_type == QDQ_F32;
    return launch_attend(c->attend, a, (cudaStream_t)stream);
}

}  // extern "C"
