// qdq_attend.cu -- causal attention of a step's new tokens over the paged cache.
#include <cmath>

#include "qdq_internal.h"
#include "qdq_paged.cuh"

namespace qdq {
namespace {

// One warp per (token, query head); the lanes hold D/32 dims each. Positions are
// taken one by one with the running maximum and sum of an online softmax.
template <typename T, int D>
__global__ void __launch_bounds__(256) attend_kernel(const AttendArgs a) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int t = (int)(unit / a.n_heads), h = (int)(unit % a.n_heads);
    if (t >= a.n_tokens) return;
    const int s = find_seq(a.q_start, a.n_seqs, t);
    if (s < 0) return;
    int first, count;
    seq_tokens(a.q_start, s, a.n_tokens, first, count);
    if (t < first || t >= first + count) return;
    const int g = h / (a.n_heads / a.n_kv_heads);
    const int p = max(a.kv_len[s], 0) - count + (t - first);
    const int64_t last = min((int64_t)p, (int64_t)a.max_pages * a.page_size - 1);
    const int lo = a.window && p >= a.window ? p - a.window + 1 : 0;
    float q[E], o[E] = {}, m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) q[i] = (float)((const T *)a.q)[t * a.q_stride + h * D + lane * E + i] * a.scale;
    for (int j = lo; j <= last; ++j) {
        const int page = a.page_table[(int64_t)s * a.max_pages + j / a.page_size];
        if (page < 0 || page >= a.n_pages) continue;
        const int64_t row = (((int64_t)page * a.page_size + j % a.page_size) * a.n_kv_heads + g) * D + lane * E;
        float x = 0.0f;
#pragma unroll
        for (int i = 0; i < E; ++i) x = fmaf(q[i], (float)((const T *)a.k_pages)[row + i], x);
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, k);
        const float mn = fmaxf(m, x), f = mn == -INFINITY ? 1.0f : expf(m - mn), w = mn == -INFINITY ? 0.0f : expf(x - mn);
        m = mn;
        l = l * f + w;
#pragma unroll
        for (int i = 0; i < E; ++i) o[i] = o[i] * f + w * (float)((const T *)a.v_pages)[row + i];
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int64_t at = t * a.out_stride + h * D + lane * E + i;
        if (a.out_f32) ((float *)a.out)[at] = o[i] * inv;
        else ((T *)a.out)[at] = Float16<T>::one(o[i] * inv);
    }
    if (a.lse && lane == 0) a.lse[(int64_t)t * a.n_heads + h] = l > 0.0f ? m + logf(l) : -INFINITY;
}

}  // namespace

int launch_attend(const AttendArgs &a, cudaStream_t stream, int) {
    const int64_t grid = ((int64_t)a.n_tokens * a.n_heads + 7) / 8;
    if (grid > 0x7FFFFFFF) return QDQ_ERR_LIMIT;
    const unsigned g = (unsigned)grid;
    if (a.head_dim == 64) {
        if (a.bf16) attend_kernel<__nv_bfloat16, 64><<<g, 256, 0, stream>>>(a);
        else attend_kernel<__half, 64><<<g, 256, 0, stream>>>(a);
    } else {
        if (a.bf16) attend_kernel<__nv_bfloat16, 128><<<g, 256, 0, stream>>>(a);
        else attend_kernel<__half, 128><<<g, 256, 0, stream>>>(a);
    }
    return cudaGetLastError() == cudaSuccess ? QDQ_OK : QDQ_ERR_CUDA;
}

}  // namespace qdq
