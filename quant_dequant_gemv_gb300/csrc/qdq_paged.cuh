// qdq_paged.cuh -- device helpers shared by the paged cache's kernels
// (qdq_paged.cu, qdq_attend.cu): the batch's arrays are device data, so every
// value read from them is clamped to its documented range before it becomes an
// address.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qdq_device.cuh"

namespace qdq {

constexpr int kMaxSeqs = 1024;

// The serving kernels are launched with programmatic stream serialisation: the CTAs of a
// call may be placed while the last kernel of the stream still runs, wait here until it
// has completed and its writes are visible, and let the next call's be placed in turn.
// First thing in a kernel, before any access to memory that another kernel may write.
QDQ_DEV void follow_last_kernel() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// The new tokens of sequence s, inside [0, n_tokens].
QDQ_DEV void seq_tokens(const int32_t *q_start, int s, int n_tokens, int &first, int &count) {
    const int a = min(max(q_start[s], 0), n_tokens), b = min(max(q_start[s + 1], 0), n_tokens);
    first = a;
    count = max(b - a, 0);
}

// The last sequence whose q_start is <= t, found by the whole warp: 32 probes a
// round, so one round for 32 sequences and two for 1024. -1 if there is none.
QDQ_DEV int find_seq(const int32_t *q_start, int n_seqs, int t) {
    const int lane = threadIdx.x & 31;
    int lo = 0, len = n_seqs;
    while (len > 0) {
        const int step = (len + 31) >> 5, at = lane * step;
        const unsigned m = __ballot_sync(0xFFFFFFFFu, at < len && q_start[lo + at] <= t);
        if (m == 0) return -1;
        const int c = 31 - __clz(m);
        lo += c * step;
        len = min(step, len - c * step);
        if (step == 1) return lo;
    }
    return -1;
}

template <typename T>
struct Float16;
template <>
struct Float16<__half> {
    static QDQ_DEV uint32_t pack(float lo, float hi) {
        uint32_t d;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
        return d;
    }
    static QDQ_DEV float2 unpack(uint32_t v) { return __half22float2(*reinterpret_cast<__half2 *>(&v)); }
};
template <>
struct Float16<__nv_bfloat16> {
    static QDQ_DEV uint32_t pack(float lo, float hi) {
        uint32_t d;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
        return d;
    }
    static QDQ_DEV float2 unpack(uint32_t v) { return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u)); }
};

// Four consecutive values, read once, as floats.
template <typename TI>
QDQ_DEV void load4(const TI *p, float *x) {
    if constexpr (sizeof(TI) == 4) {
        const float4 v = __ldcs(reinterpret_cast<const float4 *>(p));
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
        const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(p));
        const float2 a = Float16<TI>::unpack(v.x), b = Float16<TI>::unpack(v.y);
        x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
    }
}

}  // namespace qdq
