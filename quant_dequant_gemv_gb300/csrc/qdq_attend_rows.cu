// qdq_attend_rows.cu -- attention of few rows over the paged cache: over a cache of e4m3 values,
// and over the pages of a token's list in a cache of any type.
//
//   o = sum_j p_j v_j / l,  p_j = 2^(t_j - m),  l = sum_j p_j,  t_j = scale * log2(e) * q . k_j
// A block is as many whole tokens as give 8, 16 or 32 rows (row = token * group + head). Every row
// meets every position once, in one pass with a running maximum that lags by up to 2^8.
//
// Scales. A key of a block of 16 positions is 2^ek times its e4m3 value, which fp16 holds exactly, so
// the product with the fp16 query is exact up to the fp32 sums and 2^ek goes into t's factor. A
// value is 2^ev times its e4m3 value: the weight that meets it is 2^(t + ev - m), with m the
// maximum of t + ev, and l sums those weights times 2^-ev.
//
// The weights meet the values as two 16-bit terms, what the type keeps of them and what it leaves
// (16 bits in bf16, 22 in fp16). Where a block has 8 rows, the second term takes the other 8 rows of
// the matrix instruction, and costs nothing.
//
// Few rows are bound by the cache's bytes, not by the matrix instruction: mma.sync takes its operands
// from registers, where the e4m3 values are widened on their way (a matrix unit that reads shared
// memory would want them written back there), and any 8 rows fill it. A CTA has eight working warps,
// each with 16 of a tile's 128 positions (one block of scales), a maximum, a sum and an accumulator
// of its own; one warp that issues the copies, whole runs of a page's rows by tensor copies with a
// swizzle into a ring of stages of a tile's keys and values, and the queries of the next items; and
// three that join the working warps' states at an item's end, while those go on with the next.
//
// Operands. The contraction may take its terms in any order, so a lane reads 16 consecutive bytes of
// a key and its query fragments are loaded in that order. Of the values a lane reads 16 consecutive
// dims of four positions and interleaves pairs of positions; its accumulators are then 16 consecutive
// dims of two columns.
//
// The work is dealt to the CTAs in equal ranges and joined as in qdq_attend.cu (qdq_attend_plan.h).
//
// What bounds it, as measured (GB300; 32 query and 8 kv heads of 128, e4m3): HBM. 64 tokens over 30 to
// 8192 positions 103.5 us = 5.8 TB/s, 86 % of the copy rate (pages of 64 positions; at 16 a copy is 2 KB
// and it is 147 us); 64 tokens over up to 2048 chosen positions 58 us = 4.5 TB/s, of which the start and
// the joins are about 10; one token over 131001 positions 57 us. A few hundred positions take 6 us, or 9
// with a join: each step of the start (the share, a page, a copy, a counter) is one trip to L2 or HBM.
// Looked up tile by tile, pages and scales bounded the copies (64 tokens 150 us).
#include <algorithm>
#include <cmath>
#include <cuda.h>
#include <new>
#include <type_traits>

#include "qdq_attend_walk.cuh"
#include "qdq_internal.h"
#include "qdq_paged.cuh"
#include "qdq_tcgen05.cuh"

namespace qdq {

// Host state: the tensor maps of the pools, and the workspace (partial results, the joins' counters).
struct RowsState {
    CUtensorMap k_map, v_map;
    char *mem = nullptr;
    float *part_o = nullptr;
    float2 *part_ml = nullptr;
    unsigned *counters = nullptr;
    int ctas = 0;
};

namespace {

__device__ int g_rows_status;

constexpr int kWarps = 8, kJoiners = 3, kThreads = (kWarps + 1 + kJoiners) * 32, kMostRows = 32;
constexpr float kLag = 8.0f;  // log2 of how far the running maximum may lag

enum Kind { kF16, kBf16, kE4m3 };

struct RowsArgs {
    int n_seqs, n_tokens, max_pages;
    const int32_t *q_start, *kv_len, *page_table;
    const uint16_t *q;
    void *out;
    float *lse;
    int64_t q_stride, out_stride;
    int out_type;
    float scale_log2;
    int n_pages, page_shift, n_heads;
    int64_t page0;       // the layer's first page
    const uint8_t *k_scales, *v_scales;  // of the layer
    const int32_t *lists;  // [n_tokens][kv_heads][g.list], or NULL
    AttendGeometry g;
    float *part_o;
    float2 *part_ml;
    unsigned *counters;
};

struct RowsPiece {
    int n, t0;               // key tiles (0 ends the walk), the first
    int lo, hi;              // positions that the block attends to
    int tokens, token0, p0;  // the block's tokens, the row of the first, its position
    int head;
    int whole, c_first, c_last;
};

template <int HD, int KIND, int MODE>
struct Shape {
    static constexpr int kRows = 8 << MODE;
    static constexpr uint32_t kRow = HD * (KIND == kE4m3 ? 1 : 2);  // bytes of a position
    static constexpr uint32_t kHalf = kTileN * kRow;                // keys (or values) of a stage
    static constexpr uint32_t kStage = 2 * kHalf;
    static constexpr int kStages = (int)(131072 / kStage);
    static constexpr int kPieces = MODE == 0 ? 8 : MODE == 1 ? 4 : 2;  // items that the copies may be ahead
    static constexpr uint32_t kMerge = kStages * kStage;                  // [2][warp][8 rows][HD + 4]
    static constexpr uint32_t kPitch = (HD + 4) * 4, kMergeSize = kWarps * 8 * kPitch;
    static constexpr uint32_t kState = kMerge + 2 * kMergeSize;           // [2][warp][8 rows] maximum and sum
    static constexpr uint32_t kQ = kState + 2 * kWarps * 64, kQSize = kRows * HD * 2;  // [piece][row][HD]
    static constexpr uint32_t kMeta = kQ + kPieces * kQSize;              // [stage] Meta
    static constexpr uint32_t kBars = kMeta + kStages * 64;
    static constexpr uint32_t kStart = kBars + (2 * kStages + 2 * kPieces + 4) * 8;
    static constexpr uint32_t kPiece = kStart + 80;
    static constexpr uint32_t kTotal = kPiece + kPieces * sizeof(RowsPiece);
    static_assert(kQ % 16 == 0 && kMeta % 16 == 0 && kBars % 8 == 0 && kStart % 8 == 0 && kTotal <= 232448, "shared memory");
    static_assert(kStages * kStage >= 20 * kMaxSeqs && sizeof(Start) <= 80, "find_start's room, Shape::kPiece");
};

// Of each block of 16 positions of a stage: its first position (-1: absent) and its scales' exponents.
struct Meta {
    int base[8];
    int8_t ek[8], ev[8];
};
static_assert(sizeof(Meta) <= 64, "Shape::kBars");

template <int KIND>
QDQ_DEV void mma(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (KIND == kBf16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

QDQ_DEV uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t d;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
    return d;
}

QDQ_DEV void tma_rows(uint32_t dst, const CUtensorMap *map, int y, int z, uint32_t bar) { tma_load_3d(dst, map, 0, y, z, bar); }

template <int HD, int KIND, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    rows_kernel(const RowsArgs a, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
    using L = Shape<HD, KIND, MODE>;
    using F16 = Float16<typename std::conditional<KIND == kBf16, __nv_bfloat16, __half>::type>;
    constexpr bool kPacked = MODE == 0;          // a weight's second term in rows 8..15
    constexpr int kHalves = MODE == 2 ? 2 : 1;   // 32 rows: even and odd warps have 16 each, and two blocks of positions
    constexpr int kGroups = MODE == 0 ? 1 : 2;   // of 8 rows, of a warp
    constexpr int kN = HD / 8;                   // column tiles of the accumulator, dims of a lane and column
    constexpr float kLift = KIND == kBf16 ? 0.0f : 7.0f;  // (fp16's small weights: qdq_attend.cu)
    extern __shared__ __align__(1024) char smem[];
    const uint32_t sb = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int *status = &g_rows_status;
    Start *start = reinterpret_cast<Start *>(smem + L::kStart);
    RowsPiece *pieces = reinterpret_cast<RowsPiece *>(smem + L::kPiece);
    auto full = [&](int i) { return sb + L::kBars + 8u * i; };
    auto empty = [&](int i) { return sb + L::kBars + 8u * (L::kStages + i); };
    auto piece_full = [&](int i) { return sb + L::kBars + 8u * (2 * L::kStages + i); };
    auto piece_free = [&](int i) { return sb + L::kBars + 8u * (2 * L::kStages + L::kPieces + i); };
    auto merge_full = [&](int i) { return sb + L::kBars + 8u * (2 * L::kStages + 2 * L::kPieces + i); };
    auto merge_free = [&](int i) { return sb + L::kBars + 8u * (2 * L::kStages + 2 * L::kPieces + 2 + i); };
    auto piece_at = [](uint32_t items) { return (int)(items % L::kPieces); };
    auto piece_phase = [](uint32_t items) { return (items / L::kPieces) & 1; };
    follow_last_kernel();

    if (threadIdx.x == 0) {
        for (int i = 0; i < L::kStages; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), kWarps);
        }
        for (int i = 0; i < L::kPieces; ++i) {
            mbar_init(piece_full(i), 1);
            mbar_init(piece_free(i), kWarps + kJoiners);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(merge_full(i), kWarps);
            mbar_init(merge_free(i), kJoiners);
        }
        fence_mbar_init();
    }
    find_start<kThreads>(a, smem, start);
    if (!start->live) return;
    const Start s0 = *start;
    __syncthreads();
    fence_async_smem();  // the ring's memory goes over to the copies

    const int run_shift = min(a.page_shift, 7);  // log2 of the positions of one copy
    if (warp == kWarps) {
        // ---- copies ---------------------------------------------------------------------------
        const uint32_t run_bytes = L::kRow << run_shift, q_bytes = a.g.group * HD * 2;
        const int blocks_shift = a.page_shift - 4;  // log2 of a page's blocks of scales
        uint32_t stage_no = 0, items = 0;
        // An item's piece, with what its positions are found by.
        struct Source {
            const int32_t *list;  // the token's pages, or NULL
            int t0, lo, hi, token0, p0;
        };
        auto source = [&](const Walk &w) {
            Source f;
            f.token0 = w.first + w.b.i0, f.p0 = w.kv - w.count + w.b.i0, f.t0 = w.t_beg();
            // (of a list the positions are those of its pages up to the token's own)
            f.list = a.g.list ? a.lists + ((int64_t)f.token0 * a.g.kv_heads + w.head) * a.g.list : nullptr;
            f.lo = a.g.list ? 0 : w.b.lo;
            f.hi = a.g.list ? max(min(f.p0 + 1, a.g.table_end), 0) : w.b.hi;
            return f;
        };
        // Four tiles at a time, a lane has one block of 16 positions (block lane % 8 of tile lane / 8): its
        // first position and its page, or -1 where there is none, and its scales. The next four's pages, and
        // the next piece's first, are on their way while these four are copied.
        auto entry = [&](const Walk &w, const Source &f, int j, int &position, int &page) {
            position = page = -1;
            const int place = (f.t0 + j + (lane >> 3)) * kTileN + ((lane & 7) << 4);
            if (j + (lane >> 3) >= w.n || place >= w.b.hi) return;
            int at = place >> a.page_shift;
            if (f.list) {
                const int e = f.list[at], last = at ? f.list[at - 1] : -1;
                if (e < 0 || (at && e <= last) || e >= a.max_pages) return;
                at = e;
            }
            position = (at << a.page_shift) + (place & ((1 << a.page_shift) - 1));
            // (a page's run is copied whole if any of it is attended to)
            const int run = position & ~((1 << run_shift) - 1);
            if (run < f.hi && run + (1 << run_shift) > f.lo && QDQ_CHECK(status, at >= 0 && at < a.max_pages)) page = w.pages[at];
        };
        // (the bytes as they are: what is computed of them would wait for them, and with it the copies)
        uint8_t k_scale = 127, v_scale = 127;
        auto scale = [&](const Walk &w, int position, int &page) {
            if ((unsigned)page >= (unsigned)a.n_pages) page = -1;
            if (KIND != kE4m3 || page < 0) return;
            const int64_t at = (((int64_t)page * a.g.kv_heads + w.head) << blocks_shift) + ((position & ((1 << a.page_shift) - 1)) >> 4);
            k_scale = a.k_scales[at], v_scale = a.v_scales[at];
        };
        Walk w(a, s0), ahead = w;
        Source f = source(w), f_ahead = f;
        int position = -1, page = -1, next_position = -1, next_page = -1, first_position = -1, first_page = -1;
        if (w.more()) {
            entry(w, f, 0, position, page);
            entry(w, f, 4, next_position, next_page);
        }
        for (;; ++items) {
            // (after the first tile's copies have been issued: all of it is needed at once)
            auto publish = [&] {
                const int at = piece_at(items);
                RowsPiece &piece = pieces[at];
                mbar_wait(piece_free(at), piece_phase(items) ^ 1, status);
                if (lane == 0) {
                    piece.n = w.n;
                    if (w.n) {
                        piece.t0 = f.t0;
                        piece.lo = f.lo, piece.hi = f.hi;
                        piece.tokens = w.b.i1 - w.b.i0, piece.token0 = f.token0, piece.p0 = f.p0;
                        piece.head = w.head;
                        piece.whole = w.whole();
                        if (!w.whole()) {
                            piece.c_first = range_owner(s0.total, s0.ctas, w.item + a.g.item);
                            piece.c_last = range_owner(s0.total, s0.ctas, w.item + item_units(w.b, a.g.item) - 1);
                        }
                    }
                    // (the group's heads of a token lie one behind the other)
                    mbar_arrive_expect_tx(piece_full(at), w.n ? piece.tokens * q_bytes : 0u);
                }
                __syncwarp();
                if (w.more() && lane < w.b.i1 - w.b.i0 && QDQ_CHECK(status, f.token0 + lane < a.n_tokens && (lane + 1) * q_bytes <= L::kQSize))
                    bulk_g2s(sb + L::kQ + at * L::kQSize + lane * q_bytes,
                             a.q + (int64_t)(f.token0 + lane) * a.q_stride + (int64_t)w.head * a.g.group * HD, q_bytes, piece_full(at));
            };
            if (!w.more()) {
                publish();
                break;
            }
            scale(w, position, page);
            for (int j = 0; j < w.n; ++j, ++stage_no) {
                const int y = j & 3;
                if (y == 0 && j) {
                    position = next_position, page = next_page;
                    scale(w, position, page);
                    entry(w, f, j + 4, next_position, next_page);
                }
                // lane r issues the copies of the tile's run r
                const int from = y * 8 + ((lane << run_shift) >> 4);
                const int run_page = __shfl_sync(0xFFFFFFFFu, page, from & 31), run_position = __shfl_sync(0xFFFFFFFFu, position, from & 31);
                const int here = lane < (kTileN >> run_shift) ? run_page : -1;
                const uint32_t bytes = __popc(__ballot_sync(0xFFFFFFFFu, here >= 0)) * run_bytes * 2;
                const int stage = stage_no % L::kStages;
                mbar_wait(empty(stage), ((stage_no / L::kStages) & 1) ^ 1, status);
                if (here >= 0) {
                    const int in_page = run_position & ((1 << a.page_shift) - 1);
                    const uint32_t to = sb + stage * L::kStage + lane * run_bytes;
                    if (QDQ_CHECK(status, w.head < a.g.kv_heads && lane * run_bytes + run_bytes <= L::kHalf && here < a.n_pages)) {
                        if constexpr (KIND == kE4m3) {
                            const int y = (w.head << a.page_shift) + in_page, z = (int)(a.page0 + here);
                            tma_rows(to, &k_map, y, z, full(stage));
                            tma_rows(to + L::kHalf, &v_map, y, z, full(stage));
                        } else {
                            const int row8 = (int)((((a.page0 + here) << a.page_shift) + in_page) >> 3);
                            tma_load_4d(to, &k_map, 0, 0, w.head * (HD / 64), row8, full(stage));
                            tma_load_4d(to + L::kHalf, &v_map, 0, 0, w.head * (HD / 64), row8, full(stage));
                        }
                    }
                }
                if (j == 0) publish();
                if (lane >> 3 == y) {
                    Meta *m = reinterpret_cast<Meta *>(smem + L::kMeta + stage * 64);
                    m->base[lane & 7] = page < 0 ? -1 : position;
                    m->ek[lane & 7] = (int8_t)exponent_of(k_scale);
                    m->ev[lane & 7] = (int8_t)exponent_of(v_scale);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive_expect_tx(full(stage), bytes);
                if (j == 0) {
                    ahead.next(a);
                    if (ahead.more()) {
                        f_ahead = source(ahead);
                        entry(ahead, f_ahead, 0, first_position, first_page);
                    }
                }
            }
            w = ahead, f = f_ahead;
            position = first_position, page = first_page;
            if (w.more()) entry(w, f, 4, next_position, next_page);
        }
        // every copy has landed before the CTA can end, also after a wait that ran out
        for (uint32_t i = stage_no < (uint32_t)L::kStages ? 0 : stage_no - L::kStages; i < stage_no; ++i)
            mbar_wait(full(i % L::kStages), (i / L::kStages) & 1, status);
        for (uint32_t i = items < (uint32_t)L::kPieces ? 0 : items - L::kPieces + 1; i < items; ++i)
            mbar_wait(piece_full(piece_at(i)), piece_phase(i), status);
        return;
    }

    if (warp < kWarps) {
    // ---- the working warps -----------------------------------------------------------------------
    const int g = lane >> 2, c = lane & 3, half = warp % kHalves;
    uint32_t stage_no = 0, merges = 0;
    for (uint32_t items = 0;; ++items) {
        const int at = piece_at(items);
        mbar_wait(piece_full(at), piece_phase(items), status);
        const RowsPiece w = pieces[at];
        if (w.n == 0) break;
        const int rows = w.tokens * a.g.group;

        // The queries, in the order in which a lane reads a key's dims: the rows g and g + 8 of the warp's
        // 16, of each step of 16 terms the pairs that b0 and b1 hold.
        uint32_t qa[kGroups][HD / 8];
        int row_lo[kGroups], row_hi[kGroups];  // positions of the lane's rows
#pragma unroll
        for (int z = 0; z < kGroups; ++z) {
            const int r = 16 * half + 8 * z + g, tok = r / a.g.group;
            const bool live = r < rows;
            const uint32_t q = sb + L::kQ + at * L::kQSize + r * (HD * 2);
            // consecutive dims of the lane: KIND e4m3: HD / 4 from HD / 4 * c on; 16-bit: 16 from 64 h + 16 c on
            constexpr int kRun = KIND == kE4m3 ? HD / 4 : 16;
#pragma unroll
            for (int k = 0; k < HD / 4; k += 8) {
                const int dim = KIND == kE4m3 ? kRun * c + k : k / 16 * 64 + 16 * c + k % 16;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (live) v = lds128(q + 2 * dim);
                uint32_t *to = &qa[z][k / 2];
                to[0] = v.x, to[1] = v.y, to[2] = v.z, to[3] = v.w;
            }
            const int p = w.p0 + tok;
            row_lo[z] = a.g.window ? max(p - a.g.window + 1, 0) : 0;
            row_hi[z] = live ? min(p + 1, w.hi) : 0;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(piece_free(at));
        // positions that every row attends to
        const int all_lo = a.g.window ? max(w.p0 + w.tokens - a.g.window, 0) : 0, all_hi = min(w.p0 + 1, w.hi);

        float o[kN][4];
#pragma unroll
        for (int n = 0; n < kN; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;
        float m[kGroups], l[kGroups];
#pragma unroll
        for (int z = 0; z < kGroups; ++z) m[z] = -INFINITY, l[z] = 0.0f;

        for (int j = 0; j < w.n; ++j, ++stage_no) {
            const int stage = stage_no % L::kStages;
            mbar_wait(full(stage), (stage_no / L::kStages) & 1, status);
            const Meta *meta = reinterpret_cast<const Meta *>(smem + L::kMeta + stage * 64);
#pragma unroll 1
            for (int block = warp - half; block < warp - half + kHalves; ++block) {
                const int base = meta->base[block];
                if (base < 0 || base >= w.hi || base + 16 <= w.lo) continue;
                const uint32_t ks = sb + stage * L::kStage, vs = ks + L::kHalf;
                const float ev = KIND == kE4m3 ? (float)meta->ev[block] : 0.0f;
                const float c2 = KIND == kE4m3 ? a.scale_log2 * __int_as_float((127 + meta->ek[block]) << 23) : a.scale_log2;
                float s[2][4];
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.0f;
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    const int r = block * 16 + nt * 8 + g;
                    // 16 bytes of the key at a time: two (16-bit) or four (e4m3) pairs of dims
#pragma unroll
                    for (int u = 0; u < (int)L::kRow / 64; ++u) {
                        uint4 v;
                        if constexpr (KIND == kE4m3)
                            v = HD == 128 ? lds128(ks + r * 128 + (((2 * c + u) ^ g) << 4))
                                          : lds128(ks + r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
                        else
                            v = lds128(ks + (r >> 3) * (8 * L::kRow) + (u / 2) * 1024 + (r & 7) * 128 + (((2 * c + u % 2) ^ g) << 4));
                        const uint32_t x[4] = {v.x, v.y, v.z, v.w};
                        constexpr int kSteps = KIND == kE4m3 ? 4 : 2;  // of 16 terms
#pragma unroll
                        for (int k = 0; k < kSteps; ++k) {
                            uint32_t b0, b1;
                            if constexpr (KIND == kE4m3) e4m3x4_to_f16(x[k], b0, b1);
                            else b0 = x[2 * k], b1 = x[2 * k + 1];
                            const int step = u * kSteps + k;
                            if constexpr (kPacked) mma<KIND>(s[nt], qa[0][2 * step], 0u, qa[0][2 * step + 1], 0u, b0, b1);
                            else mma<KIND>(s[nt], qa[0][2 * step], qa[1][2 * step], qa[0][2 * step + 1], qa[1][2 * step + 1], b0, b1);
                        }
                    }
                }
                // ---- weights: of group z the row 8 z + g of the warp's, positions 8 nt + 2 c and the next -----------------
                const bool masked = base < all_lo || base + 16 > all_hi;
                float best[kGroups];
                bool rise = false;
#pragma unroll
                for (int z = 0; z < kGroups; ++z) {
                    float top = -INFINITY;
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float &x = s[nt][2 * z + e];
                            x = fmaf(x, c2, ev);
                            const int p = base + 8 * nt + 2 * c + e;
                            if (masked && (p < row_lo[z] || p >= row_hi[z])) x = -INFINITY;
                            top = fmaxf(top, x);
                        }
                    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                    best[z] = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                    rise |= best[z] > m[z] + (m[z] == -INFINITY ? 0.0f : kLag);
                }
                if (__any_sync(0xFFFFFFFFu, rise)) {  // raise the maximum: O and l change units
#pragma unroll
                    for (int z = 0; z < kGroups; ++z) {
                        const float to = fmaxf(m[z], best[z]), f = to == -INFINITY ? 1.0f : ex2(m[z] - to);
                        m[z] = to;
                        l[z] *= f;
#pragma unroll
                        for (int n = 0; n < kN; ++n) {
                            o[n][2 * z] *= f, o[n][2 * z + 1] *= f;
                            if constexpr (kPacked) o[n][2] *= f, o[n][3] *= f;
                        }
                    }
                }
                uint32_t p_hi[kGroups][2], p_lo[kGroups][2];  // [8 rows][positions 8 nt ..]
#pragma unroll
                for (int z = 0; z < kGroups; ++z) {
                    const float ref = kLift - (m[z] == -INFINITY ? 0.0f : m[z]);
                    float sum = 0.0f;
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt) {
                        const float x = ex2(s[nt][2 * z] + ref), y = ex2(s[nt][2 * z + 1] + ref);
                        sum += x + y;
                        p_hi[z][nt] = F16::pack(x, y);
                        const float2 h = F16::unpack(p_hi[z][nt]);
                        p_lo[z][nt] = F16::pack(x - h.x, y - h.y);
                    }
                    l[z] += KIND == kE4m3 ? sum * __int_as_float((int)(127.0f - ev) << 23) : sum;
                }
                // ---- values: positions 2 c, 2 c + 1 (b0), 2 c + 8, 2 c + 9 (b1) of the lane's kN dims ---------
                constexpr int kWords = (int)L::kRow / 32;  // of a position's share of a lane, 32 bits each
                uint32_t v[4][kWords];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int r = block * 16 + 2 * c + (y & 1) + 8 * (y >> 1);
                    if constexpr (KIND == kE4m3 && HD == 64) {
                        // 8 bytes: chunk g / 2 of the 64-byte row, which is at (g / 2) ^ (r / 2 % 4)
                        const uint32_t at = vs + r * 64 + (((g >> 1) ^ ((r >> 1) & 3)) << 4) + (g & 1) * 8;
                        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v[y][0]), "=r"(v[y][1]) : "r"(at));
                    } else {
#pragma unroll
                        for (int u = 0; u < kWords / 4; ++u) {
                            const uint32_t at = KIND == kE4m3 ? vs + r * 128 + ((g ^ (r & 7)) << 4)
                                                              : vs + (r >> 3) * (8 * L::kRow) + u * 1024 + (r & 7) * 128 + ((g ^ (r & 7)) << 4);
                            const uint4 x = lds128(at);
                            v[y][4 * u] = x.x, v[y][4 * u + 1] = x.y, v[y][4 * u + 2] = x.z, v[y][4 * u + 3] = x.w;
                        }
                    }
                }
                if (base < w.lo || base + 16 > w.hi) {
                    // rows that hold no position of the block: their weights are zero, but 0 x NaN is not
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const int p = base + 2 * c + (y & 1) + 8 * (y >> 1);
                        if (p < w.lo || p >= w.hi) {
#pragma unroll
                            for (int k = 0; k < kWords; ++k) v[y][k] = 0;
                        }
                    }
                }
                auto column = [&](int n, uint32_t b0, uint32_t b1) {
                    if constexpr (kPacked) {
                        mma<KIND>(o[n], p_hi[0][0], p_lo[0][0], p_hi[0][1], p_lo[0][1], b0, b1);
                    } else {
                        mma<KIND>(o[n], p_hi[0][0], p_hi[1][0], p_hi[0][1], p_hi[1][1], b0, b1);
                        mma<KIND>(o[n], p_lo[0][0], p_lo[1][0], p_lo[0][1], p_lo[1][1], b0, b1);
                    }
                };
#pragma unroll
                for (int k = 0; k < kWords; ++k) {
                    if constexpr (KIND == kE4m3) {
                        uint32_t b0[4], b1[4];  // of dims 4 k .. 4 k + 3
                        e4m3x4_to_f16(prmt(v[0][k], v[1][k], 0x5140), b0[0], b0[1]);
                        e4m3x4_to_f16(prmt(v[0][k], v[1][k], 0x7362), b0[2], b0[3]);
                        e4m3x4_to_f16(prmt(v[2][k], v[3][k], 0x5140), b1[0], b1[1]);
                        e4m3x4_to_f16(prmt(v[2][k], v[3][k], 0x7362), b1[2], b1[3]);
#pragma unroll
                        for (int x = 0; x < 4; ++x) column(4 * k + x, b0[x], b1[x]);
                    } else {
                        column(2 * k, prmt(v[0][k], v[1][k], 0x5410), prmt(v[2][k], v[3][k], 0x5410));
                        column(2 * k + 1, prmt(v[0][k], v[1][k], 0x7632), prmt(v[2][k], v[3][k], 0x7632));
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty(stage));
        }

        // ---- the piece's end: the warp's state, eight rows at a time --------------------------------------
#pragma unroll
        for (int z = 0; z < kGroups; ++z) {
            if (8 * z >= rows) break;
            const int room = merges & 1, mine = 16 * half + 8 * z + g;
            mbar_wait(merge_free(room), ((merges >> 1) & 1) ^ 1, status);
            ++merges;
            l[z] += __shfl_xor_sync(0xFFFFFFFFu, l[z], 1);
            l[z] += __shfl_xor_sync(0xFFFFFFFFu, l[z], 2);
            if (c == 0) reinterpret_cast<float2 *>(smem + L::kState)[(room * kWarps + warp) * 8 + g] = make_float2(m[z], l[z]);
            // the lane's columns 2 c and 2 c + 1, kN dims each
            if (mine < rows) {
                float *to = reinterpret_cast<float *>(smem + L::kMerge + room * L::kMergeSize + (warp * 8 + g) * L::kPitch);
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int n = 0; n < kN; n += 4) {
                        float e[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            e[y] = kPacked ? o[n + y][x] + o[n + y][2 + x] : o[n + y][2 * z + x];
                        const int dim = KIND == kE4m3 || HD == 64 ? (2 * c + x) * kN + n : n / 8 * 64 + (2 * c + x) * 8 + n % 8;
                        *reinterpret_cast<float4 *>(to + dim) = make_float4(e[0], e[1], e[2], e[3]);
                    }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(merge_full(room));
        }
    }
    return;
    }

    // ---- the joining warps --------------------------------------------------------------------------
    const int tid = threadIdx.x - (kWarps + 1) * 32;
    constexpr int kJoin = kJoiners * 32;
    const float ln2 = 0.6931471805599453f;
    int *flag = reinterpret_cast<int *>(smem + L::kStart);
    uint32_t merges = 0;
    for (uint32_t items = 0;; ++items) {
        const int piece_no = piece_at(items);
        mbar_wait(piece_full(piece_no), piece_phase(items), status);
        const RowsPiece w = pieces[piece_no];
        __syncwarp();
        if (lane == 0) mbar_arrive(piece_free(piece_no));
        if (w.n == 0) break;
        const int rows = w.tokens * a.g.group;
        const int part = blockIdx.x * 2 + (!w.whole && (int)blockIdx.x == w.c_first ? 1 : 0);
        auto store = [&](int row, int dim, float4 v) {
            const int tok = row / a.g.group;
            const int64_t at = (int64_t)(w.token0 + tok) * a.out_stride + (int64_t)(w.head * a.g.group + row - tok * a.g.group) * HD + dim;
            if (!QDQ_CHECK(status, at >= 0 && at + 4 <= (int64_t)(a.n_tokens - 1) * a.out_stride + (int64_t)a.n_heads * HD)) return;
            if (a.out_type == QDQ_F32) {
                *reinterpret_cast<float4 *>((float *)a.out + at) = v;
            } else if (a.out_type == QDQ_BF16) {
                *reinterpret_cast<uint2 *>((uint16_t *)a.out + at) =
                    make_uint2(Float16<__nv_bfloat16>::pack(v.x, v.y), Float16<__nv_bfloat16>::pack(v.z, v.w));
            } else {
                *reinterpret_cast<uint2 *>((uint16_t *)a.out + at) =
                    make_uint2(Float16<__half>::pack(v.x, v.y), Float16<__half>::pack(v.z, v.w));
            }
        };
        auto store_lse = [&](int row, float top, float sum) {
            const int tok = row / a.g.group;
            if (a.lse)
                a.lse[(int64_t)(w.token0 + tok) * a.n_heads + w.head * a.g.group + row - tok * a.g.group] =
                    sum != 0.0f ? (top - kLift + log2f(sum)) * ln2 : -INFINITY;
        };
        for (int z = 0; z < kGroups && 8 * z < rows; ++z, ++merges) {
            const int room = merges & 1;
            mbar_wait(merge_full(room), (merges >> 1) & 1, status);
            const float2 *state = reinterpret_cast<const float2 *>(smem + L::kState) + room * kWarps * 8;
            for (int x = tid; x < kHalves * 8 * (HD / 4); x += kJoin) {
                const int i = x / (HD / 4), dim = x % (HD / 4) * 4, r = i % 8, h = i / 8, row = 16 * h + 8 * z + r;
                if (row >= rows) continue;
                float top = -INFINITY, sum = 0.0f;
                float4 acc = make_float4(0, 0, 0, 0);
#pragma unroll
                for (int y = h; y < kWarps; y += kHalves) top = fmaxf(top, state[y * 8 + r].x);
#pragma unroll
                for (int y = h; y < kWarps; y += kHalves) {
                    const float2 ml = state[y * 8 + r];
                    const float f = ml.y != 0.0f ? ex2(ml.x - top) : 0.0f;  // (a sum that is no number stays none)
                    const float4 v = *reinterpret_cast<const float4 *>(smem + L::kMerge + room * L::kMergeSize + (y * 8 + r) * L::kPitch + dim * 4);
                    sum = fmaf(ml.y, f, sum);
                    acc.x = fmaf(v.x, f, acc.x), acc.y = fmaf(v.y, f, acc.y), acc.z = fmaf(v.z, f, acc.z), acc.w = fmaf(v.w, f, acc.w);
                }
                if (w.whole) {
                    const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
                    store(row, dim, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
                    if (dim == 0) store_lse(row, top, sum);
                } else {
                    __stcg(reinterpret_cast<float4 *>(a.part_o + ((int64_t)part * kMostRows + row) * HD + dim), acc);
                    if (dim == 0) __stcg(a.part_ml + part * kMostRows + row, make_float2(top, sum));
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(merge_free(room));
        }
        if (w.whole) continue;

        // ---- the last of an item's parts joins them all, in CTA order ---------------------------------------
        named_bar_sync(1, kJoin);
        if (tid == 0) {
            // (the fence covers the warps' stores, which the barrier has shown this thread; the count
            // goes back to zero by itself)
            __threadfence();
            const unsigned others = (unsigned)(w.c_last - w.c_first);
            unsigned *counter = a.counters + (QDQ_CHECK(status, w.c_first >= 0 && w.c_first < (int)gridDim.x) ? w.c_first : 0);
            *flag = atomicInc(counter, others) == others;
            __threadfence();
        }
        named_bar_sync(1, kJoin);
        const bool last = *flag != 0;
        named_bar_sync(1, kJoin);
        if (!last) continue;
        // (as many loads in flight as there may be parts)
        auto join = [&](auto at_once) {
            constexpr int kAtOnce = decltype(at_once)::value;
            for (int x = tid; x < rows * (HD / 4); x += kJoin) {
                const int row = x / (HD / 4), dim = x % (HD / 4) * 4;
                float top = -INFINITY, sum = 0.0f;
                float4 acc = make_float4(0, 0, 0, 0);
                for (int cta = w.c_first; cta <= w.c_last; cta += kAtOnce) {
                    float2 ml[kAtOnce];
                    float4 v[kAtOnce];
    #pragma unroll
                    for (int y = 0; y < kAtOnce; ++y) {
                        const int at = min(cta + y, w.c_last), pt = 2 * at + (at == w.c_first ? 1 : 0);
                        ml[y] = __ldcg(a.part_ml + pt * kMostRows + row);
                        v[y] = __ldcg(reinterpret_cast<const float4 *>(a.part_o + ((int64_t)pt * kMostRows + row) * HD + dim));
                    }
    #pragma unroll
                    for (int y = 0; y < kAtOnce; ++y) {
                        if (cta + y > w.c_last || ml[y].y == 0.0f) continue;
                        const float to = fmaxf(top, ml[y].x), h = sum != 0.0f ? ex2(top - to) : 0.0f, f = ex2(ml[y].x - to);
                        top = to;
                        sum = fmaf(sum, h, ml[y].y * f);
                        acc.x = fmaf(v[y].x, f, acc.x * h), acc.y = fmaf(v[y].y, f, acc.y * h);
                        acc.z = fmaf(v[y].z, f, acc.z * h), acc.w = fmaf(v[y].w, f, acc.w * h);
                    }
                }
                const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
                store(row, dim, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
                if (dim == 0) store_lse(row, top, sum);
            }
        };
        if (w.c_last - w.c_first < 6) join(std::integral_constant<int, 6>());
        else join(std::integral_constant<int, 16>());
    }
}

bool encode(CUtensorMap *map, CUtensorMapDataType type, int rank, const void *base, const cuuint64_t *dims,
            const cuuint64_t *strides, const cuuint32_t *box, CUtensorMapSwizzle swizzle) {
    const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
    EncodeTiled enc = encode_fn();
    return enc && enc(map, type, rank, const_cast<void *>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                      swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

using Kernel = void (*)(RowsArgs, CUtensorMap, CUtensorMap);
template <int HD, int KIND>
Kernel kernel_of(int mode) {
    return mode == 0 ? rows_kernel<HD, KIND, 0> : mode == 1 ? rows_kernel<HD, KIND, 1> : rows_kernel<HD, KIND, 2>;
}
struct Choice {
    Kernel kernel;
    uint32_t smem;
};
Choice choose(int head_dim, int type, int mode) {
#define QDQ_ROWS(HD, KIND)                                                                      \
    Choice{kernel_of<HD, KIND>(mode), mode == 0   ? Shape<HD, KIND, 0>::kTotal                  \
                                      : mode == 1 ? Shape<HD, KIND, 1>::kTotal                  \
                                                  : Shape<HD, KIND, 2>::kTotal}
    if (head_dim == 64) return type == QDQ_E4M3 ? QDQ_ROWS(64, kE4m3) : type == QDQ_BF16 ? QDQ_ROWS(64, kBf16) : QDQ_ROWS(64, kF16);
    return type == QDQ_E4M3 ? QDQ_ROWS(128, kE4m3) : type == QDQ_BF16 ? QDQ_ROWS(128, kBf16) : QDQ_ROWS(128, kF16);
#undef QDQ_ROWS
}

}  // namespace

int rows_create(const AttendPools &p, int sm_count, RowsState **out) {
    *out = nullptr;
    RowsState *st = new (std::nothrow) RowsState();
    if (!st) return QDQ_ERR_CUDA;
    const cuuint32_t run = p.page_size < 128 ? p.page_size : 128;
    bool ok = true;
    for (int i = 0; i < 2; ++i) {
        CUtensorMap *map = i ? &st->v_map : &st->k_map;
        const void *base = i ? p.v_pages : p.k_pages;
        if (p.type == QDQ_E4M3) {
            // [page][head and position][head_dim]: a box is a run of positions of one kv head
            const cuuint64_t rows = (cuuint64_t)p.n_kv_heads * p.page_size;
            const cuuint64_t dims[3] = {(cuuint64_t)p.head_dim, rows, (cuuint64_t)p.n_layers * p.n_pages};
            const cuuint64_t strides[2] = {(cuuint64_t)p.head_dim, rows * p.head_dim};
            const cuuint32_t box[3] = {(cuuint32_t)p.head_dim, run, 1};
            ok = ok && encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, base, dims, strides, box,
                              p.head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
        } else {
            // as in qdq_attend.cu: [row / 8][64-wide block of a row][row % 8][64]
            const int blocks = p.n_kv_heads * p.head_dim / 64;
            const cuuint64_t row = (cuuint64_t)p.n_kv_heads * p.head_dim * 2;
            const cuuint64_t rows = (cuuint64_t)p.n_layers * p.n_pages * p.page_size;
            const cuuint64_t dims[4] = {64, 8, (cuuint64_t)blocks, rows / 8}, strides[3] = {row, 128, 8 * row};
            const cuuint32_t box[4] = {64, 8, (cuuint32_t)(p.head_dim / 64), run / 8};
            ok = ok && encode(map, p.type == QDQ_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                              base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
        }
    }
    st->ctas = sm_count;
    // two parts per CTA: rows of O, a maximum and a sum; the joins' counters
    const size_t parts = (size_t)sm_count * 2, n_o = parts * kMostRows * p.head_dim * 4, n_s = parts * kMostRows * 8;
    const size_t bytes = n_o + n_s + (size_t)sm_count * sizeof(unsigned);
    ok = ok && cudaMalloc((void **)&st->mem, bytes) == cudaSuccess && cudaMemset(st->mem, 0, bytes) == cudaSuccess;
    for (int mode = 0; mode < 3; ++mode) {
        const Choice c = choose(p.head_dim, p.type, mode);
        ok = ok && cudaFuncSetAttribute(c.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, c.smem) == cudaSuccess;
    }
    if (!ok) {
        cudaGetLastError();
        rows_destroy(st);
        return QDQ_ERR_CUDA;
    }
    st->part_o = (float *)st->mem;
    st->part_ml = (float2 *)(st->mem + n_o);
    st->counters = (unsigned *)(st->mem + n_o + n_s);
    *out = st;
    return QDQ_OK;
}

void rows_destroy(RowsState *st) {
    if (st == nullptr) return;
    if (st->mem) cudaFree(st->mem);
    delete st;
}

int launch_rows(const RowsState *st, const AttendArgs &a, cudaStream_t stream) {
    RowsArgs k = {};
    const AttendPools &p = *a.pools;
    k.n_seqs = a.n_seqs, k.n_tokens = a.n_tokens, k.max_pages = a.max_pages;
    k.q_start = a.q_start, k.kv_len = a.kv_len, k.page_table = a.page_table;
    k.q = (const uint16_t *)a.q, k.out = a.out, k.lse = a.lse;
    k.q_stride = a.q_stride, k.out_stride = a.out_stride, k.out_type = a.out_type;
    k.scale_log2 = (float)((double)a.scale * 1.4426950408889634);
    k.n_pages = p.n_pages, k.n_heads = p.n_heads;
    while ((1 << k.page_shift) < p.page_size) ++k.page_shift;
    k.page0 = (int64_t)a.layer * p.n_pages;
    if (p.type == QDQ_E4M3) {
        const int64_t scales = k.page0 * p.n_kv_heads * (p.page_size / 16);
        k.k_scales = p.k_scales + scales, k.v_scales = p.v_scales + scales;
    }
    const int group = p.n_heads / p.n_kv_heads;
    // Rows of a block: those of one token, of a list; else of a sequence's new tokens on average, as
    // far as 32 go.
    const int tokens = a.lists ? 1 : (a.n_tokens + a.n_seqs - 1) / a.n_seqs;
    const int64_t rows = (int64_t)tokens * group;
    const int mode = rows <= 8 ? 0 : rows <= 16 ? 1 : 2;
    k.lists = a.lists;
    k.g.group = group;
    k.g.tokens = k.g.block = a.lists ? 1 : (8 << mode) / group;
    k.g.kv_heads = p.n_kv_heads;
    k.g.window = a.window < INT32_MAX - a.n_tokens ? a.window : INT32_MAX - a.n_tokens;
    k.g.table_end = a.max_pages * p.page_size;
    k.g.list = a.lists ? a.list : 0;
    k.g.item = 2;
    k.g.page_shift = k.page_shift;
    k.part_o = st->part_o, k.part_ml = st->part_ml, k.counters = st->counters;
    const Choice c = choose(p.head_dim, p.type, mode);
    return launch_following(c.kernel, st->ctas, kThreads, c.smem, 1, stream, k, st->k_map, st->v_map);
}

int take_status_rows() {
    int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_rows_status, sizeof(int)) != cudaSuccess) {
        cudaGetLastError();
        return QDQ_ERR_CUDA;
    }
    if (v && cudaMemcpyToSymbol(g_rows_status, &zero, sizeof(int)) != cudaSuccess) {
        cudaGetLastError();
        return QDQ_ERR_CUDA;
    }
    return v;
}

}  // namespace qdq
