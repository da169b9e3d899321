// qdq_attend.cu -- causal attention of a step's new tokens over the paged cache, on the
// tcgen05 tensor cores.
//
//   o = sum_j p_j v_j / l,  p_j = 2^(c s_j - m),  l = sum_j p_j,  c = scale * log2(e)
// in one pass over the keys with a running maximum m and sum l (fp32). For a tile of 128
// rows (tokens x the query heads that share a kv head) and a tile of 128 positions,
// S = Q K^T goes to tensor memory, 128 threads take a row each, write P back, and O += P V
// accumulates in tensor memory. The maximum that p is taken against lags the true one by up
// to 2^8, so that O is rescaled a few times a row and not every tile; the factor cancels in
// o and in l.
//
// The matrix instruction takes P in the cache's 16-bit type. A weight rounded to it once is off by
// as much as a 16-bit result is by its own rounding (the whole error is 1.37 times that); two
// terms, what the type keeps of a weight and what it leaves, and a second product make the
// result's rounding all the error. Two terms are multiplied
// * for an fp32 result always: a caller who asks for more bits than the cache has gets them
//   (8191 tokens 557 us and not 433, ragged pieces 117 and not 86);
// * of a block of one tile of rows, single tokens as a rule, in any type, since it waits for memory
//   (64 single tokens bf16: 1.66e-3 and not 2.2e-3 off, 194 us and not 189; one over 131001
//   positions fp16: 2.1e-4 and not 2.9e-4, 93 and not 90; one over 520: 10.8 and not 10.2).
// Two tiles of rows with a 16-bit result have one term: the products bound them (8191 tokens bf16:
// 2.15e-3 and not 1.64e-3 off, 413 us and not the 540 that a second term takes; a window at 64
// dims 84 and not 101, ragged pieces 83 and not 103).
//
// A CTA (one per SM) has ten working warps: two groups of four that each own one S/P/O set
// (the softmax), one that issues the matrix instructions and one that issues the copies.
// * Chunks: the two sets are two tiles of rows against the same keys, so that one
//   group's exponentials run while the other's products do.
// * Few rows (one tile, as in single-token steps): the two sets take alternate key tiles
//   of the same rows; the first joins both states, which lie in tensor memory.
// Keys and values arrive page by page through one ring of slots (4-D tensor copies with
// the 128-byte swizzle: a slot is groups of 8 positions, each group head_dim / 64 blocks
// of 8 x 128 bytes, which is the operand layout for K (K-major) and for V (N-major)).
// A page that lies outside the block's positions is not read.
//
// The work of all items is dealt to the CTAs in equal contiguous ranges
// (qdq_attend_plan.h); the parts of an item that several CTAs hold are written to a
// workspace, and the CTA that finishes last (an integer counter) joins them in CTA
// order, so the result does not depend on which one that was. No CTA waits for another.
// The copying warp walks the range and publishes each piece; the rest follow it.
//
// What bounds it, as measured (GB300; 32 query and 8 kv heads of 128 unless said):
// * single tokens: HBM. 64 sequences of 30 to 8192 positions 190 to 196 us = 6.1 to 6.3 TB/s, 90
//   to 93 % of the copy rate; one sequence of 131001 positions 91.5 to 93 us, 85 % (the rest is the
//   start, the first tile's latency and the join, about 10 us, which is all of a 520-position
//   call, and the weights' second term).
// * prompts: the chain S -> softmax -> P V -> next S of each set, about 3000 clocks a tile
//   where the matrix instructions of both sets need 2048: 8191 tokens 412 us = 1.33 PFLOP/s,
//   67 % of the cuBLAS bf16 rate, tensor pipe 59 % busy. At 64 dims the softmax alone (some
//   2500 clocks a tile and set) bounds it.
//
// Values in rows of V outside the block's positions are zeroed in shared memory before
// their product (their weights are zero, but 0 x NaN is not), scores there are replaced
// by -inf whatever K held.
//
// A cache of e4m3 values (KV8): four further warps widen the copied bytes to fp16
// into the ring that the matrix instructions read (and leave out the rows outside the block's
// positions there), in units of a power of two for each tile and kind, 2^-7 of the largest scale of
// its blocks: exactly where a block's scale is 2^-22 of the largest or more, else off by less than
// 2^-31 of the tile's largest values. The units stay out of the products: the keys'
// goes into the scores' factor, and with the values' 2^e the weight that meets them is 2^(t + e - m),
// m the maximum of t + e, l the sum of those weights times 2^-e. (Block by block in the softmax, as in
// qdq_attend_rows.cu, which takes the batches of few rows, the 8191 tokens took 530 us with two
// widening warps; so 490 with four, 1.12 PFLOP/s; ragged pieces of 11 to 642 tokens 104.) The widening
// bounds it (with a quarter of it done 425 us): its instructions, and shared memory, of which a tile of
// both sets reads 192 KB of operands and moves 128 KB to be widened.
#include <cmath>
#include <cuda.h>
#include <limits>
#include <new>
#include <type_traits>

#include "qdq_attend_walk.cuh"
#include "qdq_internal.h"
#include "qdq_paged.cuh"
#include "qdq_tcgen05.cuh"

namespace qdq {

// Host state of the attention of one cache: the tensor maps of the pools and the
// workspace (partial results and the counters that the joins leave at zero).
struct AttendState {
    CUtensorMap k_map, v_map;
    char *mem = nullptr;
    float *part_o = nullptr;
    float2 *part_ml = nullptr;
    unsigned *counters = nullptr;
    int ctas = 0;
};

namespace {

__device__ int g_attend_status;

constexpr int kWarpMma = 8, kWarpLoad = 9;
constexpr int kWiden = 4;  // KV8: warps that widen the bytes, behind these
template <bool KV8>
constexpr int kThreadsOf = KV8 ? 512 : 384;
constexpr float kLag = 8.0f;  // log2 of how far the running maximum may lag
constexpr int kColO = 256;
// log2 of what weights are kept times. fp16's last step below 2^-14 is 2^-24: with the largest weight
// at 2^7 (and up to 2^15 where the maximum lags) half of it is 2^-32 of that weight, and many small
// weights beside a large one keep their sum (at 1 they would vanish below 2^-25 of it). The factor is
// in m and cancels in o and l. bf16 has fp32's range.
template <bool BF16>
constexpr float kLift = BF16 ? 0.0f : 7.0f;

struct KernelArgs {
    int n_seqs, n_tokens, max_pages;
    const int32_t *q_start, *kv_len, *page_table;
    void *out;
    float *lse;
    int64_t out_stride;
    float scale_log2;  // |scale| * log2(e); a negative scale negates Q in the instruction
    uint32_t idesc_qk, idesc_pv;
    int n_pages, page_shift, row8_layer;  // row8_layer: first group of 8 rows of the layer
    int page0, out_bf16;                  // KV8: the layer's first page; whether 16-bit results are bf16
    const uint8_t *k_scales, *v_scales;   // KV8: of the layer
    int n_heads;
    AttendGeometry g;
    float *part_o;
    float2 *part_ml;
    unsigned *counters;
};

// KV8, of a tile: the scores' factor and the values' unit, and of its eight blocks of 16 positions the
// rows that hold a position of the block and what brings them to the tile's units.
struct Note {
    float f, e, h;       // scale * log2(e) * the keys' unit; log2 of the values', and its inverse
    uint32_t reserved;
    uint16_t rows[8];
    uint16_t times[2][8];  // fp16: keys, values
};

template <int HD, bool KV8>
struct Shape {
    static constexpr int kHalves = HD / 64;
    static constexpr uint32_t kQTile = 128u * HD * 2u;
    static constexpr uint32_t kSlot = (uint32_t)kTileN * HD * 2u;
    static constexpr int kSlots = KV8 ? (HD == 128 ? 3 : 6) : HD == 128 ? 5 : 10;
    static constexpr uint32_t kGroup8 = (uint32_t)kHalves * 1024u;  // 8 positions of a slot
    static constexpr uint32_t kQ = 0, kRing = 2 * kQTile;
    // KV8: the ring of bytes as they are copied, and each of kNotes tiles' scales and rows. (A tile's notes
    // are written over when the copies are kNotes tiles on: its bytes' slots have then been taken up
    // 2 kNotes - kRawSlots copies on, whose slots of the ring were free once its weights had been used.)
    static constexpr int kRawSlots = KV8 ? (HD == 128 ? 3 : 8) : 0, kNotes = 8;
    static constexpr uint32_t kRawSlot = (uint32_t)kTileN * HD, kRaw = kRing + kSlots * kSlot;
    static_assert(!KV8 || 2 * kNotes >= kRawSlots + kSlots + 2, "kNotes");
    static constexpr uint32_t kBars = kRaw + kRawSlots * kRawSlot;
    static constexpr uint32_t kScratch = kBars + (KV8 ? 304 + 2 * 8 * 8 : 304);        // a state handed from set to set, a join's flag
    static constexpr uint32_t kStart = kScratch + 2 * 128 * 8;  // the CTA's first piece, tensor-memory base
    // Tensor memory: S of the two sets in columns 0..255, O from kColO on. A weight's two terms
    // lie over S, 64 columns each. One term alone has, at 64 dims, columns of its own, so that the
    // next S can be computed while the weights still are; at 128 dims none are left.
    static constexpr bool kApart = HD == 64;
    static constexpr int kColOne = kApart ? kColO + 2 * HD : 0, kPitchOne = kApart ? 64 : 128;
    static constexpr int kColRest = 64;  // of the second term, from the first one's
    static constexpr uint32_t kPieces = kStart + 80;
    static constexpr uint32_t kNote = (kPieces + 192 + 15) / 16 * 16;
    static constexpr uint32_t kTotal = kNote + (KV8 ? kNotes * sizeof(Note) : 0);
    static_assert(kTotal <= 232448 && sizeof(Start) + 8 <= 80 && kSlots * kSlot >= 20 * kMaxSeqs, "shared memory, Start, find_start's room");
};

// barriers (8 bytes each) at kBars
constexpr int kBarFull = 0, kBarEmpty = 10, kBarQFull = 20, kBarQEmpty = 21, kBarS = 22, kBarP = 24, kBarPv = 26,
              kBarOFree = 28, kBarDrain = 30, kBarPiece = 31, kBarPieceFree = 33,
              kBarSFree = 35, kBarRawFull = 38, kBarRawEmpty = 46;

// What the other warps need of a piece, in one of two places in shared memory.
struct Piece {
    const int32_t *pages;  // the sequence's page table
    int n;                 // key tiles; 0 ends the walk
    int t0;                // the first
    int lo, hi;            // positions that the block attends to
    int tokens, token0, p0;  // the block's tokens, the row of the first, its position
    int head;
    int tile_t0[2], tile_t1[2];
    int alt, whole;        // alternate key tiles of one tile of rows; the whole item
    int c_first, c_last;   // the CTAs that hold parts of the item, if not
};
static_assert(2 * sizeof(Piece) <= 192, "Shape::kPieces");

// The pages of key tile j that hold positions of [lo, hi): lane l's entry of the page
// table (for the tile's l-th run of min(page, 128) positions), or -1 where there is none.
// The entry is checked where it is used, a tile later, so that nothing waits for the load.
QDQ_DEV int tile_page(const KernelArgs &a, const Piece &w, int j, int run_shift) {
    const int lane = threadIdx.x & 31;
    const int64_t p = (int64_t)j * kTileN + (lane << run_shift);
    int page = -1;
    if (lane < (kTileN >> run_shift) && p < w.hi && p + (1 << run_shift) > w.lo)
        if (QDQ_CHECK(&g_attend_status, ((int)p >> a.page_shift) >= 0 && ((int)p >> a.page_shift) < a.max_pages))
            page = w.pages[(int)p >> a.page_shift];  // (inside the table: hi is)
    return page;
}

QDQ_DEV float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// KV8, bytes to fp16: the warp's kTileN / kWiden positions of each tile. A lane takes 16 bytes of a row, which
// are two 16-byte pieces of the widened row. Eight lanes that go to shared memory together have four
// pieces of each of two neighbouring rows (of 128 dims, the other half of the second one): they read 128
// bytes of different banks, and store to the eight places of the swizzle.
template <int HD>
QDQ_DEV void widen(char *smem, const Piece *pieces, int mine, int *status) {
    using L = Shape<HD, true>;
    constexpr int kChunks = HD / 16, kRows = 32 / kChunks;  // lanes of a row, rows at once
    constexpr int kDeep = HD == 128 ? 4 : 2;                 // loads in flight
    const uint32_t sb = smem_u32(smem);
    auto bar = [&](int i) { return sb + L::kBars + 8u * i; };
    const int lane = threadIdx.x & 31;
    const int sub = HD == 128 ? (lane >> 4) * 2 + ((lane >> 2) & 1) : lane / kChunks;
    const int chunk = HD == 128 ? (lane & 3) | (((lane >> 2) ^ (lane >> 3)) & 1) << 2 : lane % kChunks;
    const uint32_t piece = (2 * chunk) & 7;
    uint32_t seq_no = 0;
    for (uint32_t items = 0;; ++items) {
        mbar_wait(bar(kBarPiece + (items & 1)), (items >> 1) & 1, status);
        const int n = pieces[items & 1].n;
        __syncwarp();
        if (n == 0) break;
        if (lane == 0) mbar_arrive(bar(kBarPieceFree + (items & 1)));
        for (int x = 0; x < 2 * n; ++x, ++seq_no) {
            const int raw = seq_no % L::kRawSlots, slot = seq_no % L::kSlots;
            mbar_wait(bar(kBarRawFull + raw), (seq_no / L::kRawSlots) & 1, status);
            mbar_wait(bar(kBarEmpty + slot), ((seq_no / L::kSlots) & 1) ^ 1, status);
            const Note &note = reinterpret_cast<const Note *>(smem + L::kNote)[(seq_no >> 1) % L::kNotes];
            const uint16_t *times = note.times[seq_no & 1];
            const uint32_t from = sb + L::kRaw + raw * L::kRawSlot + chunk * 16;
            const uint32_t to = sb + L::kRing + slot * L::kSlot + (HD == 128 ? (chunk / 4) * 1024u : 0u);
#pragma unroll 1
            for (int r0 = mine * (kTileN / kWiden); r0 < (mine + 1) * (kTileN / kWiden); r0 += kDeep * kRows) {
                uint4 v[kDeep];
#pragma unroll
                for (int y = 0; y < kDeep; ++y) v[y] = lds128(from + (r0 + y * kRows + sub) * HD);
                const __half2 by = __half2half2(__ushort_as_half(times[r0 / 16]));
                const uint32_t rows = note.rows[r0 / 16];
                if (rows != 0xFFFFu) {
#pragma unroll
                    for (int y = 0; y < kDeep; ++y)
                        if (!((rows >> (r0 % 16 + y * kRows + sub)) & 1)) v[y] = make_uint4(0, 0, 0, 0);
                }
                static_assert(16 % (kDeep * kRows) == 0, "one block at a time");
#pragma unroll
                for (int y = 0; y < kDeep; ++y) {
                    const int r = r0 + y * kRows + sub;
                    uint4 f, g;
                    e4m3x4_to_f16(v[y].x, f.x, f.y);
                    e4m3x4_to_f16(v[y].y, f.z, f.w);
                    e4m3x4_to_f16(v[y].z, g.x, g.y);
                    e4m3x4_to_f16(v[y].w, g.z, g.w);
                    auto scaled = [&](uint32_t &u) { *reinterpret_cast<__half2 *>(&u) = __hmul2(*reinterpret_cast<__half2 *>(&u), by); };
                    scaled(f.x), scaled(f.y), scaled(f.z), scaled(f.w), scaled(g.x), scaled(g.y), scaled(g.z), scaled(g.w);
                    const uint32_t row = to + (r >> 3) * L::kGroup8 + (r & 7) * 128;
                    const uint32_t first = row + ((piece ^ (r & 7)) << 4), second = first ^ 16;
                    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(first), "r"(f.x), "r"(f.y), "r"(f.z), "r"(f.w) : "memory");
                    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(second), "r"(g.x), "r"(g.y), "r"(g.z), "r"(g.w) : "memory");
                }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(kBarFull + slot));
                mbar_arrive(bar(kBarRawEmpty + raw));
            }
        }
    }
}

template <int HD, bool BF16, bool OUT32, bool KV8>
QDQ_DEV void attend(const KernelArgs &a, const CUtensorMap &q_map, const CUtensorMap &k_map, const CUtensorMap &v_map) {
    using L = Shape<HD, KV8>;
    constexpr int kThreads = kThreadsOf<KV8>;
    using F16 = Float16<typename std::conditional<BF16, __nv_bfloat16, __half>::type>;
    // Whether both terms of the weights are multiplied, with the sets on alternate key tiles and on two
    // tiles of rows.
    using TwoAlternate = std::true_type;
    using TwoTiles = std::bool_constant<OUT32>;
    extern __shared__ __align__(1024) char smem[];
    const uint32_t sb = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int *status = &g_attend_status;
    Start *start = reinterpret_cast<Start *>(smem + L::kStart);
    auto bar = [&](int i) { return sb + L::kBars + 8u * i; };
    follow_last_kernel();

    if (threadIdx.x == 0) {
        for (int i = 0; i < L::kSlots; ++i) {
            mbar_init(bar(kBarFull + i), KV8 ? kWiden : 1);
            mbar_init(bar(kBarEmpty + i), 1);
        }
        for (int i = 0; i < L::kRawSlots; ++i) {
            mbar_init(bar(kBarRawFull + i), 1);
            mbar_init(bar(kBarRawEmpty + i), kWiden);
        }
        mbar_init(bar(kBarQFull), 1);
        mbar_init(bar(kBarQEmpty), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(kBarS + i), 1);
            mbar_init(bar(kBarP + i), 4);
            mbar_init(bar(kBarPv + i), 1);
            mbar_init(bar(kBarOFree + i), 4);
            mbar_init(bar(kBarSFree + i), 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(kBarPiece + i), 1);
            mbar_init(bar(kBarPieceFree + i), 9 + (KV8 ? kWiden : 0));
        }
        mbar_init(bar(kBarDrain), 1);
        fence_mbar_init();
    }
    find_start<kThreads>(a, smem + L::kRing, start);
    if (!start->live) return;
    const Start s0 = *start;
    __syncthreads();
    fence_async_smem();  // the ring's memory goes over to the copies
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kStart);
    if (warp == kWarpMma) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *reinterpret_cast<volatile uint32_t *>(tmem_slot), 0);

    const int run_shift = min(a.page_shift, 7), tq = a.g.tokens;
    Piece *pieces = reinterpret_cast<Piece *>(smem + L::kPieces);

    // Registers: launched with 168 a thread, three warpgroups of them; the softmax groups go
    // up to 216, which holds a row's 128 scores without spilling, and the third, of which two
    // warps work, comes down to 72: 2 x 216 + 72 = 3 x 168 (the build refuses to make a library
    // with another number, attend_create to run one). KV8: launched with 128 a thread, four warpgroups,
    // 2 x 208 + 2 x 48 = 4 x 128.
    if (warp >= kWarpMma) {
        if constexpr (!KV8) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        if (warp == kWarpLoad) {
            // ---- copies ---------------------------------------------------------------------
            const uint32_t q_rows = (uint32_t)(tq * a.g.group), run_bytes = (L::kGroup8 << run_shift) >> 3;
            uint32_t seq_no = 0, items = 0;
            for (Walk w(a, s0);; w.next(a), ++items) {
                const int n = w.n, t0 = w.t_beg();
                Piece &piece = pieces[items & 1];
                mbar_wait(bar(kBarPieceFree + (items & 1)), ((items >> 1) & 1) ^ 1, status);
                if (lane == 0) {
                    piece.n = n;
                    if (n) {
                        piece.pages = w.pages;
                        piece.t0 = t0;
                        piece.lo = w.b.lo, piece.hi = w.b.hi;
                        piece.tokens = w.b.i1 - w.b.i0, piece.token0 = w.first + w.b.i0, piece.p0 = w.kv - w.count + w.b.i0;
                        piece.head = w.head;
                        for (int i = 0; i < 2; ++i) piece.tile_t0[i] = w.b.tile_t0[i], piece.tile_t1[i] = w.b.tile_t1[i];
                        piece.alt = block_alternates(a.g, w.b);
                        piece.whole = w.whole();
                        if (!w.whole()) {
                            piece.c_first = range_owner(s0.total, s0.ctas, w.item + kItemUnits);
                            piece.c_last = range_owner(s0.total, s0.ctas, w.item + item_units(w.b) - 1);
                        }
                    }
                    mbar_arrive(bar(kBarPiece + (items & 1)));
                }
                __syncwarp();
                if (!w.more()) break;
                const int tiles = w.b.i1 - w.b.i0 > tq ? 2 : 1;
                mbar_wait(bar(kBarQEmpty), (items & 1) ^ 1, status);
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar(kBarQFull), tiles * L::kHalves * q_rows * 128u);
                    for (int i = 0; i < tiles; ++i)
                        for (int h = 0; h < L::kHalves; ++h)
                            if (QDQ_CHECK(status, w.first + w.b.i0 + i * tq < a.n_tokens && (w.head + 1) * a.g.group <= a.n_heads &&
                                                      q_rows * 128u <= 16384u))
                                tma_load_3d(sb + L::kQ + i * L::kQTile + h * 16384u, &q_map, h * 64, w.head * a.g.group,
                                            w.first + w.b.i0 + i * tq, bar(kBarQFull));
                }
                int page = tile_page(a, piece, t0, run_shift);
                for (int j = 0; j < n; ++j) {
                    const int here = (unsigned)page < (unsigned)a.n_pages ? page : -1;
                    if (j + 1 < n) page = tile_page(a, piece, t0 + j + 1, run_shift);
                    const unsigned have = __ballot_sync(0xFFFFFFFFu, here >= 0);
                    const uint32_t bytes = __popc(have) * run_bytes;
                    if constexpr (KV8) {
                        const uint32_t raw_run = (uint32_t)HD << run_shift;
                        const int in_page = ((t0 + j) * kTileN + (lane << run_shift)) & ((1 << a.page_shift) - 1);
                        // block `lane` of the tile lies in run lane * 16 >> run_shift
                        const int run = ((lane & 7) << 4) >> run_shift, p0 = (t0 + j) * kTileN + ((lane & 7) << 4);
                        const int run_page = __shfl_sync(0xFFFFFFFFu, here, run);
                        constexpr int kNone = -1000;
                        int ek = kNone, ev = kNone;
                        if (run_page >= 0 && lane < 8) {
                            const int64_t at = (((int64_t)run_page * a.g.kv_heads + w.head) << (a.page_shift - 4)) +
                                               ((p0 & ((1 << a.page_shift) - 1)) >> 4);
                            ek = exponent_of(a.k_scales[at]), ev = exponent_of(a.v_scales[at]);
                        }
                        const int all_k = __reduce_max_sync(0xFFFFFFFFu, ek), all_v = __reduce_max_sync(0xFFFFFFFFu, ev);
                        const int unit_k = all_k == kNone ? 0 : all_k - 7, unit_v = all_v == kNone ? 0 : all_v - 7;
                        // 2^d in fp16, d at most 7
                        auto half_power = [](int d) { return (uint16_t)(d >= -14 ? (15 + d) << 10 : d >= -24 ? 1 << (24 + d) : 0); };
#pragma unroll
                        for (int kv = 0; kv < 2; ++kv, ++seq_no) {
                            const int slot = seq_no % L::kRawSlots;
                            mbar_wait(bar(kBarRawEmpty + slot), ((seq_no / L::kRawSlots) & 1) ^ 1, status);
                            if (here >= 0 && QDQ_CHECK(status, here < a.n_pages && w.head < a.g.kv_heads && lane * raw_run + raw_run <= L::kRawSlot))
                                tma_load_3d(sb + L::kRaw + slot * L::kRawSlot + (uint32_t)lane * raw_run, kv ? &v_map : &k_map, 0,
                                            (w.head << a.page_shift) + in_page, a.page0 + here, bar(kBarRawFull + slot));
                            if (kv == 0 && lane < 8) {
                                Note *note = reinterpret_cast<Note *>(smem + L::kNote) + (seq_no >> 1) % L::kNotes;
                                const int b = min(max(w.b.lo - p0, 0), 16), e = min(max(w.b.hi - p0, 0), 16);
                                if (lane == 0) note->f = a.scale_log2 * power_of_two(unit_k), note->e = (float)unit_v, note->h = power_of_two(-unit_v);
                                note->times[0][lane] = half_power(ek - unit_k), note->times[1][lane] = half_power(ev - unit_v);
                                note->rows[lane] = run_page >= 0 && e > b ? (uint16_t)((1u << e) - (1u << b)) : 0;
                            }
                            __syncwarp();
                            if (lane == 0) mbar_arrive_expect_tx(bar(kBarRawFull + slot), __popc(have) * raw_run);
                        }
                        continue;
                    }
                    // the lane's run of positions: its first group of 8 rows in the pools
                    const int in_page = ((t0 + j) * kTileN + (lane << run_shift)) & ((1 << a.page_shift) - 1);
                    const int row8 = a.row8_layer + (int)((((int64_t)here << a.page_shift) + in_page) >> 3);
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv, ++seq_no) {
                        const int slot = seq_no % L::kSlots;
                        mbar_wait(bar(kBarEmpty + slot), ((seq_no / L::kSlots) & 1) ^ 1, status);
                        if (lane == 0) mbar_arrive_expect_tx(bar(kBarFull + slot), bytes);
                        __syncwarp();
                        if (here >= 0 &&
                            QDQ_CHECK(status, row8 >= a.row8_layer && w.head < a.g.kv_heads && lane * run_bytes + run_bytes <= L::kSlot &&
                                                  row8 + (1 << run_shift >> 3) <= a.row8_layer + (int)(((int64_t)a.n_pages << a.page_shift) >> 3)))
                            tma_load_4d(sb + L::kRing + slot * L::kSlot + (uint32_t)lane * run_bytes, kv ? &v_map : &k_map, 0,
                                        0, w.head * L::kHalves, row8, bar(kBarFull + slot));
                    }
                }
            }
            // every copy has landed before the CTA can end, also after a wait that ran out
            constexpr uint32_t kLast = KV8 ? L::kRawSlots : L::kSlots;
            for (uint32_t i = seq_no < kLast ? 0 : seq_no - kLast; i < seq_no; ++i)
                mbar_wait(bar((KV8 ? kBarRawFull : kBarFull) + i % kLast), (i / kLast) & 1, status);
            if (items) mbar_wait(bar(kBarQFull), (items - 1) & 1, status);
        } else if (warp == kWarpMma) {
            // ---- matrix instructions ----------------------------------------------------------
            // Everything that an instruction's operands depend on is kept known to be the same in
            // every lane (values out of memory go through a shuffle), or each operand costs moves.
            constexpr uint32_t q_hi = sdesc_hi(1024), kv_hi = sdesc_hi(L::kGroup8);
            uint32_t items = 0, np = 0, no = 0, nf = 0;  // np, no, nf: bit i is the phase of set i's barrier
            const uint32_t q_lo = sdesc_lo(16) | ((sb + L::kQ) >> 4);
            const uint32_t k_lo = sdesc_lo(16) | ((sb + L::kRing) >> 4), v_lo = sdesc_lo(1024) | ((sb + L::kRing) >> 4);
            auto uniform = [](int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); };
            // A place in the ring; keys and values alternate, so the next of a kind is two on.
            struct Place {
                int slot;
                uint32_t phase;
                QDQ_DEV void step(int by) {
                    slot += by;
                    if (slot >= L::kSlots) slot -= L::kSlots, phase ^= 1;
                }
            };
            auto full = [&](const Place &p) { mbar_wait(bar(kBarFull + p.slot), p.phase, status); };
            auto release = [&](const Place &p) {
                if (elect_one()) mma_commit(bar(kBarEmpty + p.slot));
                __syncwarp();
            };
            // S_i = Q K^T with rows of tile qi (in an elected lane)
            auto qk = [&](int i, int qi, const Place &p) {
                const uint32_t kd = k_lo + (uint32_t)p.slot * (L::kSlot >> 4), qd = q_lo + qi * (L::kQTile >> 4);
#pragma unroll
                for (int k = 0; k < HD / 16; ++k)
                    mma_ss(tmem + 128u * i, desc64(qd + (k / 4) * 1024u + (k % 4) * 2u, q_hi),
                              desc64(kd + (k / 4) * 64u + (k % 4) * 2u, kv_hi), a.idesc_qk, k > 0);
                mma_commit(bar(kBarS + i));
            };
            auto begin = [&](int i, int qi, const Place &p) {
                if (elect_one()) qk(i, qi, p);
                __syncwarp();
            };
            // O_i (+)= P_i V, and, if there is a next tile, its S_i: once the last one has been read, or
            // (over P_i, which the instructions before it have read) right behind
            auto turn = [&](int i, int qi, const Place &v, bool first, const Place &k_next, bool more, auto two) {
                constexpr bool apart = L::kApart && !decltype(two)::value;
                const uint32_t p = tmem + (two.value ? 128u * i : (uint32_t)(L::kColOne + L::kPitchOne * i));
                const uint32_t vd = v_lo + (uint32_t)v.slot * (L::kSlot >> 4);
                if (first) {
                    mbar_wait(bar(kBarOFree + i), ((no >> i) & 1) ^ 1, status);
                    no ^= 1u << i;
                }
                if (apart) {
                    mbar_wait_spin(bar(kBarSFree + i), (nf >> i) & 1, status);
                    nf ^= 1u << i;
                    tc_fence_after();
                    if (more) begin(i, qi, k_next);
                }
                mbar_wait_spin(bar(kBarP + i), (np >> i) & 1, status);
                np ^= 1u << i;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < kTileN / 16; ++k)
                        mma_ts(tmem + kColO + (uint32_t)HD * i, p + 8u * k,
                                  desc64(vd + k * (2 * L::kGroup8 >> 4), kv_hi), a.idesc_pv, !first || k > 0);
                    if constexpr (two.value) {
#pragma unroll
                        for (int k = 0; k < kTileN / 16; ++k)
                            mma_ts(tmem + kColO + (uint32_t)HD * i, p + L::kColRest + 8u * k,
                                      desc64(vd + k * (2 * L::kGroup8 >> 4), kv_hi), a.idesc_pv, true);
                    }
                    mma_commit(bar(kBarPv + i));
                    if (!apart && more) qk(i, qi, k_next);
                }
                __syncwarp();
            };
            Place kp = {0, 0}, vp = {1, 0};
            for (;; ++items) {
                const Piece &w = pieces[items & 1];
                mbar_wait(bar(kBarPiece + (items & 1)), (items >> 1) & 1, status);
                const int n = uniform(w.n), t0 = uniform(w.t0);
                if (n == 0) break;
                mbar_wait(bar(kBarQFull), items & 1, status);
                if (uniform(w.alt)) {
                    for (int k = 0; k < 2 && k < n; ++k, kp.step(2)) {
                        full(kp);
                        begin(k, 0, kp);
                        release(kp);
                    }
                    for (int k = 0; k < n; ++k, vp.step(2)) {
                        // (few rows wait for memory: no key is waited for ahead of a product that could run)
                        full(vp);
                        turn(k & 1, 0, vp, k < 2, kp, false, TwoAlternate());
                        release(vp);
                        if (k + 2 < n) {
                            full(kp);
                            begin(k & 1, 0, kp);
                            release(kp);
                            kp.step(2);
                        }
                    }
                } else {
                    // the sets' key tiles, counted from the piece's first
                    const int b0 = uniform(w.tile_t0[0] - t0), e0 = uniform(min(w.tile_t1[0] - t0, n));
                    const int b1 = uniform(w.tile_t0[1] - t0), e1 = uniform(min(w.tile_t1[1] - t0, n));
                    bool begun0 = false, begun1 = false;
                    full(kp);
                    if (b0 <= 0 && 0 < e0) begin(0, 0, kp);
                    if (b1 <= 0 && 0 < e1) begin(1, 1, kp);
                    release(kp);
                    kp.step(2);
                    for (int k = 0; k < n; ++k, vp.step(2)) {
                        const bool more = k + 1 < n;
                        const bool on0 = b0 <= k && k < e0, next0 = b0 <= k + 1 && k + 1 < e0;
                        const bool on1 = b1 <= k && k < e1, next1 = b1 <= k + 1 && k + 1 < e1;
                        full(vp);
                        if (more) full(kp);
                        if (on0) {
                            turn(0, 0, vp, !begun0, kp, next0, TwoTiles());
                            begun0 = true;
                        } else if (next0) {
                            begin(0, 0, kp);
                        }
                        if (on1) {
                            turn(1, 1, vp, !begun1, kp, next1, TwoTiles());
                            begun1 = true;
                        } else if (next1) {
                            begin(1, 1, kp);
                        }
                        release(vp);
                        if (more) {
                            release(kp);
                            kp.step(2);
                        }
                    }
                }
                if (elect_one()) {
                    mma_commit(bar(kBarQEmpty));
                    mbar_arrive(bar(kBarPieceFree + (items & 1)));
                }
                __syncwarp();
            }
            if (elect_one()) mma_commit(bar(kBarDrain));
            __syncwarp();
            mbar_wait(bar(kBarDrain), 0, status);
        } else if constexpr (KV8) {
            if (warp <= kWarpLoad + kWiden) widen<HD>(smem, pieces, warp - kWarpLoad - 1, status);
        }
    } else {
        if constexpr (!KV8) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        // ---- softmax, output ----------------------------------------------------------------
        const int i = warp >> 2, r = threadIdx.x & 127;  // set; row = tensor-memory lane
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const uint32_t t_s = tmem + lanes + 128u * i, t_o = tmem + lanes + kColO + (uint32_t)HD * i;
        const float c = a.scale_log2;
        const uint64_t c2 = pack2(c, c);
        float2 *scratch = reinterpret_cast<float2 *>(smem + L::kScratch) + i * 128;
        const int r_token = r / a.g.group, r_head = r - r_token * a.g.group;
        uint32_t seq_no = 0, ns = 0, npv = 0;
        bool lent = false;  // the second set's scratch holds a state that the first may not have read
        for (uint32_t items = 0;; ++items) {
            const Piece &w = pieces[items & 1];
            mbar_wait(bar(kBarPiece + (items & 1)), (items >> 1) & 1, status);
            const int n = w.n, t0 = w.t0;
            if (n == 0) break;
            const auto done = [&] {  // the piece's place is free again
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kBarPieceFree + (items & 1)));
            };
            const uint32_t base = seq_no;
            seq_no += 2 * n;
            const bool alt = w.alt != 0, apart = L::kApart && !TwoTiles::value && !alt;
            // this set's rows and key tiles of the piece
            const int qi = alt ? 0 : i, tokens = min(tq, w.tokens - qi * tq), rows = tokens * a.g.group;
            if (rows <= 0) {
                done();
                continue;
            }
            const bool idle = (warp & 3) * 32 >= rows;  // no row of the warp's lanes is one
            // (lanes past the last row hold the next sequence's queries or what was in the tile: they
            // have no say in when the maximum is raised)
            const float lag = r < rows ? kLag : INFINITY;
            const int step = alt ? 2 : 1;
            const int j0 = alt ? t0 + i : max(t0, w.tile_t0[qi]);
            const int j1 = alt ? t0 + n : min(t0 + n, w.tile_t1[qi]);
            const int p_first = w.p0 + qi * tq;
            int lo, hi, lo_last, hi_first, x;
            span(a.g, p_first + min(r_token, tokens - 1), 1, lo, hi);
            span(a.g, p_first, 1, x, hi_first);
            span(a.g, p_first + tokens - 1, 1, lo_last, x);

            float m = -INFINITY, l = 0.0f;
            int page = j0 < j1 ? tile_page(a, w, j0, run_shift) : -1;
            for (int j = j0; j < j1; j += step) {
                const unsigned have = __ballot_sync(0xFFFFFFFFu, (unsigned)page < (unsigned)a.n_pages);
                if (j + step < j1) page = tile_page(a, w, j + step, run_shift);
                const int p0 = j * kTileN;
                const unsigned all = (1u << (kTileN >> run_shift)) - 1;
                const bool dirty = have != all || p0 < w.lo || p0 + kTileN > w.hi;
                const bool masked = dirty || p0 < lo_last || p0 + kTileN > hi_first;
                // columns 32 k .. 32 k + 31 of a masked tile: those outside [lo, hi) and whole
                // runs of absent pages become -inf
                auto mask = [&](float *s, int k) {
                    const int b = min(max(lo - p0 - 32 * k, 0), 32), e = min(max(hi - p0 - 32 * k, 0), 32);
                    uint32_t keep = e > b ? (uint32_t)(((1ull << e) - 1) & ~((1ull << b) - 1)) : 0u;
                    if (run_shift >= 5) keep = (have >> ((32 * k) >> run_shift)) & 1 ? keep : 0u;
                    else keep &= ((have >> (2 * k)) & 1 ? 0xFFFFu : 0u) | ((have >> (2 * k + 1)) & 1 ? 0xFFFF0000u : 0u);
#pragma unroll
                    for (int y = 0; y < 32; ++y) s[y] = (keep >> y) & 1 ? s[y] : -INFINITY;
                };
                mbar_wait_spin(bar(kBarS + i), ns++ & 1, status);
                tc_fence_after();
                const auto s_read = [&] {  // S may be overwritten
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kBarSFree + i));
                };
                const auto p_free = [&] {  // the last tile's weights have been read
                    if (npv == 0) return;
                    mbar_wait_spin(bar(kBarPv + i), (npv - 1) & 1, status);
                    tc_fence_after();
                };
                if (apart && idle) {
                    // (S comes ahead of the last tile's P V, so a warp without rows has to wait here
                    // too, or its arrival would count for the last tile's weights)
                    s_read();
                    p_free();
                }
                if (!idle) {
                    float s[4][32], mx[4];
                    float f_tile = c, e_tile = 0.0f, h_tile = 1.0f;
                    if constexpr (KV8) {
                        const uint4 x = lds128(sb + L::kNote + ((base >> 1) + (j - t0)) % L::kNotes * (uint32_t)sizeof(Note));
                        f_tile = __uint_as_float(x.x), e_tile = __uint_as_float(x.y), h_tile = __uint_as_float(x.z);
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) tc_ld32(t_s + 32 * k, s[k]);
#pragma unroll
                    for (int k = 0; k < 4; ++k) tc_wait_ld<32>(s[k]);
                    if (masked) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) mask(s[k], k);
                    }
#pragma unroll
                    for (int y = 0; y < 4; ++y) mx[y] = fmaxf(s[y][0], s[y][1]);
#pragma unroll
                    for (int k = 2; k < 32; k += 2)
#pragma unroll
                        for (int y = 0; y < 4; ++y) mx[y] = max3(mx[y], s[y][k], s[y][k + 1]);
                    const float unit = KV8 ? 1.0f : c;  // of the maximum, in weights' exponents
                    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    const float mn = fmaxf(m, KV8 ? fmaf(top, f_tile, e_tile) : top);
                    if (j == j0) {
                        m = mn;
                    } else if (__any_sync(0xFFFFFFFFu, (mn - m) * unit > lag)) {
                        // raise the maximum of the warp's rows: O and l change units
                        const float f = mn == -INFINITY ? 1.0f : ex2((m - mn) * unit);
                        m = mn;
                        l *= f;
                        mbar_wait_spin(bar(kBarPv + i), (npv - 1) & 1, status);
                        tc_fence_after();
                        const uint64_t f2 = pack2(f, f);
#pragma unroll
                        for (int k = 0; k < HD / 16; ++k) {
                            float o[16];
                            tc_ld16(t_o + 16 * k, o);
                            tc_wait_ld<16>(o);
#pragma unroll
                            for (int y = 0; y < 16; y += 2) {
                                const uint64_t v = fmul2(pack2(o[y], o[y + 1]), f2);
                                o[y] = lo_of(v);
                                o[y + 1] = hi_of(v);
                            }
                            tc_st16(t_o + 16 * k, reinterpret_cast<uint32_t *>(o));
                        }
                        tmem_wait_st();
                    }
                    const float mc = m == -INFINITY ? 0.0f : fmaf(m, unit, -kLift<BF16>);
                    const uint64_t mc2 = KV8 ? pack2(e_tile - mc, e_tile - mc) : pack2(-mc, -mc), f2 = KV8 ? pack2(f_tile, f_tile) : c2;
                    uint64_t sum[2] = {};
                    auto weights = [&](const float *s, uint32_t *to, uint32_t *left, auto rest) {
#pragma unroll
                        for (int k = 0; k < 32; k += 2) {
                            const uint64_t e = ffma2(pack2(s[k], s[k + 1]), f2, mc2);
                            const float p = ex2(lo_of(e)), q = ex2(hi_of(e));
                            sum[(k / 2) & 1] = fadd2(sum[(k / 2) & 1], pack2(p, q));
                            to[k / 2] = F16::pack(p, q);
                            if constexpr (rest.value) {
                                const float2 h = F16::unpack(to[k / 2]);
                                left[k / 2] = F16::pack(p - h.x, q - h.y);
                            }
                        }
                    };
                    auto store = [&](auto rest) {
                        uint32_t u[32], left[32];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            weights(s[2 * h], u, left, rest);
                            weights(s[2 * h + 1], u + 16, left + 16, rest);
                            if constexpr (rest.value) {
                                tc_st32(t_s + 32 * h, u);
                                tc_st32(t_s + L::kColRest + 32 * h, left);
                            } else {
                                if (L::kApart && h == 0) p_free();
                                tc_st32(tmem + lanes + L::kColOne + L::kPitchOne * i + 32 * h, u);
                            }
                        }
                    };
                    if (apart) s_read();
                    if (!alt) store(TwoTiles());
                    else store(TwoAlternate());
                    const uint64_t t = fadd2(sum[0], sum[1]);
                    l = KV8 ? fmaf(lo_of(t) + hi_of(t), h_tile, l) : l + (lo_of(t) + hi_of(t));
                }
                if (!KV8 && dirty) {
                    // zero the rows of V that hold no position of the block (row r of the slot)
                    const uint32_t vs = base + 2 * (j - t0) + 1;
                    mbar_wait(bar(kBarFull + vs % L::kSlots), (vs / L::kSlots) & 1, status);
                    if (p0 + r < w.lo || p0 + r >= w.hi || !((have >> (r >> run_shift)) & 1)) {
                        char *row = smem + L::kRing + (vs % L::kSlots) * L::kSlot + (r / 8) * L::kGroup8 + (r % 8) * 128;
#pragma unroll
                        for (int k = 0; k < HD / 8; ++k)
                            if (QDQ_CHECK(status, row + (k / 8) * 1024 + (k % 8) * 16 + 16 <= smem + L::kBars))
                                *reinterpret_cast<uint4 *>(row + (k / 8) * 1024 + (k % 8) * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_async_smem();
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kBarP + i));
                ++npv;
            }

            // ---- the piece's end ------------------------------------------------------------
            const bool any = j1 > j0;
            float mc = m == -INFINITY ? -INFINITY : fmaf(m, KV8 ? 1.0f : c, -kLift<BF16>), f0 = 1.0f, f1 = 0.0f;
            if (any) {
                mbar_wait_spin(bar(kBarPv + i), (npv - 1) & 1, status);
                tc_fence_after();
            }
            const bool both = alt && n >= 2;  // two states of the same rows
            if (alt && i == 1) {
                if (lent) named_bar_sync(4, 256);
                lent = both;
                if (both) {
                    scratch[r] = make_float2(mc, l);
                    tc_fence_before();
                    named_bar_arrive(3, 256);
                }
                done();
                continue;
            }
            if (both) {
                named_bar_sync(3, 256);
                tc_fence_after();
                const float2 o = scratch[128 + r];
                named_bar_arrive(4, 256);
                const float M = fmaxf(mc, o.x);
                f0 = l != 0.0f ? ex2(mc - M) : 0.0f;
                f1 = o.y != 0.0f ? ex2(o.x - M) : 0.0f;
                l = l * f0 + o.y * f1;
                mc = M;
            }
            // 32 columns of the row's accumulator (both sets' where they share the rows)
            auto read = [&](int k, float *o) {
                if (!any) {
#pragma unroll
                    for (int y = 0; y < 32; ++y) o[y] = 0.0f;
                    return;
                }
                tc_ld32(t_o + 32 * k, o);
                tc_wait_ld<32>(o);
                if (both) {
                    float e[32];
                    tc_ld32(t_o + HD + 32 * k, e);
                    tc_wait_ld<32>(e);
#pragma unroll
                    for (int y = 0; y < 32; ++y) o[y] = fmaf(e[y], f1, o[y] * f0);
                }
            };
            auto read_done = [&] {  // the next piece may overwrite the accumulators
                tc_fence_before();
                __syncwarp();
                if (any && lane == 0) {
                    mbar_arrive(bar(kBarOFree + i));
                    if (both) mbar_arrive(bar(kBarOFree + 1));
                }
            };
            const int64_t first_token = w.token0 + qi * tq, first_head = (int64_t)w.head * a.g.group;
            auto put8 = [&](int64_t at, const float *o, float f) {
                if (!QDQ_CHECK(status, at >= 0 && at % 8 == 0 && at + 8 <= (a.n_tokens - 1) * a.out_stride + (int64_t)a.n_heads * HD)) return;
                if constexpr (OUT32) {
                    float4 *to = reinterpret_cast<float4 *>((float *)a.out + at);
                    to[0] = make_float4(o[0] * f, o[1] * f, o[2] * f, o[3] * f);
                    to[1] = make_float4(o[4] * f, o[5] * f, o[6] * f, o[7] * f);
                } else {
                    auto pack = [&](float x, float y) {
                        return KV8 && a.out_bf16 ? Float16<__nv_bfloat16>::pack(x, y) : F16::pack(x, y);
                    };
                    *reinterpret_cast<uint4 *>((uint16_t *)a.out + at) =
                        make_uint4(pack(o[0] * f, o[1] * f), pack(o[2] * f, o[3] * f), pack(o[4] * f, o[5] * f), pack(o[6] * f, o[7] * f));
                }
            };
            const float ln2 = 0.6931471805599453f;
            if (w.whole) {
                const float inv = l != 0.0f ? 1.0f / l : 0.0f;
                const int64_t token = first_token + r_token, head = first_head + r_head;
                const int64_t at = token * a.out_stride + head * HD;
                if (!idle) {
#pragma unroll
                    for (int k = 0; k < HD / 32; ++k) {
                        float o[32];
                        read(k, o);
                        if (r < rows) {
#pragma unroll
                            for (int y = 0; y < 32; y += 8) {
                                if (l == 0.0f) {
#pragma unroll
                                    for (int z = 0; z < 8; ++z) o[y + z] = 0.0f;  // (nothing to attend to)
                                }
                                put8(at + 32 * k + y, o + y, inv);
                            }
                        }
                    }
                }
                read_done();
                if (a.lse && r < rows) a.lse[token * a.n_heads + head] = l != 0.0f ? (mc + log2f(l)) * ln2 : -INFINITY;
                done();
                continue;
            }
            // partial state: O as [column / 4][row][4], so that rows of a warp are contiguous
            const int c_first = w.c_first, c_last = w.c_last;
            done();
            auto part_of = [&](int cta) {
                const int part = (cta * 2 + (cta == c_first ? 1 : 0)) * 2 + i;
                return QDQ_CHECK(status, part >= 0 && part < 4 * (int)gridDim.x) ? part : i;
            };
            // One more part onto a joined state, in CTA order on every path: g and f are the factors
            // of what is there and of what comes.
            auto onto = [](float2 p, float &M, float &S, float &g, float &f) {
                const float mn = fmaxf(M, p.x);
                g = M == -INFINITY ? 0.0f : ex2(M - mn);
                f = p.y != 0.0f ? ex2(p.x - mn) : 0.0f;  // (a sum that is no number stays none)
                M = mn;
                S = fmaf(S, g, p.y * f);
            };
            if (lent) {
                named_bar_sync(4, 256);
                lent = false;
            }
            // Many rows, and the other parts are all written: this one is joined as it is, a thread
            // its row (writing it and reading all back costs some 15 000 clocks at 128 rows).
            unsigned *counter = a.counters + (QDQ_CHECK(status, c_first >= 0 && c_first < (int)gridDim.x) ? 2 * c_first : 0) + i;
            const int pieces = rows * (HD / 8);
            if (pieces > 256) {
                if (r == 0) {
                    const bool rest = ld_acquire_gpu(counter) == (unsigned)(c_last - c_first);
                    if (rest) *counter = 0;
                    scratch[0].x = rest ? 1.0f : 0.0f;
                }
                named_bar_sync(1 + i, 128);
                const bool rest = scratch[0].x != 0.0f;
                named_bar_sync(1 + i, 128);
                if (rest) {
                    const int row = min(r, rows - 1);
                    const int64_t token = first_token + r_token, head = first_head + r_head;
                    float M, S;
#pragma unroll 1
                    for (int k = 0; k < HD / 32; ++k) {
                        float acc[32] = {};
                        M = -INFINITY, S = 0.0f;
                        for (int cta = c_first; cta <= c_last; ++cta) {
                            float o[32], g, f;
                            float2 ml = make_float2(mc, l);
                            if (cta == (int)blockIdx.x) {
                                read(k, o);
                            } else {
                                ml = __ldcg(a.part_ml + part_of(cta) * 128 + row);
                                const float4 *src = reinterpret_cast<const float4 *>(a.part_o) + ((int64_t)part_of(cta) * (HD / 4) + 8 * k) * 128 + row;
#pragma unroll
                                for (int y = 0; y < 8; ++y) {
                                    const float4 v = __ldcg(src + y * 128);
                                    o[4 * y] = v.x, o[4 * y + 1] = v.y, o[4 * y + 2] = v.z, o[4 * y + 3] = v.w;
                                }
                            }
                            onto(ml, M, S, g, f);
#pragma unroll
                            for (int y = 0; y < 32; ++y) acc[y] = fmaf(f, f > 0.0f ? o[y] : 0.0f, acc[y] * g);
                        }
                        if (r < rows) {
                            const float inv = S != 0.0f ? 1.0f / S : 0.0f;
#pragma unroll
                            for (int y = 0; y < 32; y += 8) put8(token * a.out_stride + head * HD + 32 * k + y, acc + y, inv);
                        }
                    }
                    read_done();
                    if (a.lse && r < rows) a.lse[token * a.n_heads + head] = S != 0.0f ? (M + log2f(S)) * ln2 : -INFINITY;
                    continue;
                }
            }
            {
                const int part = part_of(blockIdx.x);
                float4 *po = reinterpret_cast<float4 *>(a.part_o) + (int64_t)part * (HD / 4) * 128;
                if (!idle) {
#pragma unroll
                    for (int k = 0; k < HD / 32; ++k) {
                        float o[32];
                        read(k, o);
                        if (r < rows) {
#pragma unroll
                            for (int y = 0; y < 32; y += 4)
                                __stcg(po + (8 * k + y / 4) * 128 + r, make_float4(o[y], o[y + 1], o[y + 2], o[y + 3]));
                        }
                    }
                }
                read_done();
                if (r < rows) __stcg(a.part_ml + part * 128 + r, make_float2(mc, l));
            }
            // the last of the item's parts joins them all
            named_bar_sync(1 + i, 128);
            if (r == 0) {
                // (the fence covers the whole set's stores, which the barrier has shown this thread;
                // the count goes back to zero by itself)
                __threadfence();
                const bool last = atomicInc(counter, (unsigned)(c_last - c_first)) == (unsigned)(c_last - c_first);
                __threadfence();
                scratch[0].x = last ? 1.0f : 0.0f;
            }
            named_bar_sync(1 + i, 128);
            const bool last = scratch[0].x != 0.0f;
            named_bar_sync(1 + i, 128);  // (scratch is free again)
            if (!last) continue;
            // thread by thread eight columns of a row; many loads in flight: several such, or several parts
            auto join = [&](auto items_at_once, auto parts_at_once) {
                constexpr int U = decltype(items_at_once)::value, P = decltype(parts_at_once)::value;
                for (int k = r; k < pieces; k += 128 * U) {
                    float acc[U][8] = {}, M[U], S[U] = {};
                    int row[U], col[U];
#pragma unroll
                    for (int z = 0; z < U; ++z) {
                        const int x = min(k + 128 * z, pieces - 1);
                        col[z] = x / rows;
                        row[z] = x - col[z] * rows;
                        M[z] = -INFINITY;
                    }
                    for (int cta = c_first; cta <= c_last; cta += P) {
                        float2 p[P][U];
                        float4 v[P][U][2];
#pragma unroll
                        for (int y = 0; y < P; ++y)
#pragma unroll
                            for (int z = 0; z < U; ++z) {
                                const int pt = part_of(min(cta + y, c_last));
                                const float4 *src = reinterpret_cast<const float4 *>(a.part_o) + ((int64_t)pt * (HD / 4) + 2 * col[z]) * 128 + row[z];
                                p[y][z] = __ldcg(a.part_ml + pt * 128 + row[z]);
                                v[y][z][0] = __ldcg(src);
                                v[y][z][1] = __ldcg(src + 128);
                            }
#pragma unroll
                        for (int y = 0; y < P; ++y)
#pragma unroll
                            for (int z = 0; z < U; ++z) {
                                if (cta + y > c_last) continue;
                                float g, f;
                                onto(p[y][z], M[z], S[z], g, f);
                                const float e[8] = {v[y][z][0].x, v[y][z][0].y, v[y][z][0].z, v[y][z][0].w,
                                                    v[y][z][1].x, v[y][z][1].y, v[y][z][1].z, v[y][z][1].w};
#pragma unroll
                                for (int t = 0; t < 8; ++t) acc[z][t] = fmaf(f, f > 0.0f ? e[t] : 0.0f, acc[z][t] * g);
                            }
                    }
#pragma unroll
                    for (int z = 0; z < U; ++z) {
                        if (k + 128 * z >= pieces) continue;
                        const int64_t token = first_token + row[z] / a.g.group, head = first_head + row[z] % a.g.group;
                        put8(token * a.out_stride + head * HD + 8 * col[z], acc[z], S[z] != 0.0f ? 1.0f / S[z] : 0.0f);
                        if (a.lse && col[z] == 0) a.lse[token * a.n_heads + head] = S[z] != 0.0f ? (M[z] + log2f(S[z])) * ln2 : -INFINITY;
                    }
                }
            };
            if (pieces > 256) join(std::integral_constant<int, 4>(), std::integral_constant<int, 1>());
            else join(std::integral_constant<int, 1>(), std::integral_constant<int, 4>());
        }
        if (lent) named_bar_sync(4, 256);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int HD, bool BF16, bool OUT32>
__global__ void __launch_bounds__(kThreadsOf<false>, 1)
    attend_kernel(const KernelArgs a, const __grid_constant__ CUtensorMap q_map,
                  const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
    attend<HD, BF16, OUT32, false>(a, q_map, k_map, v_map);
}
template <int HD, bool OUT32>
__global__ void __launch_bounds__(kThreadsOf<true>, 1)
    attend8_kernel(const KernelArgs a, const __grid_constant__ CUtensorMap q_map,
                   const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
    attend<HD, false, OUT32, true>(a, q_map, k_map, v_map);
}

bool encode(CUtensorMap *map, CUtensorMapDataType type, int rank, const void *base, const cuuint64_t *dims,
            const cuuint64_t *strides, const cuuint32_t *box, CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
    const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
    EncodeTiled enc = encode_fn();
    return enc && enc(map, type, rank, const_cast<void *>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                      swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

using Kernel = void (*)(KernelArgs, CUtensorMap, CUtensorMap, CUtensorMap);
template <int HD, bool OUT32>
Kernel kernel_of(int type) {
    return type == QDQ_E4M3   ? attend8_kernel<HD, OUT32>
           : type == QDQ_BF16 ? attend_kernel<HD, true, OUT32>
                              : attend_kernel<HD, false, OUT32>;
}
Kernel kernel_of(int head_dim, int type, bool out_f32) {
    if (head_dim == 64) return out_f32 ? kernel_of<64, true>(type) : kernel_of<64, false>(type);
    return out_f32 ? kernel_of<128, true>(type) : kernel_of<128, false>(type);
}
uint32_t smem_of(int head_dim, int type) {
    if (type == QDQ_E4M3) return head_dim == 64 ? Shape<64, true>::kTotal : Shape<128, true>::kTotal;
    return head_dim == 64 ? Shape<64, false>::kTotal : Shape<128, false>::kTotal;
}
CUtensorMapDataType data_type(int type) { return type == QDQ_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16; }

}  // namespace

int attend_create(const AttendPools &p, int sm_count, AttendState **out) {
    *out = nullptr;
    AttendState *st = new (std::nothrow) AttendState();
    if (!st) return QDQ_ERR_CUDA;
    // the pools as [row / 8][64-wide block of a row][row % 8][64]: one box is a run of
    // positions of one kv head, in the order that the matrix instructions read
    const int run = p.page_size < 128 ? p.page_size : 128, blocks = p.n_kv_heads * p.head_dim / 64;
    const cuuint64_t row = (cuuint64_t)p.n_kv_heads * p.head_dim * 2;
    const cuuint64_t rows = (cuuint64_t)p.n_layers * p.n_pages * p.page_size;
    const cuuint64_t dims[4] = {64, 8, (cuuint64_t)blocks, rows / 8}, strides[3] = {row, 128, 8 * row};
    const cuuint32_t box[4] = {64, 8, (cuuint32_t)(p.head_dim / 64), (cuuint32_t)run / 8};
    bool ok;
    if (p.type == QDQ_E4M3) {
        // [page][head and position][head_dim]: a box is a run of positions of one kv head
        const cuuint64_t r = (cuuint64_t)p.n_kv_heads * p.page_size, d[3] = {(cuuint64_t)p.head_dim, r, (cuuint64_t)p.n_layers * p.n_pages};
        const cuuint64_t t[2] = {(cuuint64_t)p.head_dim, r * p.head_dim};
        const cuuint32_t x[3] = {(cuuint32_t)p.head_dim, (cuuint32_t)run, 1};
        ok = encode(&st->k_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, p.k_pages, d, t, x, CU_TENSOR_MAP_SWIZZLE_NONE) &&
             encode(&st->v_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, p.v_pages, d, t, x, CU_TENSOR_MAP_SWIZZLE_NONE);
    } else {
        ok = encode(&st->k_map, data_type(p.type), 4, p.k_pages, dims, strides, box) &&
             encode(&st->v_map, data_type(p.type), 4, p.v_pages, dims, strides, box);
    }
    st->ctas = sm_count;
    // two parts per CTA and set: 128 rows of O, a maximum and a sum; the joins' counters
    const size_t parts = (size_t)sm_count * 4, n_o = parts * 128 * p.head_dim * 4, n_s = parts * 128 * 8;
    const size_t bytes = n_o + n_s + (size_t)sm_count * 2 * sizeof(unsigned);
    ok = ok && cudaMalloc((void **)&st->mem, bytes) == cudaSuccess && cudaMemset(st->mem, 0, bytes) == cudaSuccess;
    for (bool out_f32 : {false, true}) {
        cudaFuncAttributes fa;  // (the kernel's shares of registers add up to its launch's)
        const Kernel f = kernel_of(p.head_dim, p.type, out_f32);
        ok = ok && cudaFuncGetAttributes(&fa, f) == cudaSuccess && fa.numRegs == (p.type == QDQ_E4M3 ? 128 : 168);
        ok = ok && cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_of(p.head_dim, p.type)) == cudaSuccess;
    }
    if (!ok) {
        cudaGetLastError();
        attend_destroy(st);
        return QDQ_ERR_CUDA;
    }
    st->part_o = (float *)st->mem;
    st->part_ml = (float2 *)(st->mem + n_o);
    st->counters = (unsigned *)(st->mem + n_o + n_s);
    *out = st;
    return QDQ_OK;
}

void attend_destroy(AttendState *st) {
    if (st == nullptr) return;
    if (st->mem) cudaFree(st->mem);
    delete st;
}

int launch_attend(const AttendState *st, const AttendArgs &a, cudaStream_t stream) {
    KernelArgs k = {};
    const AttendPools &p = *a.pools;
    k.n_seqs = a.n_seqs, k.n_tokens = a.n_tokens, k.max_pages = a.max_pages;
    k.q_start = a.q_start, k.kv_len = a.kv_len, k.page_table = a.page_table;
    k.out = a.out, k.lse = a.lse, k.out_stride = a.out_stride;
    // (masked scores are -inf and are multiplied by the scale: for a scale of 0 by the smallest number
    // instead, which leaves them -inf and moves the weight of any finite score by less than 2^-20 of it;
    // times a scale of 2^-40 .. 2^40, over e4m3 values, by 2^-100, which leaves 2^-140 at least)
    const float least = p.type == QDQ_E4M3 ? 0x1p-100f : std::numeric_limits<float>::denorm_min();
    k.scale_log2 = std::fmax((float)(std::fabs((double)a.scale) * 1.4426950408889634), least);
    k.n_pages = p.n_pages;
    while ((1 << k.page_shift) < p.page_size) ++k.page_shift;
    k.row8_layer = (int)((int64_t)a.layer * p.n_pages * p.page_size / 8);
    k.page0 = a.layer * p.n_pages;
    k.out_bf16 = a.out_type == QDQ_BF16;
    if (p.type == QDQ_E4M3) {
        const int64_t scales = (int64_t)a.layer * p.n_pages * p.n_kv_heads * (p.page_size / 16);
        k.k_scales = p.k_scales + scales, k.v_scales = p.v_scales + scales;
    }
    k.n_heads = p.n_heads;
    k.g.group = p.n_heads / p.n_kv_heads;
    k.g.tokens = kTileM / k.g.group;
    k.g.kv_heads = p.n_kv_heads;
    k.g.window = a.window < INT32_MAX - a.n_tokens ? a.window : INT32_MAX - a.n_tokens;
    k.g.table_end = a.max_pages * p.page_size;
    k.part_o = st->part_o, k.part_ml = st->part_ml, k.counters = st->counters;
    // fp32 accumulators, both operands of the pools' type, M = 128; S: N = 128, both K-major
    // (a negative scale negates Q); O: N = head_dim, V is N-major
    const uint32_t common = (1u << 4) | (p.type == QDQ_BF16 ? (1u << 7) | (1u << 10) : 0u) | ((uint32_t)(kTileM >> 4) << 24);
    k.idesc_qk = common | ((uint32_t)(kTileN >> 3) << 17) | (a.scale < 0.0f ? 1u << 13 : 0u);
    k.idesc_pv = common | ((uint32_t)(p.head_dim >> 3) << 17) | (1u << 16);
    // Q as [token][head][dim]: a box is 64 dims of the group's heads of a tile's tokens
    CUtensorMap q_map;
    const cuuint64_t dims[3] = {(cuuint64_t)p.head_dim, (cuuint64_t)p.n_heads, (cuuint64_t)a.n_tokens};
    const cuuint64_t q_row = a.n_tokens > 1 ? (cuuint64_t)a.q_stride * 2 : (cuuint64_t)p.n_heads * p.head_dim * 2;
    const cuuint64_t strides[2] = {(cuuint64_t)p.head_dim * 2, q_row};
    const cuuint32_t box[3] = {64, (cuuint32_t)k.g.group, (cuuint32_t)k.g.tokens};
    if (!encode(&q_map, data_type(p.type), 3, a.q, dims, strides, box)) return QDQ_ERR_CUDA;
    return launch_following(kernel_of(p.head_dim, p.type, a.out_type == QDQ_F32), st->ctas, p.type == QDQ_E4M3 ? kThreadsOf<true> : kThreadsOf<false>, smem_of(p.head_dim, p.type), 1, stream, k, q_map,
                            st->k_map, st->v_map);
}

int take_status_attend() {
    int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_attend_status, sizeof(int)) != cudaSuccess) {
        cudaGetLastError();
        return QDQ_ERR_CUDA;
    }
    if (v && cudaMemcpyToSymbol(g_attend_status, &zero, sizeof(int)) != cudaSuccess) {
        cudaGetLastError();
        return QDQ_ERR_CUDA;
    }
    return v;
}

}  // namespace qdq
