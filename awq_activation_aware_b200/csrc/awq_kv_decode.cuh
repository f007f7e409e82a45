// Attention over the paged 8-bit cache for few query rows per key head: single
// tokens and short drafts (sm_100a).  See awq_kv.cuh for the cache.
//
// A step reads every key and value once and does 4 * rows operations per byte, so
// HBM bounds it: rows <= 32 keep the tensor cores far from their rate, and what
// matters is that the codes stream without a pause and that the instructions to
// turn them into operands fit beside the stream (an SM takes in 27 bytes a clock).
//
//  * Work.  A unit is 64 keys (128 for D = 64) of one (sequence, key head, tile of 8, 16 or 32 rows); a
//    row is (new token, query head of the key head's group), so a group shares each
//    key.  The units of a launch, in order, are cut into equal contiguous ranges,
//    one per block of threads (two or three blocks an SM, by the registers), whatever the lengths: a ragged
//    batch and one long sequence fill the machine alike.  Lengths are read on the
//    device.  A segment (the units of one sequence, head and row tile) that crosses
//    a cut leaves partial results, summed in order by a second kernel: the result
//    does not depend on timing.
//  * Stream.  One warp feeds a ring of 16 KB stages by TMA, one box per page (one unit
//    at most), 128-byte rows swizzled (64-byte rows for D = 64), and the blocks' scales
//    by 4-byte asynchronous copies; it reads 32 page numbers at a time, a batch ahead.
//    Four warps consume, 32 keys (two blocks of scales) of a unit each, so for D = 128
//    two of them every other unit: what a unit costs beside its keys (waits, masks,
//    votes) is shared by more of them, and two chains of dependent instructions run
//    side by side (131072 keys of 8 heads: 288 instructions for 16 keys, 342 with one
//    block at a time).
//  * Products (mma m16n8k16, fp16 operands, binary32 sums), both with the codes as
//    the 16-row operand: S^T = K Q^T and O^T = V^T P^T, so 8 query rows cost half of
//    what 16 do and hold half the registers.  The codes are exact in fp16, and any
//    order of the contracted index will do: a lane takes 16 neighbouring codes of a
//    key in one 16-byte load and the fragments' k indices are whatever those are;
//    the query fragments are loaded to match.  For the second product a lane takes 16
//    codes of four keys; pairs of keys are interleaved by byte permutes, and the
//    probabilities change lanes by a transposing 8 x 8 move.  Both load patterns are
//    free of bank conflicts under the TMA swizzle.
//  * Scales.  The key scale multiplies the score.  The value scale 2^e enters the
//    exponent: P' = 2^(x + e - m + 9), so P' stays in fp16's range whatever the
//    scales, and the row sum adds 2^-e P'.  m, a running reference per row, is some
//    earlier largest x + e; it is raised only when a value exceeds it by 2^6
//    (P' <= 2^15 < 65504), which one vote finds out: no reductions across lanes and
//    no rescaling of the accumulators in the ordinary step.
//  * Masks.  Keys past the sequence may hold anything: their scores become -inf and
//    their codes zero.  A NaN value in a key that some rows of a partly masked block
//    do not see is taken out of the product and put into the sums of the rows that do
//    (all their elements become NaN; elsewhere only those that the product reaches).
//  * Measured (us on the device): 131072 keys of 8 heads, dim 128: 52 with 8 rows a
//    head, 56 with 16, 88 with 32 (floor 41); 524288 keys 173, 6.2 TB/s; 64 sequences
//    of 4096 keys 94, 5.75 TB/s; 516 keys 9.7.  About 12 us of a long call do not grow
//    with the keys: lengths, page numbers and keys come one after another, and the
//    join.  Dim 64 and 17 to 32 rows are bound by instructions, not by HBM.  With dim
//    128 the forms of 16 and 32 rows spill 104 bytes a thread at 168 registers,
//    that of 8 rows 16 to 20 at 128; those of dim 64 none.
#pragma once

#include <type_traits>

#include "awq_kv.cuh"

namespace awq {
namespace kv {
namespace dec {

constexpr int WARPS = 4;                   // consumer warps
constexpr int THREADS = 32 * (WARPS + 1);
constexpr float kLift = 9.0f, kSlack = 6.0f;       // see Scales above

// NT tiles of 8 query rows a warp, GR groups of warps with rows of their own.
template <int D, int NT, int GR> struct Shape {
    static constexpr int ROWS = 8 * NT * GR;
    static constexpr int BLOCKS = NT == 1 ? 3 : 2;         // resident per SM: 128 or 168 registers a thread
    static constexpr int TILE = GR == 2 ? 64 : 8192 / D;   // keys per unit and stage
    static constexpr int NB = TILE / kBlock;               // blocks of scales of a unit
    static constexpr int PARTS = NB / 2;                   // warps that share a unit's keys, 32 each
    static constexpr int TURNS = WARPS / GR / PARTS;       // 2: a warp takes every other unit
    static constexpr int SUMS = WARPS / GR;                // warps whose sums of a row are joined
    static constexpr int STAGE = 2 * TILE * D;             // keys, values
    static constexpr int STAGES = 4 * (16384 / STAGE);
    static_assert(TURNS >= 1 && STAGES % TURNS == 0, "a stage's phases must all be waited for by the same warps");
    static constexpr int PER = D / 8;                      // elements of a row that one lane holds
    static constexpr int LD = D + 36;                      // row of the merge area: 4 floats after every PER, 4 more
    static constexpr int OFF_SCALES = STAGES * STAGE;      // float [STAGES][2 * NB]
    static constexpr int OFF_BARS = OFF_SCALES + STAGES * 2 * NB * 4;
    static constexpr int OFF_ML = OFF_BARS + STAGES * 16;  // float [SUMS][ROWS][2]
    static constexpr int OFF_O = OFF_ML + SUMS * ROWS * 8;
    static constexpr bool Q_APART = NT > 1;                // query fragments in shared memory, a copy a warp: registers
    static constexpr int OFF_Q = (OFF_O + ROWS * LD * 4 + 15) / 16 * 16;   // uint2 [WARPS][NT][D / 16][32]
    static constexpr int Q_BYTES = Q_APART ? NT * (D / 16) * 32 * 8 : 0;
    static constexpr int BYTES = OFF_Q + WARPS * Q_BYTES + 1024;   // + alignment
};

struct Meta {                              // a segment whose units lie in the ranges of several blocks
    int32_t b, head, rt;
    int32_t first, last;                   // the blocks of its first and last unit; last -1: no such segment
};
struct Args {
    Cache C;
    Batch B;
    int64_t T;
    Rows q, out;
    float scale_log2;
    int64_t window;
    float *lse;
    int group;                             // query heads per key head
    int rows, tile;                        // query rows per tile (8, 16 or 32), keys per unit
    int box_rows;                          // keys per TMA box: min(page, tile)
    // Where the join finds a split segment: by its own number (b heads + head) rt_most + rt while those are
    // fewer than the blocks (by_segment), else by the block that starts it (at most one split segment each).
    Meta *meta;
    int by_segment, rt_most, max_tokens;
    float *part_ml;                        // [grid][2][rows][2]: slot 0 ends a segment begun earlier, slot 1 starts one
    float *part_o;                         // [grid][2][rows][D]
    uint64_t timeout_ns;
};

// The units of sequence b: heads * rt * nt.
struct Span {
    Seq s;
    int lo, hi;                            // keys that exist and that some row may see
    int t0, nt, rt;
};
constexpr int64_t kMaxLen = 1 << 30;       // positions fit 32 bits with room to spare
__device__ __forceinline__ Span span_of(const Args &A, int b) {
    Span p;
    p.s = seq_info(A.B, b, A.T, A.max_tokens);
    int64_t cap = A.B.max_pages * A.C.page;
    if (cap > kMaxLen) cap = kMaxLen;
    p.hi = (int)(p.s.len < cap ? p.s.len : cap);
    const int64_t lo = A.window ? p.s.start + 1 - A.window : 0;
    p.lo = lo < 0 ? 0 : (lo > p.hi ? p.hi : (int)lo);
    p.t0 = p.lo / A.tile;
    p.nt = (p.hi + A.tile - 1) / A.tile - p.t0;
    if (p.nt < 1) p.nt = 1;                // rows without keys still get their zeros
    p.rt = (int)(((int64_t)p.s.n * A.group + A.rows - 1) / A.rows);
    return p;
}
// What a segment's start and end (query fragments, joining the warps, its first keys' latency) cost beside its units,
// about 4500 clocks to their 1100: counted in, or blocks of threads that get many short sequences finish last.
constexpr int kStart = 4;
__device__ __forceinline__ int64_t units_of(const Args &A, int b) {
    const Span p = span_of(A, b);
    return (int64_t)A.C.heads * p.rt * (p.nt + kStart);
}

// Where a block's range starts, found by all threads: sums of units over the
// sequences, a chunk of blockDim.x at a time.
struct Range {
    int64_t first, end;                    // units of this block
    int b;                                 // sequence of `first`
    int64_t base;                          // units before sequence b
    int64_t total;
    int64_t blocks;                        // blocks that have units: every one of them at least one
};
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *warp_sums, int64_t &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int i = 1; i < 32; i <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, v, i);
        if (lane >= i) v += o;
    }
    __syncthreads();
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    int64_t before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < WARPS + 1; ++w) {
        if (w < warp) before += warp_sums[w];
        total += warp_sums[w];
    }
    return before + v;                     // inclusive
}
__device__ __forceinline__ Range find_range(const Args &A, int64_t *sums, int64_t *found) {
    Range r;
    const int n = A.B.n_seqs;
    int64_t total = 0, incl = 0, mine = 0;
    for (int b0 = 0; b0 < n; b0 += THREADS) {
        const int b = b0 + threadIdx.x;
        int64_t part;
        mine = b < n ? units_of(A, b) : 0;
        incl = block_scan(mine, sums, part);
        total += part;
    }
    r.total = total;
    r.blocks = total < gridDim.x ? total : gridDim.x;
    r.b = 0;
    r.base = r.first = r.end = 0;
    if ((int64_t)blockIdx.x >= r.blocks) return r;
    r.first = total * blockIdx.x / r.blocks;
    r.end = total * (blockIdx.x + 1) / r.blocks;
    int64_t base = 0;
    for (int b0 = 0; b0 < n; b0 += THREADS) {
        int64_t part = total;
        if (n > THREADS) {                 // otherwise the only chunk is still in registers
            const int b = b0 + threadIdx.x;
            mine = b < n ? units_of(A, b) : 0;
            incl = block_scan(mine, sums, part);
        }
        if (base + incl - mine <= r.first && r.first < base + incl) {
            found[0] = b0 + threadIdx.x;
            found[1] = base + incl - mine;
        }
        base += part;
        if (base > r.first) break;
    }
    __syncthreads();
    r.b = (int)found[0];
    r.base = found[1];
    return r;
}

// The block's place in its range.
struct Cursor {
    int b, head, rt;
    Span p;
    int64_t seg0;                          // number of the segment's first unit (kStart after the end of the one before)
    int64_t u;                             // the block's first unit of it
    // false: the range lies within the start of a segment, whose units are another block's
    __device__ __forceinline__ bool start(const Args &A, const Range &r) {
        b = r.b;
        p = span_of(A, b);
        const int64_t i = (r.first - r.base) / (p.nt + kStart);
        seg0 = r.base + i * (p.nt + kStart) + kStart;
        u = r.first > seg0 ? r.first : seg0;
        head = (int)(i / p.rt);
        rt = (int)(i % p.rt);
        return u < r.end;
    }
    __device__ __forceinline__ int64_t seg_end() const { return seg0 + p.nt; }
    // on to the next segment, if it has a unit below `end`
    __device__ __forceinline__ bool next(const Args &A, int64_t end) {
        if (seg_end() + kStart >= end) return false;
        seg0 += p.nt + kStart;
        u = seg0;
        if (++rt < p.rt) return true;
        rt = 0;
        if (++head < A.C.heads) return true;
        head = 0;
        do {
            p = span_of(A, ++b);
        } while (p.rt == 0);
        return true;
    }
};

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t cvt_lo(uint32_t w) {        // two codes to two fp16, exactly
    uint32_t d;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(d) : "r"(w));
    return d;
}
__device__ __forceinline__ uint32_t cvt_hi(uint32_t w) {
    uint32_t d;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(d) : "r"(w));
    return d;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {   // a in the low half
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
    return d;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
// The 8 x 8 matrix of 16-bit elements that a warp holds, row g in lanes 4 g .. 4 g + 3, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t w) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(w));
    return d;
}
// Bytes of a word that hold a NaN code (0x7f or 0xff): 0x80 in each, else 0.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

// What a part of a row, of reference m, weighs beside the reference `top` of them all.  A part without a reference saw no
// score but -inf or NaN: its sum is 0 or NaN.  Its sum is added like any other (0 * NaN is NaN), so a NaN stays.
__device__ __forceinline__ float part_weight(float m, float top) { return m > -INFINITY ? ex2(m - top) : 0.0f; }

// 0, or NaN where a query's elements (fp16 pairs) are not all finite: 0 * inf is NaN.  Every score of a row with an infinite
// element is infinite or NaN, so its softmax is NaN; the factor of its scores says so, or scores of -inf alone would pass
// for a row without keys.
__device__ __forceinline__ __half2 add_unless_finite(uint32_t w, __half2 z) {
    return __hfma2(*reinterpret_cast<const __half2 *>(&w), __float2half2_rn(0.0f), z);
}

__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * WARPS) : "memory"); }

// Query fragments (the 8-column operand) of row g of each tile: 16 neighbouring elements of
// chunk 2 c + i (D = 128) or c (D = 64) per i, as fp16.  bf16 rows are lifted by a power of two
// to fp16's upper range, exact for every element above 2^-28 of the row's largest; the return
// value takes it back (NaN for a row that is not finite).
template <typename TQ, int D>
__device__ __forceinline__ float load_query(const Args &A, const Cursor &cur, int row, uint32_t (&qf)[D / 16][2]) {
    const int lane = threadIdx.x & 31, c = lane & 3;
    constexpr int NI = D / 64;
    const int i = row / A.group, h = cur.head * A.group + row % A.group;
    uint32_t w[NI][8] = {};
    if (i < cur.p.s.n) {
        const TQ *q = static_cast<const TQ *>(A.q.data) + (int64_t)(cur.p.s.row0 + i) * A.q.ld_tok +
                      (int64_t)h * A.q.ld_head;
#pragma unroll
        for (int k = 0; k < NI; ++k) {
            const uint4 *p = reinterpret_cast<const uint4 *>(q + 16 * (NI * c + k));
            const uint4 v0 = p[0], v1 = p[1];
            w[k][0] = v0.x; w[k][1] = v0.y; w[k][2] = v0.z; w[k][3] = v0.w;
            w[k][4] = v1.x; w[k][5] = v1.y; w[k][6] = v1.z; w[k][7] = v1.w;
        }
    }
    float unscale = 1.0f;
    if (!std::is_same<TQ, __half>::value) {
        uint32_t top = 0;                                          // largest magnitude, as bf16 bits
#pragma unroll
        for (int k = 0; k < NI; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) top = max(top, max(w[k][j] & 0x7fffu, (w[k][j] >> 16) & 0x7fffu));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = min(max((int)(top >> 7) - 127, -100), 126);        // 2^e <= largest < 2^(e + 1)
        const float f = pow2(14 - e);
        unscale = top < 0x7f80u ? pow2(e - 14) : NAN;
#pragma unroll
        for (int k = 0; k < NI; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                w[k][j] = pack_f16(__uint_as_float(w[k][j] << 16) * f, __uint_as_float(w[k][j] & 0xffff0000u) * f);
    } else {
        __half2 z = __float2half2_rn(0.0f);
#pragma unroll
        for (int k = 0; k < NI; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) z = add_unless_finite(w[k][j], z);
        unscale += __low2float(z) + __high2float(z);
        unscale += __shfl_xor_sync(0xffffffffu, unscale, 1);               // of the four lanes that hold the row
        unscale += __shfl_xor_sync(0xffffffffu, unscale, 2);
        unscale *= 0.25f;
    }
#pragma unroll
    for (int k = 0; k < NI; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {                              // step (k, j): elements 4 j .. 4 j + 3 of the chunk
            qf[4 * k + j][0] = w[k][2 * j];
            qf[4 * k + j][1] = w[k][2 * j + 1];
        }
    return unscale;
}

// Byte offset of the 16-byte chunk of a swizzled row.
template <int D> __device__ __forceinline__ uint32_t chunk_at(uint32_t row, uint32_t chunk) {
    return D == 128 ? row * 128 + ((chunk ^ (row & 7)) << 4) : row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4);
}

template <typename TQ, int D, int NT, int GR>
__global__ void __launch_bounds__(THREADS, Shape<D, NT, GR>::BLOCKS)
kv_decode_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v, const Args A) {
    using S = Shape<D, NT, GR>;
    constexpr int ROWS = S::ROWS;
    extern __shared__ uint8_t raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    float *scales = reinterpret_cast<float *>(sm + S::OFF_SCALES);
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + S::OFF_BARS), *empty = full + S::STAGES;
    __shared__ int64_t sums[WARPS + 1], found[2];
    __shared__ int abort_flag;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

    if (threadIdx.x == 0) {
        abort_flag = 0;
        found[0] = found[1] = 0;
        for (int i = 0; i < S::STAGES; ++i) {
            mbar_init(full + i, 4 * S::NB);
            mbar_init(empty + i, WARPS / S::TURNS);
        }
        fence_mbar_init();
    }
    griddep_launch_dependents();
    griddep_wait();                        // everything above runs beside the end of the kernel before
    if (threadIdx.x == 0 && !A.by_segment) A.meta[blockIdx.x].last = -1;
    __syncthreads();
    const Range R = find_range(A, sums, found);
    if (R.first >= R.end) return;
    Cursor cur;
    if (!cur.start(A, R)) return;

    if (warp == WARPS) {
        // ---- the stream: 2 NB lanes for boxes of keys or values, 2 NB lanes for the blocks' scales
        const int which = (lane / S::NB) & 1, j = lane % S::NB;
        const bool boxes = lane < 2 * S::NB, mine = lane < 4 * S::NB;
        const int rows = boxes ? A.box_rows : kBlock;              // keys this lane looks after
        const bool active = mine && j * rows < S::TILE;
        const void *tmap = which ? &tmap_v : &tmap_k;
        const int page_bits = 31 - __clz(A.C.page);
        // page numbers: entries [32 k, 32 k + 32) of a sequence's row, one a lane.  A unit's never straddle two batches.
        auto fetch = [&](int b, int k) -> int32_t {
            const int64_t i = (int64_t)k * 32 + lane;
            return i < A.B.max_pages ? A.B.pages[(int64_t)b * A.B.ld_pages + i] : -1;
        };
        auto batch_of = [&](int64_t u) { return ((cur.p.t0 + (int)(u - cur.seg0)) * S::TILE >> page_bits) >> 5; };
        if (lane == 0 && cur.p.s.len > cur.p.hi) atomicOr(&g_dev_error, kDevErrBadIndex);
        int hold_b = cur.b, hold_k = batch_of(cur.u);
        int32_t hold = fetch(hold_b, hold_k), ahead = fetch(hold_b, hold_k + 1);
        int stage = 0;
        uint32_t phase = 1;                                        // the first round finds the stages empty
        int64_t issued = 0;
        bool ok = true, more = true;
        for (int64_t u = cur.u; more;) {
            const int pos = (cur.p.t0 + (int)(u - cur.seg0)) * S::TILE + j * rows, head = cur.head;
            int64_t page = __shfl_sync(0xffffffffu, hold, (pos >> page_bits) & 31);
            if (!active || pos >= cur.p.hi) page = -1;             // nothing there
            else if (page < 0 || page >= A.C.n_pages) page = -2;   // a bad page
            ++u;
            if (u >= cur.seg_end()) {
                more = cur.next(A, R.end);
                u = cur.u;
                if (more && lane == 0 && cur.p.s.len > cur.p.hi) atomicOr(&g_dev_error, kDevErrBadIndex);
            } else {
                more = u < R.end;
            }
            if (more) {                                            // the next unit's page numbers are on their way meanwhile
                const int k = batch_of(u);
                if (cur.b != hold_b || k != hold_k) {
                    hold = cur.b == hold_b && k == hold_k + 1 ? ahead : fetch(cur.b, k);
                    ahead = fetch(cur.b, k + 1);
                    hold_b = cur.b;
                    hold_k = k;
                }
            }
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(empty + stage, phase, &abort_flag, A.timeout_ns));
            if (!ok) break;
            const int64_t tile = (page * A.C.heads + head) * A.C.page + (pos & (A.C.page - 1));  // its first row
            if (boxes) {
                if (page >= 0) {
                    mbar_arrive_expect_tx(full + stage, rows * D);
                    tma_load_2d(sm + stage * S::STAGE + (which * S::TILE + j * rows) * D, tmap, 0, (int32_t)tile, full + stage);
                } else {
                    mbar_arrive(full + stage);
                }
            } else if (mine) {
                float *dst = scales + (stage * 2 + which) * S::NB + j;
                if (page >= 0) {
                    cp_async_4(dst, A.C.scales[which] + tile / kBlock);
                    cp_async_arrive_noinc(full + stage);
                } else {
                    *dst = -1.0f;                                  // no such block
                    if (page == -2) atomicOr(&g_dev_error, kDevErrBadIndex);
                    mbar_arrive(full + stage);
                }
            }
            __syncwarp();
            ++issued;
            if (++stage == S::STAGES) {
                stage = 0;
                phase ^= 1;
            }
        }
        if (!ok) {                                                 // given up: let the copies in flight land
            for (int k = 0; k < S::STAGES && k < issued; ++k) {
                const int64_t n = issued - 1 - k;
                uint64_t t0 = global_timer_ns();
                while (!mbar_try_wait_hint(full + n % S::STAGES, (uint32_t)((n / S::STAGES) & 1), 20000u))
                    if (global_timer_ns() - t0 > A.timeout_ns) break;
            }
        }
        return;
    }

    // ---- consumers: 32 keys of a unit each; TURNS = 2: warps 0, 1 every other unit, warps 2, 3 the ones between
    const int g = lane >> 2, c = lane & 3, part = warp % S::PARTS, group = GR == 1 ? 0 : warp / S::SUMS;
    const int own = 8 * NT * group, sums_at = warp % S::SUMS;      // this warp's first row of a tile; its place in the join
    constexpr int NJ = D / 16;                                     // 16-row tiles of the second product
    constexpr int KB = 2;                                          // blocks of 16 keys taken at once
    uint32_t qf[S::Q_APART ? 1 : NT][D / 16][2];
    const uint32_t q_at = smem_u32(sm + S::OFF_Q + warp * S::Q_BYTES) + 8 * lane;
    float rowf[NT][2], base[NT][2], l[NT][2], o[NT][NJ][4];        // base: m - kLift of rows 2 c, 2 c + 1 of a tile,
    uint32_t has = 0;                                              // once they saw a key (bit 2 t + x), else 0
    bool settled = false;                                          // every row of the warp has
    int pos_of[NT][2];                                             // their positions
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    int count = 0;                                                 // units of the segments before
    do {
        // ---- a segment, or this block's part of it
        const int n = cur.p.s.n, row0 = cur.rt * ROWS + own;
        int all_lo, all_hi;                                        // keys that every row of the tile sees
        {
            int last = (row0 + 8 * NT - 1) / A.group, first = row0 / A.group;
            if (last >= n) last = n - 1;
            if (first >= n) first = n - 1;
            const int64_t p0 = cur.p.s.start + first + 1, p1 = cur.p.s.start + last + 1 - A.window;
            all_hi = p0 < 0 ? 0 : (p0 < cur.p.hi ? (int)p0 : cur.p.hi);
            all_lo = A.window && p1 > 0 ? (p1 < kMaxLen ? (int)p1 : (int)kMaxLen) : 0;
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const float unscale = load_query<TQ, D>(A, cur, row0 + 8 * t + g, qf[S::Q_APART ? 0 : t]) * A.scale_log2;
            if (S::Q_APART) {                                      // read back by the lane that wrote it
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(q_at + (t * (D / 16) + k) * 256), "r"(qf[0][k][0]), "r"(qf[0][k][1]) : "memory");
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                rowf[t][x] = __shfl_sync(0xffffffffu, unscale, 4 * (2 * c + x));           // from the lane that loaded the row
                base[t][x] = 0.0f;
                l[t][x] = 0.0f;
                int i = (row0 + 8 * t + 2 * c + x) / A.group;
                if (i >= n) i = n - 1;                             // rows of nobody follow the last token
                const int64_t at = cur.p.s.start + i;
                pos_of[t][x] = at < kMaxLen ? (at < -1 ? -1 : (int)at) : (int)kMaxLen;
            }
#pragma unroll
            for (int j = 0; j < NJ; ++j) o[t][j][0] = o[t][j][1] = o[t][j][2] = o[t][j][3] = 0.0f;
        }
        has = 0;
        settled = false;
        const int units = (int)((cur.seg_end() < R.end ? cur.seg_end() : R.end) - cur.u);
        int key0 = (cur.p.t0 + (int)(cur.u - cur.seg0)) * S::TILE + 32 * part;
        int turn = count & 1;
        for (int left = units; left > 0; --left, key0 += S::TILE, turn ^= 1) {
            if (S::TURNS == 1 || turn == warp / S::PARTS) {
                // a wait that ran out skips the keys but not the barriers below
                ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(full + stage, phase, &abort_flag, A.timeout_ns));
                float ks[KB], vs[KB];
#pragma unroll
                for (int b = 0; b < KB; ++b) {
                    ks[b] = scales[stage * 2 * S::NB + 2 * part + b];
                    vs[b] = scales[stage * 2 * S::NB + S::NB + 2 * part + b];
                }
                const uint32_t kt = smem_u32(sm + stage * S::STAGE) + 32 * part * D, vt = kt + S::TILE * D;
                const bool whole = key0 >= all_lo && key0 + 16 * KB <= all_hi && fminf(ks[0], ks[KB - 1]) >= 0.0f;
                if (ok && (whole || key0 < cur.p.hi)) {
                    float s[KB][NT][4];                            // keys g (0, 1), g + 8 (2, 3) of rows 2 c, 2 c + 1
#pragma unroll
                    for (int b = 0; b < KB; ++b)
#pragma unroll
                        for (int t = 0; t < NT; ++t) s[b][t][0] = s[b][t][1] = s[b][t][2] = s[b][t][3] = 0.0f;
#pragma unroll
                    for (int i = 0; i < D / 64; ++i)
#pragma unroll
                        for (int b = 0; b < KB; ++b) {
                            const uint4 k0 = lds128(kt + chunk_at<D>(16 * b + g, (D / 64) * c + i));
                            const uint4 k1 = lds128(kt + chunk_at<D>(16 * b + 8 + g, (D / 64) * c + i));
                            const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const uint32_t a[4] = {cvt_lo(w0[j]), cvt_lo(w1[j]), cvt_hi(w0[j]), cvt_hi(w1[j])};
#pragma unroll
                                for (int t = 0; t < NT; ++t) {
                                    if (S::Q_APART) {
                                        const uint2 q = lds64(q_at + (t * (D / 16) + 4 * i + j) * 256);
                                        mma_16816(s[b][t], a, q.x, q.y);
                                    } else {
                                        mma_16816(s[b][t], a, qf[t][4 * i + j][0], qf[t][4 * i + j][1]);
                                    }
                                }
                            }
                        }
                    // z = x + e - base, hidden keys -inf; 2^e = the value scale, inv_v = 2^-e
                    float top = -INFINITY, inv_v[KB];
#pragma unroll
                    for (int b = 0; b < KB; ++b) {
                        const uint32_t bits = __float_as_uint(vs[b]);
                        const float ev = __fsub_rn(__uint_as_float(0x4b400000u + (bits >> 23)), kMagic + 127.0f);
                        inv_v[b] = __uint_as_float(0x7f000000u - bits);
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            const float f0 = rowf[t][0] * ks[b], f1 = rowf[t][1] * ks[b];
                            const float c0 = ev - base[t][0], c1 = ev - base[t][1];
                            s[b][t][0] = __fmaf_rn(s[b][t][0], f0, c0);
                            s[b][t][1] = __fmaf_rn(s[b][t][1], f1, c1);
                            s[b][t][2] = __fmaf_rn(s[b][t][2], f0, c0);
                            s[b][t][3] = __fmaf_rn(s[b][t][3], f1, c1);
                            if (!whole) {
                                const bool none = ks[b] < 0.0f;        // a block that is not there
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    const int key = key0 + 16 * b + g + 8 * (k >> 1), at = pos_of[t][k & 1];
                                    if (none || key > at || key >= cur.p.hi || (A.window && key <= at - A.window))
                                        s[b][t][k] = -INFINITY;
                                }
                            }
                            top = fmax3(fmax3(top, s[b][t][0], s[b][t][1]), s[b][t][2], s[b][t][3]);
                        }
                    }
                    if (!settled || __any_sync(0xffffffffu, top > kLift + kSlack)) {       // seldom: raise the references
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                float mx = fmaxf(fmaxf(s[0][t][x], s[0][t][2 + x]), fmaxf(s[KB - 1][t][x], s[KB - 1][t][2 + x]));
                                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                                const uint32_t bit = 1u << (2 * t + x);
                                float up = 0.0f, f = 1.0f;
                                if (has & bit) {
                                    up = fmaxf(mx - kLift, 0.0f);
                                    f = ex2(-up);
                                } else if (mx > -INFINITY) {
                                    up = mx - kLift;               // the row's first keys: its sums are still 0
                                    has |= bit;
                                }
                                base[t][x] += up;
                                l[t][x] *= f;
#pragma unroll
                                for (int j = 0; j < NJ; ++j) {
                                    o[t][j][x] *= f;
                                    o[t][j][2 + x] *= f;
                                }
#pragma unroll
                                for (int b = 0; b < KB; ++b) {
                                    s[b][t][x] -= up;
                                    s[b][t][2 + x] -= up;
                                }
                            }
                        settled = __all_sync(0xffffffffu, has == (1u << (2 * NT)) - 1);
                    }
                    uint32_t pb[KB][NT][2];
#pragma unroll
                    for (int b = 0; b < KB; ++b)
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) s[b][t][k] = ex2(s[b][t][k]);
                            l[t][0] = __fmaf_rn(s[b][t][0] + s[b][t][2], inv_v[b], l[t][0]);
                            l[t][1] = __fmaf_rn(s[b][t][1] + s[b][t][3], inv_v[b], l[t][1]);
                            pb[b][t][0] = transpose8x8(pack_f16(s[b][t][0], s[b][t][1]));  // keys 2 c, 2 c + 1 of row g
                            pb[b][t][1] = transpose8x8(pack_f16(s[b][t][2], s[b][t][3]));  // keys 2 c + 8, 2 c + 9
                        }
#pragma unroll
                    for (int b = 0; b < KB; ++b) {
                        // values of keys 2 c, 2 c + 1, 2 c + 8, 2 c + 9: D / 8 codes of each
                        uint32_t v[4][D / 32];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t row = 16 * b + 2 * c + (k & 1) + 8 * (k >> 1);
                            if constexpr (D == 128) {
                                const uint4 x = lds128(vt + chunk_at<D>(row, g));
                                v[k][0] = x.x; v[k][1] = x.y; v[k][2] = x.z; v[k][3] = x.w;
                            } else {
                                const uint2 x = lds64(vt + chunk_at<D>(row, g >> 1) + (g & 1) * 8);
                                v[k][0] = x.x; v[k][1] = x.y;
                            }
                        }
                        if (!whole) {
                            // keys that do not exist: zeros.  NaN codes: zeros here, NaN in the sums of the rows that see them.
                            const int exist = ks[b] < 0.0f ? 0 : cur.p.hi - (key0 + 16 * b);
                            uint32_t bad = 0;                      // bit i: key i of the 16
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const int key = 2 * c + (k & 1) + 8 * (k >> 1);
#pragma unroll
                                for (int w = 0; w < D / 32; ++w) {
                                    if (key >= exist) v[k][w] = 0;
                                    const uint32_t nan = nan_bytes(v[k][w]);
                                    if (nan) {
                                        bad |= 1u << key;
                                        v[k][w] &= ~((nan >> 7) * 0xffu);
                                    }
                                }
                            }
                            bad = __reduce_or_sync(0xffffffffu, bad);
#pragma unroll
                            for (int t = 0; t < NT; ++t)
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    const int i = g + 8 * (k >> 1), key = key0 + 16 * b + i, at = pos_of[t][k & 1];
                                    if (((bad >> i) & 1) && key <= at && (!A.window || key > at - A.window)) l[t][k & 1] = NAN;
                                }
                        }
#pragma unroll
                        for (int w = 0; w < D / 32; ++w) {
                            const uint32_t x0 = __byte_perm(v[0][w], v[1][w], 0x5140), x1 = __byte_perm(v[0][w], v[1][w], 0x7362);
                            const uint32_t y0 = __byte_perm(v[2][w], v[3][w], 0x5140), y1 = __byte_perm(v[2][w], v[3][w], 0x7362);
                            const uint32_t a0[4] = {cvt_lo(x0), cvt_hi(x0), cvt_lo(y0), cvt_hi(y0)};   // elements 4 w, 4 w + 1
                            const uint32_t a1[4] = {cvt_lo(x1), cvt_hi(x1), cvt_lo(y1), cvt_hi(y1)};   // elements 4 w + 2, 4 w + 3
#pragma unroll
                            for (int t = 0; t < NT; ++t) {
                                mma_16816(o[t][2 * w], a0, pb[b][t][0], pb[b][t][1]);
                                mma_16816(o[t][2 * w + 1], a1, pb[b][t][0], pb[b][t][1]);
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(empty + stage);
            }
            if (++stage == S::STAGES) {
                stage = 0;
                phase ^= 1;
            }
        }
        count += units;
        // ---- join the warps: each brings its sums to the common reference and adds them in turn
        float *ml = reinterpret_cast<float *>(sm + S::OFF_ML), *oa = reinterpret_cast<float *>(sm + S::OFF_O);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float sum = l[t][x];
                sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                if (g == 0) {
                    float *p = ml + (sums_at * ROWS + own + 8 * t + 2 * c + x) * 2;
                    p[0] = (has >> (2 * t + x)) & 1 ? base[t][x] : -INFINITY;
                    p[1] = sum;
                }
            }
        consumers_sync();
        auto common = [&](int r) {
            float m = ml[2 * r];
#pragma unroll
            for (int w = 1; w < S::SUMS; ++w) m = fmaxf(m, ml[2 * (w * ROWS + r)]);
            return m;
        };
        for (int w = 0; w < S::SUMS; ++w) {
            if (w == sums_at) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int r = own + 8 * t + 2 * c + x;
                        const float f = (has >> (2 * t + x)) & 1 ? ex2(base[t][x] - common(r)) : 0.0f;
                        float *row = oa + r * S::LD + g * (S::PER + 4);
#pragma unroll
                        for (int j = 0; j < NJ; j += 2) {
                            float4 *p = reinterpret_cast<float4 *>(row + 2 * j);
                            float4 v = w ? *p : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                            v.x = __fmaf_rn(f, o[t][j][x], v.x);
                            v.y = __fmaf_rn(f, o[t][j][2 + x], v.y);
                            v.z = __fmaf_rn(f, o[t][j + 1][x], v.z);
                            v.w = __fmaf_rn(f, o[t][j + 1][2 + x], v.w);
                            *p = v;
                        }
                    }
            }
            consumers_sync();
        }
        const bool begins = cur.seg0 >= R.first, ends = cur.seg_end() <= R.end;
        const int tid = threadIdx.x;
        for (int i = tid; i < ROWS * D / 8; i += 32 * WARPS) {
            const int r = i / (D / 8), d = (i % (D / 8)) * 8;
            const int row = cur.rt * ROWS + r, tok = row / A.group, hq = cur.head * A.group + row % A.group;
            if (tok >= cur.p.s.n) continue;
            const float mx = common(r);
            float L = 0.0f;
#pragma unroll
            for (int w = 0; w < S::SUMS; ++w) {
                L = __fmaf_rn(part_weight(ml[(w * ROWS + r) * 2], mx), ml[(w * ROWS + r) * 2 + 1], L);
            }
            const float4 *p = reinterpret_cast<const float4 *>(oa + r * S::LD + d + 4 * (d / S::PER));
            const float4 a = p[0], b = p[1];
            float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
            if (begins && ends) {
                const float inv = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] *= inv;
                store_n(static_cast<TQ *>(const_cast<void *>(A.out.data)) + (int64_t)(cur.p.s.row0 + tok) * A.out.ld_tok +
                            (int64_t)hq * A.out.ld_head + d, v);
                if (A.lse && d == 0)
                    A.lse[(int64_t)(cur.p.s.row0 + tok) * A.q.heads + hq] =
                        L == 0.0f ? -INFINITY : (mx + log2f(L)) * 0.6931471805599453f;
            } else {
                const int64_t slot = ((int64_t)blockIdx.x * 2 + (begins ? 1 : 0)) * ROWS + r;
                store_n(A.part_o + slot * D + d, v);
                if (d == 0) {
                    A.part_ml[slot * 2] = mx;
                    A.part_ml[slot * 2 + 1] = L;
                }
            }
        }
        if (begins && tid == 0 && (A.by_segment || !ends)) {
            // the block of the segment's last unit x: the last i with total i / blocks <= x
            const int64_t last = ends ? -1 : (cur.seg_end() * R.blocks - 1) / R.total;
            A.meta[A.by_segment ? (cur.b * A.C.heads + cur.head) * A.rt_most + cur.rt : (int)blockIdx.x] =
                {cur.b, cur.head, cur.rt, (int32_t)blockIdx.x, (int32_t)last};
        }
        consumers_sync();
    } while (cur.next(A, R.end));
}

// The parts of a split segment's row, summed in order.  WPR warps a row: eight where there are few segments, each of
// many parts (by_segment), one where there are many, of two or three parts as a rule; a warp's loads are all on their
// way together.
constexpr int JOIN_WARPS = 8;
template <typename TQ, int D, int WPR>
__global__ void __launch_bounds__(32 * JOIN_WARPS) kv_decode_join_kernel(const Args A) {
    constexpr int N = D / 32, DEEP = 8;
    __shared__ float sm[JOIN_WARPS], sl[JOIN_WARPS], so[WPR == 1 ? 1 : WPR][D];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = WPR == 1 ? blockIdx.y * JOIN_WARPS + warp : blockIdx.y, part = WPR == 1 ? 0 : warp;
    Meta M;
    Seq s;
    if (A.by_segment) {
        const int rt = blockIdx.x % A.rt_most, bh = blockIdx.x / A.rt_most;
        s = seq_info(A.B, bh / A.C.heads, A.T, A.max_tokens);      // beside the load of M
        M = A.meta[blockIdx.x];
        if ((int64_t)rt * A.rows >= (int64_t)s.n * A.group) return;      // there is no such segment
        if (M.last < 0) return;
    } else {
        M = A.meta[blockIdx.x];
        if (M.last < 0) return;
        s = seq_info(A.B, M.b, A.T, A.max_tokens);
    }
    const int row = M.rt * A.rows + r, tok = row / A.group, hq = M.head * A.group + row % A.group;
    if (r >= A.rows || tok >= s.n) return;
    auto slot_of = [&](int i) { return ((int64_t)i * 2 + (i == M.first ? 1 : 0)) * A.rows + r; };
    float mx = -INFINITY, L = 0.0f, v[N] = {};                     // mx: reference of L and v
    for (int i0 = M.first + part; i0 <= M.last; i0 += WPR * DEEP) {
        float2 p[DEEP];
        float x[DEEP][N];
#pragma unroll
        for (int k = 0; k < DEEP; ++k) {
            const int i = i0 + k * WPR;
            p[k] = make_float2(-INFINITY, 0.0f);
            if (i <= M.last) {
                p[k] = *reinterpret_cast<const float2 *>(A.part_ml + slot_of(i) * 2);
                load_n(A.part_o + slot_of(i) * D + lane * N, x[k]);
            }
        }
        float top = mx;
#pragma unroll
        for (int k = 0; k < DEEP; ++k) top = fmaxf(top, p[k].x);
        const float f0 = part_weight(mx, top);
        L *= f0;
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] *= f0;
#pragma unroll
        for (int k = 0; k < DEEP; ++k) {
            const float f = part_weight(p[k].x, top);
            L = __fmaf_rn(f, p[k].y, L);
            if (p[k].x > -INFINITY) {
#pragma unroll
                for (int n = 0; n < N; ++n) v[n] = __fmaf_rn(f, x[k][n], v[n]);
            }
        }
        mx = top;
    }
    if (WPR > 1) {
        if (lane == 0) {
            sm[warp] = mx;
            sl[warp] = L;
        }
#pragma unroll
        for (int n = 0; n < N; ++n) so[part][lane * N + n] = v[n];
        __syncthreads();
        if (warp) return;
        mx = sm[0];
#pragma unroll
        for (int w = 1; w < WPR; ++w) mx = fmaxf(mx, sm[w]);
        L = 0.0f;
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] = 0.0f;
#pragma unroll
        for (int w = 0; w < WPR; ++w) {
            const float f = part_weight(sm[w], mx);
            L = __fmaf_rn(f, sl[w], L);
#pragma unroll
            for (int n = 0; n < N; ++n) v[n] = __fmaf_rn(f, so[w][lane * N + n], v[n]);
        }
    }
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] *= inv;
    store_n(static_cast<TQ *>(const_cast<void *>(A.out.data)) + (int64_t)(s.row0 + tok) * A.out.ld_tok +
                (int64_t)hq * A.out.ld_head + lane * N, v);
    if (A.lse && lane == 0)
        A.lse[(int64_t)(s.row0 + tok) * A.q.heads + hq] = L == 0.0f ? -INFINITY : (mx + log2f(L)) * 0.6931471805599453f;
}

}  // namespace dec
}  // namespace kv
}  // namespace awq
